// Latent attention over a paged cache: how the work is divided (see paged.h; a unit is one tile of (token, head) pairs and one
// sequence's keys), and each CTA's walk over its share.
#pragma once

#include "paged.cuh"

namespace sdpa {

constexpr int kLatentMinPiece = 1;  // blocks; see paged.h
constexpr int kLatentMinWork = 1;

struct LatentPiece {
  int b, tok0, jb0;
  int n_blocks;             // 0: no more pieces
  int slot;                 // partial slot, or -1: the whole unit, which stores O itself
  int q_off, n, len, sk;
  int pad[7];
};
static_assert(sizeof(LatentPiece) == 64, "the producer announces a piece in 64 bytes");

// The plan, made by each CTA for itself where the sequences are few and have few tiles: the line lies sequence by
// sequence and tile by tile, and a cut is {sequence, tile, block, 0}.  Spares the planning kernel (drafts of 16 sequences,
// 128 heads: 108 -> 104 us).  scratch: 8 KB of shared memory that nobody uses yet.  All threads; returns this team's cuts in `mine`.
constexpr int kInlineTiles = 8;  // of a sequence

__host__ __device__ __forceinline__ int latent_unit(const PagedParams& p, int n, int len, int tile) {
  return paged_tile_blocks(n, len, min(max(len, 0), p.max_kv), p.tok_tile, p.causal, tile) + kUnitCost;
}

// Cut c of n_ctas; sequence b lies from pos[b] to pos[b + 1].
__host__ __device__ __forceinline__ int4 latent_cut(const PagedParams& p, const long long* pos, int c, int n_ctas) {
  if (c >= n_ctas) return make_int4(p.B, 0, 0, 0);
  const long long total = pos[p.B];
  const long long x = total >> 31 ? total / n_ctas * c + total % n_ctas * c / n_ctas
                                  : static_cast<uint32_t>(total) / n_ctas * static_cast<long long>(c) +
                                        static_cast<uint32_t>(total) % n_ctas * c / n_ctas;
  int lo = 0, hi = p.B;  // the last sequence that starts at or before x (it has tokens)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pos[mid] <= x) lo = mid; else hi = mid;
  }
  const int n = plan_ld(p.cu_q + lo + 1) - plan_ld(p.cu_q + lo), len = plan_ld(p.kv_len + lo);
  long long r = x - pos[lo];
  int tile = 0, unit = latent_unit(p, n, len, 0);
  while (r >= unit) {
    r -= unit;
    unit = latent_unit(p, n, len, ++tile);
  }
  const int blocks = unit - kUnitCost;
  int off = static_cast<int>(r) - kUnitCost;
  if (p.cut ? off < p.min_piece : 2 * off < blocks) {
    off = 0;
  } else if (!p.cut || blocks - off < p.min_piece) {
    off = 0;
    if (++tile * p.tok_tile >= n) tile = 0, ++lo;
  }
  // no cut names a sequence without tokens
  while (lo < p.B && pos[lo + 1] == pos[lo]) ++lo;
  return make_int4(lo, tile, off, 0);
}

template <int THREADS>
__device__ __forceinline__ void latent_inline_plan(const PagedParams& p, uint8_t* scratch, int4* mine, int team, bool store) {
  static_assert(THREADS >= kInlinePlanSeqs && THREADS > kPagedMaxCtas, "one thread per sequence and per cut");
  long long* pos = reinterpret_cast<long long*>(scratch);               // [kInlinePlanSeqs + 1]
  long long* warp_sum = pos + kInlinePlanSeqs + 1;                       // [THREADS / 32]
  int4* cuts = reinterpret_cast<int4*>(scratch + 4096);                  // [kPagedMaxCtas + 1]
  int* n_groups = reinterpret_cast<int*>(cuts + kPagedMaxCtas + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int bad = 0;
  long long v = 0;
  if (tid < p.B) {
    const int q0 = __ldg(p.cu_q + tid), q1 = __ldg(p.cu_q + tid + 1), len = __ldg(p.kv_len + tid);
    bad = paged_bad(p, tid, q0, q1);
    if (!bad)
      for (int i = 0; i * p.tok_tile < q1 - q0; ++i) v += latent_unit(p, q1 - q0, len, i);
  }
  long long incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (tid == 0) *n_groups = 0, pos[0] = 0;
  bad = __syncthreads_or(bad);
  for (int w = 0; w < warp; ++w) incl += warp_sum[w];
  if (tid < p.B) pos[tid + 1] = incl;
  __syncthreads();
  const int n_ctas = bad ? 0 : static_cast<int>(min(static_cast<long long>(p.sms), pos[p.B] / p.min_work));
  if (team < n_ctas) {
    if (tid == 0) mine[0] = latent_cut(p, pos, team, n_ctas);
    if (tid == 32) mine[1] = latent_cut(p, pos, team + 1, n_ctas);
  } else if (tid == 0) {
    mine[0] = mine[1] = make_int4(0, 0, 0, 0);
  }
  if (store) {  // for the merge
    if (tid <= n_ctas) p.plan.cuts[tid] = cuts[tid] = bad ? make_int4(0, 0, 0, 0) : latent_cut(p, pos, tid, n_ctas);
    __syncthreads();
    if (tid < n_ctas && cuts[tid].z != 0) {
      const int b = cuts[tid].x, q0 = __ldg(p.cu_q + b);
      PagedGroup g;
      if (paged_group(cuts, tid, n_ctas, make_int2(b, cuts[tid].y), q0, __ldg(p.cu_q + b + 1) - q0, __ldg(p.kv_len + b), g))
        p.plan.groups[atomicAdd(n_groups, 1)] = g;
    }
    __syncthreads();
    if (tid == 0) {
      p.plan.head->n_ctas = n_ctas;
      p.plan.head->n_groups = *n_groups;
      if (bad) atomicOr(p.status, kStatusBadSeqlens);
    }
  }
  fence_proxy_async_smem();  // TMA writes the scratch next
  __syncthreads();
}

// The pieces of a CTA's stretch, in order.  A place is {sequence, tile, block} with the plan above, {tile, 0, block} with the
// planning kernel's.
struct LatentWalk {
  int team, at, sub, off, first;
  int4 end;

  __host__ __device__ __forceinline__ LatentWalk(int team, int4 from, int4 to)
      : team(team), at(from.x), sub(from.y), off(from.z), first(1), end(to) {}
  __host__ __device__ __forceinline__ LatentPiece next(const PagedParams& p) {
    LatentPiece w{};
    if (p.inline_plan)
      while (at < end.x && plan_ld(p.cu_q + at) == plan_ld(p.cu_q + at + 1)) ++at;
    if (!(at < end.x || (at == end.x && (sub < end.y || (sub == end.y && off < end.z))))) return w;
    const int2 tile = p.inline_plan ? make_int2(at, sub) : walk_ld(p.plan.tiles + at);
    w.b = tile.x;
    w.q_off = plan_ld(p.cu_q + w.b);
    w.n = plan_ld(p.cu_q + w.b + 1) - w.q_off;
    w.len = paged_len(p, w.b);
    w.sk = min(max(w.len, 0), p.max_kv);
    w.tok0 = tile.y * p.tok_tile;
    w.jb0 = off;
    const int all = paged_tile_blocks(w.n, w.len, w.sk, p.tok_tile, p.causal, tile.y);
    const int stop = at == end.x && sub == end.y ? end.z : all;
    w.n_blocks = stop - off;
    w.slot = (off > 0 || stop < all) ? 2 * team + 1 - first : -1;
    first = 0;
    off = 0;
    if (!p.inline_plan || ++sub * p.tok_tile >= w.n) sub = 0, ++at;
    return w;
  }
};

}  // namespace sdpa
