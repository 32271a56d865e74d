// Chunk attention over a paged cache: the work plan, the merge of partial results, and the C entry
// points (see paged.cuh for the kernel).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "sdpa.h"
#include "paged.h"
#include "ptx.cuh"

namespace sdpa {

namespace {

constexpr int kPlanThreads = 1024;

// Inclusive sum of v over the block's threads so far (before: the sum of earlier calls); total: the
// sum of all of them.  Two barriers.
__device__ __forceinline__ long long block_scan(long long v, long long before, long long (&warp_sum)[33], long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += y;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  long long s = warp_sum[lane];  // every warp scans the 32 sums itself
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  total = before + __shfl_sync(0xffffffffu, s, 31);
  const long long prev = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return before + v + (warp > 0 ? prev : 0);
}

__device__ __forceinline__ int unit_blocks(const PagedParams& p, int n, int len, int i) {
  const int sk = min(max(len, 0), p.max_kv);
  return max(paged_tile_blocks(n, len, sk, p.tok_tile, p.causal, i * kTilesPerCta),
             paged_tile_blocks(n, len, sk, p.tok_tile, p.causal, i * kTilesPerCta + 1));
}

// One block lays out the tiles, measures the line and places the cuts.  Offsets that are not sorted
// within [0, total_q], or a sequence of more than max_seqlen_q tokens, raise a status and leave no
// work, so nothing is stored.  Up to kSmall sequences and tiles are kept in shared memory as well.
constexpr int kSmall = 1024;

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PagedParams p) {
  __shared__ long long warp_sum[33];
  __shared__ int4 s_cuts[kPagedMaxCtas + 1];
  __shared__ int s_groups;
  __shared__ int s_seq[kSmall];
  __shared__ int2 s_tile[kSmall];
  __shared__ long long s_pos[kSmall];
  const int tid = threadIdx.x;
  pdl_launch_dependents();  // the attention kernel may set itself up meanwhile
  if (tid == 0) s_groups = 0;
  const int tok_unit = kTilesPerCta * p.tok_tile;
  int bad = 0;
  long long n_tiles = 0;
  for (int base = 0; base < p.B; base += kPlanThreads) {
    const int b = base + tid;
    int v = 0;
    if (b < p.B) {
      const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
      if (q0 < 0 || q1 < q0 || q1 > p.total_q || static_cast<long long>(q1) - q0 > p.max_seqlen_q)
        bad = 1;
      else
        v = (q1 - q0 + tok_unit - 1) / tok_unit;
    }
    const long long before = n_tiles;
    const long long incl = block_scan(v, before, warp_sum, n_tiles);
    if (b < p.B) {
      const int at = static_cast<int>(min(incl - v, static_cast<long long>(p.max_tiles)));
      if (p.B <= kSmall)
        s_seq[b] = at;
      else
        p.plan.seq_tiles[b] = at;
    }
  }
  if (__syncthreads_or(bad) || n_tiles > p.max_tiles) {
    if (tid == 0) {
      p.plan.head->n_ctas = p.plan.head->n_groups = 0;
      atomicOr(p.status, kStatusBadSeqlens);
    }
    return;
  }
  const int* seq = p.B <= kSmall ? s_seq : p.plan.seq_tiles;
  const bool small = n_tiles <= kSmall;
  long long total = 0;
  for (int base = 0; base < n_tiles; base += kPlanThreads) {
    const int tile = base + tid;
    long long v = 0;
    if (tile < n_tiles) {
      int lo = 0, hi = p.B;  // the last sequence that starts at or before the tile
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq[mid] <= tile) lo = mid; else hi = mid;
      }
      const int2 at = make_int2(lo, tile - seq[lo]);
      p.plan.tiles[tile] = at;
      if (small) s_tile[tile] = at;
      const int n = __ldg(p.cu_q + lo + 1) - __ldg(p.cu_q + lo);
      v = static_cast<long long>(unit_blocks(p, n, __ldg(p.kv_len + lo), at.y) + kUnitCost) * p.Hkv;
    }
    const long long before = total;
    const long long incl = block_scan(v, before, warp_sum, total);
    if (tile < n_tiles) {
      if (small)
        s_pos[tile] = incl - v;
      else
        p.plan.tile_pos[tile] = incl - v;
    }
  }
  __syncthreads();
  const long long* pos = small ? s_pos : p.plan.tile_pos;
  const int2* tiles = small ? s_tile : p.plan.tiles;
  // as many CTAs as have kMinWork each, and at least one for every unit
  const int n_ctas = static_cast<int>(min(static_cast<long long>(p.sms), max(n_tiles * p.Hkv, total / kMinWork)));
  for (int c = tid; c <= n_ctas; c += kPlanThreads) {
    int4 cut = make_int4(static_cast<int>(n_tiles), 0, 0, 0);
    if (c < n_ctas) {
      const long long x = total / n_ctas * c + total % n_ctas * c / n_ctas;
      int lo = 0, hi = static_cast<int>(n_tiles);
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pos[mid] <= x) lo = mid; else hi = mid;
      }
      const int2 at = tiles[lo];
      const int n = __ldg(p.cu_q + at.x + 1) - __ldg(p.cu_q + at.x);
      cut = paged_cut(p, x, pos[lo], lo, unit_blocks(p, n, __ldg(p.kv_len + at.x), at.y));
    }
    s_cuts[c] = cut;
    p.plan.cuts[c] = cut;
  }
  __syncthreads();
  for (int c = tid; c < n_ctas; c += kPlanThreads) {
    if (s_cuts[c].z == 0) continue;
    const int2 at = tiles[s_cuts[c].x];
    const int q0 = __ldg(p.cu_q + at.x);
    PagedGroup g;
    if (paged_group(s_cuts, c, n_ctas, at, q0, __ldg(p.cu_q + at.x + 1) - q0, __ldg(p.kv_len + at.x), g))
      p.plan.groups[atomicAdd(&s_groups, 1)] = g;
  }
  __syncthreads();
  if (tid == 0) {
    p.plan.head->n_ctas = n_ctas;
    p.plan.head->n_groups = s_groups;
  }
}

// Merges the pieces of every cut unit: O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i, M = max m_i, the
// pieces in order.  A CTA takes kMergeRows rows of a unit, DV / 8 threads a row, so that all its loads of
// one piece are in flight together.
constexpr int kMergeRows = 16;

template <bool BF16, int DV>
__global__ void __launch_bounds__(kMergeRows * DV / 8) paged_combine_kernel(const PagedParams p) {
  constexpr int LANES = DV / 8;  // threads per row, 8 columns each
  pdl_wait();
  // read at once, whether the group exists or not
  const int n_groups = ld_dep(&p.plan.head->n_groups);
  const int4* record = reinterpret_cast<const int4*>(p.plan.groups + blockIdx.x);
  const int4 g0 = ld_dep(record), g1 = ld_dep(record + 1);
  if (static_cast<int>(blockIdx.x) >= n_groups) return;
  const int tile_u = g0.x, kvh = g0.y, first = g0.z, pieces = g0.w, slot0 = g1.x, q_off = g1.y, n = g1.z, len = g1.w;
  const int sk = min(max(len, 0), p.max_kv);
  const int prow = blockIdx.y * kMergeRows + threadIdx.x / LANES, col = 8 * (threadIdx.x % LANES);
  const int t = prow / kBlockQ, row = prow - t * kBlockQ;
  const int row_tok = static_cast<int>(fast_div(row, p.div_group));
  const int tile = tile_u * kTilesPerCta + t;
  const int tok = tile * p.tok_tile + row_tok;
  if (prow >= p.slot_rows || row_tok >= p.tok_tile || tok >= n) return;
  const int head = kvh * p.group + (row - row_tok * p.group);
  const int blocks = paged_tile_blocks(n, len, sk, p.tok_tile, p.causal, tile);
  float M = -INFINITY, L = 0.f;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int i = 0; i < pieces; ++i) {
    if (i > 0 && ld_dep(&p.plan.cuts[first + i].z) >= blocks) break;  // this tile ends before
    const int64_t r = static_cast<int64_t>(i == 0 ? slot0 : 2 * (first + i)) * p.slot_rows + prow;
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + r * 2);
    const float4 a = *reinterpret_cast<const float4*>(p.part_o + r * DV + col);
    const float4 b = *reinterpret_cast<const float4*>(p.part_o + r * DV + col + 4);
    const float top = fmaxf(M, ml.x);
    const float w0 = M == -INFINITY ? 0.f : ex2(M - top), w1 = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
    M = top;
    L = L * w0 + w1 * ml.y;
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] = acc[c] * w0 + w1 * v[c];
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  uint32_t pk[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    pk[i] = BF16 ? pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv) : pack_f16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + static_cast<int64_t>(q_off + tok) * p.o_s +
                            static_cast<int64_t>(head) * p.o_h + col) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  if (p.lse != nullptr && col == 0)
    p.lse[static_cast<int64_t>(head) * p.total_q + q_off + tok] = L > 0.f ? (M + lg2(L)) * 0.6931471805599453f : -INFINITY;
}

// Work tiles that calls of these sizes can have.
long long tiles_bound(int B, int total_q, int max_seqlen_q, int group) {
  const long long tok_unit = kTilesPerCta * (kBlockQ / group);
  return std::min(static_cast<long long>(B) * ((max_seqlen_q + tok_unit - 1) / tok_unit),
                  (static_cast<long long>(total_q) + (tok_unit - 1) * B) / tok_unit);
}

// Rows of a partial slot: both query tiles, or the rows of the longest chunk where one tile holds it.
int slot_rows(int group, int max_seqlen_q) {
  const int tok_tile = kBlockQ / group;
  return max_seqlen_q <= tok_tile ? max_seqlen_q * group : kCtaRows;
}

// Bytes of partial results: two slots per CTA; none where no unit is long enough to be cut.
size_t partial_bytes(int group, int max_seqlen_q, int max_kv, int Dv) {
  if ((max_kv + kBlockK - 1) / kBlockK < 2 * kMinPiece) return 0;
  return 2ull * kPagedMaxCtas * slot_rows(group, max_seqlen_q) * (Dv + 2) * sizeof(float);
}

bool encode_q(CUtensorMap* map, const void* q, bool bf16, int total_q, int Hq, int D, int64_t q_s, int64_t q_h, int group) {
  // [total_q, Hq, D] with a box of tok_tile tokens x G heads x 64 columns: rows (token, head)
  return encode_tiled3(map, q, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, D, Hq, total_q,
                       q_h, q_s, 64, group, kBlockQ / group, CU_TENSOR_MAP_SWIZZLE_128B);
}

int fwd_paged(bool quant, const void* q, const void* k_pool, const void* v_pool, const float* k_scale,
              const float* v_scale, const int32_t* page_table, const int32_t* kv_len, const int32_t* cu_q, void* o,
              float* lse, int B, int Hq, int Hkv, int total_q, int max_seqlen_q, int page_size, int max_pages,
              int n_pages, int D, int Dv, const int64_t* strides, float scale, int causal, void* workspace,
              size_t workspace_bytes, int dtype, void* stream) {
  // ---- validation (no CUDA call before this block passes)
  if (!q || !k_pool || !v_pool || !page_table || !kv_len || !cu_q || !o || (quant && (!k_scale || !v_scale)))
    return SDPA_ERR_INVALID;
  if (B < 1 || Hq < 1 || Hkv < 1 || total_q < 1 || max_seqlen_q < 1 || max_seqlen_q > total_q || D < 1 || Dv < 1)
    return SDPA_ERR_INVALID;
  if (Hq % Hkv != 0) return SDPA_ERR_INVALID;
  if (!(std::isfinite(scale) && scale > 0.f)) return SDPA_ERR_INVALID;
  int rc = page_check(page_size, max_pages, n_pages);
  if (rc != SDPA_OK) return rc;
  if (dtype != SDPA_F16 && dtype != SDPA_BF16) return SDPA_ERR_UNSUPPORTED;
  if (!((D == 64 && Dv == 64) || (D == 128 && Dv == 128) || (D == 192 && Dv == 128))) return SDPA_ERR_UNSUPPORTED;
  const int group = Hq / Hkv;
  if (group > kBlockQ) return SDPA_ERR_UNSUPPORTED;  // the heads of a KV head share one 128-row tile
  int64_t st[SDPA_FWD_PAGED_NSTRIDES] = {(int64_t)Hq * D, D, (int64_t)page_size * Hkv * D, (int64_t)Hkv * D, D,
                                         (int64_t)page_size * Hkv * Dv, (int64_t)Hkv * Dv, Dv, (int64_t)Hq * Dv, Dv,
                                         max_pages};
  if (strides) std::memcpy(st, strides, sizeof(st));
  for (int i = 0; i < 10; ++i)
    if (!stride_ok(st[i], quant && i >= 2 && i < 8 ? 16 : 8)) return SDPA_ERR_UNSUPPORTED;
  if (st[10] < max_pages) return SDPA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(o)) return SDPA_ERR_UNSUPPORTED;
  if (quant && (!aligned16(k_scale) || !aligned16(v_scale))) return SDPA_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(kv_len) | reinterpret_cast<uintptr_t>(cu_q) |
       reinterpret_cast<uintptr_t>(lse)) & 3u)
    return SDPA_ERR_INVALID;
  const int max_kv = max_pages * page_size;
  const long long tiles = tiles_bound(B, total_q, max_seqlen_q, group);
  if (tiles * Hkv >= (1ll << 30)) return SDPA_ERR_UNSUPPORTED;
  const size_t plan = paged_plan_bytes(B, tiles), partials = partial_bytes(group, max_seqlen_q, max_kv, Dv);
  if (!workspace || !aligned16(workspace) || workspace_bytes < plan) return SDPA_ERR_INVALID;

  PagedParams p{};
  p.o = o, p.lse = lse, p.o_s = st[8], p.o_h = st[9];
  p.cu_q = cu_q, p.kv_len = kv_len, p.page_table = page_table, p.pt_b = st[10];
  p.k_scale = k_scale, p.v_scale = v_scale;
  p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.total_q = total_q, p.max_seqlen_q = max_seqlen_q, p.group = group;
  p.causal = causal ? 1 : 0;
  p.tok_tile = kBlockQ / group;
  p.page_size = page_size, p.log2_page = __builtin_ctz((unsigned)page_size);
  p.max_pages = max_pages, p.n_pages = n_pages, p.max_kv = max_kv;
  p.scale2 = (float)((double)scale * 1.4426950408889634);
  p.div_group = make_fastdiv((uint32_t)group);
  p.slot_rows = slot_rows(group, max_seqlen_q);
  p.cut = partials > 0 && workspace_bytes >= plan + partials;
  p.max_tiles = (int)tiles;
  p.inline_plan = B <= kInlinePlanSeqs && max_seqlen_q <= p.tok_tile && !(quant && D == 192);
  p.plan = paged_plan_at(workspace, tiles);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan);
  p.part_ml = p.part_o + 2ull * kPagedMaxCtas * p.slot_rows * Dv;
  int dev = 0;
  if (current_device_sms(&dev, &p.sms) != cudaSuccess || device_status_ptr(&p.status) != cudaSuccess) return SDPA_ERR_CUDA;
  p.sms = std::min(p.sms, kPagedMaxCtas);

  alignas(64) CUtensorMap tq, tk, tv;
  const int rows = std::min(kBlockK, page_size);
  bool ok = encode_q(&tq, q, dtype == SDPA_BF16, total_q, Hq, D, st[0], st[1], group);
  if (quant) {
    auto codes = [&](CUtensorMap* map, const void* pool, int dim, const int64_t* s) {
      const int w = dim % 128 == 0 ? 128 : 64;
      return encode_bshd(map, pool, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, n_pages, page_size, Hkv, dim, s[0], s[1], s[2], w,
                         rows, w == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
    };
    ok = ok && codes(&tk, k_pool, D, st + 2) && codes(&tv, v_pool, Dv, st + 5);
  } else {
    const CUtensorMapDataType dt = dtype == SDPA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    ok = ok && encode_bshd(&tk, k_pool, dt, 2, n_pages, page_size, Hkv, D, st[2], st[3], st[4], 64, rows,
                           CU_TENSOR_MAP_SWIZZLE_128B) &&
         encode_bshd(&tv, v_pool, dt, 2, n_pages, page_size, Hkv, Dv, st[5], st[6], st[7], 64, rows,
                     CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (!ok) return SDPA_ERR_CUDA;
  p.stall_first_stage = take_stall_flag();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == SDPA_BF16;
  cudaError_t e = p.inline_plan ? cudaSuccess : launch_paged_plan(p, s);
  if (e == cudaSuccess)
    e = quant ? launch_paged_fp8(bf16, D, tq, tk, tv, p, s)
              : (bf16 ? launch_paged_bf16(D, tq, tk, tv, p, s) : launch_paged_f16(D, tq, tk, tv, p, s));
  if (e == cudaSuccess && p.cut) e = launch_paged_combine(bf16, Dv, p, s);
  return e == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

}  // namespace

cudaError_t launch_paged_plan(const PagedParams& p, cudaStream_t st) {
  paged_plan_kernel<<<1, kPlanThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_paged_combine(bool bf16, int Dv, const PagedParams& p, cudaStream_t st) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // at most sms - 1 units are cut
  cfg.gridDim = dim3(static_cast<unsigned>(std::max(p.sms - 1, 1)), static_cast<unsigned>((p.slot_rows + kMergeRows - 1) / kMergeRows));
  cfg.blockDim = dim3(kMergeRows * Dv / 8);
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  if (Dv == 64)
    return bf16 ? cudaLaunchKernelEx(&cfg, paged_combine_kernel<true, 64>, p)
                : cudaLaunchKernelEx(&cfg, paged_combine_kernel<false, 64>, p);
  return bf16 ? cudaLaunchKernelEx(&cfg, paged_combine_kernel<true, 128>, p)
              : cudaLaunchKernelEx(&cfg, paged_combine_kernel<false, 128>, p);
}

}  // namespace sdpa

using namespace sdpa;

extern "C" {

size_t sdpa_fwd_paged_workspace_size(int B, int Hq, int Hkv, int total_q, int max_seqlen_q, int max_kv, int Dv) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > kBlockQ || total_q < 1 || max_seqlen_q < 1 ||
      max_seqlen_q > total_q || max_kv < 1 || max_kv > (1 << 30) || Dv < 1)
    return 0;
  const int group = Hq / Hkv;
  return paged_plan_bytes(B, tiles_bound(B, total_q, max_seqlen_q, group)) + partial_bytes(group, max_seqlen_q, max_kv, Dv);
}

int sdpa_fwd_paged(const void* q, const void* k_pool, const void* v_pool, const int32_t* page_table,
                   const int32_t* kv_len, const int32_t* cu_seqlens_q, void* o, float* lse, int B, int Hq, int Hkv,
                   int total_q, int max_seqlen_q, int page_size, int max_pages, int n_pages, int D, int Dv,
                   const int64_t* strides, float scale, int causal, void* workspace, size_t workspace_bytes,
                   sdpa_dtype dtype, void* stream) {
  return fwd_paged(false, q, k_pool, v_pool, nullptr, nullptr, page_table, kv_len, cu_seqlens_q, o, lse, B, Hq, Hkv,
                   total_q, max_seqlen_q, page_size, max_pages, n_pages, D, Dv, strides, scale, causal, workspace,
                   workspace_bytes, dtype, stream);
}

int sdpa_fwd_paged_fp8(const void* q, const void* k_pool, const void* v_pool, const float* k_scale,
                       const float* v_scale, const int32_t* page_table, const int32_t* kv_len,
                       const int32_t* cu_seqlens_q, void* o, float* lse, int B, int Hq, int Hkv, int total_q,
                       int max_seqlen_q, int page_size, int max_pages, int n_pages, int D, int Dv,
                       const int64_t* strides, float scale, int causal, void* workspace, size_t workspace_bytes,
                       sdpa_dtype dtype, void* stream) {
  return fwd_paged(true, q, k_pool, v_pool, k_scale, v_scale, page_table, kv_len, cu_seqlens_q, o, lse, B, Hq, Hkv,
                   total_q, max_seqlen_q, page_size, max_pages, n_pages, D, Dv, strides, scale, causal, workspace,
                   workspace_bytes, dtype, stream);
}

}  // extern "C"
