// Attention of a chunk of new tokens per sequence over a paged cache (16-bit pages, or e4m3 pages
// with one scale per row), for sm_103a: TMA by page table -> shared-memory ring -> tcgen05 MMAs with
// accumulators in tensor memory -> blocked online softmax -> P.V, warp-specialised.
//
// The mathematics is that of the prefill kernels (running row max, lazily rescaled O, fp32 row sums).
// What the paged cache and the chunk change:
//   * a query tile's 128 rows are (token, head) pairs: the G query heads of a KV head ride in one
//     tile, tok_tile = 128 / G tokens high, so a short chunk still fills the rows and every K/V byte
//     serves all heads of its group.  One TMA box [tok_tile tokens, G heads, 64 columns] loads a chunk of columns;
//   * the keys of a 128-key block come in boxes of min(128, page_size) rows, one page each, issued
//     by the lanes of the producer warp side by side; pages past the cache read as zeros;
//   * rows of the last page past kv_len may hold anything: their scores are masked, and their V rows
//     are zeroed in shared memory before the P.V product (0 * NaN would poison it);
//   * all the work, every (query tile, KV head, key block), is one line that the SMs divide equally, so
//     that few query rows over long caches, ragged batches and long chunks alike keep every SM busy to the end.
//     A unit whose keys a cut divides writes partials (unnormalised O, max, sum) that a second
//     kernel merges.  The cuts are planned on the device, where the lengths are (paged_plan_kernel).
// Bound by the tensor cores for long chunks and by memory for short ones.  32 / 8 heads of 128, pages of 64, bf16:
// 8192 tokens over 32768 rows 2375-2490 us in a short run (1.55-1.6 PFLOP/s) and 2670-2730 under the power cap, drafts
// of 3-8 tokens of 16 sequences of 1024-16384 rows 102 us (5.6 TB/s); over e4m3 pages 4 x 2048 tokens of 16384 rows
// 1526 us (1.35 PFLOP/s), the drafts 88 us (3.4 TB/s).
// K and V blocks have a ring each and are loaded in the order of their use: K(0), then K(j) and V(j-1)
// for each j, then the last V.  A slot is so held for little longer than its MMAs take, and the rest of
// the rings is loads in flight.
//
// Quantised pages.  Every e4m3 value is exact in fp16, so converter warps turn a block's codes into fp16
// operands (one thread per row) and both products are fp16, whatever the query's type.  Long chunks have four
// such warps, which alternate between K and V and leave the softmax registers for a row's 128 scores; short ones,
// where the conversion of a block stands between its arrival and its MMAs, four for K and four for V (one
// warpgroup for both: 1760 -> 1590 us for 2048 tokens of 16384 rows of four sequences, but 95 -> 103 for drafts):
//   * K' = code * (k_scale / 2^ek), 2^(ek + 6) the power of two of the block's largest scale: the
//     largest row lies just below fp16's largest value, rows of power-of-two scales stay exact down
//     to 2^-21 of the largest scale and lose a bit for each one below (K' is read as 0 under
//     2^-30).  Other scales cost two roundings, of the factor and of the product (2^-11 each; a single one would
//     need the products in fp32, and the conversions to it and back).  The block's scores are multiplied by 2^ek;
//   * V' likewise with ev, and 2^ev joins the exponent: with y = s + ev the running maximum is taken
//     over y, P = 2^(y - m) meets V', and the row sum takes 2^-ev of the block's sum.  P stays in
//     fp16's best range whatever the scales are;
//   * a bf16 query is brought into fp16's range by a power of two per row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.h"
#include "ptx.cuh"

namespace sdpa {

constexpr float kPagedRescaleLog2 = 8.0f;
constexpr float kPagedLn2 = 0.6931471805599453f;
constexpr int kMinBlockExp = -100;  // exponent floor of a block's scales: 2^100 * sums stays finite
constexpr int kBlockExpRoom = 6;    // codes reach 448 < 2^9, fp16 65504: six powers of two to spare
constexpr float kMinBlkScale2 = 1.1754944e-38f;  // a factor of 0 would turn masked scores into NaN
constexpr int kFixRing = 8;         // v_ragged barriers: more than the ring holds blocks
constexpr int kExpRing = 8;         // blocks whose exponents are kept: more than the ring can run ahead

// ONE: no sequence has more tokens than one query tile holds.  In a graph, by this form and by the other, us over
// 16-bit and over e4m3 pages (32 / 8 heads of 128): drafts of 16 sequences of 1024-16384 rows 102 / 107 and 88 / 111, full
// tiles there (32 tokens) 107 / 110 and 97 / 119, full tiles of one head (8 / 8 heads, 128 tokens of 16384 rows)
// 184 / 188 and 155 / 202, 64 sequences of one key block 21.0 / 21.4 and 26 / 27, of two 23 / 26 and 30 / 35, 200 of 512-1024
// rows 121 / 130 and 173 / 190.  Shared memory then keeps one query tile,
// the two accumulators take the even and the odd key blocks ("readers" 0 and 1, each with half of the
// rings), so that one's softmax runs beside the other's MMAs, and slot 0's warps merge the two at the
// end of a piece.  Otherwise accumulator t serves query tile t and both read every block.
template <bool QUANT, int D, int DV, bool ONE>
struct PagedCfg {
  static constexpr int NCH_D = D / 64, NCH_V = DV / 64;
  static constexpr int Q_BYTES = kBlockQ * D * 2;
  static constexpr int K_BYTES = kBlockK * D * 2;
  static constexpr int V_BYTES = kBlockK * DV * 2;
  static constexpr int Q_TILES = ONE ? 1 : 2;
  // slots of the rings: what 227 KB hold beside the query tiles
  static constexpr int KS = D == 64 ? 4 : D == 128 ? (QUANT || ONE ? 2 : 3) : QUANT ? 1 : 2;
  static constexpr int VS = D == 64 ? 4 : D == 128 ? (ONE && !QUANT ? 4 : 2) : ONE ? 2 : 1;
  static constexpr int READERS = ONE ? 2 : 1;
  static constexpr int KR = KS / READERS, VR = VS / READERS;  // slots of a reader
  static_assert(KS % READERS == 0 && VS % READERS == 0, "every reader has the same slots");
  // raw codes: boxes of 128 (or 64) codes a row
  static constexpr int KW = D % 128 == 0 ? 128 : 64, VW = DV % 128 == 0 ? 128 : 64;
  static constexpr int KRAW = QUANT ? kBlockK * D : 0, VRAW = QUANT ? kBlockK * DV : 0;
  static constexpr int RAWS = !QUANT ? 0 : D == 64 ? 3 : ONE ? 2 : 1;  // of K, and of V
  static constexpr int QK_STEPS = D / 16, PV_STEPS = kBlockK / 16;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + Q_TILES * Q_BYTES;
  static constexpr int OFF_V = OFF_K + KS * K_BYTES;
  static constexpr int OFF_KRAW = OFF_V + VS * V_BYTES;
  static constexpr int OFF_VRAW = OFF_KRAW + RAWS * KRAW;
  static constexpr int OFF_BAR = OFF_VRAW + RAWS * VRAW;
  static constexpr int BARS = D == 64 ? 768 : 640;
  static constexpr int OFF_EXP = OFF_BAR + BARS;                    // int2 [kExpRing][4]
  static constexpr int OFF_QEXP = OFF_EXP + (QUANT ? kExpRing * 32 : 0);  // int8 [2 tiles][2][128]
  // pieces announced by the producer: more than it can run ahead of the slowest role.  Of the pieces
  // behind the one whose last V is used up, each has a V that waits in the rings for its softmax; of those
  // in which a role has no block, one at a time waits for it (passed).
  static constexpr int PIECES = D == 64 ? 16 : 8;
  static constexpr int OFF_PIECE = OFF_QEXP + (QUANT ? 512 : 0);
  static constexpr int OFF_ML = OFF_PIECE + PIECES * 64;            // float2 [128]: max and sum of slot 1
  static constexpr int SMEM = OFF_ML + 1024;
  static_assert((KS > VS ? KS : VS) + 2 <= kExpRing, "the exponent ring holds what the converters write");
  static_assert(VS + RAWS + 4 <= PIECES, "the piece ring holds what the producer announces");
  // warpgroups: control (producer, MMA, helpers), converters (quantised: of K and of V, or one of both), two softmax
  static constexpr int CONVERTERS = !QUANT ? 0 : ONE ? 2 : 1;
  static constexpr int SOFTMAX_WARP = 4 + 4 * CONVERTERS;
  static constexpr int THREADS = SOFTMAX_WARP * 32 + 256;
  // scores of its row that a softmax thread holds at a time
  static constexpr int HELD = CONVERTERS == 2 ? 64 : kBlockK;
  // registers per thread; the sums must stay within what the block is launched with
  static constexpr uint32_t REGS_CONTROL = CONVERTERS == 1 ? 56 : QUANT ? 64 : 96;
  static constexpr uint32_t REGS_CONVERT = 72;
  static constexpr uint32_t REGS_SOFTMAX = CONVERTERS == 1 ? 192 : QUANT ? 136 : 200;
  static constexpr uint32_t REGS_LAUNCH = CONVERTERS == 1 ? 128 : QUANT ? 96 : 168;
  static_assert(128 * REGS_CONTROL + 128 * CONVERTERS * REGS_CONVERT + 256 * REGS_SOFTMAX <= THREADS * REGS_LAUNCH,
                "register split exceeds the launch");
  static_assert(SMEM <= 227 * 1024, "more shared memory than a CTA may opt in to");
  static_assert(Q_BYTES % 1024 == 0 && K_BYTES % 1024 == 0 && V_BYTES % 1024 == 0 && KRAW % 1024 == 0 && VRAW % 1024 == 0,
                "1 KB tile alignment");
};

// One piece of a work unit: two query tiles (2 * tok_tile tokens of one sequence, the G heads of one KV
// head) against the key blocks [jb0, jb0 + n_blocks).
struct PagedPiece {
  int b, kvh, tok0, jb0;
  int n_blocks;            // 0: no more pieces
  int n_s[2];              // blocks that each accumulator takes: those its tile sees, or the even and the odd ones
  int slot;                // partial slot, or -1: the whole unit, which stores O itself
  int q_off, n, len, sk;
  int k_off;               // packed keys: the sequence's first row
  int pad[3];
};
static_assert(sizeof(PagedPiece) == 64, "the producer announces a piece in 64 bytes");

// The tiles of the plan; the host, where tests replay the walk, reads them plainly.
__host__ __device__ __forceinline__ int2 walk_ld(const int2* p) {
#ifdef __CUDA_ARCH__
  return ld_dep(p);
#else
  return *p;
#endif
}

// The pieces of a CTA's stretch of the line, in order (the producer's walk; the other roles read
// what it announces).
struct PagedWalk {
  int cta, tile, kvh, off, first;
  int4 end;

  __host__ __device__ __forceinline__ PagedWalk(int cta, int4 from, int4 to)
      : cta(cta), tile(from.x), kvh(from.y), off(from.z), first(1), end(to) {}
  template <bool ONE>
  __host__ __device__ __forceinline__ PagedPiece next(const PagedParams& p) {
    PagedPiece w{};
    // planned by this kernel, tiles are sequences, and those without tokens are passed over
    if (ONE && p.inline_plan)
      while (tile < end.x && plan_ld(p.cu_q + tile) == plan_ld(p.cu_q + tile + 1)) ++tile;
    if (!(tile < end.x || (tile == end.x && (kvh < end.y || (kvh == end.y && off < end.z))))) return w;
    const int2 at = ONE && p.inline_plan ? make_int2(tile, 0) : walk_ld(p.plan.tiles + tile);
    const int all = unit<ONE>(p, at, w);
    const int stop = (tile == end.x && kvh == end.y) ? end.z : all;
    w.kvh = kvh;
    w.jb0 = off;
    w.n_blocks = stop - off;
#pragma unroll
    for (int t = 0; t < 2; ++t)
      w.n_s[t] = ONE ? (w.n_blocks + 1 - t) / 2 : min(max(w.n_s[t] - off, 0), w.n_blocks);
    w.slot = (off > 0 || stop < all) ? 2 * cta + 1 - first : -1;
    first = 0;
    off = 0;
    if (++kvh == p.Hkv) kvh = 0, ++tile;
    return w;
  }
  // Item i of the list: a whole unit.
  __host__ __device__ __forceinline__ static PagedPiece item(const PagedParams& p, int i, int n_items) {
    const int tiles = n_items / p.Hkv, per = tiles * p.list_heads;
    const int g = i / per, heads = min(p.list_heads, p.Hkv - g * p.list_heads);
    const int r = i - g * per, rank = r / heads;
    PagedPiece w{};
    w.n_blocks = unit<false>(p, walk_ld(p.plan.tiles + rank), w);
    w.kvh = g * p.list_heads + (r - rank * heads);
    w.slot = -1;
    return w;
  }

 private:
  // Fills in the sequence of a unit, and in n_s the blocks that its tiles see; returns the longer one's.
  template <bool ONE>
  __host__ __device__ __forceinline__ static int unit(const PagedParams& p, int2 at, PagedPiece& w) {
    w.b = at.x;
    w.q_off = plan_ld(p.cu_q + w.b);
    w.n = plan_ld(p.cu_q + w.b + 1) - w.q_off;
    w.len = paged_len(p, w.b);
    w.k_off = p.cu_k != nullptr ? plan_ld(p.cu_k + w.b) : 0;
    w.sk = min(max(w.len, 0), p.max_kv);
    w.tok0 = at.y * kTilesPerCta * p.tok_tile;
#pragma unroll
    for (int t = 0; t < kTilesPerCta; ++t)
      w.n_s[t] = paged_tile_blocks(w.n, w.len, w.sk, p.tok_tile, p.causal, at.y * kTilesPerCta + t);
    return max(w.n_s[0], w.n_s[1]);
  }
};

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Converts row r of a raw tile (boxes of W codes a row, swizzled) into `chunks` 128-byte-swizzled fp16
// chunks of 64 columns, as the MMAs read them, times the pair factor f; f = 0 stores zeros whatever
// the codes are.  One thread per row: both the reads and the writes of eight neighbouring rows
// fall on all banks.  The loop over chunks is not unrolled: the kernel's loops together must fit the
// instruction cache (drafts of 16 sequences: 92.5 us so, 100 with two chunks an iteration, 96 with half a one).
template <int W>
__device__ __forceinline__ void convert_row(const uint8_t* raw, uint8_t* dst, int chunks, int r, uint32_t f) {
  const int x = (r & 7) << 4;
  const bool live = f != 0u;
#pragma unroll 1
  for (int ch = 0; ch < chunks; ++ch) {
    const uint8_t* src = W == 128 ? raw + (ch >> 1) * kBlockK * 128 + r * 128 : raw + ch * kBlockK * 64 + r * 64;
    uint4 c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int off = W == 128 ? ((((ch & 1) * 4 + i) << 4) ^ x) : ((i << 4) ^ (((r >> 1) & 3) << 4));
      c[i] = *reinterpret_cast<const uint4*>(src + off);
    }
    uint8_t* d = dst + ch * kBlockK * 128 + r * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
      uint32_t h[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        e4m3x4_to_f16x4(live ? w[q] : 0u, h[2 * q], h[2 * q + 1]);
        h[2 * q] = mul_f16x2(h[2 * q], f);
        h[2 * q + 1] = mul_f16x2(h[2 * q + 1], f);
      }
      *reinterpret_cast<uint4*>(d + (((2 * i) << 4) ^ x)) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(d + (((2 * i + 1) << 4) ^ x)) = make_uint4(h[4], h[5], h[6], h[7]);
    }
  }
}

// Exponents of a block's largest scales of K and V from those of its four 32-row parts (biased as in
// fp32), less the room that fp16 leaves above the codes.
__device__ __forceinline__ int2 block_exp(const int2* parts) {
  const int4 a = *reinterpret_cast<const int4*>(parts), b = *reinterpret_cast<const int4*>(parts + 2);
  return make_int2(max(max(max(a.x, a.z), max(b.x, b.z)) - 127 - kBlockExpRoom, kMinBlockExp),
                   max(max(max(a.y, a.w), max(b.y, b.w)) - 127 - kBlockExpRoom, kMinBlockExp));
}

// One arrival for a warp whose lanes have all done their part (their fences included).
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// The plan where every sequence has one query tile, by each CTA for itself: a scan over the sequences'
// lengths on the line, then this CTA's two cuts; CTA 0 stores all of them and the cut units for the merge.
// Spares the launch of a planning kernel and the wait for it (in a graph, 16-bit and e4m3 pages: drafts of 16 sequences
// 104.5 -> 101.7 us and 89.1 -> 87.9, 64 sequences of one key block 22.7 -> 21.0 and 28.0 -> 26.3, 200 of 512-1024 rows
// 123 -> 122 and 174 -> 173).
// scratch: 8 KB of shared memory that nobody uses yet.  All threads; returns the cuts in `mine`.
template <int THREADS>
__device__ __forceinline__ void paged_inline_plan(const PagedParams& p, uint8_t* scratch, int4* mine) {
  static_assert(THREADS >= kInlinePlanSeqs && THREADS > kPagedMaxCtas, "one thread per sequence and per cut");
  long long* pos = reinterpret_cast<long long*>(scratch);               // [kInlinePlanSeqs + 1]
  long long* warp_sum = pos + kInlinePlanSeqs + 1;                       // [THREADS / 32]
  int4* cuts = reinterpret_cast<int4*>(scratch + 4096);                  // [kPagedMaxCtas + 1]
  int* n_groups = reinterpret_cast<int*>(cuts + kPagedMaxCtas + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int bad = 0, n = 0, len = 0;
  long long v = 0;
  if (tid < p.B) {
    const int q0 = __ldg(p.cu_q + tid), q1 = __ldg(p.cu_q + tid + 1);
    len = paged_len(p, tid);
    bad = paged_bad(p, tid, q0, q1);
    n = q1 - q0;
    if (!bad && n > 0)
      v = static_cast<long long>(paged_tile_blocks(n, len, min(max(len, 0), p.max_kv), p.tok_tile, p.causal, 0) + kUnitCost) *
          p.Hkv;
  }
  long long incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  if (tid == 0) *n_groups = 0;
  bad = __syncthreads_or(bad);
  const int units = __syncthreads_count(v > 0) * p.Hkv;
  for (int w = 0; w < warp; ++w) incl += warp_sum[w];
  if (tid < p.B) pos[tid + 1] = incl;
  if (tid == 0) pos[0] = 0;
  __syncthreads();
  const long long total = pos[p.B];
  const int n_ctas = bad ? 0 : static_cast<int>(min(static_cast<long long>(p.sms), max(static_cast<long long>(units), total / p.min_work)));
  const int cta = blockIdx.x;
  auto cut_at = [&](int c) { return bad ? make_int4(0, 0, 0, 0) : paged_inline_cut(p, pos, c, n_ctas); };
  if (cta < n_ctas) {
    if (tid == 0) mine[0] = cut_at(cta);
    if (tid == 32) mine[1] = cut_at(cta + 1);
  } else if (tid == 0) {
    mine[0] = mine[1] = make_int4(0, 0, 0, 0);
  }
  if (cta == 0) {  // for the merge
    if (tid <= n_ctas) p.plan.cuts[tid] = cuts[tid] = cut_at(tid);
    __syncthreads();
    if (tid < n_ctas && cuts[tid].z != 0) {
      const int b = cuts[tid].x, q0 = __ldg(p.cu_q + b);
      PagedGroup g;
      if (paged_group(cuts, tid, n_ctas, make_int2(b, 0), q0, __ldg(p.cu_q + b + 1) - q0, paged_len(p, b), g))
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

// Barriers (phases continue from piece to piece; the arrivals of warps are one each):
//   piece[i % PIECES]     : the producer announced piece i
//   passed[r]             : softmax r (all its threads), or the helper (r = 2), has passed a piece in which it has no
//                           block; nothing else holds the producer for it there (e4m3 mixed batch 258 -> 261 us;
//                           a barrier that every role arrives at in every piece: 267)
//   q_full[t] / q_empty[t]: Q tile t landed / accumulator t's last QK MMA of the piece finished
//   q_ready[t]            : quantised pages and a bf16 query: tile t converted to fp16
//   kv_full / kv_empty    : a slot of the K or V ring holds its block / the issuers that read it are done
//   kc_full[3 s + c]      : shared slots: chunk c of K's block s (mod 2) landed, in kv_full's place
//   raw_full / raw_empty  : quantised pages: codes of K (0) or V (1) landed / read by the converters
//   e_full[i % 8 (+ 8)]   : quantised pages: each converter warp of K (of V, where those are others) has stored
//                           the exponents of its 32 rows of block i (the block's are the largest of the four)
//   turn[t]               : issuer t may issue (both tiles active)
//   v_ragged[i % 8]       : 16-bit pages: the i-th V block that ends past kv_len landed; a helper warp
//                           then zeroes those rows and completes kv_full in the copy's place
//   s_full[t], p_half[t], p_full[t], o_full[t], o_empty[t]: as in the prefill kernels, per accumulator
//   ml_full               : ONE: accumulator 1's max and sum are there
//
// PACKED: keys and values are packed rows instead of pages, and the last 64 columns of the keys come from a tensor of
// their own without heads (tm_r; unused otherwise).  Only the loads differ: a block is one box of 128 rows a column chunk.
template <bool BF16, bool QUANT, int D, int DV, bool ONE, bool PACKED>
__global__ void __launch_bounds__(PagedCfg<QUANT, D, DV, ONE>::THREADS, 1)
    paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_r, const PagedParams p) {
  static_assert(!(PACKED && QUANT), "packed keys are 16 bits wide");
  using C = PagedCfg<QUANT, D, DV, ONE>;
  // Packed keys of D = 192: beside two query tiles there is room for K of two blocks and V of one, and a single slot of V
  // leaves its load no more time than one tile's Q K^T.  So K and V share eight 16 KB slots: block g's three chunks of K
  // are numbers 5 g .. 5 g + 2, its V's two halves (64 keys) 5 g + 3 and 5 g + 4, number i lies in slot i % 8.  V(g) then takes
  // the place of K(g - 1), loaded two steps before its use, and K(g) those of K(g - 2) and V(g - 2), which are free before the
  // second tile's last Q K^T: every load has at least three products' time (8192 tokens x 128 heads: 2529 -> 2200 us).
  constexpr bool SHARED = PACKED && !ONE;
  constexpr int KS = C::KS, VS = SHARED ? 2 : C::VS, KR = C::KR, VR = SHARED ? 2 : C::VR;
  constexpr int kSlot = 16 * 1024;
  static_assert(!SHARED || (C::NCH_D == 3 && C::NCH_V == 2 && C::KS * C::K_BYTES + C::VS * C::V_BYTES == 8 * kSlot), "eight slots");
  constexpr int NR = C::RAWS > 0 ? C::RAWS : 1;
  constexpr int HELD = C::HELD;
  constexpr bool CONVERT_Q = QUANT && BF16;
  constexpr bool F16_MATH = QUANT || !BF16;
  // D = 128 fills the shared memory, without room to align the window by hand
  extern __shared__ __align__(1024) uint8_t paged_smem[];
  uint8_t* smem = paged_smem;
  if (smem_u32(smem) & 1023u) {  // never: nothing static lies in front of it
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars;              // [2]
  uint64_t* q_empty = q_full + 2;       // [2]
  uint64_t* q_ready = q_empty + 2;      // [2]
  uint64_t* s_full = q_ready + 2;       // [2]
  uint64_t* p_half = s_full + 2;        // [2]
  uint64_t* p_full = p_half + 2;        // [2]
  uint64_t* o_full = p_full + 2;        // [2]
  uint64_t* o_empty = o_full + 2;       // [2]
  uint64_t* mma_done = o_empty + 2;     // [2]
  uint64_t* turn = mma_done + 2;        // [2]
  uint64_t* v_ragged = turn + 2;        // [kFixRing]
  // one array for K (first KS or NR) and V (behind them)
  uint64_t* kv_full = v_ragged + kFixRing;   // [KS + VS]
  uint64_t* kv_empty = kv_full + KS + VS;    // [KS + VS]
  uint64_t* raw_full = kv_empty + KS + VS;   // [2 NR]
  uint64_t* raw_empty = raw_full + 2 * NR;   // [2 NR]
  uint64_t* e_full = raw_empty + 2 * NR;    // [2 kExpRing]
  uint64_t* piece = e_full + 2 * kExpRing;  // [PIECES]
  uint64_t* passed = piece + C::PIECES;   // [3]
  uint64_t* ml_full = passed + 3;         // [1]
  uint64_t* kc_full = ml_full + 1;        // [6], shared slots only: chunk c of the K block in ring slot s, 3 s + c
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(kc_full + (SHARED ? 6 : 0));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int2* blk_exp = reinterpret_cast<int2*>(smem + C::OFF_EXP);
  int8_t* q_exp = reinterpret_cast<int8_t*>(smem + C::OFF_QEXP);
  PagedPiece* pieces = reinterpret_cast<PagedPiece*>(smem + C::OFF_PIECE);
  float2* ml_x = reinterpret_cast<float2*>(smem + C::OFF_ML);  // [128]
  static_assert(((SHARED ? 30 : 24) + kFixRing + 2 * kExpRing + 2 * (KS + VS) + 4 * NR + C::PIECES) * 8 + 8 <= C::BARS, "barriers fit their area");

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  pdl_launch_dependents();  // the combine may be scheduled early; it waits for this grid

  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_ready[t], 4);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_half[t], 4);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_full[t], 1);
      mbar_init(&o_empty[t], 4);
      mbar_init(&mma_done[t], 1);
      mbar_init(&turn[t], 1);
    }
    mbar_init(ml_full, 4);
    for (int s = 0; s < (SHARED ? 6 : 0); ++s) mbar_init(&kc_full[s], 1);
    for (int t = 0; t < 2; ++t) mbar_init(&q_empty[t], 1);
    for (int s = 0; s < kFixRing; ++s) mbar_init(&v_ragged[s], 1);
    for (int s = 0; s < KS + VS; ++s) {
      mbar_init(&kv_full[s], QUANT ? 4 : 1);
      mbar_init(&kv_empty[s], ONE ? 1 : 2);
    }
    for (int s = 0; s < 2 * kExpRing; ++s) mbar_init(&e_full[s], 4);
    for (int s = 0; s < 2 * NR; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    for (int s = 0; s < C::PIECES; ++s) mbar_init(&piece[s], 1);
    for (int r = 0; r < 3; ++r) mbar_init(&passed[r], r < 2 ? 128 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  int4 cuts[2] = {make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0)};
  if (ONE && p.inline_plan) {
    int4* mine = reinterpret_cast<int4*>(&pieces[C::PIECES - 1]);  // not announced before the producer has read it
    paged_inline_plan<C::THREADS>(p, sQ, mine);
    if (warp == 0) cuts[0] = mine[0], cuts[1] = mine[1];
  } else {
    pdl_wait();  // the plan comes from the kernel launched before
    if (warp == 0 && static_cast<int>(blockIdx.x) < ld_dep(&p.plan.head->n_ctas)) {
      cuts[0] = ld_dep(p.plan.cuts + blockIdx.x);
      cuts[1] = ld_dep(p.plan.cuts + blockIdx.x + 1);
    }
  }
  // the next announced piece, for the other roles
  int n_piece = 0;
  auto next_piece = [&](bool& ok) -> const PagedPiece& {
    const PagedPiece& w = pieces[n_piece % C::PIECES];
    ok = mbar_wait(&piece[n_piece % C::PIECES], (n_piece / C::PIECES) & 1, abort_flag, p.status);
    ++n_piece;
    return w;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (one warp)
    regs_dec<C::REGS_CONTROL>();
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      if (PACKED) tma_prefetch_desc(&tm_r);
    }
    const int rows = PACKED ? kBlockK : min(kBlockK, p.page_size);  // rows per box
    const int nsub = kBlockK / rows;             // boxes per column chunk: 1 .. 8
    constexpr int KPARTS = QUANT ? D / C::KW : C::NCH_D, VPARTS = QUANT ? DV / C::VW : C::NCH_V;
    constexpr int KCOLS = QUANT ? C::KW : 64, VCOLS = QUANT ? C::VW : 64;    // columns per box
    constexpr int KROW = QUANT ? C::KW : 128, VROW = QUANT ? C::VW : 128;    // bytes of a box row
    constexpr int KTX = QUANT ? kBlockK * D : C::K_BYTES, VTX = QUANT ? kBlockK * DV : C::V_BYTES;
    // the rings that TMA fills: raw ones in the order of the blocks, or those of the readers
    constexpr int LK = QUANT ? NR : KR, LV = QUANT ? NR : VR;
    uint64_t* ld_full = QUANT ? raw_full : kv_full;
    uint64_t* ld_empty = QUANT ? raw_empty : kv_empty;
    const int q_tx = p.tok_tile * p.group * D * 2;
    PagedWalk walk(blockIdx.x, cuts[0], cuts[1]);
    // from a list: the next item is asked for while this one is loaded
    int n_items = 0, item = 0;
    auto take = [&]() { return lane == 0 ? atomicAdd(&p.plan.head->next_item, 1) : 0; };
    if constexpr (SHARED) {
      n_items = ld_dep(&p.plan.head->n_items);
      if (n_items > 0) item = take();
    }
    int qn[2] = {0, 0};     // pieces of each accumulator
    int nl[2][2] = {};      // blocks of K and of V issued (16-bit pages: per reader)
    int nr = 0;             // ragged V blocks among them
    int np[3] = {0, 0, 0};  // pieces without a block for softmax 0, softmax 1, the helper
    bool ok = true;
    while (ok) {
      PagedPiece w;
      if (SHARED && n_items > 0) {
        const int i = __shfl_sync(0xffffffffu, item, 0);
        w = i < n_items ? PagedWalk::item(p, i, n_items) : PagedPiece{};
        if (i < n_items) item = take();
      } else {
        w = walk.template next<ONE>(p);
      }
      if (w.n_blocks > 0) {
#pragma unroll
        for (int r = 0; r < (QUANT ? 2 : 3); ++r) {
          if (r < 2 ? w.n_s[r] > 0 : (w.jb0 + w.n_blocks) * kBlockK > w.sk) continue;
          if (np[r] > 0) ok = ok && mbar_wait_warp(&passed[r], (np[r] - 1) & 1, abort_flag, p.status);
          ++np[r];
        }
        if (!ok) break;
      }
      if (lane == 0) {
        pieces[n_piece % C::PIECES] = w;
        mbar_arrive(&piece[n_piece % C::PIECES]);
      }
      ++n_piece;
      if (w.n_blocks == 0) break;
      for (int t = 0; t < kTilesPerCta && ok; ++t) {
        if (ONE ? t == 1 : w.n_s[t] == 0) continue;
        // ONE: both accumulators have used the tile
        if ((qn[t] > 0 && !mbar_wait_warp(&q_empty[t], (qn[t] - 1) & 1, abort_flag, p.status)) ||
            (ONE && qn[1] > 0 && !mbar_wait_warp(&q_empty[1], (qn[1] - 1) & 1, abort_flag, p.status))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&q_full[t], q_tx);
          for (int c = 0; c < C::NCH_D; ++c)
            tma_load_3d(sQ + t * C::Q_BYTES + c * kBlockQ * 128, &tm_q, &q_full[t], c * 64, w.kvh * p.group,
                        w.q_off + w.tok0 + t * p.tok_tile);
        }
        ++qn[t];
        if (ONE) ++qn[1];
      }
      const int32_t* table = PACKED ? nullptr : p.page_table + w.b * p.pt_b;
      const int used = (w.sk + p.page_size - 1) >> p.log2_page;  // pages that hold visible rows
      const int sub = lane & 7;                                  // page of the block: lane % 8 < nsub
      int phys_k = p.n_pages, row_k = 0;  // page and row of this lane's box; outside the pool: zeros
      for (int j = 0; ok && j <= w.n_blocks; ++j) {
        const int phys_v = phys_k, row_v = row_k;
        if (j < w.n_blocks) {
          const int key = (w.jb0 + j) * kBlockK + sub * rows;
          if constexpr (PACKED) {  // rows of the next sequence or past the last one: masked, as V's are zeroed
            row_k = w.k_off + key, phys_k = 0;
          } else {
            const int lp = key >> p.log2_page;
            row_k = key & (p.page_size - 1);
            phys_k = p.n_pages;
            if (sub < nsub && lp < used) phys_k = __ldg(table + lp);
          }
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (kv == 0 || SHARED ? j == w.n_blocks : j == 0) continue;  // K(j), then V(j-1) (V(j) where they share slots)
          const int rd = ONE && !QUANT ? (j - kv) & 1 : 0;
          const int ring = kv == 0 ? LK : LV, base = (kv == 0 ? 0 : QUANT ? NR : KS) + rd * ring;
          const int c = rd ? nl[kv][1]++ : nl[kv][0]++;
          const int s = c % ring, r = c / ring;
          if (r > 0 && !mbar_wait_warp(&ld_empty[base + s], (r - 1) & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          // shared slots: V(c) comes in the place of K(c - 1), too
          if (SHARED && kv == 1 && c > 0 && !mbar_wait_warp(&ld_empty[(c - 1) % 2], ((c - 1) / 2) & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          if (p.stall_first_stage && c == 0) continue;  // test hook: the first slots never fill
          uint64_t* bar = &ld_full[base + s];
          if (!QUANT && kv == 1 && (w.jb0 + j + (SHARED ? 1 : 0)) * kBlockK > w.sk) {
            bar = &v_ragged[nr % kFixRing];
            ++nr;
          }
          if (lane == 0 && !(SHARED && kv == 0)) mbar_arrive_expect_tx(bar, kv == 0 ? KTX : VTX);
          __syncwarp();
          const int at = rd * ring + s;
          uint8_t* dst = kv == 0 ? (QUANT ? smem + C::OFF_KRAW + at * C::KRAW : sK + at * C::K_BYTES)
                                 : (QUANT ? smem + C::OFF_VRAW + at * C::VRAW : sV + at * C::V_BYTES);
          const int parts = kv == 0 ? KPARTS : VPARTS, row_b = kv == 0 ? KROW : VROW;
          const int part = lane >> 3;  // column chunk
          if constexpr (SHARED) {
            if (kv == 1) {  // V's halves of 64 keys, two boxes each
              if (sub == 0 && part < 4)
                tma_load_4d(sK + ((5 * c + 3 + (part >> 1)) & 7) * kSlot + (part & 1) * (kSlot / 2), &tm_v, bar, (part & 1) * 64,
                            w.kvh, row_k + (part >> 1) * 64, 0);
              continue;
            }
            // K's first chunk in the place of K(c - 2)'s last, the others in those of V(c - 2)
#pragma unroll 1
            for (int ch = 0; ch < 3; ++ch) {
              if (ch == 1 && c > 1 && !mbar_wait_warp(&ld_empty[KS + c % 2], ((c - 2) / 2) & 1, abort_flag, p.status)) {
                ok = false;
                break;
              }
              if (lane == 0) {
                mbar_arrive_expect_tx(&kc_full[3 * s + ch], kSlot);
                tma_load_4d(sK + ((5 * c + ch) & 7) * kSlot, ch == 2 ? &tm_r : &tm_k, &kc_full[3 * s + ch], ch == 2 ? 0 : ch * 64,
                            ch == 2 ? 0 : w.kvh, row_k, 0);
              }
            }
            __syncwarp();
            if (!ok) break;
            continue;
          }
          const bool shared = PACKED && kv == 0 && part == parts - 1;
          if (sub < nsub && part < parts)
            tma_load_4d(dst + part * kBlockK * row_b + sub * rows * row_b, shared ? &tm_r : kv == 0 ? &tm_k : &tm_v, bar,
                        shared ? 0 : part * (kv == 0 ? KCOLS : VCOLS), shared ? 0 : w.kvh, kv == 0 ? row_k : row_v,
                        kv == 0 ? phys_k : phys_v);
        }
      }
    }
    if (!ok && lane == 0) {
      // let every copy already in flight land before the CTA's shared memory goes away
      for (int t = 0; t < kTilesPerCta; ++t)
        if (qn[t] > 0) mbar_drain(&q_full[t], (qn[t] - 1) & 1);
      for (int j = max(0, nr - kFixRing); j < nr; ++j) mbar_drain(&v_ragged[j % kFixRing], (j / kFixRing) & 1);
      for (int kv = 0; kv < 2; ++kv)
        for (int rd = 0; rd < 2; ++rd) {
          const int ring = kv == 0 ? LK : LV, base = (kv == 0 ? 0 : QUANT ? NR : KS) + rd * ring;
          for (int j = max(0, nl[kv][rd] - ring); j < nl[kv][rd]; ++j) {
            if (SHARED && kv == 0)
              for (int ch = 0; ch < 3; ++ch) mbar_drain(&kc_full[3 * (j % ring) + ch], (j / ring) & 1);
            else
              mbar_drain(&ld_full[base + j % ring], (j / ring) & 1);
          }
        }
    }
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------ MMA issuers: one thread per query tile
    // An issuing thread blocks while the tensor core is busy, and whatever it does between two MMAs
    // (a wait that succeeds at once costs some 75 cycles) leaves the tensor core idle if nobody else
    // feeds it: with one issuer for both tiles that was 1800 of 4000 cycles a block.  So each tile
    // has its own, and the two take turns: an issuer waits for everything its step reads, then for
    // its turn, issues P.V and Q K^T, hands the turn over and does its commits while the other's MMAs
    // run.  Without turns the tiles drift into step and both softmaxes leave the tensor core alone.
    regs_dec<C::REGS_CONTROL>();
    if (lane == 0) {
      constexpr uint32_t fmt = F16_MATH ? 0 : 1;
      constexpr uint32_t idesc_qk = make_idesc(fmt, fmt, 0, 0, kBlockQ, kBlockK);
      constexpr uint32_t idesc_pv = make_idesc(fmt, fmt, 0, 1, kBlockQ, DV);
      const int t = warp >> 1;
      const uint64_t dq0 = make_smem_desc(smem_u32(sQ), 16, 1024, kSwizzle128B);
      const uint64_t dk0 = make_smem_desc(smem_u32(sK), 16, 1024, kSwizzle128B);
      const uint64_t dv0 = make_smem_desc(smem_u32(SHARED ? sK : sV), SHARED ? kSlot / 2 : kBlockK * 128, 1024, kSwizzle128B);
      const uint32_t q_lo = static_cast<uint32_t>(dq0), q_hi = static_cast<uint32_t>(dq0 >> 32);
      const uint32_t k_lo = static_cast<uint32_t>(dk0), k_hi = static_cast<uint32_t>(dk0 >> 32);
      const uint32_t v_lo = static_cast<uint32_t>(dv0), v_hi = static_cast<uint32_t>(dv0 >> 32);
      const uint32_t tS = tmem_base + t * 128;
      int gk = 0, gv = 0;         // shared slots: blocks of K and of V so far
      const uint32_t tO = tmem_base + 256 + t * 128;
      int qn = 0;                 // loads of this accumulator's query tile so far
      int on = 0, pn = 0;         // pieces and blocks of this slot so far
      uint32_t turns = 1 - t;     // parity of the turn barrier's next phase; tile 0 begins
      // slots of this reader's next K and V blocks and the parities of their phases
      const int k0 = ONE ? t * KR : 0, v0 = ONE ? t * VR : 0;
      int ks = k0, vs = v0;
      uint32_t kph = 0, vph = 0;
      bool ok = true;
      auto next_k = [&]() {
        if (++ks == k0 + KR) ks = k0, kph ^= 1u;
      };
      auto next_v = [&]() {
        if (++vs == v0 + VR) vs = v0, vph ^= 1u;
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, abort_flag, p.status); };
      const uint32_t dq = q_lo + static_cast<uint32_t>(((ONE ? 0 : t) * C::Q_BYTES) >> 4);
      // O (+)= P V for keys 0-63 or 64-127 of the V block in slot v, and S = Q K^T of the K block in slot k (with shared
      // slots: of block v and k)
      auto pv_half = [&](int half, int v, uint32_t acc) {
        const uint32_t dv = v_lo + static_cast<uint32_t>((SHARED ? ((5 * v + 3 + half) & 7) * kSlot - half * 64 * 128 : v * C::V_BYTES) >> 4);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < C::PV_STEPS / 2; ++kk) {
          const int q = half * C::PV_STEPS / 2 + kk;
          mma_f16_ts(tO, tS + q * 8, dv + static_cast<uint32_t>((q * 16 * 128) >> 4), v_hi, idesc_pv, kk > 0 ? 1u : acc);
        }
      };
      // Shared slots: chunk by chunk, those that had not landed before this tile's turn (landed) as they do.
      auto qk_chunks = [&](int k, int slot, uint32_t parity, const bool (&landed)[3]) {
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          if (!landed[c] && !wait(&kc_full[3 * slot + c], parity)) return false;
          tc_fence_after();
          const uint32_t b = k_lo + static_cast<uint32_t>((((5 * k + c) & 7) * kSlot) >> 4);
          const uint32_t a = dq + static_cast<uint32_t>((c * kBlockQ * 128) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_ss(tS, a + static_cast<uint32_t>((kk * 32) >> 4), q_hi, b + static_cast<uint32_t>((kk * 32) >> 4), k_hi, idesc_qk,
                       c > 0 || kk > 0 ? 1u : 0u);
        }
        return true;
      };
      auto qk = [&](int k) {
        const uint32_t dk = k_lo + static_cast<uint32_t>((k * C::K_BYTES) >> 4);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < C::QK_STEPS; ++kk) {
          const uint32_t off = static_cast<uint32_t>(((kk / 4) * kBlockQ * 128 + (kk % 4) * 32) >> 4);
          mma_f16_ss(tS, dq + off, q_hi, dk + off, k_hi, idesc_qk, kk > 0 ? 1u : 0u);
        }
      };
      while (true) {
        const PagedPiece& w = next_piece(ok);
        const int nb = ok ? w.n_blocks : 0;
        if (nb == 0) break;
        const int n = w.n_s[t];
        if constexpr (ONE) {
          // both issuers see every query tile and pass it on, so that none misses a phase
          if (!(ok = wait(CONVERT_Q ? &q_ready[0] : &q_full[0], qn & 1))) break;
          if (n == 0) mbar_arrive(&q_empty[t]);
          if (n > 0) {
            int vu = 0;  // slot of the last V and the parity of its phase
            uint32_t vup = 0;
            for (int i = 0;; ++i) {  // the reader's i-th block
              const int ku = ks;
              if (i < n) {
                if (!(ok = wait(&kv_full[ku], kph))) break;
                next_k();
              }
              if (i > 0) {  // O += P(i-1) V(i-1)
                if (!(ok = (i > 1 || on == 0 || wait(&o_empty[t], (on - 1) & 1)) && wait(&kv_full[KS + vu], vup) &&
                           wait(&p_half[t], pn & 1)))
                  break;
                pv_half(0, vu, i > 1 ? 1u : 0u);  // while the second half of P is computed
                if (!(ok = wait(&p_full[t], pn & 1))) break;
                pv_half(1, vu, 1u);
                ++pn;
                mma_commit(&kv_empty[KS + vu]);
              }
              if (i == n) {
                mma_commit(&o_full[t]);
                break;
              }
              qk(ku);
              mma_commit(&s_full[t]);
              mma_commit(&kv_empty[ku]);
              if (i == n - 1) mma_commit(&q_empty[t]);
              vu = vs, vup = vph;
              next_v();
            }
            if (!ok) break;
          }
          ++qn;
        } else {
          if (n > 0 && !(ok = wait(CONVERT_Q ? &q_ready[t] : &q_full[t], qn & 1))) break;
          // Step j: O += P(j-1) V(j-1), then S = Q K(j)^T.  A block that this tile does not see is seen
          // landing and passed on.
          for (int j = 0; j <= nb; ++j) {
            const int ku = ks, vu = vs;
            const uint32_t kpar = kph;
            bool landed[3] = {false, false, false};
            if (j < nb) {
              if (SHARED) {  // P V does not wait for them; a block that this tile does not see has to have landed
                if (j >= n && !(ok = wait(&kc_full[3 * ku], kpar) && wait(&kc_full[3 * ku + 1], kpar) && wait(&kc_full[3 * ku + 2], kpar))) break;
              } else if (!(ok = wait(&kv_full[ku], kph))) {
                break;
              }
              next_k();
            }
            if (j > 0) {
              if (!(ok = wait(&kv_full[KS + vu], vph))) break;
              next_v();
            }
            const bool pv = j > 0 && j <= n;
            if (pv && !(ok = (j > 1 || on == 0 || wait(&o_empty[t], (on - 1) & 1)) && wait(&p_full[t], pn & 1))) break;
            if (SHARED && j < n)
#pragma unroll
              for (int c = 0; c < 3; ++c) landed[c] = mbar_test(&kc_full[3 * ku + c], kpar);
            if (!(ok = wait(&turn[t], turns))) break;
            turns ^= 1u;
            if (pv) {
              pv_half(0, SHARED ? gv : vu, j > 1 ? 1u : 0u);
              pv_half(1, SHARED ? gv : vu, 1u);
              ++pn;
              if (SHARED) mma_commit(&kv_empty[KS + vu]);  // its slots are K's after next: at once
            }
            if (SHARED) {
              if (j < n && !(ok = qk_chunks(gk, ku, kpar, landed))) break;
            } else if (j < n) {
              qk(ku);
            }
            mbar_arrive(&turn[1 - t]);
            gk += j < nb, gv += j > 0;
            if (j < n) {
              mma_commit(&s_full[t]);
              mma_commit(&kv_empty[ku]);
              if (j == n - 1) mma_commit(&q_empty[t]);
            } else if (j < nb) {
              mbar_arrive(&kv_empty[ku]);
            }
            if (pv) {
              if (!SHARED) mma_commit(&kv_empty[KS + vu]);
              if (j == n) mma_commit(&o_full[t]);
            } else if (j > 0) {
              mbar_arrive(&kv_empty[KS + vu]);
            }
          }
          if (!ok) break;
          if (n > 0) ++qn;
        }
        if (n > 0) ++on;
      }
      // every MMA issued so far has finished before tensor memory is released
      mma_commit(&mma_done[t]);
      mbar_drain(&mma_done[t], 0);
    }
  } else if (warp < 4) {
    regs_dec<C::REGS_CONTROL>();
    if constexpr (!QUANT) {
      // ---------------------------------------------------------- V rows past kv_len -> 0 (one warp)
      if (warp == 2) {
        int nv[2] = {0, 0}, nr = 0;  // V blocks of each reader in the pieces before; ragged blocks
        bool ok = true;
        while (true) {
          const PagedPiece& w = next_piece(ok);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok || w.n_blocks == 0) break;
          const int last = w.n_blocks - 1;  // only the last block can end past kv_len
          const int live = w.sk - (w.jb0 + last) * kBlockK;
          if (live < kBlockK) {
            const int rd = ONE ? last & 1 : 0;
            const int s = rd * VR + (rd ? nv[1] + (last >> 1) : nv[0] + (ONE ? last >> 1 : last)) % VR;
            if (!mbar_wait_warp(&v_ragged[nr % kFixRing], (nr / kFixRing) & 1, abort_flag, p.status)) break;
            ++nr;
            uint8_t* v = sV + s * C::V_BYTES;
            // whole 128-byte rows of every column chunk: the swizzle stays inside a row
            const int g = nv[0] + last;  // shared slots: the block
            for (int u = lane + max(live, 0) * 8; u < kBlockK * 8; u += 32)
#pragma unroll
              for (int c = 0; c < C::NCH_V; ++c)
                *reinterpret_cast<uint4*>(SHARED ? sK + ((5 * g + 3 + (u >> 9)) & 7) * kSlot + c * (kSlot / 2) + (u & 511) * 16
                                                 : v + c * kBlockK * 128 + u * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&kv_full[KS + s]);
          }
          nv[0] += ONE ? w.n_s[0] : w.n_blocks;
          nv[1] += ONE ? w.n_s[1] : 0;
          if (live >= kBlockK) warp_arrive(&passed[2], lane);
        }
      }
    }
  } else if (QUANT && warp < C::SOFTMAX_WARP) {
    // ------------------------------------------------------------ converters: codes -> fp16 operands
    regs_dec<C::REGS_CONVERT>();
    const int row = tid & 127;        // tile row of this thread
    // A bf16 query tile into fp16's range; two buffers of exponents, as the next piece's tile may be
    // converted before this one's softmax has begun.
    auto convert_q = [&](int t, int buf) {
      uint8_t* q = sQ + t * C::Q_BYTES + row * 128;
      float amax = 0.f;
#pragma unroll 4
      for (int u = 0; u < D / 8; ++u) {
        const uint4 v = *reinterpret_cast<const uint4*>(q + (u >> 3) * kBlockQ * 128 + (((u & 7) ^ (row & 7)) << 4));
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16lo_f32(x[i])), fabsf(bf16hi_f32(x[i]))));
      }
      float mul, back;
      q_f16_scale(amax, mul, back);
#pragma unroll 4
      for (int u = 0; u < D / 8; ++u) {
        uint4* ptr = reinterpret_cast<uint4*>(q + (u >> 3) * kBlockQ * 128 + (((u & 7) ^ (row & 7)) << 4));
        const uint4 v = *ptr;
        *ptr = make_uint4(pack_f16x2(bf16lo_f32(v.x) * mul, bf16hi_f32(v.x) * mul),
                          pack_f16x2(bf16lo_f32(v.y) * mul, bf16hi_f32(v.y) * mul),
                          pack_f16x2(bf16lo_f32(v.z) * mul, bf16hi_f32(v.z) * mul),
                          pack_f16x2(bf16lo_f32(v.w) * mul, bf16hi_f32(v.w) * mul));
      }
      // exponent of `back`, in [-126, 113]
      q_exp[(t * 2 + buf) * 128 + row] = static_cast<int8_t>(static_cast<int>(__float_as_uint(back) >> 23) - 127);
      fence_proxy_async_smem();
      warp_arrive(&q_ready[t], lane);
    };
    if constexpr (C::CONVERTERS == 1) {
      // One warpgroup: K(0), then K(j) and V(j-1), the order in which the issuers use them.
      int qn[2] = {0, 0};
      int blk = 0;
      bool ok = true;
      while (true) {
        const PagedPiece& w = next_piece(ok);
        ok = __all_sync(0xffffffffu, ok);
        const int nb = ok ? w.n_blocks : 0;
        if (nb == 0) break;
        const int sk = w.sk, jb0 = w.jb0, kvh = w.kvh;
        const int32_t* table = p.page_table + w.b * p.pt_b;
        // as for two warpgroups (below): exponents one block ahead of their use, scales two, pages three
        // (always loaded, from the first page where there is none: a load under a condition is waited for at once);
        // rows past kv_len or without a page take the factor 0.
        int page2 = 0;
        bool has_page = false, has_scale = false;
        float cur_k = 0.f, cur_v = 0.f, nxt_k = 0.f, nxt_v = 0.f;
        auto fetch_page = [&](int j) {
          const int key = (jb0 + j) * kBlockK + row;
          has_page = j < nb && key < sk;
          page2 = ld_dep(table + (has_page ? key >> p.log2_page : 0));
        };
        auto fetch_scale = [&](int j) {
          has_scale = has_page && page2 >= 0 && page2 < p.n_pages;
          const int64_t at = ((static_cast<int64_t>(has_scale ? page2 : 0) * p.Hkv + kvh) << p.log2_page) +
                             (((jb0 + j) * kBlockK + row) & (p.page_size - 1));
          nxt_k = ld_dep(p.k_scale + at);
          nxt_v = ld_dep(p.v_scale + at);
        };
        auto store_exp = [&](int j) {
          cur_k = has_scale ? nxt_k : 0.f, cur_v = has_scale ? nxt_v : 0.f;
          const int ek = static_cast<int>(__reduce_max_sync(0xffffffffu, __float_as_uint(cur_k)) >> 23);
          const int ev = static_cast<int>(__reduce_max_sync(0xffffffffu, __float_as_uint(cur_v)) >> 23);
          const int be = (blk + j) % kExpRing;
          if (lane == 0) {
            blk_exp[be * 4 + (row >> 5)] = make_int2(ek, ev);
            mbar_arrive(&e_full[be]);
          }
        };
        fetch_page(0);
        fetch_scale(0);
        fetch_page(1);
        if constexpr (CONVERT_Q) {
#pragma unroll 1
          for (int t = 0; t < 2; ++t) {
            if (w.n_s[t] == 0) continue;
            const int n = t ? qn[1]++ : qn[0]++;
            if (!(ok = mbar_wait_warp(&q_full[t], n & 1, abort_flag, p.status))) break;
            convert_q(t, n & 1);
          }
          if (!ok) break;
        }
        store_exp(0);
        fetch_scale(1);
        fetch_page(2);
        uint32_t f_v = 0u;  // factors of V(j-1)
#pragma unroll 1
        for (int j = 0; j <= nb; ++j) {
          uint32_t f[2] = {0u, f_v};
          if (j < nb) {
            const int be = (blk + j) % kExpRing;
            if (!(ok = mbar_wait_warp(&e_full[be], ((blk + j) / kExpRing) & 1, abort_flag, p.status))) break;
            const int2 e = block_exp(blk_exp + be * 4);
            // scale / 2^e, below 2^7: exact in fp16 for power-of-two scales down to 2^-24
            const float rk = cur_k * __uint_as_float(static_cast<uint32_t>(127 - e.x) << 23);
            const float rv = cur_v * __uint_as_float(static_cast<uint32_t>(127 - e.y) << 23);
            f[0] = pack_f16x2(rk, rk);
            f_v = pack_f16x2(rv, rv);
            if (j + 1 < nb) {
              store_exp(j + 1);
              fetch_scale(j + 2);
              fetch_page(j + 3);
            }
          }
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            if (kv == 0 ? j == nb : j == 0) continue;
            const int c = blk + j - kv;
            const int rs = c % NR, ring = kv == 0 ? KR : VR, s = c % ring, at = (kv == 0 ? 0 : KS) + s;
            ok = mbar_wait_warp(&raw_full[kv * NR + rs], (c / NR) & 1, abort_flag, p.status) &&
                 (c < ring || mbar_wait_warp(&kv_empty[at], (c / ring - 1) & 1, abort_flag, p.status));
            if (!ok) break;
            const uint8_t* raw = kv == 0 ? smem + C::OFF_KRAW + rs * C::KRAW : smem + C::OFF_VRAW + rs * C::VRAW;
            uint8_t* dst = kv == 0 ? sK + s * C::K_BYTES : sV + s * C::V_BYTES;
            if (C::KW == C::VW || kv == 1)
              convert_row<C::VW>(raw, dst, kv == 0 ? C::NCH_D : C::NCH_V, row, kv == 0 ? f[0] : f[1]);
            else
              convert_row<C::KW>(raw, dst, C::NCH_D, row, f[0]);
            fence_proxy_async_smem();
            warp_arrive(&kv_full[at], lane);
            if (lane == 0) mbar_arrive(&raw_empty[kv * NR + rs]);
          }
          if (!ok) break;
        }
        if (!ok) break;
        blk += nb;
      }
    } else {
      const int kv = (warp - 4) >> 2;   // 0: K, 1: V
      const float* scale = kv == 0 ? p.k_scale : p.v_scale;
      int qn = 0;
      int blk = 0;                      // blocks of the pieces before this one
      int nc[2] = {0, 0};               // those of each reader
      bool ok = true;
      while (true) {
        const PagedPiece& w = next_piece(ok);
        ok = __all_sync(0xffffffffu, ok);
        const int nb = ok ? w.n_blocks : 0;
        if (nb == 0) break;
        const int sk = w.sk, jb0 = w.jb0, kvh = w.kvh;
        const int32_t* table = p.page_table + w.b * p.pt_b;
        // The scale of this thread's row in each block.  The exponents of a block are stored one block
        // ahead of their use, the scales loaded one ahead of that, and the row's page another one, as
        // the two loads depend on each other.
        int page2 = -1;
        float cur = 0.f, nxt = 0.f;
        auto fetch_page = [&](int j) {
          const int key = (jb0 + j) * kBlockK + row;
          page2 = j < nb && key < sk ? ld_dep(table + (key >> p.log2_page)) : -1;
        };
        auto fetch_scale = [&](int j) {
          nxt = 0.f;  // rows past kv_len or without a page: factor 0
          if (page2 >= 0 && page2 < p.n_pages)
            nxt = ld_dep(scale + ((static_cast<int64_t>(page2) * p.Hkv + kvh) << p.log2_page) +
                         (((jb0 + j) * kBlockK + row) & (p.page_size - 1)));
        };
        auto store_exp = [&](int j) {  // scales are not negative: their bits order like they do
          cur = nxt;
          const int e = static_cast<int>(__reduce_max_sync(0xffffffffu, __float_as_uint(cur)) >> 23);
          const int be = (blk + j) % kExpRing;
          if (lane == 0) {
            reinterpret_cast<int*>(blk_exp + be * 4 + (row >> 5))[kv] = e;
            mbar_arrive(&e_full[kv * kExpRing + be]);
          }
        };
        fetch_page(0);
        fetch_scale(0);
        fetch_page(1);
        if constexpr (CONVERT_Q) {
          const int t = kv;  // the converters of K take query tile 0, those of V tile 1
          if (ONE ? t == 0 : w.n_s[t] > 0) {
            if (!mbar_wait_warp(&q_full[t], qn & 1, abort_flag, p.status)) break;
            convert_q(t, qn & 1);
            ++qn;
          }
        }
        store_exp(0);
        fetch_scale(1);
        fetch_page(2);
#pragma unroll 1
        for (int j = 0; j < nb; ++j) {
          const int be = blk + j;
          const int rs = be % NR;
          const int rd = ONE ? j & 1 : 0;
          const int ring = kv == 0 ? KR : VR, c = ONE ? (rd ? nc[1] : nc[0]) + (j >> 1) : be;
          const int s = rd * ring + c % ring, base = kv == 0 ? 0 : KS;
          ok = mbar_wait_warp(&e_full[kv * kExpRing + be % kExpRing], (be / kExpRing) & 1, abort_flag, p.status);
          if (!ok) break;
          const int2 e = block_exp(blk_exp + be % kExpRing * 4);
          // scale / 2^e, below 2^7: exact in fp16 for power-of-two scales down to 2^-24
          const float r = cur * __uint_as_float(static_cast<uint32_t>(127 - (kv == 0 ? e.x : e.y)) << 23);
          const uint32_t f = pack_f16x2(r, r);
          if (j + 1 < nb) {
            store_exp(j + 1);
            fetch_scale(j + 2);
            fetch_page(j + 3);
          }
          ok = mbar_wait_warp(&raw_full[kv * NR + rs], (be / NR) & 1, abort_flag, p.status) &&
               (c < ring || mbar_wait_warp(&kv_empty[base + s], (c / ring - 1) & 1, abort_flag, p.status));
          if (!ok) break;
          const uint8_t* raw = kv == 0 ? smem + C::OFF_KRAW + rs * C::KRAW : smem + C::OFF_VRAW + rs * C::VRAW;
          uint8_t* dst = kv == 0 ? sK + s * C::K_BYTES : sV + s * C::V_BYTES;
          if (C::KW == C::VW || kv == 1)
            convert_row<C::VW>(raw, dst, kv == 0 ? C::NCH_D : C::NCH_V, row, f);
          else
            convert_row<C::KW>(raw, dst, C::NCH_D, row, f);
          fence_proxy_async_smem();
          warp_arrive(&kv_full[base + s], lane);
          if (lane == 0) mbar_arrive(&raw_empty[kv * NR + rs]);
        }
        if (!ok) break;
        blk += nb;
        nc[0] += (nb + 1) / 2, nc[1] += nb / 2;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    regs_inc<C::REGS_SOFTMAX>();
    const int t = (warp - C::SOFTMAX_WARP) >> 2;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem_base + lane_off + t * 128;
    const uint32_t tO = tmem_base + lane_off + 256 + t * 128;
    // (token, head) of this thread's row
    const int row_tok = static_cast<int>(fast_div(static_cast<uint32_t>(row), p.div_group));
    const int row_head = row - row_tok * p.group;
    int sn = 0, on[2] = {0, 0};  // S blocks of this accumulator; pieces of each
    int qn = 0;                  // loads of its query tile
    int blk = 0, merges = 0;
    bool ok = true;
    while (true) {
      const PagedPiece& w = next_piece(ok);
      ok = __all_sync(0xffffffffu, ok);
      const int nb = ok ? w.n_blocks : 0;
      if (nb == 0) break;
      const int blk0 = blk;
      blk += nb;
      const int n = w.n_s[t], n_other = w.n_s[1 - t];
      const bool merge = ONE && w.n_s[1] > 0;
      const int qt = ONE ? 0 : t;
      const int q_par = qn & 1;
      if (ONE || n > 0) ++qn;
      if (n == 0) {
        if (n_other > 0) ++on[1 - t];
        mbar_arrive(&passed[t]);
        continue;
      }
      const int tok = w.tok0 + qt * p.tok_tile + row_tok;
      const bool row_valid = row_tok < p.tok_tile && tok < w.n;
      // keys this row sees, and those every row of the tile sees
      const int lim_row = p.causal ? min(w.sk, w.len - w.n + tok + 1) : w.sk;
      const int lim_all = p.causal ? min(w.sk, w.len - w.n + w.tok0 + qt * p.tok_tile + 1) : w.sk;
      // a warp without a valid row keeps the barriers going and leaves what tensor memory holds in P:
      // it reaches only O rows that nobody stores
      const bool live = __any_sync(0xffffffffu, row_valid);
      const int jb0 = w.jb0, step = ONE ? 2 : 1, j0 = ONE ? t : 0;  // its blocks: j0 + i * step
      float row_scale2 = p.scale2;
      // Exponents of a block.  Its predecessor in the ring is stored: for the first block of a piece because
      // its scores are there, for the others because those of the block before were.
      int2 exps = make_int2(0, 0);
      auto get_exp = [&](int j) {
        const int be = blk0 + j;
        for (int kv = 0; kv < C::CONVERTERS; ++kv)
          if (!mbar_wait_warp(&e_full[kv * kExpRing + be % kExpRing], (be / kExpRing) & 1, abort_flag, p.status)) return false;
        exps = block_exp(blk_exp + be % kExpRing * 4);
        return true;
      };
      float m_used = -INFINITY;
      float l = 0.f;
      for (int i = 0; i < n; ++i, ++sn) {
        const int j = j0 + i * step;
        if (!mbar_wait_warp(&s_full[t], sn & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        if (!live) {
          warp_arrive(&p_half[t], lane);
          warp_arrive(&p_full[t], lane);
          continue;
        }
        // the query's exponent was stored before q_ready, which the MMAs behind s_full waited for
        if (CONVERT_Q && i == 0)
          row_scale2 *= __uint_as_float(
              static_cast<uint32_t>(127 + static_cast<int>(q_exp[(qt * 2 + q_par) * 128 + row])) << 23);
        if (QUANT && i == 0 && !(ok = get_exp(j))) break;
        const float blk_scale2 =
            QUANT ? fmaxf(row_scale2 * __uint_as_float(static_cast<uint32_t>(127 + exps.x) << 23), kMinBlkScale2) : row_scale2;
        const float shift = static_cast<float>(exps.y);
        const float unshift = __uint_as_float(static_cast<uint32_t>(127 - exps.y) << 23);
        tc_fence_after();
        const int k0 = (jb0 + j) * kBlockK;
        const bool edge = k0 + kBlockK > lim_all;  // the diagonal and the ragged last block hide keys
        const int lim = lim_row - k0;
        if (HELD < kBlockK && edge) {  // in place, once for both readings
#pragma unroll 1
          for (int c = 0; c < kBlockK; c += 32) {
            uint32_t r[32];
            tmem_ld32(tS + c, r);
            tmem_ld_wait();
            reg_fence(r);
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (c + q >= lim) r[q] = 0xFF800000u;
            tmem_st32(tS + c, r);
          }
          tmem_st_wait();
        }
        // The row's 128 scores stay in registers where there are enough.  Beside two warpgroups of
        // converters they are read twice, 64 columns at a time, in loops that are not unrolled.
        uint32_t r[HELD / 32][32];
        auto load = [&](int pass) {
#pragma unroll
          for (int q = 0; q < HELD / 32; ++q) tmem_ld32(tS + pass * HELD + q * 32, r[q]);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < HELD / 32; ++q) reg_fence(r[q]);
          if (HELD == kBlockK && edge) {
#pragma unroll
            for (int c = 0; c < HELD; ++c)
              if (c >= lim) r[c >> 5][c & 31] = 0xFF800000u;
          }
        };
        auto score = [&](int c) { return __uint_as_float(r[c >> 5][c & 31]); };
        float mb = -INFINITY;
#pragma unroll 1
        for (int pass = 0; pass < kBlockK / HELD; ++pass) {
          load(pass);
          float mx[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) mx[q] = fmaxf(score(q), score(8 + q));
#pragma unroll
          for (int gi = 1; gi < HELD / 16; ++gi)
#pragma unroll
            for (int q = 0; q < 8; ++q) mx[q] = fmax3(mx[q], score(16 * gi + q), score(16 * gi + 8 + q));
          mb = fmaxf(mb, fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])));
        }
        const float m_cand = fmaxf(m_used, QUANT ? fmaf(mb, blk_scale2, shift) : mb * blk_scale2);
        // Rows without a token have no say in when the warp rescales: they may be another sequence's queries or, behind
        // the last full token of a tile, what an earlier kernel left in shared memory, and the others' rounding
        // would depend on them.
        const bool need = row_valid && m_cand > m_used + kPagedRescaleLog2;
        const bool rescale = __any_sync(0xffffffffu, need);
        float alpha = 1.f;
        if (rescale) {
          alpha = (m_cand == -INFINITY) ? 1.f : ex2(m_used - m_cand);
          l *= alpha;
          m_used = m_cand;
        }
        // O holds the P.V of the earlier blocks (finished: s_full covers them)
        auto rescale_o = [&]() {
#pragma unroll 1
          for (int c = 0; c < DV / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + c * 32, o);
            tmem_ld_wait();
            reg_fence(o);
#pragma unroll
            for (int q = 0; q < 32; q += 2) {
              float a = __uint_as_float(o[q]), b = __uint_as_float(o[q + 1]);
              fmul2_scalar(a, b, alpha);
              o[q] = __float_as_uint(a);
              o[q + 1] = __float_as_uint(b);
            }
            tmem_st32(tO + c * 32, o);
          }
        };
        // P = 2^(y - m), rounded to 16 bits for the P.V product; the row sum takes the fp32 values.  P
        // goes over the scores in two halves (the first one's columns hold scores that have been read),
        // so that P.V starts on the first.
        const float neg_m = (m_used == -INFINITY) ? 0.f : (QUANT ? shift - m_used : -m_used);
        float ls[4] = {0.f, 0.f, 0.f, 0.f};
        auto half_row = [&](int half, int c0) {  // P of keys 64 half .. + 63, whose scores are held from c0 on
          uint32_t pk[32];
#pragma unroll
          for (int w2 = 0; w2 < 32; ++w2) {
            float x0, x1;
            ffma2_scalar(x0, x1, score(c0 + 2 * w2), score(c0 + 2 * w2 + 1), blk_scale2, neg_m);
            const float p0 = ex2(x0), p1 = ex2(x1);
            pk[w2] = F16_MATH ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
            if (w2 & 1)
              fadd2(ls[2], ls[3], p0, p1);
            else
              fadd2(ls[0], ls[1], p0, p1);
          }
          tmem_st32(tS + half * 32, pk);
        };
        auto publish = [&](uint64_t* bar) {
          tmem_st_wait();
          tc_fence_before();
          warp_arrive(bar, lane);
        };
        if constexpr (HELD < kBlockK) {
          if (rescale && i > 0) rescale_o();
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            load(half);
            half_row(half, 0);
            publish(half == 0 ? &p_half[t] : &p_full[t]);
          }
        } else {
          half_row(0, 0);
          if (rescale && i > 0) rescale_o();
          publish(&p_half[t]);
          half_row(1, 64);
          publish(&p_full[t]);
        }
        const float sum = (ls[0] + ls[1]) + (ls[2] + ls[3]);
        l = QUANT ? fmaf(sum, unshift, l) : l + sum;
        // the next block's, while its scores are on their way
        if (QUANT && i + 1 < n && !(ok = get_exp(j + step))) break;
      }
      if (!ok) break;

      // ---------------------------------------------------------- epilogue: O / l and LSE, or a partial
      if (merge && t == 1) {
        // accumulator 0's warps merge: hand them the max and sum; they read O from tensor memory
        // (o_empty: they have read the piece before)
        if (on[1] > 0 && !mbar_wait_warp(&o_empty[1], (on[1] - 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        ml_x[row] = make_float2(m_used, l);
        warp_arrive(ml_full, lane);
        ++on[0], ++on[1];
        continue;
      }
      if (!mbar_wait_warp(&o_full[t], on[t] & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      float w0 = 1.f, w1 = 0.f;  // weights of this O and, merging, of accumulator 1's
      if (merge) {
        if (!mbar_wait_warp(ml_full, merges & 1, abort_flag, p.status) ||
            !mbar_wait_warp(&o_full[1], on[1] & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        const float2 other = ml_x[row];
        ++merges;
        const float top = fmaxf(m_used, other.x);
        w0 = m_used == -INFINITY ? 0.f : ex2(m_used - top);
        w1 = other.x == -INFINITY ? 0.f : ex2(other.x - top);
        l = l * w0 + other.y * w1;
        m_used = top;
      }
      ++on[t];
      if (n_other > 0) ++on[1 - t];
      tc_fence_after();
      const bool partial = w.slot >= 0;
      // a score of +infinity: where only its product with the scale was, the sum is 0
      if (m_used == INFINITY) l = __uint_as_float(0x7FC00000u);
      const float inv = partial ? 1.f : (l == 0.f ? 0.f : 1.f / l);  // NaN stays NaN
      w0 *= inv, w1 *= inv;
      const int64_t prow = static_cast<int64_t>(w.slot) * p.slot_rows + qt * kBlockQ + row;
      const int head = w.kvh * p.group + row_head;
      const int q_row = w.q_off + tok;
      uint16_t* orow = static_cast<uint16_t*>(p.o) + static_cast<int64_t>(q_row) * p.o_s + static_cast<int64_t>(head) * p.o_h;
#pragma unroll 1
      for (int c = 0; c < (live ? DV / 32 : 0); ++c) {
        uint32_t o[32];
        tmem_ld32(tO + c * 32, o);
        tmem_ld_wait();
        reg_fence(o);
        if (merge) {
          uint32_t o1[32];
          tmem_ld32(tO + 128 + c * 32, o1);
          tmem_ld_wait();
          reg_fence(o1);
#pragma unroll
          for (int q = 0; q < 32; ++q)
            o[q] = __float_as_uint(__uint_as_float(o[q]) * w0 + __uint_as_float(o1[q]) * w1);
        } else if (!partial) {
#pragma unroll
          for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * w0);
        }
        if (row_valid) {
          if (partial) {
            uint4* dst = reinterpret_cast<uint4*>(p.part_o + prow * DV + c * 32);
#pragma unroll
            for (int q = 0; q < 8; ++q) dst[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          } else {
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const float a = __uint_as_float(o[2 * q]), b = __uint_as_float(o[2 * q + 1]);
              pk[q] = BF16 ? pack_bf16x2(a, b) : pack_f16x2(a, b);
            }
            uint4* dst = reinterpret_cast<uint4*>(orow + c * 32);
#pragma unroll
            for (int q = 0; q < 4; ++q) dst[q] = make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      warp_arrive(&o_empty[t], lane);
      if (merge && lane == 0) mbar_arrive(&o_empty[1]);
      if (row_valid) {
        if (partial)
          *reinterpret_cast<float2*>(p.part_ml + prow * 2) = make_float2(m_used, l);
        else if (p.lse != nullptr)
          p.lse[static_cast<int64_t>(head) * p.total_q + q_row] = l == 0.f ? -INFINITY : (m_used + lg2(l)) * kPagedLn2;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Launches the kernel, one CTA per SM: as a programmatic dependent of the plan kernel, if there is one.
template <bool BF16, bool QUANT, int D, int DV, bool ONE, bool PACKED>
cudaError_t launch_paged_one(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tr,
                             const PagedParams& p, cudaStream_t st) {
  using C = PagedCfg<QUANT, D, DV, ONE>;
  auto kern = paged_kernel<BF16, QUANT, D, DV, ONE, PACKED>;
  int dev = 0, sms = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> opted{0};
  if ((e = smem_opt_in(kern, C::SMEM, dev, opted)) != cudaSuccess) return e;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.sms));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = p.inline_plan ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, tr, p);
}

template <bool BF16, bool QUANT, int D, int DV>
cudaError_t launch_paged_instance(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                  const PagedParams& p, cudaStream_t st) {
  if constexpr (!(QUANT && D == 192))  // as paged_choose has it
    if (p.one) return launch_paged_one<BF16, QUANT, D, DV, true, false>(tq, tk, tv, tv, p, st);
  return launch_paged_one<BF16, QUANT, D, DV, false, false>(tq, tk, tv, tv, p, st);
}

}  // namespace sdpa
