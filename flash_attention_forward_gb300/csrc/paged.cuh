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
// K and V blocks take turns in one ring of equal slots, in the order of their use: K(0), then K(j) and
// V(j-1) for each j, then the last V.  A slot is so held for little longer than its MMAs take, and the
// rest of the ring is loads in flight.
//
// Quantised pages.  Every e4m3 value is exact in fp16, so four converter warps turn a block's codes
// into fp16 operands (one thread per row) and both products are fp16, whatever the query's type:
//   * K' = code * (k_scale / 2^ek), 2^(ek + 6) the power of two of the block's largest scale: the
//     largest row lies just below fp16's largest value, rows of power-of-two scales stay exact down
//     to 2^-21 of the largest scale and lose a bit for each one below (K' is read as 0 under
//     2^-30).  The block's scores are multiplied by 2^ek;
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

// ONE: no sequence has more tokens than one query tile holds, so shared memory keeps one and the ring
// takes the other's place (such calls are bound by reading the cache).
template <bool QUANT, int D, int DV, bool ONE>
struct PagedCfg {
  static constexpr int NCH_D = D / 64, NCH_V = DV / 64;
  static constexpr int Q_BYTES = kBlockQ * D * 2;
  static constexpr int K_BYTES = kBlockK * D * 2;
  static constexpr int V_BYTES = kBlockK * DV * 2;
  static constexpr int SLOT = K_BYTES > V_BYTES ? K_BYTES : V_BYTES;
  static constexpr int Q_TILES = ONE ? 1 : 2;
  static constexpr int SLOTS = D == 64 ? 8 : D == 128 ? (QUANT ? 4 : ONE ? 6 : 5) : (ONE && !QUANT ? 3 : 2);
  // raw codes: boxes of 128 (or 64) codes a row
  static constexpr int KW = D % 128 == 0 ? 128 : 64, VW = DV % 128 == 0 ? 128 : 64;
  static constexpr int RAW = QUANT ? kBlockK * D : 0;
  static constexpr int RAWS = !QUANT ? 0 : D == 64 ? 6 : D == 128 ? (ONE ? 4 : 2) : (ONE ? 3 : 1);
  static constexpr int QK_STEPS = D / 16, PV_STEPS = kBlockK / 16;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_SLOT = OFF_Q + Q_TILES * Q_BYTES;
  static constexpr int OFF_RAW = OFF_SLOT + SLOTS * SLOT;
  static constexpr int OFF_BAR = OFF_RAW + RAWS * RAW;
  static constexpr int BARS = D == 64 ? 768 : 640;
  static constexpr int OFF_EXP = OFF_BAR + BARS;                    // int2 [kExpRing][4]
  static constexpr int OFF_QEXP = OFF_EXP + (QUANT ? kExpRing * 32 : 0);  // int8 [2 tiles][2][128]
  // pieces announced by the producer: more than it can run ahead of the slowest role.  With m pieces behind
  // the one whose V is used up, 2 m - 1 items lie in the rings (each piece's V waits for its softmax).
  static constexpr int PIECES = D == 64 ? 16 : 8;
  static constexpr int OFF_PIECE = OFF_QEXP + (QUANT ? 512 : 0);
  static constexpr int OFF_ML = OFF_PIECE + PIECES * 64;            // float2 [128]: max and sum of slot 1
  static constexpr int SMEM = OFF_ML + 1024;
  static_assert(SLOTS / 2 + 3 <= kExpRing, "the exponent ring holds what the converters write");
  static_assert((SLOTS + RAWS) / 2 + 2 <= PIECES, "the piece ring holds what the producer announces");
  // warpgroups: control (producer, MMA, helpers), converters (quantised), two softmax
  static constexpr int THREADS = QUANT ? 512 : 384;
  static constexpr int SOFTMAX_WARP = QUANT ? 8 : 4;
  // registers per thread; the sums must stay within what the block is launched with
  static constexpr uint32_t REGS_CONTROL = QUANT ? 64 : 96;
  static constexpr uint32_t REGS_CONVERT = 64;
  static constexpr uint32_t REGS_SOFTMAX = QUANT ? 192 : 200;
  static constexpr uint32_t REGS_LAUNCH = QUANT ? 128 : 168;
  static_assert(128 * REGS_CONTROL + (QUANT ? 128 * REGS_CONVERT : 0) + 256 * REGS_SOFTMAX <= THREADS * REGS_LAUNCH,
                "register split exceeds the launch");
  static_assert(SMEM <= 227 * 1024, "more shared memory than a CTA may opt in to");
  static_assert(Q_BYTES % 1024 == 0 && SLOT % 1024 == 0 && RAW % 1024 == 0, "1 KB tile alignment");
};

// One piece of a work unit: two query tiles (2 * tok_tile tokens of one sequence, the G heads of one KV
// head) against the key blocks [jb0, jb0 + n_blocks).  There are two S / O accumulators ("slots").
// Normally slot t serves query tile t, and both read every block.  A unit whose tokens all lie in tile
// 0 ("alternating") gives the even blocks to slot 0 and the odd ones to slot 1, so that one slot's
// softmax runs beside the other's MMAs there too; slot 0's warps merge the two at the end.
struct PagedPiece {
  int b, kvh, tok0, jb0;
  int n_blocks;            // 0: no more pieces
  int n_s[2];              // blocks of each slot
  int slot;                // partial slot, or -1: the whole unit, which stores O itself
  int q_off, n, len, sk;
  int alt;                 // alternating
  int pad[3];
};
static_assert(sizeof(PagedPiece) == 64, "the producer announces a piece in 64 bytes");

// The pieces of this CTA's stretch of the line, in order (the producer's walk; the other roles read
// what it announces).
struct PagedWalk {
  int tile, kvh, off, first;
  int4 end;

  __device__ __forceinline__ explicit PagedWalk(const PagedParams& p) : first(1) {
    const int n = ld_dep(&p.plan.head->n_ctas);
    int4 c = make_int4(0, 0, 0, 0);
    end = c;
    if (static_cast<int>(blockIdx.x) < n) {
      c = ld_dep(p.plan.cuts + blockIdx.x);
      end = ld_dep(p.plan.cuts + blockIdx.x + 1);
    }
    tile = c.x, kvh = c.y, off = c.z;
  }
  __device__ __forceinline__ PagedPiece next(const PagedParams& p) {
    PagedPiece w{};
    if (!(tile < end.x || (tile == end.x && (kvh < end.y || (kvh == end.y && off < end.z))))) return w;
    const int2 at = ld_dep(p.plan.tiles + tile);
    w.b = at.x;
    w.kvh = kvh;
    w.q_off = __ldg(p.cu_q + w.b);
    w.n = __ldg(p.cu_q + w.b + 1) - w.q_off;
    w.len = __ldg(p.kv_len + w.b);
    w.sk = min(max(w.len, 0), p.max_kv);
    w.tok0 = at.y * kTilesPerCta * p.tok_tile;
    w.jb0 = off;
    int blocks[kTilesPerCta];
#pragma unroll
    for (int t = 0; t < kTilesPerCta; ++t)
      blocks[t] = paged_tile_blocks(w.n, w.len, w.sk, p.tok_tile, p.causal, at.y * kTilesPerCta + t);
    const int all = max(blocks[0], blocks[1]);
    const int stop = (tile == end.x && kvh == end.y) ? end.z : all;
    w.n_blocks = stop - off;
    w.alt = blocks[1] == 0;
#pragma unroll
    for (int t = 0; t < 2; ++t)
      w.n_s[t] = w.alt ? (w.n_blocks + 1 - t) / 2 : min(max(blocks[t] - off, 0), w.n_blocks);
    w.slot = (off > 0 || stop < all) ? 2 * static_cast<int>(blockIdx.x) + 1 - first : -1;
    first = 0;
    off = 0;
    if (++kvh == p.Hkv) kvh = 0, ++tile;
    return w;
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
// instruction cache (unrolled for K and V, fetches stalled 2 of 10 resident warps and the softmax took twice
// as long; 2048 tokens of 8192 rows 284 us against 217 us).
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

// Barriers (phases continue from piece to piece; the arrivals of warps are one each):
//   piece[i % PIECES]     : the producer announced piece i
//   q_full[t] / q_empty[t]: Q tile t landed / its last QK MMA finished (q_empty[2]: slot 1's last one
//                           on tile 0 in an alternating piece)
//   q_ready[t]            : quantised pages and a bf16 query: tile t converted to fp16
//   full[s] / empty[s]    : ring slot s holds its item / both issuers are done with it
//   raw_full / raw_empty  : quantised pages: codes landed / read by the converters
//   e_full[i % 8]         : quantised pages: each converter warp has stored the exponents of its 32
//                           rows of block i (the block's are the largest of the four)
//   turn[t]               : issuer t may issue (both tiles active)
//   v_ragged[i % 8]       : 16-bit pages: the i-th V block that ends past kv_len landed; a helper warp
//                           then zeroes those rows and completes full[s] in the copy's place
//   s_full[t], p_half[t], p_full[t], o_full[t], o_empty[t]: as in the prefill kernels, per slot
//   ml_full               : alternating pieces: slot 1's max and sum are there
template <bool BF16, bool QUANT, int D, int DV, bool ONE>
__global__ void __launch_bounds__(PagedCfg<QUANT, D, DV, ONE>::THREADS, 1)
    paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const PagedParams p) {
  using C = PagedCfg<QUANT, D, DV, ONE>;
  constexpr int NS = C::SLOTS;
  constexpr int NR = C::RAWS > 0 ? C::RAWS : 1;
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
  uint8_t* sKV = smem + C::OFF_SLOT;
  uint8_t* sRaw = smem + C::OFF_RAW;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars;              // [2]
  uint64_t* q_empty = q_full + 2;       // [3]
  uint64_t* q_ready = q_empty + 3;      // [2]
  uint64_t* s_full = q_ready + 2;       // [2]
  uint64_t* p_half = s_full + 2;        // [2]
  uint64_t* p_full = p_half + 2;        // [2]
  uint64_t* o_full = p_full + 2;        // [2]
  uint64_t* o_empty = o_full + 2;       // [2]
  uint64_t* mma_done = o_empty + 2;     // [2]
  uint64_t* turn = mma_done + 2;        // [2]
  uint64_t* v_ragged = turn + 2;        // [kFixRing]
  uint64_t* full = v_ragged + kFixRing;  // [NS]
  uint64_t* empty = full + NS;          // [NS]
  uint64_t* raw_full = empty + NS;      // [NR]
  uint64_t* raw_empty = raw_full + NR;  // [NR]
  uint64_t* e_full = raw_empty + NR;    // [kExpRing]
  uint64_t* piece = e_full + kExpRing;  // [PIECES]
  uint64_t* ml_full = piece + C::PIECES;  // [1]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ml_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int2* blk_exp = reinterpret_cast<int2*>(smem + C::OFF_EXP);
  int8_t* q_exp = reinterpret_cast<int8_t*>(smem + C::OFF_QEXP);
  PagedPiece* pieces = reinterpret_cast<PagedPiece*>(smem + C::OFF_PIECE);
  float2* ml_x = reinterpret_cast<float2*>(smem + C::OFF_ML);  // [128]
  static_assert((22 + kFixRing + kExpRing + 2 * NS + 2 * NR + C::PIECES) * 8 + 8 <= C::BARS, "barriers fit their area");

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
    for (int t = 0; t < 3; ++t) mbar_init(&q_empty[t], 1);
    for (int s = 0; s < kFixRing; ++s) mbar_init(&v_ragged[s], 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], QUANT ? 4 : 1);
      mbar_init(&empty[s], 2);
    }
    for (int s = 0; s < kExpRing; ++s) mbar_init(&e_full[s], 4);
    for (int s = 0; s < NR; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    for (int s = 0; s < C::PIECES; ++s) mbar_init(&piece[s], 1);
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
  pdl_wait();  // the plan comes from the kernel launched before
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
    }
    const int rows = min(kBlockK, p.page_size);  // rows per box
    const int nsub = kBlockK / rows;             // boxes per column chunk: 1 .. 8
    constexpr int KPARTS = QUANT ? D / C::KW : C::NCH_D, VPARTS = QUANT ? DV / C::VW : C::NCH_V;
    constexpr int KCOLS = QUANT ? C::KW : 64, VCOLS = QUANT ? C::VW : 64;    // columns per box
    constexpr int KROW = QUANT ? C::KW : 128, VROW = QUANT ? C::VW : 128;    // bytes of a box row
    constexpr int KTX = QUANT ? kBlockK * D : C::K_BYTES, VTX = QUANT ? kBlockK * DV : C::V_BYTES;
    constexpr int NL = QUANT ? NR : NS;          // ring that TMA fills
    uint64_t* ld_full = QUANT ? raw_full : full;
    uint64_t* ld_empty = QUANT ? raw_empty : empty;
    const int q_tx = p.tok_tile * p.group * D * 2;
    PagedWalk walk(p);
    int qn[2] = {0, 0}, alts = 0;
    bool last_alt = false;  // tile 0's last piece was alternating, with blocks for slot 1
    int g = 0, nr = 0;      // items, and ragged V blocks, issued
    bool ok = true;
    while (ok) {
      const PagedPiece w = walk.next(p);
      if (lane == 0) {
        pieces[n_piece % C::PIECES] = w;
        mbar_arrive(&piece[n_piece % C::PIECES]);
      }
      ++n_piece;
      if (w.n_blocks == 0) break;
      for (int t = 0; t < kTilesPerCta && ok; ++t) {
        if (t == 0 ? w.n_s[0] == 0 : (w.alt || w.n_s[1] == 0)) continue;
        if ((qn[t] > 0 && !mbar_wait_warp(&q_empty[t], (qn[t] - 1) & 1, abort_flag, p.status)) ||
            (t == 0 && last_alt && !mbar_wait_warp(&q_empty[2], (alts - 1) & 1, abort_flag, p.status))) {
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
        if (t == 0) {
          last_alt = w.alt && w.n_s[1] > 0;
          alts += last_alt;
        }
      }
      const int32_t* table = p.page_table + w.b * p.pt_b;
      const int used = (w.sk + p.page_size - 1) >> p.log2_page;  // pages that hold visible rows
      const int sub = lane & 7;                                  // page of the block: lane % 8 < nsub
      int phys_k = p.n_pages, row_k = 0;  // page and row of this lane's box; outside the pool: zeros
      for (int j = 0; ok && j <= w.n_blocks; ++j) {
        const int phys_v = phys_k, row_v = row_k;
        if (j < w.n_blocks) {
          const int key = (w.jb0 + j) * kBlockK + sub * rows;
          const int lp = key >> p.log2_page;
          row_k = key & (p.page_size - 1);
          phys_k = p.n_pages;
          if (sub < nsub && lp < used) phys_k = __ldg(table + lp);
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (kv == 0 ? j == w.n_blocks : j == 0) continue;  // K(j), then V(j-1)
          const int s = g % NL, r = g / NL;
          if (r > 0 && !mbar_wait_warp(&ld_empty[s], (r - 1) & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          if (p.stall_first_stage && g == 0) {  // test hook: slot 0 never fills
            ++g;
            continue;
          }
          uint64_t* bar = &ld_full[s];
          if (!QUANT && kv == 1 && (w.jb0 + j) * kBlockK > w.sk) {
            bar = &v_ragged[nr % kFixRing];
            ++nr;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar, kv == 0 ? KTX : VTX);
          __syncwarp();
          uint8_t* dst = QUANT ? sRaw + s * C::RAW : sKV + s * C::SLOT;
          const int parts = kv == 0 ? KPARTS : VPARTS, row_b = kv == 0 ? KROW : VROW;
          const int part = lane >> 3;  // column chunk
          if (sub < nsub && part < parts)
            tma_load_4d(dst + part * kBlockK * row_b + sub * rows * row_b, kv == 0 ? &tm_k : &tm_v, bar,
                        part * (kv == 0 ? KCOLS : VCOLS), w.kvh, kv == 0 ? row_k : row_v, kv == 0 ? phys_k : phys_v);
          ++g;
        }
      }
    }
    if (!ok && lane == 0) {
      // let every copy already in flight land before the CTA's shared memory goes away
      for (int t = 0; t < kTilesPerCta; ++t)
        if (qn[t] > 0) mbar_drain(&q_full[t], (qn[t] - 1) & 1);
      for (int j = max(0, nr - kFixRing); j < nr; ++j) mbar_drain(&v_ragged[j % kFixRing], (j / kFixRing) & 1);
      for (int j = max(0, g - NL); j < g; ++j) mbar_drain(&ld_full[j % NL], (j / NL) & 1);
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
      const uint64_t dk0 = make_smem_desc(smem_u32(sKV), 16, 1024, kSwizzle128B);
      const uint64_t dv0 = make_smem_desc(smem_u32(sKV), kBlockK * 128, 1024, kSwizzle128B);
      const uint32_t q_lo = static_cast<uint32_t>(dq0), q_hi = static_cast<uint32_t>(dq0 >> 32);
      const uint32_t k_lo = static_cast<uint32_t>(dk0), k_hi = static_cast<uint32_t>(dk0 >> 32);
      const uint32_t v_lo = static_cast<uint32_t>(dv0), v_hi = static_cast<uint32_t>(dv0 >> 32);
      const uint32_t tS = tmem_base + t * 128;
      const uint32_t tO = tmem_base + 256 + t * 128;
      int qn[2] = {0, 0};         // Q tiles loaded so far
      int on = 0, pn = 0;         // pieces and blocks of this slot so far
      uint32_t turns = 1 - t;     // parity of the turn barrier's next phase; tile 0 begins
      int s = 0;                  // ring slot of the next item and the parity of its phase
      uint32_t ph = 0;
      bool ok = true;
      auto next = [&]() {
        if (++s == NS) s = 0, ph ^= 1u;
      };
      while (true) {
        const PagedPiece& w = next_piece(ok);
        const int nb = ok ? w.n_blocks : 0;
        if (nb == 0) break;
        const int n = w.n_s[t];
        const bool alt = w.alt != 0, both = !alt && w.n_s[0] > 0 && w.n_s[1] > 0;
        const int qt = alt ? 0 : t;  // query tile of this slot
        if (n > 0) ok = mbar_wait(CONVERT_Q ? &q_ready[qt] : &q_full[qt], qn[qt] & 1, abort_flag, p.status);
        if (w.n_s[0] > 0) ++qn[0];
        if (!alt && w.n_s[1] > 0) ++qn[1];
        const uint32_t dq = q_lo + static_cast<uint32_t>((qt * C::Q_BYTES) >> 4);
        // Step j takes K(j) and V(j-1) from the ring: O += P(j-1) V(j-1), then S = Q K(j)^T.  In an
        // alternating piece block j is this slot's if j % 2 == t, and S = Q K(j)^T follows
        // O += P(j-2) V(j-2).  An item that this slot does not read is seen and passed on.
        int vs = 0;  // slot of the V to be used next
        for (int j = 0; ok && j <= nb + (alt ? 1 : 0); ++j) {
          const bool qk = alt ? j < nb && (j & 1) == t : j < n;
          const bool pv = alt ? j >= 2 && (j & 1) == t : j >= 1 && j <= n;
          const int ks = s;
          if (j < nb) {
            if (!mbar_wait(&full[ks], ph, abort_flag, p.status)) {
              ok = false;
              break;
            }
            if (!qk) mbar_arrive(&empty[ks]);
            next();
          }
          const bool v_here = j >= 1 && j <= nb;
          if (v_here && !alt) {
            vs = s;
            if (!mbar_wait(&full[vs], ph, abort_flag, p.status)) {
              ok = false;
              break;
            }
            if (!pv) mbar_arrive(&empty[vs]);
            next();
          }
          if (pv) {
            if ((alt ? j < 4 : j == 1) && on > 0 && !mbar_wait(&o_empty[t], (on - 1) & 1, abort_flag, p.status)) {
              ok = false;
              break;
            }
            if (!mbar_wait(&p_half[t], pn & 1, abort_flag, p.status) ||
                (both && !mbar_wait(&p_full[t], pn & 1, abort_flag, p.status))) {
              ok = false;
              break;
            }
          }
          if (both) {
            if (!mbar_wait(&turn[t], turns, abort_flag, p.status)) {
              ok = false;
              break;
            }
            turns ^= 1u;
          }
          if (pv) {
            const uint32_t dv = v_lo + static_cast<uint32_t>((vs * C::SLOT) >> 4);
            const uint32_t acc0 = (alt ? j >= 4 : j > 1) ? 1u : 0u;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < C::PV_STEPS / 2; ++kk)
              mma_f16_ts(tO, tS + kk * 8, dv + static_cast<uint32_t>((kk * 16 * 128) >> 4), v_hi, idesc_pv,
                         kk > 0 ? 1u : acc0);
            // without turns, P.V starts on the first half of P while the second is computed
            if (!both) {
              if (!mbar_wait(&p_full[t], pn & 1, abort_flag, p.status)) {
                ok = false;
                break;
              }
              tc_fence_after();
            }
#pragma unroll
            for (int kk = C::PV_STEPS / 2; kk < C::PV_STEPS; ++kk)
              mma_f16_ts(tO, tS + kk * 8, dv + static_cast<uint32_t>((kk * 16 * 128) >> 4), v_hi, idesc_pv, 1u);
            ++pn;
            if (!both) mma_commit(&empty[vs]);
          }
          if (qk) {
            tc_fence_after();
            const uint32_t dk = k_lo + static_cast<uint32_t>((ks * C::SLOT) >> 4);
#pragma unroll
            for (int kk = 0; kk < C::QK_STEPS; ++kk) {
              const uint32_t off = static_cast<uint32_t>(((kk / 4) * kBlockQ * 128 + (kk % 4) * 32) >> 4);
              mma_f16_ss(tS, dq + off, q_hi, dk + off, k_hi, idesc_qk, kk > 0 ? 1u : 0u);
            }
          }
          if (both) mbar_arrive(&turn[1 - t]);
          if (qk) {
            mma_commit(&s_full[t]);
            mma_commit(&empty[ks]);
          }
          if (pv && both) mma_commit(&empty[vs]);
          if (pv && (alt ? j >= nb : j == n)) mma_commit(&o_full[t]);
          if (qk && (alt ? j + 2 >= nb : j == n - 1)) mma_commit(&q_empty[alt && t == 1 ? 2 : t]);
          if (v_here && alt) {  // V(j-1), behind this step's MMAs
            if (!mbar_wait(&full[s], ph, abort_flag, p.status)) {
              ok = false;
              break;
            }
            if (((j - 1) & 1) == t)
              vs = s;
            else
              mbar_arrive(&empty[s]);
            next();
          }
        }
        if (!ok) break;
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
        int g = 0, nr = 0;
        bool ok = true;
        while (true) {
          const PagedPiece& w = next_piece(ok);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok || w.n_blocks == 0) break;
          const int last = w.n_blocks - 1;  // only the last block can end past kv_len
          const int live = w.sk - (w.jb0 + last) * kBlockK;
          if (live < kBlockK) {
            const int s = (g + 2 * last + 1) % NS;
            if (!mbar_wait_warp(&v_ragged[nr % kFixRing], (nr / kFixRing) & 1, abort_flag, p.status)) break;
            ++nr;
            uint8_t* v = sKV + s * C::SLOT;
            // whole 128-byte rows of every column chunk: the swizzle stays inside a row
            for (int u = lane + max(live, 0) * 8; u < kBlockK * 8; u += 32)
#pragma unroll
              for (int c = 0; c < C::NCH_V; ++c)
                *reinterpret_cast<uint4*>(v + c * kBlockK * 128 + u * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
          }
          g += 2 * w.n_blocks;
        }
      }
    }
  } else if (QUANT && warp < 8) {
    // ------------------------------------------------------------ converters: codes -> fp16 operands
    regs_dec<C::REGS_CONVERT>();
    const int row = tid - 128;  // tile row of this thread
    int qn[2] = {0, 0};
    int g = 0, blk = 0;
    bool ok = true;
    while (true) {
      const PagedPiece& w = next_piece(ok);
      ok = __all_sync(0xffffffffu, ok);
      const int nb = ok ? w.n_blocks : 0;
      if (nb == 0) break;
      const int sk = w.sk, jb0 = w.jb0, kvh = w.kvh;
      if constexpr (CONVERT_Q) {
        for (int t = 0; t < kTilesPerCta && ok; ++t) {
          if (t == 0 ? w.n_s[0] == 0 : (w.alt || w.n_s[1] == 0)) continue;
          if (!mbar_wait_warp(&q_full[t], qn[t] & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
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
          // exponent of `back`, in [-126, 113]; two buffers, as the next unit's tile may be converted
          // before this one's softmax has begun
          q_exp[(t * 2 + (qn[t] & 1)) * 128 + row] =
              static_cast<int8_t>(static_cast<int>(__float_as_uint(back) >> 23) - 127);
          fence_proxy_async_smem();
          warp_arrive(&q_ready[t], lane);
          ++qn[t];
        }
        if (!ok) break;
      }
      const int32_t* table = p.page_table + w.b * p.pt_b;
      // Each thread's row has a scale of K and one of V per block.  The exponents of a block are stored
      // one block ahead of their use, the scales loaded one ahead of that, and the row's page another
      // one, as the two loads depend on each other.
      int page2 = -1;
      float2 cur = make_float2(0.f, 0.f), nxt = cur;  // scales of K and V
      auto fetch_page = [&](int j) {
        const int key = (jb0 + j) * kBlockK + row;
        page2 = j < nb && key < sk ? ld_dep(table + (key >> p.log2_page)) : -1;
      };
      auto fetch_scales = [&](int j) {
        nxt = make_float2(0.f, 0.f);  // rows past kv_len or without a page: factor 0
        if (page2 >= 0 && page2 < p.n_pages) {
          const int64_t at = ((static_cast<int64_t>(page2) * p.Hkv + kvh) << p.log2_page) +
                             (((jb0 + j) * kBlockK + row) & (p.page_size - 1));
          nxt = make_float2(ld_dep(p.k_scale + at), ld_dep(p.v_scale + at));
        }
      };
      auto store_exps = [&](int j) {  // scales are not negative: their bits order like they do
        cur = nxt;
        const int ek = static_cast<int>(__reduce_max_sync(0xffffffffu, __float_as_uint(cur.x)) >> 23);
        const int ev = static_cast<int>(__reduce_max_sync(0xffffffffu, __float_as_uint(cur.y)) >> 23);
        const int be = (blk + j) % kExpRing;
        if (lane == 0) {
          blk_exp[be * 4 + (row >> 5)] = make_int2(ek, ev);
          mbar_arrive(&e_full[be]);
        }
      };
      fetch_page(0);
      fetch_scales(0);
      fetch_page(1);
      store_exps(0);
      fetch_scales(1);
      fetch_page(2);
      uint32_t f_v = 0;  // factor of this thread's V row, one step behind
      for (int j = 0; ok && j <= nb; ++j) {
        const uint32_t f_prev = f_v;
        uint32_t f_k = 0;
        if (j < nb) {
          const int be = blk + j;
          if (!mbar_wait_warp(&e_full[be % kExpRing], (be / kExpRing) & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const int2 e = block_exp(blk_exp + be % kExpRing * 4);
          // scale / 2^e, below 2^7: exact in fp16 for power-of-two scales down to 2^-24
          const float rk = cur.x * __uint_as_float(static_cast<uint32_t>(127 - e.x) << 23);
          const float rv = cur.y * __uint_as_float(static_cast<uint32_t>(127 - e.y) << 23);
          f_k = pack_f16x2(rk, rk), f_v = pack_f16x2(rv, rv);
          if (j + 1 < nb) {
            store_exps(j + 1);
            fetch_scales(j + 2);
            fetch_page(j + 3);
          }
        }
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          if (kv == 0 ? j == nb : j == 0) continue;  // K(j), then V(j-1)
          const int rs = g % NR, s = g % NS;
          if (!mbar_wait_warp(&raw_full[rs], (g / NR) & 1, abort_flag, p.status) ||
              (g >= NS && !mbar_wait_warp(&empty[s], (g / NS - 1) & 1, abort_flag, p.status))) {
            ok = false;
            break;
          }
          ++g;
          const uint8_t* raw = sRaw + rs * C::RAW;
          uint8_t* dst = sKV + s * C::SLOT;
          if (C::KW == C::VW)
            convert_row<C::KW>(raw, dst, kv == 0 ? C::NCH_D : C::NCH_V, row, kv == 0 ? f_k : f_prev);
          else if (kv == 0)
            convert_row<C::KW>(raw, dst, C::NCH_D, row, f_k);
          else
            convert_row<C::VW>(raw, dst, C::NCH_V, row, f_prev);
          fence_proxy_async_smem();
          warp_arrive(&full[s], lane);
          if (lane == 0) mbar_arrive(&raw_empty[rs]);
        }
      }
      if (!ok) break;
      blk += nb;
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
    int sn = 0, on[2] = {0, 0};  // S blocks of this slot; pieces of each slot
    int qn[2] = {0, 0};          // Q tiles loaded
    int blk = 0, alts = 0;
    bool ok = true;
    while (true) {
      const PagedPiece& w = next_piece(ok);
      ok = __all_sync(0xffffffffu, ok);
      const int nb = ok ? w.n_blocks : 0;
      if (nb == 0) break;
      const int blk0 = blk;
      blk += nb;
      const int n = w.n_s[t], n_other = w.n_s[1 - t];
      const bool alt = w.alt != 0, merge = alt && w.n_s[1] > 0;
      const int qt = alt ? 0 : t;
      const int q_par = qn[qt] & 1;
      if (w.n_s[0] > 0) ++qn[0];
      if (!alt && w.n_s[1] > 0) ++qn[1];
      if (n == 0) {
        if (n_other > 0) ++on[1 - t];
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
      const int jb0 = w.jb0, step = alt ? 2 : 1, j0 = alt ? t : 0;  // this slot's blocks: j0 + i * step
      float row_scale2 = p.scale2;
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
        float blk_scale2 = row_scale2, shift = 0.f, unshift = 1.f;
        if constexpr (QUANT) {
          const int be = blk0 + j;
          if (!mbar_wait_warp(&e_full[be % kExpRing], (be / kExpRing) & 1, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const int2 e = block_exp(blk_exp + be % kExpRing * 4);
          blk_scale2 = fmaxf(blk_scale2 * __uint_as_float(static_cast<uint32_t>(127 + e.x) << 23), kMinBlkScale2);
          shift = static_cast<float>(e.y);
          unshift = __uint_as_float(static_cast<uint32_t>(127 - e.y) << 23);
        }
        tc_fence_after();
        const int k0 = (jb0 + j) * kBlockK;
        const bool edge = k0 + kBlockK > lim_all;  // the diagonal and the ragged last block hide keys
        const int lim = lim_row - k0;
        if (QUANT && edge) {  // in place, once for both readings
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
        // 16-bit pages: the row's 128 scores stay in registers.  Quantised pages: they are read twice,
        // 64 columns at a time, in loops that are not unrolled (see convert_row on the instruction
        // cache; measured 263 -> 245 us there, and 2412 -> 2582 us for 16-bit pages, which keep the short way).
        constexpr int HELD = QUANT ? 64 : kBlockK;
        uint32_t r[HELD / 32][32];
        auto load = [&](int pass) {
#pragma unroll
          for (int q = 0; q < HELD / 32; ++q) tmem_ld32(tS + pass * HELD + q * 32, r[q]);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < HELD / 32; ++q) reg_fence(r[q]);
          if (!QUANT && edge) {
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
        const bool need = m_cand > m_used + kPagedRescaleLog2;
        const bool rescale = __any_sync(0xffffffffu, need);
        float alpha = 1.f;
        if (rescale) {
          alpha = (m_cand == -INFINITY) ? 1.f : ex2(m_used - m_cand);
          l *= alpha;
          m_used = m_cand;
        }
        // O holds the P.V of this slot's earlier blocks (finished: s_full covers them)
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
        if constexpr (QUANT) {
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
      }
      if (!ok) break;

      // ---------------------------------------------------------- epilogue: O / l and LSE, or a partial
      if (merge && t == 1) {
        // slot 0's warps merge: hand them this slot's max and sum; they read O from tensor memory
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
      float w0 = 1.f, w1 = 0.f;  // weights of this slot's O and, merging, of slot 1's
      if (merge) {
        if (!mbar_wait_warp(ml_full, alts & 1, abort_flag, p.status) ||
            !mbar_wait_warp(&o_full[1], on[1] & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        const float2 other = ml_x[row];
        ++alts;
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
      const float inv = partial ? 1.f : (l > 0.f ? 1.f / l : 0.f);
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
          p.lse[static_cast<int64_t>(head) * p.total_q + q_row] = l > 0.f ? (m_used + lg2(l)) * kPagedLn2 : -INFINITY;
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

// Launches the kernel as a programmatic dependent of the plan kernel, one CTA per SM.
template <bool BF16, bool QUANT, int D, int DV, bool ONE>
cudaError_t launch_paged_one(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p,
                             cudaStream_t st) {
  using C = PagedCfg<QUANT, D, DV, ONE>;
  auto kern = paged_kernel<BF16, QUANT, D, DV, ONE>;
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
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, p);
}

template <bool BF16, bool QUANT, int D, int DV>
cudaError_t launch_paged_instance(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                  const PagedParams& p, cudaStream_t st) {
  return p.max_seqlen_q <= p.tok_tile ? launch_paged_one<BF16, QUANT, D, DV, true>(tq, tk, tv, p, st)
                                      : launch_paged_one<BF16, QUANT, D, DV, false>(tq, tk, tv, p, st);
}

}  // namespace sdpa
