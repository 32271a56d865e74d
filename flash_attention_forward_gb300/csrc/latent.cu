// Latent attention in its absorbed form over a paged cache, for sm_103a: every head's query meets the cached rows
// themselves, a row of 512 + 64 values being the key of all heads and, but for its last 64, their value.
//
// A row of 1152 bytes serves up to 128 heads, 2 * (576 + 512) FLOP each: with all 128 on one GPU the products weigh as much
// as the memory traffic, with the 16 of one of eight shards they are far below it.  What decides the layout is
// on-chip memory.  A block of 128 keys takes 147 KB of shared memory, and an output tile of 128 heads x 512 dims all of
// tensor memory, which leaves no room for the scores.  So both products are computed transposed, keys and dims in the
// rows of the MMAs and R = 16, 32 or 64 (token, head) pairs in their columns:
//     S^T [128 keys x R] = K Q^T          nine 64-column chunks of a key block as A, as they lie in the cache
//     O^T [4 x 128 dims x R] += V^T P^T   the same chunks, read key-major, as A; P^T [128 keys x R] from shared memory
// Every byte that arrives serves both products from one place, tensor memory holds 5 R columns, and few heads cost
// few columns.  More than 64 heads are divided over two CTAs that walk the same keys side by side, so that
// the second one's reads are served by the L2.
//
// A block of 128 keys is four pairs of chunks (128 dims), and the rotary chunk, which only the first product reads.  A pair is
// free as soon as its 128 output dims have had their product, and is refilled while the others still wait for theirs: with
// R = 64 the ring holds a single block, and P^T goes over its rotary chunk.
//
// A softmax thread holds one key's scores of 16 columns; 16 columns have a warpgroup of their own.  The running maximum
// of a column is kept until a score passes it by 2^8 (exact, as O and the sum share it), so the common block needs
// no maximum at all: P is computed with the one there is, and a barrier with an OR over the warpgroup says whether that held.
// P is rounded to the cache's type for the product; sums stay per thread, in fp32 of the unrounded P, until the end of a piece.
//
// The work is divided over the SMs as in the chunk attention (latent_plan.cuh): a unit is one tile of R pairs and one
// sequence's keys, cuts inside it write fp32 partials, which latent_combine_kernel merges.
//
// What bounds it.  16 heads: memory.  A block takes 3.4 us an SM, 6.5 TB/s, 97% of the copy rate; 64 sequences of 1024-16384
// rows take 123 us in all (5.2 TB/s), 11 being the start and the first loads, 10 the last pieces and the merge.  64 columns:
// the chain of the two products and the softmax between them, as there is room for a single block of keys beside the queries.  An
// MMA of 128 rows takes the tensor core 49 cycles whatever the columns up to 64 (64 for 128), so a block's 68 are
// 3400 of its 6500 cycles; 1700 pass between the last score's MMA and the first of P V (16 softmax warps: 210 to wake, 260 to
// load, 570 of arithmetic, 170 for the vote, 130 for the fence, 400 until the issuer sees the last arrival), the rest are waits
// and commits.  128 heads over the same sequences: 210 us, 740 TFLOP/s, 3.1 TB/s.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "sdpa.h"
#include "latent_plan.cuh"

namespace sdpa {

namespace {

constexpr int kChunkBytes = kBlockK * 128;     // 128 keys x 64 columns
constexpr int kPairBytes = 2 * kChunkBytes;
constexpr int kPairs = kLatentDim / 128;       // of a key block
constexpr int kLatentCols = 16;                // columns of a softmax warpgroup
constexpr int kLatentMaxRows = 64;
constexpr float kNoMax = 1e38f;                // minus the running maximum before the first visible key: finite, so that
                                               // a hidden key's -inf stays -inf

template <int R>
struct LatentCfg {
  static constexpr int NC = kLatentCols;
  static constexpr int WGS = R / NC;
  static constexpr int THREADS = 128 + 128 * WGS;
  static constexpr int Q_CHUNK = R * 128;
  static constexpr int Q_BYTES = (kLatentRow / 64) * Q_CHUNK;
  static constexpr bool P_OVER_ROPE = R == 64;
  static constexpr int PAIRS = R == 64 ? 4 : 5, ROPES = R == 16 ? 2 : 1;  // room for so many
  // A slot of the ring, with a barrier for its arrival and one for its release, is a pair; with R = 64, where the single
  // issuing thread sets the pace and every wait costs it some 110 cycles and every commit 55, half a block, the
  // second one with the rotary chunk (128 heads of 64 sequences: 244 -> 212 us).
  static constexpr int SLOT_PAIRS = R == 64 ? 2 : 1, SLOTS = PAIRS / SLOT_PAIRS, BLOCK_SLOTS = kPairs / SLOT_PAIRS;
  static constexpr int P_ROW = 2 * R, P_BYTES = kBlockK * P_ROW;
  static constexpr uint32_t P_SWIZZLE = R == 64 ? kSwizzle128B : R == 32 ? kSwizzle64B : kSwizzle32B;
  static constexpr int P_XOR = R == 64 ? 7 : R == 32 ? 3 : 1;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_PAIR = OFF_Q + Q_BYTES;
  static constexpr int OFF_ROPE = OFF_PAIR + PAIRS * kPairBytes;
  static constexpr int OFF_P = P_OVER_ROPE ? OFF_ROPE : OFF_ROPE + ROPES * kChunkBytes;
  static constexpr int OFF_BAR = OFF_ROPE + ROPES * kChunkBytes + (P_OVER_ROPE ? 0 : P_BYTES);
  static constexpr int PIECES = 8;  // announced pieces: more than the producer can run ahead of the softmax
  static constexpr int N_BARS = SLOTS + PAIRS + 2 * ROPES + 7 + PIECES;
  static constexpr int OFF_PIECE = OFF_BAR + 256;
  static constexpr int OFF_RED = OFF_PIECE + PIECES * 64;          // float [2][WGS][4][NC]: maxima, sums
  static constexpr int OFF_ROW = OFF_RED + 2 * WGS * 4 * NC * 4;  // int64 [R], float [2][R]: rows of O, factors, maxima
  static constexpr int SMEM = OFF_ROW + R * 16;
  static constexpr int S_COL = 0, O_COL = R;                       // tensor memory columns
  static constexpr uint32_t TMEM = R == 64 ? 512 : R == 32 ? 256 : 128;
  static_assert(N_BARS * 8 + 8 <= 256, "barriers fit their area");
  static_assert(SMEM <= 227 * 1024, "more shared memory than a CTA may opt in to");
  static_assert(O_COL + kPairs * R <= static_cast<int>(TMEM), "tensor memory holds S and O");
  static_assert(Q_BYTES % 1024 == 0 && OFF_P % 1024 == 0, "1 KB tile alignment");
  static_assert(!P_OVER_ROPE || P_BYTES == kChunkBytes, "P takes the rotary chunk's place");
};

// What a call adds to the plan's parameters.
struct LatentParams {
  int groups, group_heads;  // head groups of a tile's tokens, and the heads of one
  FastDiv div_heads;        // by group_heads
};

// Whether any of the `count` threads at barrier `id` says so; a barrier among them.
__device__ __forceinline__ bool barrier_any(uint32_t id, uint32_t count, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}

// (x0, x1) = (a0, a1) * b + (c0, c1)
__device__ __forceinline__ void ffma2_pair(float& x0, float& x1, float a0, float a1, float b, float c0, float c1) {
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\t"
      "mov.b64 rb, {%4, %4};\n\t"
      "mov.b64 rc, {%5, %6};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\t"
      "mov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(x0), "=f"(x1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}

// Barriers (phases continue from piece to piece):
//   piece[i % PIECES]         : the producer announced piece i
//   q_full / q_empty          : the query tile landed / its last Q K^T of the piece is done
//   pair_full / pair_empty    : a ring slot holds its dims of 128 keys / the P V of a pair of it is done
//   rope_full / rope_empty    : a rotary chunk landed / its K Q^T is done (R = 64: part of the second slot; P lies there, too)
//   s_full, p_full            : the scores are there (and all P V before them done) / P is written, O rescaled
//   o_full, o_empty           : the piece's last P V is done / O has been read
template <bool BF16, int R>
__global__ void __launch_bounds__(LatentCfg<R>::THREADS, 1)
    latent_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_c, const PagedParams p,
                  const LatentParams lp) {
  using C = LatentCfg<R>;
  extern __shared__ __align__(1024) uint8_t latent_smem[];
  uint8_t* smem = latent_smem;
  if (smem_u32(smem) & 1023u) {  // never: nothing static lies in front of it
    if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
    return;
  }
  uint8_t* sQ = smem + C::OFF_Q;
  uint64_t* pair_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);  // [SLOTS]
  uint64_t* pair_empty = pair_full + C::SLOTS;                            // [PAIRS]
  uint64_t* rope_full = pair_empty + C::PAIRS;                            // [ROPES]
  uint64_t* rope_empty = rope_full + C::ROPES;
  uint64_t* q_full = rope_empty + C::ROPES;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;
  uint64_t* p_full = s_full + 1;
  uint64_t* o_full = p_full + 1;
  uint64_t* o_empty = o_full + 1;
  uint64_t* mma_done = o_empty + 1;
  uint64_t* piece = mma_done + 1;                                         // [PIECES]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(piece + C::PIECES);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  LatentPiece* pieces = reinterpret_cast<LatentPiece*>(smem + C::OFF_PIECE);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int team = blockIdx.x / lp.groups, hg = blockIdx.x - team * lp.groups;
  pdl_launch_dependents();  // the combine may be scheduled early; it waits for this grid

  if (tid == 64) {  // not in the warp that allocates
    for (int s = 0; s < C::SLOTS; ++s) mbar_init(&pair_full[s], 1);
    for (int s = 0; s < C::PAIRS; ++s) mbar_init(&pair_empty[s], 1);
    for (int s = 0; s < C::ROPES; ++s) mbar_init(&rope_full[s], 1), mbar_init(&rope_empty[s], 1);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(p_full, 4 * C::WGS);
    mbar_init(o_full, 1);
    mbar_init(o_empty, 4 * C::WGS);
    mbar_init(mma_done, 1);
    for (int s = 0; s < C::PIECES; ++s) mbar_init(&piece[s], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  int4 cuts[2] = {make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0)};
  if (p.inline_plan) {
    int4* mine = reinterpret_cast<int4*>(&pieces[C::PIECES - 1]);  // free until eight pieces are announced
    latent_inline_plan<C::THREADS>(p, sQ, mine, team, blockIdx.x == 0);  // barriers of the whole block
    cuts[0] = mine[0], cuts[1] = mine[1];
    __syncthreads();  // read before it is a piece's place
  } else {
    __syncthreads();
    pdl_wait();  // the plan comes from the kernel launched before
    if (team < ld_dep(&p.plan.head->n_ctas)) {
      cuts[0] = ld_dep(p.plan.cuts + team);
      cuts[1] = ld_dep(p.plan.cuts + team + 1);
    }
  }
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  int n_piece = 0;
  auto next_piece = [&](bool& ok) -> const LatentPiece& {
    const LatentPiece& w = pieces[n_piece % C::PIECES];
    ok = mbar_wait(&piece[n_piece % C::PIECES], (n_piece / C::PIECES) & 1, abort_flag, p.status);
    ++n_piece;
    return w;
  };

  if (warp == 0 || warp == 2 || warp == 3) {
    // ------------------------------------------------------------ TMA producers (three warps)
    // One announces the pieces and loads the query tile and the first chunk of every pair, one the second chunk, one the
    // rotary chunk: pages of 16 rows take eight boxes a chunk, and a warp issues them one after the other.
    const int part = warp == 0 ? 0 : warp - 1;
    const bool rope = part == 2;
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_c);
    }
    const int rows = min(kBlockK, p.page_size);  // rows per box
    const int nsub = kBlockK / rows;             // boxes per chunk: 1 .. 8, one lane each
    const uint32_t box_at = (part & 1) * kChunkBytes + lane * rows * 128;
    const bool own_ring = rope && !C::P_OVER_ROPE;
    const int ring = own_ring ? C::ROPES : C::SLOTS;
    uint64_t* full = own_ring ? rope_full : pair_full;
    uint64_t* empty = own_ring ? rope_empty : pair_empty;
    uint8_t* base = smem + (rope ? C::OFF_ROPE : C::OFF_PAIR) + box_at;
    const int q_tx = p.tok_tile * lp.group_heads * kLatentRow * 2;
    LatentWalk walk(team, cuts[0], cuts[1]);
    int qn = 0, nl = 0;  // pieces and slots so far
    bool ok = true;
    while (ok) {
      const LatentPiece w = walk.next(p);
      if (part == 0) {
        if (lane == 0) {
          pieces[n_piece % C::PIECES] = w;
          mbar_arrive(&piece[n_piece % C::PIECES]);
        }
        ++n_piece;
      }
      if (w.n_blocks == 0) break;
      const int32_t* table = p.page_table + w.b * p.pt_b;
      const int used = (w.sk + p.page_size - 1) >> p.log2_page;  // pages that hold visible rows
      auto page_of = [&](int j) {  // of this lane's box in block j; outside the pool: the zeros behind it, for prefetches as well
        const int page = ((w.jb0 + j) * kBlockK + lane * rows) >> p.log2_page;
        const int at = j < w.n_blocks && lane < nsub && page < used ? __ldg(table + page) : p.n_pages;
        return static_cast<unsigned>(at) < static_cast<unsigned>(p.n_pages) ? at : p.n_pages;
      };
      auto row_of = [&](int j) { return ((w.jb0 + j) * kBlockK + lane * rows) & (p.page_size - 1); };
      int next = page_of(0);
      if (part == 0) {
        if (qn > 0 && !mbar_wait_warp(q_empty, (qn - 1) & 1, abort_flag, p.status)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, q_tx);
          for (int c = 0; c < kLatentRow / 64; ++c)
            tma_load_3d(sQ + c * C::Q_CHUNK, &tm_q, q_full, c * 64, hg * lp.group_heads, w.q_off + w.tok0);
        }
        ++qn;
      }
      for (int j = 0; ok && j < w.n_blocks; ++j) {
        const int page = next, row = row_of(j);
        next = page_of(j + 1);
#pragma unroll 1
        for (int g = 0; g < (own_ring ? 1 : C::BLOCK_SLOTS); ++g, ++nl) {  // the block's slots
          const int s = nl % ring, r = nl / ring;
          const bool last = g == C::BLOCK_SLOTS - 1;
          if (C::P_OVER_ROPE && rope && !last) continue;
          // where a slot is two pairs, each is loaded as it gets free; P, in the rotary chunk's place, with the last one
          auto free_slot = [&](int i) {
            return r == 0 || mbar_wait_warp(&empty[own_ring ? s : s * C::SLOT_PAIRS + i], (r - 1) & 1, abort_flag, p.status);
          };
          if (!free_slot(rope && !own_ring ? C::SLOT_PAIRS - 1 : 0)) {
            ok = false;
            break;
          }
          if (p.stall_first_stage && nl == 0) continue;  // test hook: the first slots never fill
          // one arrival announces all bytes of a slot, which may have landed by then
          if (lane == 0 && (part == 0 || own_ring))
            mbar_arrive_expect_tx(&full[s], own_ring ? kChunkBytes
                                                     : C::SLOT_PAIRS * kPairBytes + (C::P_OVER_ROPE && last ? kChunkBytes : 0));
          __syncwarp();
          if (rope) {
            if (lane < nsub) tma_load_3d(base + (own_ring ? s * kChunkBytes : 0), &tm_c, &full[s], kLatentDim, row, page);
          } else {
#pragma unroll
            for (int i = 0; i < C::SLOT_PAIRS; ++i) {
              if (i > 0 && !(ok = free_slot(i))) break;
              if (lane < nsub)
                tma_load_3d(base + (s * C::SLOT_PAIRS + i) * kPairBytes, &tm_c, &full[s], (g * C::SLOT_PAIRS + i) * 128 + part * 64, row, page);
            }
            if (!ok) break;
          }
        }
        // With one block in the ring the next one's boxes go to the L2 meanwhile (64 / 128 heads of 64 sequences: 151 -> 144,
        // 248 -> 244 us; with more in the ring, or further ahead, it loses: 16 heads 124 -> 152).  Not for small pages, whose
        // many boxes keep the copy engine busy as it is.
        if (C::P_OVER_ROPE && rope && nsub <= 2 && hg == 0 && j + 1 < w.n_blocks && lane < nsub)
          for (int c = 0; c < kLatentRow / 64; ++c) tma_prefetch_3d(&tm_c, c * 64, row_of(j + 1), next);
      }
    }
    if (!ok && lane == 0) {
      // let every copy already in flight land before the CTA's shared memory goes away
      if (qn > 0) mbar_drain(q_full, (qn - 1) & 1);
      for (int i = max(0, nl - ring); i < nl; ++i) mbar_drain(&full[i % ring], (i / ring) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (one thread)
    if (lane == 0) {
      constexpr uint32_t fmt = BF16 ? 1 : 0;
      constexpr uint32_t idesc_qk = make_idesc(fmt, fmt, 0, 0, kBlockK, R);
      constexpr uint32_t idesc_pv = make_idesc(fmt, fmt, 1, 1, 128, R);  // both operands lie key-major
      const uint64_t dq = make_smem_desc(smem_u32(sQ), 16, 1024, kSwizzle128B);
      const uint64_t dk = make_smem_desc(smem_u32(smem + C::OFF_PAIR), 16, 1024, kSwizzle128B);
      const uint64_t dr = make_smem_desc(smem_u32(smem + C::OFF_ROPE), 16, 1024, kSwizzle128B);
      const uint64_t dv = make_smem_desc(smem_u32(smem + C::OFF_PAIR), kChunkBytes, 1024, kSwizzle128B);
      const uint64_t dp = make_smem_desc(smem_u32(smem + C::OFF_P), kChunkBytes, 8 * C::P_ROW, C::P_SWIZZLE);
      const uint32_t q_lo = static_cast<uint32_t>(dq), q_hi = static_cast<uint32_t>(dq >> 32);
      const uint32_t k_lo = static_cast<uint32_t>(dk), k_hi = static_cast<uint32_t>(dk >> 32);
      const uint32_t r_lo = static_cast<uint32_t>(dr), r_hi = static_cast<uint32_t>(dr >> 32);
      const uint32_t v_lo = static_cast<uint32_t>(dv), v_hi = static_cast<uint32_t>(dv >> 32);
      const uint32_t p_lo = static_cast<uint32_t>(dp), p_hi = static_cast<uint32_t>(dp >> 32);
      const uint32_t tS = tmem_base + C::S_COL, tO = tmem_base + C::O_COL;
      int qn = 0, nl = 0, bn = 0;  // pieces, slots, blocks so far
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, abort_flag, p.status); };
      // slot g of the block; a single block in the ring always lies in the same ones
      auto slot_of = [&](int g) { return C::SLOTS == C::BLOCK_SLOTS ? g : (nl + g) % C::SLOTS; };
      while (true) {
        const LatentPiece& w = next_piece(ok);
        const int nb = ok ? w.n_blocks : 0;
        if (nb == 0 || !wait(q_full, qn & 1)) break;
        for (int j = 0; ok && j < nb; ++j) {
          // S^T = K Q^T, slot by slot as they land
#pragma unroll
          for (int g = 0; g < C::BLOCK_SLOTS; ++g) {
            const int s = slot_of(g);
            if (!(ok = wait(&pair_full[s], ((nl + g) / C::SLOTS) & 1))) break;
            tc_fence_after();
            const uint32_t a = k_lo + static_cast<uint32_t>((s * C::SLOT_PAIRS * kPairBytes) >> 4);
            const uint32_t b = q_lo + static_cast<uint32_t>((2 * g * C::SLOT_PAIRS * C::Q_CHUNK) >> 4);
#pragma unroll
            for (int kk = 0; kk < 8 * C::SLOT_PAIRS; ++kk)
              mma_f16_ss(tS, a + static_cast<uint32_t>(((kk / 4) * kChunkBytes + (kk % 4) * 32) >> 4), k_hi,
                         b + static_cast<uint32_t>(((kk / 4) * C::Q_CHUNK + (kk % 4) * 32) >> 4), q_hi, idesc_qk,
                         g > 0 || kk > 0 ? 1u : 0u);
          }
          const int rs = bn % C::ROPES;
          if (!ok || !(ok = C::P_OVER_ROPE || wait(&rope_full[rs], (bn / C::ROPES) & 1))) break;
          if (!C::P_OVER_ROPE) tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_ss(tS, r_lo + static_cast<uint32_t>((rs * kChunkBytes + kk * 32) >> 4), r_hi,
                       q_lo + static_cast<uint32_t>((2 * kPairs * C::Q_CHUNK + kk * 32) >> 4), q_hi, idesc_qk, 1u);
          mma_commit(s_full);
          if (!C::P_OVER_ROPE) mma_commit(&rope_empty[rs]);
          if (j == nb - 1) mma_commit(q_empty);
          // O^T += V^T P^T, 128 dims at a time
          if (!(ok = (j > 0 || qn == 0 || wait(o_empty, (qn - 1) & 1)) && wait(p_full, bn & 1))) break;
          ++bn;
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < C::BLOCK_SLOTS; ++g) {
            const int s = slot_of(g);
#pragma unroll
            for (int i = 0; i < C::SLOT_PAIRS; ++i) {
              const uint32_t a = v_lo + static_cast<uint32_t>(((s * C::SLOT_PAIRS + i) * kPairBytes) >> 4);
#pragma unroll
              for (int kk = 0; kk < kBlockK / 16; ++kk)
                mma_f16_ss(tO + (g * C::SLOT_PAIRS + i) * R, a + static_cast<uint32_t>((kk * 16 * 128) >> 4), v_hi,
                           p_lo + static_cast<uint32_t>((kk * 16 * C::P_ROW) >> 4), p_hi, idesc_pv, j > 0 || kk > 0 ? 1u : 0u);
              mma_commit(&pair_empty[s * C::SLOT_PAIRS + i]);
            }
          }
          nl += C::BLOCK_SLOTS;
          if (j == nb - 1) mma_commit(o_full);
        }
        if (!ok) break;
        ++qn;
      }
      // Every MMA issued so far has finished before tensor memory is released: the softmax has waited for the last ones
      // (o_full), unless a wait gave up.
      if (*abort_flag) {
        mma_commit(mma_done);
        mbar_drain(mma_done, 0);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax: a warpgroup for NC columns
    constexpr int NC = C::NC;
    const int wg = (warp - 4) >> 2, wq = warp & 3;
    const int row = wq * 32 + lane;   // key of the block; dim of 128
    const int col0 = wg * NC;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem_base + lane_off + C::S_COL + col0, tO = tmem_base + lane_off + C::O_COL + col0;
    const uint32_t bar_id = 1 + wg;
    float* red_max = reinterpret_cast<float*>(smem + C::OFF_RED) + wg * 4 * NC;  // [4][16]
    float* red_sum = red_max + C::WGS * 4 * NC;
    int64_t* row_at = reinterpret_cast<int64_t*>(smem + C::OFF_ROW) + wg * NC;
    float* row_inv = reinterpret_cast<float*>(smem + C::OFF_ROW + C::WGS * NC * 8) + wg * NC;
    float* neg_max = row_inv + C::WGS * NC;
    // P^T row of this key: this warpgroup's columns
    uint8_t* p_row[NC / 8];
#pragma unroll
    for (int i = 0; i < NC / 8; ++i) {
      const int off = row * C::P_ROW + col0 * 2 + i * 16;
      p_row[i] = smem + C::OFF_P + (off ^ (((off >> 7) & C::P_XOR) << 4));
    }
    const int heads = min(lp.group_heads, p.Hq - hg * lp.group_heads);
    int sn = 0, on = 0;  // blocks and pieces so far
    bool ok = true;
    while (true) {
      bool got;
      const LatentPiece& w = next_piece(got);
      got = __all_sync(0xffffffffu, got);
      // the four warps leave together: they meet at barriers
      if (barrier_any(bar_id, 128, !(ok && got))) break;
      const int nb = w.n_blocks;
      if (nb == 0) break;
      const int q_off = w.q_off, tok0 = w.tok0, sk = w.sk, slot = w.slot, jb0 = w.jb0;
      const int tokens = min(p.tok_tile, w.n - tok0);
      const int base = p.causal ? w.len - w.n + tok0 + 1 : sk;  // keys that the tile's first token sees, but for sk
      const int lim_all = min(sk, base);
      // Minus the columns' running maxima, in powers of two, lie in shared memory.  A column without a (token, head), whose
      // scores may be anything, has P = 0 and no say in the votes.
      if (row < NC) {
        const int t = static_cast<int>(fast_div(static_cast<uint32_t>(col0 + row), lp.div_heads));
        neg_max[row] = t < tokens && col0 + row - t * lp.group_heads < heads ? kNoMax : -INFINITY;
      }
      named_barrier_sync(bar_id, 128);
      float l[NC];  // this key's sums
#pragma unroll
      for (int c = 0; c < NC; ++c) l[c] = 0.f;
      for (int j = 0; j < nb; ++j, ++sn) {
        ok = mbar_wait_warp(s_full, sn & 1, abort_flag, p.status);
        const int k0 = (jb0 + j) * kBlockK;
        auto scores = [&](uint32_t (&r)[NC]) {  // of this thread's key; hidden ones -inf
          tmem_ld16(tS, r);
          tmem_ld_wait();
          reg_fence(r);
          if (k0 + kBlockK > lim_all) {  // the diagonal and the last block hide keys
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              const int t = static_cast<int>(fast_div(static_cast<uint32_t>(col0 + c), lp.div_heads));
              if (k0 + row >= min(sk, p.causal ? base + t : sk)) r[c] = 0xFF800000u;
            }
          }
        };
        // P with the maxima as they are, which nearly always holds: the barrier that says so comes behind the work
        uint32_t pk[NC / 2];
        float sums[NC];
        auto probabilities = [&](const uint32_t (&r)[NC]) {  // and the largest distance from a running maximum
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < NC; c += 2) {
            const float2 nm = *reinterpret_cast<const float2*>(neg_max + c);
            float x0, x1;
            ffma2_pair(x0, x1, __uint_as_float(r[c]), __uint_as_float(r[c + 1]), p.scale2, nm.x, nm.y);
            top = fmax3(top, x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            sums[c] = l[c], sums[c + 1] = l[c + 1];
            fadd2(sums[c], sums[c + 1], p0, p1);
            pk[c / 2] = BF16 ? pack_bf16x2(p0, p1) : pack_f16x2(p0, p1);
          }
          return top;
        };
        bool need = !ok;
        if (ok) {
          tc_fence_after();
          uint32_t r[NC];
          scores(r);
          need = probabilities(r) > kPagedRescaleLog2;
          // rows of V past the cache: 0 * NaN would poison the product.  The block's pairs have all landed.
          if (k0 + kBlockK > sk && k0 + row >= sk) {
            for (int c = wg; c < kPairs; c += C::WGS) {
              uint8_t* v = smem + C::OFF_PAIR + ((kPairs * sn + c) % C::PAIRS) * kPairBytes + row * 128;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                *reinterpret_cast<uint4*>(v + (i >> 3) * kChunkBytes + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          __syncwarp();
        }
        if (barrier_any(bar_id, 128, need)) {
          // the columns' maxima over the block's keys, new running maxima, O and the sums rescaled
          uint32_t r[NC];
          if (ok) {
            scores(r);
            float mx[NC];
#pragma unroll
            for (int c = 0; c < NC; ++c) mx[c] = __uint_as_float(r[c]);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1)
#pragma unroll
              for (int c = 0; c < NC; ++c) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], d));
            if (lane == 0)
#pragma unroll
              for (int c = 0; c < NC; c += 4)
                *reinterpret_cast<float4*>(red_max + wq * NC + c) = make_float4(mx[c], mx[c + 1], mx[c + 2], mx[c + 3]);
            __syncwarp();
          }
          float nm[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) nm[c] = neg_max[c];
          const float nm_l = neg_max[lane % NC];
          if (barrier_any(bar_id, 128, !ok)) {
            ok = false;
            break;
          }
          auto block_max = [&](int c) {
            return fmaxf(fmaxf(red_max[c], red_max[NC + c]), fmaxf(red_max[2 * NC + c], red_max[3 * NC + c]));
          };
          // A column with a score of +infinity takes that as its maximum (its P is NaN or 0 from here on, and it asks for no
          // further vote), but moves no other: an infinite query does not touch the rounding of the rows beside it.  So whether
          // a finite score passed its column's maximum is asked again, a column a lane.
          const float mb_l = block_max(lane % NC);
          const bool far = __any_sync(0xffffffffu, mb_l * p.scale2 < INFINITY && fmaf(mb_l, p.scale2, nm_l) > kPagedRescaleLog2);
          float alpha[NC];
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float least = fminf(nm[c], -(block_max(c) * p.scale2));
            const float neg = far || least == -INFINITY ? least : nm[c];
            alpha[c] = neg == nm[c] ? 1.f : ex2(neg - nm[c]);
            if (row == c) neg_max[c] = neg;
            l[c] *= alpha[c];
          }
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < kPairs; ++c) {
              uint32_t o[NC];
              tmem_ld16(tO + c * R, o);
              tmem_ld_wait();
              reg_fence(o);
#pragma unroll
              for (int i = 0; i < NC; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[i]);
              tmem_st16(tO + c * R, o);
            }
            tmem_st_wait();
          }
          named_barrier_sync(bar_id, 128);  // the new maxima are there
          probabilities(r);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) l[c] = sums[c];
#pragma unroll
        for (int i = 0; i < NC / 8; ++i)
          *reinterpret_cast<uint4*>(p_row[i]) = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(p_full, lane);
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue: O / l and LSE, or a partial
#pragma unroll
      for (int d = 16; d > 0; d >>= 1)
#pragma unroll
        for (int c = 0; c < NC; ++c) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
      if (lane == 0) {
#pragma unroll
        for (int c = 0; c < NC; c += 4)
          *reinterpret_cast<float4*>(red_sum + wq * NC + c) = make_float4(l[c], l[c + 1], l[c + 2], l[c + 3]);
      }
      __syncwarp();
      named_barrier_sync(bar_id, 128);
      const bool partial = slot >= 0;
      if (row < NC) {
        // this thread's column: where its row of O goes (among the partials or to O; < 0: nowhere), its factor
        const int t = static_cast<int>(fast_div(static_cast<uint32_t>(col0 + row), lp.div_heads));
        const int h = col0 + row - t * lp.group_heads;  // of the group
        const float neg = neg_max[row];
        float sum = (red_sum[row] + red_sum[NC + row]) + (red_sum[2 * NC + row] + red_sum[3 * NC + row]);
        // a score of +infinity: where only its product with the scale was, the sum is 0
        if (neg == -INFINITY) sum = __uint_as_float(0x7FC00000u);
        int64_t at = -1;
        if (t < tokens && h < heads) {
          const int head = hg * lp.group_heads + h;
          if (partial) {
            const int64_t prow = static_cast<int64_t>(slot) * p.slot_rows + t * p.Hq + head;
            at = prow * kLatentDim;
            *reinterpret_cast<float2*>(p.part_ml + prow * 2) = make_float2(-neg, sum);
          } else {
            const int q_row = q_off + tok0 + t;
            at = q_row * p.o_s + head * p.o_h;
            if (p.lse != nullptr)
              p.lse[static_cast<int64_t>(head) * p.total_q + q_row] = sum == 0.f ? -INFINITY : (lg2(sum) - neg) * kPagedLn2;
          }
        }
        row_at[row] = at;
        row_inv[row] = partial ? 1.f : sum == 0.f ? 0.f : 1.f / sum;  // NaN stays NaN
      }
      ok = mbar_wait_warp(o_full, on & 1, abort_flag, p.status);
      ++on;
      if (barrier_any(bar_id, 128, !ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < kPairs; ++c) {
        uint32_t o[NC];
        tmem_ld16(tO + c * R, o);
        tmem_ld_wait();
        reg_fence(o);
        if (partial) {
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            const int64_t at = row_at[i];
            if (at >= 0) p.part_o[at + c * 128 + row] = __uint_as_float(o[i]);
          }
        } else {
          // neighbouring lanes hold neighbouring dims: an even lane takes both of column i, an odd one of column i + 1
#pragma unroll
          for (int i = 0; i < NC; i += 2) {
            const int mine = i + (lane & 1);
            const float a = __uint_as_float(o[i]) * row_inv[i], b = __uint_as_float(o[i + 1]) * row_inv[i + 1];
            const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : b, 1);
            const float lo = lane & 1 ? other : a, hi = lane & 1 ? b : other;
            const int64_t at = row_at[mine];
            if (at >= 0)
              *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + at + c * 128 + (row & ~1)) =
                  BF16 ? pack_bf16x2(lo, hi) : pack_f16x2(lo, hi);
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      warp_arrive(o_empty, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM);
  }
}

// Merges the pieces of the cut units, as paged_combine_kernel, for rows of 512 values: O = sum w_i O_i / sum w_i l_i, w_i =
// 2^(m_i - max m).  Two warps a row; a warp's lanes fetch the maxima and sums of up to 32 pieces side by side, so that the
// loads of O depend on one load only and are in flight together.
constexpr int kLatentMergeRows = 4;

template <bool BF16>
__global__ void __launch_bounds__(64 * kLatentMergeRows) latent_combine_kernel(const PagedParams p) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  // read at once, whether the group exists or not
  const int n_groups = ld_dep(&p.plan.head->n_groups);
  const int4* record = reinterpret_cast<const int4*>(p.plan.groups + blockIdx.x);
  const int4 g0 = ld_dep(record), g1 = ld_dep(record + 1);
  if (static_cast<int>(blockIdx.x) >= n_groups) return;
  const int tile = g0.x, first = g0.z, pieces = g0.w, slot0 = g1.x, q_off = g1.y, n = g1.z;
  const int row = blockIdx.y * kLatentMergeRows + threadIdx.x / 64, col = (threadIdx.x % 64) * 4;  // and col + 256
  const int row_tok = static_cast<int>(fast_div(row, p.div_group));
  const int tok = tile * p.tok_tile + row_tok;
  if (row >= p.slot_rows || tok >= n) return;
  auto row_of = [&](int i) { return static_cast<int64_t>(i == 0 ? slot0 : 2 * (first + i)) * p.slot_rows + row; };
  float M = -INFINITY, L = 0.f;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int base = 0; base < pieces; base += 32) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (base + lane < pieces) ml = *reinterpret_cast<const float2*>(p.part_ml + row_of(base + lane) * 2);
    float top = fmaxf(M, ml.x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    const float old = M == -INFINITY ? 0.f : ex2(M - top);
    M = top;
    const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
    float sum = w * ml.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    L = L * old + sum;
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] *= old;
    const int count = min(32, pieces - base);
#pragma unroll 4
    for (int i = 0; i < count; ++i) {
      const float* o = p.part_o + row_of(base + i) * kLatentDim + col;
      const float4 a = *reinterpret_cast<const float4*>(o), b = *reinterpret_cast<const float4*>(o + 256);
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] += wi * v[c];
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;  // NaN stays NaN
  const int head = row - row_tok * p.group;
  uint16_t* o = static_cast<uint16_t*>(p.o) + static_cast<int64_t>(q_off + tok) * p.o_s + static_cast<int64_t>(head) * p.o_h + col;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* a = acc + 4 * h;
    *reinterpret_cast<uint2*>(o + 256 * h) =
        BF16 ? make_uint2(pack_bf16x2(a[0] * inv, a[1] * inv), pack_bf16x2(a[2] * inv, a[3] * inv))
             : make_uint2(pack_f16x2(a[0] * inv, a[1] * inv), pack_f16x2(a[2] * inv, a[3] * inv));
  }
  if (p.lse != nullptr && col == 0)
    p.lse[static_cast<int64_t>(head) * p.total_q + q_off + tok] = L == 0.f ? -INFINITY : (M + lg2(L)) * kPagedLn2;
}

cudaError_t launch_latent_combine(bool bf16, const PagedParams& p, cudaStream_t st) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // at most p.sms - 1 units are cut
  cfg.gridDim = dim3(static_cast<unsigned>(std::max(p.sms - 1, 1)),
                     static_cast<unsigned>((p.slot_rows + kLatentMergeRows - 1) / kLatentMergeRows));
  cfg.blockDim = dim3(64 * kLatentMergeRows);
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return bf16 ? cudaLaunchKernelEx(&cfg, latent_combine_kernel<true>, p) : cudaLaunchKernelEx(&cfg, latent_combine_kernel<false>, p);
}

template <bool BF16, int R>
cudaError_t launch_latent(const CUtensorMap& tq, const CUtensorMap& tc, const PagedParams& p, const LatentParams& lp,
                          cudaStream_t st) {
  using C = LatentCfg<R>;
  auto kern = latent_kernel<BF16, R>;
  int dev = 0, sms = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> opted{0};
  if ((e = smem_opt_in(kern, C::SMEM, dev, opted)) != cudaSuccess) return e;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.sms * lp.groups));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = p.inline_plan ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tq, tc, p, lp);
}

// How the heads of a token and the tokens of a tile fill R columns.
struct LatentTile {
  int groups, group_heads, tok_tile, rows;
};
LatentTile latent_tile(int Hq, int max_seqlen_q) {
  LatentTile t;
  t.groups = (Hq + kLatentMaxRows - 1) / kLatentMaxRows;
  t.group_heads = (Hq + t.groups - 1) / t.groups;
  t.tok_tile = std::min(kLatentMaxRows / t.group_heads, max_seqlen_q);
  if (t.groups > 1) t.tok_tile = 1;  // a slot of partials holds one token's heads of all groups
  const int used = t.tok_tile * t.group_heads;
  t.rows = used <= 16 ? 16 : used <= 32 ? 32 : 64;
  return t;
}
long long latent_tiles(int B, int total_q, int max_seqlen_q, int tok_tile) {
  return std::min(static_cast<long long>(B) * ((max_seqlen_q + tok_tile - 1) / tok_tile),
                  (static_cast<long long>(total_q) + static_cast<long long>(tok_tile - 1) * B) / tok_tile);
}
// Two slots per team of CTAs; none where no unit is long enough to be cut.
size_t latent_partial_bytes(const LatentTile& t, int Hq, int max_kv) {
  if ((max_kv + kBlockK - 1) / kBlockK < 2 * kLatentMinPiece) return 0;
  return 2ull * (kPagedMaxCtas / t.groups) * t.tok_tile * Hq * (kLatentDim + 2) * sizeof(float);
}

}  // namespace

}  // namespace sdpa

using namespace sdpa;

extern "C" {

size_t sdpa_fwd_latent_paged_workspace_size(int B, int Hq, int total_q, int max_seqlen_q, int max_kv) {
  if (B < 1 || Hq < 1 || Hq > 2 * kLatentMaxRows || total_q < 1 || max_seqlen_q < 1 || max_seqlen_q > total_q || max_kv < 1 ||
      max_kv > (1 << 30) || B > kMaxCount || total_q > kMaxCount)
    return 0;
  const LatentTile t = latent_tile(Hq, max_seqlen_q);
  return paged_plan_bytes(B, latent_tiles(B, total_q, max_seqlen_q, t.tok_tile)) + latent_partial_bytes(t, Hq, max_kv);
}

int sdpa_fwd_latent_paged(const void* q, const void* pool, const int32_t* page_table, const int32_t* kv_len,
                          const int32_t* cu_seqlens_q, void* o, float* lse, int B, int Hq, int total_q, int max_seqlen_q,
                          int page_size, int max_pages, int n_pages, int latent_dim, int rotary_dim, const int64_t* strides,
                          float scale, int causal, void* workspace, size_t workspace_bytes, sdpa_dtype dtype, void* stream) {
  // ---- validation (no CUDA call before this block passes)
  if (!q || !pool || !page_table || !kv_len || !cu_seqlens_q || !o) return SDPA_ERR_INVALID;
  if (B < 1 || Hq < 1 || total_q < 1 || max_seqlen_q < 1 || max_seqlen_q > total_q || latent_dim < 1 || rotary_dim < 1)
    return SDPA_ERR_INVALID;
  if (!(std::isfinite(scale) && scale > 0.f)) return SDPA_ERR_INVALID;
  const int rc = page_check(page_size, max_pages, n_pages);
  if (rc != SDPA_OK) return rc;
  if (dtype != SDPA_F16 && dtype != SDPA_BF16) return SDPA_ERR_UNSUPPORTED;
  if (latent_dim != kLatentDim || rotary_dim != kLatentRot || Hq > 2 * kLatentMaxRows || B > kMaxCount || total_q > kMaxCount)
    return SDPA_ERR_UNSUPPORTED;
  int64_t st[SDPA_FWD_LATENT_PAGED_NSTRIDES] = {(int64_t)Hq * kLatentRow, kLatentRow, (int64_t)page_size * kLatentRow,
                                                kLatentRow, (int64_t)Hq * kLatentDim, kLatentDim, max_pages};
  if (strides) std::memcpy(st, strides, sizeof(st));
  for (int i = 0; i < 6; ++i)
    if (!stride_ok(st[i], 8)) return SDPA_ERR_UNSUPPORTED;
  if (st[6] < max_pages || rows_coincide(total_q, st[4]) || rows_coincide(Hq, st[5])) return SDPA_ERR_INVALID;
  if (rows_coincide(total_q, st[0]) || rows_coincide(Hq, st[1]) || rows_coincide(n_pages, st[2]) || rows_coincide(page_size, st[3]))
    return SDPA_ERR_UNSUPPORTED;  // no tensor map of such a layout
  if (!aligned16(q) || !aligned16(pool) || !aligned16(o)) return SDPA_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(kv_len) |
       reinterpret_cast<uintptr_t>(cu_seqlens_q) | reinterpret_cast<uintptr_t>(lse)) & 3u)
    return SDPA_ERR_INVALID;
  const int max_kv = max_pages * page_size;
  const LatentTile t = latent_tile(Hq, max_seqlen_q);
  const long long tiles = latent_tiles(B, total_q, max_seqlen_q, t.tok_tile);
  if (tiles >= (1ll << 30)) return SDPA_ERR_UNSUPPORTED;
  const size_t plan = paged_plan_bytes(B, tiles), partials = latent_partial_bytes(t, Hq, max_kv);
  if (!workspace || !aligned16(workspace) || workspace_bytes < plan) return SDPA_ERR_INVALID;

  // One "KV head" whose group are all heads: the head groups of a unit are the CTAs of a team.
  PagedParams p{};
  p.o = o, p.lse = lse, p.o_s = st[4], p.o_h = st[5];
  p.cu_q = cu_seqlens_q, p.kv_len = kv_len, p.page_table = page_table, p.pt_b = st[6];
  p.B = B, p.Hq = Hq, p.Hkv = 1, p.total_q = total_q, p.max_seqlen_q = max_seqlen_q, p.group = Hq;
  p.causal = causal ? 1 : 0;
  p.tok_tile = t.tok_tile;
  p.unit_tiles = 1, p.min_piece = kLatentMinPiece, p.min_work = kLatentMinWork;
  p.page_size = page_size, p.log2_page = __builtin_ctz((unsigned)page_size);
  p.max_pages = max_pages, p.n_pages = n_pages, p.max_kv = max_kv;
  p.scale2 = (float)((double)scale * 1.4426950408889634);
  p.div_group = make_fastdiv((uint32_t)Hq);
  p.slot_rows = t.tok_tile * Hq;
  p.cut = partials > 0 && workspace_bytes >= plan + partials;
  p.max_tiles = (int)tiles;
  p.inline_plan = B <= kInlinePlanSeqs && max_seqlen_q <= kInlineTiles * t.tok_tile;
  p.plan = paged_plan_at(workspace, tiles);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan);
  p.part_ml = p.part_o + 2ull * (kPagedMaxCtas / t.groups) * p.slot_rows * kLatentDim;
  int dev = 0;
  if (current_device_sms(&dev, &p.sms) != cudaSuccess || device_status_ptr(&p.status) != cudaSuccess) return SDPA_ERR_CUDA;
  p.sms = std::max(1, std::min(p.sms, kPagedMaxCtas) / t.groups);
  LatentParams lp{t.groups, t.group_heads, make_fastdiv((uint32_t)t.group_heads)};

  alignas(64) CUtensorMap tq, tc;
  const bool bf16 = dtype == SDPA_BF16;
  const CUtensorMapDataType dt = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  if (!encode_tiled3(&tq, q, dt, 2, kLatentRow, Hq, total_q, st[1], st[0], 64, t.group_heads, t.tok_tile,
                     CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tiled3(&tc, pool, dt, 2, kLatentRow, page_size, n_pages, st[3], st[2], 64, std::min(kBlockK, page_size), 1,
                     CU_TENSOR_MAP_SWIZZLE_128B))
    return SDPA_ERR_CUDA;
  p.stall_first_stage = take_stall_flag();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = p.inline_plan ? cudaSuccess : launch_paged_plan(p, s);
  if (e == cudaSuccess) {
    if (t.rows == 16)
      e = bf16 ? launch_latent<true, 16>(tq, tc, p, lp, s) : launch_latent<false, 16>(tq, tc, p, lp, s);
    else if (t.rows == 32)
      e = bf16 ? launch_latent<true, 32>(tq, tc, p, lp, s) : launch_latent<false, 32>(tq, tc, p, lp, s);
    else
      e = bf16 ? launch_latent<true, 64>(tq, tc, p, lp, s) : launch_latent<false, 64>(tq, tc, p, lp, s);
  }
  if (e == cudaSuccess && p.cut) e = launch_latent_combine(bf16, p, s);
  return e == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

}  // extern "C"
