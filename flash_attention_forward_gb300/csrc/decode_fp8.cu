// Split-KV decode over a quantised paged cache (e4m3 codes, one fp32 scale per row of K and of V)
// for sm_103a: one query token per sequence.
//
// The two phases are those of the 16-bit decode: a CTA owns one (sequence, KV head, split of keys)
// and writes a partial (unnormalised O, max, sum); the combine merges the splits.  What differs is
// the arithmetic between the codes and the tensor cores:
//   * every e4m3 value is exact in fp16, so the codes go to fp16 fragments unscaled and both
//     products are fp16 with fp32 accumulation.  A bf16 query is moved into fp16's range by a power
//     of two per row (its largest entry to [2^14, 2^15)), which keeps all 8 of its bits down to
//     2^-29 of that entry;
//   * K's scale multiplies the fp32 score of its key;
//   * V's scale joins the exponent: with y_j = s_j + log2(v_scale_j) and the running maximum taken
//     over y, P_j = 2^(y_j - m) feeds the P.V product against the bare codes and
//     l = sum 2^(s_j - m) is the matching denominator.  P then stays in fp16's best range whatever
//     the scales are, where a product P * v_scale could leave it.
// Bound by memory: D + Dv + 8 bytes per row against 2 (D + Dv) flops per query head.  64 sequences of
// 1024-16384 rows, 32 / 8 heads of 128, pages of 64: 193 us with the combine in a graph, 6.1 TB/s of codes
// and scales; the same loads without the arithmetic took 194 when the whole took 196.  The products with
// keys and value dims in the 16 rows of an MMA (below) brought it from 225: with heads there, half of each
// MMA, of the accumulators and of the softmax's shuffles were for empty rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <algorithm>
#include <atomic>

#include "sdpa.h"
#include "internal.h"
#include "ptx.cuh"

namespace sdpa {

namespace {

constexpr float kRescaleLog2F8 = 8.0f;
constexpr int kF8Chunk = 64;                   // keys per ring stage
constexpr int kF8Box = kF8Chunk * 128;         // one box of 128 codes a row: 8 KB
constexpr int kF8Threads = (kDecodeWarps + 1) * 32;
// A zero scale (the filling of pages outside the pool) counts as 2^-100, so that the maximum stays
// finite and the sum stays below fp32's largest value.  For V's scales in [2^-80, 2^80], as the header asks, the terms
// 2^(s_j - m) of the sum lie between 2^88 and 2^-80 where their weight is the row's largest, and vanish (2^-126)
// only under 2^-46 of it.
constexpr float kMinLog2Scale = -100.f;
constexpr int kF8MinSplit = 256;

template <int D>
struct DecF8Cfg {
  static constexpr int KBOX = (D + 127) / 128;          // K boxes per chunk (columns past D read as zeros)
  static constexpr int UNITS = D / 64;                  // 16-code units of a K row per thread
  static constexpr int CODES = (KBOX + 1) * kF8Box;     // 16 KB (D = 128) or 24 KB (D = 192)
  static constexpr int SCALES = 2 * kF8Chunk * 4;       // bytes of K and V scales that land per stage
  static constexpr int SCALE_AREA = 1024;               // ... in pieces of at least 128 B each (TMA's alignment)
  static constexpr int STAGES = D == 128 ? 6 : 4;       // about 100 KB in flight per CTA, two CTAs per SM
  static constexpr int SMEM = STAGES * (CODES + SCALE_AREA) + 256 + 1024;
  static_assert(D % 64 == 0 && STAGES * CODES >= kDecodeWarps * 16 * kDecodeDv * 4, "merge buffer fits the ring");
};

// The order of the eight keys of a fragment and of the eight 16-code units of a V row: neighbours
// differ in bit 2, which spreads the 16-byte reads of a quarter-warp (two rows x four units of K,
// four rows x two units of V) over all banks of the 128-byte swizzle.
__constant__ int kOrder[8] = {0, 4, 1, 5, 2, 6, 3, 7};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit values held as an MMA fragment (thread (g, t): row g, columns 2t, 2t + 1).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t byte_perm(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

__device__ __forceinline__ uint4 lds16(const uint8_t* base, int row, int unit) {
  return *reinterpret_cast<const uint4*>(base + row * 128 + ((unit ^ (row & 7)) << 4));
}

// WIDE: groups of 9-16 query heads per KV head (a second tile of 8 columns).
template <bool BF16, int D, bool WIDE>
__global__ void __launch_bounds__(kF8Threads, 2)
    decode_f8_split_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs,
                           const DecodeParams p) {
  using C = DecF8Cfg<D>;
  constexpr int ST = C::STAGES;
  constexpr int RH = WIDE ? 2 : 1;
  constexpr int R = 8 * RH;
  constexpr int CH = WIDE ? 1 : 2;  // chains of MMAs per score: two in all hide half of their latency
  extern __shared__ uint8_t f8_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(f8_smem_raw) + 1023) & ~uintptr_t(1023));
  float* scales = reinterpret_cast<float*>(smem + ST * C::CODES);  // [ST][K, V][128]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + ST * (C::CODES + C::SCALE_AREA));
  uint64_t* empty = full + ST;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + ST);

  pdl_launch_dependents();  // the combine may be scheduled early; it waits for this grid
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = min(max(__ldg(p.kv_len + b), 0), p.max_kv);
  const int start = split << p.log2_split;
  if (start >= L) return;
  const int end = min(start + (1 << p.log2_split), L);
  const int nchunks = (end - start + kF8Chunk - 1) / kF8Chunk;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kDecodeWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();

  __shared__ float sm_m[kDecodeWarps][R];
  __shared__ float sm_l[kDecodeWarps][R];
  const int G = p.group;

  if (warp == kDecodeWarps) {
    // ---------------------------------------------------------- producer (one warp)
    // A chunk is `parts` boxes (K columns 0-127 (and 128-255), V, K scales, V scales) for each of
    // its pages; the lanes take one box each, so that page-table reads and issues overlap.
    constexpr int PARTS = C::KBOX + 3;
    const int rows = min(kF8Chunk, p.page_size);
    const int nsub = kF8Chunk / rows;  // pages per chunk: 1, 2 or 4
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_ks);
      tma_prefetch_desc(&tm_vs);
    }
    const int part = lane % PARTS, sub = lane / PARTS;
    int c = 0;
    for (; c < nchunks; ++c) {
      const int s = c % ST, r = c / ST;
      // page and row of this lane's box; logical pages past the table read as zeros
      const int key = start + c * kF8Chunk + sub * rows;
      const int lp = key >> p.log2_page;
      int phys = p.n_pages;
      if (sub < nsub && lp < p.max_pages) phys = __ldg(p.page_table + b * p.pt_b + lp);
      const int prow = key & (p.page_size - 1);
      if (r > 0 && !mbar_wait_warp(&empty[s], (r - 1) & 1, abort_flag, p.status)) break;
      if (lane == 0) mbar_arrive_expect_tx(&full[s], C::CODES + C::SCALES);
      __syncwarp();
      if (sub < nsub) {
        uint8_t* st = smem + s * C::CODES;
        float* sc = scales + s * 256 + sub * max(rows, 32);
        if (part < C::KBOX)
          tma_load_4d(st + part * kF8Box + sub * rows * 128, &tm_k, &full[s], 128 * part, kvh, prow, phys);
        else if (part == C::KBOX)
          tma_load_4d(st + C::KBOX * kF8Box + sub * rows * 128, &tm_v, &full[s], 0, kvh, prow, phys);
        else
          tma_load_3d(sc + (part == C::KBOX + 1 ? 0 : 128), part == C::KBOX + 1 ? &tm_ks : &tm_vs, &full[s],
                      prow, kvh, phys);
      }
    }
    if (c < nchunks && lane == 0)  // aborted: let the copies in flight land
      for (int j = max(0, c - ST); j < c; ++j) mbar_drain(&full[j % ST], (j / ST) & 1);
  } else {
    // ---------------------------------------------------------- consumers
    // Both products are taken transposed, S^T = K Q^T and O^T = V^T P^T: the 16 rows of an MMA are
    // keys and value dims, its 8 columns the heads of the group, so that no row of it is empty.
    // g = lane / 4, t = lane % 4.  K (A operand): thread (g, t) holds dims [64 i + 16 t, +16), i < D / 64,
    // of the keys g and g + 8 (in kOrder); one 32-bit word of four codes is one k-step.  V^T (A operand):
    // keys 2t, 2t + 1 (+ 8) in kOrder, dims [16 kOrder[g], +16), two of them per tile.  Accumulators:
    // acc[rh][i] holds dims 16 kOrder[g] + 2 i (+ 1) of the heads 2t, 2t + 1 (+ 8 rh).
    const int g = lane >> 2, t = lane & 3;
    uint32_t qf[RH][C::UNITS][8];  // head g + 8 rh (B operand)
    float qs[RH][2];               // score scale of heads 2t, 2t + 1 (+ 8 rh), exp2 units
#pragma unroll
    for (int rh = 0; rh < RH; ++rh) {
      const int head = g + 8 * rh;
      qs[rh][0] = qs[rh][1] = p.scale2;
#pragma unroll
      for (int i = 0; i < C::UNITS; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) qf[rh][i][j] = 0u;
      if (head < G) {
        const uint16_t* qrow = static_cast<const uint16_t*>(p.q) + b * p.q_b + static_cast<int64_t>(kvh * G + head) * p.q_h;
#pragma unroll
        for (int i = 0; i < C::UNITS; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(qrow + 64 * i + 16 * t + 8 * h));
            qf[rh][i][4 * h] = v.x, qf[rh][i][4 * h + 1] = v.y, qf[rh][i][4 * h + 2] = v.z, qf[rh][i][4 * h + 3] = v.w;
          }
      }
      if constexpr (BF16) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < C::UNITS; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            amax = fmaxf(amax, fmaxf(fabsf(bf16lo_f32(qf[rh][i][j])), fabsf(bf16hi_f32(qf[rh][i][j]))));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        float mul, back;
        q_f16_scale(amax, mul, back);
        qs[rh][0] *= __shfl_sync(0xffffffffu, back, 8 * t);
        qs[rh][1] *= __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < C::UNITS; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            qf[rh][i][j] = pack_f16x2(bf16lo_f32(qf[rh][i][j]) * mul, bf16hi_f32(qf[rh][i][j]) * mul);
      }
    }
    const int order_g = kOrder[g];
    const int krow = 16 * warp + order_g;                             // chunk rows krow, krow + 8: this thread's scores
    const int srow = krow + (p.page_size == 16 ? 16 * warp : 0);      // ... and scales: 16-row pages take 32 floats each
    int vrow[4];                                                      // chunk rows of its V codes
#pragma unroll
    for (int u = 0; u < 4; ++u) vrow[u] = 16 * warp + 8 * (u >> 1) + kOrder[2 * t + (u & 1)];

    float acc[RH][8][4];
    float m[RH][2], l[RH][2];  // m is the same in all lanes of one t; l is this thread's part of the sum
#pragma unroll
    for (int rh = 0; rh < RH; ++rh) {
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[rh][i][0] = acc[rh][i][1] = acc[rh][i][2] = acc[rh][i][3] = 0.f;
      m[rh][0] = m[rh][1] = -INFINITY, l[rh][0] = l[rh][1] = 0.f;
    }
    bool ok = true;

    for (int c = 0; c < nchunks; ++c) {
      const int s = c % ST;
      if (!mbar_wait_warp(&full[s], (c / ST) & 1, abort_flag, p.status)) {
        ok = false;
        break;
      }
      const uint8_t* kS = smem + s * C::CODES;
      const uint8_t* vS = kS + C::KBOX * kF8Box;
      const float* sc_s = scales + s * 256;
      const int left = end - (start + c * kF8Chunk);  // rows of the chunk before kv_len
      uint4 kr[2][C::UNITS], vr[4];
      float ks[2], lvs[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ks[h] = sc_s[srow + 8 * h];
        lvs[h] = sc_s[128 + srow + 8 * h];
#pragma unroll
        for (int i = 0; i < C::UNITS; ++i) kr[h][i] = lds16(kS + (i >> 1) * kF8Box, krow + 8 * h, (i & 1) * 4 + t);
      }
      auto load_v = [&]() {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 x = lds16(vS, vrow[u], order_g);
          vr[u] = vrow[u] < left ? x : make_uint4(0u, 0u, 0u, 0u);  // rows past kv_len may hold anything
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);  // everything is in registers: the stage may refill
      };
      if constexpr (!WIDE) load_v();  // two tiles of heads leave no registers for V's codes yet

      float sc[RH][CH][4];
#pragma unroll
      for (int rh = 0; rh < RH; ++rh)
#pragma unroll
        for (int e = 0; e < CH; ++e) sc[rh][e][0] = sc[rh][e][1] = sc[rh][e][2] = sc[rh][e][3] = 0.f;
#pragma unroll
      for (int i = 0; i < C::UNITS; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x4(word_of(kr[0][i], w), a0, a2);
          e4m3x4_to_f16x4(word_of(kr[1][i], w), a1, a3);
#pragma unroll
          for (int rh = 0; rh < RH; ++rh)
            mma_f16_16816(sc[rh][w % CH], a0, a1, a2, a3, qf[rh][i][2 * w], qf[rh][i][2 * w + 1]);
        }
      if constexpr (WIDE) load_v();
#pragma unroll
      for (int h = 0; h < 2; ++h) lvs[h] = fmaxf(lg2(lvs[h]), kMinLog2Scale);
      float x[RH][4], y[RH][4];  // [2 h + e]: key h, head e
      bool need = false;
#pragma unroll
      for (int rh = 0; rh < RH; ++rh)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          x[rh][u] = (CH == 1 ? sc[rh][0][u] : sc[rh][0][u] + sc[rh][CH - 1][u]) * qs[rh][u & 1] * ks[u >> 1];
          y[rh][u] = x[rh][u] + lvs[u >> 1];
          if (krow + 8 * (u >> 1) >= left) x[rh][u] = y[rh][u] = -INFINITY;
          need |= y[rh][u] > m[rh][u & 1] + kRescaleLog2F8;
        }
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int rh = 0; rh < RH; ++rh)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mb = fmaxf(y[rh][e], y[rh][2 + e]);
#pragma unroll
            for (int d = 4; d < 32; d *= 2) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, d));
            mb = fmaxf(mb, m[rh][e]);
            const float alpha = (mb == -INFINITY) ? 1.f : ex2(m[rh][e] - mb);
            l[rh][e] *= alpha;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[rh][i][e] *= alpha, acc[rh][i][2 + e] *= alpha;
            m[rh][e] = mb;
          }
      }
      uint32_t pt[RH][2];  // P^T (B operand): keys 2t, 2t + 1 (+ 8) of head g
#pragma unroll
      for (int rh = 0; rh < RH; ++rh) {
        float neg_m[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          neg_m[e] = (m[rh][e] == -INFINITY) ? 0.f : -m[rh][e];
          l[rh][e] += ex2(x[rh][e] + neg_m[e]) + ex2(x[rh][2 + e] + neg_m[e]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          pt[rh][h] = movmatrix_trans(pack_f16x2(ex2(y[rh][2 * h] + neg_m[0]), ex2(y[rh][2 * h + 1] + neg_m[1])));
      }
      // O^T += V^T P^T: bytes of two keys interleaved, so that one conversion gives an A register
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t sel = h ? 0x7362u : 0x5140u;
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x4(byte_perm(word_of(vr[0], w), word_of(vr[1], w), sel), a0, a1);
          e4m3x4_to_f16x4(byte_perm(word_of(vr[2], w), word_of(vr[3], w), sel), a2, a3);
#pragma unroll
          for (int rh = 0; rh < RH; ++rh) mma_f16_16816(acc[rh][2 * w + h], a0, a1, a2, a3, pt[rh][0], pt[rh][1]);
        }
    }

#pragma unroll
    for (int rh = 0; rh < RH; ++rh)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[rh][e] += __shfl_xor_sync(0xffffffffu, l[rh][e], d);
        if (!ok) {
          m[rh][e] = -INFINITY;
          l[rh][e] = 0.f;
        }
      }
    // merge the four warps: per-warp O goes to the (now idle) ring memory
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(kDecodeWarps * 32));
    float* sm_o = reinterpret_cast<float*>(smem);  // [warp][head][dv]
#pragma unroll
    for (int rh = 0; rh < RH; ++rh)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int head = 2 * t + e + 8 * rh;
        if (head < G) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float2*>(sm_o + (warp * R + head) * kDecodeDv + 16 * order_g + 2 * i) =
                make_float2(acc[rh][i][e], acc[rh][i][2 + e]);
          if (g == 0) {
            sm_m[warp][head] = m[rh][e];
            sm_l[warp][head] = l[rh][e];
          }
        }
      }
    asm volatile("bar.sync 1, %0;" ::"n"(kDecodeWarps * 32));
    const int dv = threadIdx.x;  // kDecodeWarps * 32 == kDecodeDv
    for (int r = 0; r < G; ++r) {
      float M = -INFINITY;
#pragma unroll
      for (int wi = 0; wi < kDecodeWarps; ++wi) M = fmaxf(M, sm_m[wi][r]);
      float o = 0.f, ls = 0.f;
#pragma unroll
      for (int wi = 0; wi < kDecodeWarps; ++wi) {
        const float mw = sm_m[wi][r];
        const float e = (mw == -INFINITY) ? 0.f : ex2(mw - M);
        o += e * sm_o[(wi * R + r) * kDecodeDv + dv];
        ls += e * sm_l[wi][r];
      }
      const int h = kvh * G + r;
      float* part = p.ws + (static_cast<int64_t>(b * p.Hq + h) * p.n_splits_max + split) * (kDecodeDv + 2);
      part[dv] = o;
      if (dv == 0) {
        part[kDecodeDv] = M;
        part[kDecodeDv + 1] = ls;
      }
    }
  }
}

template <bool BF16, int D, bool WIDE>
cudaError_t launch_f8_instance(const DecodeParams& p, const CUtensorMap (&tm)[4], cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  static std::atomic<uint64_t> opted{0};
  auto kern = decode_f8_split_kernel<BF16, D, WIDE>;
  if ((e = smem_opt_in(kern, DecF8Cfg<D>::SMEM, dev, opted)) != cudaSuccess) return e;
  kern<<<dim3(p.n_splits_max, p.Hkv, p.B), kF8Threads, DecF8Cfg<D>::SMEM, st>>>(tm[0], tm[1], tm[2], tm[3], p);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t launch_f8(int D, const DecodeParams& p, const CUtensorMap (&tm)[4], cudaStream_t st) {
  const bool wide = p.group > 8;
  if (D == 192)
    return wide ? launch_f8_instance<BF16, 192, true>(p, tm, st) : launch_f8_instance<BF16, 192, false>(p, tm, st);
  return wide ? launch_f8_instance<BF16, 128, true>(p, tm, st) : launch_f8_instance<BF16, 128, false>(p, tm, st);
}

// Keys per split: the largest of 2048 .. 256 that gives every SM of the card two CTAs (304), or
// 256.  Longer splits write fewer partials and start fewer CTAs (the batch above: 4096 cost
// 4 us more, 1024 14, 512 44); a few short sequences need more CTAs than that gives.  The lengths are on the
// device, so max_kv stands for them: a page table wider than they need gives longer splits than they would take, and
// CTAs without keys (3 sequences of 3000 rows, 32 / 4 heads: 9 us with a tight table, 10 with one 8 times as wide,
// 21 with one for 131072 rows; 64 sequences of 4000 rows, 32 / 8 heads: 101, 116, 145).
int f8_log2_split(int B, int Hkv, int max_kv) {
  int log2 = 11;  // 2048
  while ((1 << log2) > kF8MinSplit &&
         static_cast<long long>(B) * Hkv * ((max_kv + (1 << log2) - 1) >> log2) < 304)
    --log2;
  return log2;
}

size_t f8_partials_bytes(int B, int Hq, int Hkv, int max_kv, int Dv) {
  const int log2 = f8_log2_split(B, Hkv, max_kv);
  const size_t n = static_cast<size_t>((max_kv + (1 << log2) - 1) >> log2);
  return split_round16(static_cast<size_t>(B) * Hq * n * static_cast<size_t>(Dv + 2) * sizeof(float));
}

}  // namespace

}  // namespace sdpa

using namespace sdpa;

extern "C" {

size_t sdpa_decode_paged_fp8_workspace_size(int B, int Hq, int Hkv, int max_kv, int Dv) {
  if (B < 1 || Hq < 1 || Hkv < 1 || max_kv < 1 || Dv < 1 || max_kv > (1 << 30)) return 0;
  return f8_partials_bytes(B, Hq, Hkv, max_kv, Dv);
}

int sdpa_decode_paged_fp8(const void* q, const void* k_pool, const void* v_pool, const float* k_scale,
                          const float* v_scale, const int32_t* page_table, const int32_t* kv_len, void* o, float* lse,
                          int B, int Hq, int Hkv, int page_size, int max_pages, int n_pages, int D, int Dv,
                          const int64_t* strides, float scale, void* workspace, size_t workspace_bytes,
                          sdpa_dtype dtype, void* stream) {
  if (!page_table || !k_scale || !v_scale) return SDPA_ERR_INVALID;
  int rc = page_check(page_size, max_pages, n_pages);
  if (rc != SDPA_OK) return rc;
  const int max_kv = max_pages * page_size;
  DecodeCall call;
  rc = decode_check(q, k_pool, v_pool, page_table, kv_len, o, lse, B, Hq, Hkv, max_kv, page_size, max_pages, n_pages, D,
                    Dv, strides, scale, dtype, &call);
  if (rc != SDPA_OK) return rc;
  DecodeParams& p = call.p;
  const int64_t pool_strides[6] = {p.k_b, p.k_s, p.k_h, p.v_b, p.v_s, p.v_h};
  for (int64_t s : pool_strides)
    if (!stride_ok(s, 16)) return SDPA_ERR_UNSUPPORTED;
  if (!aligned16(k_scale) || !aligned16(v_scale)) return SDPA_ERR_UNSUPPORTED;
  if (!workspace || !aligned16(workspace) || workspace_bytes < f8_partials_bytes(B, Hq, Hkv, max_kv, Dv))
    return SDPA_ERR_INVALID;
  p.log2_split = f8_log2_split(B, Hkv, max_kv);
  p.n_splits_max = (max_kv + (1 << p.log2_split) - 1) >> p.log2_split;
  p.ws = static_cast<float*>(workspace);

  alignas(64) CUtensorMap tm[4];
  const int rows = std::min(kF8Chunk, page_size);
  if (!encode_bshd(&tm[0], k_pool, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, n_pages, page_size, Hkv, D, p.k_b, p.k_s, p.k_h,
                   128, rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_bshd(&tm[1], v_pool, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, n_pages, page_size, Hkv, Dv, p.v_b, p.v_s, p.v_h,
                   128, rows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_scales(&tm[2], k_scale, n_pages, Hkv, page_size, rows) ||
      !encode_scales(&tm[3], v_scale, n_pages, Hkv, page_size, rows))
    return SDPA_ERR_CUDA;
  if (device_status_ptr(&p.status) != cudaSuccess) return SDPA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = call.elem == kBF16 ? launch_f8<true>(D, p, tm, st) : launch_f8<false>(D, p, tm, st);
  if (e == cudaSuccess) e = launch_decode_combine(call.elem, p, st);
  return e == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

}  // extern "C"
