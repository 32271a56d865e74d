// Rotary positions for sm_103a: queries and keys turned by their positions, and the rows of a latent
// cache (a token's latent vector beside the rotary key that all heads share) turned as they are written
// into their pages.
//
// Pair i of a head is turned by the angle position * inv_freq[i]:
//     (a, b) -> factor * (a cos - b sin, b cos + a sin),
// in fp32, rounded once.  Far into a long context the angle passes 10^6 radians, where fp32 holds it to
// 0.06; so it is taken in turns, as a 64-bit fraction: inv_freq / 2 pi is the 24-bit significand times 66
// bits of 1 / 2 pi, and the product with the position is a 64-bit multiplication whose overflow drops
// whole turns.  What is lost is 2^-64 of the angle and 2^-64 turns a position; the fraction's upper 32 bits
// go through sincospif.  That costs three integer multiplications a pair, against five fp64
// instructions at a rate of two a cycle and SM.
//
// Both kernels are bound by memory: 32767 tokens of 32 heads of 128 are turned in 84 us (537 MB, 6.4 TB/s; 32768 tokens of 40
// heads, all dims, 104), 66,000 latent rows written in 26 (153 MB, 5.8 TB/s), a decode step's 64 tokens in 4 and 3 us (in a
// graph).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "sdpa.h"
#include "internal.h"
#include "ptx.cuh"
#include "rows16.cuh"

namespace sdpa {

namespace {

constexpr int kRopeThreads = 128;

// cos and sin of position * inv_freq, times factor.  inv_freq of 2^25 and above, infinite or NaN: NaN.
struct Turn {
  float c, s;
};
__device__ __forceinline__ Turn turn_at(float inv_freq, int pos, float factor) {
  const uint32_t bits = __float_as_uint(inv_freq);
  const int ex = static_cast<int>(bits >> 23) & 255;
  // inv_freq = m 2^(e - 150), e = ex (1 for subnormals); 1 / 2 pi = kInv2Pi 2^-66
  constexpr uint64_t kInv2Pi = 0xA2F9836E4E44152Aull;
  const uint64_t m = (bits & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
  const int shift = 152 - max(ex, 1);  // turns a position in units of 2^-64: (m kInv2Pi) >> shift
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  uint64_t step = shift >= 64 ? (shift >= 128 ? 0ull : hi >> (shift - 64)) : shift > 0 ? (lo >> shift) | (hi << (64 - shift)) : lo;
  if (bits >> 31) step = 0ull - step;
  const uint64_t phase = step * static_cast<uint64_t>(static_cast<int64_t>(pos));
  Turn t;
  sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &t.s, &t.c);
  if (shift <= 0) t.c = t.s = __uint_as_float(0x7FC00000u);
  t.c *= factor, t.s *= factor;
  return t;
}

// (a, b) turned
__device__ __forceinline__ void turn_pair(float& a, float& b, const Turn& t) {
  const float x = a * t.c - b * t.s;
  b = b * t.c + a * t.s;
  a = x;
}

struct RopeParams {
  const uint16_t *q, *k;
  uint16_t *qo, *ko;
  const int32_t* positions;
  const float* inv_freq;
  int64_t q_s, q_h, k_s, k_h, qo_s, qo_h, ko_s, ko_h;
  int total, Hq, H;        // H: heads of q and k together
  int half;                // pairs of a head
  int units, turn_units;   // units of a head's row; those that turn
  int lanes;               // threads that share the heads of a (token, unit)
  int copy_q, copy_k;      // the dims that are not turned are copied
  float factor;
  FastDiv div_units, div_lanes;
};

// Heads whose loads are in flight together, twice over, as the next batch is loaded while one is turned (in us, the two
// cases above: without that 103 and 112; batches of four 90 and 112, blocks of 256 threads 87 and 106).
constexpr int kRopeBatch = 2;
// Threads that keep the SMs busy at all, and those that many heads are spread over (32767 x 32 heads, 4096 tokens x 129 heads of
// 192: one thread a token's unit 115 and 108 us, 152 * 4096 threads 101 and 81, 152 * 32768 122 and 104, before the double batch).
constexpr long long kRopeBusy = 152 * 1024, kRopeFull = 152 * 4096;

// A thread keeps one unit of a head's row (half pairs: vectors i and i + half; interleaved: one vector;
// behind the turned dims a vector that is copied) and the angles of its pairs for every lanes-th head.
template <bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  constexpr int NV = INTERLEAVED ? 1 : 2;
  const uint32_t g = blockIdx.x * kRopeThreads + threadIdx.x;
  const uint32_t rest = fast_div(g, p.div_units);
  const int unit = static_cast<int>(g - rest * p.units);
  const int tok = static_cast<int>(fast_div(rest, p.div_lanes));
  const int h0 = static_cast<int>(rest) - tok * p.lanes;
  if (tok >= p.total) return;
  const bool turns = unit < p.turn_units;
  const int d0 = turns ? 8 * unit : 2 * p.half + 8 * (unit - p.turn_units);
  const int d1 = d0 + p.half;  // the pairs' second vector (half layout)
  const uint16_t* q = p.q + tok * p.q_s;
  const uint16_t* k = p.k + tok * p.k_s;
  uint16_t* qo = p.qo + tok * p.qo_s;
  uint16_t* ko = p.ko + tok * p.ko_s;
  uint4 x[kRopeBatch][NV], next[kRopeBatch][NV];
  auto load = [&](uint4 (&x)[kRopeBatch][NV], int h) {
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i, h += p.lanes) {
      if (h >= p.H || !(turns || (h < p.Hq ? p.copy_q : p.copy_k))) continue;
      const uint16_t* row = h < p.Hq ? q + h * p.q_h : k + (h - p.Hq) * p.k_h;
      x[i][0] = *reinterpret_cast<const uint4*>(row + d0);
      if (!INTERLEAVED && turns) x[i][NV - 1] = *reinterpret_cast<const uint4*>(row + d1);
    }
  };
  load(x, h0);
  Turn t[INTERLEAVED ? 4 : 8];
  if (turns) {
    const int pos = __ldg(p.positions + tok);
#pragma unroll
    for (int i = 0; i < (INTERLEAVED ? 4 : 8); ++i) t[i] = turn_at(__ldg(p.inv_freq + (INTERLEAVED ? 4 : 8) * unit + i), pos, p.factor);
  }
  for (int h = h0; h < p.H; h += kRopeBatch * p.lanes) {
    load(next, h + kRopeBatch * p.lanes);  // while this batch is turned
    int hs = h;
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i, hs += p.lanes) {
      if (hs >= p.H || !(turns || (hs < p.Hq ? p.copy_q : p.copy_k))) continue;
      uint16_t* row = hs < p.Hq ? qo + hs * p.qo_h : ko + (hs - p.Hq) * p.ko_h;
      if (turns) {
        float a[8];
        unpack8<BF16>(x[i][0], a);
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int j = 0; j < 4; ++j) turn_pair(a[2 * j], a[2 * j + 1], t[j]);
        } else {
          float b[8];
          unpack8<BF16>(x[i][NV - 1], b);
#pragma unroll
          for (int j = 0; j < 8; ++j) turn_pair(a[j], b[j], t[j]);
          *reinterpret_cast<uint4*>(row + d1) = pack8<BF16>(b);
        }
        x[i][0] = pack8<BF16>(a);
      }
      *reinterpret_cast<uint4*>(row + d0) = x[i][0];
    }
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i)
#pragma unroll
      for (int v = 0; v < NV; ++v) x[i][v] = next[i][v];
  }
}

struct LatentWriteParams {
  const uint16_t *c, *r;
  uint16_t* pool;
  const int64_t* slots;
  const int32_t* positions;  // null: the rotary part is stored as it is
  const float* inv_freq;
  uint32_t* status;
  int64_t c_s, r_s, p_page, p_row;
  int64_t n_slots;
  int total, log2_page;
  float factor;
};

constexpr int kWriteThreads = 256;
constexpr int kWriteTokens = 16;  // a block's latent vectors: four 16-byte vectors a thread
constexpr int kTurnTokens = 32;   // a block's rotary parts: four pairs a thread
static_assert(kTurnTokens == 2 * kWriteTokens, "two blocks of vectors to one of rotary parts");

// Of three blocks two copy latent vectors, the third turns the rotary parts beside them (in one block the copies of some
// warps waited for their angles: 66,000 rows 28.9 -> 28.1 us; what is read once leaving the L2 first, 26.2 us).
template <bool BF16, bool INTERLEAVED>
__global__ void __launch_bounds__(kWriteThreads) latent_write_kernel(const LatentWriteParams p) {
  auto slot_row = [&](int64_t slot) {
    return p.pool + (slot >> p.log2_page) * p.p_page + (slot & ((int64_t(1) << p.log2_page) - 1)) * p.p_row;
  };
  const int group = blockIdx.x / 3, role = blockIdx.x - 3 * group;
  if (role < 2) {
    constexpr int VECS = kLatentDim / 8, REPS = kWriteTokens * VECS / kWriteThreads;
    const int t0 = (2 * group + role) * kWriteTokens + threadIdx.x / VECS, v = threadIdx.x % VECS;
    uint4 x[REPS];
    int64_t slot[REPS];
#pragma unroll
    for (int i = 0; i < REPS; ++i) {
      const int tok = t0 + i * (kWriteThreads / VECS);
      slot[i] = -1;
      if (tok < p.total) {
        slot[i] = __ldg(p.slots + tok);
        x[i] = __ldcs(reinterpret_cast<const uint4*>(p.c + tok * p.c_s) + v);
      }
    }
#pragma unroll
    for (int i = 0; i < REPS; ++i)
      if (slot[i] >= 0 && slot[i] < p.n_slots) reinterpret_cast<uint4*>(slot_row(slot[i]))[v] = x[i];
    return;
  }
  const int tok = group * kTurnTokens + threadIdx.x / 8, u = threadIdx.x % 8;
  if (tok >= p.total) return;
  // pairs 4 u .. 4 u + 3: dims 8 u .. + 7 (interleaved), or 4 u .. + 3 and 32 + 4 u .. + 3
  const int64_t slot = __ldg(p.slots + tok);
  const uint16_t* src = p.r + tok * p.r_s;
  const int d0 = INTERLEAVED ? 8 * u : 4 * u, d1 = INTERLEAVED ? d0 + 4 : d0 + kLatentRot / 2;
  const uint2 lo = __ldg(reinterpret_cast<const uint2*>(src + d0)), hi = __ldg(reinterpret_cast<const uint2*>(src + d1));
  if (slot < 0) return;
  if (slot >= p.n_slots) {
    atomicOr(p.status, kStatusBadSeqlens);  // behind the pool
    return;
  }
  uint4 w = make_uint4(lo.x, lo.y, hi.x, hi.y);
  if (p.positions != nullptr) {
    const int pos = __ldg(p.positions + tok);
    float a[8];
    unpack8<BF16>(w, a);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const Turn t = turn_at(__ldg(p.inv_freq + 4 * u + j), pos, p.factor);
      if constexpr (INTERLEAVED)
        turn_pair(a[2 * j], a[2 * j + 1], t);
      else
        turn_pair(a[j], a[4 + j], t);
    }
    w = pack8<BF16>(a);
  }
  uint16_t* dst = slot_row(slot) + kLatentDim;
  *reinterpret_cast<uint2*>(dst + d0) = make_uint2(w.x, w.y);
  *reinterpret_cast<uint2*>(dst + d1) = make_uint2(w.z, w.w);
}

}  // namespace

}  // namespace sdpa

using namespace sdpa;

extern "C" {

int sdpa_rope(const void* q, const void* k, void* q_out, void* k_out, const int32_t* positions, const float* inv_freq,
              int total, int Hq, int Hk, int D, int rotary_dim, int interleaved, float factor, const int64_t* strides,
              sdpa_dtype dtype, void* stream) {
  // ---- validation (no CUDA call before this block passes)
  if (!q || !q_out || !positions || !inv_freq || (Hk > 0 && (!k || !k_out))) return SDPA_ERR_INVALID;
  if (total < 1 || Hq < 1 || Hk < 0 || D < 1 || rotary_dim < 1 || rotary_dim > D || !std::isfinite(factor)) return SDPA_ERR_INVALID;
  if (dtype != SDPA_F16 && dtype != SDPA_BF16) return SDPA_ERR_UNSUPPORTED;
  if (D % 8 != 0 || rotary_dim % (interleaved ? 8 : 16) != 0 || static_cast<long long>(Hq) + Hk > kMaxCount) return SDPA_ERR_UNSUPPORTED;
  int64_t st[SDPA_ROPE_NSTRIDES] = {(int64_t)Hq * D, D, (int64_t)Hk * D, D, (int64_t)Hq * D, D, (int64_t)Hk * D, D};
  if (strides) std::memcpy(st, strides, sizeof(st));
  for (int i = 0; i < SDPA_ROPE_NSTRIDES; ++i)
    if (!stride_ok(st[i], 8)) return SDPA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out)) return SDPA_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(inv_freq)) & 3u) return SDPA_ERR_INVALID;
  // an output's rows are places of their own
  if (rows_coincide(total, st[4]) || rows_coincide(Hq, st[5]) || (Hk > 0 && rows_coincide(total, st[6])) || rows_coincide(Hk, st[7]))
    return SDPA_ERR_INVALID;
  // in place: the rows have to lie alike
  if ((q == q_out && (st[0] != st[4] || st[1] != st[5])) || (Hk > 0 && k == k_out && (st[2] != st[6] || st[3] != st[7])))
    return SDPA_ERR_INVALID;

  RopeParams p{};
  p.q = static_cast<const uint16_t*>(q), p.k = static_cast<const uint16_t*>(Hk > 0 ? k : q);
  p.qo = static_cast<uint16_t*>(q_out), p.ko = static_cast<uint16_t*>(Hk > 0 ? k_out : q_out);
  p.positions = positions, p.inv_freq = inv_freq;
  p.q_s = st[0], p.q_h = st[1], p.k_s = st[2], p.k_h = st[3];
  p.qo_s = st[4], p.qo_h = st[5], p.ko_s = st[6], p.ko_h = st[7];
  p.total = total, p.Hq = Hq, p.H = Hq + Hk, p.half = rotary_dim / 2;
  p.copy_q = q != q_out, p.copy_k = Hk > 0 && k != k_out;
  p.turn_units = rotary_dim / (interleaved ? 8 : 16);
  p.units = p.turn_units + (p.copy_q || p.copy_k ? (D - rotary_dim) / 8 : 0);
  p.factor = factor;
  // A token's heads are shared by as many threads as keep the SMs busy, but a thread that has a batch of heads to itself
  // computes its angles once for them.
  const long long rows = static_cast<long long>(total) * p.units;
  const long long busy = (kRopeBusy + rows - 1) / rows, full = (kRopeFull + rows - 1) / rows, batches = (p.H + kRopeBatch - 1) / kRopeBatch;
  p.lanes = static_cast<int>(std::min<long long>(p.H, std::max(busy, std::min(full, batches))));
  if (rows * p.lanes >= (1ll << 31)) return SDPA_ERR_UNSUPPORTED;
  p.div_units = make_fastdiv(static_cast<uint32_t>(p.units));
  p.div_lanes = make_fastdiv(static_cast<uint32_t>(p.lanes));
  const unsigned grid = static_cast<unsigned>((rows * p.lanes + kRopeThreads - 1) / kRopeThreads);
  const bool bf16 = dtype == SDPA_BF16;
  auto kern = interleaved ? (bf16 ? rope_kernel<true, true> : rope_kernel<false, true>)
                          : (bf16 ? rope_kernel<true, false> : rope_kernel<false, false>);
  kern<<<grid, kRopeThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

int sdpa_latent_write(const void* c, const void* k_rope, void* pool, const int64_t* slots, const int32_t* positions,
                      const float* inv_freq, int total, int page_size, int n_pages, int latent_dim, int rotary_dim,
                      int interleaved, float factor, const int64_t* strides, sdpa_dtype dtype, void* stream) {
  // ---- validation (no CUDA call before this block passes)
  if (!c || !k_rope || !pool || !slots || (positions == nullptr) != (inv_freq == nullptr)) return SDPA_ERR_INVALID;
  if (total < 1 || latent_dim < 1 || rotary_dim < 1 || !std::isfinite(factor)) return SDPA_ERR_INVALID;
  const int rc = page_check(page_size, 1, n_pages);
  if (rc != SDPA_OK) return rc;
  if (dtype != SDPA_F16 && dtype != SDPA_BF16) return SDPA_ERR_UNSUPPORTED;
  if (latent_dim != kLatentDim || rotary_dim != kLatentRot || total > kMaxCount) return SDPA_ERR_UNSUPPORTED;
  int64_t st[SDPA_LATENT_WRITE_NSTRIDES] = {kLatentDim, kLatentRot, (int64_t)page_size * kLatentRow, kLatentRow};
  if (strides) std::memcpy(st, strides, sizeof(st));
  for (int i = 0; i < SDPA_LATENT_WRITE_NSTRIDES; ++i)
    if (!stride_ok(st[i], 8)) return SDPA_ERR_UNSUPPORTED;
  if (rows_coincide(n_pages, st[2]) || rows_coincide(page_size, st[3])) return SDPA_ERR_INVALID;
  if (!aligned16(c) || !aligned16(k_rope) || !aligned16(pool)) return SDPA_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(slots) & 7u) ||
      ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(inv_freq)) & 3u))
    return SDPA_ERR_INVALID;

  LatentWriteParams p{};
  p.c = static_cast<const uint16_t*>(c), p.r = static_cast<const uint16_t*>(k_rope);
  p.pool = static_cast<uint16_t*>(pool);
  p.slots = slots, p.positions = positions, p.inv_freq = inv_freq;
  p.c_s = st[0], p.r_s = st[1], p.p_page = st[2], p.p_row = st[3];
  p.total = total, p.log2_page = __builtin_ctz((unsigned)page_size);
  p.n_slots = static_cast<int64_t>(n_pages) << p.log2_page;
  p.factor = factor;
  if (device_status_ptr(&p.status) != cudaSuccess) return SDPA_ERR_CUDA;
  const bool bf16 = dtype == SDPA_BF16;
  auto kern = interleaved ? (bf16 ? latent_write_kernel<true, true> : latent_write_kernel<false, true>)
                          : (bf16 ? latent_write_kernel<true, false> : latent_write_kernel<false, false>);
  const unsigned grid = 3 * ((static_cast<unsigned>(total) + kTurnTokens - 1) / kTurnTokens);
  kern<<<grid, kWriteThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

}  // extern "C"
