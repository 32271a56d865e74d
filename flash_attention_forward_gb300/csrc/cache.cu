// Quantised paged K/V cache for sm_103a: new tokens' K and V rounded to e4m3 codes as they are
// written into their pages, and cached rows read back as packed 16-bit tensors.
//
// One row is the D (or Dv) values of one (token, KV head).  Its scale is the least power of two
// 2^k that keeps the row within e4m3's range, amax <= 448 * 2^k, so
//     code = e4m3(x * 2^-k),   value = code * 2^k,
// the scaling is exact and the only rounding is that of the code (3 mantissa bits, half a step is
// 2^-4 relative).  A scale of amax / 448 would round twice and gain nothing: a floating-point code
// has the same relative step wherever in its range a value lies.  k >= -80 (rows of zeros take it):
// the attention kernels hold 1 / scale in fp32.  NaN stays NaN and does not move the scale; a row
// with an infinity gets 2^120, from which the infinity reads back as one (448 * 2^120 is none of fp32's
// values), entries of at most 2^110 as zeros and larger ones as they are rounded.  From 1.9375 * 2^127 on, where
// the rounding reaches 2^128, finite values read back as infinities too.
//
// Both kernels are bound by memory: 3 (D + Dv) + 8 bytes move per row of K and V against some 40
// instructions per 8 values.  66,000 tokens of 8 heads of 128 are written in 68 us (6.1 TB/s: 271 MB read,
// 135 MB of codes and 4 MB of scales written), 139,000 read back in 131 (6.6 TB/s), both in a graph.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sdpa.h"
#include "internal.h"
#include "ptx.cuh"

namespace sdpa {

namespace {

constexpr int kCacheThreads = 128;

// The rows of K and V ((token, KV head), token major) are taken kLanes threads at a time, eight
// values a thread; a block takes REPS passes of kCacheThreads / LANES rows.  4 x 128 threads wrote the
// tokens above in 76 us, 2 x 256 in 82, 8 x 128 in 81, all before the scales' joint stores, which took 4 us off.
template <int D, int DV>
struct CacheCfg {
  static constexpr int LANES = D > 128 ? 32 : D / 8;  // a power of two; 8 of the 32 idle for D = 192
  static constexpr int ROWS = kCacheThreads / LANES;  // rows a pass
  static constexpr int REPS = 4;                      // passes, all their loads in flight together
  static constexpr int BLOCK_ROWS = ROWS * REPS;
  static_assert(DV <= D && 8 * LANES >= D, "one group of lanes holds a row");
};

// Cache slot of packed row r: sequence b by binary search in cu (any values keep the search inside
// cu[0 .. B]), position pos of the row in it, then the page.  first = kv_len - length for the
// writer (the rows are the last of the sequence), 0 for the reader (kv_len null).
struct Slot {
  int page;  // physical page, or < 0: no slot
  int row;   // row in the page
};
constexpr int kNoRow = -1;    // r belongs to no sequence: nothing is written
constexpr int kBadSlot = -2;  // outside the table or the pool: reported

__device__ __forceinline__ Slot cache_slot(const CacheParams& p, int r) {
  Slot s{kNoRow, 0};
  int lo = 0, hi = p.B;  // cu[lo] <= r < cu[hi] where the offsets are sorted
  if (r < __ldg(p.cu) || r >= __ldg(p.cu + p.B)) return s;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu + mid) <= r) lo = mid; else hi = mid;
  }
  const int c0 = __ldg(p.cu + lo), c1 = __ldg(p.cu + lo + 1);
  s.page = kBadSlot;
  if (r < c0 || r >= c1) return s;  // unsorted offsets
  long long pos = static_cast<long long>(r) - c0;
  if (p.kv_len != nullptr) pos += static_cast<long long>(__ldg(p.kv_len + lo)) - (static_cast<long long>(c1) - c0);
  if (pos < 0 || pos >= (static_cast<long long>(p.max_pages) << p.log2_page)) return s;
  const int phys = __ldg(p.page_table + lo * p.pt_b + (pos >> p.log2_page));
  if (phys < 0 || phys >= p.n_pages) return s;
  s.page = phys;
  s.row = static_cast<int>(pos) & ((1 << p.log2_page) - 1);
  return s;
}

// The block's rows span at most BLOCK_ROWS tokens: one thread finds each token's slot.
template <int BLOCK_ROWS>
__device__ __forceinline__ void block_slots(const CacheParams& p, int row0, int n_rows, Slot (&slots)[BLOCK_ROWS]) {
  const int t0 = static_cast<int>(fast_div(row0, p.div_h));
  const int t1 = static_cast<int>(fast_div(row0 + n_rows - 1, p.div_h));
  for (int i = threadIdx.x; i <= t1 - t0; i += kCacheThreads) {
    const Slot s = cache_slot(p, t0 + i);
    if (s.page == kBadSlot) atomicOr(p.status, kStatusBadSeqlens);
    slots[i] = s;
  }
  __syncthreads();
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      x[2 * i] = bf16lo_f32(w[i]), x[2 * i + 1] = bf16hi_f32(w[i]);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
}

// Exponent k of the row's scale from its largest magnitude m * 2^e (1 <= m < 2): 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int k = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(k, kCacheMinExp);
}
__device__ __forceinline__ float exp2_int(int k) { return __uint_as_float(static_cast<uint32_t>(127 + k) << 23); }

template <bool BF16, int D, int DV>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheParams p) {
  using C = CacheCfg<D, DV>;
  __shared__ Slot slots[C::BLOCK_ROWS];
  __shared__ float scales[2][C::BLOCK_ROWS];
  const int row0 = blockIdx.x * C::BLOCK_ROWS;
  const int n_rows = min(C::BLOCK_ROWS, p.rows - row0);
  const int t0 = static_cast<int>(fast_div(row0, p.div_h));
  const int sub = threadIdx.x / C::LANES, lane = threadIdx.x % C::LANES;
  // the source rows do not depend on the slots: their loads are in flight while those are found
  uint4 raw[C::REPS][2];
  int tok[C::REPS], head[C::REPS];
#pragma unroll
  for (int i = 0; i < C::REPS; ++i) {
    const int rr = row0 + i * C::ROWS + sub;
    tok[i] = static_cast<int>(fast_div(min(rr, p.rows - 1), p.div_h));
    head[i] = min(rr, p.rows - 1) - tok[i] * p.Hkv;
    raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
    if (i * C::ROWS + sub < n_rows) {
      if (8 * lane < D)
        raw[i][0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.k) + tok[i] * p.k_s +
                                                         head[i] * p.k_h + 8 * lane));
      if (8 * lane < DV)
        raw[i][1] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.v) + tok[i] * p.v_s +
                                                         head[i] * p.v_h + 8 * lane));
    }
  }
  block_slots(p, row0, n_rows, slots);
#pragma unroll
  for (int i = 0; i < C::REPS; ++i) {
    float x[2][8], amax[2] = {0.f, 0.f};
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      unpack8<BF16>(raw[i][kv], x[kv]);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax[kv] = fmaxf(amax[kv], fabsf(x[kv][j]));
    }
#pragma unroll
    for (int d = C::LANES / 2; d > 0; d >>= 1) {
      amax[0] = fmaxf(amax[0], __shfl_xor_sync(0xffffffffu, amax[0], d));
      amax[1] = fmaxf(amax[1], __shfl_xor_sync(0xffffffffu, amax[1], d));
    }
    if (i * C::ROWS + sub >= n_rows) continue;
    const Slot s = slots[tok[i] - t0];
    if (s.page < 0) continue;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const int k = scale_exponent(amax[kv]);
      const float inv = exp2_int(-k);
      uint8_t* dst = kv == 0 ? p.k_pool + s.page * p.kp_p + s.row * p.kp_r + head[i] * p.kp_h
                             : p.v_pool + s.page * p.vp_p + s.row * p.vp_r + head[i] * p.vp_h;
      if (8 * lane < (kv == 0 ? D : DV)) {
        const float* f = x[kv];
        *reinterpret_cast<uint2*>(dst + 8 * lane) =
            make_uint2(pack_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                       pack_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
      }
      if (lane == 0) scales[kv][i * C::ROWS + sub] = exp2_int(k);
    }
  }
  // The scales of a head's tokens are neighbours: written by one warp, they share sectors.
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * C::BLOCK_ROWS; i += kCacheThreads) {
    const int kv = i / C::BLOCK_ROWS, rr = i % C::BLOCK_ROWS;
    if (rr >= n_rows) continue;
    const int t = static_cast<int>(fast_div(row0 + rr, p.div_h));
    const Slot s = slots[t - t0];
    if (s.page < 0) continue;
    const int64_t at = static_cast<int64_t>(s.page) * p.Hkv + (row0 + rr - t * p.Hkv);
    (kv == 0 ? p.k_scale : p.v_scale)[(at << p.log2_page) + s.row] = scales[kv][rr];
  }
}

template <bool BF16, int D, int DV>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheParams p) {
  using C = CacheCfg<D, DV>;
  __shared__ Slot slots[C::BLOCK_ROWS];
  const int row0 = blockIdx.x * C::BLOCK_ROWS;
  const int n_rows = min(C::BLOCK_ROWS, p.rows - row0);
  const int t0 = static_cast<int>(fast_div(row0, p.div_h));
  const int sub = threadIdx.x / C::LANES, lane = threadIdx.x % C::LANES;
  block_slots(p, row0, n_rows, slots);
  uint2 raw[C::REPS][2];
  float sc[C::REPS][2];
  int page[C::REPS];
#pragma unroll
  for (int i = 0; i < C::REPS; ++i) {
    const int rr = row0 + i * C::ROWS + sub;
    page[i] = kNoRow;
    raw[i][0] = raw[i][1] = make_uint2(0u, 0u);
    sc[i][0] = sc[i][1] = 0.f;
    if (i * C::ROWS + sub >= n_rows) continue;
    const int tok = static_cast<int>(fast_div(rr, p.div_h)), head = rr - tok * p.Hkv;
    const Slot s = slots[tok - t0];
    page[i] = s.page;
    if (s.page < 0) continue;  // a bad slot reads as zeros
    if (8 * lane < D)
      raw[i][0] = __ldg(reinterpret_cast<const uint2*>(p.k_pool + s.page * p.kp_p + s.row * p.kp_r + head * p.kp_h +
                                                       8 * lane));
    if (8 * lane < DV)
      raw[i][1] = __ldg(reinterpret_cast<const uint2*>(p.v_pool + s.page * p.vp_p + s.row * p.vp_r + head * p.vp_h +
                                                       8 * lane));
    const int64_t si = ((static_cast<int64_t>(s.page) * p.Hkv + head) << p.log2_page) + s.row;
    sc[i][0] = __ldg(p.k_scale + si), sc[i][1] = __ldg(p.v_scale + si);
  }
#pragma unroll
  for (int i = 0; i < C::REPS; ++i) {
    if (page[i] == kNoRow) continue;
    const int rr = row0 + i * C::ROWS + sub;
    const int tok = static_cast<int>(fast_div(rr, p.div_h)), head = rr - tok * p.Hkv;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      if (8 * lane >= (kv == 0 ? D : DV)) continue;
      const uint4 h = e4m3x8_to_f16x8(raw[i][kv]);
      const uint32_t w[4] = {h.x, h.y, h.z, h.w};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        o[j] = BF16 ? pack_bf16x2(f.x * sc[i][kv], f.y * sc[i][kv]) : pack_f16x2(f.x * sc[i][kv], f.y * sc[i][kv]);
      }
      uint16_t* dst = kv == 0 ? static_cast<uint16_t*>(p.k_out) + tok * p.k_s + head * p.k_h
                              : static_cast<uint16_t*>(p.v_out) + tok * p.v_s + head * p.v_h;
      *reinterpret_cast<uint4*>(dst + 8 * lane) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <int D, int DV>
cudaError_t launch_cache(bool write, bool bf16, const CacheParams& p, cudaStream_t st) {
  constexpr int BR = CacheCfg<D, DV>::BLOCK_ROWS;
  const unsigned grid = static_cast<unsigned>((p.rows + BR - 1) / BR);
  auto kern = write ? (bf16 ? cache_write_kernel<true, D, DV> : cache_write_kernel<false, D, DV>)
                    : (bf16 ? cache_read_kernel<true, D, DV> : cache_read_kernel<false, D, DV>);
  kern<<<grid, kCacheThreads, 0, st>>>(p);
  return cudaGetLastError();
}

// One checked call of either direction (write: k, v in, pools out; else the reverse).
int cache_call(bool write, const void* k, const void* v, const void* k_pool, const void* v_pool, const float* k_scale,
               const float* v_scale, const int32_t* page_table, const int32_t* kv_len, const int32_t* cu, int B,
               int Hkv, int total, int page_size, int max_pages, int n_pages, int D, int Dv, const int64_t* strides,
               int dtype, cudaStream_t stream) {
  // ---- validation (no CUDA call before this block passes)
  if (!k || !v || !k_pool || !v_pool || !k_scale || !v_scale || !page_table || !cu || (write && !kv_len))
    return SDPA_ERR_INVALID;
  if (B < 1 || Hkv < 1 || total < 1 || D < 1 || Dv < 1) return SDPA_ERR_INVALID;
  int rc = page_check(page_size, max_pages, n_pages);
  if (rc != SDPA_OK) return rc;
  if (dtype != SDPA_F16 && dtype != SDPA_BF16) return SDPA_ERR_UNSUPPORTED;
  if (!((D == 64 && Dv == 64) || (D == 128 && Dv == 128) || (D == 192 && Dv == 128))) return SDPA_ERR_UNSUPPORTED;
  if (static_cast<long long>(total) * Hkv >= (1ll << 30)) return SDPA_ERR_UNSUPPORTED;
  int64_t st[SDPA_CACHE_NSTRIDES] = {(int64_t)Hkv * D, D, (int64_t)Hkv * Dv, Dv,
                                     (int64_t)page_size * Hkv * D, (int64_t)Hkv * D, D,
                                     (int64_t)page_size * Hkv * Dv, (int64_t)Hkv * Dv, Dv, max_pages};
  if (strides)
    for (int i = 0; i < SDPA_CACHE_NSTRIDES; ++i) st[i] = strides[i];
  for (int i = 0; i < 4; ++i)
    if (!stride_ok(st[i], 8)) return SDPA_ERR_UNSUPPORTED;
  for (int i = 4; i < 10; ++i)
    if (!stride_ok(st[i], 16)) return SDPA_ERR_UNSUPPORTED;
  if (st[10] < max_pages) return SDPA_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_pool) || !aligned16(v_pool)) return SDPA_ERR_UNSUPPORTED;
  if (!aligned16(k_scale) || !aligned16(v_scale)) return SDPA_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(kv_len) | reinterpret_cast<uintptr_t>(cu)) & 3u)
    return SDPA_ERR_INVALID;

  CacheParams p{};
  p.k = p.k_out = const_cast<void*>(k);
  p.v = p.v_out = const_cast<void*>(v);
  p.k_pool = static_cast<uint8_t*>(const_cast<void*>(k_pool));
  p.v_pool = static_cast<uint8_t*>(const_cast<void*>(v_pool));
  p.k_scale = const_cast<float*>(k_scale);
  p.v_scale = const_cast<float*>(v_scale);
  p.page_table = page_table, p.kv_len = kv_len, p.cu = cu;
  p.k_s = st[0], p.k_h = st[1], p.v_s = st[2], p.v_h = st[3];
  p.kp_p = st[4], p.kp_r = st[5], p.kp_h = st[6], p.vp_p = st[7], p.vp_r = st[8], p.vp_h = st[9], p.pt_b = st[10];
  p.B = B, p.Hkv = Hkv, p.rows = total * Hkv;
  p.log2_page = __builtin_ctz((unsigned)page_size), p.max_pages = max_pages, p.n_pages = n_pages;
  p.div_h = make_fastdiv((uint32_t)Hkv);
  if (device_status_ptr(&p.status) != cudaSuccess) return SDPA_ERR_CUDA;
  const bool bf16 = dtype == SDPA_BF16;
  const cudaError_t e = D == 64    ? launch_cache<64, 64>(write, bf16, p, stream)
                        : D == 128 ? launch_cache<128, 128>(write, bf16, p, stream)
                                   : launch_cache<192, 128>(write, bf16, p, stream);
  return e == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

}  // namespace

int page_check(int page_size, int max_pages, int n_pages) {
  if (page_size < 1 || max_pages < 1 || n_pages < 1 || (page_size & (page_size - 1))) return SDPA_ERR_INVALID;
  if (page_size < 16 || static_cast<long long>(max_pages) * page_size > (1ll << 30)) return SDPA_ERR_UNSUPPORTED;
  return SDPA_OK;
}

}  // namespace sdpa

using namespace sdpa;

extern "C" {

int sdpa_cache_write_fp8(const void* k, const void* v, void* k_pool, void* v_pool, float* k_scale, float* v_scale,
                         const int32_t* page_table, const int32_t* kv_len, const int32_t* cu_seqlens, int B, int Hkv,
                         int total, int page_size, int max_pages, int n_pages, int D, int Dv, const int64_t* strides,
                         sdpa_dtype in_dtype, void* stream) {
  return cache_call(true, k, v, k_pool, v_pool, k_scale, v_scale, page_table, kv_len, cu_seqlens, B, Hkv, total,
                    page_size, max_pages, n_pages, D, Dv, strides, in_dtype, static_cast<cudaStream_t>(stream));
}

int sdpa_cache_read_fp8(const void* k_pool, const void* v_pool, const float* k_scale, const float* v_scale,
                        const int32_t* page_table, const int32_t* cu_seqlens, void* k, void* v, int B, int Hkv,
                        int total, int page_size, int max_pages, int n_pages, int D, int Dv, const int64_t* strides,
                        sdpa_dtype out_dtype, void* stream) {
  return cache_call(false, k, v, k_pool, v_pool, k_scale, v_scale, page_table, nullptr, cu_seqlens, B, Hkv, total,
                    page_size, max_pages, n_pages, D, Dv, strides, out_dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
