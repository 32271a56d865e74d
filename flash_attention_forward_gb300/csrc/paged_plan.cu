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

// Costs in units of one 128-key block of a work unit: what a unit spends before its first and
// after its last block, and what the merge adds once anything is cut.
constexpr float kUnitOverhead = 3.f, kMergeOverhead = 4.f;
constexpr int kPlanThreads = 1024;
constexpr int kPlanCandidates = 64;  // segments of the longest sequence: 1 .. 64

__device__ __forceinline__ int plan_tiles(const PagedParams& p, int b, int& blocks, int& n_out) {
  const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
  const int n = max(0, q1 - q0);
  const int sk = min(max(__ldg(p.kv_len + b), 0), p.max_kv);
  blocks = n > 0 ? max(1, (sk + kBlockK - 1) / kBlockK) : 0;
  n_out = n;
  const int tok_unit = kTilesPerCta * p.tok_tile;
  return (n + tok_unit - 1) / tok_unit;
}

// One block decides how the key ranges are cut and lays out the units.  Candidate i cuts the longest
// sequence into i + 1 segments of `seg` blocks and every other one by the same `seg`; each warp
// costs candidates over all sequences:
//   rounds = ceil(units / SMs),  cost = max(rounds * blocks per unit, seg) + rounds * overhead (+ merge)
// and the cheapest that fits the workspace's partial slots wins, the first on ties.  Offsets that are
// not sorted within [0, total_q], or a sequence of more than max_seqlen_q tokens, raise a status and
// leave no units, so nothing is stored.
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PagedParams p) {
  __shared__ int s_max_blocks;
  __shared__ unsigned long long s_best;
  __shared__ int warp_sum[3][32];
  __shared__ int carry[3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();  // the attention kernel may set itself up meanwhile
  if (tid == 0) {
    s_max_blocks = 0;
    s_best = ~0ull;
    carry[0] = carry[1] = carry[2] = 0;
  }
  __syncthreads();
  int bad = 0, top = 0;
  for (int b = tid; b < p.B; b += kPlanThreads) {
    const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
    if (q0 < 0 || q1 < q0 || q1 > p.total_q || q1 - q0 > p.max_seqlen_q) bad = 1;
    int blocks, n;
    plan_tiles(p, b, blocks, n);
    top = max(top, blocks);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) atomicMax(&s_max_blocks, top);
  int32_t* prefix = p.plan + kPlanHeader;
  if (__syncthreads_or(bad)) {
    for (int i = tid; i < 3 * (p.B + 1); i += kPlanThreads) prefix[i] = 0;
    if (tid == 0) {
      p.plan[kPlanUnits] = p.plan[kPlanGroups] = 0;
      p.plan[kPlanSeg] = 1;
      atomicOr(p.status, kStatusBadSeqlens);
    }
    return;
  }
  const int max_blocks = max(s_max_blocks, 1);
  for (int i = warp; i < kPlanCandidates; i += kPlanThreads / 32) {
    const int seg = (max_blocks + i) / (i + 1);
    if (i > 0 && (p.max_slots == 0 || seg < 2)) break;  // the same for the whole warp
    float units = 0.f, work = 0.f, slots = 0.f;
    for (int b = lane; b < p.B; b += 32) {
      int blocks, n;
      const float tiles = static_cast<float>(plan_tiles(p, b, blocks, n)) * p.Hkv;
      if (n == 0) continue;
      const float segs = static_cast<float>((blocks + seg - 1) / seg);
      units += tiles * segs;
      work += tiles * blocks;
      if (segs > 1.f) slots += tiles * segs;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      units += __shfl_xor_sync(0xffffffffu, units, d);
      work += __shfl_xor_sync(0xffffffffu, work, d);
      slots += __shfl_xor_sync(0xffffffffu, slots, d);
    }
    if (lane == 0 && units > 0.f && (i == 0 || slots <= static_cast<float>(p.max_slots))) {
      const float rounds = ceilf(units / static_cast<float>(p.sms));
      const float cost = fmaxf(rounds * work / units, static_cast<float>(min(seg, max_blocks))) + rounds * kUnitOverhead +
                         (slots > 0.f ? kMergeOverhead : 0.f);
      // positive floats order like their bits
      atomicMin(&s_best, (static_cast<unsigned long long>(__float_as_uint(cost)) << 32) | static_cast<unsigned>(i));
    }
  }
  __syncthreads();
  const int best = s_best == ~0ull ? 0 : static_cast<int>(s_best & 0xFFFFFFFFu);
  const int seg = (max_blocks + best) / (best + 1);
  // exclusive prefixes of units, slots and groups over the sequences
  for (int base = 0; base < p.B; base += kPlanThreads) {
    const int b = base + tid;
    int v[3] = {0, 0, 0};
    if (b < p.B) {
      int blocks, n;
      const int tiles = plan_tiles(p, b, blocks, n) * p.Hkv;
      const int segs = n > 0 ? (blocks + seg - 1) / seg : 0;
      v[0] = tiles * segs;
      v[1] = segs > 1 ? v[0] : 0;
      v[2] = segs > 1 ? tiles : 0;
    }
    int x[3] = {v[0], v[1], v[2]};
#pragma unroll
    for (int q = 0; q < 3; ++q) {
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x[q], d);
        if (lane >= d) x[q] += y;
      }
      if (lane == 31) warp_sum[q][warp] = x[q];
    }
    __syncthreads();
    if (warp < 3) {
      int s = warp_sum[warp][lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
      }
      warp_sum[warp][lane] = s;
    }
    __syncthreads();
    int incl[3];
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      incl[q] = carry[q] + x[q] + (warp > 0 ? warp_sum[q][warp - 1] : 0);
      if (b < p.B) prefix[q * (p.B + 1) + b] = incl[q] - v[q];
    }
    __syncthreads();
    if (tid == kPlanThreads - 1)
      for (int q = 0; q < 3; ++q) carry[q] = incl[q];
    __syncthreads();
  }
  if (tid < 3) prefix[tid * (p.B + 1) + p.B] = carry[tid];
  if (tid == 0) {
    p.plan[kPlanUnits] = carry[0];
    p.plan[kPlanSeg] = seg;
    p.plan[kPlanGroups] = carry[2];
  }
}

// Merges the segments of every cut (work tile, KV head): one warp per (group, row), the segments in
// order, M = max m_i, O = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
template <bool BF16, int DV>
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedParams p) {
  constexpr int VEC = DV / 32;  // columns per lane
  pdl_wait();
  const int32_t* prefix = p.plan + kPlanHeader;
  const int32_t* slot_prefix = prefix + (p.B + 1);
  const int32_t* group_prefix = slot_prefix + (p.B + 1);
  const int groups = ld_dep(p.plan + kPlanGroups), seg = ld_dep(p.plan + kPlanSeg);
  const int lane = threadIdx.x & 31;
  const int64_t items = static_cast<int64_t>(groups) * p.slot_rows;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items; it += static_cast<int64_t>(gridDim.x) * 8) {
    const int grp = static_cast<int>(it / p.slot_rows), prow = static_cast<int>(it - static_cast<int64_t>(grp) * p.slot_rows);
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (ld_dep(group_prefix + mid) <= grp) lo = mid; else hi = mid;
    }
    const int local = grp - ld_dep(group_prefix + lo);  // rank * Hkv + kvh
    const int q_off = __ldg(p.cu_q + lo), n = __ldg(p.cu_q + lo + 1) - q_off;
    const int len = __ldg(p.kv_len + lo), sk = min(max(len, 0), p.max_kv);
    const int tok_unit = kTilesPerCta * p.tok_tile;
    const int tiles = (n + tok_unit - 1) / tok_unit;
    const int rank = local / p.Hkv, kvh = local - rank * p.Hkv;
    const int t = prow / kBlockQ, row = prow - t * kBlockQ;
    const int row_tok = static_cast<int>(fast_div(row, p.div_group));
    const int tile = (tiles - 1 - rank) * kTilesPerCta + t;
    const int tok = tile * p.tok_tile + row_tok;
    if (row_tok >= p.tok_tile || tok >= n) continue;  // the same for the whole warp
    const int head = kvh * p.group + (row - row_tok * p.group);
    const int blocks = paged_tile_blocks(n, len, sk, p.tok_tile, p.causal, tile);
    const int segs = (blocks + seg - 1) / seg;         // segments this tile reaches
    const int stride = tiles * p.Hkv;                   // slots from one segment to the next
    const int64_t slot0 = ld_dep(slot_prefix + lo) + local;
    float M = -INFINITY;
    for (int s = lane; s < segs; s += 32)
      M = fmaxf(M, p.part_ml[((slot0 + static_cast<int64_t>(s) * stride) * p.slot_rows + prow) * 2]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    float acc[VEC], L = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int s = 0; s < segs; ++s) {
      const int64_t at = (slot0 + static_cast<int64_t>(s) * stride) * p.slot_rows + prow;
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
      const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
      L += w * ml.y;
      const float* src = p.part_o + at * DV + lane * VEC;
      if constexpr (VEC == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        acc[0] += w * v.x, acc[1] += w * v.y, acc[2] += w * v.z, acc[3] += w * v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        acc[0] += w * v.x, acc[1] += w * v.y;
      }
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    uint32_t* orow = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + static_cast<int64_t>(q_off + tok) * p.o_s +
                                                 static_cast<int64_t>(head) * p.o_h + lane * VEC);
    uint32_t pk[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i)
      pk[i] = BF16 ? pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv) : pack_f16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    if constexpr (VEC == 4)
      *reinterpret_cast<uint2*>(orow) = make_uint2(pk[0], pk[1]);
    else
      *orow = pk[0];
    if (p.lse != nullptr && lane == 0)
      p.lse[static_cast<int64_t>(head) * p.total_q + q_off + tok] =
          L > 0.f ? (M + lg2(L)) * 0.6931471805599453f : -INFINITY;
  }
}

size_t plan_bytes(int B) { return split_round16((kPlanHeader + 3 * (static_cast<size_t>(B) + 1)) * sizeof(int32_t)); }

// Rows of a partial slot: both query tiles, or the rows of the longest chunk where one tile holds it.
int slot_rows(int group, int max_seqlen_q) {
  const int tok_tile = kBlockQ / group;
  return max_seqlen_q <= tok_tile ? max_seqlen_q * group : kCtaRows;
}

// Partial slots a workspace is sized for: 64 MB of them, at least 304 (two cuts for every SM), at
// most 4096 and what the sizes can produce at all; none where no sequence has two blocks of keys.
long long slots_wanted(int B, int Hkv, int total_q, int max_seqlen_q, int group, int max_kv, size_t slot_bytes) {
  const long long blocks = (max_kv + kBlockK - 1) / kBlockK;
  if (blocks < 2) return 0;
  const long long tok_unit = kTilesPerCta * (kBlockQ / group);
  const long long by_max = static_cast<long long>(B) * ((max_seqlen_q + tok_unit - 1) / tok_unit);
  const long long by_total = (static_cast<long long>(total_q) + (tok_unit - 1) * B) / tok_unit;
  const long long most = std::min(by_max, by_total) * Hkv * std::min<long long>(blocks, kPlanCandidates);
  return std::min(most, std::min<long long>(4096, std::max<long long>(304, (64ll << 20) / static_cast<long long>(slot_bytes))));
}

size_t slot_size(int rows, int Dv) { return static_cast<size_t>(rows) * (Dv + 2) * sizeof(float); }

size_t paged_ws_bytes(int B, int Hq, int Hkv, int total_q, int max_seqlen_q, int max_kv, int Dv) {
  const int group = Hq / Hkv;
  const size_t one = slot_size(slot_rows(group, max_seqlen_q), Dv);
  return plan_bytes(B) + static_cast<size_t>(slots_wanted(B, Hkv, total_q, max_seqlen_q, group, max_kv, one)) * one;
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
  const long long tok_unit = kTilesPerCta * (kBlockQ / group);
  const long long tiles = std::min(static_cast<long long>(B) * ((max_seqlen_q + tok_unit - 1) / tok_unit),
                                   (static_cast<long long>(total_q) + (tok_unit - 1) * B) / tok_unit);
  if (tiles * Hkv * kPlanCandidates >= (1ll << 30)) return SDPA_ERR_UNSUPPORTED;
  if (!workspace || !aligned16(workspace) || workspace_bytes < plan_bytes(B)) return SDPA_ERR_INVALID;

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
  p.div_group = make_fastdiv((uint32_t)group), p.div_hkv = make_fastdiv((uint32_t)Hkv);
  p.slot_rows = slot_rows(group, max_seqlen_q);
  const size_t one = slot_size(p.slot_rows, Dv);
  const long long fit = static_cast<long long>((workspace_bytes - plan_bytes(B)) / one);
  p.max_slots = static_cast<int>(std::min(fit, slots_wanted(B, Hkv, total_q, max_seqlen_q, group, max_kv, one)));
  char* ws = static_cast<char*>(workspace);
  p.plan = reinterpret_cast<int32_t*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + plan_bytes(B));
  p.part_ml = p.part_o + static_cast<size_t>(p.max_slots) * p.slot_rows * Dv;
  int dev = 0;
  if (current_device_sms(&dev, &p.sms) != cudaSuccess || device_status_ptr(&p.status) != cudaSuccess) return SDPA_ERR_CUDA;

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
  cudaError_t e = launch_paged_plan(p, s);
  if (e == cudaSuccess)
    e = quant ? launch_paged_fp8(bf16, D, tq, tk, tv, p, s)
              : (bf16 ? launch_paged_bf16(D, tq, tk, tv, p, s) : launch_paged_f16(D, tq, tk, tv, p, s));
  if (e == cudaSuccess && p.max_slots > 0) e = launch_paged_combine(bf16, Dv, p, s);
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
  // one warp per row, at most four CTAs per SM walking the rows
  const long long rows = static_cast<long long>(p.max_slots) * p.slot_rows;
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>((rows + 7) / 8, 4ll * p.sms)));
  cfg.blockDim = dim3(256);
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
  return paged_ws_bytes(B, Hq, Hkv, total_q, max_seqlen_q, max_kv, Dv);
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
