// Page allocation for paged caches: a step's change of every sequence's length, on the device.
//
// The free pages are a stack, free_pages[0 .. n_free).  Sequence b goes from n rows to n + change[b]; the pages
// it no longer needs are pushed, sequence by sequence and page by page, and then those that are needed are popped in
// the same order.  With F pages pushed and A popped the r-th page popped is stack entry n_free + F - 1 - r: one of
// the old entries, or, from n_free on, the j-th page given back, which stands in the page table of a sequence
// that shrinks.  So nothing depends on anything another thread writes: prefix sums of the counts, then every new
// page, every page that stays on the stack and every new token is found by itself.  A thread looks its item up
// in the sums by binary search.
//
// Bound by latency for a decode step (64 sequences: one block, one launch, 5.6 us in a graph) and for a scheduler's step over
// 1024 sequences with 843,000 new tokens (17 us, of which the sums of the one block are some 7; 11.7 MB).
#include <algorithm>

#include "sdpa.h"
#include "internal.h"
#include "ptx.cuh"
#include "scan.cuh"

namespace sdpa {

namespace {

constexpr int kResizeThreads = 1024;
constexpr int kResizeTokens = 1024;  // tokens a block of the second kernel
// One block does all of it where that is little: the sequences fit its shared memory, and the tokens and the pages that
// could be given back are few.
constexpr int kResizeSeqs = 1024;
bool one_block(int B, int total, int max_pages) {
  return B <= kResizeSeqs && total <= 4 * kResizeThreads && static_cast<long long>(B) * max_pages <= 64 * kResizeThreads;
}

struct ResizeHead {
  int32_t ok, n_free, freed, taken;
};
// A sequence's rows before and after, and the pages given back and taken by those before it.
struct ResizeSeq {
  int32_t before, after, freed, taken;
};
static_assert(sizeof(ResizeHead) == sizeof(int4) && sizeof(ResizeSeq) == sizeof(int4), "read as one vector");

struct ResizeParams {
  int32_t* table;
  const int32_t *kv_len, *change, *n_free;
  int32_t* free_pages;
  int32_t *kv_len_out, *n_free_out, *cu, *positions;
  int64_t* slots;
  int4* head;              // workspace: ResizeHead, then ResizeSeq [B + 1]
  int4* seqs;
  uint32_t* status;
  int64_t pt_b;
  int B, total, log2_page, max_pages, n_pages;
};

__device__ __forceinline__ int pages_of(int rows, int log2_page) {
  return static_cast<int>((static_cast<long long>(rows) + (1 << log2_page) - 1) >> log2_page);
}

// The last sequence in [lo, hi) whose sum, seqs[b].z (given back) or .w (taken), is at most x.
template <bool TAKEN>
__device__ __forceinline__ int find_seq(const int4* seqs, int lo, int hi, int x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const int4 s = seqs[mid];
    if ((TAKEN ? s.w : s.z) <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// The j-th page given back.
__device__ __forceinline__ int freed_page(const ResizeParams& p, int j) {
  const int b = find_seq<false>(p.seqs, 0, p.B, j);
  const int4 s = p.seqs[b];
  return p.table[b * p.pt_b + pages_of(s.y, p.log2_page) + (j - s.z)];
}
// The r-th page taken.
__device__ __forceinline__ int taken_page(const ResizeParams& p, const int4& head, int r) {
  const int at = head.y + head.z - 1 - r;
  return at < head.y ? p.free_pages[at] : freed_page(p, at - head.y);
}

// The items of thread `first` of `threads`: new pages, pages that stay on the stack, tokens.
__device__ __forceinline__ void resize_pages(const ResizeParams& p, const int4& head, long long first, long long threads) {
  for (long long r = first; r < head.w; r += threads) {
    const int b = find_seq<true>(p.seqs, 0, p.B, static_cast<int>(r));
    const int4 s = p.seqs[b];
    p.table[b * p.pt_b + pages_of(s.x, p.log2_page) + (r - s.w)] = taken_page(p, head, static_cast<int>(r));
  }
  for (long long j = first; j < static_cast<long long>(head.z) - head.w; j += threads)
    p.free_pages[head.y + j] = freed_page(p, static_cast<int>(j));
}

// Position and slot of token t, which belongs to a sequence in [lo, hi) if to any.
__device__ __forceinline__ void resize_token(const ResizeParams& p, const int4& head, int t, int lo, int hi) {
  int pos = 0;
  int64_t slot = -1;
  if (head.x && t < p.cu[p.B]) {
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] <= t) lo = mid; else hi = mid;
    }
    const int4 s = p.seqs[lo];
    pos = s.x + (t - p.cu[lo]);
    const int page = pos >> p.log2_page, had = pages_of(s.x, p.log2_page);
    // a page taken by this call may not stand in the table yet
    const int phys = page < had ? p.table[lo * p.pt_b + page] : taken_page(p, head, s.w + (page - had));
    slot = (static_cast<int64_t>(phys) << p.log2_page) + (pos & ((1 << p.log2_page) - 1));
  }
  p.positions[t] = pos;
  p.slots[t] = slot;
}

// One block: the sums.  ALL: the items too.
template <bool ALL>
__global__ void __launch_bounds__(kResizeThreads) resize_plan_kernel(ResizeParams p) {
  __shared__ long long warp_sum[33];
  __shared__ int4 s_seqs[ALL ? kResizeSeqs : 1];
  const int tid = threadIdx.x;
  if (ALL) p.seqs = s_seqs;
  if (!ALL) pdl_launch_dependents();
  long long tokens = 0, freed = 0, taken = 0;
  int bad = 0;
  const int n_free = *p.n_free;  // it and the lengths may be overwritten below: no read-only loads
  for (int base = 0; base < p.B; base += kResizeThreads) {
    const int b = base + tid;
    int before = 0, after = 0, more = 0, back = 0, n_new = 0;
    if (b < p.B) {
      before = p.kv_len[b];
      const int d = __ldg(p.change + b);
      const long long to = static_cast<long long>(before) + d;
      if (before < 0 || before > (p.max_pages << p.log2_page) || to < 0 || to > (static_cast<long long>(p.max_pages) << p.log2_page)) {
        bad = 1;
        after = before;
      } else {
        after = static_cast<int>(to);
        const int grow = pages_of(after, p.log2_page) - pages_of(before, p.log2_page);
        more = max(grow, 0), back = max(-grow, 0), n_new = max(d, 0);
      }
    }
    const long long t0 = tokens, f0 = freed, a0 = taken;
    const long long ti = block_scan(n_new, t0, warp_sum, tokens);
    const long long fi = block_scan(back, f0, warp_sum, freed);
    const long long ai = block_scan(more, a0, warp_sum, taken);
    if (b < p.B) {
      // sums past 31 bits mean a bad call: nothing is taken from them
      p.seqs[b] = make_int4(before, after, static_cast<int>(fi - back), static_cast<int>(ai - more));
      p.cu[b] = static_cast<int>(ti - n_new);
    }
  }
  bad |= n_free < 0 || n_free > p.n_pages || tokens > p.total || taken > n_free + freed || n_free + freed - taken > p.n_pages ||
         freed > p.n_pages;
  bad = __syncthreads_or(bad);
  const int4 head = bad ? make_int4(0, n_free, 0, 0) : make_int4(1, n_free, static_cast<int>(freed), static_cast<int>(taken));
  for (int b = tid; b < p.B; b += kResizeThreads) {
    const int4 s = p.seqs[b];
    p.kv_len_out[b] = bad ? s.x : s.y;
    if (bad) p.cu[b] = 0;
  }
  if (tid == 0) {
    p.cu[p.B] = bad ? 0 : static_cast<int>(tokens);
    p.n_free_out[0] = head.y + head.z - head.w;
    if (!ALL) p.head[0] = head;
    if (bad) atomicOr(p.status, kStatusBadSeqlens);
  }
  if (ALL) {
    __syncthreads();
    resize_pages(p, head, tid, kResizeThreads);
    for (int t = tid; t < p.total; t += kResizeThreads) resize_token(p, head, t, 0, p.B);
  }
}

__global__ void __launch_bounds__(256) resize_items_kernel(const ResizeParams p) {
  __shared__ int range[2];
  pdl_wait();
  const int4 head = ld_dep(p.head);
  resize_pages(p, head, static_cast<long long>(blockIdx.x) * 256 + threadIdx.x, static_cast<long long>(gridDim.x) * 256);
  // the block's tokens lie in a few sequences: two threads look for them, the others between those
  const int t0 = blockIdx.x * kResizeTokens, t1 = min(t0 + kResizeTokens, p.total);
  if (t0 >= t1) return;
  if (threadIdx.x < 2) {
    const int t = threadIdx.x == 0 ? t0 : t1 - 1;
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] <= t) lo = mid; else hi = mid;
    }
    range[threadIdx.x] = lo;
  }
  __syncthreads();
  for (int t = t0 + threadIdx.x; t < t1; t += 256) resize_token(p, head, t, range[0], range[1] + 1);
}

}  // namespace

}  // namespace sdpa

using namespace sdpa;

extern "C" {

size_t sdpa_cache_resize_workspace_size(int B, int total, int max_pages) {
  if (B < 1 || total < 1 || max_pages < 1 || B > kMaxCount || total > kMaxCount) return 0;
  return one_block(B, total, max_pages) ? 0 : (static_cast<size_t>(B) + 1) * sizeof(int4);
}

int sdpa_cache_resize(int32_t* page_table, const int32_t* kv_len, const int32_t* change, int32_t* free_pages,
                      const int32_t* n_free, int32_t* kv_len_out, int32_t* n_free_out, int32_t* cu_seqlens,
                      int32_t* positions, int64_t* slots, int B, int total, int page_size, int max_pages, int n_pages,
                      int64_t table_stride, void* workspace, size_t workspace_bytes, void* stream) {
  // ---- validation (no CUDA call before this block passes)
  if (!page_table || !kv_len || !change || !free_pages || !n_free || !kv_len_out || !n_free_out || !cu_seqlens || !positions || !slots)
    return SDPA_ERR_INVALID;
  if (B < 1 || total < 1) return SDPA_ERR_INVALID;
  const int rc = page_check(page_size, max_pages, n_pages);
  if (rc != SDPA_OK) return rc;
  if (B > kMaxCount || total > kMaxCount) return SDPA_ERR_UNSUPPORTED;
  if (table_stride < max_pages) return SDPA_ERR_INVALID;
  const void* words[] = {page_table, kv_len, change, free_pages, n_free, kv_len_out, n_free_out, cu_seqlens, positions};
  for (const void* w : words)
    if (reinterpret_cast<uintptr_t>(w) & 3u) return SDPA_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(slots) & 7u) return SDPA_ERR_INVALID;
  const size_t need = sdpa_cache_resize_workspace_size(B, total, max_pages);
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return SDPA_ERR_INVALID;

  ResizeParams p{};
  p.table = page_table, p.kv_len = kv_len, p.change = change, p.n_free = n_free, p.free_pages = free_pages;
  p.kv_len_out = kv_len_out, p.n_free_out = n_free_out, p.cu = cu_seqlens, p.positions = positions, p.slots = slots;
  if (need > 0) p.head = static_cast<int4*>(workspace), p.seqs = p.head + 1;
  p.pt_b = table_stride;
  p.B = B, p.total = total, p.log2_page = __builtin_ctz((unsigned)page_size), p.max_pages = max_pages, p.n_pages = n_pages;
  if (device_status_ptr(&p.status) != cudaSuccess) return SDPA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (one_block(B, total, max_pages)) {
    resize_plan_kernel<true><<<1, kResizeThreads, 0, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
  }
  resize_plan_kernel<false><<<1, kResizeThreads, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SDPA_ERR_CUDA;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // a block per kResizeTokens tokens, and enough of them for the pages of long tables
  const long long entries = std::min<long long>(static_cast<long long>(B) * max_pages, n_pages);
  const long long blocks = std::max<long long>((static_cast<long long>(total) + kResizeTokens - 1) / kResizeTokens,
                                               std::min<long long>(152, (entries + 1023) / 1024));
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, resize_items_kernel, p) == cudaSuccess ? SDPA_OK : SDPA_ERR_CUDA;
}

}  // extern "C"
