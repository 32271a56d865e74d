// Chunk attention over a paged cache: parameter blocks, the work plan that lives in the caller's
// workspace, and the launch functions.  Internal.
#pragma once

#include "internal.h"

namespace sdpa {

// The plan, written by paged_plan_kernel at the start of the workspace: a header of kPlanHeader
// ints, then three prefixes of B + 1 entries each over the sequences.
enum PlanHeader : int { kPlanUnits = 0, kPlanSeg = 1, kPlanGroups = 2, kPlanHeader = 4 };
// prefix 0: work units; prefix 1: partial slots (units of sequences cut into several key ranges);
// prefix 2: groups (work tile, KV head) that the combine merges.

struct PagedParams {
  void* o;                 // [total_q, Hq, Dv]
  float* lse;              // [Hq, total_q] or null
  int64_t o_s, o_h;        // element strides of o
  const int32_t* cu_q;     // [B + 1]
  const int32_t* kv_len;   // [B]
  const int32_t* page_table;
  int64_t pt_b;
  const float* k_scale;    // quantised caches: [n_pages, Hkv, page_size]
  const float* v_scale;
  int32_t* plan;           // workspace: the plan ...
  float* part_o;           // ... then partial O [slot][slot_rows][DV] ...
  float* part_ml;          // ... and (max, sum) [slot][slot_rows][2]
  uint32_t* status;
  int B, Hq, Hkv, total_q, max_seqlen_q, group, causal;
  int tok_tile;            // tokens per 128-row query tile: 128 / group
  int page_size, log2_page, max_pages, n_pages;
  int max_kv;              // max_pages * page_size
  int slot_rows, max_slots, sms;
  int stall_first_stage;   // test hook
  float scale2;            // scale * log2(e)
  FastDiv div_group, div_hkv;
};

// Key blocks that query tile `tile` (tok_tile tokens) of a sequence sees: 0 past its last token, else
// at least 1 (a tile without visible keys runs one masked block and stores O = 0, LSE = -inf).
#ifdef __CUDACC__
__host__ __device__ __forceinline__ int paged_tile_blocks(int n, int len, int sk, int tok_tile, int causal, int tile) {
  const int first = tile * tok_tile;
  if (first >= n) return 0;
  int keys = sk;
  if (causal) {
    const int end = first + tok_tile < n ? first + tok_tile : n;
    const int vis = len - n + end;  // keys the tile's last token sees
    keys = keys < vis ? keys : vis;
  }
  return keys > kBlockK ? (keys + kBlockK - 1) / kBlockK : 1;
}
#endif

cudaError_t launch_paged_plan(const PagedParams& p, cudaStream_t st);
cudaError_t launch_paged_f16(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedParams& p, cudaStream_t st);
cudaError_t launch_paged_bf16(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const PagedParams& p, cudaStream_t st);
cudaError_t launch_paged_fp8(bool bf16, int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedParams& p, cudaStream_t st);
cudaError_t launch_paged_combine(bool bf16, int Dv, const PagedParams& p, cudaStream_t st);

}  // namespace sdpa
