// Chunk attention over a paged cache: parameter blocks, the work plan that lives in the caller's
// workspace, and the launch functions.  Internal.
#pragma once

#include "internal.h"

namespace sdpa {

// The work, as one line.  A work unit is unit_tiles query tiles (of tok_tile tokens of one sequence each) and one
// KV head against all the key blocks the tiles see; units lie in the order (sequence, tile, KV
// head), each as long as its key blocks plus kUnitCost for its prologue and epilogue.  CTA c takes the
// stretch from cut c to cut c + 1, all of one length, so every SM has the same to do whatever the
// lengths are.  A cut inside a unit divides its keys; the two or more pieces write partials that a
// second kernel merges.  Cuts that would leave fewer than min_piece blocks on a side move to the
// unit's edge.
constexpr int kUnitCost = 2;         // blocks' time of a unit's prologue and epilogue
constexpr int kMinPiece = 3;         // blocks (of the chunk attention; its min_piece and min_work)
constexpr int kMinWork = 6;          // blocks per CTA below which more CTAs do not pay (unless units are left)
constexpr int kPagedMaxCtas = 160;

// The plan, at the start of the workspace: written by paged_plan_kernel, or by the attention kernel
// itself where every sequence has one query tile (kInlinePlanSeqs sequences at most); a "tile" is then a sequence.
constexpr int kInlinePlanSeqs = 256;
// A cut unit, for the merge.
struct PagedGroup {
  int32_t tile, kvh;       // tile in its sequence, KV head
  int32_t first, pieces;   // CTA of the first piece; the others follow
  int32_t slot0;           // partial slot of the first piece (the others: 2 * CTA)
  int32_t q_off, n, len;   // the sequence's packed offset, tokens and cache length
};
static_assert(sizeof(PagedGroup) == 2 * sizeof(int4), "read as two vectors");
struct PagedPlanHeader {
  int32_t n_ctas, n_groups;
  int32_t n_items, next_item;  // work as a list (see kListUnits), or n_items = 0
};
// Packed keys, sequences of more than one query tile, many units: nothing is cut, and the CTAs take whole units from a list,
// one after the other as they get done.  The list takes some KV heads at a time, as many as have their keys and values in
// kListBytes, and their units longest first: what runs at one time then shares K and V in the L2.  Equal stretches of the line have every CTA at heads
// of its own (8192 tokens x 128 heads: 10.8 GB of reads that miss it, 2200 us against 1900).
constexpr int kListUnits = 4;                 // per SM, from which on work is a list
constexpr int64_t kListBytes = 32 << 20;
struct PagedPlan {
  PagedPlanHeader* head;
  int4* cuts;              // [kPagedMaxCtas + 1] {tile, KV head, key block, 0}
  PagedGroup* groups;      // [kPagedMaxCtas] cut units
  int2* tiles;             // [n_tiles] {sequence, tile in it}
  long long* tile_pos;     // [n_tiles + 1] start of a tile's units on the line
  int32_t* seq_tiles;      // [B + 1] tiles of the sequences before b
};
inline size_t paged_plan_bytes(int B, long long n_tiles) {
  return split_round16(sizeof(PagedPlanHeader) + (kPagedMaxCtas + 1) * sizeof(int4) + kPagedMaxCtas * sizeof(PagedGroup) +
                       static_cast<size_t>(n_tiles) * (sizeof(int2) + sizeof(long long)) + sizeof(long long) +
                       (static_cast<size_t>(B) + 1) * sizeof(int32_t));
}
inline PagedPlan paged_plan_at(void* ws, long long n_tiles) {
  PagedPlan p;
  char* c = static_cast<char*>(ws);
  p.head = reinterpret_cast<PagedPlanHeader*>(c);
  p.cuts = reinterpret_cast<int4*>(p.head + 1);
  p.groups = reinterpret_cast<PagedGroup*>(p.cuts + kPagedMaxCtas + 1);
  p.tile_pos = reinterpret_cast<long long*>(p.groups + kPagedMaxCtas);
  p.tiles = reinterpret_cast<int2*>(p.tile_pos + n_tiles + 1);
  p.seq_tiles = reinterpret_cast<int32_t*>(p.tiles + n_tiles);
  return p;
}

struct PagedParams {
  void* o;                 // [total_q, Hq, Dv]
  float* lse;              // [Hq, total_q] or null
  int64_t o_s, o_h;        // element strides of o
  const int32_t* cu_q;     // [B + 1]
  const int32_t* kv_len;   // [B], or null: packed keys
  const int32_t* cu_k;     // packed keys: [B + 1], sequence b's are rows cu_k[b] .. of [total_k, Hkv, .]
  const int32_t* page_table;
  int64_t pt_b;
  const float* k_scale;    // quantised caches: [n_pages, Hkv, page_size]
  const float* v_scale;
  PagedPlan plan;          // workspace: the plan ...
  float* part_o;           // ... then partial O [2 * CTA + (0: the CTA's first piece, 1: its last)][slot_rows][DV] ...
  float* part_ml;          // ... and (max, sum) [slot][slot_rows][2]
  uint32_t* status;
  int B, Hq, Hkv, total_q, max_seqlen_q, group, causal;
  int one;                 // the kernel for sequences of one query tile (see paged_choose)
  int list_heads;          // packed keys: KV heads that the list takes at a time; 0: work is never a list
  int tok_tile;            // tokens per 128-row query tile: 128 / group
  int page_size, log2_page, max_pages, n_pages;
  int max_kv;              // max_pages * page_size, or total_k
  int unit_tiles = kTilesPerCta;  // query tiles of a work unit
  int min_piece = kMinPiece, min_work = kMinWork;
  int slot_rows, cut, sms; // cut: the workspace holds partials, units may be cut
  int max_tiles;           // tiles the plan has room for
  int inline_plan;         // the attention kernel plans for itself
  int stall_first_stage;   // test hook
  float scale2;            // scale * log2(e)
  FastDiv div_group;
};

// Which kernel a call gets and which plans go with it.  The kernel for one query tile a sequence walks a line with cuts and
// knows no list; it plans for itself where the sequences are few.  The other one takes a list where its keys are packed.
// Everything that depends on the choice (launch, boxes, planning kernel) asks what this has written.  head_bytes: keys and
// values of a head where they are packed, else 0.
inline void paged_choose(PagedParams& p, bool quant, int D, int64_t head_bytes) {
  // three-block operands leave no room for two readers' rings beside the raw codes
  p.one = !(quant && D == 192) && p.max_seqlen_q <= p.tok_tile;
  p.inline_plan = p.one && p.B <= kInlinePlanSeqs;
  p.list_heads = 0;
  if (head_bytes > 0 && !p.one) {
    const int64_t heads = kListBytes / head_bytes;
    p.list_heads = static_cast<int>(heads < 1 ? 1 : heads < p.Hkv ? heads : p.Hkv);
  }
}

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

#ifdef __CUDACC__
// Loads of what the plan is made from; the host, where tests replay it, has no read-only form.
__host__ __device__ __forceinline__ int plan_ld(const int32_t* p) {
#ifdef __CUDA_ARCH__
  return __ldg(p);
#else
  return *p;
#endif
}
// Whether the planning kernel leaves a list.
__host__ __device__ __forceinline__ bool paged_is_list(const PagedParams& p, long long n_tiles) {
  return p.list_heads > 0 && n_tiles * p.Hkv >= static_cast<long long>(kListUnits) * p.sms;
}
// Keys of sequence b.
__host__ __device__ __forceinline__ int paged_len(const PagedParams& p, int b) {
  return p.cu_k != nullptr ? plan_ld(p.cu_k + b + 1) - plan_ld(p.cu_k + b) : plan_ld(p.kv_len + b);
}
// Whether sequence b's offsets break the rules (q0, q1: its query rows).
__host__ __device__ __forceinline__ bool paged_bad(const PagedParams& p, int b, int q0, int q1) {
  bool bad = q0 < 0 || q1 < q0 || q1 > p.total_q || static_cast<long long>(q1) - q0 > p.max_seqlen_q;
  if (p.cu_k != nullptr) {
    const int k0 = plan_ld(p.cu_k + b), k1 = plan_ld(p.cu_k + b + 1);
    bad = bad || k0 < 0 || k1 < k0 || k1 > p.max_kv;
  }
  return bad;
}
// Where cut c of n_ctas lies: position x of the line falls into a unit of `blocks` key blocks that starts
// at `start` for KV head 0 (the tile's units follow one another).  {tile, KV head, block}.
__host__ __device__ __forceinline__ int4 paged_cut(const PagedParams& p, long long x, long long start, int tile, int blocks) {
  const long long unit = blocks + kUnitCost, r = x - start;  // many KV heads of a long sequence: past 32 bits
  int kvh = static_cast<int>(r / unit);
  int off = static_cast<int>(r - kvh * unit) - kUnitCost;
  if (p.cut ? off < p.min_piece : 2 * off < blocks) {
    off = 0;
  } else if (!p.cut || blocks - off < p.min_piece) {
    off = 0;
    if (++kvh == p.Hkv) kvh = 0, ++tile;
  }
  return make_int4(tile, kvh, off, 0);
}
// Cut c of n_ctas where tiles are sequences and sequence b lies from pos[b] to pos[b + 1].  Those without tokens
// have no length, and no cut names one: the walk passes over them, and the unit that it begins with has to be the
// one that the cut names, as paged_group tells a CTA's first piece by that.
__host__ __device__ __forceinline__ int4 paged_inline_cut(const PagedParams& p, const long long* pos, int c, int n_ctas) {
  if (c >= n_ctas) return make_int4(p.B, 0, 0, 0);
  const long long total = pos[p.B];
  const long long x = total / n_ctas * c + total % n_ctas * c / n_ctas;
  int lo = 0, hi = p.B;  // the last sequence that starts at or before x (it has tokens)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pos[mid] <= x) lo = mid; else hi = mid;
  }
  int4 cut = paged_cut(p, x, pos[lo], lo, static_cast<int>((pos[lo + 1] - pos[lo]) / p.Hkv) - kUnitCost);
  while (cut.x < p.B && pos[cut.x + 1] == pos[cut.x]) ++cut.x;
  return cut;
}
// The group of a unit whose first cut is cut c (cuts[c].z > 0 and not cut before), or false.
__host__ __device__ __forceinline__ bool paged_group(const int4* cuts, int c, int n_ctas, int2 at, int q_off, int n,
                                                     int len, PagedGroup& g) {
  const int4 cut = cuts[c];
  if (cut.z == 0) return false;
  const int4 prev = cuts[c - 1];  // c > 0: the line starts with a whole unit
  if (prev.x == cut.x && prev.y == cut.y && prev.z > 0) return false;
  int pieces = 2;
  while (c + pieces - 1 < n_ctas && cuts[c + pieces - 1].x == cut.x && cuts[c + pieces - 1].y == cut.y) ++pieces;
  // the first piece is CTA c - 1's last one, and its first one too if the CTA starts with it
  const int slot0 = 2 * (c - 1) + (prev.x == cut.x && prev.y == cut.y ? 0 : 1);
  g = PagedGroup{at.y, cut.y, c - 1, pieces, slot0, q_off, n, len};
  return true;
}
#endif

cudaError_t launch_paged_plan(const PagedParams& p, cudaStream_t st);
cudaError_t launch_paged_f16(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedParams& p, cudaStream_t st);
cudaError_t launch_paged_bf16(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const PagedParams& p, cudaStream_t st);
cudaError_t launch_paged_fp8(bool bf16, int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedParams& p, cudaStream_t st);
// Packed keys [total_k, Hkv, 128] and their shared part [total_k, 64] (tr), D = 192.
cudaError_t launch_paged_packed(bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CUtensorMap& tr, const PagedParams& p, cudaStream_t st);
cudaError_t launch_paged_combine(bool bf16, int Dv, const PagedParams& p, cudaStream_t st);

}  // namespace sdpa
