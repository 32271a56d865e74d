// Host replay of the chunk attention's choice of kernel and plan (paged_choose, paged_is_list): what the planning kernel, or the
// attention kernel for itself, lays out is walked as the chosen kernel walks it.  Checks that every unit is worked on once,
// whole where it comes from a list.
#include <cstdio>
#include <map>
#include <tuple>
#include <vector>

#include "paged.cuh"

using namespace sdpa;

// Whether the kernel that a call gets takes its work as the plan leaves it.  Returns 0, or a code and a line in msg; form: {one,
// inline_plan, list}.  cu_k: packed keys, of head_bytes a head; null: pages, of kv_len keys.
extern "C" int paged_form_replay(int B, int Hq, int Hkv, const int* cu_q, const int* cu_k, const int* kv_len, int max_seqlen_q,
                                 int quant, int D, long long head_bytes, int max_kv, int causal, int sms, int cut, int* form, char* msg) {
  PagedParams p{};
  p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.group = Hq / Hkv, p.causal = causal, p.cu_q = cu_q, p.cu_k = cu_k, p.kv_len = kv_len;
  p.max_seqlen_q = max_seqlen_q, p.tok_tile = kBlockQ / p.group, p.max_kv = max_kv, p.sms = sms, p.cut = cut;
  paged_choose(p, quant, D, head_bytes);
  std::vector<int2> tiles;  // {sequence, tile pair in it}
  std::vector<long long> pos{0};
  std::map<std::tuple<int, int, int>, int> units, done;  // (sequence, tile pair, KV head) -> key blocks
  for (int b = 0; b < B; ++b) {
    const int n = cu_q[b + 1] - cu_q[b], len = paged_len(p, b), sk = std::min(std::max(len, 0), max_kv);
    const int unit = kTilesPerCta * p.tok_tile, count = p.inline_plan ? 1 : (n + unit - 1) / unit;
    for (int i = 0; i < count; ++i) {
      const int blocks = std::max(paged_tile_blocks(n, len, sk, p.tok_tile, causal, kTilesPerCta * i),
                                  paged_tile_blocks(n, len, sk, p.tok_tile, causal, kTilesPerCta * i + 1));
      tiles.push_back(make_int2(b, i));
      pos.push_back(pos.back() + (n > 0 ? static_cast<long long>(blocks + kUnitCost) * Hkv : 0));
      for (int h = 0; n > 0 && h < Hkv; ++h) units[{b, i, h}] = blocks;
    }
  }
  p.plan.tiles = tiles.data();
  const bool list = !p.inline_plan && paged_is_list(p, static_cast<long long>(tiles.size()));
  form[0] = p.one, form[1] = p.inline_plan, form[2] = list;
  if (p.inline_plan && !p.one) return sprintf(msg, "the kernel for more tiles does not plan"), 1;
  if (list) {
    // the kernel for one tile and the one over pages read the cuts, which a list does not have
    if (p.one || cu_k == nullptr) return sprintf(msg, "a list for a kernel that reads cuts"), 2;
    const int n_items = static_cast<int>(tiles.size()) * Hkv;
    for (int i = 0; i < n_items; ++i) {
      const PagedPiece w = PagedWalk::item(p, i, n_items);
      if (w.slot != -1) return sprintf(msg, "item %d is a piece", i), 3;
      if (!done.emplace(std::make_tuple(w.b, w.tok0 / (kTilesPerCta * p.tok_tile), w.kvh), w.n_blocks).second)
        return sprintf(msg, "item %d comes twice", i), 4;
    }
  } else {
    const long long total = pos.back();
    const int n_ctas = static_cast<int>(std::min<long long>(sms, std::max<long long>(units.size(), total / kMinWork)));
    std::vector<int4> cuts(n_ctas + 1);
    for (int c = 0; c <= n_ctas; ++c) {
      if (p.inline_plan) {
        cuts[c] = paged_inline_cut(p, pos.data(), c, n_ctas);
        continue;
      }
      cuts[c] = make_int4(static_cast<int>(tiles.size()), 0, 0, 0);
      if (c == n_ctas) break;
      const long long x = total / n_ctas * c + total % n_ctas * c / n_ctas;
      size_t lo = 0;
      while (lo + 1 < tiles.size() && pos[lo + 1] <= x) ++lo;
      cuts[c] = paged_cut(p, x, pos[lo], static_cast<int>(lo), units[{tiles[lo].x, tiles[lo].y, 0}]);
    }
    for (int c = 0; c < n_ctas; ++c) {
      PagedWalk walk(c, cuts[c], cuts[c + 1]);
      while (true) {
        const PagedPiece w = p.one ? walk.next<true>(p) : walk.next<false>(p);
        if (w.n_blocks == 0) break;
        int& at = done[{w.b, w.tok0 / (kTilesPerCta * p.tok_tile), w.kvh}];
        if (w.n_blocks < 0 || w.jb0 != at) return sprintf(msg, "CTA %d: %d blocks from %d, %d before", c, w.n_blocks, w.jb0, at), 5;
        at += w.n_blocks;
      }
    }
  }
  return done == units ? 0 : (sprintf(msg, "%zu units worked on, %zu exist, or not all blocks of them", done.size(), units.size()), 6);
}
