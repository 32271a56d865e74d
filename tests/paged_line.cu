// Host replay of the chunk attention's plan: the kernels' own cut, walk and group functions over one batch.
// Checks that the CTAs' pieces cover every unit once and that the merge reads the slots they write.
#include <cstdio>
#include <map>
#include <tuple>
#include <vector>

#include "paged.cuh"

using namespace sdpa;

namespace {

struct Piece {
  int slot, jb0, blocks;
};

int tile_blocks(const PagedParams& p, int b, int tile) {
  const int n = p.cu_q[b + 1] - p.cu_q[b], len = p.kv_len[b];
  return paged_tile_blocks(n, len, min(max(len, 0), p.max_kv), p.tok_tile, p.causal, tile);
}

}  // namespace

// one: sequences of one query tile, planned by the attention kernel; else by the planning kernel.  cut: room for
// partials.  Returns 0, or a code and a line in msg.
extern "C" int paged_line_replay(int B, int Hq, int Hkv, const int* cu_q, const int* kv_len, int max_kv, int causal, int sms,
                                 int one, int cut, char* msg) {
  PagedParams p{};
  p.B = B, p.Hq = Hq, p.Hkv = Hkv, p.group = Hq / Hkv, p.causal = causal, p.cu_q = cu_q, p.kv_len = kv_len;
  p.tok_tile = kBlockQ / p.group, p.max_kv = max_kv, p.sms = sms, p.cut = cut, p.inline_plan = one;
  // the line: tiles {sequence, tile pair in it} and their starts
  std::vector<int2> tiles;
  std::vector<long long> pos{0};
  std::map<std::tuple<int, int, int>, int> units;  // (sequence, tile pair, KV head) -> key blocks
  long long n_units = 0;
  for (int b = 0; b < B; ++b) {
    const int n = cu_q[b + 1] - cu_q[b], unit = kTilesPerCta * p.tok_tile;
    const int count = one ? 1 : (n + unit - 1) / unit;
    for (int i = 0; i < count; ++i) {
      const int blocks = max(tile_blocks(p, b, kTilesPerCta * i), tile_blocks(p, b, kTilesPerCta * i + 1));
      tiles.push_back(make_int2(b, i));
      pos.push_back(pos.back() + (n > 0 ? static_cast<long long>(blocks + kUnitCost) * Hkv : 0));
      if (n == 0) continue;
      n_units += Hkv;
      for (int h = 0; h < Hkv; ++h) units[{b, i, h}] = blocks;
    }
  }
  p.plan.tiles = tiles.data();
  const long long total = pos.back();
  const int n_ctas = static_cast<int>(std::min<long long>(sms, std::max<long long>(n_units, total / kMinWork)));
  std::vector<int4> cuts(n_ctas + 1);
  for (int c = 0; c <= n_ctas; ++c) {
    if (one) {
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
  // what the CTAs do
  std::map<std::tuple<int, int, int>, std::vector<Piece>> done;
  for (int c = 0; c < n_ctas; ++c) {
    PagedWalk walk(c, cuts[c], cuts[c + 1]);
    while (true) {
      const PagedPiece w = one ? walk.next<true>(p) : walk.next<false>(p);
      if (w.n_blocks == 0) break;
      if (w.n_blocks < 0) return sprintf(msg, "CTA %d: a piece of %d blocks", c, w.n_blocks), 1;
      done[{w.b, w.tok0 / (kTilesPerCta * p.tok_tile), w.kvh}].push_back({w.slot, w.jb0, w.n_blocks});
    }
  }
  // what the merge reads
  std::map<std::tuple<int, int, int>, PagedGroup> groups;
  for (int c = 0; c < n_ctas; ++c) {
    if (cuts[c].z == 0) continue;
    const int2 at = tiles[cuts[c].x];
    PagedGroup g;
    if (!paged_group(cuts.data(), c, n_ctas, at, cu_q[at.x], cu_q[at.x + 1] - cu_q[at.x], kv_len[at.x], g)) continue;
    if (!groups.emplace(std::make_tuple(at.x, at.y, g.kvh), g).second)
      return sprintf(msg, "sequence %d head %d is merged twice", at.x, g.kvh), 2;
  }
  for (const auto& [unit, blocks] : units) {
    const auto& [b, tile, kvh] = unit;
    const std::vector<Piece>& pieces = done[unit];
    int at = 0;
    for (const Piece& x : pieces) {
      if (x.jb0 != at) return sprintf(msg, "sequence %d tile %d head %d: block %d follows %d", b, tile, kvh, x.jb0, at), 3;
      at += x.blocks;
    }
    if (at != blocks) return sprintf(msg, "sequence %d tile %d head %d: %d of %d blocks", b, tile, kvh, at, blocks), 4;
    const auto g = groups.find(unit);
    if ((pieces.size() > 1) != (g != groups.end()) || (pieces.size() == 1 && pieces[0].slot != -1))
      return sprintf(msg, "sequence %d tile %d head %d: %zu pieces, merged %d", b, tile, kvh, pieces.size(), g != groups.end()), 5;
    if (g == groups.end()) continue;
    if (g->second.pieces != static_cast<int>(pieces.size()) || g->second.tile != tile)
      return sprintf(msg, "sequence %d tile %d head %d: %zu pieces, %d merged", b, tile, kvh, pieces.size(), g->second.pieces), 6;
    for (int i = 0; i < g->second.pieces; ++i) {
      const int slot = i == 0 ? g->second.slot0 : 2 * (g->second.first + i);
      if (slot != pieces[i].slot)
        return sprintf(msg, "sequence %d tile %d head %d: piece %d written to slot %d, read from %d", b, tile, kvh, i,
                       pieces[i].slot, slot), 7;
    }
  }
  return done.size() == units.size() ? 0 : (sprintf(msg, "%zu units worked on, %zu exist", done.size(), units.size()), 8);
}
