// Host replay of the latent attention's plan: the kernels' own cut, walk and group functions over one batch.  Checks that the
// CTAs' pieces cover every unit once and that the merge reads the slots they write.
#include <algorithm>
#include <cstdio>
#include <map>
#include <utility>
#include <vector>

#include "latent_plan.cuh"

using namespace sdpa;

// inl: planned by the attention kernel, else by the planning kernel.  cut: room for partials.  Returns 0, or a code and a line
// in msg.
extern "C" int latent_line_replay(int B, int tok_tile, const int* cu_q, const int* kv_len, int max_kv, int causal, int sms, int inl,
                                  int cut, char* msg) {
  PagedParams p{};
  p.B = B, p.Hkv = 1, p.causal = causal, p.cu_q = cu_q, p.kv_len = kv_len, p.tok_tile = tok_tile, p.max_kv = max_kv;
  p.sms = sms, p.cut = cut, p.inline_plan = inl, p.unit_tiles = 1, p.min_piece = kLatentMinPiece, p.min_work = kLatentMinWork;
  std::vector<int2> tiles;                      // {sequence, tile in it}
  std::vector<long long> seq_pos{0}, pos{0};    // starts of the sequences and of the tiles
  std::map<std::pair<int, int>, int> units;     // -> key blocks
  for (int b = 0; b < B; ++b) {
    const int n = cu_q[b + 1] - cu_q[b];
    for (int i = 0; i * tok_tile < n; ++i) {
      const int unit = latent_unit(p, n, kv_len[b], i);
      tiles.push_back(make_int2(b, i));
      pos.push_back(pos.back() + unit);
      units[{b, i}] = unit - kUnitCost;
    }
    seq_pos.push_back(pos.back());
  }
  p.plan.tiles = tiles.data();
  const long long total = pos.back();
  const int n_ctas = static_cast<int>(std::min<long long>(sms, total / p.min_work));
  std::vector<int4> cuts(n_ctas + 1);
  for (int c = 0; c <= n_ctas; ++c) {
    if (inl) {
      cuts[c] = latent_cut(p, seq_pos.data(), c, n_ctas);
      continue;
    }
    cuts[c] = make_int4(static_cast<int>(tiles.size()), 0, 0, 0);
    if (c == n_ctas) break;
    const long long x = total / n_ctas * c + total % n_ctas * c / n_ctas;
    size_t lo = 0;
    while (lo + 1 < tiles.size() && pos[lo + 1] <= x) ++lo;
    cuts[c] = paged_cut(p, x, pos[lo], static_cast<int>(lo), units[{tiles[lo].x, tiles[lo].y}]);
  }
  struct Piece {
    int slot, jb0, blocks;
  };
  std::map<std::pair<int, int>, std::vector<Piece>> done;
  for (int c = 0; c < n_ctas; ++c) {
    LatentWalk walk(c, cuts[c], cuts[c + 1]);
    while (true) {
      const LatentPiece w = walk.next(p);
      if (w.n_blocks == 0) break;
      if (w.n_blocks < 0) return sprintf(msg, "CTA %d: a piece of %d blocks", c, w.n_blocks), 1;
      done[{w.b, w.tok0 / tok_tile}].push_back({w.slot, w.jb0, w.n_blocks});
    }
  }
  std::map<std::pair<int, int>, PagedGroup> groups;
  for (int c = 0; c < n_ctas; ++c) {
    if (cuts[c].z == 0) continue;
    const int2 at = inl ? make_int2(cuts[c].x, cuts[c].y) : tiles[cuts[c].x];
    PagedGroup g;
    if (!paged_group(cuts.data(), c, n_ctas, at, cu_q[at.x], cu_q[at.x + 1] - cu_q[at.x], kv_len[at.x], g)) continue;
    if (!groups.emplace(std::make_pair(at.x, at.y), g).second) return sprintf(msg, "sequence %d tile %d is merged twice", at.x, at.y), 2;
  }
  for (const auto& [unit, blocks] : units) {
    const std::vector<Piece>& pieces = done[unit];
    int at = 0;
    for (const Piece& x : pieces) {
      if (x.jb0 != at) return sprintf(msg, "sequence %d tile %d: block %d follows %d", unit.first, unit.second, x.jb0, at), 3;
      at += x.blocks;
    }
    if (at != blocks) return sprintf(msg, "sequence %d tile %d: %d of %d blocks", unit.first, unit.second, at, blocks), 4;
    const auto g = groups.find(unit);
    if ((pieces.size() > 1) != (g != groups.end()) || (pieces.size() == 1 && pieces[0].slot != -1))
      return sprintf(msg, "sequence %d tile %d: %zu pieces, merged %d", unit.first, unit.second, pieces.size(), g != groups.end()), 5;
    if (g == groups.end()) continue;
    if (g->second.pieces != static_cast<int>(pieces.size()) || g->second.tile != unit.second)
      return sprintf(msg, "sequence %d tile %d: %zu pieces, %d merged", unit.first, unit.second, pieces.size(), g->second.pieces), 6;
    for (int i = 0; i < g->second.pieces; ++i) {
      const int slot = i == 0 ? g->second.slot0 : 2 * (g->second.first + i);
      if (slot != pieces[i].slot)
        return sprintf(msg, "sequence %d tile %d: piece %d written to slot %d, read from %d", unit.first, unit.second, i, pieces[i].slot, slot), 7;
    }
  }
  return done.size() == units.size() ? 0 : (sprintf(msg, "%zu units worked on, %zu exist", done.size(), units.size()), 8);
}
