// The plan of chunk attention as the kernel builds and follows it (chunk_plan.hpp), one call on the host for all pairs of CTAs.
#include "chunk_plan.hpp"

using namespace mfa;

extern "C" int charge(int quantised) { return quantised ? kChunkPieceUnitsQuantised : kChunkPieceUnits; }
extern "C" int tile_tokens() { return kTokens; }
extern "C" int most_pairs() { return kChunkMaxPairs; }

extern "C" long long sequence_units(int len, int n, int piece_units) { return sequence_cost(len, n, piece_units); }

// pieces: [pair, b, tile, u0, u1, units, row, tokens, seen0, seen, slot or -1, last] each, in each pair's order; parts: [row,
// tokens, pair, parts] each. Returns the number of pieces, -1 where `room` is too small.
template <bool kTurn>
static int go_through(const ChunkParams& p, PlanSmem& s, int* pieces, int room, int* parts, int* n_parts) {
  const int units = s.cost[p.B], W = busy_pairs(p, units);
  int n = 0, m = 0;
  for (int w = 0; w < W; ++w) {
    const int lo = range_of_pair(w, units, W), hi = range_of_pair(w + 1, units, W);
    LineRange range{lo, hi};
    s.rest = {0, 0};
    if (kTurn && units > p.l2_units) {
      if (lo < hi) range.from = begin_of(p, s, lo, hi);
      s.rest = {lo, range.from};
    }
    Piece q;
    while (next_piece<kTurn>(p, s, range, q)) {
      if (n == room) return -1;
      const int it[12] = {w, q.b, q.i, q.u0, q.u1, q.units, q.row, q.tokens, q.seen0, q.seen, q.whole() ? -1 : part_slot(w, q.u0 == 0), q.last};
      std::copy(it, it + 12, pieces + 12 * n++);
    }
    Piece t;
    const int k = units > 0 ? parts_from(p, s, w, units, W, t) : 0;
    if (k > 0) {
      const int it[4] = {t.row, t.tokens, w, k};
      std::copy(it, it + 4, parts + 4 * m++);
    }
  }
  *n_parts = m;
  return n;
}

extern "C" int plan(int B, const int* lens, const int* rows, int pairs, int piece_units, int l2_units, int turn, int* pieces, int room, int* parts,
         int* n_parts) {
  static PlanSmem s;
  ChunkParams p{};
  p.B = B;
  p.pairs = pairs;
  p.piece_units = piece_units;
  p.l2_units = l2_units;
  for (int b = 0; b <= B; ++b) s.row[b] = rows[b];
  s.cost[0] = 0;
  for (int b = 0; b < B; ++b) s.len[b] = lens[b];
  for (int b = 0; b < B; ++b) s.cost[b + 1] = s.cost[b] + sequence_cost(s.len[b], seeing(s, b), piece_units);
  return turn ? go_through<true>(p, s, pieces, room, parts, n_parts) : go_through<false>(p, s, pieces, room, parts, n_parts);
}

extern "C" int slot(int pair, int begins) { return part_slot(pair, begins != 0); }
