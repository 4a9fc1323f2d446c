// chunk_plan.hpp -- the plan of chunk attention: the units of all row tiles on a line, and the pieces of them that a pair of CTAs
// goes through. For the kernel, and for the host, where a test goes through it.
#pragma once

#include "mfa_serving.hpp"
#include "work_line.hpp"

namespace mfa {
namespace {

#ifndef __CUDACC__  // a host compiler: CUDA's headers leave these out
using std::max;
using std::min;
#ifndef __noinline__
#define __noinline__
#endif
#endif

constexpr int kTokens = kChunkTileTokens;

// The line of work as every CTA sees it.
constexpr int kPlanChunks = kMaxBatch / 32 + 1;
struct LineRange {
  int from, to;
};
struct PlanSmem {
  int32_t cost[kMaxBatch + 1];  // units of the sequences before b; [B]: of all
  int32_t row[kMaxBatch + 1];   // first row of sequence b's tokens, non-decreasing within [0, max_tokens]
  int32_t len[kMaxBatch];       // positions that its pages hold
  int32_t last[kPlanChunks + 1], total[kPlanChunks + 1];  // of 32 sequences
  LineRange rest;                                         // what the pair does last, if it is not empty
};

// Tile i of a sequence whose chunk of n tokens stands behind a others sees a + min(4 (i + 1), n) keys. Of the tiles that
// are full, the first i take, with z = floor((a + 127) / 4),
//     sum_{k = 1..i} ceil((a + 4 k) / 128) = sum_{k = 1..i} floor((k + z) / 32) = G(i + z) - G(z)
// units, G(m) = sum_{k = 0..m} floor(k / 32); modulo 2^32, and the host has seen to it that the sums stay below 2^31.
__host__ __device__ __forceinline__ uint32_t floor_sum(uint32_t m) {
  const uint32_t q = m >> 5;
  return 16 * q * (q - 1) + q * ((m & 31) + 1);
}
__host__ __device__ __forceinline__ int units_of(int keys) { return (keys + kUnitKeys - 1) / kUnitKeys; }
__host__ __device__ __forceinline__ int full_tiles_cost(int i, int a, int piece_units) {
  const uint32_t z = (uint32_t)(a + kUnitKeys - 1) >> 2;
  return (int)(floor_sum((uint32_t)i + z) - floor_sum(z)) + i * piece_units;
}
__host__ __device__ __forceinline__ int tiles_of(int n) { return (n + kTokens - 1) / kTokens; }
__host__ __device__ __forceinline__ int sequence_cost(int len, int n, int piece_units) {
  return n > 0 ? full_tiles_cost(tiles_of(n) - 1, len - n, piece_units) + units_of(len) + piece_units : 0;
}
// Tokens of b that see a key at all: the last len of them.
__host__ __device__ __forceinline__ int seeing(const PlanSmem& s, int b) { return min(s.row[b + 1] - s.row[b], s.len[b]); }

// Pairs that have work: with fewer units than pairs, every range holds one.
__host__ __device__ __forceinline__ int busy_pairs(const ChunkParams& p, int units) { return min(p.pairs, max(units, 1)); }

// A pair's pieces, in order: units [u0, u1) of one row tile. The rest of a tile that begins before the pair's range comes first,
// or, where the pages are more than L2 holds, last (kTurn): then all pairs begin with tiles' beginnings and go through a
// sequence's pages at about the same time, and HBM delivers them once for all of these. bf16, for seconds: 1024 tokens each
// behind 100000 and 90000 1600 -> 1870 TFLOP/s, 2048 behind 129024 1660 -> 1890, 8 chunks of 512 behind 32000 1720 -> 2050 in a
// burst; 2048 behind 63488, whose pages L2 holds, 1885 and 1890.
struct Piece {
  int b = -1, i;     // sequence, tile of it
  int a, n, row0;    // of the sequence: positions before its chunk, tokens that see any, the first one's row
  int row, tokens;   // of the tile: first row, tokens (1 to 4)
  int seen0, seen;   // keys that its first and its last token see
  int units;         // of the whole tile
  int u0, u1;
  int first, x;      // line positions: the tile's, and the one behind it
  bool last = false; // it is of what comes last
  __host__ __device__ int pages() const { return (seen + kPageSize - 1) / kPageSize; }
  __host__ __device__ int keys(int page) const { return min(max(seen - page * kPageSize, 0), kPageSize); }
  // Whether V of unit u holds rows that not all tokens see, up to the end of an MMA's 16 keys.
  __host__ __device__ bool ends(int u) const { return (u + 1) * kUnitKeys > seen0 && (tokens > 1 || (seen % kKeyStep) != 0); }
  __host__ __device__ bool whole() const { return u0 == 0 && u1 == units; }
};
template <bool kTurn>
__host__ __device__ __forceinline__ bool next_piece(const ChunkParams& p, const PlanSmem& s, LineRange range, Piece& q) {
  if (q.b < 0) q.x = range.from;
  for (;;) {
    if (kTurn && q.last) range = s.rest;
    if (q.x >= range.to) {
      if (!kTurn || q.last || s.rest.from >= s.rest.to) return false;
      q.last = true;
      q.x = s.rest.from;
      q.b = -1;
      range = s.rest;
    }
    if (q.b < 0 || q.x >= s.cost[q.b + 1]) {
      const int b = last_at_most(s.cost, p.B, q.x);
      q.b = b;
      q.n = seeing(s, b);
      q.a = s.len[b] - q.n;
      q.row0 = s.row[b + 1] - q.n;
      q.first = s.cost[b];
      int i0 = 0, i1 = tiles_of(q.n) - 1;  // the last tile that begins at or before x
      if (q.x == q.first) i1 = 0;
      while (i0 < i1) {
        const int mid = (i0 + i1 + 1) >> 1;
        if (q.first + full_tiles_cost(mid, q.a, p.piece_units) <= q.x) i0 = mid; else i1 = mid - 1;
      }
      q.i = i0;
      q.first += full_tiles_cost(i0, q.a, p.piece_units);
    } else {
      ++q.i;
      q.first = q.x;
    }
    q.tokens = min(kTokens, q.n - kTokens * q.i);
    q.row = q.row0 + kTokens * q.i;
    q.seen0 = q.a + kTokens * q.i + 1;
    q.seen = q.seen0 + q.tokens - 1;
    q.units = units_of(q.seen);
    q.u0 = max(0, q.x - q.first - p.piece_units);
    q.u1 = min(q.units, range.to - q.first - p.piece_units);
    q.x = q.first + p.piece_units + q.units;
    if (q.u0 < q.u1) return true;
  }
}

// Where a pair's range begins: at its first tile's beginning, if the rest of a tile before that is to come last.
static __host__ __device__ __noinline__ int begin_of(const ChunkParams& p, const PlanSmem& s, int lo, int hi) {
  Piece q;
  if (!next_piece<false>(p, s, LineRange{lo, hi}, q) || q.u0 == 0 || q.x >= hi) return lo;
  // units that the sequences hold together, if all are like this one, which is to have more than two tiles
  const int cost = s.cost[q.b + 1] - s.cost[q.b];
  const bool more = cost > 2 * (q.units + p.piece_units) && (float)q.units * (float)s.cost[p.B] > (float)p.l2_units * (float)cost;
  return more ? q.x : lo;
}

// The tile that begins in pair w's range and ends behind it, if any: its parts, the first of them pair w's, and its piece there.
__host__ __device__ __forceinline__ int parts_from(const ChunkParams& p, const PlanSmem& s, int w, int units, int W, Piece& q) {
  const int lo = range_of_pair(w, units, W), hi = range_of_pair(w + 1, units, W);
  if (!next_piece<false>(p, s, LineRange{hi - 1, hi}, q) || q.u1 == q.units || lo > q.first + p.piece_units) return 0;
  return pair_of_unit(q.first + p.piece_units + q.units - 1, units, W) - w + 1;
}
// Where a partial result of a pair lies, in row tiles of the workspace.
__host__ __device__ __forceinline__ int part_slot(int pair, bool begins) { return 2 * pair + begins; }

}  // namespace
}  // namespace mfa
