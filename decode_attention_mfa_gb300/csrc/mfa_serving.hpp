// mfa_serving.hpp -- parameter blocks and launch entry points of the operators of
// a serving step: page tables and slots, appends by slot, a cache read back,
// decode attention over shared prefixes, and attention of chunks of new tokens.
#pragma once

#include "mfa_internal.h"

namespace mfa {

// Rows scattered to cache slots (slot = page * 64 + row of the page; negative: no row).
struct AppendSlotsParams {
  const uint16_t* k_new;  // row i at k_new + i * k_stride (bf16 bits)
  const uint16_t* v_new;
  long long k_stride, v_stride;
  const int64_t* slot_map;  // [n_rows]
  void* k_cache;
  void* v_cache;
  float* k_scale;  // E4M3 and E2M1
  float* v_scale;
  uint32_t* err;
  int n_rows, num_pages, num_sms;
  int fmt;  // kKvBf16, kKvE4M3 or kKvE2M1
};

// Positions of a paged cache as bf16 rows: row row_starts[b] + i is position first[b] + i of sequence b.
struct KvReadParams {
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;  // E4M3 and E2M1
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* first;       // [B] (null: 0)
  const int32_t* row_starts;  // [B + 1]
  uint16_t* k_out;            // row i at k_out + i * k_stride (bf16 bits)
  uint16_t* v_out;
  long long k_stride, v_stride;
  uint32_t* err;
  int B, max_rows, max_pages, num_pages;
  int fmt;
};

// Pages taken from or given back to the stack of free page ids.
constexpr size_t kTableCounterOffset = 64;  // header byte of the arrival counter (zero between calls)
struct PageTableParams {
  const int32_t* n_new;       // [B] tokens that arrive (reserve)
  const int32_t* finished;    // [B] non-zero: the request ended (release)
  const int32_t* keep_pages;  // [B] pages a released request keeps (release; null: none)
  const int32_t* seq_lens;    // [B]
  int32_t* page_table;        // [B][max_pages]
  int32_t* free_pages;        // [num_pages] stack, top at n_free - 1
  const int32_t* n_free;
  int32_t* new_starts;        // [B + 1]
  int64_t* slot_map;          // [max_new]
  int32_t* seq_lens_out;      // [B], may be seq_lens
  int32_t* n_free_out;        // may be n_free
  uint32_t* err;
  uint32_t* counter;
  int B, max_pages, num_pages, max_new;
  bool in_place;              // an output replaces an input: written when every CTA has read
};

// Shared-prefix decode. The work is a line of row tiles: up to kPrefixTileSeqs neighbouring sequences against their
// prefix and against the pages of each. Units of a tile: its pages by two, plus kPrefixPieceUnits for loading Q and
// writing the partial results.
constexpr int kPrefixTileSeqs = 4;
constexpr int kPrefixPieceUnits = 6;
struct PrefixParams {
  const uint16_t* q;            // [B][64][256] bf16 bits
  const int32_t* group_starts;  // [n_groups + 1]
  const int32_t* prefix_pages;  // [n_groups]
  const int32_t* page_table;
  const int32_t* seq_lens;
  const float* k_scale;         // [num_pages][64] (null: bf16 cache)
  const float* v_scale;
  // partial results, rows of [64 heads][256] (and [64] LSEs): row 4 (pair + t) + s for sequence s of row tile t
  float* part_o;
  float* part_lse;
  int4* parts;                  // [B]: b's partial results, two runs of rows kPrefixTileSeqs apart: first row, number, twice
  uint16_t* out;                // [B][64][256] bf16 bits
  float* lse;                   // [B][64]
  uint32_t* err;
  float scale;
  int B, n_groups, max_pages, num_pages, pairs;
  uint64_t wait_budget_ns;
};

// Attention of chunks of new tokens. The work is a line of row tiles, up to kChunkTileTokens neighbouring tokens of a
// sequence against what they see. Units of a tile: its pages by two, and what goes by between two tiles, for which quantised
// caches split Q: with 1, 2, 3, 4, 6 of them steps that mix long and short tiles took 40.3, 39.9, 39.1, 42.4, 47.2 us on a bf16
// cache, and 1303, 1087, 935, 840, 870 us on a 4-bit one.
constexpr int kChunkTileTokens = 4, kChunkMaxPairs = 95;
constexpr int kChunkPieceUnits = 3, kChunkPieceUnitsQuantised = 4;
// What L2's 129 MB hold: lines that both dies read are in both halves.
constexpr long long kChunkL2Bytes = 80ll << 20;
struct ChunkParams {
  const uint16_t* q;         // [max_tokens][64][256] bf16 bits
  const void* v_cache;
  const int32_t* q_starts;   // [B + 1]
  const int32_t* page_table;
  const int32_t* seq_lens;
  const float* k_scale;      // [num_pages][64] (E4M3 and E2M1)
  const float* v_scale;
  // partial results, 256 rows of [256] (and LSEs) each: 2 pair of the tile that began before the pair's range, 2 pair + 1 of
  // the one that ends behind it
  float* part_o;
  float* part_lse;
  // [pairs + 1]: tiles that lie in several ranges: first row, tokens | parts << 8 (0 behind the last), first pair, first of the
  // combine's groups
  int4* parts;
  uint16_t* out;             // [max_tokens][64][256] bf16 bits
  float* lse;                // [max_tokens][64]
  uint32_t* err;
  float scale;
  int B, max_tokens, max_pages, num_pages, pairs;
  int piece_units;           // of a tile besides its pages'
  int l2_units;              // units whose K and V L2 holds
  int fmt;                   // kKvBf16, kKvE4M3 or kKvE2M1
  uint64_t wait_budget_ns;
};

// Kernel launchers (each returns the launch's cudaError_t).
cudaError_t launch_kv_append_slots(const AppendSlotsParams& p, cudaStream_t stream);
cudaError_t launch_kv_read(const KvReadParams& p, cudaStream_t stream);
cudaError_t launch_reserve_pages(const PageTableParams& p, cudaStream_t stream);
cudaError_t launch_release_pages(const PageTableParams& p, cudaStream_t stream);
cudaError_t launch_decode_prefix_tc(const PrefixParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map,
                                    const CUtensorMap& q_map, cudaStream_t stream);
cudaError_t launch_prefix_combine(const PrefixParams& p, cudaStream_t stream);
cudaError_t launch_chunk_attention_tc(const ChunkParams& p, const CUtensorMap& k_map, const CUtensorMap& v_map,
                                      const CUtensorMap& q_map, cudaStream_t stream);
cudaError_t launch_chunk_combine(const ChunkParams& p, cudaStream_t stream);

}  // namespace mfa
