// decode_prefix_tc.cu -- decode attention for a batch whose sequences share
// prefixes: the pages of a group's prefix are read once for four sequences at a
// time instead of once for each, and in the same kernel every sequence reads
// what it holds behind its prefix.
//
// A group's queries form one matrix of 64 n rows (64 heads, n sequences), and
//     S = Q K^T,  P = exp2(scale log2(e) S - m),  O = P V,  l = P 1
// over the prefix is ordinary matrix work: 4 * 64 * 256 flops a sequence and
// key, against 1 KB (bf16) a key for the whole group, so from about five
// sequences on the tensor cores bound it and not memory. What a sequence holds
// behind the prefix is bound by memory.
//
// Row tile: up to four neighbouring sequences, 256 rows, and as its keys the
// pages of their prefix, then the own pages of the first sequence, of the
// second, and so on. A page is therefore seen by all the rows of the tile or by
// those of one sequence; the others' rows skip its softmax and are left out of
// its P V MMAs (by their mask of output lanes, so that nothing in a sequence's
// pages, not even a NaN, reaches another's result). Own pages use a quarter of
// the rows, but a unit of two pages still takes the tensor cores less time (2048
// cycles of a pair of SMs) than HBM takes to deliver its 128 KB at the pair's
// share of the bandwidth.
//
// A cluster of two CTAs, each with 128 of the rows, works on units of 128 keys
// (two pages) with tcgen05 MMAs of cta_group::2: each CTA holds one of the two
// K pages and half of V's dimensions, and both halves feed the pair's MMAs.
// Against one CTA with 128 rows this halves what every SM reads from L2 (128 KB
// in 2048 tensor cycles, which L2 cannot serve to 152 SMs) and what the MMAs
// read from shared memory for B. TMEM holds S twice (2 x 128 columns; P
// overwrites S in place and is the A operand of P V from there) and O (256
// columns): all of it.
//
// Work split: the units of all row tiles, one after the other, form a line
// (kPrefixPieceUnits more for every tile: its Q load and partial results); each
// pair takes an equal range of it (stream-K) and writes, per row tile that it
// holds units of, normalised partial results and LSEs of the sequences that see
// any of them; the combine joins a sequence's parts.
//
// Warp roles:
//   warps 0-7  softmax: thread = row = TMEM lane; warp w and w + 4 share 32
//              rows, 64 keys of a unit each, and agree on the reference maximum,
//              which moves only when weights become large (then O is rescaled).
//   warp 8     producer (TMA, each CTA its own halves, completing on the
//              leader's barriers).
//   warp 9     TMEM allocation, and MMA issue (one thread of the leader's; the
//              other CTA's leaves the combine where the parts are).
//   warp 10    the rows behind a sequence's last token in V, zeroed up to the
//              end of an MMA's 16 keys: 0 * NaN of a stale row would poison P V.
//   warps 10-13 (E4M3 cache only, instead) V codes to f16, rows behind the last
//              token to zero.
// Every wait is bounded (the wait budget), as in the split kernel.
//
// Measured, combine included: 304 sequences behind 256 pages 172 to 178 us from
// card to card (1835 to 1900 TFLOP/s; cuBLAS reaches 1914 in a burst), E4M3 180 to
// 187; 32 behind 128 pages 26.2 us, of which 5 go by until the first S (plan, page
// ids, first loads), 10 in 9 units, 2.9 in the write-out of 128 KB a CTA (an SM
// writes 32 B a cycle) and 3.8 in the combine.
//
// E4M3 cache: S is 8-bit MMAs (kind::f8f6f4) on the raw K codes, with Q as two
// E4M3 terms under a power of two per row, split in shared memory when a row
// tile begins (two terms at twice the 16-bit rate cost what bf16 does). For P V
// four more warps turn the V codes times their scales into f16, and P is f16 as
// well: each is off by 2^-11, where E4M3 terms of P would flush a thousand small
// weights beside one large one. f16 holds the codes' and the scales' exponents
// for scales within [2^-16, 2), |v| of 0.007 to 900; of a scale outside, the
// power of two beyond goes to its key's weight instead, and the reference follows
// weights times that power: what neither large values without weight nor rows of
// zeros (whose scale the append sets to 1) take from the others' bits. Weights
// below 2^-18 of a row's largest are held to 2^-29 of it.
#include <type_traits>

#include "mfa_serving.hpp"
#include "tc_pair.cuh"

namespace mfa {
namespace {

constexpr int kSoftmaxWarps = 8, kProducerWarp = 8, kMmaWarp = 9, kTailWarp = 10, kConvertWarps = 4;
template <bool kFp8>
__host__ __device__ constexpr int threads() { return 32 * (kTailWarp + (kFp8 ? kConvertWarps : 1)); }
// Two K and two V slots, of even and odd units, one CTA's half of a unit each: K one page of 256 dims, V 128 dims of two
// pages. A K slot is free when S of its unit is done, a V slot when P V is, which the softmax warps are told anyway: the
// issuing thread commits twice a unit. (With a ring of 16 KB granules it waited four times and committed six times a
// unit, and a unit took 3600 cycles; 2650 with these slots; 2048, the tensor cores' own time, with elect_one.)
template <bool kFp8>
__host__ __device__ constexpr uint32_t slot_bytes() { return kFp8 ? 16384 : 32768; }  // as loaded
constexpr uint32_t kVSlotBytes = 32768, kVPageBytes = 16384;                          // V as the MMAs read it, 16 bits
constexpr int kSeqs = kPrefixTileSeqs;
constexpr int kScaleSlots = 4;         // E4M3: 128 K scales and 128 V scales a unit
constexpr int kScaleBytes = 1024;
constexpr int kQBytes = 65536;         // 128 rows x 256 dims, four 64-dim blocks of [128 rows x 128 B]
constexpr int kSeqQBytes = 32768;      // one sequence's rows
static_assert(kPrefixTileSeqs * kHeads == 256, "rows of a row tile");

enum Bar {
  KFull = 0,                 // [2] leader: both CTAs' halves landed
  VFull = KFull + 2,         // [2] leader; E4M3: one arrival per converting warp of the pair
  QFull = VFull + 2,         // bf16: leader; E4M3: both, each its own rows
  QReady,                    // E4M3, leader: Q split into terms, one arrival per softmax warp of the pair
  SFull,                     // [2] both: S of even and odd units
  PFull = SFull + 2,         // [2] leader: one arrival per softmax warp of the pair
  PvDone = PFull + 2,        // [2] both: P V of even and odd units
  OFree = PvDone + 2,        // leader: O has been read, one arrival per softmax warp of the pair
  Drain,                     // leader
  ScFull,                    // [kScaleSlots] E4M3, both
  ScEmpty = ScFull + kScaleSlots,   // [kScaleSlots] one arrival per softmax and converting warp of the CTA
  TailFull = ScEmpty + kScaleSlots, // [2] both: this CTA's V of a partial last unit landed (by V slot)
  TailReady = TailFull + 2,         // [2] leader: its rows behind the last token are zero, one arrival a CTA
  RawFull = TailReady + 2,          // [2] E4M3, both: this CTA's V codes landed
  RawEmpty = RawFull + 2,           // [2] one arrival per converting warp of the CTA
  kBars = RawEmpty + 2
};

// The line of work as every CTA sees it. Indices of sequences and tiles fit 16 bits (at most 1024 sequences).
struct PlanSmem {
  int32_t cost[kMaxBatch + 1];    // units of the row tiles before t; [tiles]: of all
  int32_t pages[kMaxBatch];       // prefix pages of tile t
  uint32_t len[kMaxBatch];        // tokens of sequence b, | kBehind
  uint16_t first[kMaxBatch + 2];  // first sequence of tile t; [tiles]: B
  uint16_t lead[kMaxBatch];       // the sequence whose table row gives tile t's prefix pages
  int32_t tiles;
};
constexpr uint32_t kBehind = 0x80000000u;  // b sees its tile's prefix, its own pages begin behind it
struct PlanScratch {
  int32_t count[kMaxBatch], lead[kMaxBatch], pages[kMaxBatch], group[kMaxBatch];
  uint16_t b0[kMaxBatch + 2];
  int32_t start[kMaxBatch];
  int32_t last[kMaxBatch / 32], units[kMaxBatch / 32];  // of 32 sequences, of 32 row tiles
  uint32_t begins[kMaxBatch / 32];
};
static_assert(kMaxBatch <= 32 * 32, "a lane for each 32 of the batch");

template <bool kFp8>
struct Smem {
  static constexpr uint32_t k = 0;
  static constexpr uint32_t v = k + 2 * slot_bytes<kFp8>();
  static constexpr uint32_t raw = v + 2 * kVSlotBytes;  // E4M3: V codes
  static constexpr uint32_t q = raw + (kFp8 ? 2 * slot_bytes<kFp8>() : 0);
  static constexpr uint32_t scales = q + kQBytes;
  static constexpr uint32_t plan = scales + (kFp8 ? kScaleSlots * kScaleBytes : 0);
  static constexpr uint32_t red = (plan + (uint32_t)sizeof(PlanSmem) + 15) & ~15u;  // [4][128] exchange of the row halves
  static constexpr uint32_t bars = red + 4 * 128 * 4;
  static constexpr uint32_t misc = bars + 8 * kBars;  // TMEM base, abort flag
  static constexpr uint32_t total = misc + 8;
};
static_assert(Smem<false>::total + 1024 <= 227 * 1024 && Smem<true>::total + 1024 <= 227 * 1024, "shared memory");
static_assert(2 * slot_bytes<true>() + 2 * kVSlotBytes >= sizeof(PlanScratch), "the plan's scratch lies in the K and V slots");

// ---------------------------------------------------------------- plan
__device__ __forceinline__ int own_tokens(const PlanSmem& s, int b, int prefix_pages) {
  const uint32_t len = s.len[b];
  return (int)(len & ~kBehind) - ((len & kBehind) ? prefix_pages * kPageSize : 0);
}

// A group shares its prefix if at least two of its sequences hold all of it;
// a sequence that ends inside it (or an empty slot of the batch) reads its own
// table row alone, so that no row has a mask within a shared page and nothing
// behind its last token is ever read for it. Row tiles: four neighbours at a time within a
// shared group, and within a run of sequences that share nothing. All threads;
// ends with a barrier.
__device__ void build_plan(const PrefixParams& p, PlanSmem& s, PlanScratch& t, uint32_t* err) {
  const int n = p.n_groups, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kThreads = blockDim.x;
  // (by other warps than the lengths, so that neither waits for the other's loads)
  for (int g = (threadIdx.x + kThreads - 128) % kThreads; g < n; g += kThreads) {
    int pages = __ldcg(p.prefix_pages + g);
    if (pages < 0 || pages > p.max_pages) {
      raise_error(err, MFA_DEVERR_CAPACITY);
      pages = pages < 0 ? 0 : p.max_pages;
    }
    t.pages[g] = pages;
    t.count[g] = 0;
    t.lead[g] = kMaxBatch;
  }
  for (int b = threadIdx.x; b < p.B; b += kThreads)
    s.len[b] = (uint32_t)clamp_len(__ldcg(p.seq_lens + b), p.max_pages * kPageSize, err);
  if (warp == kThreads / 32 - 1) {  // starts, made non-decreasing within [0, B]: no sequence lies in two groups
    int top = 0;
    for (int g0 = 0; g0 <= n; g0 += 32) {
      const int g = g0 + lane;
      const int raw = g <= n ? __ldcg(p.group_starts + g) : 0;
      int x = min(max(raw, 0), p.B);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x = max(x, y);
      }
      x = max(x, top);
      if (g <= n) {
        if (x != raw) raise_error(err, MFA_DEVERR_CAPACITY);
        t.b0[g] = (uint16_t)x;
      }
      top = __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    int of = -1;  // the group whose whole prefix b holds, | a mark where it does not
    if (b >= t.b0[0] && b < t.b0[n]) {
      of = last_at_most(t.b0, n + 1, b);
      const int pages = t.pages[of];
      if (pages > 0 && (int)s.len[b] >= pages * kPageSize) {
        s.len[b] |= kBehind;
        atomicAdd(&t.count[of], 1);
        atomicMin(&t.lead[of], b);
      }
    }
    t.group[b] = of;
  }
  __syncthreads();
  // tiles begin every four sequences from where the shared group (or the run without one) begins
  auto key = [&](int b) { return b >= 0 && t.group[b] >= 0 && t.count[t.group[b]] >= 2 ? t.group[b] : -1; };
  // A warp takes 32 sequences, or 32 tiles, at a time; what it needs of those before is read by a lane for each 32.
  const int chunks = (p.B + 31) / 32, warps = kThreads / 32;
#pragma unroll 1
  for (int c = warp; c < chunks; c += warps) {
    const int b = 32 * c + lane;
    int x = b < p.B && (b == 0 || key(b - 1) != key(b)) ? b : -1;  // where the run begins, if within these 32
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = max(x, y);
    }
    t.start[b] = x;
    if (lane == 31) t.last[c] = x;
  }
  if (chunks > 1) __syncthreads(); else __syncwarp();
#pragma unroll 1
  for (int c = warp; c < chunks; c += warps) {
    const int b = 32 * c + lane;
    const int from = max(t.start[b], __reduce_max_sync(0xffffffffu, lane < c ? t.last[lane] : -1));
    const uint32_t begins = __ballot_sync(0xffffffffu, b < p.B && (b - from) % kSeqs == 0);
    if (lane == 0) t.begins[c] = begins;
  }
  if (chunks > 1) __syncthreads(); else __syncwarp();
#pragma unroll 1
  for (int c = warp; c < chunks; c += warps) {
    const int b = 32 * c + lane, g = b < p.B ? key(b) : -1;
    const uint32_t begins = t.begins[c];
    const int before = __reduce_add_sync(0xffffffffu, lane < c ? __popc(t.begins[lane]) : 0);
    if ((begins >> lane) & 1) {
      const int i = before + __popc(begins & ((1u << lane) - 1));
      s.first[i] = (uint16_t)b;
      s.pages[i] = g >= 0 ? t.pages[g] : 0;
      s.lead[i] = g >= 0 ? (uint16_t)t.lead[g] : 0;
    }
    if (b < p.B && g < 0) s.len[b] &= ~kBehind;
    if (b == p.B - 1) {
      s.tiles = before + __popc(begins);
      s.first[before + __popc(begins)] = (uint16_t)p.B;
    }
  }
  if (chunks > 1) __syncthreads(); else __syncwarp();
  const int tiles = chunks > 1 || warp == 0 ? s.tiles : 0;
#pragma unroll 1
  for (int c = warp; 32 * c < tiles; c += warps) {
    const int i = 32 * c + lane;
    int u = 0;
    if (i < tiles) {
      int pages = s.pages[i];
      for (int b = s.first[i]; b < s.first[i + 1]; ++b) pages += pages_of(own_tokens(s, b, s.pages[i]));
      u = pages ? (pages + 1) / 2 + kPrefixPieceUnits : 0;
    }
    const int x = warp_inclusive_sum(u, lane);
    if (i < tiles) s.cost[i] = x - u;
    if (i == tiles - 1) s.cost[tiles] = x;
    if (lane == 31) t.units[c] = x;
  }
  if (tiles > 32) {
    __syncthreads();
#pragma unroll 1
    for (int c = warp; 32 * c < tiles; c += warps) {
      const int i = 32 * c + lane, before = __reduce_add_sync(0xffffffffu, lane < c ? t.units[lane] : 0);
      if (i < tiles) s.cost[i] += before;
      if (i == tiles - 1) s.cost[tiles] += before;
    }
  }
  fence_proxy_async_smem();  // the scratch is TMA's from here on
  __syncthreads();
}

// Pairs that have work: with fewer units than pairs, every range holds one.
__device__ __forceinline__ int busy_pairs(const PrefixParams& p, int units) { return min(p.pairs, max(units, 1)); }

// Where the combine finds each sequence's partial results: of the pairs that hold prefix units, and of those that hold
// pages of its own. One warp of each pair.
__device__ void publish_plan(const PrefixParams& p, const PlanSmem& s, int pair, int lane) {
  const int C = s.cost[s.tiles], W = busy_pairs(p, C);
  for (int b = 32 * pair + lane; b < p.B; b += 32 * p.pairs) {
    const int t = last_at_most(s.first, s.tiles, b), j = b - s.first[t], prefix = s.pages[t];
    int c = prefix;
    for (int i = s.first[t]; i < b; ++i) c += pages_of(own_tokens(s, i, prefix));
    const int own = pages_of(own_tokens(s, b, prefix));
    auto pair_of = [&](int page) { return pair_of_unit(s.cost[t] + kPrefixPieceUnits + page / 2, C, W); };
    auto row = [&](int w) { return (w + t) * kSeqs + j; };
    int4 parts = make_int4(0, 0, 0, 0);
    int w = -1;  // the last pair so far
    if (s.len[b] & kBehind) {
      const int w0 = pair_of(0);
      w = pair_of(prefix - 1);
      parts.x = row(w0);
      parts.y = w - w0 + 1;
    }
    if (own) {
      const int w0 = max(w + 1, pair_of(c));
      parts.z = row(w0);
      parts.w = max(0, pair_of(c + own - 1) - w0 + 1);
    }
    p.parts[b] = parts;
  }
}

// A pair's pieces, in order: units [u0, u1) of one row tile. Page k of the tile is the prefix's for k < c[0], then
// sequence s's for c[s] <= k < c[s + 1].
struct Piece {
  int t;              // row tile
  int b, seqs;        // first sequence, sequences (1 to kSeqs)
  int c[kSeqs + 1];
  uint32_t tails;     // byte s: tokens on the last own page of sequence s
  uint32_t behind;    // bit s: sequence s sees the prefix
  int u0, u1;         // units
  int x;              // line position behind the tile
  __device__ int owner(int k) const {  // kSeqs: the prefix's
    return k < c[0] ? kSeqs : k < c[1] ? 0 : k < c[2] ? 1 : k < c[3] ? 2 : 3;
  }
  // tokens on page k, 0 behind the tile's last page
  __device__ int tokens(int k) const {
    if (k < c[0]) return kPageSize;
    if (k >= c[kSeqs]) return 0;
    const int s = owner(k);
    const int end = s == 0 ? c[1] : s == 1 ? c[2] : s == 2 ? c[3] : c[4];
    return k + 1 < end ? kPageSize : (int)((tails >> (8 * s)) & 0xFF);
  }
};
__device__ __forceinline__ bool next_piece(const PlanSmem& s, int hi, Piece& q) {
  while (q.x < hi) {
    const int t = last_at_most(s.cost, s.tiles, q.x), first = s.cost[t], len = s.cost[t + 1] - first;
    q.t = t;
    q.b = s.first[t];
    q.seqs = s.first[t + 1] - q.b;
    q.c[0] = s.pages[t];
    q.tails = q.behind = 0;
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
      const int tokens = i < q.seqs ? own_tokens(s, q.b + i, q.c[0]) : 0;
      q.c[i + 1] = q.c[i] + pages_of(tokens);
      q.tails |= (uint32_t)(tokens > 0 ? (tokens - 1) % kPageSize + 1 : 0) << (8 * i);
      if (i < q.seqs && (s.len[q.b + i] & kBehind)) q.behind |= 1u << i;
    }
    q.u0 = max(0, q.x - first - kPrefixPieceUnits);
    q.u1 = min(len, hi - first) - kPrefixPieceUnits;
    q.x = first + len;
    if (q.u0 < q.u1) return true;
  }
  return false;
}

// ---------------------------------------------------------------- producer
// Page ids of a tile: a window of 64 held by the warp (32 ahead of need).
struct TilePages {
  int end, base, a, b;
  __device__ int load(int k, const PrefixParams& p, const PlanSmem& s, const Piece& q) const {
    if (k >= end) return 0;
    const int o = q.owner(k);
    const int c = o == 0 ? q.c[0] : o == 1 ? q.c[1] : o == 2 ? q.c[2] : q.c[3];
    const int seq = o == kSeqs ? s.lead[q.t] : q.b + o;
    const int at = o == kSeqs ? k : k - c + (((q.behind >> o) & 1) ? q.c[0] : 0);
    return __ldcg(p.page_table + (size_t)seq * p.max_pages + at);
  }
  __device__ int checked(int id, const PrefixParams& p) const {
    if (id >= 0 && id < p.num_pages) return id;
    raise_error(p.err, MFA_DEVERR_PAGE);
    return 0;
  }
  __device__ void start(int k, const PrefixParams& p, const PlanSmem& s, const Piece& q, int lane) {
    end = min(q.c[kSeqs], 2 * q.u1);
    base = k;
    const int x = load(base + lane, p, s, q), y = load(base + 32 + lane, p, s, q);  // both on their way at once
    a = checked(x, p);
    b = checked(y, p);
  }
  __device__ int get(int k, const PrefixParams& p, const PlanSmem& s, const Piece& q, int lane) {
    while (k >= base + 64) {
      base += 32;
      a = b;
      b = checked(load(base + 32 + lane, p, s, q), p);
    }
    const int i = k - base;
    return i < 32 ? __shfl_sync(0xffffffffu, a, i) : __shfl_sync(0xffffffffu, b, i - 32);
  }
};

template <bool kFp8>
__device__ void producer_role(const PrefixParams& p, const CUtensorMap* kmap, const CUtensorMap* vmap,
                              const CUtensorMap* qmap, const Ctx& cx, const PlanSmem& s, int pair, int lo, int hi) {
  using Sm = Smem<kFp8>;
  constexpr uint32_t kSlot = slot_bytes<kFp8>(), kPage = kSlot / 2;
  constexpr int kCols = kFp8 ? 128 : 64;  // columns of a copy: 128 bytes
  const int lane = threadIdx.x & 31, r = (int)cx.rank;
  const uint64_t pol_shared = policy_evict_normal(), pol_own = policy_evict_first();
  uint32_t pieces = 0, tails[2] = {0, 0};
  // K of unit `n` (and its scales): this CTA's page, page r of the two, on the leader's barrier, on which the leader
  // announces the bytes of both CTAs
  auto load_k = [&](uint32_t n, int pa, int pb, uint64_t pol) -> bool {
    const uint32_t slot = n & 1;
    if (n >= 2 && !cx.wait_warp(SFull + slot, ((n >> 1) & 1) ^ 1)) return false;
    const int page = r == 0 ? pa : pb;
    if (elect_one()) {
      const uint32_t dst = cx.base + Sm::k + slot * kSlot, bar = cx.leader_bar(KFull + slot);
      if (r == 0) mbar_arrive_expect_tx(cx.bar(KFull + slot), pb >= 0 ? 2 * kSlot : kSlot);
      if (page >= 0)
#pragma unroll
        for (int d = 0; d < kHeadDim / kCols; ++d)
          tma_load_2d_pair(dst + d * 8192, kmap, d * kCols, page * kPageSize, bar, pol);
    }
    if constexpr (kFp8) {  // the scales of all the unit's keys, for this CTA's rows
      const uint32_t sc_slot = n % kScaleSlots;
      if (!cx.wait_warp(ScEmpty + sc_slot, ((n / kScaleSlots) & 1) ^ 1)) return false;
      if (elect_one()) {
        const uint32_t sc = cx.base + Sm::scales + sc_slot * kScaleBytes, sb = cx.bar(ScFull + sc_slot);
        constexpr uint32_t kPageScales = kPageSize * sizeof(float);
        mbar_arrive_expect_tx(sb, (pb >= 0 ? 4 : 2) * kPageScales);
        bulk_load(sc, p.k_scale + (size_t)pa * kPageSize, kPageScales, sb);
        bulk_load(sc + 512, p.v_scale + (size_t)pa * kPageSize, kPageScales, sb);
        if (pb >= 0) {
          bulk_load(sc + kPageScales, p.k_scale + (size_t)pb * kPageSize, kPageScales, sb);
          bulk_load(sc + 512 + kPageScales, p.v_scale + (size_t)pb * kPageSize, kPageScales, sb);
        }
      }
    }
    return true;
  };
  // V of unit `n`: this CTA's 128 dims of each page. That of a tail lands on this CTA's own barrier, for the warp that
  // zeroes its rows; E4M3: all of it does, for the warps that convert it.
  auto load_v = [&](uint32_t n, int pa, int pb, bool tail, uint64_t pol) -> bool {
    const uint32_t slot = n & 1, parity = ((n >> 1) & 1) ^ 1, bytes = pb >= 0 ? kSlot : kPage;
    uint32_t dst, bar;
    if constexpr (kFp8) {
      if (!cx.wait_warp(RawEmpty + slot, parity)) return false;
      dst = cx.base + Sm::raw + slot * kSlot;
      bar = cx.bar(RawFull + slot);
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
    } else {
      if (n >= 2 && !cx.wait_warp(PvDone + slot, parity)) return false;
      dst = cx.base + Sm::v + slot * kSlot;
      bar = tail ? cx.bar(TailFull + slot) : cx.leader_bar(VFull + slot);
      if (lane == 0 && r == 0) mbar_arrive_expect_tx(cx.bar(VFull + slot), tail ? 0 : 2 * bytes);
      if (lane == 0 && tail) mbar_arrive_expect_tx(bar, bytes);
      tails[slot] += tail;
    }
    if (elect_one())
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i == 0 || pb >= 0)
#pragma unroll
          for (int d = 0; d < 128 / kCols; ++d)
            tma_load_2d_pair(dst + i * kPage + d * 8192, vmap, r * 128 + d * kCols, (i ? pb : pa) * kPageSize, bar, pol);
    return true;
  };
  Piece q;
  q.x = lo;
  uint32_t cnt = 0;      // units whose K has been loaded
  int va = -1, vb = -1;  // the last of them: its V is still to be loaded (V trails K by a unit, as the MMAs use them)
  bool vtail = false, good = true;
  uint64_t vpol = pol_own;
  while (good && next_piece(s, hi, q)) {
    // Q may be replaced once S of every unit so far is done
    good = cnt == 0 || cx.wait_warp(SFull + ((cnt - 1) & 1), ((cnt - 1) >> 1) & 1);
    if (!good) break;
    if (elect_one()) {
      const int here = min(2, max(0, q.seqs - 2 * r));  // this CTA's sequences
      if (kFp8)
        mbar_arrive_expect_tx(cx.bar(QFull), here * kSeqQBytes);
      else if (r == 0)
        mbar_arrive_expect_tx(cx.bar(QFull), q.seqs * kSeqQBytes);
      const uint32_t bar = kFp8 ? cx.bar(QFull) : cx.leader_bar(QFull);
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (h < here)
            tma_load_2d_pair(cx.base + Sm::q + d * 16384 + h * 8192, qmap, d * 64, (q.b + 2 * r + h) * kHeads, bar, pol_shared);
    }
    ++pieces;
    TilePages ids;
    ids.start(2 * q.u0, p, s, q, lane);
    for (int u = q.u0; good && u < q.u1; ++u) {
      const int pa = ids.get(2 * u, p, s, q, lane);
      const int pb = 2 * u + 1 < q.c[kSeqs] ? ids.get(2 * u + 1, p, s, q, lane) : -1;
      const uint64_t pol = 2 * u < q.c[0] ? pol_shared : pol_own;
      good = load_k(cnt, pa, pb, pol);
      if (good && va >= 0) good = load_v(cnt - 1, va, vb, vtail, vpol);
      ++cnt;
      va = pa;
      vb = pb;
      vtail = is_partial(q.tokens(2 * u)) || is_partial(q.tokens(2 * u + 1));
      vpol = pol;
    }
    if (kFp8 && good) {  // E4M3: the next row tile's Q is split only behind this one's last P V
      good = load_v(cnt - 1, va, vb, vtail, vpol);
      va = -1;
    }
  }
  if (good && va >= 0) good = load_v(cnt - 1, va, vb, vtail, vpol);
  // Every copy of both CTAs must land before either leaves: this CTA's barriers and the leader's tell, and the other CTA
  // stays until the cluster's last barrier.
  if (lane == 0) {
    for (uint32_t k = cnt > 2 ? cnt - 2 : 0; k < cnt; ++k) {
      if (r == 0) (void)mbar_wait(cx.bar(KFull + (k & 1)), (k >> 1) & 1, kDrainNs, nullptr, p.err);
      if ((kFp8 || r == 0) && (good || k + 1 < cnt))
        (void)mbar_wait(cx.bar((kFp8 ? RawFull : VFull) + (k & 1)), (k >> 1) & 1, kDrainNs, nullptr, p.err);
    }
    for (int i = 0; i < 2; ++i)
      if (tails[i]) (void)mbar_wait(cx.bar(TailFull + i), (tails[i] - 1) & 1, kDrainNs, nullptr, p.err);
    if constexpr (kFp8)
      for (uint32_t k = cnt > (uint32_t)kScaleSlots ? cnt - kScaleSlots : 0; k < cnt; ++k)
        (void)mbar_wait(cx.bar(ScFull + k % kScaleSlots), (k / kScaleSlots) & 1, kDrainNs, nullptr, p.err);
    if (pieces && (kFp8 || r == 0)) (void)mbar_wait(cx.bar(QFull), (pieces - 1) & 1, kDrainNs, nullptr, p.err);
  }
  __syncwarp();
}

// ---------------------------------------------------------------- rows behind the last token
__device__ void tail_role(const PrefixParams& p, const Ctx& cx, const PlanSmem& s, int pair, int lo, int hi) {
  const int lane = threadIdx.x & 31;
  uint32_t cnt = 0, tails[2] = {0, 0};
  Piece q;
  q.x = lo;
  while (next_piece(s, hi, q)) {
    for (int u = q.u0; u < q.u1; ++u, ++cnt) {
      const int tokens[2] = {q.tokens(2 * u), q.tokens(2 * u + 1)};
      if (!is_partial(tokens[0]) && !is_partial(tokens[1])) continue;
      const uint32_t slot = cnt & 1;
      if (!cx.wait_warp(TailFull + slot, tails[slot] & 1)) return;
      ++tails[slot];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!is_partial(tokens[i])) continue;
        const uint32_t base = cx.base + Smem<false>::v + slot * kVSlotBytes + i * kVPageBytes + tokens[i] * 128;
        const int words = (kKeyStep - tokens[i] % kKeyStep) * 8;  // 16 B words of a 64-dim chunk's rows
        for (int w = lane; w < words * 2; w += 32)
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(base + (w / words) * 8192 + (w % words) * 16), "r"(0)
                       : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(cx.leader_bar(TailReady + slot));
    }
  }
}

// E4M3: V of a unit as P V reads it, f16 of code * scale * 2^kUp without the scale's shift (off by 2^-11 for the scale
// and 2^-11 for the product), from the codes: per page [64 rows x 128 dims] to two 64-dim chunks of [64 rows x 128 B], both
// with the 128-byte swizzle. A thread takes 16 codes of a row and of every 16th row after it; rows behind the last token
// become zeros. Eight neighbouring threads take half of rows r and r ^ 5, whose swizzles differ in the bits that keep
// both the codes they read and the values they write on banks of their own. That the scales are applied here spares the
// softmax threads 64 values each from shared memory, whose bandwidth the MMAs need.
__device__ void convert_role(const PrefixParams& p, const Ctx& cx, const PlanSmem& s, int pair, int lo, int hi,
                             const uint8_t* gbase) {
  using Sm = Smem<true>;
  const int lane = threadIdx.x & 31, t = threadIdx.x - 32 * kTailWarp;
  const int row0 = (2 * (t >> 4)) ^ (t & 4 ? 5 : 0);
  const int c = (t & 3) | ((t >> 1) & 4);  // 16-code chunk: dims [16 c, 16 c + 16)
  const uint32_t from = row0 * 128 + ((c ^ (row0 & 7)) << 4);  // rows 16 apart share the swizzle
  const uint32_t to = (c >> 2) * 8192 + row0 * 128;
  const uint32_t to0 = to + (((2 * (c & 3)) ^ (row0 & 7)) << 4), to1 = to + (((2 * (c & 3) + 1) ^ (row0 & 7)) << 4);
  uint32_t n = 0;
  Piece q;
  q.x = lo;
  while (next_piece(s, hi, q)) {
    for (int u = q.u0; u < q.u1; ++u, ++n) {
      const uint32_t slot = n & 1, sc_slot = n % kScaleSlots;
      const uint32_t src = cx.base + Sm::raw + slot * slot_bytes<true>() + from, dst = cx.base + Sm::v + slot * kVSlotBytes;
      const float* sc = reinterpret_cast<const float*>(gbase + Sm::scales + sc_slot * kScaleBytes) + kUnitKeys;
      if (!cx.wait_warp(ScFull + sc_slot, (n / kScaleSlots) & 1)) return;
      if (!cx.wait_warp(RawFull + slot, (n >> 1) & 1)) return;
      if (n >= 2 && !cx.wait_warp(PvDone + slot, ((n >> 1) & 1) ^ 1)) return;
#pragma unroll
      for (int page = 0; page < 2; ++page) {
        const int valid = q.tokens(2 * u + page);
        uint4 v[4];
        __half2 scale[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = ld_shared_v4(src + page * 8192 + i * 2048);
          const float s = sc[page * kPageSize + row0 + 16 * i];
          scale[i] = __float2half2_rn(s * exp2_int(E4m3Range::kUp - scale_shift<E4m3Range>(s)));
        }
        if (valid < kPageSize) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (row0 + 16 * i >= valid) {
              v[i] = make_uint4(0u, 0u, 0u, 0u);
              scale[i] = __float2half2_rn(0.0f);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          uint32_t h[2][4];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[k >> 1] >> (16 * (k & 1))), __NV_E4M3);
            const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&r), scale[i]);
            h[k >> 2][k & 3] = *reinterpret_cast<const uint32_t*>(&y);
          }
          st_shared_v4(dst + page * kVPageBytes + i * 2048 + to0, h[0]);
          st_shared_v4(dst + page * kVPageBytes + i * 2048 + to1, h[1]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(cx.bar(RawEmpty + slot));
        mbar_arrive(cx.bar(ScEmpty + sc_slot));
        mbar_arrive_pair(cx.leader_bar(VFull + slot));
      }
    }
  }
}

// ---------------------------------------------------------------- MMA issue (one thread of the leader)
template <bool kFp8>
__device__ void mma_role(const PrefixParams& p, const Ctx& cx, const PlanSmem& s, int pair, int lo, int hi,
                         uint32_t tmem) {
  constexpr uint32_t idesc_s = idesc_f16(256, kSCols, kFp8 ? 0 : 1, 0, 0);    // A = Q, B = K, both K-major (format 0: E4M3)
  constexpr uint32_t idesc_o = idesc_f16(256, kHeadDim, kFp8 ? 0 : 1, 0, 1);  // A = P (TMEM), B = V (dim-major; format 0: f16)
  using Sm = Smem<kFp8>;
  uint32_t pieces = 0, s_cnt = 0, p_cnt = 0, tails[2] = {0, 0};
  // Descriptors of the operands' first blocks; a block `bytes` further on has bytes / 16 more in the address field, which
  // holds every shared address without a carry.
  auto ahead = [](uint64_t desc, uint32_t bytes) -> uint64_t { return desc + (bytes >> 4); };
  const uint64_t q_desc = smem_desc_sw128(cx.base + Sm::q, 16, 1024);
  const uint64_t k_desc0 = smem_desc_sw128(cx.base + Sm::k, 16, 1024);
  const uint64_t v_desc0 = smem_desc_sw128(cx.base + Sm::v, 8192, 1024);
  // The tensor cores hold a few MMAs behind the one they work on, so what this thread does between two batches of them
  // costs nothing as long as it is short: barriers are looked at in the middle of a batch, for the next one, and waited
  // for only if that found them not yet done.
  bool k_ready = false, pv_ready = false;
  auto peek = [&](int i, uint32_t parity) -> bool { return mbar_test_wait(cx.bar(i), parity); };
  // S of unit s_cnt; p_next: a P V is to follow
  auto do_s = [&](bool p_next) -> bool {
    const uint32_t buf = s_cnt & 1, d = tmem + buf * kSCols;  // its last reader, P V of two units ago, was issued before
    if (!k_ready && !cx.wait(KFull + buf, (s_cnt >> 1) & 1)) return false;
    k_ready = false;
    tc_fence_after();
    const uint64_t k_desc = ahead(k_desc0, buf * slot_bytes<kFp8>());
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i == 8) pv_ready = p_next && peek(VFull + (p_cnt & 1), (p_cnt >> 1) & 1) && peek(PFull + (p_cnt & 1), (p_cnt >> 1) & 1);
      if constexpr (kFp8) {  // Q's term i / 8, 128-dim half, 32 dims
        const int h = (i >> 2) & 1, kk = i & 3;
        tc_mma_pair_f8(d, ahead(q_desc, h * 32768 + (i >> 3) * 16384 + kk * 32), ahead(k_desc, h * 8192 + kk * 32), idesc_s, i != 0);
      } else {  // 64-dim block, 16 dims
        const int e = i >> 2, kk = i & 3;
        tc_mma_pair(d, ahead(q_desc, e * 16384 + kk * 32), ahead(k_desc, e * 8192 + kk * 32), idesc_s, i != 0);
      }
    }
    tc_commit_pair(cx.bar(SFull + buf));
    ++s_cnt;
    return true;
  };
  // P V of a unit. A page is seen by the sequences of `seen` (bits); those without O in this piece yet get theirs from
  // its first MMA, which does not add.
  struct Unit {
    int tokens[2];
    uint32_t seen[2];
    uint32_t all;  // the sequences of the tile
    bool pending, first;
    uint32_t piece;
  };
  uint32_t begun = 0;  // sequences that have O in the piece of the P V issued last
  auto do_pv = [&](const Unit& v) -> bool {
    constexpr int kSteps = kPageSize / kKeyStep;
    const uint32_t buf = p_cnt & 1, a = tmem + buf * kSCols, d = tmem + kTmemO;
    if (v.first) {
      begun = 0;
      if (!cx.wait(OFree, (v.piece & 1) ^ 1)) return false;
    }
    if (!kFp8 && (is_partial(v.tokens[0]) || is_partial(v.tokens[1])) && !cx.wait(TailReady + buf, tails[buf]++ & 1)) return false;
    if (!pv_ready && !(cx.wait(VFull + buf, (p_cnt >> 1) & 1) && cx.wait(PFull + buf, (p_cnt >> 1) & 1))) return false;
    tc_fence_after();
    const uint64_t v_desc = ahead(v_desc0, buf * kVSlotBytes);
    auto a_of = [&](int i, int kk) { return a + i * 64 + (kk >> 1) * 32 + (kk & 1) * 8; };  // page i, step kk
    if (v.tokens[0] + v.tokens[1] == kUnitKeys && v.seen[0] == v.all && v.seen[1] == v.all) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk)
          tc_mma_pair_tmem_a(d, a_of(i, kk), ahead(v_desc, i * kVPageBytes + kk * 2048), idesc_o, (i | kk) != 0 || begun != 0);
        if (i == 0) k_ready = peek(KFull + (s_cnt & 1), (s_cnt >> 1) & 1);
      }
      begun = v.all;
    } else {
      for (int i = 0; i < 2; ++i) {
        const uint32_t seen = i ? v.seen[1] : v.seen[0];
        const int steps = ((i ? v.tokens[1] : v.tokens[0]) + kKeyStep - 1) / kKeyStep;
        uint32_t off[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) off[w] = ((seen >> (w >> 1)) & 1) ? 0u : 0xFFFFFFFFu;
        for (int kk = 0; kk < steps; ++kk)
          tc_mma_pair_tmem_a_masked(d, a_of(i, kk), ahead(v_desc, i * kVPageBytes + kk * 2048), idesc_o, off,
                                    kk != 0 || (begun & seen) != 0);
        if (steps) begun |= seen;
      }
      k_ready = false;
    }
    tc_commit_pair(cx.bar(PvDone + buf));
    ++p_cnt;
    return true;
  };
  Piece q;
  q.x = lo;
  Unit pend{};  // the unit whose P V is still to be issued
  bool good = true;
  while (good && next_piece(s, hi, q)) {
    good = cx.wait(kFp8 ? QReady : QFull, pieces & 1);
    for (int u = q.u0; good && u < q.u1; ++u) {
      good = do_s(pend.pending);
      if (good && pend.pending) good = do_pv(pend);
      pend.pending = true;
      pend.first = u == q.u0;
      pend.piece = pieces;
      pend.all = (1u << q.seqs) - 1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int k = 2 * u + i, o = q.owner(k);
        pend.tokens[i] = q.tokens(k);
        pend.seen[i] = o == kSeqs ? q.behind : 1u << o;
      }
    }
    if (kFp8 && good) {  // the softmax warps split the next Q once they have read this O
      pv_ready = false;
      good = do_pv(pend);
      pend.pending = false;
    }
    ++pieces;
  }
  if (good && pend.pending) {
    pv_ready = false;
    (void)do_pv(pend);
  }
  tc_commit_pair(cx.bar(Drain));  // every MMA is done before TMEM is given back
  (void)mbar_wait(cx.bar(Drain), 0, kDrainNs, nullptr, p.err);
}

// ---------------------------------------------------------------- softmax
// E4M3: the bf16 Q of this CTA's 128 rows (four 64-dim blocks of [128 rows x 128 B], 128-byte swizzle) becomes, in
// place, two E4M3 terms of Q * 2^e ([128-dim half][term][128 rows x 128 B]): the first rounds the scaled value, the second
// the rest, which is exact unless it falls below the E4M3 normal range (2^-18.8 of the row's largest |q|). 2^e is the
// largest power of two that keeps the row within the E4M3 maximum, 448. Thread (row, half) takes the 128 dims of its
// half, whose terms lie where they did: the second block is read whole before the terms of the first replace either.
// All softmax threads; red: their exchange. Returns 2^-e, NaN for a row with an infinity (which E4M3 would hold as 448; a NaN
// stays one in the terms).
__device__ __forceinline__ float split_q(uint32_t q_addr, float* red, int row, int quad, int half) {
  const uint32_t at = q_addr + half * 32768 + row * 128;  // the first of the two blocks; the second 16 KB on
  auto chunk = [&](int j) { return ((j ^ (row & 7)) << 4); };
  uint4 v[8];
  float top = 0.0f;
  auto largest = [&](const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
  };
#pragma unroll
  for (int j = 0; j < 8; ++j) largest(ld_shared_v4(at + chunk(j)));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = ld_shared_v4(at + 16384 + chunk(j));
    largest(v[j]);
  }
  red[half * 128 + row] = top;
  barrier_rows(quad);
  top = fmaxf(red[row], red[128 + row]);
  int e = 0;
  if (top > 0.0f && top < INFINITY) {
    const uint32_t bits = __float_as_uint(top);
    e = ((bits & 0x7FFFFFu) <= 0x600000u ? 8 : 7) - ((int)((bits >> 23) & 0xFFu) - 127);  // top * 2^e in (224, 448]
    e = max(-126, min(126, e));
  }
  const float up = exp2_int(e);
  auto store = [&](int o, const uint4& x, const uint4& y) {  // 16 dims
    uint32_t a1[2], a2[2], b1[2], b2[2];
    split_q8<false>(x, up, a1, a2);
    split_q8<false>(y, up, b1, b2);
    const uint32_t t1[4] = {a1[0], a1[1], b1[0], b1[1]}, t2[4] = {a2[0], a2[1], b2[0], b2[1]};
    st_shared_v4(at + chunk(o), t1);
    st_shared_v4(at + 16384 + chunk(o), t2);
  };
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    const uint4 x = ld_shared_v4(at + chunk(2 * o)), y = ld_shared_v4(at + chunk(2 * o + 1));
    store(o, x, y);
  }
#pragma unroll
  for (int o = 4; o < 8; ++o) store(o, v[2 * o - 8], v[2 * o - 7]);
  fence_proxy_async_smem();
  return top < INFINITY ? exp2_int(-e) : __uint_as_float(0x7FFFFFFFu);
}

template <bool kFp8>
__device__ void softmax_role(const PrefixParams& p, const Ctx& cx, const PlanSmem& s, int pair, int lo, int hi, uint32_t tmem, uint8_t* gbase) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = warp >> 2, quad = warp & 3, row = 32 * quad + lane;
  const uint32_t lanes = (uint32_t)(32 * quad) << 16;
  const float c2 = p.scale == 0.0f && !kFp8 ? 1e-37f : p.scale * kLog2e;  // (0 times an infinity would be NaN)
  const uint32_t p_full = cx.leader_bar(PFull), o_free = cx.leader_bar(OFree);
  float* red = reinterpret_cast<float*>(gbase + Smem<kFp8>::red);
  uint32_t cnt = 0, pieces = 0;  // units, pieces so far
  // After a wait that gave up, the warp goes through the rest of its work without waiting, so that the warps that meet it
  // at named barriers, which have no limit, do not wait for it in vain. What it computes is meaningless.
  bool alive = true;
  auto wait = [&](int bar, uint32_t parity) { alive = alive && cx.wait_warp(bar, parity); };
  // P V of the unit before `cnt`. S of that unit is done, and with it every MMA issued before it, P V of two units
  // earlier (the last on the same barrier) among them: the parity is exact.
  auto wait_pv = [&]() { wait(PvDone + ((cnt - 1) & 1), ((cnt - 1) >> 1) & 1); };
  Piece q;
  q.x = lo;
  while (next_piece(s, hi, q)) {
    const int j = 2 * (int)cx.rank + (quad >> 1);  // sequence of the row tile
    // the pages that this row sees: those below `prefix`, and own0 .. own1 - 1, of which the last holds `tail` tokens
    const int prefix = ((q.behind >> j) & 1) ? q.c[0] : 0;
    const int own0 = j == 0 ? q.c[0] : j == 1 ? q.c[1] : j == 2 ? q.c[2] : q.c[3];
    const int own1 = j == 0 ? q.c[1] : j == 1 ? q.c[2] : j == 2 ? q.c[3] : q.c[4];
    const int tail = (int)((q.tails >> (8 * j)) & 0xFF);
    auto seen = [&](int k) { return k < prefix ? kPageSize : k < own0 || k >= own1 ? 0 : k + 1 < own1 ? kPageSize : tail; };
    bool fresh = true;              // no key so far
    bool open = true;               // a row of the warp has no finite reference
    float m = -INFINITY, l = 0.0f;  // the row's reference (log2 units), and this thread's share of its denominator
    // The same of the weights as P holds them, by which O is divided: a weight that has most of the sum then cancels its
    // rounding (relative error of out 2.4e-3 -> 1.9e-3 for 128 sequences behind 512 pages, 1% slower). Of f16 weights the
    // difference does not matter. The LSE takes the unrounded sum.
    float l_p = 0.0f;
    float mul = c2;                 // of the row's products: the softmax scale, and the power of two of its Q terms
    if constexpr (kFp8) {
      wait(QFull, pieces & 1);
      mul *= split_q(cx.base + Smem<kFp8>::q, red, row, quad, half);
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(cx.leader_bar(QReady));
      barrier_rows(quad);  // red is free again
      ++pieces;
    }
    for (int u = q.u0; u < q.u1; ++u, ++cnt) {
      const uint32_t buf = cnt & 1, ts = tmem + lanes + buf * kSCols;
      const uint32_t sc_slot = cnt % kScaleSlots;
      const float* sc = reinterpret_cast<const float*>(gbase + Smem<kFp8>::scales + sc_slot * kScaleBytes);
      const int cols = seen(2 * u + half);  // this thread's keys
      if (kFp8) wait(ScFull + sc_slot, (cnt / kScaleSlots) & 1);
      // E4M3: a look at two of the 64 V scales of this warp's page; the threads of the rows together see those of both.
      bool may = false;
      if constexpr (kFp8) {
        const float2 v = reinterpret_cast<const float2*>(sc + kUnitKeys + 64 * half)[lane];
        may = may_shift<E4m3Range>(2 * lane < cols ? v.x : 1.0f) | may_shift<E4m3Range>(2 * lane + 1 < cols ? v.y : 1.0f);
      }
      wait(SFull + buf, (cnt >> 1) & 1);
      tc_fence_after();
      if (cols + seen(2 * u + (half ^ 1)) > 0) {
        // This thread's products, 32 keys at a time. P of 32 keys replaces the first 16 columns of their S.
        float2 x[16];
        const uint32_t tx = ts + 64 * half;
        auto load = [&](int g) {
          tmem_ld32(tx + g, reinterpret_cast<float*>(x));
          if constexpr (kFp8) {  // times the scales of K, of which half arrive meanwhile
            const float4* k = reinterpret_cast<const float4*>(sc + 64 * half + g);
            float4 k4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) k4[c] = k[c];
            tc_wait_ld();
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              x[2 * c] = mul2(x[2 * c], make_float2(k4[c].x, k4[c].y));
              x[2 * c + 1] = mul2(x[2 * c + 1], make_float2(k4[c].z, k4[c].w));
            }
#pragma unroll
            for (int c = 4; c < 8; ++c) {
              const float4 y = k[c];
              x[2 * c] = mul2(x[2 * c], make_float2(y.x, y.y));
              x[2 * c + 1] = mul2(x[2 * c + 1], make_float2(y.z, y.w));
            }
          } else {
            tc_wait_ld();
          }
        };
        // Products behind the last token become infinities that give weights of 0, so that one body of code does for whole
        // and partial units, which is fetched anew in every call (4 sequences behind 16 pages 14.3 us with two bodies, 14.0
        // with one). E4M3: K's scales there may be anything, so the weights are masked themselves.
        if (!kFp8 && cols < 64) {
          const float none = mul > 0.0f ? -INFINITY : INFINITY;
#pragma unroll 1
          for (int g = 0; g < 64; g += 32) {
            if (g + 32 <= cols) continue;
            load(g);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              if (g + 2 * c >= cols) x[c].x = none;
              if (g + 2 * c + 1 >= cols) x[c].y = none;
            }
            tmem_st32(tx + g, reinterpret_cast<const float*>(x));
          }
          tc_wait_st();
        }
        uint32_t w[32];
        float2 sum, sum_p;
        // weights of this thread's keys, their sums, and P; kPart: only the first `cols` of the 64 count
        auto weights = [&](auto part) {
          constexpr bool kPart = decltype(part)::value;
          const float ref = m == -INFINITY ? 0.0f : m;  // only infinite logits so far: weights of 0
          const float2 mul_2 = make_float2(mul, mul), ref_2 = make_float2(-ref, -ref);
          sum = make_float2(0.0f, 0.0f);
          sum_p = sum;
          float2 sum1 = sum, sum_p1 = sum;
#pragma unroll
          for (int g = 0; g < 64; g += 32) {
            load(g);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              float2 y = fma2(x[c], mul_2, ref_2);
              y.x = ex2_approx(y.x);
              y.y = ex2_approx(y.y);
              if constexpr (kPart) {
                if (g + 2 * c >= cols) y.x = 0.0f;
                if (g + 2 * c + 1 >= cols) y.y = 0.0f;
              }
              if (c & 1)
                sum1 = add2(sum1, y);
              else
                sum = add2(sum, y);
              // the A operand is 16 bits, half a step of each weight: 2^-8 (bf16), 2^-11 (f16)
              const uint32_t both = kFp8 ? pack_f16(y.x, y.y) : pack_bf16(y.x, y.y);
              w[g / 2 + c] = both;
              if constexpr (!kFp8) {
                const float2 rounded = make_float2(__uint_as_float(both << 16), __uint_as_float(both & 0xFFFF0000u));
                if (c & 1)
                  sum_p1 = add2(sum_p1, rounded);
                else
                  sum_p = add2(sum_p, rounded);
              }
            }
          }
          sum = add2(sum, sum1);
          sum_p = add2(sum_p, sum_p1);
        };
        // the largest logit of this thread's first `end` keys (log2 units), or of more where these give none
        auto largest = [&](int end) -> float {
          float top = -INFINITY;
#pragma unroll 1
          for (int g = 0; g < 64; g += 32) {
            if (g >= end && !__any_sync(0xffffffffu, top == -INFINITY)) break;
            load(g);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              if (!kFp8 || g + 2 * c < cols) top = fmaxf(top, x[c].x * mul);
              if (!kFp8 || g + 2 * c + 1 < cols) top = fmaxf(top, x[c].y * mul);
            }
          }
          return top;
        };
        bool move = open, shifted = false;
#pragma unroll 1
        for (int tries = 0; tries < 2; ++tries) {
          if (move) {
            if (kFp8 && (shifted = barrier_rows_or(quad, may))) break;
            // Half the keys are enough for a first reference, the sum tells if not (32 sequences behind 128 pages 26.0 ->
            // 25.6 us; on an E4M3 cache 50.4 and 50.6, so not there).
            const float big = largest(!kFp8 && tries == 0 ? 32 : 64) - moved_to<kFp8>();
            red[half * 128 + row] = big;
            barrier_rows(quad);
            const float m_new = fmaxf(m, fmaxf(big, red[(half ^ 1) * 128 + row]));
            const float alpha = fresh || m == m_new ? 1.0f : ex2_approx(m - m_new);
            m = m_new;
            open = __any_sync(0xffffffffu, m == -INFINITY);  // the same in both warps of the rows
            l *= alpha;
            l_p *= alpha;
            if (!fresh && __any_sync(0xffffffffu, alpha != 1.0f)) {
              // O holds the units before this one; each of the two warps scales half of its columns
              wait_pv();
              tc_fence_after();
#pragma unroll 1
              for (int c = 128 * half; c < 128 * half + 128; c += 32) {
                float o[32];
                tmem_ld32(tmem + lanes + kTmemO + c, o);
                tc_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] *= alpha;
                tmem_st32(tmem + lanes + kTmemO + c, o);
              }
              tc_wait_st();  // the second try may read O again
            }
          }
          if (!kFp8 || cols >= 64)
            weights(std::false_type{});
          else
            weights(std::true_type{});
          move = barrier_rows_or(quad, sum.x + sum.y > kMostSum || may);
          if (!move) break;
        }
        if (kFp8 && shifted) {  // nothing has been done yet
          if (!fresh) wait_pv();
          tc_fence_after();
          const float2 ml = shifted_unit<E4m3Range>(tx, tmem + lanes + kTmemO, sc + 64 * half, cols, mul, m, l, fresh, red, row, half);
          m = ml.x;
          l = ml.y;
          open = __any_sync(0xffffffffu, m == -INFINITY);
        } else {
          l += sum.x + sum.y;
          l_p += sum_p.x + sum_p.y;
          tmem_st16(tx, reinterpret_cast<const float*>(w));
          tmem_st16(tx + 32, reinterpret_cast<const float*>(w + 16));
          tc_wait_st();
        }
        fresh = false;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_pair(p_full + 8 * buf);
        if (kFp8) mbar_arrive(cx.bar(ScEmpty + sc_slot));
      }
    }
    // ---- the piece's partial result: O / l and its LSE, 128 dims a thread
    wait_pv();
    tc_fence_after();
    if (!fresh) {
      red[half * 128 + row] = l;
      if (!kFp8) red[256 + half * 128 + row] = l_p;
      barrier_rows(quad);
      l += red[(half ^ 1) * 128 + row];
      if (!kFp8) l_p += red[256 + (half ^ 1) * 128 + row];
      const size_t at = ((size_t)(pair + q.t) * kSeqs + j) * kHeads + (row & 63);
      const float inv = kFp8 ? exp2_int(-E4m3Range::kUp) / l : 1.0f / l_p;
      float* dst = p.part_o + (at - (lane & 3)) * kHeadDim + 8 * (lane & 3);
#pragma unroll 1
      for (int c = 128 * half; c < 128 * half + 128; c += 32) {
        float o[32];
        tmem_ld32(tmem + lanes + kTmemO + c, o);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] *= inv;
        transpose_quad(o, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) st_global_v8(dst + k * kHeadDim + c, o + 8 * k);
      }
      if (half == 0) p.part_lse[at] = (m + log2f(l)) * kLn2;
      barrier_rows(quad);  // red is free again
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_pair(o_free);
  }
}

template <bool kFp8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads<kFp8>(), 1)
    decode_prefix_tc_kernel(const __grid_constant__ PrefixParams p, const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
  using Sm = Smem<kFp8>;
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  const uint32_t raw = smem_u32(dyn_smem);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = dyn_smem + (base - raw);
  PlanSmem& plan = *reinterpret_cast<PlanSmem*>(gbase + Sm::plan);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Sm::misc);
  int* abort_flag = reinterpret_cast<int*>(gbase + Sm::misc + 4);
  const int warp = threadIdx.x >> 5;
  Ctx cx{base, base + Sm::bars, cta_rank(), abort_flag, p.err, p.wait_budget_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) {
      const bool of_pair = i == PFull || i == PFull + 1 || i == OFree || i == QReady;  // every softmax warp of both CTAs
      const bool of_cta = i >= ScEmpty && i < ScEmpty + kScaleSlots;                   // of this one
      const bool of_converts = kFp8 && (i == VFull || i == VFull + 1);
      mbar_init(cx.bar(i), of_pair                             ? 2 * kSoftmaxWarps
                           : of_cta                            ? kSoftmaxWarps + kConvertWarps
                           : of_converts                       ? 2 * kConvertWarps
                           : i >= RawEmpty                     ? kConvertWarps
                           : i >= TailReady && i < RawFull     ? 2
                                                               : 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kProducerWarp && (threadIdx.x & 31) == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    prefetch_tensormap(&qmap);
  }
  __syncwarp();
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + Sm::misc),
                 "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncwarp();
  cluster_arrive();  // this CTA's barriers are initialised, its tensor memory is its own
  // hints only, these may still be written: what the plan, the first loads and Q need, in L2
  {
    auto hint = [](const void* at) { asm volatile("prefetch.global.L2 [%0];" ::"l"(at)); };
    const int i = threadIdx.x * 8;  // of 4-byte elements: a sector a thread
    if (blockIdx.x == 0 && i < p.B) hint(p.seq_lens + i);
    if (blockIdx.x == 0 && i < p.n_groups) hint(p.prefix_pages + i);
    if (blockIdx.x == 0 && i <= p.n_groups) hint(p.group_starts + i);
  }
  if (threadIdx.x == 0) {
    prefetch_l2_share(p.page_table, (size_t)p.B * p.max_pages * sizeof(int32_t), blockIdx.x, gridDim.x);
    prefetch_l2_share(p.q, (size_t)p.B * kHeads * kHeadDim * sizeof(uint16_t), blockIdx.x, gridDim.x);
  }
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  build_plan(p, plan, *reinterpret_cast<PlanScratch*>(gbase + Sm::k), blockIdx.x == 0 ? p.err : nullptr);
  cluster_wait();  // as are the other's; what it does to its own shared memory until its loads begin concerns no one else
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int units = plan.cost[plan.tiles], W = busy_pairs(p, units), pair = blockIdx.x >> 1;
  const int lo = pair < W ? range_of_pair(pair, units, W) : 0, hi = pair < W ? range_of_pair(pair + 1, units, W) : 0;

  if (warp < kSoftmaxWarps) {
    softmax_role<kFp8>(p, cx, plan, pair, lo, hi, tmem, gbase);
  } else if (warp == kProducerWarp) {
    producer_role<kFp8>(p, &kmap, &vmap, &qmap, cx, plan, pair, lo, hi);
  } else if (warp >= kTailWarp) {
    if constexpr (kFp8)
      convert_role(p, cx, plan, pair, lo, hi, gbase);
    else
      tail_role(p, cx, plan, pair, lo, hi);
  } else if (cx.rank == 1) {  // (its MMAs are issued by the leader)
    publish_plan(p, plan, pair, threadIdx.x & 31);
  } else if (elect_one()) {
    mma_role<kFp8>(p, cx, plan, pair, lo, hi, tmem);
  }
  __syncwarp();
  if (*cx.abort) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kSettleNs) {}
  }
  __syncwarp();
  tc_fence_before();
  cluster_arrive();
  cluster_wait();  // no copy, MMA or arrival for either CTA is left
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
}

template <bool kFp8>
cudaError_t launch_prefix(const PrefixParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                          const CUtensorMap& qmap, cudaStream_t stream) {
  const size_t smem = Smem<kFp8>::total + 1024;
  static int configured[kTrackedDevices] = {};
  const cudaError_t e = ensure_dynamic_smem(decode_prefix_tc_kernel<kFp8>, smem, configured);
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_prefix_tc_kernel<kFp8>, dim3(2 * p.pairs), dim3(threads<kFp8>()), smem, stream, p, kmap, vmap, qmap);
}
}  // namespace

cudaError_t launch_decode_prefix_tc(const PrefixParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                    const CUtensorMap& qmap, cudaStream_t stream) {
  return p.k_scale ? launch_prefix<true>(p, kmap, vmap, qmap, stream) : launch_prefix<false>(p, kmap, vmap, qmap, stream);
}

}  // namespace mfa
