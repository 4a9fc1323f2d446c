// chunk_attention_tc.cu -- attention of the new tokens of every sequence (a chunk
// of a prompt, a whole prompt, or one token) over all that its pages hold, causal
// among the new ones. With L_b positions in the cache, of which the last n_b are
// new, token t of them sees the first L_b - n_b + 1 + t:
//     S = Q K^T,  P = exp2(scale log2(e) S - m),  O = P V,  l = P 1
// for its 64 heads, which share K and V.
//
// Row tile: up to four neighbouring tokens of a sequence, 256 rows, and as its
// keys the pages up to what its last token sees. 4 * 64 * 256 flops a token and
// key against 1 KB (bf16) a key for the four tokens: matrix work, bound by the
// tensor cores, except for tiles of one token, whose pages HBM delivers more
// slowly than the pair of SMs that shares a tile works them off.
//
// A cluster of two CTAs, each with 128 of the rows, works on units of 128 keys
// (two pages) with tcgen05 MMAs of cta_group::2: each CTA holds one of the two K
// pages and half of V's dimensions, and both halves feed the pair's MMAs. TMEM
// holds S twice (2 x 128 columns; P overwrites S in place and is the A operand of
// P V from there) and O (256 columns): all of it. This is the tile of the
// shared-prefix kernel, whose parts it uses; what differs is where tiles come
// from, their masks, and that a prompt makes thousands of short tiles, so that
// what happens between two of them counts:
//   - S of a tile's first unit is issued before P V of the last tile's last one
//     where Q is there by then: its four blocks of 64 dimensions are loaded as the
//     last S of the tile before has read each of them;
//   - O of a tile is read into registers as bf16, and free for the next tile,
//     before any of it is written; on a bf16 cache by the softmax warps behind the
//     first unit of the next tile (by four warps of their own, which leave the
//     others 128 registers, 16 prompts of 512 tokens took 188 us instead of 163),
//     on a quantised one by the warps that convert V (by the softmax warps, which
//     split Q at that time, 307 us instead of 223).
//
// Work split: the units of all tiles, one after the other, form a line (a few
// more for each tile); each pair takes an equal range of it. A tile that lies
// whole in a range is written out; of the others, one at each end of a range at
// most, normalised partial results go to the workspace and the combine joins
// them. Units of the first i tiles of a sequence have a closed form, so that
// nothing is kept for a tile.
//
// Masks: a row's keys end where its token does, within the last 128 + 3 keys of
// its tile. Logits behind it become weights of zero; V's rows behind the tile's
// last token are zeroed, and of those that only some of its tokens see, up to
// three, values that are no numbers become zeros, which the rows that see them get
// added at the end: 0 * NaN of a later token never reaches an earlier one.
//
// Warp roles:
//   warps 0-7  softmax (and output): thread = row = TMEM lane; warp w and w + 4
//              share 32 rows, 64 keys of a unit each.
//   warp 8     producer (TMA, each CTA its own halves, completing on the leader's
//              barriers).
//   warp 9     TMEM allocation, and MMA issue (one thread of the leader's; the
//              first pair's other one leaves the combine where the parts are).
//   warp 10    V's rows behind the tile's last token and those that not all see.
//   warps 10-13 (E4M3 and E2M1 caches, instead) V codes to f16, with the same, and
//              the output.
// Every wait is bounded (the wait budget), as in the split kernel.
//
// E4M3 and E2M1 caches: S is 8-bit MMAs (kind::f8f6f4) on the raw K codes, with Q
// as two E4M3 terms under a power of two per row, split in shared memory when a
// tile begins; V's codes times their scales become f16, and P is f16 as well (the
// shared-prefix kernel says why).
//
// Measured, combine included: 2048 tokens behind 63488 in 4.65 to 4.7 ms called back to back (1840 to 1860 TFLOP/s; cuBLAS reaches 1896 in a
// burst, 1707 for seconds), the tensor cores 98% busy; 304 behind 16080 in 165 us, E4M3 174, E2M1 168 (replayed from graphs, as
// the following). A unit takes the 2050 cycles of its MMAs; what is lost between two tiles is 0.4 us for long tiles, and 2.6 us for
// the tiles of 2.5 units that 512-token prompts have (16 of them 161 us: a chain of Q and K from L2, 2 us each under load, the
// softmax of two units and the output), on quantised caches 3 us (Q waits for the last S, and its split takes 1.6; 220 and 223
// us). 23 tokens behind 900 take 15 us: plan 1.2, first tile, page ids and loads 1.9, a unit 2.9, 128 KB of fp32 partial results
// a CTA 2.8, combine 2.5, two launches.
#include <cuda_fp4.h>
#include <algorithm>
#include <type_traits>

#include "chunk_plan.hpp"
#include "mfa_serving.hpp"
#include "tc_pair.cuh"

namespace mfa {
namespace {

constexpr int kSoftmaxWarps = 8, kProducerWarp = 8, kMmaWarp = 9, kValueWarp = 10, kValueWarps = 4;
template <int kFmt>
constexpr bool kQuant = kFmt != kKvBf16;
template <int kFmt>
__host__ __device__ constexpr int threads() { return 32 * (kValueWarp + (kQuant<kFmt> ? kValueWarps : 1)); }
// Warps that write the output: the softmax warps on a bf16 cache, on a quantised one the value warps.
template <int kFmt>
__host__ __device__ constexpr int output_warps() { return kQuant<kFmt> ? kValueWarps : kSoftmaxWarps; }
// Two K and two V slots, of even and odd units, one CTA's half of a unit each: K one page of 256 dims, V 128 dims of two
// pages. E2M1 codes lie in shared memory as the 4-bit operands do, 16 codes in 8 bytes and 8 unused ones behind them.
template <int kFmt>
__host__ __device__ constexpr uint32_t slot_bytes() { return kQuant<kFmt> ? 16384 : 32768; }
template <int kFmt>
__host__ __device__ constexpr uint32_t slot_tx() { return kFmt == kKvE2M1 ? 8192 : slot_bytes<kFmt>(); }  // as copied
template <int kFmt>
using Range = std::conditional_t<kFmt == kKvE2M1, E2m1Range, E4m3Range>;
constexpr uint32_t kVSlotBytes = 32768, kVPageBytes = 16384;  // V as the MMAs read it, 16 bits
constexpr int kScaleSlots = 4, kScaleBytes = 1024;  // quantised: 128 K scales and 128 V scales a unit
constexpr int kQBytes = 65536;                      // 128 rows x 256 dims, four 64-dim blocks of [128 rows x 128 B]
static_assert(kTokens * kHeads == 256, "rows of a tile");

// The rows' sums of a piece, for its output: a softmax warp is at most two pieces ahead of it (S of a third follows P V of the
// second, which waits for the first one's O to be read).
constexpr int kStats = 4;
struct RowStats {
  float l[2][128], m[128];  // [half of the keys][row]
};

enum Bar {
  KFull = 0,                 // [2] leader: both CTAs' halves landed
  VFull = KFull + 2,         // [2] leader; quantised: one arrival per converting warp of the pair
  QFull = VFull + 2,         // [4] bf16: leader, by 64-dim block; quantised: the first, of both, each its own rows
  QFree = QFull + 4,         // [4] bf16, both: the last S of a piece has read the block
  QReady = QFree + 4,        // quantised, leader: Q split into terms, one arrival per softmax warp of the pair
  SFull,                     // [2] both: S of even and odd units
  PFull = SFull + 2,         // [2] leader: one arrival per softmax warp of the pair
  PvDone = PFull + 2,        // [2] both: P V of even and odd units
  OFree = PvDone + 2,        // leader: O has been read, one arrival per output warp of the pair
  StFull,                    // [kStats] quantised, both: the rows' sums of a piece, one arrival per softmax warp of the CTA
  Drain = StFull + kStats,   // leader
  ScFull,                    // [kScaleSlots] quantised, both
  ScEmpty = ScFull + kScaleSlots,   // [kScaleSlots] one arrival per softmax and converting warp of the CTA
  TailFull = ScEmpty + kScaleSlots, // [2] both: this CTA's V of a tile's end landed (by V slot)
  TailReady = TailFull + 2,         // [2] leader: it has been seen to, one arrival a CTA
  RawFull = TailReady + 2,          // [2] quantised, both: this CTA's V codes landed
  RawEmpty = RawFull + 2,           // [2] one arrival per converting warp of the CTA
  kBars = RawEmpty + 2
};

template <int kFmt>
struct Smem {
  static constexpr uint32_t k = 0;
  static constexpr uint32_t v = k + 2 * slot_bytes<kFmt>();
  static constexpr uint32_t raw = v + 2 * kVSlotBytes;  // quantised: V codes
  static constexpr uint32_t q = raw + (kQuant<kFmt> ? 2 * slot_bytes<kFmt>() : 0);
  static constexpr uint32_t scales = q + kQBytes;
  static constexpr uint32_t plan = scales + (kQuant<kFmt> ? kScaleSlots * kScaleBytes : 0);
  static constexpr uint32_t red = (plan + (uint32_t)sizeof(PlanSmem) + 15) & ~15u;  // [8][128] exchange of the row halves
  static constexpr uint32_t stats = red + 8 * 128 * 4;
  static constexpr uint32_t bars = stats + (kQuant<kFmt> ? kStats * sizeof(RowStats) : 0);
  static constexpr uint32_t odd = bars + 8 * kBars;  // [4] pieces with values that are no numbers (set_odd)
  static constexpr uint32_t misc = odd + 16;         // TMEM base, abort flag
  static constexpr uint32_t total = misc + 8;
};
static_assert(Smem<kKvBf16>::total + 1024 <= 227 * 1024 && Smem<kKvE4M3>::total + 1024 <= 227 * 1024, "shared memory");

struct Ctx {
  uint32_t base, bar0, odd, rank;
  volatile int* abort;
  uint32_t* err;
  uint64_t budget;
  __device__ uint32_t bar(int i) const { return bar0 + 8u * (uint32_t)i; }
  __device__ uint32_t leader_bar(int i) const { return map_to_leader(bar(i)); }
  __device__ bool wait(int i, uint32_t parity) const { return mbar_wait(bar(i), parity, budget, abort, err); }
  // the same for a whole warp, whose lanes give up together
  __device__ bool wait_warp(int i, uint32_t parity) const { return __all_sync(0xffffffffu, wait(i, parity)); }
};

// Rows of a tile's end held values that are no numbers: told to both CTAs' softmax warps, by piece. They look behind the
// piece's last P V, which waits for the arrival behind this; a fourth piece is not begun before they have. Rare.
__device__ __noinline__ void set_odd(uint32_t odd, uint32_t piece) {
#pragma unroll 1
  for (uint32_t r = 0; r < 2; ++r) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(odd + 4 * (piece & 3)), "r"(r));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(piece + 1) : "memory");
  }
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

// ---------------------------------------------------------------- plan
__device__ __forceinline__ int running_max(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = max(x, y);
  }
  return x;
}

// All threads; ends with a barrier.
__device__ void build_plan(const ChunkParams& p, PlanSmem& s, uint32_t* err) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kThreads = blockDim.x, warps = blockDim.x >> 5;
  if (p.B < 32) {  // one warp, without a barrier between the steps
    if (warp == 0) {
      const int raw = lane <= p.B ? __ldcg(p.q_starts + lane) : 0, raw_len = lane < p.B ? __ldcg(p.seq_lens + lane) : 0;
      const int len = clamp_len(raw_len, p.max_pages * kPageSize, err);
      const int x = running_max(min(max(raw, 0), p.max_tokens), lane);
      if (lane <= p.B && x != raw) raise_error(err, MFA_DEVERR_CAPACITY);
      const int next = __shfl_down_sync(0xffffffffu, x, 1);
      const int u = lane < p.B ? sequence_cost(len, min(next - x, len), p.piece_units) : 0;
      const int before = warp_inclusive_sum(u, lane) - u;
      if (lane < p.B) s.len[lane] = len;
      if (lane <= p.B) {
        s.row[lane] = x;
        s.cost[lane] = before;
      }
    }
    __syncthreads();
    return;
  }
  const int starts = (p.B + 32) / 32, chunks = (p.B + 31) / 32;  // 32 at a time, a warp each
#pragma unroll 1
  for (int c = warp; c < starts; c += warps) {
    const int i = 32 * c + lane, raw = i <= p.B ? __ldcg(p.q_starts + i) : 0;
    const int x = running_max(min(max(raw, 0), p.max_tokens), lane);
    if (i <= p.B) {
      if (x != raw) raise_error(err, MFA_DEVERR_CAPACITY);
      s.row[i] = x;
    }
    if (lane == 31) s.last[c] = x;
  }
  // (from the other end of the block, so that neither waits for the other's loads)
  for (int b = kThreads - 1 - threadIdx.x; b < p.B; b += kThreads)
    s.len[b] = clamp_len(__ldcg(p.seq_lens + b), p.max_pages * kPageSize, err);
  __syncthreads();
  if (starts > 1) {
#pragma unroll 1
    for (int c = warp; c < starts; c += warps) {
      const int i = 32 * c + lane, before = __reduce_max_sync(0xffffffffu, lane < c ? s.last[lane] : 0);
      if (i <= p.B && s.row[i] < before) {
        raise_error(err, MFA_DEVERR_CAPACITY);
        s.row[i] = before;
      }
    }
    __syncthreads();
  }
#pragma unroll 1
  for (int c = warp; c < chunks; c += warps) {
    const int b = 32 * c + lane, u = b < p.B ? sequence_cost(s.len[b], seeing(s, b), p.piece_units) : 0;
    const int x = warp_inclusive_sum(u, lane);
    if (b < p.B) s.cost[b] = x - u;
    if (b == p.B - 1) s.cost[p.B] = x;
    if (lane == 31) s.total[c] = x;
  }
  __syncthreads();
  if (chunks > 1) {
#pragma unroll 1
    for (int c = warp; c < chunks; c += warps) {
      const int b = 32 * c + lane, before = __reduce_add_sync(0xffffffffu, lane < c ? s.total[lane] : 0);
      if (b < p.B) s.cost[b] += before;
      if (b == p.B - 1) s.cost[p.B] += before;
    }
    __syncthreads();
  }
}

// Groups of eight warps that the combine takes for a tile: of one and two parts a warp takes two rows, of up to four one, of more
// half a row.
__device__ __forceinline__ int combine_groups(int tokens, int parts) {
  return tokens * kHeads / 8 * 2 / (parts <= 2 ? 4 : parts <= 4 ? 2 : 1);
}

// Where the combine finds the partial results: for every pair in whose range a tile begins that ends behind it, in order, then
// entries without tokens, the first of them with the number of all groups. One warp of the first pair.
__device__ void publish_parts(const ChunkParams& p, const PlanSmem& s, int lane) {
  const int units = s.cost[p.B], W = busy_pairs(p, units);
  int found = 0, groups = 0;
  for (int w0 = 0; w0 < W; w0 += 32) {
    const int w = w0 + lane;
    int row = 0, tokens = 0, parts = 0;
    Piece q;
    if (w < W && units > 0 && (parts = parts_from(p, s, w, units, W, q)) > 0) {
      row = q.row;
      tokens = q.tokens;
    }
    const uint32_t some = __ballot_sync(0xffffffffu, tokens > 0);
    const int mine = tokens > 0 ? combine_groups(tokens, parts) : 0, upto = warp_inclusive_sum(mine, lane);
    if (tokens > 0)
      p.parts[found + __popc(some & ((1u << lane) - 1))] = make_int4(row, tokens | parts << 8, w, groups + upto - mine);
    found += __popc(some);
    groups += __shfl_sync(0xffffffffu, upto, 31);
  }
  for (int i = found + lane; i <= p.pairs; i += 32) p.parts[i] = make_int4(0, 0, 0, i == found ? groups : 0x7fffffff);
}

// The output of tokens that see no key. One warp of each pair.
__device__ void write_unseeing(const ChunkParams& p, const PlanSmem& s, int pair, int lane) {
  for (int b = pair; b < p.B; b += p.pairs) {
    const int none = s.row[b + 1] - s.row[b] - seeing(s, b);
    for (int t = 0; t < none; ++t) {
      const size_t row = (size_t)(s.row[b] + t) * kHeads;
      uint4* out = reinterpret_cast<uint4*>(p.out + row * kHeadDim);
      for (int i = lane; i < kHeads * kHeadDim / 8; i += 32) out[i] = make_uint4(0u, 0u, 0u, 0u);
      for (int i = lane; i < kHeads; i += 32) p.lse[row + i] = -INFINITY;
    }
  }
}

// ---------------------------------------------------------------- producer
// Page ids of a piece: a window of 64 held by the warp (32 ahead of need). Those that a piece begins with are asked for
// when the piece before it begins.
struct TilePages {
  int end, base, a, b;
  __device__ static int load(int k, int end, const ChunkParams& p, const Piece& q) {
    return k < end ? __ldcg(p.page_table + (size_t)q.b * p.max_pages + k) : 0;
  }
  __device__ static int end_of(const Piece& q) { return min(q.pages(), 2 * q.u1); }
  __device__ int checked(int id, const ChunkParams& p) const {
    if (id >= 0 && id < p.num_pages) return id;
    raise_error(p.err, MFA_DEVERR_PAGE);
    return 0;
  }
  __device__ void start(int x, int y, const ChunkParams& p, const Piece& q) {
    end = end_of(q);
    base = 2 * q.u0;
    a = checked(x, p);
    b = checked(y, p);
  }
  __device__ int get(int k, const ChunkParams& p, const Piece& q, int lane) {
    while (k >= base + 64) {
      base += 32;
      a = b;
      b = checked(load(base + 32 + lane, end, p, q), p);
    }
    const int i = k - base;
    return i < 32 ? __shfl_sync(0xffffffffu, a, i) : __shfl_sync(0xffffffffu, b, i - 32);
  }
};

template <int kFmt, bool kTurn>
__device__ void producer_role(const ChunkParams& p, const CUtensorMap* kmap, const CUtensorMap* vmap,
                              const CUtensorMap* qmap, const Ctx& cx, const PlanSmem& s, LineRange range) {
  using Sm = Smem<kFmt>;
  constexpr bool kQ8 = kQuant<kFmt>;
  constexpr uint32_t kSlot = slot_bytes<kFmt>(), kPage = kSlot / 2, kTx = slot_tx<kFmt>();
  const int lane = threadIdx.x & 31, r = (int)cx.rank;
  const uint64_t pol = policy_evict_normal();
  uint32_t pieces = 0, tails[2] = {0, 0};
  // K of unit `n` (and its scales): this CTA's page, page r of the two, on the leader's barrier, on which the leader
  // announces the bytes of both CTAs
  auto load_k = [&](uint32_t n, int pa, int pb) -> bool {
    const uint32_t slot = n & 1;
    if (n >= 2 && !cx.wait_warp(SFull + slot, ((n >> 1) & 1) ^ 1)) return false;
    const int page = r == 0 ? pa : pb;
    if (elect_one()) {
      const uint32_t dst = cx.base + Sm::k + slot * kSlot, bar = cx.leader_bar(KFull + slot);
      if (r == 0) mbar_arrive_expect_tx(cx.bar(KFull + slot), pb >= 0 ? 2 * kTx : kTx);
      if (page >= 0) tma_load_3d_pair(dst, kmap, 0, page * kPageSize, 0, bar, pol);
    }
    if constexpr (kQ8) {  // the scales of all the unit's keys, for this CTA's rows
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
  // V of unit `n`: this CTA's 128 dims of each page. That of a tile's end lands on this CTA's own barrier, for the warp
  // that sees to its rows; quantised: all of it does, for the warps that convert it.
  auto load_v = [&](uint32_t n, int pa, int pb, bool tail) -> bool {
    const uint32_t slot = n & 1, parity = ((n >> 1) & 1) ^ 1, bytes = pb >= 0 ? kTx : kTx / 2;
    uint32_t dst, bar;
    if constexpr (kQ8) {
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
    if (elect_one()) {
      constexpr int kBlocks = kQ8 ? 1 : 2;  // of 128 dims
      tma_load_3d_pair(dst, vmap, 0, pa * kPageSize, r * kBlocks, bar, pol);
      if (pb >= 0) tma_load_3d_pair(dst + kPage, vmap, 0, pb * kPageSize, r * kBlocks, bar, pol);
    }
    return true;
  };
  uint32_t cnt = 0;  // units whose K has been loaded
  // Q of a piece, the rows of this CTA's two tokens: by block, as the piece before is done with each (quantised: with all)
  auto load_q = [&](const Piece& q) -> bool {
    if (kQ8 && pieces > 0 && !cx.wait_warp(SFull + ((cnt - 1) & 1), ((cnt - 1) >> 1) & 1)) return false;
    if (kQ8 && lane == 0) mbar_arrive_expect_tx(cx.bar(QFull), kQBytes);
    // (rows past the tensor's end, in a missing token's place, come as zeros and from nowhere)
    const int y0 = (2 * r < q.tokens ? q.row + 2 * r : p.max_tokens) * kHeads;
    const int y1 = (2 * r + 1 < q.tokens ? q.row + 2 * r + 1 : p.max_tokens) * kHeads;
#pragma unroll 1
    for (int d = 0; d < 4; ++d) {
      if (!kQ8 && pieces > 0 && !cx.wait_warp(QFree + d, (pieces - 1) & 1)) return false;
      if (elect_one()) {
        if (!kQ8 && r == 0) mbar_arrive_expect_tx(cx.bar(QFull + d), 2 * kQBytes / 4);
        const uint32_t dst = cx.base + Sm::q + d * (kQBytes / 4), bar = kQ8 ? cx.bar(QFull) : cx.leader_bar(QFull + d);
        tma_load_3d_pair(dst, qmap, 0, y0, d, bar, pol);
        tma_load_3d_pair(dst + kQBytes / 8, qmap, 0, y1, d, bar, pol);
      }
    }
    ++pieces;
    return true;
  };
  int va = -1, vb = -1;  // the last unit: its V is still to be loaded (V trails K by a unit, as the MMAs use them)
  bool vtail = false, good = true;
  Piece q, next;
  bool more = next_piece<kTurn>(p, s, range, next);
  int na = 0, nb = 0;
  auto ask = [&]() {  // what the next piece begins with
    const int end = TilePages::end_of(next);
    na = TilePages::load(2 * next.u0 + lane, end, p, next);
    nb = TilePages::load(2 * next.u0 + 32 + lane, end, p, next);
  };
  if (more) {
    ask();
    if (kQ8) good = load_q(next);  // (first, as it is split; bf16: K first, 0.1 us of a short call)
  }
  while (good && more) {
    q = next;
    TilePages ids;
    ids.start(na, nb, p, q);
    more = next_piece<kTurn>(p, s, range, next);
    if (more) {
      ask();
      const int here = min(2, max(0, next.tokens - 2 * r));  // its Q, into L2
      if (here > 0 && lane == 0)
        prefetch_l2(p.q + (size_t)(next.row + 2 * r) * kHeads * kHeadDim, here * kHeads * kHeadDim * 2);
    }
    for (int u = q.u0; good && u < q.u1; ++u) {
      const int pa = ids.get(2 * u, p, q, lane);
      const int pb = 2 * u + 1 < q.pages() ? ids.get(2 * u + 1, p, q, lane) : -1;
      // quantised: V's codes of two units earlier are converted before the MMAs are done with K of that unit, bf16: it is the other
      // way round
      if (kQ8 && va >= 0) good = load_v(cnt - 1, va, vb, vtail);
      good = good && load_k(cnt, pa, pb);
      if (!kQ8 && good && va >= 0) good = load_v(cnt - 1, va, vb, vtail);
      if (good && u == q.u0 && (!kQ8 || cnt > 0)) good = load_q(q);
      ++cnt;
      va = pa;
      vb = pb;
      vtail = q.ends(u);
    }
  }
  if (good && va >= 0) good = load_v(cnt - 1, va, vb, vtail);
  // Every copy of both CTAs must land before either leaves: this CTA's barriers and the leader's tell, and the other CTA
  // stays until the cluster's last barrier.
  if (lane == 0) {
    for (uint32_t k = cnt > 2 ? cnt - 2 : 0; k < cnt; ++k) {
      if (r == 0) (void)mbar_wait(cx.bar(KFull + (k & 1)), (k >> 1) & 1, kDrainNs, nullptr, p.err);
      if ((kQ8 || r == 0) && (good || k + 1 < cnt))
        (void)mbar_wait(cx.bar((kQ8 ? RawFull : VFull) + (k & 1)), (k >> 1) & 1, kDrainNs, nullptr, p.err);
    }
    for (int i = 0; i < 2; ++i)
      if (tails[i]) (void)mbar_wait(cx.bar(TailFull + i), (tails[i] - 1) & 1, kDrainNs, nullptr, p.err);
    if constexpr (kQ8)
      for (uint32_t k = cnt > (uint32_t)kScaleSlots ? cnt - kScaleSlots : 0; k < cnt; ++k)
        (void)mbar_wait(cx.bar(ScFull + k % kScaleSlots), (k / kScaleSlots) & 1, kDrainNs, nullptr, p.err);
    if (pieces && (kQ8 || r == 0))
      for (int d = 0; d < (kQ8 ? 1 : 4); ++d) (void)mbar_wait(cx.bar(QFull + d), (pieces - 1) & 1, kDrainNs, nullptr, p.err);
  }
  __syncwarp();
}

// ---------------------------------------------------------------- V at a tile's end
__device__ __forceinline__ bool not_number_bf16(uint32_t two) {
  return (two & 0x7F80u) == 0x7F80u || (two & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ bool not_number_f16(uint32_t two) {
  return (two & 0x7C00u) == 0x7C00u || (two & 0x7C000000u) == 0x7C000000u;
}
// bf16 words without the halves that are no numbers.
__device__ __forceinline__ uint32_t numbers_bf16(uint32_t two) {
  return ((two & 0x7F80u) == 0x7F80u ? 0u : two & 0xFFFFu) | ((two & 0x7F800000u) == 0x7F800000u ? 0u : two & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t numbers_f16(uint32_t two) {
  return ((two & 0x7C00u) == 0x7C00u ? 0u : two & 0xFFFFu) | ((two & 0x7C000000u) == 0x7C000000u ? 0u : two & 0xFFFF0000u);
}

// bf16: V of a unit at a tile's end, once it has landed: of rows that not all tokens see values that are no numbers become
// zeros, and rows behind the last one up to the end of an MMA's 16 keys do. One warp; true if there was such a value.
__device__ bool clear_tail(uint32_t unit, const Piece& q, int u, int lane) {
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int first = (2 * u + i) * kPageSize, keys = q.keys(2 * u + i);
    const uint32_t page = unit + i * kVPageBytes;
    // two rows at a time, 16 bytes of two 64-dim chunks a lane
    for (int row = max(0, q.seen0 - first) + (lane >> 4); row < keys; row += 2) {
      const uint32_t at = page + ((lane >> 3) & 1) * 8192 + row * 128 + (lane & 7) * 16;
      const uint4 v = ld_shared_v4(at);
      if (not_number_bf16(v.x) || not_number_bf16(v.y) || not_number_bf16(v.z) || not_number_bf16(v.w)) {
        const uint32_t w[4] = {numbers_bf16(v.x), numbers_bf16(v.y), numbers_bf16(v.z), numbers_bf16(v.w)};
        st_shared_v4(at, w);
        odd = true;
      }
    }
    if (is_partial(keys)) {
      const int words = (kKeyStep - keys % kKeyStep) * 8;  // 16 B words of a 64-dim chunk's rows
      for (int w = lane; w < words * 2; w += 32)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(page + keys * 128 + (w / words) * 8192 + (w % words) * 16), "r"(0)
                     : "memory");
    }
  }
  return odd;
}

// Of what a converting thread has stored (at0, at1: its words of row row0 of the unit), rows from `from` on, which not all
// tokens see, without what is no number; true if there was any. Out of line: in the loop of all units it cost a fifth of their
// time.
__device__ __noinline__ bool clear_odd_f16(uint32_t at0, uint32_t at1, int row0, int from) {
  bool odd = false;
#pragma unroll 1
  for (int i = 0; i < 8; ++i) {  // rows 16 apart, of two pages
    if ((i >> 2) * kPageSize + row0 + 16 * (i & 3) < from) continue;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t at = (k ? at1 : at0) + (i >> 2) * kVPageBytes + (i & 3) * 2048;
      const uint4 v = ld_shared_v4(at);
      if (not_number_f16(v.x) || not_number_f16(v.y) || not_number_f16(v.z) || not_number_f16(v.w)) {
        const uint32_t w[4] = {numbers_f16(v.x), numbers_f16(v.y), numbers_f16(v.z), numbers_f16(v.w)};
        st_shared_v4(at, w);
        odd = true;
      }
    }
  }
  return odd;
}

// Quantised: V of a unit as P V reads it, f16 of code * scale * 2^kUp without the scale's shift, from the codes: per page
// [64 rows x 128 dims] to two 64-dim chunks of [64 rows x 128 B], both with the 128-byte swizzle. A thread takes 16 codes of
// a row and of every 16th row after it; rows behind the tile's last token become zeros. Which rows eight neighbouring threads
// take keeps reads and writes on banks of their own, as in the shared-prefix kernel.
struct Converter {
  int row0;
  uint32_t from, to0, to1;
  __device__ explicit Converter(int t) {
    row0 = (2 * (t >> 4)) ^ (t & 4 ? 5 : 0);
    const int c = (t & 3) | ((t >> 1) & 4);  // 16-code chunk: dims [16 c, 16 c + 16)
    from = row0 * 128 + ((c ^ (row0 & 7)) << 4);  // rows 16 apart share the swizzle
    const uint32_t to = (c >> 2) * 8192 + row0 * 128;
    to0 = to + (((2 * (c & 3)) ^ (row0 & 7)) << 4);
    to1 = to + (((2 * (c & 3) + 1) ^ (row0 & 7)) << 4);
  }
};
template <int kFmt>
__device__ __forceinline__ void convert_unit(const Converter& at, uint32_t src, uint32_t dst, const float* sc, const Piece& q, int u) {
  const int row0 = at.row0;
  src += at.from;
#pragma unroll
  for (int page = 0; page < 2; ++page) {
    const int valid = q.keys(2 * u + page);
    uint4 v[4];
    __half2 scale[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = ld_shared_v4(src + page * 8192 + i * 2048);
      const float s = sc[page * kPageSize + row0 + 16 * i];
      scale[i] = __float2half2_rn(s * exp2_int(Range<kFmt>::kUp - scale_shift<Range<kFmt>>(s)));
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
        __half2_raw r;
        if constexpr (kFmt == kKvE2M1)
          r = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(w[k >> 2] >> (8 * (k & 3))), __NV_E2M1);
        else
          r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[k >> 1] >> (16 * (k & 1))), __NV_E4M3);
        const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&r), scale[i]);
        h[k >> 2][k & 3] = *reinterpret_cast<const uint32_t*>(&y);
      }
      st_shared_v4(dst + page * kVPageBytes + i * 2048 + at.to0, h[0]);
      st_shared_v4(dst + page * kVPageBytes + i * 2048 + at.to1, h[1]);
    }
  }
}

// ---------------------------------------------------------------- MMA issue (one thread of the leader)
template <int kFmt, bool kTurn>
__device__ void mma_role(const ChunkParams& p, const Ctx& cx, const PlanSmem& s, LineRange range, uint32_t tmem) {
  constexpr bool kQ8 = kQuant<kFmt>;
  // A = Q, B = K, both K-major (8-bit kinds: formats 0, E4M3, and 5, E2M1); A = P (TMEM), B = V (dim-major; format 0: f16)
  constexpr uint32_t idesc_s = idesc_f16(256, kSCols, kQ8 ? 0 : 1, 0, 0) | (kFmt == kKvE2M1 ? 5u << 10 : 0u);
  constexpr uint32_t idesc_o = idesc_f16(256, kHeadDim, kQ8 ? 0 : 1, 0, 1);
  using Sm = Smem<kFmt>;
  uint32_t pieces = 0, s_cnt = 0, p_cnt = 0, tails[2] = {0, 0};
  // Descriptors of the operands' first blocks; a block `bytes` further on has bytes / 16 more in the address field, which
  // holds every shared address without a carry.
  auto ahead = [](uint64_t desc, uint32_t bytes) -> uint64_t { return desc + (bytes >> 4); };
  const uint64_t q_desc = smem_desc_sw128(cx.base + Sm::q, 16, 1024);
  const uint64_t k_desc0 = smem_desc_sw128(cx.base + Sm::k, 16, 1024);
  const uint64_t v_desc0 = smem_desc_sw128(cx.base + Sm::v, 8192, 1024);
  // What this thread does between two batches of MMAs costs nothing as long as it is short: barriers are looked at in the
  // middle of a batch, for the next one, and waited for only if that found them not yet done.
  bool k_ready = false, pv_ready = false;
  auto peek = [&](int i, uint32_t parity) -> bool { return mbar_test_wait(cx.bar(i), parity); };
  auto peek_pv = [&]() -> bool { return peek(VFull + (p_cnt & 1), (p_cnt >> 1) & 1) && peek(PFull + (p_cnt & 1), (p_cnt >> 1) & 1); };
  // S of unit s_cnt; p_next: a P V is to follow; first, last: of its piece
  auto do_s = [&](bool p_next, bool first, bool last) -> bool {
    const uint32_t buf = s_cnt & 1, d = tmem + buf * kSCols;  // its last reader, P V of two units ago, was issued before
    if (!k_ready && !cx.wait(KFull + buf, (s_cnt >> 1) & 1)) return false;
    k_ready = false;
    tc_fence_after();
    const uint64_t k_desc = ahead(k_desc0, buf * slot_bytes<kFmt>());
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!kQ8 && first && !cx.wait(QFull + e, pieces & 1)) return false;
      if (e == 2) pv_ready = p_next && peek_pv();
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if constexpr (kQ8)  // Q's term e / 2, 128-dim half e % 2, 32 dims
          tc_mma_pair_f8(d, ahead(q_desc, (e & 1) * 32768 + (e >> 1) * 16384 + kk * 32), ahead(k_desc, (e & 1) * 8192 + kk * 32), idesc_s,
                         (e | kk) != 0);
        else  // 64-dim block, 16 dims
          tc_mma_pair(d, ahead(q_desc, e * 16384 + kk * 32), ahead(k_desc, e * 8192 + kk * 32), idesc_s, (e | kk) != 0);
      }
      if (!kQ8 && last) tc_commit_pair(cx.bar(QFree + e));
    }
    tc_commit_pair(cx.bar(SFull + buf));
    ++s_cnt;
    return true;
  };
  struct Unit {  // whose P V is still to be issued
    int keys[2];
    bool pending, first, ends;
    uint32_t piece;
  };
  auto do_pv = [&](const Unit& v) -> bool {
    constexpr int kSteps = kPageSize / kKeyStep;
    const uint32_t buf = p_cnt & 1, a = tmem + buf * kSCols, d = tmem + kTmemO;
    if (v.first && !cx.wait(OFree, (v.piece & 1) ^ 1)) return false;
    if (!kQ8 && v.ends && !cx.wait(TailReady + buf, tails[buf]++ & 1)) return false;
    if (!pv_ready && !(cx.wait(VFull + buf, (p_cnt >> 1) & 1) && cx.wait(PFull + buf, (p_cnt >> 1) & 1))) return false;
    pv_ready = false;
    tc_fence_after();
    const uint64_t v_desc = ahead(v_desc0, buf * kVSlotBytes);
    auto a_of = [&](int i, int kk) { return a + i * 64 + (kk >> 1) * 32 + (kk & 1) * 8; };  // page i, step kk
    if (v.keys[1] == kPageSize) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk)
          tc_mma_pair_tmem_a(d, a_of(i, kk), ahead(v_desc, i * kVPageBytes + kk * 2048), idesc_o, (i | kk) != 0 || !v.first);
        if (i == 0) k_ready = peek(KFull + (s_cnt & 1), (s_cnt >> 1) & 1);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        const int steps = ((i ? v.keys[1] : v.keys[0]) + kKeyStep - 1) / kKeyStep;
#pragma unroll 1
        for (int kk = 0; kk < steps; ++kk)
          tc_mma_pair_tmem_a(d, a_of(i, kk), ahead(v_desc, i * kVPageBytes + kk * 2048), idesc_o, (i | kk) != 0 || !v.first);
      }
      k_ready = false;
    }
    tc_commit_pair(cx.bar(PvDone + buf));
    ++p_cnt;
    return true;
  };
  // Between two pieces: true if the next S can be issued, false if the last P V can and the next S not yet (`good` false:
  // neither in time).
  auto s_goes_first = [&](bool& good) -> bool {
    const uint64_t t0 = globaltimer_ns();
    for (bool again = false;; again = true) {
      if (peek(QFull, pieces & 1) && peek(KFull + (s_cnt & 1), (s_cnt >> 1) & 1)) return true;
      if (peek_pv()) return false;
      if (*cx.abort) break;
      if (again && globaltimer_ns() - t0 >= cx.budget) {
        raise_error(cx.err, MFA_DEVERR_TIMEOUT);
        *cx.abort = 1;
        break;
      }
    }
    good = false;
    return true;
  };
  Piece q;
  Unit pend{};
  bool good = true;
  while (good && next_piece<kTurn>(p, s, range, q)) {
    for (int u = q.u0; good && u < q.u1; ++u) {
      if (u == q.u0) {
        // quantised: Q is split behind the last softmax, which takes longer than the last P V
        if (pend.pending && (kQ8 || !s_goes_first(good)) && good) {
          good = do_pv(pend);
          pend.pending = false;
        }
        if (kQ8 && good) good = cx.wait(QReady, pieces & 1);
        if (!good) break;
      }
      good = do_s(pend.pending, u == q.u0, u + 1 == q.u1);
      if (good && pend.pending) good = do_pv(pend);
      pend.pending = true;
      pend.first = u == q.u0;
      pend.ends = q.ends(u);
      pend.piece = pieces;
      pend.keys[0] = q.keys(2 * u);
      pend.keys[1] = q.keys(2 * u + 1);
    }
    ++pieces;
  }
  if (good && pend.pending) (void)do_pv(pend);
  tc_commit_pair(cx.bar(Drain));  // every MMA is done before TMEM is given back
  (void)mbar_wait(cx.bar(Drain), 0, kDrainNs, nullptr, p.err);
}

// ---------------------------------------------------------------- references
// A row's reference is set so that its largest weight then is 2^set_at. It moves when the sum of a thread's weights passes
// 2^most_sum_log2: of the 64 of a unit on a quantised cache, of all so far on a bf16 cache. And in units that the careful way
// below takes for another reason, when a weight passes the 64th part. A move takes a unit 2000 cycles longer.
// P as f16 ends at 2^16, and below 2^-14 its step stays 2^-24: weights below 2^-18 of the row's largest are held to 2^-29 of it,
// as in the shared-prefix kernel, so that N of them that all round the same way are off by N 2^-29 together (262144: 2^-11). With
// references at the largest logit that would be N 2^-25, and below 2^-25 nothing would be left of them in O (304 tokens behind
// 16080 on E4M3 174 us instead of 174.5, with logits of twice and four times the spread 187 and 224 instead of 201 and 235).
// P as bf16 has the same relative step everywhere, so its weights are small enough that a row's never have a sum above 1: each of
// its two threads has 2^-3 behind a whole unit, 2^-2 behind the last one, and where it has more than 2^-4 when others move its
// reference does too. O is then never larger than the largest V, and no finite V gives an infinite output. (With references at the
// largest logit, moved by units of 2^30, values of 2^90 came out infinite behind 200 such units; the times are the same.) What it
// takes from fp32's lower end: values of V below 2^-110 lose bits. Set at 2^-30, below 2^-104; at 2^-18, with which rows move
// more often, below 2^-116, but two prompts of 4096 with logits of five times the spread took 680 us instead of 620.
template <bool kQ8>
__host__ __device__ constexpr int set_at() { return kQ8 ? (int)moved_to<true>() : -24; }
template <bool kQ8>
__host__ __device__ constexpr int most_sum_log2() { return kQ8 ? 15 : -3; }

// ---------------------------------------------------------------- V and output
// V of position k of the piece's sequence, as P V would read it if nothing had been cleared, where that is no number, else 0: on a
// quantised cache also where f16 does not hold the value for its scale (convert_unit). Out of line: inlined, it costs the units'
// loop of an E2M1 cache registers (16 prompts of 512 tokens 231 -> 234 us where the table is wide, 304 tokens behind 16080 169 -> 170.5).
template <int kFmt>
__device__ __noinline__ float not_number(const ChunkParams& p, int b, int k, int dim) {
  const int page = __ldcg(p.page_table + (size_t)b * p.max_pages + k / kPageSize);
  const size_t slot = (size_t)(page >= 0 && page < p.num_pages ? page : 0) * kPageSize + k % kPageSize;
  float v;
  if constexpr (kFmt == kKvBf16) {
    v = __uint_as_float((uint32_t)__ldcg(static_cast<const uint16_t*>(p.v_cache) + slot * kHeadDim + dim) << 16);
  } else {
    __half_raw h;
    if constexpr (kFmt == kKvE4M3) {
      h = __nv_cvt_fp8_to_halfraw(__ldcg(static_cast<const uint8_t*>(p.v_cache) + slot * kHeadDim + dim), __NV_E4M3);
    } else {
      const uint8_t two = __ldcg(static_cast<const uint8_t*>(p.v_cache) + (slot * kHeadDim + dim) / 2);
      h = __nv_cvt_fp4_to_halfraw((__nv_fp4_storage_t)(dim & 1 ? two >> 4 : two & 15), __NV_E2M1);
    }
    const float s = __ldcg(p.v_scale + slot);
    v = __half2float(__hmul(*reinterpret_cast<const __half*>(&h), __float2half_rn(s * exp2_int(Range<kFmt>::kUp - scale_shift<Range<kFmt>>(s)))));
  }
  return fabsf(v) <= 3.402823466e38f ? 0.0f : v;
}

// The output of a piece whose end held values that are no numbers: O / l and, in the rows that see them, these values added
// (a weight times one of them is one). Rare and out of line. part_row: of the partial results (null: the output itself).
template <int kFmt>
__device__ __noinline__ void write_odd(const ChunkParams& p, int b, int k0, int k1, uint32_t o_addr, float inv, size_t out_row,
                                       float* part_row, int d0, int dims, bool valid) {
#pragma unroll 1
  for (int c = d0; c < d0 + dims; c += 16) {
    float o[16];
    tmem_ld16(o_addr + c, o);
    tc_wait_ld();
#pragma unroll 1
    for (int k = k0; k < k1; ++k)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] += not_number<kFmt>(p, b, k, c + j);
    if (!valid) continue;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (part_row) part_row[c + j] = o[j] * inv;
      else p.out[out_row * kHeadDim + c + j] = (uint16_t)(pack_bf16(o[j] * inv, 0.0f) & 0xFFFFu);
    }
  }
}

// O of a piece over its rows' sums, and their LSE: to the output, or as a partial result. Thread = row, kDims dims from d0 on;
// l, l_p: the sum of the row's weights, and of those that entered O.
template <int kFmt, int kDims>
__device__ __forceinline__ void write_piece(const ChunkParams& p, const Ctx& cx, const Piece& q, float l, float l_p, float m, int pair,
                                            uint32_t o_addr, uint32_t o_free, int row, int d0, bool odd) {
  const int lane = threadIdx.x & 31, j = 2 * (int)cx.rank + (row >> 6);  // token of the tile
  const bool valid = j < q.tokens, whole = q.whole();
  // rows that see no key of the piece have O = 0 and no weight
  const float inv = q.seen0 + j <= q.u0 * kUnitKeys ? 0.0f : kQuant<kFmt> ? exp2_int(-Range<kFmt>::kUp) / l_p : 1.0f / l_p;
  const size_t out_row = (size_t)(q.row + j) * kHeads + (row & 63);
  const size_t part = (size_t)part_slot(pair, q.u0 == 0) * 256 + 128 * cx.rank + row;
  if (valid && d0 == 0) {
    constexpr int kSet = kQuant<kFmt> ? 0 : set_at<false>();  // taken off both first, so that neither is far from their sum
    const float lse = ((m + kSet) + log2f(l * exp2_int(-kSet))) * kLn2;
    if (whole) p.lse[out_row] = lse;
    else p.part_lse[part] = lse;
  }
  auto free_o = [&]() {  // for the next piece's first P V
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_pair(o_free);
  };
  if (odd) {
    // keys of this piece that not all of the tile's tokens see, up to this row's
    const int k0 = max(q.seen0, q.u0 * kUnitKeys), k1 = min(q.seen0 + j, q.u1 * kUnitKeys);
    write_odd<kFmt>(p, q.b, k0, valid ? k1 : k0, o_addr, inv, out_row, whole ? nullptr : p.part_o + part * kHeadDim, d0, kDims, valid);
  }
  if (odd || !valid) {
    free_o();
    return;
  }
  // Four neighbouring lanes exchange theirs, so that each writes a part of four rows and together whole lines of them.
  if (whole) {
    // As bf16 into registers as far as they go, so that O is free before much is written. Words of 64 dims in the order in which
    // the lanes' 16 bytes lie beside each other.
    constexpr int kHeld = kDims > 128 ? 64 : kDims;  // (128 of 256 spill)
    uint16_t* dst = p.out + (out_row - (lane & 3)) * kHeadDim + d0 + 8 * (lane & 3);
#pragma unroll 1
    for (int d = 0; d < kDims; d += kHeld) {
      float w[kHeld / 64][32];
#pragma unroll
      for (int c = 0; c < kHeld / 32; ++c) {
        float o[32];
        tmem_ld32(o_addr + d0 + d + 32 * c, o);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k)
          w[c >> 1][8 * (k >> 2) + 4 * (c & 1) + (k & 3)] = __uint_as_float(pack_bf16(o[2 * k] * inv, o[2 * k + 1] * inv));
      }
      if (d + kHeld == kDims) free_o();
#pragma unroll
      for (int c = 0; c < kHeld / 64; ++c) {
        transpose_quad(w[c], lane);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float4* to = reinterpret_cast<float4*>(dst + k * kHeadDim + d + 64 * c);
          to[0] = make_float4(w[c][8 * k], w[c][8 * k + 1], w[c][8 * k + 2], w[c][8 * k + 3]);
          to[4] = make_float4(w[c][8 * k + 4], w[c][8 * k + 5], w[c][8 * k + 6], w[c][8 * k + 7]);
        }
      }
    }
  } else {
    float* dst = p.part_o + (part - (lane & 3)) * kHeadDim + 8 * (lane & 3);
#pragma unroll 1
    for (int c = d0; c < d0 + kDims; c += 32) {
      float o[32];
      tmem_ld32(o_addr + c, o);
      tc_wait_ld();
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] *= inv;
      transpose_quad(o, lane);
#pragma unroll
      for (int k = 0; k < 4; ++k) st_global_v8(dst + k * kHeadDim + c, o + 8 * k);
    }
    free_o();
  }
}

// bf16: V at the end of every tile.
template <bool kTurn>
__device__ void tail_role(const ChunkParams& p, const Ctx& cx, const PlanSmem& s, LineRange range) {
  const int lane = threadIdx.x & 31;
  uint32_t n = 0, tails[2] = {0, 0}, piece = 0;
  Piece q;
  for (; next_piece<kTurn>(p, s, range, q); ++piece) {
    for (int u = q.u0; u < q.u1; ++u, ++n) {
      if (!q.ends(u)) continue;
      const uint32_t slot = n & 1;
      if (!cx.wait_warp(TailFull + slot, tails[slot] & 1)) return;
      ++tails[slot];
      if (clear_tail(cx.base + Smem<kKvBf16>::v + slot * kVSlotBytes, q, u, lane)) set_odd(cx.odd, piece);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(cx.leader_bar(TailReady + slot));
    }
  }
}

// Quantised: V of every unit as P V needs it and, behind that of the next piece's first unit, the output of a piece.
template <int kFmt, bool kTurn>
__device__ void value_role(const ChunkParams& p, const Ctx& cx, const PlanSmem& s, int pair, LineRange range, uint32_t tmem,
                           uint8_t* gbase) {
  using Sm = Smem<kFmt>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = 32 * (warp & 3) + lane;
  const uint32_t o_addr = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kTmemO, o_free = cx.leader_bar(OFree);
  const RowStats* stats = reinterpret_cast<const RowStats*>(gbase + Sm::stats);
  volatile const uint32_t* odd = reinterpret_cast<volatile const uint32_t*>(gbase + Sm::odd);
  const Converter at(threadIdx.x - 32 * kValueWarp);
  uint32_t n = 0, piece = 0;
  Piece q, last;
  for (bool more = true; more; ++piece) {
    more = next_piece<kTurn>(p, s, range, q);
    int u = q.u0;
    do {
      if (more) {
        const uint32_t slot = n & 1, sc_slot = n % kScaleSlots, dst = cx.base + Sm::v + slot * kVSlotBytes;
        const float* sc = reinterpret_cast<const float*>(gbase + Sm::scales + sc_slot * kScaleBytes) + kUnitKeys;
        if (!cx.wait_warp(ScFull + sc_slot, (n / kScaleSlots) & 1)) return;
        if (!cx.wait_warp(RawFull + slot, (n >> 1) & 1)) return;
        if (n >= 2 && !cx.wait_warp(PvDone + slot, ((n >> 1) & 1) ^ 1)) return;
        convert_unit<kFmt>(at, cx.base + Sm::raw + slot * slot_bytes<kFmt>(), dst, sc, q, u);
        if (q.ends(u) && clear_odd_f16(dst + at.to0, dst + at.to1, at.row0, q.seen0 - u * kUnitKeys)) set_odd(cx.odd, piece);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(cx.bar(RawEmpty + slot));
          mbar_arrive(cx.bar(ScEmpty + sc_slot));
          mbar_arrive_pair(cx.leader_bar(VFull + slot));
        }
        ++n;
      }
      if (piece > 0 && u == q.u0) {
        const uint32_t done = piece - 1, unit = n - (more ? 2 : 1);  // the piece before, its last unit
        // the sums tell that S of that unit is done, and so every P V of two units earlier: the parity is exact
        if (!cx.wait_warp(StFull + (done & (kStats - 1)), (done / kStats) & 1)) return;
        if (!cx.wait_warp(PvDone + (unit & 1), (unit >> 1) & 1)) return;
        tc_fence_after();
        const RowStats& st = stats[done & (kStats - 1)];
        const float l = st.l[0][row] + st.l[1][row];
        write_piece<kFmt, kHeadDim>(p, cx, last, l, l, st.m[row], pair, o_addr, o_free, row, 0, odd[done & 3] == done + 1);
      }
    } while (more && ++u < q.u1);
    last = q;
  }
}

// ---------------------------------------------------------------- softmax
// Quantised: the bf16 Q of this CTA's 128 rows (four 64-dim blocks of [128 rows x 128 B], 128-byte swizzle) becomes, in place,
// two E4M3 terms of Q * 2^e ([128-dim half][term][128 rows x 128 B]): the first rounds the scaled value, the second the rest,
// which is exact unless it falls below the E4M3 normal range (2^-18.8 of the row's largest |q|). 2^e is the largest power of
// two that keeps the row within the E4M3 maximum, 448 (2^126 at most). Thread (row, half) takes the 128 dims of its half, whose
// terms lie where they did. All softmax threads; red: their exchange. Returns 2^-e, NaN for a row with a value that is no number.
__device__ __forceinline__ float split_queries(uint32_t q_addr, float* red, int row, int quad, int half) {
  const uint32_t at = q_addr + half * 32768 + row * 128;  // the first of the two blocks; the second 16 KB on
  auto chunk = [&](int j) { return (j ^ (row & 7)) << 4; };
  uint4 v[8];
  uint32_t tops = 0;  // the largest magnitudes of even and odd dims, as bits: what is no number is larger than any
  auto largest = [&](const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) tops = __vmaxu2(tops, w[k] & 0x7FFF7FFFu);
  };
#pragma unroll
  for (int j = 0; j < 8; ++j) largest(ld_shared_v4(at + chunk(j)));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = ld_shared_v4(at + 16384 + chunk(j));
    largest(v[j]);
  }
  red[half * 128 + row] = __uint_as_float(max(tops << 16, tops & 0xFFFF0000u));
  barrier_rows(quad);
  const uint32_t top = max(__float_as_uint(red[row]), __float_as_uint(red[128 + row]));
  int e = 0;
  if (top != 0 && top < 0x7F800000u) e = ((top & 0x7FFFFFu) <= 0x600000u ? 8 : 7) - ((int)(top >> 23) - 127);  // in (224, 448]
  e = max(-120, min(126, e));
  const float up = exp2_int(e);
#pragma unroll
  for (int o = 0; o < 8; ++o) {  // 16 dims; those of the second block have been read
    const uint4 x = o < 4 ? ld_shared_v4(at + chunk(2 * o)) : v[2 * o - 8], y = o < 4 ? ld_shared_v4(at + chunk(2 * o + 1)) : v[2 * o - 7];
    uint32_t a1[2], a2[2], b1[2], b2[2];
    split_q8<true>(x, up, a1, a2);
    split_q8<true>(y, up, b1, b2);
    const uint32_t t1[4] = {a1[0], a1[1], b1[0], b1[1]}, t2[4] = {a2[0], a2[1], b2[0], b2[1]};
    st_shared_v4(at + chunk(o), t1);
    st_shared_v4(at + 16384 + chunk(o), t2);
  }
  fence_proxy_async_smem();
  return top < 0x7F800000u ? exp2_int(-e) : __uint_as_float(0x7FFFFFFFu);
}

// A row's state over the units of its keys: the reference (log2 units), and this thread's share of the denominator.
struct RowState {
  bool fresh = true;  // no key so far
  bool open = true;   // a row of the warp has no finite reference
  float m = -INFINITY, l = 0.0f;
  // The same of the weights as P holds them, by which O is divided: a weight that has most of the sum then cancels its
  // rounding (relative error of out 2.4e-3 -> 1.9e-3 for 128 sequences behind 512 pages, 1% slower). Of f16 weights the
  // difference does not matter. The LSE takes the unrounded sum.
  float l_p = 0.0f;
};

// The weights of one unit, S in tensor memory replaced by P. tx: this thread's 64 products, of which `cols` count (the two
// warps of the rows together at least one; `whole`: all 128); o_addr: O's first column in its lane; sc: the K scales of its
// keys, 128 before their V scales (quantised); may: some V scale among the warp's may have a shift; wait_pv: O holds every
// unit before this one. Both warps of the rows. A whole unit of rows that have a reference takes the first way, in which the
// products come 32 at a time and no maximum is looked for, unless its weights are too large; the other way holds all 64 in
// registers between the maximum and the weights, so that masks and references take no second trip to tensor memory.
template <bool kQ8, typename R, typename WaitPv>
__device__ __forceinline__ void softmax_tile_unit(RowState& st, uint32_t tx, uint32_t o_addr, const float* sc, int cols, bool whole,
                                                  bool may, float mul, float* red, bool& turn, int row, int quad, int half, WaitPv&& wait_pv) {
  // 32 products; P of 32 keys replaces the first 16 columns of their S
  auto load = [&](int g, float2 (&x)[16]) {
    tmem_ld32(tx + g, reinterpret_cast<float*>(x));
    if constexpr (kQ8) {  // times the scales of K, of which half arrive meanwhile
      const float4* k = reinterpret_cast<const float4*>(sc + g);
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
  float2 sum[2], sum_p[2];
  auto clear = [&]() { sum[0] = sum[1] = sum_p[0] = sum_p[1] = make_float2(0.0f, 0.0f); };
  // the weights of keys 2 c, 2 c + 1 into the sums, and as the A operand: 16 bits, half a step of each weight is 2^-8 (bf16)
  // or 2^-11 (f16)
  auto weigh = [&](float2 y, int c) -> uint32_t {
    y.x = ex2_approx(y.x);
    y.y = ex2_approx(y.y);
    sum[c & 1] = add2(sum[c & 1], y);
    const uint32_t both = kQ8 ? pack_f16(y.x, y.y) : pack_bf16(y.x, y.y);
    if constexpr (!kQ8)
      sum_p[c & 1] = add2(sum_p[c & 1], make_float2(__uint_as_float(both << 16), __uint_as_float(both & 0xFFFF0000u)));
    return both;
  };
  uint32_t w[32];
  bool done = false, over = false;
  if (whole && !st.open) {
    const float2 mul_2 = make_float2(mul, mul), ref_2 = make_float2(-st.m, -st.m);
    clear();
#pragma unroll
    for (int g = 0; g < 64; g += 32) {
      float2 x[16];
      load(g, x);
#pragma unroll
      for (int c = 0; c < 16; ++c) w[g / 2 + c] = weigh(fma2(x[c], mul_2, ref_2), c);
    }
    const float2 all = add2(sum[0], sum[1]);
    float total = all.x + all.y;
    if constexpr (!kQ8) total += st.l;
    done = !barrier_rows_or(quad, total > exp2_int(most_sum_log2<kQ8>()) || may);
    over = !done;
  }
  if (!done) {
    float2 y[32];
    load(0, *reinterpret_cast<float2 (*)[16]>(y));
    load(32, *reinterpret_cast<float2 (*)[16]>(y + 16));
    // all 64 count: the largest product, which times a positive factor stays the largest; else each by itself
    float top = -INFINITY, factor = 1.0f;
    if (cols == kPageSize && mul > 0.0f) {
#pragma unroll
      for (int c = 0; c < 32; ++c) top = fmaxf(top, fmaxf(y[c].x, y[c].y));
      top *= mul;
      factor = mul;
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        y[c] = mul2(y[c], make_float2(mul, mul));
        if (2 * c >= cols) y[c].x = -INFINITY;
        if (2 * c + 1 >= cols) y[c].y = -INFINITY;
        top = fmaxf(top, fmaxf(y[c].x, y[c].y));
      }
    }
    float ask = top - set_at<kQ8>();  // for the row's reference
    if constexpr (!kQ8) ask = fmaxf(ask, st.l > 0x1p-4f ? st.m + 8.0f : -INFINITY);
    float* mine = red + (turn ? 256 : 0);  // two turns: who is two exchanges ahead has seen the other read
    turn = !turn;
    mine[half * 128 + row] = ask;
    bool shifted = false;
    if constexpr (kQ8) shifted = barrier_rows_or(quad, may);
    else barrier_rows(quad);
    if (kQ8 && shifted) {  // nothing has been done yet
      if (!st.fresh) wait_pv();
      tc_fence_after();
      const float2 ml = shifted_unit<R>(tx, o_addr, sc, cols, mul, st.m, st.l, st.fresh, red + 4 * 128, row, half);
      st.m = ml.x;
      st.l = ml.y;
      st.open = __any_sync(0xffffffffu, st.m == -INFINITY);
      st.fresh = false;
      return;
    }
    ask = fmaxf(ask, mine[(half ^ 1) * 128 + row]);
    // where one row moves, all do
    const float m_new = st.open || over || ask > st.m + (most_sum_log2<kQ8>() - 6 - set_at<kQ8>()) ? fmaxf(st.m, ask) : st.m;
    const float alpha = st.fresh || st.m == m_new ? 1.0f : ex2_approx(st.m - m_new);
    st.m = m_new;
    st.open = __any_sync(0xffffffffu, st.m == -INFINITY);  // the same in both warps of the rows
    st.l *= alpha;
    st.l_p *= alpha;
    const float ref = st.m == -INFINITY ? 0.0f : st.m;  // only infinite logits so far: weights of 0
    clear();
#pragma unroll
    for (int c = 0; c < 32; ++c) w[c] = weigh(fma2(y[c], make_float2(factor, factor), make_float2(-ref, -ref)), c);
    if (!st.fresh && __any_sync(0xffffffffu, alpha != 1.0f)) {
      // O holds the units before this one; each of the two warps scales half of its columns
      wait_pv();
      tc_fence_after();
#pragma unroll 1
      for (int c = 128 * half; c < 128 * half + 128; c += 32) {
        float o[32];
        tmem_ld32(o_addr + c, o);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] *= alpha;
        tmem_st32(o_addr + c, o);
      }
    }
  }
  st.l += sum[0].x + sum[1].x + sum[0].y + sum[1].y;
  st.l_p += sum_p[0].x + sum_p[1].x + sum_p[0].y + sum_p[1].y;
  tmem_st16(tx, reinterpret_cast<const float*>(w));
  tmem_st16(tx + 32, reinterpret_cast<const float*>(w + 16));
  tc_wait_st();
  st.fresh = false;
}

template <int kFmt, bool kTurn>
__device__ void softmax_role(const ChunkParams& p, const Ctx& cx, const PlanSmem& s, int pair, LineRange range, uint32_t tmem,
                             uint8_t* gbase) {
  constexpr bool kQ8 = kQuant<kFmt>;
  using Sm = Smem<kFmt>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = warp >> 2, quad = warp & 3, row = 32 * quad + lane;
  const int j = 2 * (int)cx.rank + (quad >> 1);  // token of the tile
  const uint32_t lanes = (uint32_t)(32 * quad) << 16, o_addr = tmem + lanes + kTmemO;
  const float c2 = p.scale == 0.0f && !kQ8 ? 1e-37f : p.scale * kLog2e;  // (0 times an infinity would be NaN)
  const uint32_t p_full = cx.leader_bar(PFull), o_free = cx.leader_bar(OFree);
  float* red = reinterpret_cast<float*>(gbase + Sm::red);
  uint32_t cnt = 0, pieces = 0;  // units, pieces so far
  bool turn = false;             // of the exchanges between the two warps of the rows
  // After a wait that gave up, the warp goes through the rest of its work without waiting, so that the warps that meet it
  // at named barriers, which have no limit, do not wait for it in vain. What it computes is meaningless.
  bool alive = true;
  auto wait = [&](int bar, uint32_t parity) { alive = alive && cx.wait_warp(bar, parity); };
  // P V of unit n. S of that unit is done, and with it every MMA issued before it, P V of two units earlier (the last on the
  // same barrier) among them: the parity is exact.
  auto wait_pv = [&](uint32_t n) { wait(PvDone + (n & 1), (n >> 1) & 1); };
  Piece q, last;
  RowState st, last_st;
  for (bool more = true; more; ++pieces) {
    more = next_piece<kTurn>(p, s, range, q);
    if (kQ8 && !more) break;
    const int seen = more && j < q.tokens ? q.seen0 + j : 0;  // keys that this row sees
    st = RowState();
    float mul = c2;  // of the row's products: the softmax scale, and the power of two of its Q terms
    if constexpr (kQ8) {
      wait(QFull, pieces & 1);
      mul *= split_queries(cx.base + Sm::q, red + 4 * 128, row, quad, half);
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(cx.leader_bar(QReady));
      barrier_rows(quad);  // red is free again
    }
    int u = q.u0;
    do {
      if (more) {
        const uint32_t buf = cnt & 1, tx = tmem + lanes + buf * kSCols + 64 * half;
        const uint32_t sc_slot = cnt % kScaleSlots;
        const float* sc = reinterpret_cast<const float*>(gbase + Sm::scales + sc_slot * kScaleBytes) + 64 * half;
        const int cols = min(max(seen - u * kUnitKeys - half * kPageSize, 0), kPageSize);  // this thread's keys
        if (kQ8) wait(ScFull + sc_slot, (cnt / kScaleSlots) & 1);
        // quantised: a look at two of the 64 V scales of this warp's page; the threads of the rows together see those of both.
        bool may = false;
        if constexpr (kQ8) {
          const float2 v = reinterpret_cast<const float2*>(sc + kUnitKeys)[lane];
          may = may_shift<Range<kFmt>>(2 * lane < cols ? v.x : 1.0f) | may_shift<Range<kFmt>>(2 * lane + 1 < cols ? v.y : 1.0f);
        }
        wait(SFull + buf, (cnt >> 1) & 1);
        tc_fence_after();
        if (seen > u * kUnitKeys) {
          softmax_tile_unit<kQ8, Range<kFmt>>(st, tx, o_addr, sc, cols, seen >= (u + 1) * kUnitKeys, may, mul, red, turn, row, quad, half,
                                              [&]() { wait_pv(cnt - 1); });
        } else {  // no key of this unit: weights of zero
          const float none[16] = {};
          tmem_st16(tx, none);
          tmem_st16(tx + 32, none);
          tc_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_pair(p_full + 8 * buf);
          if (kQ8) mbar_arrive(cx.bar(ScEmpty + sc_slot));
        }
        ++cnt;
      }
      if (!kQ8 && pieces > 0 && u == q.u0) {  // the output of the piece before
        wait_pv(cnt - (more ? 2 : 1));
        tc_fence_after();
        red[(4 + half) * 128 + row] = last_st.l;
        red[(6 + half) * 128 + row] = last_st.l_p;
        barrier_rows(quad);
        const uint32_t done = pieces - 1;
        const bool odd = reinterpret_cast<volatile const uint32_t*>(gbase + Sm::odd)[done & 3] == done + 1;
        write_piece<kFmt, 128>(p, cx, last, last_st.l + red[(4 + (half ^ 1)) * 128 + row], last_st.l_p + red[(6 + (half ^ 1)) * 128 + row],
                               last_st.m, pair, o_addr, o_free, row, 128 * half, odd);
        barrier_rows(quad);  // red is free again
      }
    } while (more && ++u < q.u1);
    if constexpr (kQ8) {
      RowStats& to = reinterpret_cast<RowStats*>(gbase + Sm::stats)[pieces & (kStats - 1)];
      to.l[half][row] = st.l;
      if (half == 0) to.m[row] = st.m;
      __syncwarp();
      if (lane == 0) mbar_arrive(cx.bar(StFull + (pieces & (kStats - 1))));
    } else {
      last = q;
      last_st = st;
    }
  }
}

template <int kFmt, bool kTurn>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads<kFmt>(), 1)
    chunk_attention_tc_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap kmap,
                              const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
  using Sm = Smem<kFmt>;
  constexpr bool kQ8 = kQuant<kFmt>;
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  const uint32_t raw = smem_u32(dyn_smem);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = dyn_smem + (base - raw);
  PlanSmem& plan = *reinterpret_cast<PlanSmem*>(gbase + Sm::plan);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Sm::misc);
  int* abort_flag = reinterpret_cast<int*>(gbase + Sm::misc + 4);
  const int warp = threadIdx.x >> 5;
  Ctx cx{base, base + Sm::bars, base + Sm::odd, cta_rank(), abort_flag, p.err, p.wait_budget_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) {
      const bool of_pair = i == PFull || i == PFull + 1 || i == QReady;  // every softmax warp of both CTAs
      const bool of_cta = i >= ScEmpty && i < ScEmpty + kScaleSlots;     // and value warp of this one
      const bool of_values = kQ8 && (i == VFull || i == VFull + 1);
      mbar_init(cx.bar(i), of_pair                         ? 2 * kSoftmaxWarps
                           : of_cta                        ? kSoftmaxWarps + kValueWarps
                           : of_values                     ? 2 * kValueWarps
                           : i == OFree                    ? 2 * output_warps<kFmt>()
                           : i >= StFull && i < Drain      ? kSoftmaxWarps
                           : i >= RawEmpty                 ? kValueWarps
                           : i >= TailReady && i < RawFull ? 2
                                                           : 1);
    }
    *abort_flag = 0;
    plan.rest = {0, 0};
    for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(gbase + Sm::odd)[i] = 0;
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
  {  // hints only, these may still be written: what the plan needs, in L2
    const int i = threadIdx.x * 8;  // of 4-byte elements: a sector a thread
    if (blockIdx.x == 0 && i < p.B) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.seq_lens + i));
    if (blockIdx.x == 0 && i <= p.B) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q_starts + i));
  }
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  build_plan(p, plan, blockIdx.x == 0 ? p.err : nullptr);
  cluster_wait();  // as are the other's; what it does to its own shared memory until its loads begin concerns no one else
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int units = plan.cost[p.B], W = busy_pairs(p, units), pair = blockIdx.x >> 1;
  const int lo = pair < W ? range_of_pair(pair, units, W) : 0, hi = pair < W ? range_of_pair(pair + 1, units, W) : 0;
  LineRange range{lo, hi};
  if (kTurn && units > p.l2_units) {
    if (lo < hi) range.from = begin_of(p, plan, lo, hi);
    __syncthreads();
    if (threadIdx.x == 0) plan.rest = {lo, range.from};
    __syncthreads();
  }

  if (warp < kSoftmaxWarps) {
    softmax_role<kFmt, kTurn>(p, cx, plan, pair, range, tmem, gbase);
  } else if (warp == kProducerWarp) {
    producer_role<kFmt, kTurn>(p, &kmap, &vmap, &qmap, cx, plan, range);
  } else if (warp >= kValueWarp) {
    if constexpr (kQ8)
      value_role<kFmt, kTurn>(p, cx, plan, pair, range, tmem, gbase);
    else
      tail_role<kTurn>(p, cx, plan, range);
  } else if (cx.rank == 1) {  // (its MMAs are issued by the leader)
    if (pair == 0) publish_parts(p, plan, threadIdx.x & 31);
    write_unseeing(p, plan, pair, threadIdx.x & 31);
  } else if (elect_one()) {
    mma_role<kFmt, kTurn>(p, cx, plan, range, tmem);
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

// ---------------------------------------------------------------- combine
// Joins the parts of the tiles that lie in several ranges. With O_s and lse_s of part s, M = max_s lse_s and
// w_s = exp(lse_s - M):  out = sum_s w_s O_s / sum_s w_s,  lse = M + ln sum_s w_s.  A warp takes half a row, eight parts at a
// time, with a running M, or, of tiles with up to four and two parts, one or two rows: eight loads of 16 bytes in flight a
// lane. The first part is the second partial result of its pair (a tile that begins there), the others are the first ones of
// the pairs behind it. Bound by latency: the list of tiles, then the parts, of groups on one line that the blocks share. Three
// blocks an SM are there at once; with more a call without parts took 1 us longer, and with four parts of a row at a time 23
// tokens behind 900 took 1.7 us longer.
constexpr int kCombineThreads = 256, kCombineWarps = kCombineThreads / 32, kCombineBlocksPerPair = 6;
static_assert(kCombineWarps == 8, "combine_groups");
// Of the part with the largest LSE: the weights of all have a sum of at most 1, and what they join is no larger than the parts.
constexpr float kPartWeight = 1.0f / 128;
static_assert(kChunkMaxPairs + 1 <= 128, "parts of a tile");
// kRows rows from r on of a tile whose first row is `first` and whose first part is pair `pair`'s; kHalves halves of them from
// `half` on, kParts parts at a time; dims 4 lane .. 4 lane + 3 of a half.
template <int kRows, int kHalves, int kParts>
__device__ __forceinline__ void combine_rows(const ChunkParams& p, int first, int pair, int parts, int r, int half, int lane) {
  static_assert(kRows * kHalves * kParts == 8, "loads in flight");
  float mx[kRows], den[kRows], acc[kRows][kHalves][4];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    mx[j] = -INFINITY;
    den[j] = 0.0f;
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[j][h][c] = 0.0f;
  }
#pragma unroll 1
  for (int i0 = 0; i0 < parts; i0 += kParts) {
    float4 x[kRows][kHalves][kParts];
    float z[kRows][kParts];
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      const int i = min(i0 + k, parts - 1);  // (behind the last part: the last one, without weight)
      const size_t part = (size_t)part_slot(pair + i, i == 0) * 256 + r;
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        z[j][k] = __ldcg(p.part_lse + part + j);
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          x[j][h][k] = __ldcg(reinterpret_cast<const float4*>(p.part_o + (part + j) * kHeadDim) + 32 * (half + h) + lane);
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const float before = mx[j];
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        if (i0 + k >= parts) z[j][k] = -INFINITY;
        mx[j] = fmaxf(mx[j], z[j][k]);
      }
      const float base = mx[j] == -INFINITY ? 0.0f : mx[j];  // (no finite logit so far: weights of 0)
      const float old = exp2f((before - base) * kLog2e);
      den[j] *= old;
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[j][h][c] = old == 0.0f ? 0.0f : acc[j][h][c] * old;
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        const float w = exp2f((z[j][k] - base) * kLog2e) * kPartWeight;
        den[j] += w;
        if (w != 0.0f) {  // of weight 0 (or no part): left out, never scaled
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            acc[j][h][0] = fmaf(w, x[j][h][k].x, acc[j][h][0]);
            acc[j][h][1] = fmaf(w, x[j][h][k].y, acc[j][h][1]);
            acc[j][h][2] = fmaf(w, x[j][h][k].z, acc[j][h][2]);
            acc[j][h][3] = fmaf(w, x[j][h][k].w, acc[j][h][3]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const float inv = 1.0f / den[j];
    const size_t row = (size_t)first * kHeads + r + j;
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
      reinterpret_cast<uint2*>(p.out + row * kHeadDim)[32 * (half + h) + lane] =
          make_uint2(pack_bf16(acc[j][h][0] * inv, acc[j][h][1] * inv), pack_bf16(acc[j][h][2] * inv, acc[j][h][3] * inv));
    if (half == 0 && lane == 0) p.lse[row] = mx[j] + log2f(den[j] / kPartWeight) * kLn2;
  }
}
__global__ void __launch_bounds__(kCombineThreads, 3) chunk_combine_kernel(const ChunkParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  // The list by one warp of a block: by all of them, their requests for the same lines take the call 1.4 us.
  static_assert((kChunkMaxPairs + 1) % 32 == 0, "lanes");
  __shared__ int4 list[kChunkMaxPairs + 1];
  __shared__ int s_groups;
  if (warp == 0) {
    constexpr int kHeld = (kChunkMaxPairs + 32) / 32;
    int4 e[kHeld];
    int groups = 0x7fffffff;
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      e[k] = 32 * k + lane <= p.pairs ? __ldcg(p.parts + 32 * k + lane) : make_int4(0, 0, 0, 0x7fffffff);
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      list[32 * k + lane] = e[k];
      if (e[k].y == 0) groups = min(groups, e[k].w);
    }
    groups = __reduce_min_sync(0xffffffffu, groups);
    if (lane == 0) s_groups = groups;
  }
  __syncthreads();
  int i = 0;  // the tile of group g
#pragma unroll 1
  for (int g = blockIdx.x; g < s_groups; g += gridDim.x) {
    while (g >= list[i + 1].w) ++i;
    const int4 at = list[i];  // first row, tokens | parts << 8, first pair, first group
    const int first = at.x, parts = at.y >> 8, item = (g - at.w) * kCombineWarps + warp;
    if (parts <= 2)
      combine_rows<2, 2, 2>(p, first, at.z, parts, 2 * item, 0, lane);
    else if (parts <= 4)
      combine_rows<1, 2, 4>(p, first, at.z, parts, item, 0, lane);
    else
      combine_rows<1, 1, 8>(p, first, at.z, parts, item >> 1, item & 1, lane);
  }
}

template <int kFmt, bool kTurn>
cudaError_t launch_chunk(const ChunkParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, const CUtensorMap& qmap,
                         cudaStream_t stream) {
  const size_t smem = Smem<kFmt>::total + 1024;
  static int configured[kTrackedDevices] = {};
  const cudaError_t e = ensure_dynamic_smem(chunk_attention_tc_kernel<kFmt, kTurn>, smem, configured);
  if (e != cudaSuccess) return e;
  return launch_pdl(chunk_attention_tc_kernel<kFmt, kTurn>, dim3(2 * p.pairs), dim3(threads<kFmt>()), smem, stream, p, kmap, vmap, qmap);
}
template <int kFmt>
cudaError_t launch_chunk(const ChunkParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap, const CUtensorMap& qmap,
                         cudaStream_t stream) {
  // Pieces that may turn cost a short prompt or few tiles 1 to 2% even where none does (16 of 512 tokens 160.0 -> 163.9 us, E4M3
  // 233.5 -> 235.5, E2M1 233.4 -> 238.1; 304 tokens behind 16080 168.3 -> 169.6), so there is a kernel without, for calls whose
  // pages fit L2 whatever their lengths. The host knows capacities alone: tables and a pool as small as that are a small server's
  // or a test's, and one whose pool fills the card has the other kernel in every step. Half a unit a page.
  const bool turn = 0.5 * std::min((long long)p.B * p.max_pages, (long long)p.num_pages) > p.l2_units;
  return turn ? launch_chunk<kFmt, true>(p, kmap, vmap, qmap, stream) : launch_chunk<kFmt, false>(p, kmap, vmap, qmap, stream);
}
}  // namespace

cudaError_t launch_chunk_attention_tc(const ChunkParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                      const CUtensorMap& qmap, cudaStream_t stream) {
  return p.fmt == kKvBf16   ? launch_chunk<kKvBf16>(p, kmap, vmap, qmap, stream)
         : p.fmt == kKvE4M3 ? launch_chunk<kKvE4M3>(p, kmap, vmap, qmap, stream)
                            : launch_chunk<kKvE2M1>(p, kmap, vmap, qmap, stream);
}

cudaError_t launch_chunk_combine(const ChunkParams& p, cudaStream_t stream) {
  return launch_pdl(chunk_combine_kernel, dim3(kCombineBlocksPerPair * p.pairs), dim3(kCombineThreads), 0, stream, p);
}

}  // namespace mfa
