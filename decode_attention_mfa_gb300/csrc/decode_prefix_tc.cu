// decode_prefix_tc.cu -- decode attention for a batch whose sequences share
// prefixes: the pages of a group's prefix are read once for four sequences at a
// time instead of once for each, and in the same kernel every sequence reads
// what it holds behind its prefix.
//
// A group's queries form one matrix of 64 n rows (64 heads, n sequences), and
//     S = Q K^T,  P = exp2(scale log2(e) S - m),  O = P V,  l = P 1
// over the prefix is ordinary matrix work: 4 * 64 * 256 flops a sequence and
// key, against 1 KB (bf16) a key for the whole group, so from about five
// sequences on the tensor cores bound it and not memory. The tokens behind the
// prefix are bound by memory. Both are row tiles of one line of work, so that some SMs
// stream while others compute; the LSE combine joins a sequence's parts.
//
// Tile: a cluster of two CTAs works on 256 rows (four sequences of a group, two
// a CTA; one sequence for its own tokens) against units of 128 keys (two pages)
// with tcgen05 MMAs of cta_group::2: each CTA holds the Q rows of its
// sequences, one of the two K pages and half of V's dimensions, and both halves
// feed the pair's MMAs. Against one CTA with 128 rows this halves what every SM
// reads from L2 (128 KB in 2048 tensor cycles, which L2 cannot serve to 152
// SMs) and what the MMAs read from shared memory for B. A sequence's own tokens
// use a quarter of the rows, but then a unit still takes the tensor cores less
// time (2048 cycles for a pair) than HBM at its share of the bandwidth (128 KB).
// TMEM holds S twice (2 x 128 columns; P overwrites S in place and is the A
// operand of P V from there) and O (256 columns): all of it.
//
// Work split: the row tiles, one after the other, form a line of units
// (kPrefixPieceUnits more for every tile: its Q load and partial result); each
// pair takes an equal range of it (stream-K) and writes a normalised partial
// result and its LSE per row tile that it holds units of.
//
// Warp roles:
//   warps 0-7  softmax: thread = row = TMEM lane; warp w and w + 4 share 32
//              rows, 64 keys of a unit each, and agree on the reference maximum, which moves
//              only when a row exceeds it by 2^8 (then O is rescaled).
//   warp 8     producer (TMA, each CTA its own halves, completing on the leader's barriers).
//   warp 9     MMA issue (one thread of the leader) and TMEM allocation.
//   warp 10    the rows behind a sequence's last token in V, zeroed up to the
//              end of an MMA's 16 (E4M3: 32) keys: 0 * NaN of a stale row would poison P V.
// Every wait is bounded (the wait budget), as in the split kernel.
//
// E4M3 cache: both products are 8-bit MMAs (kind::f8f6f4) on the raw codes. Q
// enters as two E4M3 terms under a power of two per row, split in shared memory
// when a row tile begins; P times the V scale enters as two E4M3 terms, kept
// within 2^8 by the same moving reference: with a the reference and p =
// 2^(logit - a), O sums p * v_scale * code and l sums p, so that any a gives
// the same O / l, and a follows max(logit) + log2(largest V scale of the unit).
// Two terms at twice the 16-bit rate cost the tensor cores what bf16 does.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <type_traits>

#include "mfa_device.cuh"

namespace mfa {
namespace {

constexpr int kSoftmaxWarps = 8, kProducerWarp = 8, kMmaWarp = 9, kTailWarp = 10;
constexpr int kThreads = 352;
// Two K and two V slots, of even and odd units, one CTA's half of a unit each: K one page of 256 dims, V 128 dims of two
// pages (each page's half at kHalf). A K slot is free when S of its unit is done, a V slot when P V is, which the
// softmax warps are told anyway: the issuing thread commits twice a unit. (With a ring of 16 KB granules it waited
// four times and committed six times a unit, and a unit took 3600 cycles instead of XXXX.)
template <bool kFp8>
__host__ __device__ constexpr uint32_t slot_bytes() { return kFp8 ? 16384 : 32768; }
constexpr int kUnitKeys = 2 * kPageSize;
constexpr int kScaleSlots = 4;         // E4M3: 128 K scales and 128 V scales a unit
constexpr int kScaleBytes = 1024;
constexpr int kQBytes = 65536;         // 128 rows x 256 dims, four 64-dim blocks of [128 rows x 128 B]
constexpr int kSeqQBytes = 32768;      // one sequence's rows
constexpr int kTmemCols = 512, kTmemO = 256, kSCols = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// log2 units: P (E4M3: P * v_scale) stays below 2^top between moves of the reference, and a move leaves the largest of
// them `headroom` below that. E4M3: below 2^0, held as codes of 2^8 times it (split_p2), so that a move leaves 2^5 as the
// largest code and the small weights above the smallest steps.
template <bool kFp8>
__host__ __device__ constexpr float top_weight() { return kFp8 ? 0.0f : 8.0f; }
template <bool kFp8>
__host__ __device__ constexpr float headroom() { return kFp8 ? 3.0f : 8.0f; }
// Keys of one MMA of P V.
template <bool kFp8>
__host__ __device__ constexpr int key_step() { return kFp8 ? 32 : 16; }
static_assert(kPrefixTileSeqs * kHeads == 256, "rows of a row tile");

enum Bar {
  KFull = 0,                 // [2] leader: both CTAs' halves landed
  VFull = KFull + 2,         // [2] leader
  QFull = VFull + 2,         // bf16: leader; E4M3: both, each its own rows
  QReady,                    // E4M3, leader: Q split into terms, one arrival per softmax warp of the pair
  SFull,                     // [2] both: S of even and odd units
  PFull = SFull + 2,         // [2] leader: one arrival per softmax warp of the pair
  PvDone = PFull + 2,        // [2] both: P V of even and odd units
  OFree = PvDone + 2,        // leader: O has been read, one arrival per softmax warp of the pair
  Drain,                     // leader
  ScFull,                    // [kScaleSlots] E4M3, both
  ScEmpty = ScFull + kScaleSlots,   // [kScaleSlots] one arrival per softmax warp of the CTA
  TailFull = ScEmpty + kScaleSlots, // [2] both: this CTA's V of a partial last unit landed (by V slot)
  TailReady = TailFull + 2,         // [2] leader: its rows behind the last token are zero, one arrival a CTA
  kBars = TailReady + 2
};

// The line of work as every CTA sees it. Indices of sequences and tiles fit 16 bits (at most 1024 sequences).
struct PlanSmem {
  int32_t cost[kMaxBatch + 1];   // units of the prefix tiles of the groups before g; [n_groups]: of all
  int32_t own[kMaxBatch + 1];    // units of the own tokens of the sequences before b
  uint16_t b0[kMaxBatch + 2];    // first sequence of group g
  uint16_t lead[kMaxBatch];      // the sequence whose table row gives the prefix pages, | kOdd; kUnshared: not shared
  uint16_t tile[kMaxBatch + 2];  // prefix tiles of the groups before g
  uint16_t tail[kMaxBatch];      // keys in the last unit of b's own tokens (0: it has none), | kBehind
};
constexpr uint16_t kOdd = 0x8000;       // the prefix has an odd number of pages
constexpr uint16_t kUnshared = 0x7FFF;
constexpr uint16_t kBehind = 0x8000;    // b's own tokens begin behind its group's prefix
struct PlanScratch {
  int32_t count[kMaxBatch], lead[kMaxBatch], pages[kMaxBatch], len[kMaxBatch], group[kMaxBatch];
};

template <bool kFp8>
struct Smem {
  static constexpr uint32_t k = 0;
  static constexpr uint32_t v = k + 2 * slot_bytes<kFp8>();
  static constexpr uint32_t q = v + 2 * slot_bytes<kFp8>();
  static constexpr uint32_t scales = q + kQBytes;
  static constexpr uint32_t plan = scales + (kFp8 ? kScaleSlots * kScaleBytes : 0);
  static constexpr uint32_t red = (plan + (uint32_t)sizeof(PlanSmem) + 15) & ~15u;  // [2][128] exchange of the row halves
  static constexpr uint32_t bars = red + 2 * 128 * 4;
  static constexpr uint32_t misc = bars + 8 * kBars;  // TMEM base, abort flag
  static constexpr uint32_t total = misc + 8;
};
static_assert(Smem<false>::total + 1024 <= 227 * 1024 && Smem<true>::total + 1024 <= 227 * 1024, "shared memory");
static_assert(4 * slot_bytes<true>() >= sizeof(PlanScratch), "the plan's scratch lies in the K and V slots");

// ---------------------------------------------------------------- cluster pair
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_to_leader(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrival on a barrier of the other CTA. What it announces lies in tensor memory, which the tcgen05 fences order, so no
// release at cluster scope is needed: that one waits for all of the thread's memory operations (a unit took 3800
// cycles with it).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// The same behind writes to shared memory that the other CTA's MMAs read.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Whether a phase is complete, without waiting for it.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// TMA load into this CTA's shared memory that completes on a barrier of the pair's leader.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y,
                                                 uint32_t leader_bar, uint64_t cache_hint) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(leader_bar), "l"(cache_hint)
      : "memory");
}
__device__ __forceinline__ void tc_mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tc_mma_pair_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                   uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tc_mma_pair_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A from tensor memory: 8-bit elements 4j .. 4j + 3 of a row in column j.
__device__ __forceinline__ void tc_mma_pair_f8_tmem_a(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                      uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrival on the barrier at the same offset of both CTAs once every MMA issued so far is done.
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// True in one thread of a converged warp. The compiler knows that it is one, and then issues a tcgen05 instruction behind
// it without a loop over the threads that might be active.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
  return ok != 0;
}

struct Ctx {
  uint32_t base, bar0, rank;
  volatile int* abort;
  uint32_t* err;
  uint64_t budget;
  __device__ uint32_t bar(int i) const { return bar0 + 8u * (uint32_t)i; }
  __device__ uint32_t leader_bar(int i) const { return map_to_leader(bar(i)); }
  __device__ bool wait(int i, uint32_t parity) const { return mbar_wait(bar(i), parity, budget, abort, err); }
  // the same for a whole warp, whose lanes give up together
  __device__ bool wait_warp(int i, uint32_t parity) const { return __all_sync(0xffffffffu, wait(i, parity)); }
  // a barrier that threads of the other CTA arrive on
  __device__ __noinline__ bool wait_pair_slow(int i, uint32_t parity) const {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_cluster(bar(i), parity)) {
      if (*abort) return false;
      if (globaltimer_ns() - t0 > budget) {
        raise_error(err, MFA_DEVERR_TIMEOUT);
        *abort = 1;
        return false;
      }
    }
    return true;
  }
  __device__ bool wait_pair(int i, uint32_t parity) const {
    return mbar_try_wait_cluster(bar(i), parity) || wait_pair_slow(i, parity);
  }
};

// ---------------------------------------------------------------- plan
// Largest g in [0, n) with a[g] <= x (a is non-decreasing and a[0] <= x).
template <typename T>
__device__ __forceinline__ int last_at_most(const T* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int)a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ int warp_inclusive_sum(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
__device__ __forceinline__ int tiles_of_group(const PlanSmem& s, int g) {
  return (s.b0[g + 1] - s.b0[g] + kPrefixTileSeqs - 1) / kPrefixTileSeqs;
}
// Pages of a shared group's prefix.
__device__ __forceinline__ int pages_of_group(const PlanSmem& s, int g) {
  const int units = (s.cost[g + 1] - s.cost[g]) / tiles_of_group(s, g) - kPrefixPieceUnits;
  return 2 * units - ((s.lead[g] & kOdd) ? 1 : 0);
}

// A group shares its prefix if at least two of its sequences hold all of it;
// a sequence that ends inside it (or an empty slot of the batch) is read on its
// own, so that no row of a shared product has a mask and nothing behind its
// last token is ever read for it. All threads; ends with a barrier.
__device__ void build_plan(const PrefixParams& p, PlanSmem& s, PlanScratch& t, uint32_t* err) {
  const int n = p.n_groups, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int g = threadIdx.x; g < n; g += kThreads) {
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
    t.len[b] = clamp_len(__ldcg(p.seq_lens + b), p.max_pages * kPageSize, err);
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
        s.b0[g] = (uint16_t)x;
      }
      top = __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    int of = -1;
    if (b >= s.b0[0] && b < s.b0[n]) {
      const int g = last_at_most(s.b0, n + 1, b), pages = t.pages[g];
      if (pages > 0 && t.len[b] >= pages * kPageSize) {
        of = g;
        atomicAdd(&t.count[g], 1);
        atomicMin(&t.lead[g], b);
      }
    }
    t.group[b] = of;
  }
  __syncthreads();
  if (warp == 0) {
    int units = 0, tiles = 0;
    for (int g0 = 0; g0 < n; g0 += 32) {
      const int g = g0 + lane;
      const bool shared = g < n && t.count[g] >= 2;
      const int nt = shared ? tiles_of_group(s, g) : 0;
      const int nu = shared ? nt * ((t.pages[g] + 1) / 2 + kPrefixPieceUnits) : 0;
      const int x = warp_inclusive_sum(nu, lane), y = warp_inclusive_sum(nt, lane);
      if (g < n) {
        s.cost[g] = units + x - nu;
        s.tile[g] = (uint16_t)(tiles + y - nt);
        s.lead[g] = shared ? (uint16_t)(t.lead[g] | ((t.pages[g] & 1) ? kOdd : 0)) : kUnshared;
      }
      units += __shfl_sync(0xffffffffu, x, 31);
      tiles += __shfl_sync(0xffffffffu, y, 31);
    }
    if (lane == 0) s.cost[n] = units;
  } else if (warp == 1) {
    int units = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      int rest = 0, u = 0;
      uint16_t behind = 0;
      if (b < p.B) {
        const int g = t.group[b];
        rest = t.len[b];
        if (g >= 0 && t.count[g] >= 2) {
          rest -= t.pages[g] * kPageSize;
          behind = kBehind;
        }
        u = rest > 0 ? (rest + kUnitKeys - 1) / kUnitKeys + kPrefixPieceUnits : 0;
      }
      const int x = warp_inclusive_sum(u, lane);
      if (b < p.B) {
        s.own[b] = units + x - u;
        s.tail[b] = (uint16_t)((rest > 0 ? (rest - 1) % kUnitKeys + 1 : 0) | behind);
      }
      units += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) s.own[p.B] = units;
  }
  fence_proxy_async_smem();  // the scratch is TMA's from here on
  __syncthreads();
}

// Pairs that have work: with fewer units than pairs, every range holds one.
__device__ __forceinline__ int busy_pairs(const PrefixParams& p, int units) { return min(p.pairs, max(units, 1)); }

// Where the combine finds each sequence's partial results.
__device__ void publish_plan(const PrefixParams& p, const PlanSmem& s) {
  const int n = p.n_groups, C1 = s.cost[n], C = C1 + s.own[p.B], W = busy_pairs(p, C);
  for (int b = blockIdx.x * kThreads + threadIdx.x; b < p.B; b += gridDim.x * kThreads) {
    int4 parts = make_int4(0, 0, 0, 0);
    if (s.tail[b] & kBehind) {
      const int g = last_at_most(s.b0, n + 1, b), j = b - s.b0[g], i = j / kPrefixTileSeqs;
      const int len = (s.cost[g + 1] - s.cost[g]) / tiles_of_group(s, g);  // units of one tile
      const long long x = s.cost[g] + (long long)i * len;
      const int w = cta_of_cost(x + kPrefixPieceUnits, C, W);
      parts.x = (w + s.tile[g] + i) * kPrefixTileSeqs + j % kPrefixTileSeqs;
      parts.y = cta_of_cost(x + len - 1, C, W) - w + 1;
    }
    if (s.tail[b] & ~kBehind) {
      const int w = cta_of_cost((long long)C1 + s.own[b] + kPrefixPieceUnits, C, W);
      parts.z = p.own_row0 + w + b;
      parts.w = cta_of_cost((long long)C1 + s.own[b + 1] - 1, C, W) - w + 1;
    }
    p.parts[b] = parts;
  }
}

// A pair's pieces, in order: units [u0, u1) of one row tile.
struct Piece {
  const int32_t* pages;  // page-table entries of the tile's keys
  int b, seqs;           // first sequence, sequences (1 to kPrefixTileSeqs)
  int keys;              // keys of the tile
  int u0, u1;            // units
  int row;               // partial result of its first sequence
  bool own;              // a sequence's own tokens
  long long x;           // line position behind the tile
};
__device__ __forceinline__ bool next_piece(const PrefixParams& p, const PlanSmem& s, int pair, long long hi, Piece& q) {
  const int n = p.n_groups, C1 = s.cost[n];
  while (q.x < hi) {
    long long first;
    int len;
    q.own = q.x >= C1;
    if (!q.own) {
      const int g = last_at_most(s.cost, n, (int)q.x), lead = s.lead[g] & ~kOdd;
      len = (s.cost[g + 1] - s.cost[g]) / tiles_of_group(s, g);
      const int i = ((int)q.x - s.cost[g]) / len;
      first = s.cost[g] + (long long)i * len;
      q.b = s.b0[g] + i * kPrefixTileSeqs;
      q.seqs = min(kPrefixTileSeqs, s.b0[g + 1] - q.b);
      q.keys = (len - kPrefixPieceUnits) * kUnitKeys - ((s.lead[g] & kOdd) ? kPageSize : 0);
      q.pages = p.page_table + (size_t)lead * p.max_pages;
      q.row = (pair + s.tile[g] + i) * kPrefixTileSeqs;
    } else {
      const int b = last_at_most(s.own, p.B, (int)(q.x - C1)), tail = s.tail[b];
      len = s.own[b + 1] - s.own[b];
      first = (long long)C1 + s.own[b];
      q.b = b;
      q.seqs = 1;
      q.keys = (len - kPrefixPieceUnits - 1) * kUnitKeys + (tail & ~kBehind);
      q.pages = p.page_table + (size_t)b * p.max_pages;
      if (tail & kBehind) q.pages += pages_of_group(s, last_at_most(s.b0, n + 1, b));
      q.row = p.own_row0 + pair + b;
    }
    q.u0 = max(0, (int)(q.x - first) - kPrefixPieceUnits);
    q.u1 = (int)min((long long)len, hi - first) - kPrefixPieceUnits;
    q.x = first + len;
    if (q.u0 < q.u1) return true;
  }
  return false;
}
__device__ __forceinline__ int keys_in_unit(const Piece& q, int u) { return min(kUnitKeys, q.keys - u * kUnitKeys); }
// A last unit whose last MMA of P V reaches behind the sequence's last token.
template <bool kFp8>
__device__ __forceinline__ bool is_tail(const Piece& q, int valid) { return q.own && valid % key_step<kFp8>() != 0; }

// ---------------------------------------------------------------- producer
// Page ids of a tile: a window of 64 held by the warp (32 ahead of need).
struct TilePages {
  const int32_t* row;
  int end, base, a, b;
  __device__ int fetch(int pg, const PrefixParams& p) const {
    if (pg >= end) return 0;
    const int id = __ldg(row + pg);
    if (id >= 0 && id < p.num_pages) return id;
    raise_error(p.err, MFA_DEVERR_PAGE);
    return 0;
  }
  __device__ void start(int pg, const PrefixParams& p, int lane) {
    base = pg;
    a = fetch(base + lane, p);
    b = fetch(base + 32 + lane, p);
  }
  __device__ int get(int pg, const PrefixParams& p, int lane) {
    while (pg >= base + 64) {
      base += 32;
      a = b;
      b = fetch(base + 32 + lane, p);
    }
    const int i = pg - base;
    return i < 32 ? __shfl_sync(0xffffffffu, a, i) : __shfl_sync(0xffffffffu, b, i - 32);
  }
};

template <bool kFp8>
__device__ void producer_role(const PrefixParams& p, const CUtensorMap* kmap, const CUtensorMap* vmap,
                              const CUtensorMap* qmap, const Ctx& cx, const PlanSmem& s, int pair, long long lo,
                              long long hi) {
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
    if (lane == 0) {
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
      if (lane == 0) {
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
  // zeroes its rows.
  auto load_v = [&](uint32_t n, int pa, int pb, bool tail, uint64_t pol) -> bool {
    const uint32_t slot = n & 1;
    if (n >= 2 && !cx.wait_warp(PvDone + slot, ((n >> 1) & 1) ^ 1)) return false;
    if (lane == 0) {
      const uint32_t dst = cx.base + Sm::v + slot * kSlot, bytes = pb >= 0 ? kSlot : kPage;
      if (r == 0) mbar_arrive_expect_tx(cx.bar(VFull + slot), tail ? 0 : 2 * bytes);
      if (tail) mbar_arrive_expect_tx(cx.bar(TailFull + slot), bytes);
      const uint32_t bar = tail ? cx.bar(TailFull + slot) : cx.leader_bar(VFull + slot);
      for (int i = 0; i < (pb >= 0 ? 2 : 1); ++i)
#pragma unroll
        for (int d = 0; d < 128 / kCols; ++d)
          tma_load_2d_pair(dst + i * kPage + d * 8192, vmap, r * 128 + d * kCols, (i ? pb : pa) * kPageSize, bar, pol);
    }
    tails[slot] += tail;
    return true;
  };
  Piece q;
  q.x = lo;
  uint32_t cnt = 0;      // units whose K has been loaded
  int va = -1, vb = -1;  // the last of them: its V is still to be loaded (V trails K by a unit, as the MMAs use them)
  bool vtail = false, good = true;
  uint64_t vpol = pol_own;
  while (good && next_piece(p, s, pair, hi, q)) {
    TilePages ids;
    ids.row = q.pages;
    ids.end = min((q.keys + kPageSize - 1) / kPageSize, 2 * q.u1);
    ids.start(2 * q.u0, p, lane);
    const uint64_t pol = q.own ? pol_own : pol_shared;
    // Q may be replaced once S of every unit so far is done
    good = cnt == 0 || cx.wait_warp(SFull + ((cnt - 1) & 1), ((cnt - 1) >> 1) & 1);
    if (!good) break;
    if (lane == 0) {
      const int here = min(2, max(0, q.seqs - 2 * r));  // this CTA's sequences
      if (kFp8)
        mbar_arrive_expect_tx(cx.bar(QFull), here * kSeqQBytes);
      else if (r == 0)
        mbar_arrive_expect_tx(cx.bar(QFull), q.seqs * kSeqQBytes);
      const uint32_t bar = kFp8 ? cx.bar(QFull) : cx.leader_bar(QFull);
      for (int d = 0; d < 4; ++d)
        for (int h = 0; h < here; ++h)
          tma_load_2d_pair(cx.base + Sm::q + d * 16384 + h * 8192, qmap, d * 64, (q.b + 2 * r + h) * kHeads, bar, pol_shared);
    }
    ++pieces;
    for (int u = q.u0; good && u < q.u1; ++u) {
      const int valid = keys_in_unit(q, u);
      const int pa = ids.get(2 * u, p, lane);
      const int pb = valid > kPageSize ? ids.get(2 * u + 1, p, lane) : -1;
      good = load_k(cnt, pa, pb, pol);
      if (good && va >= 0) good = load_v(cnt - 1, va, vb, vtail, vpol);
      ++cnt;
      va = pa;
      vb = pb;
      vtail = is_tail<kFp8>(q, valid);
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
      if (r == 0) (void)mbar_wait(cx.bar(KFull + (k & 1)), (k >> 1) & 1, cx.budget, nullptr, p.err);
      if (r == 0 && (good || k + 1 < cnt)) (void)mbar_wait(cx.bar(VFull + (k & 1)), (k >> 1) & 1, cx.budget, nullptr, p.err);
    }
    for (int i = 0; i < 2; ++i)
      if (tails[i]) (void)mbar_wait(cx.bar(TailFull + i), (tails[i] - 1) & 1, cx.budget, nullptr, p.err);
    if constexpr (kFp8)
      for (uint32_t k = cnt > (uint32_t)kScaleSlots ? cnt - kScaleSlots : 0; k < cnt; ++k)
        (void)mbar_wait(cx.bar(ScFull + k % kScaleSlots), (k / kScaleSlots) & 1, cx.budget, nullptr, p.err);
    if (pieces && (kFp8 || r == 0)) (void)mbar_wait(cx.bar(QFull), (pieces - 1) & 1, cx.budget, nullptr, p.err);
  }
  __syncwarp();
}

// ---------------------------------------------------------------- rows behind the last token
template <bool kFp8>
__device__ void tail_role(const PrefixParams& p, const Ctx& cx, const PlanSmem& s, int pair, long long lo, long long hi) {
  constexpr int kStep = key_step<kFp8>(), kChunks = kFp8 ? 1 : 2;  // 128 B chunks of a V row half: 128 or 64 dims
  const int lane = threadIdx.x & 31;
  uint32_t cnt = 0, tails[2] = {0, 0};
  Piece q;
  q.x = lo;
  while (next_piece(p, s, pair, hi, q)) {
    cnt += q.u1 - q.u0;
    const int valid = keys_in_unit(q, q.u1 - 1);
    if (!is_tail<kFp8>(q, valid)) continue;
    const uint32_t slot = (cnt - 1) & 1;
    if (!cx.wait_warp(TailFull + slot, tails[slot] & 1)) return;
    ++tails[slot];
    const uint32_t base = cx.base + Smem<kFp8>::v + slot * slot_bytes<kFp8>() + (valid / kPageSize) * (slot_bytes<kFp8>() / 2);
    const int row = valid % kPageSize, words = (kStep - valid % kStep) * 8;  // 16 B words of a chunk's rows
    for (int i = lane; i < words * kChunks; i += 32) {
      const uint32_t at = base + (i / words) * 8192 + row * 128 + (i % words) * 16;
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(cx.leader_bar(TailReady + slot));
  }
}

// ---------------------------------------------------------------- MMA issue (one thread of the leader)
template <bool kFp8>
__device__ void mma_role(const PrefixParams& p, const Ctx& cx, const PlanSmem& s, int pair, long long lo, long long hi,
                         uint32_t tmem) {
  constexpr uint32_t idesc_s = idesc_f16(256, kSCols, kFp8 ? 0 : 1, 0, 0);    // A = Q, B = K, both K-major (E4M3: format 0)
  constexpr uint32_t idesc_o = idesc_f16(256, kHeadDim, kFp8 ? 0 : 1, 0, 1);  // A = P (TMEM), B = V (dim-major)
  using Sm = Smem<kFp8>;
  uint32_t pieces = 0, s_cnt = 0, p_cnt = 0, tails[2] = {0, 0};
  // Descriptors of the operands' first blocks; a block `bytes` further on has bytes / 16 more in the address field, which
  // holds every shared address without a carry.
  auto ahead = [](uint64_t desc, uint32_t bytes) -> uint64_t { return desc + (bytes >> 4); };
  const uint64_t q_desc = smem_desc_sw128(cx.base + Sm::q, 16, 1024);
  const uint64_t k_desc0 = smem_desc_sw128(cx.base + Sm::k, 16, 1024);
  const uint64_t v_desc0 = smem_desc_sw128(cx.base + Sm::v, kFp8 ? 16 : 8192, 1024);
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
        tc_mma_pair_f8(d, ahead(q_desc, (i >> 3) * 32768 + h * 16384 + kk * 32), ahead(k_desc, h * 8192 + kk * 32), idesc_s, i != 0);
      } else {  // 64-dim block, 16 dims
        const int e = i >> 2, kk = i & 3;
        tc_mma_pair(d, ahead(q_desc, e * 16384 + kk * 32), ahead(k_desc, e * 8192 + kk * 32), idesc_s, i != 0);
      }
    }
    tc_commit_pair(cx.bar(SFull + buf));
    ++s_cnt;
    return true;
  };
  // P V of a unit of `valid` keys: as many MMAs as hold one
  struct Unit {
    int valid;
    bool tail, first;
    uint32_t piece;
  };
  auto do_pv = [&](const Unit& v) -> bool {
    constexpr int kStep = key_step<kFp8>(), kSteps = kPageSize / kStep;
    const uint32_t buf = p_cnt & 1, a = tmem + buf * kSCols, d = tmem + kTmemO;
    if (v.first && !cx.wait(OFree, (v.piece & 1) ^ 1)) return false;
    if (v.tail && !cx.wait_pair(TailReady + buf, tails[buf]++ & 1)) return false;
    if (!pv_ready && !(cx.wait(VFull + buf, (p_cnt >> 1) & 1) && cx.wait(PFull + buf, (p_cnt >> 1) & 1))) return false;
    tc_fence_after();
    const uint64_t v_desc = ahead(v_desc0, buf * slot_bytes<kFp8>());
    auto mma = [&](int i, int t, int kk, bool add) {  // page i, term t of P (E4M3), step kk
      if constexpr (kFp8)
        tc_mma_pair_f8_tmem_a(d, a + t * 32 + i * 16 + kk * 8, ahead(v_desc, i * 8192 + kk * 4096), idesc_o, add);
      else
        tc_mma_pair_tmem_a(d, a + i * 32 + kk * 8, ahead(v_desc, i * 16384 + kk * 2048), idesc_o, add);
    };
    constexpr int kTerms = kFp8 ? 2 : 1;
    if (v.valid == kUnitKeys) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
#pragma unroll
          for (int kk = 0; kk < kSteps; ++kk) mma(i, t, kk, (i | t | kk) != 0 || !v.first);
        if (i == 0) k_ready = peek(KFull + (s_cnt & 1), (s_cnt >> 1) & 1);
      }
    } else {
      for (int i = 0; i * kPageSize < v.valid; ++i)
        for (int t = 0; t < kTerms; ++t)
          for (int kk = 0; kk < min(kSteps, (v.valid - i * kPageSize + kStep - 1) / kStep); ++kk)
            mma(i, t, kk, (i | t | kk) != 0 || !v.first);
      k_ready = false;
    }
    tc_commit_pair(cx.bar(PvDone + buf));
    ++p_cnt;
    return true;
  };
  Piece q;
  q.x = lo;
  Unit pend{0, false, false, 0};  // the unit whose P V is still to be issued (valid = 0: none)
  bool good = true;
  while (good && next_piece(p, s, pair, hi, q)) {
    good = kFp8 ? cx.wait_pair(QReady, pieces & 1) : cx.wait(QFull, pieces & 1);
    for (int u = q.u0; good && u < q.u1; ++u) {
      good = do_s(pend.valid != 0);
      if (good && pend.valid) good = do_pv(pend);
      const int valid = keys_in_unit(q, u);
      pend = Unit{valid, is_tail<kFp8>(q, valid), u == q.u0, pieces};
    }
    if (kFp8 && good) {  // the softmax warps split the next Q once they have read this O
      pv_ready = false;
      good = do_pv(pend);
      pend.valid = 0;
    }
    ++pieces;
  }
  if (good && pend.valid) {
    pv_ready = false;
    (void)do_pv(pend);
  }
  tc_commit_pair(cx.bar(Drain));  // every MMA is done before TMEM is given back
  (void)mbar_wait(cx.bar(Drain), 0, cx.budget, nullptr, p.err);
}

// ---------------------------------------------------------------- softmax
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 32 bytes at once: a whole sector of one row a thread.
__device__ __forceinline__ void st_global_v8(float* dst, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
// Barriers of the two warps that share 32 rows, and of all softmax warps.
__device__ __forceinline__ void barrier_rows(int quad) { asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory"); }
__device__ __forceinline__ bool barrier_rows_or(int quad, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, %2, 64, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(1 + quad)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void barrier_softmax() { asm volatile("bar.sync 5, 256;" ::: "memory"); }

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

// E4M3: the bf16 Q of this CTA's 128 rows (four 64-dim blocks of [128 rows x 128 B], 128-byte swizzle) becomes, in
// place, two E4M3 terms of Q * 2^e ([term][128-dim half][128 rows x 128 B]): t1 rounds the scaled value, t2 the rest,
// which is exact unless it falls below the E4M3 normal range (2^-18.8 of the row's largest |q|). 2^e is the largest
// power of two that keeps the row within the E4M3 maximum, 448. Thread (row, half) takes 128 dims of its row. All
// softmax threads; red: their exchange. Returns 2^-e.
__device__ __noinline__ float split_q(uint32_t q_addr, float* red, int row, int half) {
  uint4 v[16];  // 8 dims each
#pragma unroll
  for (int j = 0; j < 16; ++j)
    v[j] = ld_shared_v4(q_addr + (2 * half + (j >> 3)) * 16384 + row * 128 + (((j & 7) ^ (row & 7)) << 4));
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
  }
  red[half * 128 + row] = top;
  barrier_softmax();  // every row is in registers: the terms may overwrite it
  top = fmaxf(red[row], red[128 + row]);
  int e = 0;
  if (top > 0.0f && top <= 3.0e38f) {
    const uint32_t bits = __float_as_uint(top);
    e = ((bits & 0x7FFFFFu) <= 0x600000u ? 8 : 7) - ((int)((bits >> 23) & 0xFFu) - 127);  // top * 2^e in (224, 448]
    e = max(-126, min(126, e));
  }
  const float up = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
  for (int o = 0; o < 8; ++o) {  // 16 dims
    uint32_t t1[4], t2[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t w[4] = {v[2 * o + u].x, v[2 * o + u].y, v[2 * o + u].z, v[2 * o + u].w};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t a = 0, b = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float x = __uint_as_float(w[2 * i + k] << 16) * up, y = __uint_as_float(w[2 * i + k] & 0xFFFF0000u) * up;
          const __nv_fp8x2_storage_t c1 = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
          const __half2_raw h1 = __nv_cvt_fp8x2_to_halfraw2(c1, __NV_E4M3);
          const float2 d1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
          const __nv_fp8x2_storage_t c2 = __nv_cvt_float2_to_fp8x2(make_float2(x - d1.x, y - d1.y), __NV_SATFINITE, __NV_E4M3);
          a |= (uint32_t)c1 << (16 * k);
          b |= (uint32_t)c2 << (16 * k);
        }
        t1[2 * u + i] = a;
        t2[2 * u + i] = b;
      }
    }
    const uint32_t at = q_addr + half * 16384 + row * 128 + ((o ^ (row & 7)) << 4);
    st_shared_v4(at, t1);
    st_shared_v4(at + 32768, t2);
  }
  fence_proxy_async_smem();
  return __uint_as_float((uint32_t)(127 - e) << 23);
}

// Two weights times their V scales, y in [-1, 1], as two E4M3 terms each of 2^8 y. E4M3 has exponent bias 7 and f16 has
// 15, so the f16 bits of y (of which the exponent's top one is 0), the sign moved behind that bit and without the low
// seven, are the E4M3 code of 2^8 y, subnormals included: integer arithmetic on both halves gives the first term, y's
// bits rounded, and an f16 difference without error what is left. kConvert: the second term by a conversion, else by
// the same arithmetic. A conversion keeps the unit that also does the exponentials for 8 cycles a warp, the integer form
// the ALU for about as long, so that neither alone is best (with three conversions a pair the softmax took 2600 cycles a
// unit, with integers alone 3600).
struct TermPair {
  uint32_t hi;  // codes of the first terms in bytes 1 and 3
  uint32_t lo;  // of the second ones: bytes 0 and 1 if converted, else 1 and 3
};
__device__ __forceinline__ uint32_t e4m3_bytes(uint32_t f) { return ((f + f) & 0x7FFF7FFFu) | (f & 0x80008000u); }
template <bool kConvert>
__device__ __forceinline__ TermPair split_p2(float2 y) {
  TermPair t;
  const __half2 h = __floats2half2_rn(y.x, y.y);
  const uint32_t up = *reinterpret_cast<const uint32_t*>(&h) + 0x00400040u, first = up & 0xFF80FF80u;
  t.hi = e4m3_bytes(up);
  __half2 rest = __hsub2(h, *reinterpret_cast<const __half2*>(&first));
  if constexpr (kConvert) {
    rest = __hmul2(rest, __half2half2(__ushort_as_half(0x5C00)));  // 2^8
    t.lo = __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&rest), __NV_SATFINITE, __NV_E4M3);
  } else {
    t.lo = e4m3_bytes(*reinterpret_cast<const uint32_t*>(&rest) + 0x00400040u);
  }
  return t;
}

template <bool kFp8>
__device__ void softmax_role(const PrefixParams& p, const Ctx& cx, const PlanSmem& s, int pair, long long lo,
                             long long hi, uint32_t tmem, uint8_t* gbase) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = warp >> 2, quad = warp & 3, row = 32 * quad + lane;
  const uint32_t lanes = (uint32_t)(32 * quad) << 16;
  const float c2 = p.scale * kLog2e;
  const bool neg = p.scale < 0.0f;  // the smallest product then makes the largest logit
  const uint32_t p_full = cx.leader_bar(PFull), o_free = cx.leader_bar(OFree);
  float* red = reinterpret_cast<float*>(gbase + Smem<kFp8>::red);
  uint32_t cnt = 0, pieces = 0;  // units, pieces so far
  // P V of the unit before `cnt`. S of that unit is done, and with it every MMA issued before it, P V of two units
  // earlier (the last on the same barrier) among them: the parity is exact.
  auto wait_pv = [&]() -> bool { return cx.wait_warp(PvDone + ((cnt - 1) & 1), ((cnt - 1) >> 1) & 1); };
  Piece q;
  q.x = lo;
  while (next_piece(p, s, pair, hi, q)) {
    const int j = 2 * (int)cx.rank + (quad >> 1);  // sequence of the row tile
    const bool mine = j < q.seqs;
    float m = -INFINITY, l = 0.0f;  // the row's reference (log2 units), and this thread's share of its denominator
    float mul = c2;                 // of the row's products: the softmax scale, and 2^-e of its Q terms
    if constexpr (kFp8) {
      if (!cx.wait_warp(QFull, pieces & 1)) return;
      mul *= split_q(cx.base + Smem<kFp8>::q, red, row, half);
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cx.leader_bar(QReady));
      barrier_rows(quad);  // red is free again
      ++pieces;
    }
    for (int u = q.u0; u < q.u1; ++u, ++cnt) {
      const uint32_t buf = cnt & 1, ts = tmem + lanes + buf * kSCols;
      const uint32_t sc_slot = cnt % kScaleSlots;
      const float* sc = reinterpret_cast<const float*>(gbase + Smem<kFp8>::scales + sc_slot * kScaleBytes);
      if (kFp8 && !cx.wait_warp(ScFull + sc_slot, (cnt / kScaleSlots) & 1)) return;
      if (!cx.wait_warp(SFull + buf, (cnt >> 1) & 1)) return;
      tc_fence_after();
      if (mine) {
        const int valid = keys_in_unit(q, u), cols = min(64, valid - 64 * half);  // this thread's keys (none: <= 0)
        float2 x[32];
        tmem_ld32(ts + 64 * half, reinterpret_cast<float*>(x));
        tmem_ld32(ts + 64 * half + 32, reinterpret_cast<float*>(x) + 32);
        float lift = 0.0f;  // E4M3: log2 of the unit's largest V scale
        if constexpr (kFp8) {
          float4 v4 = reinterpret_cast<const float4*>(sc + 128)[lane];
          if (4 * lane + 3 >= valid) {  // scales behind the last key are stale
            if (4 * lane >= valid) v4.x = 0.0f;
            if (4 * lane + 1 >= valid) v4.y = 0.0f;
            if (4 * lane + 2 >= valid) v4.z = 0.0f;
            v4.w = 0.0f;
          }
          const float most = fmaxf(fmaxf(fabsf(v4.x), fabsf(v4.y)), fmaxf(fabsf(v4.z), fabsf(v4.w)));
          lift = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
          l += lift - lift;                     // NaN for a scale that is not finite: the integer codes would hide it
          lift = fmaxf(__log2f(lift), -90.0f);  // so that p stays far from 2^128 whatever the scales are
        }
        tc_wait_ld();
        if constexpr (kFp8) {  // products times the K scales
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float4 k4 = reinterpret_cast<const float4*>(sc + 64 * half)[c / 2];
            x[c] = mul2(x[c], make_float2(k4.x, k4.y));
            x[c + 1] = mul2(x[c + 1], make_float2(k4.z, k4.w));
          }
        }
        if (cols < 64) {  // behind the last key: out of the maximum, and weights of 0 below
          const float out = neg ? 3.0e38f : -3.0e38f;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (2 * c >= cols) x[c].x = out;
            if (2 * c + 1 >= cols) x[c].y = out;
          }
        }
        float top[4];
        if (!neg) {
#pragma unroll
          for (int c = 0; c < 32; ++c) top[c & 3] = c < 4 ? fmaxf(x[c].x, x[c].y) : max3(top[c & 3], x[c].x, x[c].y);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) top[c & 3] = c < 4 ? fmaxf(-x[c].x, -x[c].y) : max3(top[c & 3], -x[c].x, -x[c].y);
        }
        float big = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * fabsf(mul);
        big = cols > 0 ? big + (lift - (top_weight<kFp8>() - headroom<kFp8>())) : -INFINITY;
        // the barrier also lets P overwrite the columns that the other warp has read
        if (barrier_rows_or(quad, big > m + headroom<kFp8>() || u == q.u0)) {
          red[half * 128 + row] = big;
          barrier_rows(quad);
          const float m_new = fmaxf(m, fmaxf(big, red[(half ^ 1) * 128 + row]));
          const float alpha = u == q.u0 || m == m_new ? 1.0f : ex2_approx(m - m_new);
          m = m_new;
          l *= alpha;
          if (u != q.u0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
            // O holds the units before this one; each of the two warps scales half of its columns
            if (!wait_pv()) return;
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
          }
        }
        const float ref = m == -INFINITY ? 0.0f : m;  // only infinite logits so far: weights of 0
        const float2 mul_2 = make_float2(mul, mul), ref_2 = make_float2(-ref, -ref);
        // weights, their sum, and P; kPart: only the first `cols` keys count
        auto weights = [&](auto part) {
          constexpr bool kPart = decltype(part)::value;
          float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
          uint32_t w[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            x[c] = fma2(x[c], mul_2, ref_2);
            x[c].x = ex2_approx(x[c].x);
            x[c].y = ex2_approx(x[c].y);
            if constexpr (kPart) {
              if (2 * c >= cols) x[c].x = 0.0f;
              if (2 * c + 1 >= cols) x[c].y = 0.0f;
            }
            sum[c & 1] = add2(sum[c & 1], x[c]);
            if constexpr (!kFp8) w[c] = pack_bf16(x[c].x, x[c].y);  // the A operand is 16 bits: half a step, 2^-8, of each weight
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          if constexpr (kFp8) {  // words 0-15: first terms of the 64 keys, 16-31: second ones
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float4 v4 = reinterpret_cast<const float4*>(sc + 128 + 64 * half)[c / 2];
              float2 a = mul2(x[c], make_float2(v4.x, v4.y)), b = mul2(x[c + 1], make_float2(v4.z, v4.w));
              if constexpr (kPart) {  // a stale scale may be NaN
                if (2 * c >= cols) a.x = 0.0f;
                if (2 * c + 1 >= cols) a.y = 0.0f;
                if (2 * c + 2 >= cols) b.x = 0.0f;
                if (2 * c + 3 >= cols) b.y = 0.0f;
              }
              const TermPair ta = split_p2<true>(a), tb = split_p2<true>(b);
              w[c / 2] = __byte_perm(ta.hi, tb.hi, 0x7531);
              w[16 + c / 2] = __byte_perm(ta.lo, tb.lo, 0x5410);
            }
            tmem_st16(ts + 16 * half, reinterpret_cast<const float*>(w));
            tmem_st16(ts + 32 + 16 * half, reinterpret_cast<const float*>(w + 16));
          } else {
            tmem_st32(ts + 32 * half, reinterpret_cast<const float*>(w));
          }
        };
        if (cols >= 64)
          weights(std::false_type{});
        else
          weights(std::true_type{});
        tc_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_pair(p_full + 8 * buf);
        if (kFp8) mbar_arrive(cx.bar(ScEmpty + sc_slot));
      }
    }
    // ---- the piece's partial result: O / l and its LSE, 128 dims a thread
    if (!wait_pv()) return;
    tc_fence_after();
    if (mine) {
      red[half * 128 + row] = l;
      barrier_rows(quad);
      l += red[(half ^ 1) * 128 + row];
      const size_t at = (size_t)(q.row + (q.own ? 0 : j)) * kHeads + (row & 63);
      const float inv = (kFp8 ? 0x1p-8f : 1.0f) / l;  // E4M3: the codes of P stand for 2^8 of it
      float* dst = p.part_o + at * kHeadDim;
#pragma unroll 1
      for (int c = 128 * half; c < 128 * half + 128; c += 32) {
        float o[32];
        tmem_ld32(tmem + lanes + kTmemO + c, o);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] *= inv;
#pragma unroll
        for (int k = 0; k < 32; k += 8) st_global_v8(dst + c + k, o + k);
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
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
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
      mbar_init(cx.bar(i), of_pair ? 2 * kSoftmaxWarps : of_cta ? kSoftmaxWarps : i >= TailReady ? 2 : 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kProducerWarp && (threadIdx.x & 31) == 0) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    prefetch_tensormap(&qmap);
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + Sm::misc),
                 "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  build_plan(p, plan, *reinterpret_cast<PlanScratch*>(gbase + Sm::k), blockIdx.x == 0 ? p.err : nullptr);
  publish_plan(p, plan);
  cluster_sync();  // the other CTA's barriers are initialised, its scratch is done with
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int units = plan.cost[p.n_groups] + plan.own[p.B], W = busy_pairs(p, units), pair = blockIdx.x >> 1;
  const long long lo = pair < W ? cta_cost_lo(pair, units, W) : 0, hi = pair < W ? cta_cost_lo(pair + 1, units, W) : 0;

  if (warp < kSoftmaxWarps) {
    softmax_role<kFp8>(p, cx, plan, pair, lo, hi, tmem, gbase);
  } else if (warp == kProducerWarp) {
    producer_role<kFp8>(p, &kmap, &vmap, &qmap, cx, plan, pair, lo, hi);
  } else if (warp == kTailWarp) {
    tail_role<kFp8>(p, cx, plan, pair, lo, hi);
  } else if (cx.rank == 0 && elect_one()) {
    mma_role<kFp8>(p, cx, plan, pair, lo, hi, tmem);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // no copy, MMA or arrival for either CTA is left
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
  return launch_pdl(decode_prefix_tc_kernel<kFp8>, dim3(2 * p.pairs), dim3(kThreads), smem, stream, p, kmap, vmap, qmap);
}
}  // namespace

cudaError_t launch_decode_prefix_tc(const PrefixParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                    const CUtensorMap& qmap, cudaStream_t stream) {
  return p.k_scale ? launch_prefix<true>(p, kmap, vmap, qmap, stream) : launch_prefix<false>(p, kmap, vmap, qmap, stream);
}

}  // namespace mfa
