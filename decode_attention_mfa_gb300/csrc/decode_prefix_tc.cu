// decode_prefix_tc.cu -- the shared-prefix part of decode attention: the
// queries of all the sequences of a group against the group's prefix, whose
// pages are read once for four sequences at a time instead of once for each.
//
// A group's queries form one matrix of 64 n rows (64 heads, n sequences), and
//     S = Q K^T,  P = exp2(scale log2(e) S - m),  O = P V,  l = P 1
// over the prefix is ordinary matrix work: 4 * 64 * 256 flops a sequence and
// key, against 1 KB (bf16) a key for the whole group, so from about five
// sequences on the tensor cores bound it and not memory. What a sequence has
// behind the prefix is left to the split kernel, and the LSE combine joins both
// by their log-sum-exps.
//
// Tile: a cluster of two CTAs works on 256 rows (four sequences, two a CTA)
// against 128 keys (two pages) with tcgen05 MMAs of cta_group::2: each CTA
// holds the Q rows of its two sequences, one of the two K pages and half of
// V's dimensions, and both halves feed the pair's MMAs. Against one CTA with
// 128 rows this halves what every SM reads from L2 (128 KB in 2048 tensor
// cycles, which L2 cannot serve to 152 SMs) and what the MMAs read from shared
// memory for B. TMEM holds S twice (2 x 128 columns, P overwrites S in place as
// 64 columns of bf16 pairs, and is the A operand of P V from there) and O (256
// columns): all of it.
//
// Work split: the row tiles of all groups, one after the other, form a line of
// units (one unit = one tile of 128 keys, and kPieceUnits for every tile's Q load and
// partial result); each pair takes an equal range of it (stream-K) and writes
// a normalised partial result and its LSE per row tile that it holds units of.
//
// Warp roles: warps 0-3 softmax (thread = row = TMEM lane: no exchange between
// threads; the reference maximum moves only when a row exceeds it by 2^8, then
// O is rescaled), warp 4 producer (TMA, each CTA its own halves, completing on
// the leader's barriers), warp 5 MMA issue (the leader's only).
// Every wait is bounded (the wait budget), as in the split kernel.
//
// E4M3 cache: both products are 8-bit MMAs (kind::f8f6f4) on the raw codes. Q
// enters as two E4M3 terms under a power of two per row, split in shared memory
// when a row tile begins; P times the V scale enters as two E4M3 terms, kept
// within [0, 2^8] by the same moving reference: with a the reference and p =
// 2^(logit - a), O sums p * v_scale * code and l sums p, so that any a gives
// the same O / l, and a follows max(logit) + log2(largest V scale of the unit).
// Two terms at twice the 16-bit rate cost the tensor cores what bf16 does.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "mfa_device.cuh"

namespace mfa {
namespace {

constexpr int kThreads = 192;
constexpr int kSoftmaxWarps = 4, kProducerWarp = 4, kMmaWarp = 5;
// Ring of 16 KB granules. bf16: half of a K page (128 dims), or 128 dims of a V page; E4M3: a K page, or 128 dims of
// two V pages.
template <bool kFp8>
__host__ __device__ constexpr int slots() { return kFp8 ? 8 : 9; }
constexpr int kGranule = 16384;
constexpr int kScaleSlots = 4;         // E4M3: 128 K scales and 128 V scales a unit
constexpr int kScaleBytes = 1024;
constexpr int kQBytes = 65536;         // 128 rows x 256 dims, four 64-dim blocks of [128 rows x 128 B]
constexpr int kTmemCols = 512, kTmemO = 256, kSCols = 128;
constexpr int kTileRows = 256;         // of the pair, 128 a CTA
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTop = 8.0f;           // log2 units: P (E4M3: P * v_scale) stays below 2^8 between moves of the reference
// Where a move leaves the largest of them: 2^0, and 2^5 for E4M3, whose small weights then lie above its smallest steps.
template <bool kFp8>
__host__ __device__ constexpr float headroom() { return kFp8 ? 3.0f : kTop; }
static_assert(kTileRows == kPrefixTileSeqs * kHeads, "rows of a row tile");

constexpr int kMaxSlots = 9;
enum Bar {
  Full = 0,                  // [slots] leader: both CTAs' halves landed
  Empty = Full + kMaxSlots,  // [slots] both: the MMAs reading the granule are done
  QFull = Empty + kMaxSlots, // bf16: leader; E4M3: both, each its own rows
  QReady,                    // E4M3, leader: Q split into terms, one arrival per softmax warp of the pair
  QEmpty,                    // both
  SFull,                    // [2] both
  PFull = SFull + 2,        // [2] leader: one arrival per softmax warp of the pair
  PvDone = PFull + 2,       // [2] both: P V of even and odd units
  OFree = PvDone + 2,                   // leader: O has been read, one arrival per softmax warp of the pair
  Drain,                    // leader
  ScFull,                   // [kScaleSlots] E4M3, both
  ScEmpty = ScFull + kScaleSlots,  // one arrival per softmax warp of the CTA
  kBars = ScEmpty + kScaleSlots
};

// Groups as every CTA sees them. Sizes and indices of sequences and tiles fit
// 16 bits (at most 1024 sequences).
struct PlanSmem {
  int32_t cost[kMaxBatch + 1];    // units before group g
  int32_t pages[kMaxBatch];       // prefix pages
  uint16_t b0[kMaxBatch + 2];     // first sequence
  uint16_t lead[kMaxBatch];       // the sequence whose table row gives the prefix pages; kUnshared: not shared
  uint16_t tile[kMaxBatch + 2];   // row tiles before group g
};
constexpr uint16_t kUnshared = 0xFFFF;

template <bool kFp8>
struct Smem {
  static constexpr uint32_t ring = 0;
  static constexpr uint32_t q = slots<kFp8>() * kGranule;
  static constexpr uint32_t scales = q + kQBytes;
  static constexpr uint32_t plan = scales + (kFp8 ? kScaleSlots * kScaleBytes : 0);
  static constexpr uint32_t bars = (plan + (uint32_t)sizeof(PlanSmem) + 7) & ~7u;
  static constexpr uint32_t misc = bars + 8 * kBars;
  static constexpr uint32_t total = misc + 16;
};
static_assert(Smem<false>::total + 1024 <= 227 * 1024 && Smem<true>::total + 1024 <= 227 * 1024, "shared memory");
static_assert(slots<true>() * kGranule >= 2 * 4 * kMaxBatch, "the plan's scratch lies in the ring");

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
__device__ __forceinline__ int units_of(int pages) { return (pages + 1) / 2; }

// A group shares its prefix if at least two of its sequences hold all of it;
// a sequence that ends inside it (or an empty slot of the batch) is left to the
// split kernel as a whole, so that no row of the shared product has a mask and
// nothing behind its last token is ever read for it. All threads; ends with a
// barrier. t: 2 * kMaxBatch ints of scratch.
__device__ void build_plan(const PrefixParams& p, PlanSmem& s, int32_t* t, uint32_t* err) {
  const int n = p.n_groups;
  int32_t* cnt = t;
  int32_t* lead = t + kMaxBatch;
  for (int g = threadIdx.x; g < n; g += kThreads) {
    int pages = __ldcg(p.prefix_pages + g);
    if (pages < 0 || pages > p.max_pages) {
      raise_error(err, MFA_DEVERR_CAPACITY);
      pages = pages < 0 ? 0 : p.max_pages;
    }
    s.pages[g] = pages;
    cnt[g] = 0;
    lead[g] = kMaxBatch;
  }
  if (threadIdx.x < 32) {  // starts, made non-decreasing within [0, B]: no sequence lies in two groups
    const int lane = threadIdx.x;
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
  const int b_end = s.b0[n];
  for (int b = s.b0[0] + (int)threadIdx.x; b < b_end; b += kThreads) {
    const int g = last_at_most(s.b0, n + 1, b), pages = s.pages[g];
    if (pages > 0 && __ldcg(p.seq_lens + b) >= pages * kPageSize) {
      atomicAdd(cnt + g, 1);
      atomicMin(lead + g, b);
    }
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int units = 0, tiles = 0;
    for (int g0 = 0; g0 < n; g0 += 32) {
      const int g = g0 + lane;
      const bool shared = g < n && cnt[g] >= 2;
      const int nt = shared ? (s.b0[g + 1] - s.b0[g] + kPrefixTileSeqs - 1) / kPrefixTileSeqs : 0;
      const int nu = shared ? nt * (units_of(s.pages[g]) + kPrefixPieceUnits) : 0;
      int x = nu, y = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
          x += a;
          y += b;
        }
      }
      if (g < n) {
        s.cost[g] = units + x - nu;
        s.tile[g] = (uint16_t)(tiles + y - nt);
        s.lead[g] = shared ? (uint16_t)lead[g] : kUnshared;
      }
      units += __shfl_sync(0xffffffffu, x, 31);
      tiles += __shfl_sync(0xffffffffu, y, 31);
    }
    if (lane == 0) s.cost[n] = units;
  }
  fence_proxy_async_smem();  // the scratch is TMA's from here on
  __syncthreads();
}

// Pairs that have work: with fewer units than pairs, every range holds one.
__device__ __forceinline__ int busy_pairs(const PrefixParams& p, int units) { return min(p.pairs, max(units, 1)); }

// What the later kernels of the call need to know of each sequence: the pages
// they skip, and where its partial results over the prefix are.
__device__ void publish_plan(const PrefixParams& p, const PlanSmem& s) {
  const int n = p.n_groups, C = s.cost[n], W = busy_pairs(p, C);
  for (int b = blockIdx.x * kThreads + threadIdx.x; b < p.B; b += gridDim.x * kThreads) {
    int skip = 0;
    int2 parts = make_int2(0, 0);
    if (b >= s.b0[0] && b < s.b0[n]) {
      const int g = last_at_most(s.b0, n + 1, b), pages = s.pages[g];
      if (s.lead[g] != kUnshared && __ldcg(p.seq_lens + b) >= pages * kPageSize) {
        const int u = units_of(pages), j = b - s.b0[g], i = j / kPrefixTileSeqs;
        const long long x0 = (long long)s.cost[g] + (long long)i * (u + kPrefixPieceUnits) + kPrefixPieceUnits;
        const int w0 = cta_of_cost(x0, C, W), w1 = cta_of_cost(x0 + u - 1, C, W);
        skip = pages;
        parts = make_int2((w0 + s.tile[g] + i) * kPrefixTileSeqs + j % kPrefixTileSeqs, w1 - w0 + 1);
      }
    }
    p.skip[b] = skip;
    p.parts[b] = parts;
  }
}

// A pair's pieces, in order: units [u0, u1) of one row tile.
struct Piece {
  int g, i;        // group, row tile of the group
  int u0, u1;      // units
  int pages;       // pages of the prefix
  long long x;     // line position behind the tile
};
__device__ __forceinline__ bool next_piece(const PlanSmem& s, int n, long long hi, Piece& q) {
  while (q.x < hi) {
    q.g = last_at_most(s.cost, n, (int)q.x);
    q.pages = s.pages[q.g];
    const int len = units_of(q.pages) + kPrefixPieceUnits;
    const int local = (int)q.x - s.cost[q.g];
    q.i = local / len;
    const long long first = (long long)s.cost[q.g] + (long long)q.i * len;
    q.u0 = max(0, (int)(q.x - first) - kPrefixPieceUnits);
    q.u1 = (int)min((long long)len, hi - first) - kPrefixPieceUnits;
    q.x = first + len;
    if (q.u0 < q.u1) return true;
  }
  return false;
}
__device__ __forceinline__ int pages_in_unit(const Piece& q, int u) { return 2 * u + 1 < q.pages ? 2 : 1; }

// ---------------------------------------------------------------- producer
// Page ids of the prefix: a window of 64 held by the warp (32 ahead of need).
struct PrefixPages {
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
                              const CUtensorMap* qmap, const Ctx& cx, const PlanSmem& s, long long lo, long long hi) {
  const int lane = threadIdx.x & 31;
  constexpr int kSlots = slots<kFp8>();
  using Sm = Smem<kFp8>;
  const int r = (int)cx.rank;
  const uint64_t pol = policy_evict_normal();
  uint32_t cc = 0, pieces = 0, units = 0;
  // The next granule: its address, and the leader's barrier of it, on which the leader announces `bytes` of both CTAs.
  auto next_slot = [&](uint32_t bytes, uint32_t& dst, uint32_t& bar) -> bool {
    const uint32_t slot = cc % kSlots, n = cc / kSlots;
    if (!cx.wait_warp(Empty + slot, (n & 1) ^ 1)) return false;
    dst = cx.base + Sm::ring + slot * kGranule;
    bar = cx.leader_bar(Full + slot);
    if (lane == 0 && r == 0) mbar_arrive_expect_tx(cx.bar(Full + slot), bytes);
    ++cc;
    return true;
  };
  // K of one unit: this CTA's page (page r of the two); bf16: in two granules of 128 dims
  auto load_k = [&](int pa, int pb) -> bool {
    const int page = r == 0 ? pa : pb;
    if constexpr (kFp8) {
      uint32_t dst, bar;
      if (!next_slot(pb >= 0 ? 2 * kGranule : kGranule, dst, bar)) return false;
      if (lane == 0 && page >= 0) {
        tma_load_2d_pair(dst, kmap, 0, page * kPageSize, bar, pol);
        tma_load_2d_pair(dst + 8192, kmap, 128, page * kPageSize, bar, pol);
      }
      // the scales of all the unit's keys, for this CTA's rows
      const uint32_t slot = units % kScaleSlots;
      if (!cx.wait_warp(ScEmpty + slot, ((units / kScaleSlots) & 1) ^ 1)) return false;
      ++units;
      if (lane == 0) {
        const uint32_t sc = cx.base + Sm::scales + slot * kScaleBytes, sb = cx.bar(ScFull + slot);
        constexpr uint32_t kPageScales = kPageSize * sizeof(float);
        mbar_arrive_expect_tx(sb, (pb >= 0 ? 4 : 2) * kPageScales);
        bulk_load(sc, p.k_scale + (size_t)pa * kPageSize, kPageScales, sb);
        bulk_load(sc + 512, p.v_scale + (size_t)pa * kPageSize, kPageScales, sb);
        if (pb >= 0) {
          bulk_load(sc + kPageScales, p.k_scale + (size_t)pb * kPageSize, kPageScales, sb);
          bulk_load(sc + 512 + kPageScales, p.v_scale + (size_t)pb * kPageSize, kPageScales, sb);
        }
      }
      return true;
    }
    for (int h = 0; h < 2; ++h) {
      uint32_t dst, bar;
      if (!next_slot(pb >= 0 ? 2 * kGranule : kGranule, dst, bar)) return false;
      if (lane == 0 && page >= 0) {
        tma_load_2d_pair(dst, kmap, h * 128, page * kPageSize, bar, pol);
        tma_load_2d_pair(dst + 8192, kmap, h * 128 + 64, page * kPageSize, bar, pol);
      }
    }
    return true;
  };
  // V of one unit: this CTA's 128 dims of each page; bf16: a granule a page
  auto load_v = [&](int pa, int pb) -> bool {
    if constexpr (kFp8) {
      uint32_t dst, bar;
      if (!next_slot(pb >= 0 ? 2 * kGranule : kGranule, dst, bar)) return false;
      if (lane == 0) {
        tma_load_2d_pair(dst, vmap, r * 128, pa * kPageSize, bar, pol);
        if (pb >= 0) tma_load_2d_pair(dst + 8192, vmap, r * 128, pb * kPageSize, bar, pol);
      }
      return true;
    }
    for (int i = 0; i < (pb >= 0 ? 2 : 1); ++i) {
      uint32_t dst, bar;
      if (!next_slot(2 * kGranule, dst, bar)) return false;
      const int page = i ? pb : pa;
      if (lane == 0) {
        tma_load_2d_pair(dst, vmap, r * 128, page * kPageSize, bar, pol);
        tma_load_2d_pair(dst + 8192, vmap, r * 128 + 64, page * kPageSize, bar, pol);
      }
    }
    return true;
  };
  Piece q;
  q.x = lo;
  int va = -1, vb = -1;  // the unit whose V is still to be loaded: V trails K by a unit, as the MMAs use them
  bool good = true;
  while (good && next_piece(s, p.n_groups, hi, q)) {
    PrefixPages ids;
    ids.row = p.page_table + (size_t)s.lead[q.g] * p.max_pages;
    ids.end = min(q.pages, 2 * q.u1);
    ids.start(2 * q.u0, p, lane);
    good = cx.wait_warp(QEmpty, (pieces & 1) ^ 1);
    if (!good) break;
    if (lane == 0) {
      const int row0 = (s.b0[q.g] + q.i * kPrefixTileSeqs + 2 * r) * kHeads;  // rows past the batch read zeros
      if (kFp8)
        mbar_arrive_expect_tx(cx.bar(QFull), kQBytes);
      else if (r == 0)
        mbar_arrive_expect_tx(cx.bar(QFull), 2 * kQBytes);
      const uint32_t bar = kFp8 ? cx.bar(QFull) : cx.leader_bar(QFull);
      for (int d = 0; d < 4; ++d)
        for (int h = 0; h < 2; ++h)
          tma_load_2d_pair(cx.base + Sm::q + d * 16384 + h * 8192, qmap, d * 64, row0 + h * 64, bar, pol);
    }
    ++pieces;
    for (int u = q.u0; good && u < q.u1; ++u) {
      const int pa = ids.get(2 * u, p, lane);
      const int pb = pages_in_unit(q, u) == 2 ? ids.get(2 * u + 1, p, lane) : -1;
      good = load_k(pa, pb);
      if (good && va >= 0) good = load_v(va, vb);
      va = pa;
      vb = pb;
    }
    if (kFp8 && good) {  // E4M3: the next row tile's Q is split only behind this one's last P V
      good = load_v(va, vb);
      va = -1;
    }
  }
  if (good && va >= 0) good = load_v(va, vb);
  // Every copy of both CTAs must land before either leaves: the leader's barriers tell, and the other CTA stays
  // until the cluster's last barrier.
  if (kFp8 && lane == 0) {
    for (uint32_t k = (units > (uint32_t)kScaleSlots ? units - kScaleSlots : 0); k < units; ++k)
      (void)mbar_wait(cx.bar(ScFull + k % kScaleSlots), (k / kScaleSlots) & 1, cx.budget, nullptr, p.err);
    if (pieces) (void)mbar_wait(cx.bar(QFull), (pieces - 1) & 1, cx.budget, nullptr, p.err);
  }
  if (r == 0 && lane == 0) {
    for (uint32_t k = (cc > (uint32_t)kSlots ? cc - kSlots : 0); k < cc; ++k)
      (void)mbar_wait(cx.bar(Full + k % kSlots), (k / kSlots) & 1, cx.budget, nullptr, p.err);
    if (!kFp8 && pieces) (void)mbar_wait(cx.bar(QFull), (pieces - 1) & 1, cx.budget, nullptr, p.err);
  }
  __syncwarp();
}

// ---------------------------------------------------------------- MMA issue (one thread of the leader)
template <bool kFp8>
__device__ void mma_role(const PrefixParams& p, const Ctx& cx, const PlanSmem& s, long long lo, long long hi,
                         uint32_t tmem) {
  constexpr uint32_t idesc_s = idesc_f16(256, kSCols, 1, 0, 0);  // A = Q, B = K, both K-major
  constexpr uint32_t idesc_o = idesc_f16(256, kHeadDim, 1, 0, 1);  // A = P (TMEM), B = V (dim-major)
  constexpr uint32_t idesc_s8 = idesc_f16(256, kSCols, 0, 0, 0), idesc_o8 = idesc_f16(256, kHeadDim, 0, 0, 1);  // E4M3
  constexpr int kSlots = slots<kFp8>();
  using Sm = Smem<kFp8>;
  uint32_t cc = 0, pieces = 0, s_cnt = 0, p_cnt = 0;
  auto do_s = [&]() -> bool {
    const uint32_t d = tmem + (s_cnt & 1) * kSCols;  // its last reader, P V of two units ago, was issued before
    if constexpr (kFp8) {
      const uint32_t slot = cc % kSlots;
      if (!cx.wait(Full + slot, (cc / kSlots) & 1)) return false;
      tc_fence_after();
      const uint32_t kb = cx.base + Sm::ring + slot * kGranule, qa = cx.base + Sm::q;
#pragma unroll
      for (int t = 0; t < 2; ++t)  // Q's terms
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_pair_f8(d, smem_desc_sw128(qa + t * 32768 + h * 16384 + kk * 32, 16, 1024),
                           smem_desc_sw128(kb + h * 8192 + kk * 32, 16, 1024), idesc_s8, (t | h | kk) != 0);
      tc_commit_pair(cx.bar(Empty + slot));
      ++cc;
    }
    for (int h = 0; !kFp8 && h < 2; ++h) {
      const uint32_t slot = cc % kSlots;
      if (!cx.wait(Full + slot, (cc / kSlots) & 1)) return false;
      tc_fence_after();
      const uint32_t kb = cx.base + Sm::ring + slot * kGranule;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t qa = cx.base + Sm::q + (2 * h + e) * 16384;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_pair(d, smem_desc_sw128(qa + kk * 32, 16, 1024), smem_desc_sw128(kb + e * 8192 + kk * 32, 16, 1024),
                      idesc_s, (h | e | kk) != 0);
      }
      tc_commit_pair(cx.bar(Empty + slot));
      ++cc;
    }
    tc_commit_pair(cx.bar(SFull + (s_cnt & 1)));
    ++s_cnt;
    return true;
  };
  auto do_pv = [&](int np, bool first, uint32_t piece) -> bool {
    const uint32_t buf = p_cnt & 1;
    if (first && !cx.wait_pair(OFree, (piece & 1) ^ 1)) return false;
    if (!cx.wait_pair(PFull + buf, (p_cnt >> 1) & 1)) return false;
    if constexpr (kFp8) {
      const uint32_t slot = cc % kSlots;
      if (!cx.wait(Full + slot, (cc / kSlots) & 1)) return false;
      tc_fence_after();
      const uint32_t vb = cx.base + Sm::ring + slot * kGranule;
      for (int i = 0; i < np; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)  // P's terms
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            tc_mma_pair_f8_tmem_a(tmem + kTmemO, tmem + buf * kSCols + t * 32 + i * 16 + kk * 8,
                                  smem_desc_sw128(vb + i * 8192 + kk * 4096, 16, 1024), idesc_o8,
                                  !(first && (i | t | kk) == 0));
      tc_commit_pair(cx.bar(Empty + slot));
      ++cc;
    }
    for (int i = 0; !kFp8 && i < np; ++i) {
      const uint32_t slot = cc % kSlots;
      if (!cx.wait(Full + slot, (cc / kSlots) & 1)) return false;
      tc_fence_after();
      const uint32_t vb = cx.base + Sm::ring + slot * kGranule;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        tc_mma_pair_tmem_a(tmem + kTmemO, tmem + buf * kSCols + i * 32 + kk * 8, smem_desc_sw128(vb + kk * 2048, 8192, 1024),
                           idesc_o, !(first && i == 0 && kk == 0));
      tc_commit_pair(cx.bar(Empty + slot));
      ++cc;
    }
    tc_commit_pair(cx.bar(PvDone + buf));
    ++p_cnt;
    return true;
  };
  Piece q;
  q.x = lo;
  int pend = 0;  // pages of the unit whose P V is still to be issued (0: none)
  bool pend_first = false, good = true;
  uint32_t pend_piece = 0;
  while (good && next_piece(s, p.n_groups, hi, q)) {
    good = kFp8 ? cx.wait_pair(QReady, pieces & 1) : cx.wait(QFull, pieces & 1);
    for (int u = q.u0; good && u < q.u1; ++u) {
      good = do_s();
      if (good && u == q.u1 - 1) tc_commit_pair(cx.bar(QEmpty));
      if (good && pend) good = do_pv(pend, pend_first, pend_piece);
      pend = pages_in_unit(q, u);
      pend_first = u == q.u0;
      pend_piece = pieces;
    }
    if (kFp8 && good) {  // the softmax warps split the next Q once they have read this O
      good = do_pv(pend, pend_first, pend_piece);
      pend = 0;
    }
    ++pieces;
  }
  if (good && pend) (void)do_pv(pend, pend_first, pend_piece);
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
// 32 lanes x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// 32 bytes at once: a whole sector of one row a thread.
__device__ __forceinline__ void st_global_v8(float* dst, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// ---- E4M3: this thread's row of Q (four 64-dim blocks of [128 rows x 128 B], 128-byte swizzle) becomes, in place, two
// E4M3 terms of Q * 2^e ([term][128-dim half][128 rows x 128 B]): t1 rounds the scaled value, t2 the rest, which is
// exact unless it falls below the E4M3 normal range (2^-18.8 of the row's largest |q|). 2^e is the largest power of two
// that keeps the row within the E4M3 maximum, 448. Returns 2^-e. All 128 threads.
__device__ __noinline__ float split_q_row(uint32_t q_addr, int row) {
  auto ld = [](uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
  };
  uint4 v[32];  // 8 dims each
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = ld(q_addr + (j >> 3) * 16384 + row * 128 + (((j & 7) ^ (row & 7)) << 4));
  asm volatile("bar.sync 1, 128;" ::: "memory");  // every row is in registers
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
  }
  int e = 0;
  if (top > 0.0f && top <= 3.0e38f) {
    const uint32_t bits = __float_as_uint(top);
    e = ((bits & 0x7FFFFFu) <= 0x600000u ? 8 : 7) - ((int)((bits >> 23) & 0xFFu) - 127);  // top * 2^e in (224, 448]
    e = max(-126, min(126, e));
  }
  const float up = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
  for (int o = 0; o < 16; ++o) {  // 16 dims
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
    const uint32_t at = q_addr + (o >> 3) * 16384 + row * 128 + (((o & 7) ^ (row & 7)) << 4);
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(t1[0]), "r"(t1[1]), "r"(t1[2]), "r"(t1[3]) : "memory");
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + 32768), "r"(t2[0]), "r"(t2[1]), "r"(t2[2]), "r"(t2[3]) : "memory");
  }
  fence_proxy_async_smem();
  return __uint_as_float((uint32_t)(127 - e) << 23);
}

// Two weights (times their V scales, at most 2^8) as two E4M3 terms each: c1 rounds them, c2 the rest, formed in f16
// (c1 is exact in f16, and so is the difference).
__device__ __forceinline__ void split_p2(float a, float b, uint32_t& c1, uint32_t& c2) {
  const __half2 x = __floats2half2_rn(a, b);
  const __nv_fp8x2_storage_t t1 = __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&x), __NV_SATFINITE, __NV_E4M3);
  const __half2_raw d1 = __nv_cvt_fp8x2_to_halfraw2(t1, __NV_E4M3);
  const __half2 rest = __hsub2(x, *reinterpret_cast<const __half2*>(&d1));
  c1 = t1;
  c2 = __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&rest), __NV_SATFINITE, __NV_E4M3);
}

template <bool kFp8>
__device__ void softmax_role(const PrefixParams& p, const Ctx& cx, const PlanSmem& s, long long lo, long long hi,
                             uint32_t tmem, int pair, const uint8_t* gbase) {
  const int row = threadIdx.x & 127, lane = row & 31;
  uint32_t pieces = 0;
  const uint32_t lanes = (uint32_t)(row & ~31) << 16;
  const float c2 = p.scale * kLog2e;
  const uint32_t p_full = cx.leader_bar(PFull), o_free = cx.leader_bar(OFree);
  uint32_t cnt = 0;  // units so far
  // P V of the unit before `cnt`. S of that unit is done, and with it every MMA issued before it, P V of two units
  // earlier (the last on the same barrier) among them: the parity is exact.
  auto wait_pv = [&]() -> bool { return cx.wait_warp(PvDone + ((cnt - 1) & 1), ((cnt - 1) >> 1) & 1); };
  Piece q;
  q.x = lo;
  while (next_piece(s, p.n_groups, hi, q)) {
    const int j = 2 * (int)cx.rank + (row >> 6);  // sequence of the row tile (the same for the whole warp)
    const bool mine = s.b0[q.g] + q.i * kPrefixTileSeqs + j < s.b0[q.g + 1];
    float m = -INFINITY, l = 0.0f;  // reference maximum (log2 units) and this row's denominator
    float mul = c2;                 // of this row's products: the softmax scale, and 2^-e of its Q terms
    if constexpr (kFp8) {
      if (!cx.wait_warp(QFull, pieces & 1)) return;
      mul *= split_q_row(cx.base + Smem<kFp8>::q, row);
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cx.leader_bar(QReady));
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
        const bool both = pages_in_unit(q, u) == 2;
        float x[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, x + 32 * c);
        tc_wait_ld();
        float lift = 0.0f;  // E4M3: log2 of the unit's largest V scale
        if constexpr (kFp8) {
          // products times the K scales; an absent page's scales are not there either
#pragma unroll
          for (int c = 0; c < 128; c += 4) {
            if (c == 64 && !both) break;
            const float4 k4 = reinterpret_cast<const float4*>(sc)[c / 4];
            x[c] *= k4.x;
            x[c + 1] *= k4.y;
            x[c + 2] *= k4.z;
            x[c + 3] *= k4.w;
          }
          float4 v4 = make_float4(0.f, 0.f, 0.f, 0.f);
          if (both || lane < 16) v4 = reinterpret_cast<const float4*>(sc + 128)[lane];
          const float most = fmaxf(fmaxf(fabsf(v4.x), fabsf(v4.y)), fmaxf(fabsf(v4.z), fabsf(v4.w)));
          lift = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
          lift = fmaxf(log2f(lift), -90.0f);  // so that p stays far from 2^128 whatever the scales are
        }
        // the largest logit of the unit (of one page: the other half of S is not of this prefix); a negative scale
        // makes it of the smallest product
        float top[4];
        if (mul >= 0.0f) {
#pragma unroll
          for (int c = 0; c < 64; ++c) top[c & 3] = c < 4 ? x[c] : fmaxf(top[c & 3], x[c]);
          if (both)
#pragma unroll
            for (int c = 64; c < 128; ++c) top[c & 3] = fmaxf(top[c & 3], x[c]);
        } else {
#pragma unroll
          for (int c = 0; c < 64; ++c) top[c & 3] = c < 4 ? -x[c] : fmaxf(top[c & 3], -x[c]);
          if (both)
#pragma unroll
            for (int c = 64; c < 128; ++c) top[c & 3] = fmaxf(top[c & 3], -x[c]);
        }
        float big = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * fabsf(mul);
        big += lift - (kTop - headroom<kFp8>());
        if (__any_sync(0xffffffffu, big > m + headroom<kFp8>() || u == q.u0)) {
          const float m_new = fmaxf(m, big);
          const float alpha = u == q.u0 || m == m_new ? 1.0f : ex2_approx(m - m_new);
          m = m_new;
          l *= alpha;
          if (u != q.u0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
            // O holds the units before this one: their last P V is done when its phase is
            if (!wait_pv()) return;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kHeadDim; c += 32) {
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
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c == 2 && !both) break;
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float a = ex2_approx(fmaf(x[32 * c + 2 * k], mul, -ref));
            float b = ex2_approx(fmaf(x[32 * c + 2 * k + 1], mul, -ref));
            sum[(2 * k) & 3] += a;
            sum[(2 * k + 1) & 3] += b;
            if constexpr (kFp8) {  // words 0-7: first terms of 32 keys, 8-15: second ones
              const float2 v2 = reinterpret_cast<const float2*>(sc + 128)[16 * c + k];
              uint32_t c1, c2;
              split_p2(a * v2.x, b * v2.y, c1, c2);
              w[k >> 1] = k & 1 ? w[k >> 1] | c1 << 16 : c1;
              w[8 + (k >> 1)] = k & 1 ? w[8 + (k >> 1)] | c2 << 16 : c2;
            } else {
              w[k] = pack_bf16(a, b);  // the A operand is 16 bits: half a step, 2^-8, of each weight
            }
          }
          if constexpr (kFp8) {
            tmem_st8(ts + 8 * c, w);
            tmem_st8(ts + 32 + 8 * c, w + 8);
          } else {
            tmem_st16(ts + 16 * c, reinterpret_cast<const float*>(w));
          }
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tc_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_cluster(p_full + 8 * buf);
        if (kFp8) mbar_arrive(cx.bar(ScEmpty + sc_slot));
      }
    }
    // ---- the piece's partial result: O / l and its LSE
    if (!wait_pv()) return;
    tc_fence_after();
    if (mine) {
      const size_t at = ((size_t)(pair + s.tile[q.g] + q.i) * kPrefixTileSeqs + j) * kHeads + (row & 63);
      const float inv = 1.0f / l;
      float* dst = p.part_o + at * kHeadDim;
#pragma unroll 1
      for (int c = 0; c < kHeadDim; c += 32) {
        float o[32];
        tmem_ld32(tmem + lanes + kTmemO + c, o);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] *= inv;
#pragma unroll
        for (int k = 0; k < 32; k += 8) st_global_v8(dst + c + k, o + k);
      }
      p.part_lse[at] = (m + log2f(l)) * kLn2;
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(o_free);
  }
}

template <bool kFp8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    decode_prefix_tc_kernel(const __grid_constant__ PrefixParams p, const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ __align__(1024) uint8_t dyn_smem[];
  const uint32_t raw = smem_u32(dyn_smem);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = dyn_smem + (base - raw);
  PlanSmem& plan = *reinterpret_cast<PlanSmem*>(gbase + Smem<kFp8>::plan);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Smem<kFp8>::misc);
  int* abort_flag = reinterpret_cast<int*>(gbase + Smem<kFp8>::misc + 4);
  const int warp = threadIdx.x >> 5;
  Ctx cx{base, base + Smem<kFp8>::bars, cta_rank(), abort_flag, p.err, p.wait_budget_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBars; ++i) {
      const bool of_pair = i == PFull || i == PFull + 1 || i == OFree || i == QReady;
      mbar_init(cx.bar(i), of_pair ? 2 * kSoftmaxWarps : i >= ScEmpty ? kSoftmaxWarps : 1);
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
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + Smem<kFp8>::misc),
                 "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  build_plan(p, plan, reinterpret_cast<int32_t*>(gbase + Smem<kFp8>::ring), blockIdx.x == 0 ? p.err : nullptr);
  publish_plan(p, plan);
  cluster_sync();  // the other CTA's barriers are initialised, its scratch is done with
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int units = plan.cost[p.n_groups], W = busy_pairs(p, units), pair = blockIdx.x >> 1;
  const long long lo = pair < W ? cta_cost_lo(pair, units, W) : 0, hi = pair < W ? cta_cost_lo(pair + 1, units, W) : 0;

  if (warp < kSoftmaxWarps) {
    softmax_role<kFp8>(p, cx, plan, lo, hi, tmem, pair, gbase);
  } else if (warp == kProducerWarp) {
    producer_role<kFp8>(p, &kmap, &vmap, &qmap, cx, plan, lo, hi);
  } else if (cx.rank == 0 && (threadIdx.x & 31) == 0) {
    mma_role<kFp8>(p, cx, plan, lo, hi, tmem);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // no copy, MMA or arrival for either CTA is left
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
}

}  // namespace

namespace {
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
