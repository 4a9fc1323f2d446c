// page_tables.cu -- the bookkeeping of a paged cache on the GPU: pages taken
// from and given back to a device-owned stack of free page ids, the page
// tables of the requests, and the slot of every token that arrives.
//
// With h_b = ceil(L_b / 64) the pages request b holds and a_b = ceil((L_b +
// n_b) / 64) those it needs, one exclusive prefix sum over the requests gives
//     start_b = sum_{c<b} n_c          (first token of b in the step's rows)
//     take_b  = sum_{c<b} (a_c - h_c)  (pages taken before b)
// and every output follows from them without a further dependence: page h_b + i
// of b is the free page at stack position n_free - 1 - (take_b + i), and token
// t of b sits at position L_b + t, i.e. row (L_b + t) % 64 of page
// (L_b + t) / 64. Releasing is the same sum over the pages given back.
//
// Split: the sums over at most 1024 requests take well under a microsecond of a
// CTA's time, less than a second launch or a grid-wide wait would, so every
// CTA forms them itself and then works on its share of the tokens and pages.
// The calls are bound by latency (launch, two dependent loads, the sums): 3.2 us
// for 128 requests with a token each, 5.4 us for 1000 requests with 250,000
// tokens (2 MB), 3.4 us for the release of 63 of 1000 requests. With outputs that
// replace inputs the arrival of all CTAs adds 0.8 us where there are many.
#include "mfa_device.cuh"
#include "mfa_serving.hpp"

namespace mfa {
namespace {

constexpr int kTableThreads = 1024;  // a thread a request
constexpr int kTableWarps = kTableThreads / 32;
static_assert(kTableThreads >= kMaxBatch && kTableWarps == 32, "the sums take one round, and one warp the warps' sums");

struct Pair {
  uint32_t a, b;
};
// Sums that stop at 2^31 - 1 instead of wrapping: the counts are the caller's. Where a sum matters it is exact, because
// it is compared with a bound below that first.
__device__ __forceinline__ uint32_t add_sat(uint32_t x, uint32_t y) { return min(x + y, 0x7fffffffu); }

// Sums up to and including this thread's values, and before them, in thread order, by the whole block.
struct Sums {
  Pair before, upto;
};
__device__ __forceinline__ Sums block_scan(Pair own, Pair* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [lane](Pair x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t ya = __shfl_up_sync(0xffffffffu, x.a, o), yb = __shfl_up_sync(0xffffffffu, x.b, o);
      if (lane >= o) x = Pair{add_sat(x.a, ya), add_sat(x.b, yb)};
    }
    return x;
  };
  Pair x = scan(own);
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  const Pair warps = scan(s_warp[lane]);  // every warp for itself
  Pair base{__shfl_sync(0xffffffffu, warps.a, max(warp - 1, 0)), __shfl_sync(0xffffffffu, warps.b, max(warp - 1, 0))};
  if (warp == 0) base = Pair{0, 0};
  Pair prev{__shfl_up_sync(0xffffffffu, x.a, 1), __shfl_up_sync(0xffffffffu, x.b, 1)};
  if (lane == 0) prev = Pair{0, 0};
  return Sums{{add_sat(base.a, prev.a), add_sat(base.b, prev.b)}, {add_sat(base.a, x.a), add_sat(base.b, x.b)}};
}

// First b with upto[b] > i (upto is non-decreasing); B if there is none.
__device__ __forceinline__ int first_above(const int* upto, int B, int i) {
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (upto[mid] > i) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// True in the one block that arrives last: every other block of the grid has
// read its inputs by then, so outputs that replace inputs may be written. The
// counter wraps to zero for the next call.
__device__ __forceinline__ bool last_block(uint32_t* counter) {
  __shared__ int s_last;
  if (gridDim.x == 1) return true;  // (its threads have met since they read)
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicInc(counter, gridDim.x - 1) == gridDim.x - 1;
  }
  __syncthreads();
  return s_last;
}

// Pages of len + more tokens.
__device__ __forceinline__ int pages_held(int len, int more) {
  return (int)(((long long)len + more + kPageSize - 1) / kPageSize);
}

__device__ __forceinline__ int checked_count(int n, int most, uint32_t* err) {
  if (n >= 0 && n <= most) return n;
  raise_error(err, MFA_DEVERR_CAPACITY);
  return n < 0 ? 0 : most;
}

__global__ void __launch_bounds__(kTableThreads) reserve_pages_kernel(const PageTableParams p) {
  __shared__ Pair s_warp[kTableWarps];
  __shared__ int s_upto[kMaxBatch];  // tokens up to and including request b
  __shared__ int s_page[kMaxBatch];  // pages up to and including request b
  __shared__ int s_len[kMaxBatch];
  __shared__ int s_take[kMaxBatch];  // pages taken before request b, -1: not served
  __shared__ int s_taken;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const bool first = blockIdx.x == 0;  // device faults are reported once
  uint32_t* err = first ? p.err : nullptr;
  const int b = threadIdx.x;  // this thread's request
  const int free_raw = __ldcg(p.n_free);
  const int n = b < p.B ? __ldcg(p.n_new + b) : 0, len = b < p.B ? __ldcg(p.seq_lens + b) : 0;
  if (b == 0) s_taken = 0;
  const int n_free = checked_count(free_raw, p.num_pages, err);
  // One pass of sums for tokens and pages: which requests fit the step's rows depends on the tokens before them, but those
  // that do not are the last ones, and no request's pages depend on a later one.
  const bool good = n >= 0 && len >= 0 && (long long)len + n <= (long long)p.max_pages * kPageSize;
  const uint32_t need = good ? (uint32_t)(pages_held(len, n) - pages_held(len, 0)) : 0u;
  const Sums sums = block_scan(Pair{(uint32_t)max(n, 0), need}, s_warp);
  const bool fits = sums.upto.a <= (uint32_t)p.max_new;
  const bool served = good && fits && (need == 0 || sums.upto.b <= (uint32_t)n_free);
  const uint32_t most = __reduce_max_sync(0xffffffffu, b < p.B && served && need > 0 ? sums.upto.b : 0u);
  if ((b & 31) == 0) atomicMax(&s_taken, (int)most);
  if (b < p.B) {
    if (!good || !fits) raise_error(err, MFA_DEVERR_CAPACITY);
    if (good && fits && !served) raise_error(err, MFA_DEVERR_NO_PAGES);
    s_len[b] = len;
    s_upto[b] = (int)sums.upto.a;
    s_page[b] = (int)min(sums.upto.b, (uint32_t)n_free);  // behind the last served request only its order matters
    s_take[b] = served ? (int)min(sums.before.b, (uint32_t)n_free) : -1;
  }
  __syncthreads();
  const int taken = s_taken;
  const uint32_t t0 = blockIdx.x * kTableThreads + threadIdx.x, step = gridDim.x * kTableThreads;  // sums stay below 2^32
  // the new entries of the page tables
  for (uint32_t u = t0; u < (uint32_t)taken; u += step) {
    const int i = (int)u, b = first_above(s_page, p.B, i);
    const int held = pages_held(s_len[b], 0);
    const int page = __ldcg(p.free_pages + (n_free - 1 - i));
    if (page < 0 || page >= p.num_pages) raise_error(p.err, MFA_DEVERR_PAGE);
    p.page_table[(size_t)b * p.max_pages + held + (i - s_take[b])] = page;
  }
  // the slots of the tokens; -1 for tokens that are not served and past the last one
  for (uint32_t u = t0; u < (uint32_t)p.max_new; u += step) {
    const int i = (int)u, b = first_above(s_upto, p.B, i);
    long long slot = -1;
    if (b < p.B && s_take[b] >= 0) {
      const int pos = s_len[b] + i - (b ? s_upto[b - 1] : 0);
      const int held = pages_held(s_len[b], 0), pg = pos / kPageSize;
      // a page held before the call stands in the table, a new one is read where the table's entry comes from
      const int page = pg < held ? __ldcg(p.page_table + (size_t)b * p.max_pages + pg)
                                 : __ldcg(p.free_pages + (n_free - 1 - (s_take[b] + pg - held)));
      if (page >= 0 && page < p.num_pages)
        slot = (long long)page * kPageSize + pos % kPageSize;
      else
        raise_error(p.err, MFA_DEVERR_PAGE);
    }
    p.slot_map[u] = slot;
  }
  if (first && b < p.B) p.new_starts[b + 1] = s_upto[b];
  if (first && b == 0) p.new_starts[0] = 0;
  if (p.in_place ? last_block(p.counter) : first) {
    if (b < p.B) p.seq_lens_out[b] = s_take[b] >= 0 ? len + n : len;
    if (b == 0) *p.n_free_out = n_free - taken;
  }
}

__global__ void __launch_bounds__(kTableThreads) release_pages_kernel(const PageTableParams p) {
  __shared__ Pair s_warp[kTableWarps];
  __shared__ int s_upto[kMaxBatch];  // pages given back up to and including request b
  __shared__ int s_kept[kMaxBatch];  // pages request b keeps at the start of its row, -1: it is left as it is
  __shared__ int s_total;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const bool first = blockIdx.x == 0;
  uint32_t* err = first ? p.err : nullptr;
  const long long cap = (long long)p.max_pages * kPageSize;
  const int b = threadIdx.x;  // this thread's request
  const int free_raw = __ldcg(p.n_free);
  const int len = b < p.B ? __ldcg(p.seq_lens + b) : 0;
  const bool ended = b < p.B && __ldcg(p.finished + b) != 0;
  const int keep = ended && p.keep_pages ? __ldcg(p.keep_pages + b) : 0;
  if (b == 0) s_total = 0;
  const int n_free = checked_count(free_raw, p.num_pages, err);
  const bool good = ended && len >= 0 && len <= cap && keep >= 0;
  if (ended && !good) raise_error(err, MFA_DEVERR_CAPACITY);
  const int held = good ? pages_held(len, 0) : 0;
  int kept = good ? min(keep, held) : -1;
  const uint32_t count = good ? (uint32_t)(held - kept) : 0u, room = (uint32_t)(p.num_pages - n_free);
  const Sums sums = block_scan(Pair{count, 0u}, s_warp);
  const bool fits = count == 0 || sums.upto.a <= room;
  const uint32_t most = __reduce_max_sync(0xffffffffu, fits && count > 0 ? sums.upto.a : 0u);
  if ((b & 31) == 0) atomicMax(&s_total, (int)most);
  if (b < p.B) {
    if (!fits) {
      raise_error(err, MFA_DEVERR_CAPACITY);
      kept = -1;
    }
    s_kept[b] = kept;
    s_upto[b] = (int)min(sums.upto.a, room);
  }
  __syncthreads();
  const int total = s_total;
  for (uint32_t u = blockIdx.x * kTableThreads + threadIdx.x; u < (uint32_t)total; u += gridDim.x * kTableThreads) {
    const int i = (int)u, b = first_above(s_upto, p.B, i);
    const int page = __ldcg(p.page_table + (size_t)b * p.max_pages + s_kept[b] + (i - (b ? s_upto[b - 1] : 0)));
    if (page < 0 || page >= p.num_pages) raise_error(p.err, MFA_DEVERR_PAGE);
    p.free_pages[n_free + i] = page;
  }
  if (p.in_place ? last_block(p.counter) : first) {
    if (b < p.B) p.seq_lens_out[b] = kept >= 0 ? (int)min((long long)len, (long long)kept * kPageSize) : len;
    if (b == 0) *p.n_free_out = n_free + total;
  }
}

// A thread a token or table entry, up to one CTA per SM (beyond that every CTA would repeat the sums over the requests
// only to wait for an SM).
int table_grid(long long items) {
  constexpr long long kItemsPerCta = kTableThreads, kMostCtas = 152;
  const long long g = (items + kItemsPerCta - 1) / kItemsPerCta;
  return (int)(g < 1 ? 1 : g > kMostCtas ? kMostCtas : g);
}

}  // namespace

cudaError_t launch_reserve_pages(const PageTableParams& p, cudaStream_t stream) {
  return launch_pdl(reserve_pages_kernel, dim3(table_grid(p.max_new)), dim3(kTableThreads), 0, stream, p);
}

cudaError_t launch_release_pages(const PageTableParams& p, cudaStream_t stream) {
  return launch_pdl(release_pages_kernel, dim3(table_grid((long long)p.B * p.max_pages)), dim3(kTableThreads), 0, stream, p);
}

}  // namespace mfa
