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
// The calls are bound by latency (launch, two dependent loads, the sums): the
// step of 1000 requests with 250,000 tokens moves 2 MB.
#include "mfa_device.cuh"

namespace mfa {
namespace {

constexpr int kTableThreads = 512;
constexpr int kTableWarps = kTableThreads / 32;

struct Pair {
  long long a, b;
};

// Exclusive prefix sums of two values per request, in request order, by the
// whole block: f(b) gives the values of request b, g(b, before, own) receives
// the sums before it. Returns the totals. Sums are 64-bit: the lengths are the
// caller's and 1024 of them may pass 32 bits.
template <typename F, typename G>
__device__ __forceinline__ Pair block_scan(int B, Pair* s_warp, F f, G g) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Pair base{0, 0};
  for (int b0 = 0; b0 < B; b0 += kTableThreads) {
    const int b = b0 + (int)threadIdx.x;
    Pair own{0, 0};
    if (b < B) own = f(b);
    Pair x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long ya = __shfl_up_sync(0xffffffffu, x.a, o), yb = __shfl_up_sync(0xffffffffu, x.b, o);
      if (lane >= o) {
        x.a += ya;
        x.b += yb;
      }
    }
    __syncthreads();  // the previous round's warp sums have been read
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    Pair before = base;
    for (int w = 0; w < kTableWarps; ++w) {
      const Pair y = s_warp[w];
      if (w < warp) {
        before.a += y.a;
        before.b += y.b;
      }
      base.a += y.a;
      base.b += y.b;
    }
    if (b < B) g(b, Pair{before.a + x.a - own.a, before.b + x.b - own.b}, own);
  }
  return base;
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
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = gridDim.x == 1 || atomicInc(counter, gridDim.x - 1) == gridDim.x - 1;
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
  const long long cap = (long long)p.max_pages * kPageSize;
  const int free_raw = __ldcg(p.n_free);
  for (int b = threadIdx.x; b < p.B; b += kTableThreads) {
    s_take[b] = __ldcg(p.n_new + b);
    s_len[b] = __ldcg(p.seq_lens + b);
  }
  if (threadIdx.x == 0) s_taken = 0;
  const int n_free = checked_count(free_raw, p.num_pages, err);
  // One pass for tokens and pages: which requests fit the step's rows depends on the tokens before them, but those that
  // do not are the last ones, and no request's pages depend on a later one.
  block_scan(
      p.B, s_warp,
      [&](int b) {
        const int n = s_take[b], len = s_len[b];
        const bool good = n >= 0 && len >= 0 && (long long)len + n <= cap;
        if (!good) raise_error(err, MFA_DEVERR_CAPACITY);
        return Pair{n < 0 ? 0 : n, good ? pages_held(len, n) - pages_held(len, 0) : 0};
      },
      [&](int b, Pair before, Pair own) {
        const int n = s_take[b], len = s_len[b];
        const long long end = before.a + own.a, pages = before.b + own.b;
        const bool good = n >= 0 && len >= 0 && (long long)len + n <= cap, fits = end <= p.max_new;
        if (good && !fits) raise_error(err, MFA_DEVERR_CAPACITY);
        const bool served = good && fits && (own.b == 0 || pages <= n_free);
        if (good && fits && !served) raise_error(err, MFA_DEVERR_NO_PAGES);
        s_upto[b] = (int)min(end, 0x7fffffffLL);
        s_page[b] = (int)min(pages, (long long)n_free);  // behind the last served request only its order matters
        s_take[b] = served ? (int)min(before.b, (long long)n_free) : -1;
        if (served && own.b > 0) atomicMax(&s_taken, (int)pages);
      });
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
  // the slots of the tokens; -1 for tokens that are not served and past the last one. kAtOnce tokens a thread: their
  // searches and page loads overlap.
  constexpr int kAtOnce = 4;
  for (uint32_t u0 = t0; u0 < (uint32_t)p.max_new; u0 += kAtOnce * step) {
    int page[kAtOnce], row[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const uint32_t u = u0 + k * step;
      const int i = (int)u, b = u < (uint32_t)p.max_new ? first_above(s_upto, p.B, i) : p.B;
      row[k] = -1;
      page[k] = 0;
      if (b < p.B && s_take[b] >= 0) {
        const int pos = s_len[b] + i - (b ? s_upto[b - 1] : 0);
        const int held = pages_held(s_len[b], 0), pg = pos / kPageSize;
        row[k] = pos % kPageSize;
        // a page held before the call stands in the table, a new one is read where the table's entry comes from
        page[k] = pg < held ? __ldcg(p.page_table + (size_t)b * p.max_pages + pg)
                            : __ldcg(p.free_pages + (n_free - 1 - (s_take[b] + pg - held)));
      }
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const uint32_t u = u0 + k * step;
      if (u >= (uint32_t)p.max_new) break;
      const bool good = page[k] >= 0 && page[k] < p.num_pages;
      if (!good) raise_error(p.err, MFA_DEVERR_PAGE);
      p.slot_map[u] = row[k] >= 0 && good ? (long long)page[k] * kPageSize + row[k] : -1;
    }
  }
  if (first)
    for (int b = threadIdx.x; b <= p.B; b += kTableThreads) p.new_starts[b] = b ? s_upto[b - 1] : 0;
  if (last_block(p.counter)) {
    for (int b = threadIdx.x; b < p.B; b += kTableThreads)
      p.seq_lens_out[b] = s_take[b] >= 0 ? s_len[b] + s_upto[b] - (b ? s_upto[b - 1] : 0) : s_len[b];
    if (threadIdx.x == 0) *p.n_free_out = n_free - taken;
  }
}

__global__ void __launch_bounds__(kTableThreads) release_pages_kernel(const PageTableParams p) {
  __shared__ Pair s_warp[kTableWarps];
  __shared__ int s_upto[kMaxBatch];  // pages given back up to and including request b
  __shared__ int s_kept[kMaxBatch];  // pages request b keeps at the start of its row, -1: it is left as it is
  __shared__ int s_len[kMaxBatch];
  __shared__ int s_total;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  const bool first = blockIdx.x == 0;
  uint32_t* err = first ? p.err : nullptr;
  const long long cap = (long long)p.max_pages * kPageSize;
  const int free_raw = __ldcg(p.n_free);
  for (int b = threadIdx.x; b < p.B; b += kTableThreads) {
    s_len[b] = __ldcg(p.seq_lens + b);
    s_kept[b] = __ldcg(p.finished + b);
    s_upto[b] = p.keep_pages ? __ldcg(p.keep_pages + b) : 0;
  }
  if (threadIdx.x == 0) s_total = 0;
  const int n_free = checked_count(free_raw, p.num_pages, err);
  block_scan(
      p.B, s_warp,
      [&](int b) {
        const int len = s_len[b], keep = s_upto[b];
        int kept = -1, count = 0;
        if (s_kept[b] != 0) {
          if (len < 0 || len > cap || keep < 0) {
            raise_error(err, MFA_DEVERR_CAPACITY);
          } else {
            const int held = pages_held(len, 0);
            kept = min(keep, held);
            count = held - kept;
          }
        }
        s_kept[b] = kept;
        return Pair{count, 0};
      },
      [&](int b, Pair before, Pair own) {
        const long long upto = before.a + own.a, room = p.num_pages - n_free;
        if (own.a > 0 && upto > room) {
          raise_error(err, MFA_DEVERR_CAPACITY);
          s_kept[b] = -1;
        }
        s_upto[b] = (int)min(upto, room);
        if (own.a > 0 && upto <= room) atomicMax(&s_total, (int)upto);
      });
  __syncthreads();
  const int total = s_total;
  for (uint32_t u = blockIdx.x * kTableThreads + threadIdx.x; u < (uint32_t)total; u += gridDim.x * kTableThreads) {
    const int i = (int)u, b = first_above(s_upto, p.B, i);
    const int page = __ldcg(p.page_table + (size_t)b * p.max_pages + s_kept[b] + (i - (b ? s_upto[b - 1] : 0)));
    if (page < 0 || page >= p.num_pages) raise_error(p.err, MFA_DEVERR_PAGE);
    p.free_pages[n_free + i] = page;
  }
  if (last_block(p.counter)) {
    for (int b = threadIdx.x; b < p.B; b += kTableThreads)
      p.seq_lens_out[b] = s_kept[b] >= 0 ? (int)min((long long)s_len[b], (long long)s_kept[b] * kPageSize) : s_len[b];
    if (threadIdx.x == 0) *p.n_free_out = n_free + total;
  }
}

// One CTA per 2048 tokens or table entries, four a thread, at most one per SM:
// fewer items a CTA would repeat the sums over the requests for too little work.
int table_grid(long long items) {
  constexpr long long kItemsPerCta = 4 * kTableThreads, kMostCtas = 152;
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
