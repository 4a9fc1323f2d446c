// kv_read.cu -- positions of a paged cache read back as bf16 rows: a request
// that moves to another server or into a cache of another format, or whose
// values a caller wants as the attention sees them,
//     out[row_starts[b] + i] = bf16(decode(code) * scale),  position first[b] + i.
//
// Bound by memory (1024, 520 or 264 B in and 1024 B out a token), for few rows by
// a chain of three trips to L2: starts, page id, rows. 201 rows take 2.3 us, 58,778
// from E4M3 17.2 us, 65,111 from E2M1 16.8 us: what is written bounds these, a fill
// of 63 MB alone takes 16.4 us, and without the conversions they take as long.
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "mfa_device.cuh"
#include "mfa_serving.hpp"

namespace mfa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
  const __nv_bfloat162 h = __float22bfloat162_rn(v);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two codes to fp32, times the scale, to bf16: the product of the code's few bits and the scale's 24 is rounded to fp32
// first, which moves the bf16 result only where that rounding lands between two of its values.
__device__ __forceinline__ uint32_t scaled(const __half2_raw& codes, float s) {
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&codes));
  return pack_bf16(make_float2(v.x * s, v.y * s));
}
__device__ __forceinline__ uint32_t from_e4m3(uint32_t two, float s) {
  return scaled(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3), s);
}
__device__ __forceinline__ uint32_t from_e2m1(uint32_t two, float s) {
  return scaled(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)two, __NV_E2M1), s);
}

// A warp takes kRows rows, their K and their V; lane i has elements [8 i, 8 i + 8) of each.
template <int kFmt, int kRows>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadParams p) {
  __shared__ int s_start[kMaxBatch + 1];
  const int lane = threadIdx.x & 31;
  const long long r0 = ((long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kRows;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  for (int b = threadIdx.x; b <= p.B; b += kThreads) s_start[b] = __ldcg(p.row_starts + b);
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.B; b += kThreads)
      if (s_start[b] < 0 || s_start[b + 1] < s_start[b] || s_start[b + 1] > p.max_rows) raise_error(p.err, MFA_DEVERR_CAPACITY);
  const long long cap = (long long)p.max_pages * kPageSize;
  // lane j looks row r0 + j up: its slot, or -1
  long long slot = -1;
  if (lane < kRows && r0 + lane < p.max_rows && r0 + lane >= s_start[0] && r0 + lane < s_start[p.B]) {
    const int r = (int)(r0 + lane);
    int lo = 0, hi = p.B - 1;  // the last sequence that begins at or before r: those behind it with no rows begin later
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_start[mid] <= r) lo = mid; else hi = mid - 1;
    }
    const long long pos = (long long)r - s_start[lo] + (p.first ? __ldcg(p.first + lo) : 0);
    if (pos < 0 || pos >= cap) {
      raise_error(p.err, MFA_DEVERR_CAPACITY);
    } else {
      const int page = __ldcg(p.page_table + (size_t)lo * p.max_pages + pos / kPageSize);
      if (page < 0 || page >= p.num_pages) raise_error(p.err, MFA_DEVERR_PAGE);
      else slot = (long long)page * kPageSize + pos % kPageSize;
    }
  }
  constexpr int kBytes = kFmt == kKvBf16 ? 16 : kFmt == kKvE4M3 ? 8 : 4;  // of a lane
  using Word = std::conditional_t<kFmt == kKvBf16, uint4, std::conditional_t<kFmt == kKvE4M3, uint2, uint32_t>>;
  static_assert(sizeof(Word) == kBytes, "a lane's codes");
  Word w[2 * kRows];
  float s[2 * kRows];
  long long at[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    at[j] = __shfl_sync(0xffffffffu, slot, j);
    if (at[j] < 0) continue;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      w[2 * j + v] = __ldcg(reinterpret_cast<const Word*>(v ? p.v_cache : p.k_cache) + at[j] * 32 + lane);
      if (kFmt != kKvBf16) s[2 * j + v] = __ldcg((v ? p.v_scale : p.k_scale) + at[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    if (at[j] < 0) continue;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      uint16_t* row = (v ? p.v_out + (r0 + j) * p.v_stride : p.k_out + (r0 + j) * p.k_stride);
      uint4 y;
      if constexpr (kFmt == kKvBf16) {
        y = w[2 * j + v];
      } else if constexpr (kFmt == kKvE4M3) {
        const uint2 c = w[2 * j + v];
        const float z = s[2 * j + v];
        y = make_uint4(from_e4m3(c.x & 0xFFFFu, z), from_e4m3(c.x >> 16, z), from_e4m3(c.y & 0xFFFFu, z), from_e4m3(c.y >> 16, z));
      } else {
        const uint32_t c = w[2 * j + v];
        const float z = s[2 * j + v];
        y = make_uint4(from_e2m1(c & 0xFFu, z), from_e2m1((c >> 8) & 0xFFu, z), from_e2m1((c >> 16) & 0xFFu, z), from_e2m1(c >> 24, z));
      }
      reinterpret_cast<uint4*>(row)[lane] = y;
    }
  }
}

template <int kFmt, int kRows>
cudaError_t launch_rows(const KvReadParams& p, cudaStream_t stream) {
  constexpr int kPerBlock = kThreads / 32 * kRows;
  return launch_pdl(kv_read_kernel<kFmt, kRows>, dim3(((unsigned)p.max_rows + kPerBlock - 1) / kPerBlock), dim3(kThreads), 0,
                    stream, p);
}
template <int kFmt>
cudaError_t launch_fmt(const KvReadParams& p, cudaStream_t stream) {
  // Four rows a warp of many: 58,778 from E4M3 in 17.2 us, with two or eight 17.5 and 17.8, and 17.5 with blocks that stay and
  // look their next rows' pages up meanwhile. One of few, whose trips to L2 are what counts.
  constexpr int kManyRows = 8192;
  return p.max_rows < kManyRows ? launch_rows<kFmt, 1>(p, stream) : launch_rows<kFmt, 4>(p, stream);
}

}  // namespace

cudaError_t launch_kv_read(const KvReadParams& p, cudaStream_t stream) {
  return p.fmt == kKvBf16   ? launch_fmt<kKvBf16>(p, stream)
         : p.fmt == kKvE4M3 ? launch_fmt<kKvE4M3>(p, stream)
                            : launch_fmt<kKvE2M1>(p, stream);
}

}  // namespace mfa
