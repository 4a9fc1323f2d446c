// kv_append.cu -- in-place KV append into the paged cache (bf16 copy or
// per-token E4M3 or E2M1 quantisation), advancing the device-owned length
// counter.
//
// Semantics: "DuckLLM decode fixed-cost reduction" page, sections 7.2 (static
// KV cache written at a fixed slot, never re-materialised) and 7.6 (the append
// offset and the attention length come from one device-owned counter, and the
// attention after an append includes the new token). FP8 storage: "Step-3 is
// Large yet Affordable" (paper summary page), section 7 (8-bit KV, 512 bytes
// per token per layer); one fp32 scale per token (absmax / 448) because the
// pages do not fix the granularity. 4-bit storage: same page, section 5.2 (KV
// kept in 4 bits, attention computed in 8 bits), as OCP MX FP4 (E2M1) codes
// with one fp32 scale per token (absmax / 6), two codes per byte.
#include <algorithm>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "mfa_device.cuh"
#include "mfa_serving.hpp"

namespace mfa {
namespace {

constexpr int kAppendThreads = 256;  // 8 warps, one token row (K or V) per warp at a time

// Rows are 512 bytes of bf16: lane i holds elements [8i, 8i + 8).
// Quantise one bf16 row to E4M3 with scale = absmax / 448 (1 for a zero row).
// Divisions are IEEE round-to-nearest; the conversion rounds to nearest even
// and saturates to +-448.
__device__ __forceinline__ void quantise_row_e4m3(const uint4 raw, uint8_t* __restrict__ dst,
                                                  float* __restrict__ scale_out, int lane) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float s = (amax > 0.0f) ? __fdiv_rn(amax, 448.0f) : 1.0f;
  uint32_t packed[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 pr = make_float2(__fdiv_rn(x[4 * i + 2 * j], s), __fdiv_rn(x[4 * i + 2 * j + 1], s));
      const __nv_fp8x2_storage_t c2 = __nv_cvt_float2_to_fp8x2(pr, __NV_SATFINITE, __NV_E4M3);
      word |= (uint32_t)c2 << (16 * j);
    }
    packed[i] = word;
  }
  reinterpret_cast<uint2*>(dst)[lane] = make_uint2(packed[0], packed[1]);
  if (lane == 0) *scale_out = s;
}

// Nearest E2M1 code to y, a tie going to the code with mantissa bit 0, beyond 6
// saturating; the sign is kept (sign bit 3, also on zero). The candidate
// magnitudes are 0, 0.5, 1, 1.5, 2, 3, 4, 6: the comparisons are against the
// midpoints, each tie resolved toward the even code.
__device__ __forceinline__ uint32_t e2m1_code(float y) {
  const float a = fabsf(y);
  const uint32_t c = a <= 0.25f ? 0u : a < 0.75f ? 1u : a <= 1.25f ? 2u : a < 1.75f ? 3u
                   : a <= 2.5f ? 4u : a < 3.5f ? 5u : a <= 5.0f ? 6u : 7u;
  return c | (signbit(y) ? 8u : 0u);
}

// Quantise one bf16 row to E2M1 with scale = absmax / 6 (1 for a zero row):
// lane i packs elements [8i, 8i + 8) into 4 bytes, element 2k in the low nibble.
__device__ __forceinline__ void quantise_row_e2m1(const uint4 raw, uint8_t* __restrict__ dst,
                                                  float* __restrict__ scale_out, int lane) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float s = (amax > 0.0f) ? __fdiv_rn(amax, 6.0f) : 1.0f;
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) word |= e2m1_code(__fdiv_rn(x[i], s)) << (4 * i);
  reinterpret_cast<uint32_t*>(dst)[lane] = word;
  if (lane == 0) *scale_out = s;
}

constexpr int kMaxStagedPages = 64;  // page ids validated once and kept in shared memory

__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(AppendParams p) {
  __shared__ int s_start;
  __shared__ int s_bad;
  __shared__ int s_pages[kMaxStagedPages];
  const int b = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kWarps = kAppendThreads / 32;
  pdl_launch_dependents();  // the decode kernel may run its prologue meanwhile
  pdl_wait_prior_grid();    // launched early too: whatever ran before must be complete and visible
  // the row of this warp's first work item (token t = i / 2, K or V) is read
  // while warp 0 looks up and checks where the tokens go
  const int first = warp;
  uint4 first_row = make_uint4(0u, 0u, 0u, 0u);
  if (first < 2 * p.n_new) {
    const uint16_t* src = ((first & 1) ? p.v_new : p.k_new) + ((size_t)b * p.n_new + (first >> 1)) * kHeadDim;
    first_row = __ldcg(reinterpret_cast<const uint4*>(src) + lane);
  }
  if (warp == 0) {
    const int start = p.seq_lens[b];
    const long long cap = (long long)p.max_pages * kPageSize;
    bool bad_cap = start < 0 || (long long)start + p.n_new > cap;
    bool bad_page = false;
    if (!bad_cap) {
      // every page id the new tokens land in is checked before anything is written
      const int pg_first = start / kPageSize, pg_last = (start + p.n_new - 1) / kPageSize;
      for (int pg = pg_first + lane; pg <= pg_last; pg += 32) {
        const int page = p.page_table[(size_t)b * p.max_pages + pg];
        if (page < 0 || page >= p.num_pages) bad_page = true;
        if (pg - pg_first < kMaxStagedPages) s_pages[pg - pg_first] = page;
      }
      bad_page = __any_sync(0xffffffffu, bad_page);
    }
    if (lane == 0) {
      if (bad_cap) raise_error(p.err, MFA_DEVERR_CAPACITY);
      if (bad_page) raise_error(p.err, MFA_DEVERR_PAGE);
      s_bad = (bad_cap || bad_page) ? 1 : 0;
      s_start = start;
    }
  }
  __syncthreads();
  if (s_bad) return;
  const int start = s_start;
  const int pg_first = start / kPageSize;
  for (int i = warp; i < 2 * p.n_new; i += kWarps) {
    const int t = i >> 1;
    const bool is_v = i & 1;
    const int pos = start + t;
    const int pg = pos / kPageSize;
    const int page = (pg - pg_first < kMaxStagedPages) ? s_pages[pg - pg_first]
                                                        : p.page_table[(size_t)b * p.max_pages + pg];
    const size_t slot = (size_t)page * kPageSize + (pos % kPageSize);
    const uint16_t* src = (is_v ? p.v_new : p.k_new) + ((size_t)b * p.n_new + t) * kHeadDim;
    const uint4 row = (i == first) ? first_row : __ldcg(reinterpret_cast<const uint4*>(src) + lane);
    if (p.fmt == kKvE2M1) {
      uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + slot * (kHeadDim / 2);
      float* sc = (is_v ? p.v_scale : p.k_scale) + slot;
      quantise_row_e2m1(row, dst, sc, lane);
    } else if (p.fmt == kKvE4M3) {
      uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + slot * kHeadDim;
      float* sc = (is_v ? p.v_scale : p.k_scale) + slot;
      quantise_row_e4m3(row, dst, sc, lane);
    } else {
      uint16_t* dst = static_cast<uint16_t*>(is_v ? p.v_cache : p.k_cache) + slot * kHeadDim;
      reinterpret_cast<uint4*>(dst)[lane] = row;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) p.seq_lens[b] = start + p.n_new;
}

// Quotients x / s, two at a time, as IEEE division rounds them: Markstein's
// method (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990). With y the rounded reciprocal of s, q = x y is
// corrected by its exact remainder, q -= (q s - x) y. For any s that takes two
// such steps; for the scales of a row, absmax / 6 or / 448 rounded, and its bf16
// values one gives the rounded quotient (tests/test_quantiser_host.py goes through
// all of their mantissas). The remainders are exact while nothing underflows, which
// s in [2^-60, 2^60] and quotients above 2^-10 (smaller ones are code 0 whatever
// their last bits) ensure. Written in -x and -y, which also keeps the sign of a
// zero. With divisions the call took 33.6 us for 65,000 tokens to E4M3.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
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
__device__ __forceinline__ float2 unpack_bf16x2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// quantise_row_e4m3 and quantise_row_e2m1, with the same codes and scales, by kLanes lanes: lane l has elements 8 l to 8 l + 7, and
// of 16 lanes those 128 further on. An E2M1 code is the conversion's (nearest, a tie to the even code, beyond 6 saturating, NaN
// to 6).
template <bool kFp4, int kLanes>
__device__ __forceinline__ void quantise_row_slots(const uint4 (&raw)[32 / kLanes], uint8_t* __restrict__ dst,
                                                   float* __restrict__ scale_out, int l) {
  constexpr int kPairs = 4 * (32 / kLanes);
  uint32_t w[kPairs];
#pragma unroll
  for (int h = 0; h < 32 / kLanes; ++h) {
    w[4 * h] = raw[h].x;
    w[4 * h + 1] = raw[h].y;
    w[4 * h + 2] = raw[h].z;
    w[4 * h + 3] = raw[h].w;
  }
  // the largest magnitude, a NaN left out of it as by fmaxf
  const __nv_bfloat162* pairs = reinterpret_cast<const __nv_bfloat162*>(w);
  __nv_bfloat162 top = __habs2(pairs[0]);
#pragma unroll
  for (int i = 1; i < kPairs; ++i) top = __hmax2(top, __habs2(pairs[i]));
  const float2 both = unpack_bf16x2(*reinterpret_cast<const uint32_t*>(&top));
  float amax = fmaxf(fmaxf(both.x, both.y), 0.0f);
  if constexpr (kLanes == 32) {
    // not negative (and of NaN alone 0): ordered as integers
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  } else {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  }
  // absmax over 6 or 448 in the same way, 1 / 6 and 1 / 448 being known (bf16's 128 mantissas are in that test too)
  constexpr float kMost = kFp4 ? 6.0f : 448.0f, kInverse = 1.0f / kMost;
  const float q0 = amax * kInverse;
  float s = fmaf(fmaf(-kMost, q0, amax), kInverse, q0);
  if (!(amax >= 0x1p-100f && amax <= 0x1p100f)) s = (amax > 0.0f) ? __fdiv_rn(amax, kMost) : 1.0f;
  auto convert = [](float2 q) -> uint32_t {
    if constexpr (kFp4) return __nv_cvt_float2_to_fp4x2(q, __NV_E2M1, cudaRoundNearest);
    else return __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
  };
  uint32_t code[kPairs];
  if (s >= 0x1p-60f && s <= 0x1p60f) {
    const float y = -__frcp_rn(s);
    const float2 minus_y = make_float2(y, y), ss = make_float2(s, s);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const float2 minus_x = unpack_bf16x2(w[i] ^ 0x80008000u);
      const float2 q = mul2(minus_x, minus_y);
      code[i] = convert(fma2(fma2(ss, q, minus_x), minus_y, q));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const float2 x = unpack_bf16x2(w[i]);
      code[i] = convert(make_float2(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s)));
    }
  }
#pragma unroll
  for (int h = 0; h < 32 / kLanes; ++h) {
    const uint32_t* c = code + 4 * h;
    if constexpr (kFp4)
      reinterpret_cast<uint32_t*>(dst)[kLanes * h + l] = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
    else
      reinterpret_cast<uint2*>(dst)[kLanes * h + l] = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  }
  if (l == 0) *scale_out = s;
}

// Rows scattered to the slots of a slot map. No row depends on another, so the
// call is bound by latency for a decode step's rows and by memory bandwidth for a
// prefill's (read 1 KB, write 1 KB, 520 or 264 B a token): 128 rows 1.2 us, 16384
// rows 3.7 us (9 TB/s, L2 among it), 65536 rows to E4M3 17.5 us (5.8
// TB/s), to E2M1 16.0 us (5.3 TB/s).
constexpr int kSlotThreads = 256;
// bf16: a warp a row of K or of V, kRows such items a warp, all of whose loads are in flight before the first store.
template <int kRows>
__global__ void __launch_bounds__(kSlotThreads) kv_append_slots_kernel(const AppendSlotsParams p) {
  const int lane = threadIdx.x & 31;
  const long long items = 2ll * p.n_rows;  // item i: row i / 2, K (even) or V (odd)
  const long long i0 = ((long long)blockIdx.x * (kSlotThreads / 32) + (threadIdx.x >> 5)) * kRows;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  uint4 row[kRows];
  long long slot[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const long long i = i0 + j, r = i >> 1;
    slot[j] = -1;
    if (i < items) {
      slot[j] = __ldcg(reinterpret_cast<const long long*>(p.slot_map) + r);
      const uint16_t* src = (i & 1) ? p.v_new + r * p.v_stride : p.k_new + r * p.k_stride;
      row[j] = __ldcg(reinterpret_cast<const uint4*>(src) + lane);
    }
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    if (slot[j] < 0) continue;  // a padded row
    if (slot[j] >= (long long)p.num_pages * kPageSize) {
      if (lane == 0) raise_error(p.err, MFA_DEVERR_PAGE);
      continue;
    }
    uint16_t* dst = static_cast<uint16_t*>((i0 + j) & 1 ? p.v_cache : p.k_cache) + slot[j] * kHeadDim;
    reinterpret_cast<uint4*>(dst)[lane] = row[j];
  }
}
template <bool kFp4>
__device__ __forceinline__ constexpr int code_row_bytes() { return kFp4 ? kHeadDim / 2 : kHeadDim; }
// Quantised: kLanes lanes a row of K or of V. With half a warp, what there is to do for a row (its maximum, its scale and the
// scale's reciprocal) takes half the instructions; the halves of a warp then take K and V of one row.
template <bool kFp4, int kLanes>
__global__ void __launch_bounds__(kSlotThreads) kv_append_slots_quantised_kernel(const AppendSlotsParams p) {
  const int l = threadIdx.x & (kLanes - 1);
  const long long item = (long long)blockIdx.x * (kSlotThreads / kLanes) + threadIdx.x / kLanes, r = item >> 1;
  const bool is_v = item & 1;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  uint4 row[32 / kLanes] = {};
  long long slot = -1;
  if (r < p.n_rows) {
    slot = __ldcg(reinterpret_cast<const long long*>(p.slot_map) + r);
    const uint4* src = reinterpret_cast<const uint4*>(is_v ? p.v_new + r * p.v_stride : p.k_new + r * p.k_stride);
#pragma unroll
    for (int h = 0; h < 32 / kLanes; ++h) row[h] = __ldcg(src + kLanes * h + l);
  }
  if (slot >= (long long)p.num_pages * kPageSize) {
    if (l == 0) raise_error(p.err, MFA_DEVERR_PAGE);
    slot = -1;
  }
  if (slot < 0) return;  // a padded row, of the warp's K and V alike
  quantise_row_slots<kFp4, kLanes>(row, static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + slot * code_row_bytes<kFp4>(),
                                   (is_v ? p.v_scale : p.k_scale) + slot, l);
}
// The same with half a warp a row for very many rows: the blocks that are there at once go through all of them, each warp with
// its next row's loads in flight while it works on one. With a block for every 8 rows the memory waits for that work. Five
// blocks an SM: with three, four and six, 65536 rows to E2M1 took 19.9, 16.5 and 18.9 us instead of 16.0.
constexpr int kStreamBlocksPerSm = 5, kStreamRows = kSlotThreads / 32;
template <bool kFp4>
__global__ void __launch_bounds__(kSlotThreads, kStreamBlocksPerSm) kv_append_slots_stream_kernel(const AppendSlotsParams p) {
  constexpr int kLanes = 16;
  const int l = threadIdx.x & (kLanes - 1);
  const bool is_v = threadIdx.x & kLanes;
  const uint32_t rows = p.n_rows, step = gridDim.x * kStreamRows;
  uint32_t r = blockIdx.x * kStreamRows + threadIdx.x / 32;
  uint8_t* cache = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache);
  float* scales = is_v ? p.v_scale : p.k_scale;
  const long long end = (long long)p.num_pages * kPageSize, stride = (is_v ? p.v_stride : p.k_stride) / 8;  // in uint4
  const uint4* src = reinterpret_cast<const uint4*>(is_v ? p.v_new : p.k_new) + r * stride + l;
  const long long* at = reinterpret_cast<const long long*>(p.slot_map) + r;
  pdl_launch_dependents();
  pdl_wait_prior_grid();
  if (r >= rows) return;
  uint4 next[2] = {__ldcg(src), __ldcg(src + kLanes)};
  long long next_slot = __ldcg(at);
#pragma unroll 1
  for (bool more = true; more;) {  // (of the warp)
    const uint4 row[2] = {next[0], next[1]};
    const long long slot = next_slot;
    more = rows - r > step;
    if (more) {
      r += step;
      src += step * stride;
      at += step;
      next[0] = __ldcg(src);
      next[1] = __ldcg(src + kLanes);
      next_slot = __ldcg(at);
    }
    if (slot >= end) {
      if (l == 0) raise_error(p.err, MFA_DEVERR_PAGE);
    } else if (slot >= 0) {  // else a padded row
      quantise_row_slots<kFp4, kLanes>(row, cache + slot * code_row_bytes<kFp4>(), scales + slot, l);
    }
  }
}

unsigned slot_blocks(long long warps) { return (unsigned)((warps + kSlotThreads / 32 - 1) / (kSlotThreads / 32)); }
template <int kRows>
cudaError_t launch_slots(const AppendSlotsParams& p, cudaStream_t stream) {
  const unsigned blocks = slot_blocks((2ll * p.n_rows + kRows - 1) / kRows);
  return launch_pdl(kv_append_slots_kernel<kRows>, dim3(blocks), dim3(kSlotThreads), 0, stream, p);
}
template <bool kFp4>
cudaError_t launch_slots_quantised(const AppendSlotsParams& p, cudaStream_t stream) {
  // a warp a row, half a warp, and with the loop, E4M3: 128 rows 1.55, 1.75 and 1.6 us, 4096 rows 2.7, 2.6 and 2.6, 8192 rows
  // 3.9, 3.1 and 3.4. Half a warp and the loop, replayed on the same rows, part of which L2 then holds: 8192 rows 2.8 and 3.1
  // (E2M1 3.0 and 3.3), 12160 rows 3.51 and 3.54 (3.72 and 3.77), 16384 rows 4.24 and 4.24 (4.56 and 4.55), 24320 rows 5.8 and
  // 5.8 (6.27 and 6.13), 65536 rows 15.7 and 14.6 (15.5 and 14.7), 200000 rows 48.2 and 46.7 (48.0 and 43.4). The loop gains at
  // 4096 to 6080 rows too, 0.1 to 0.4 us, where all rows are in its first turn, and loses where few are in its second.
  constexpr int kManyRows = 2048, kVeryManyRows = 16384;
  if (p.n_rows < kManyRows)
    return launch_pdl(kv_append_slots_quantised_kernel<kFp4, 32>, dim3(slot_blocks(2ll * p.n_rows)), dim3(kSlotThreads), 0, stream, p);
  if (p.n_rows < kVeryManyRows)
    return launch_pdl(kv_append_slots_quantised_kernel<kFp4, 16>, dim3(slot_blocks(p.n_rows)), dim3(kSlotThreads), 0, stream, p);
  const unsigned blocks = std::min((unsigned)(kStreamBlocksPerSm * p.num_sms), (unsigned)(((long long)p.n_rows + kStreamRows - 1) / kStreamRows));
  return launch_pdl(kv_append_slots_stream_kernel<kFp4>, dim3(blocks), dim3(kSlotThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_kv_append_slots(const AppendSlotsParams& p, cudaStream_t stream) {
  if (p.fmt == kKvE4M3) return launch_slots_quantised<false>(p, stream);
  if (p.fmt == kKvE2M1) return launch_slots_quantised<true>(p, stream);
  // Two items a warp halve the blocks that many rows take to launch, one is the shorter wait for few rows: 16384 rows 4.6
  // us with one and 3.5 with two; 4096 rows 1.8 and 2.1.
  constexpr int kManyRows = 8192;
  return p.n_rows >= kManyRows ? launch_slots<2>(p, stream) : launch_slots<1>(p, stream);
}

cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream) {
  return launch_pdl(kv_append_kernel, dim3(p.B), dim3(kAppendThreads), 0, stream, p);
}

}  // namespace mfa
