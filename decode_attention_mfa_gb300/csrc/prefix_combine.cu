// prefix_combine.cu -- merges a sequence's partial results of the shared-prefix
// kernel (of the pairs of CTAs that held pages it sees). With O_s and
// lse_s of part s, M = max_s lse_s and w_s = exp(lse_s - M):
//     out = sum_s w_s O_s / sum_s w_s,   lse = M + ln sum_s w_s.
//
// The kernel's plan has left where a sequence's parts are (PrefixParams::parts),
// so a CTA reads nothing but them. One CTA of 256 threads per (sequence, kH
// heads): warp i < kH turns the LSEs of head i into weights while the parts' O
// rows, kH KB each, come into shared memory by bulk copies; then 256 / kH
// threads a head sum them in fp32. A row of weight 0 (an underflowed exponent,
// or a part without a finite logit) is skipped, never scaled. Bound by latency,
// and for large batches by reading the parts from L2: 2.3 us behind the prefix
// kernel for 4 sequences, 3.8 us for 32 with 19 MB of parts.
#include "mfa_device.cuh"
#include "mfa_serving.hpp"

namespace mfa {
namespace {

constexpr int kThreads = 256;
// Rows in shared memory a round: with four and eight heads a CTA the parts of a batch of 32 (up to about twelve a
// sequence) and of larger ones (about four) come in one round; four CTAs of that size share an SM.
template <int kH>
__host__ __device__ constexpr int chunk_bytes() { return kH >= 4 ? 48 * 1024 : 32 * 1024; }
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint64_t kDrainNs = 200000000ull;

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int kH>
__global__ void __launch_bounds__(kThreads, 4) prefix_combine_kernel(const PrefixParams p) {
  constexpr int kPerHead = kThreads / kH;               // threads of a head
  constexpr int kDimThreads = kPerHead < 64 ? kPerHead : 64;
  constexpr int kVec = kHeadDim / (4 * kDimThreads);    // float4s a thread
  constexpr int kSubsets = kPerHead / kDimThreads;      // the parts are dealt to this many sets of threads
  constexpr int kChunkBytes = chunk_bytes<kH>();
  constexpr int kPartBytes = kH * 1024;
  constexpr int kChunk = kChunkBytes / kPartBytes;      // parts a round
  static_assert(kDimThreads * kVec * 4 == kHeadDim && kH <= 8 && kChunk <= 32, "shape");
  extern __shared__ __align__(128) uint8_t smem_raw[];
  float* s_w = reinterpret_cast<float*>(smem_raw + kChunkBytes);  // [kH][2 * pairs] normalised weights
  __shared__ float s_lse[kH];
  __shared__ float4 s_acc[kSubsets > 1 ? kThreads * kVec : 1];
  __shared__ __align__(8) uint64_t s_bar;
  const uint32_t o_base = smem_u32(smem_raw), bar = smem_u32(&s_bar);
  const int b = blockIdx.y, h0 = blockIdx.x * kH;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hl = threadIdx.x / kPerHead, r = threadIdx.x % kPerHead;
  const int dt = r % kDimThreads, sub = r / kDimThreads;
  uint16_t* out = p.out + ((size_t)b * kHeads + h0 + hl) * kHeadDim;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait_prior_grid();
  const int4 at = __ldcg(p.parts + b);
  const int n = at.y + at.w;
  if (n == 0) {  // an empty sequence
    if (sub == 0) {
#pragma unroll
      for (int v = 0; v < kVec; ++v) reinterpret_cast<uint2*>(out)[dt * kVec + v] = make_uint2(0u, 0u);
      if (dt == 0) p.lse[(size_t)b * kHeads + h0 + hl] = -INFINITY;
    }
    return;
  }
  auto part = [&](int i) -> size_t {  // row of part i
    return i < at.y ? (size_t)at.x + (size_t)i * kPrefixTileSeqs : (size_t)at.z + (size_t)(i - at.y) * kPrefixTileSeqs;
  };
  auto issue_round = [&](int k) {  // warp 0, one copy a lane
    const int i0 = k * kChunk, cnt = min(kChunk, n - i0);
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(cnt * kPartBytes));
    __syncwarp();
    if (lane < cnt)
      bulk_load(o_base + (uint32_t)(lane * kPartBytes), p.part_o + (part(i0 + lane) * kHeads + h0) * kHeadDim, kPartBytes, bar);
  };
  if (warp == 0) issue_round(0);
  if (warp < kH) {
    float* w = s_w + warp * 2 * p.pairs;
    float mx = -INFINITY;
    for (int i = lane; i < n; i += 32) {
      const float v = __ldcg(p.part_lse + part(i) * kHeads + h0 + warp);
      w[i] = v;
      mx = fmaxf(mx, v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    float den = 0.0f;
    for (int i = lane; i < n; i += 32) {
      const float e = exp2f((w[i] - mx) * kLog2e);
      w[i] = e;
      den += e;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    const float inv = 1.0f / den;
    for (int i = lane; i < n; i += 32) w[i] *= inv;
    if (lane == 0) s_lse[warp] = mx + log2f(den) * kLn2;
  }
  __syncthreads();

  const float* w = s_w + hl * 2 * p.pairs;
  float4 acc[kVec];
#pragma unroll
  for (int v = 0; v < kVec; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int rounds = (n + kChunk - 1) / kChunk;
  for (int k = 0; k < rounds; ++k) {
    if (k > 0) {
      __syncthreads();  // every thread is done with the previous round's rows
      if (warp == 0) issue_round(k);
    }
    // bounded, but not by the wait budget: these are this CTA's own copies. On expiry the error word records it, and every
    // thread still reaches the barriers.
    (void)mbar_wait(bar, k & 1, kDrainNs, nullptr, p.err);
    const int i0 = k * kChunk, cnt = min(kChunk, n - i0);
    for (int i = sub; i < cnt; i += kSubsets) {
      const float wi = w[i0 + i];
      if (wi != 0.0f) {
        const float4* row = reinterpret_cast<const float4*>(smem_raw + i * kPartBytes + hl * 1024) + dt * kVec;
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          const float4 y = row[v];
          acc[v].x = fmaf(wi, y.x, acc[v].x);
          acc[v].y = fmaf(wi, y.y, acc[v].y);
          acc[v].z = fmaf(wi, y.z, acc[v].z);
          acc[v].w = fmaf(wi, y.w, acc[v].w);
        }
      }
    }
  }
  if constexpr (kSubsets > 1) {
#pragma unroll
    for (int v = 0; v < kVec; ++v) s_acc[threadIdx.x * kVec + v] = acc[v];
    __syncthreads();
    if (sub == 0) {
      for (int k = 1; k < kSubsets; ++k) {
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
          const float4 y = s_acc[(threadIdx.x + k * kDimThreads) * kVec + v];
          acc[v].x += y.x;
          acc[v].y += y.y;
          acc[v].z += y.z;
          acc[v].w += y.w;
        }
      }
    }
  }
  if (sub == 0) {
#pragma unroll
    for (int v = 0; v < kVec; ++v)
      reinterpret_cast<uint2*>(out)[dt * kVec + v] =
          make_uint2(pack_bf16x2(acc[v].x, acc[v].y), pack_bf16x2(acc[v].z, acc[v].w));
    if (dt == 0) p.lse[(size_t)b * kHeads + h0 + hl] = s_lse[hl];
  }
}

template <int kH>
cudaError_t launch_kh(const PrefixParams& p, cudaStream_t stream) {
  const size_t smem = chunk_bytes<kH>() + sizeof(float) * (size_t)kH * 2 * p.pairs;
  static int configured[kTrackedDevices] = {};
  const cudaError_t e = ensure_dynamic_smem(prefix_combine_kernel<kH>, smem, configured);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefix_combine_kernel<kH>, dim3(kHeads / kH, p.B), dim3(kThreads), smem, stream, p);
}

}  // namespace

// Heads a CTA: as in the LSE combine, about two to four CTAs an SM.
cudaError_t launch_prefix_combine(const PrefixParams& p, cudaStream_t stream) {
  if (p.B <= 8) return launch_kh<1>(p, stream);
  if (p.B <= 16) return launch_kh<2>(p, stream);
  if (p.B <= 48) return launch_kh<4>(p, stream);
  return launch_kh<8>(p, stream);
}

}  // namespace mfa
