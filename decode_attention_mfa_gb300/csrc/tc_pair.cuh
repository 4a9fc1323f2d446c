// tc_pair.cuh -- building blocks of the kernels in which a cluster of two CTAs
// works on one matrix of 256 query rows (64 heads of four sequences or of four
// tokens) with tcgen05 MMAs of cta_group::2: barriers and copies of the pair,
// the split of a line of work among pairs, the values of an 8-bit cache, and
// what a softmax thread, whose row is its TMEM lane, does with its row.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "mfa_device.cuh"
#include "work_line.hpp"

namespace mfa {

// Exponents of V's scales that f16 holds beside the codes' (V' = code * scale * 2^kUp): E4M3, V' at most 448 * 2^7 and its
// scale at least 2^-10; E2M1, 6 * 2^13 and 2^-13.
struct E4m3Range {
  static constexpr int kLeast = -16, kMost = 0, kUp = 6;
};
struct E2m1Range {
  static constexpr int kLeast = -16, kMost = 9, kUp = 3;
};
// The most that a weight takes of a scale outside: far enough from 2^127 for their sums.
constexpr int kMostShift = 100;
constexpr int kTmemCols = 512, kTmemO = 256, kSCols = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A move of the reference leaves the row's largest weight at 2^moved_to: of bf16, whose relative step is the same
// everywhere, anything will do, of f16 a value that leaves room both ways. The next move comes when the sum of
// a thread's 64 weights of a unit passes kMostSum, so that none of them passes f16's range; the sum is needed anyway,
// and a maximum is looked for only then.
template <bool kFp8>
__host__ __device__ constexpr float moved_to() { return kFp8 ? 4.0f : 0.0f; }
constexpr float kMostSum = 32768.0f;
// Waits for what this CTA itself has in flight, before it leaves, do not shrink with the wait budget; and after a wait
// that gave up, copies that no barrier of this CTA tells of get this long to land.
constexpr uint64_t kDrainNs = 200000000ull, kSettleNs = 1000000ull;

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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Arrival on a barrier of the pair's leader. What it announces is read by the MMAs alone, and lies in tensor memory,
// which the tcgen05 fences order, or in this CTA's shared memory, which the proxy fence before it has made visible to
// them, so no release at cluster scope is needed: that one takes 1500 cycles, most of a unit's time.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
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
// TMA loads into this CTA's shared memory that complete on a barrier of the pair's leader.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y,
                                                 uint32_t leader_bar, uint64_t cache_hint) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(leader_bar), "l"(cache_hint)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t leader_bar,
                                                 uint64_t cache_hint) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(leader_bar), "l"(cache_hint)
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
// The same without the output lanes (rows) of `off`: bit i of word w stands for row 32 w + i of the pair's 256.
__device__ __forceinline__ void tc_mma_pair_tmem_a_masked(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                                          const uint32_t (&off)[8], uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8, %9, %10, %11, %12}, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]),
      "r"(off[4]), "r"(off[5]), "r"(off[6]), "r"(off[7])
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
// it, or a TMA copy, without a loop over the threads that might be active (80 cycles an MMA, of which a unit has 32; the
// eight copies of a Q took 0.6 us).
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
};

__device__ __forceinline__ int warp_inclusive_sum(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kPageSize - 1) / kPageSize; }

// Whether the last MMA of P V on a page of so many tokens reaches behind them.
__device__ __forceinline__ bool is_partial(int tokens) { return tokens % kKeyStep != 0; }

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// The exponent that a key's weight takes of its V scale: what lies outside [kLeast, kMost]. A scale of zero (or below the
// fp32 normal range) has none, its row adds nothing.
template <typename R>
__device__ __forceinline__ int scale_shift(float scale) {
  const int e = (int)((__float_as_uint(scale) >> 23) & 0xFFu) - 127;
  return e == -127 ? 0 : max(-kMostShift, min(kMostShift, e - max(R::kLeast, min(R::kMost, e))));
}
// Whether it may have one (zeros are taken for such, too).
template <typename R>
__device__ __forceinline__ bool may_shift(float scale) {
  constexpr uint32_t kLeast = (uint32_t)(127 + R::kLeast) << 23, kSpan = (uint32_t)(R::kMost - R::kLeast + 1) << 23;
  return (__float_as_uint(scale) & 0x7FFFFFFFu) - kLeast >= kSpan;
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
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
// Four neighbouring lanes, each with 32 values of its row, exchange them so that lane j has values 8 j .. 8 j + 7 of all
// four rows (row k's at v[8 k]): a store then writes whole 128 B lines instead of 32 B of as many rows as lanes (a tile's
// result took 4 us that way).
__device__ __forceinline__ void transpose_quad(float (&v)[32], int lane) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float other = __shfl_xor_sync(0xffffffffu, (lane & 2) ? v[i] : v[16 + i], 2);
    if (lane & 2) v[i] = other; else v[16 + i] = other;
  }
#pragma unroll
  for (int h = 0; h < 32; h += 16)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? v[h + i] : v[h + 8 + i], 1);
      if (lane & 1) v[h + i] = other; else v[h + 8 + i] = other;
    }
}
// 32 bytes at once.
__device__ __forceinline__ void st_global_v8(float* dst, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
// Barriers of the two warps that share 32 rows.
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

// Eight bf16 values times `up` (at most 448 then) as two E4M3 terms: codes of four in a word. Between them the values are
// f16, which holds their eight bits exactly from 2^-17 on (the second term's last step is 2^-9); in fp32 the two prompts
// on an 8-bit cache take 0.4 us more.
// kPairs: the product, which is exact, as bf16 pairs, one operation of ten less; the chunk kernel gains 0.5% by it (two prompts of
// 4096 672.7 -> 669.4 us), the shared-prefix kernel loses 0.4 to 3% (128 sequences behind 512 pages 182.4 -> 188.4), whose loops the
// compiler then lays out otherwise.
template <bool kPairs>
__device__ __forceinline__ void split_q8(const uint4 v, float up, uint32_t (&t1)[2], uint32_t (&t2)[2]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const __nv_bfloat162 up_2 = __float2bfloat162_rn(up);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t a = 0, b = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      __half2 x;
      if constexpr (kPairs) {
        const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[2 * i + k]), up_2);
        const uint32_t bits = *reinterpret_cast<const uint32_t*>(&y);
        x = __floats2half2_rn(__uint_as_float(bits << 16), __uint_as_float(bits & 0xFFFF0000u));
      } else {
        x = __floats2half2_rn(__uint_as_float(w[2 * i + k] << 16) * up, __uint_as_float(w[2 * i + k] & 0xFFFF0000u) * up);
      }
      const __nv_fp8x2_storage_t c1 =
          __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&x), __NV_SATFINITE, __NV_E4M3);
      const __half2_raw h1 = __nv_cvt_fp8x2_to_halfraw2(c1, __NV_E4M3);
      const __half2 rest = __hsub2(x, *reinterpret_cast<const __half2*>(&h1));
      const __nv_fp8x2_storage_t c2 =
          __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&rest), __NV_SATFINITE, __NV_E4M3);
      a |= (uint32_t)c1 << (16 * k);
      b |= (uint32_t)c2 << (16 * k);
    }
    t1[i] = a;
    t2[i] = b;
  }
}

// E4M3: a unit whose V scales have shifts, which is rare and out of line: in the usual units' loop it cost them 9% (304
// sequences behind 256 pages 182 -> 199 us), the threads' look for such scales alone at most 1%. P takes the shifts, the
// denominator does not. The reference is looked for among all keys, so no second try follows and P may replace S at once.
// tx: this thread's 64 products, sc: their K scales, 128 before their V scales. Returns the row's reference and this thread's
// share of its denominator. Both warps of the rows; what O holds is complete.
template <typename R>
static __device__ __noinline__ float2 shifted_unit(uint32_t tx, uint32_t o_addr, const float* sc, int cols, float mul, float m,
                                                   float l, bool fresh, float* red, int row, int half) {
  const float* v_scale = sc + kUnitKeys;
  float x[32];
  float top = -INFINITY;
#pragma unroll 1
  for (int g = 0; g < 64; g += 32) {
    tmem_ld32(tx + g, x);
    tc_wait_ld();
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (g + k < cols) top = fmaxf(top, x[k] * sc[g + k] * mul + (float)scale_shift<R>(v_scale[g + k]));
  }
  red[half * 128 + row] = top - moved_to<true>();
  barrier_rows(row >> 5);
  const float m_new = fmaxf(m, fmaxf(red[row], red[128 + row]));
  const float alpha = fresh || m == m_new ? 1.0f : ex2_approx(m - m_new);
  if (!fresh && __any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll 1
    for (int c = 128 * half; c < 128 * half + 128; c += 32) {
      tmem_ld32(o_addr + c, x);
      tc_wait_ld();
#pragma unroll
      for (int k = 0; k < 32; ++k) x[k] *= alpha;
      tmem_st32(o_addr + c, x);
    }
  }
  const float ref = m_new == -INFINITY ? 0.0f : m_new;
  float sum = 0.0f;
#pragma unroll 1
  for (int g = 0; g < 64; g += 32) {
    tmem_ld32(tx + g, x);
    tc_wait_ld();
    uint32_t w[16];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float y = g + k < cols ? ex2_approx(fmaf(x[k] * sc[g + k], mul, -ref)) : 0.0f;
      sum += y;
      x[k] = y * exp2_int(scale_shift<R>(v_scale[g + k]));
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) w[c] = pack_f16(x[2 * c], x[2 * c + 1]);
    tmem_st16(tx + g, reinterpret_cast<const float*>(w));
  }
  tc_wait_st();
  barrier_rows(row >> 5);  // red is free again
  return make_float2(m_new, l * alpha + sum);
}

}  // namespace mfa
