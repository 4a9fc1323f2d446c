// work_line.hpp -- a line of work units cut into equal ranges, one for each pair of CTAs, and where a unit or an element of a
// running sum lies. For the kernels' plans, and for the host, where a test goes through them.
#pragma once

#include <algorithm>

#include "mfa_internal.h"

namespace mfa {

constexpr int kUnitKeys = 2 * kPageSize;
constexpr int kKeyStep = 16;  // keys of one MMA of P V

// Largest g in [0, n) with a[g] <= x (a is non-decreasing and a[0] <= x).
template <typename T>
__host__ __device__ __forceinline__ int last_at_most(const T* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int)a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// a b / c, in 32 bits where the product allows it.
__host__ __device__ __forceinline__ int share(uint32_t a, uint32_t b, uint32_t c) {
  const unsigned long long x = (unsigned long long)a * b;
  return (x >> 32) ? (int)(x / c) : (int)((uint32_t)x / c);
}
// First unit of pair w's range of the line of C units, of W pairs; and the pair whose range holds unit x.
__host__ __device__ __forceinline__ int range_of_pair(int w, int C, int W) { return share(w, C, W); }
__host__ __device__ __forceinline__ int pair_of_unit(int x, int C, int W) {
  const unsigned long long y = ((unsigned long long)x + 1) * W - 1;
  return (y >> 32) ? (int)(y / (uint32_t)C) : (int)((uint32_t)y / (uint32_t)C);
}

}  // namespace mfa
