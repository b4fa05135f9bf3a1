// Numbers in 8 bits (e4m3: 4 exponent bits, 3 of the significand, largest 448) with
// a scale for each block of 128 columns of a row, or of 128 rows.
//
// A block's largest magnitude a, at least 2^-100 (so that neither quotient leaves
// fp32's range, whatever the block holds), gives
//   scale = a / 448,   q = e4m3(x * (448 / a)),
// each step rounded to the nearest, ties to even: the same bits wherever it is done.
// A NaN in a block makes its scale and all its numbers NaN; an infinity makes the
// scale infinite, the infinite numbers NaN and the others 0.
#pragma once

#include "rows.cuh"

namespace flce {

constexpr int kBlock8 = 128;
constexpr float kMax8 = 448.0f;
constexpr float kLeast8 = 7.888609052210118e-31f;  // 2^-100

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Largest over the aligned group of kLanes lanes.
template <int kLanes>
__device__ __forceinline__ float group_max_nan(float m) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// The largest of each of NV values over a group of L lanes: afterwards lane i of the
// group has that of value i / (L / NV).  Halves of the values are exchanged, so that
// NV values take about NV + log2(L / NV) shuffles, not NV log2(L).
template <int NV, int L>
__device__ __forceinline__ float group_max_of(float (&m)[NV]) {
  const int lane = threadIdx.x & (L - 1);
  int o = L / 2;
#pragma unroll
  for (int n = NV / 2; n > 0; n /= 2, o /= 2) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = upper ? m[i] : m[i + n], keep = upper ? m[i + n] : m[i];
      m[i] = max_nan(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  return group_max_nan<L / NV>(m[0]);
}

struct Scale8 {
  float scale, times;
  __device__ __forceinline__ explicit Scale8(float largest) {
    const float a = max_nan(largest, kLeast8);
    scale = __fdiv_rn(a, kMax8);
    times = __fdiv_rn(kMax8, a);
  }
};

// Two numbers in 8 bits, lo in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}

inline int64_t blocks8(int64_t n) { return (n + kBlock8 - 1) / kBlock8; }

// A matrix in 8 bits: rows of 16-byte blocks.
inline int check_matrix8(const void* q, int64_t rows, int64_t cols, int64_t ld) {
  if (rows > 0 && q == nullptr) return FLCE_EINVAL;
  if (ld < cols || ld >= (int64_t(1) << 40)) return FLCE_ESHAPE;
  if (rows > 0 && ld > (int64_t(1) << 60) / rows) return FLCE_ESHAPE;
  if (ld % 16 != 0 || !aligned(q, 16)) return FLCE_EALIGN;
  return FLCE_OK;
}

}  // namespace flce
