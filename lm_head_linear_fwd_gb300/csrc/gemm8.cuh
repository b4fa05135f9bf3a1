// The product of two matrices in 8 bits (eight.cuh):
//   y[m, n] = sum over blocks k of a_scales[m, k] b_scales[n, k]
//             sum over the block's columns j of a[m, j] b[n, j]      (+ bias[n])
//
// tcgen05.mma forms a block's sums (products of two e4m3 numbers are exact in fp32)
// in tensor memory; its 128 columns are 128 bytes, one stage of the ring in shared
// memory and four instructions.  The scales change from block to block, so every
// block's sums are read back and added up in fp32 registers, times their scales:
// while the next block's are formed, in another part of tensor memory.
#pragma once

#include <cuda.h>

#include "eight.cuh"

namespace flce {

// D (+)= A B^T, both 8 bits in shared memory, fp32 sums.
__device__ __forceinline__ void mma_8bit(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// One lane of a warp whose lanes are all here.  The products are issued by a warp that
// goes through its loop as a whole, so that descriptors and addresses stay in the
// registers that a warp shares, where the instruction wants them: with one lane in
// the loop four products and their two commits took 450 cycles to issue.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// This thread's warp, known to be the same for all its lanes.
__device__ __forceinline__ int warp_index() {
  return __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
}

// K columns of fp32 of this thread's lane of tensor memory (16 or 32).
template <int K>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float (&v)[K]) {
  if constexpr (K == 32) {
    tmem_ld32(taddr, v);
  } else {
    static_assert(K == 16, "16 or 32 columns");
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
  }
}

struct Gemm8Args {
  int64_t M, N;  // rows of a (tokens) and of b (weights)
  int blocks;    // of 128 columns
  const float* a_scales;  // [M, blocks]
  const float* b_scales;  // [N / b_rows, blocks]
  int b_rows;             // 1 or 128
  const void* bias;       // [N] or null
  int bias_f32;
  void* y;
  int64_t ldy;
  int y_f32, accumulate;
  int32_t* status;  // may be null
  int64_t tiles_m, tiles_n;
  int split;        // CTAs of a cluster, which share a tile's blocks
};

__device__ __forceinline__ float2 both_nan() {
  return make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
}

__device__ __forceinline__ float bias_at(const Gemm8Args& g, int64_t n) {
  if (g.bias == nullptr || n >= g.N) return 0.0f;
  return g.bias_f32 ? static_cast<const float*>(g.bias)[n]
                    : Elem<__nv_bfloat16>::load(static_cast<const __nv_bfloat16*>(g.bias) + n);
}

}  // namespace flce
