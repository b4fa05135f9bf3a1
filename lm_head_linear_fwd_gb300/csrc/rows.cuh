// Helpers shared by the operators around the loss head (embedding.cu, norm.cu,
// head4.cu): argument checks and element access.
#pragma once

#include <atomic>
#include <numeric>

#include "common.cuh"
#include "host.h"

namespace flce {

// The bytes of a [rows, cols] matrix whose rows start ld elements of es bytes apart.
struct Span {
  uintptr_t p;
  int64_t rows, row, step;  // bytes of a row, and from one to the next
  Span(const void* base, int64_t rows, int64_t cols, int64_t ld, size_t es)
      : p(reinterpret_cast<uintptr_t>(base)),
        rows(base == nullptr ? 0 : rows),
        row(cols * static_cast<int64_t>(es)),
        step(rows > 1 ? ld * static_cast<int64_t>(es) : 0) {}
  bool empty() const { return rows <= 0 || row <= 0; }
  uintptr_t end() const { return p + static_cast<uintptr_t>((rows - 1) * step + row); }
};

// Whether two matrices share a byte.  The distance from a row of b to a row of a is
// a.p - b.p plus some multiple of g = gcd(a.step, b.step); rows meet where it lies
// between -a.row and b.row.  Column slices of one buffer, and its even and odd rows,
// are apart.  Exact for equal strides; different ones may count as meeting though
// the rows that would are not there.
inline bool overlap(const Span& a, const Span& b) {
  if (a.empty() || b.empty() || a.p >= b.end() || b.p >= a.end()) return false;
  const int64_t g = std::gcd(a.step, b.step);
  if (g == 0) return true;  // one row each
  const int64_t far = static_cast<int64_t>(a.p >= b.p ? a.p - b.p : b.p - a.p) % g;
  const int64_t r = a.p >= b.p || far == 0 ? far : g - far;
  return r < b.row || g - r < a.row;
}

// A [rows, cols] matrix argument: present when it has rows, element-aligned,
// with a row stride that covers its columns and byte offsets that fit 63 bits.
inline int check_matrix(const void* p, int dt, int64_t rows, int64_t cols, int64_t ld) {
  if (rows > 0 && p == nullptr) return FLCE_EINVAL;
  if (ld < cols || ld >= (int64_t(1) << 40)) return FLCE_ESHAPE;
  if (rows > 0 && ld > (int64_t(1) << 60) / rows) return FLCE_ESHAPE;
  if (!aligned(p, dtype_size(dt))) return FLCE_EALIGN;
  return FLCE_OK;
}

// Allows a kernel `bytes` of dynamic shared memory, once per device.
template <typename K>
inline int raise_smem(K* kernel, int bytes, std::atomic<uint64_t>& raised) {
  int dev = 0;
  int rc = cuda_status(cudaGetDevice(&dev), "cudaGetDevice");
  if (rc != FLCE_OK) return rc;
  const uint64_t bit = 1ull << (dev & 63);
  if (raised.load() & bit) return FLCE_OK;
  rc = cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes),
                   "cudaFuncSetAttribute(shared memory of a kernel)");
  if (rc == FLCE_OK) raised.fetch_or(bit);
  return rc;
}

// Asynchronous copies of 16 bytes to shared memory; !valid: zeros instead.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// VEC consecutive elements of T in fp32, loaded and stored as one access of
// VEC * sizeof(T) bytes (2 to 16).
template <typename T, int VEC>
struct Vec {
  static_assert(VEC * sizeof(T) <= 16, "one access");
  float x[VEC];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == Elem<T>::kPerVec) {
      Elem<T>::unpack(*reinterpret_cast<const uint4*>(p), x);
    } else if constexpr (VEC == 2 && sizeof(T) == 2) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
      x[0] = bf16_lo(w);
      x[1] = bf16_hi(w);
    } else {
      static_assert(VEC == 1, "16 or 4 bytes, or one element");
      x[0] = Elem<T>::load(p);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VEC == Elem<T>::kPerVec) {
      *reinterpret_cast<uint4*>(p) = Elem<T>::pack(x);
    } else if constexpr (VEC == 2 && sizeof(T) == 2) {
      *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(x[0], x[1]);
    } else {
      static_assert(VEC == 1, "16 or 4 bytes, or one element");
      Elem<T>::store(p, x[0]);
    }
  }
};

// VEC elements of T as they lie in memory, to be unpacked when used (half the
// registers of Vec for bf16).
template <typename T, int VEC>
struct RawVec {
  static constexpr int kWords = VEC * sizeof(T) >= 4 ? VEC * sizeof(T) / 4 : 1;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (VEC * sizeof(T) == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      static_assert(VEC * sizeof(T) == 2, "16, 4 or 2 bytes");
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void unpack(float (&x)[VEC]) const {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if constexpr (sizeof(T) == 4)
        x[e] = __uint_as_float(w[e]);
      else
        x[e] = (e & 1) ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
    }
  }
};

// VEC values of type G as fp32, in accesses of at most 16 bytes (the address is
// aligned to them).
template <typename G, int VEC>
__device__ __forceinline__ void load_as(const G* p, float (&x)[VEC]) {
  constexpr int W = VEC < Elem<G>::kPerVec ? VEC : Elem<G>::kPerVec;
#pragma unroll
  for (int k = 0; k < VEC; k += W) {
    if constexpr (W == 4 && sizeof(G) == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p + k);
      x[k] = bf16_lo(v.x);
      x[k + 1] = bf16_hi(v.x);
      x[k + 2] = bf16_lo(v.y);
      x[k + 3] = bf16_hi(v.y);
    } else {
      Vec<G, W> v;
      v.load(p + k);
#pragma unroll
      for (int e = 0; e < W; ++e) x[k + e] = v.x[e];
    }
  }
}

// VEC fp32 values stored as type G in accesses of at most 16 bytes.
template <typename G, int VEC>
__device__ __forceinline__ void store_as(G* p, const float (&x)[VEC]) {
  constexpr int W = VEC < Elem<G>::kPerVec ? VEC : Elem<G>::kPerVec;
#pragma unroll
  for (int k = 0; k < VEC; k += W) {
    if constexpr (W == 2 && sizeof(G) == 4) {
      *reinterpret_cast<float2*>(p + k) = make_float2(x[k], x[k + 1]);
    } else if constexpr (W == 4 && sizeof(G) == 2) {
      *reinterpret_cast<uint2*>(p + k) =
          make_uint2(pack_bf16x2(x[k], x[k + 1]), pack_bf16x2(x[k + 2], x[k + 3]));
    } else {
      Vec<G, W> v;
#pragma unroll
      for (int e = 0; e < W; ++e) v.x[e] = x[k + e];
      v.store(p + k);
    }
  }
}

}  // namespace flce
