// Helpers shared by the operators around the loss head (embedding.cu, norm.cu,
// head4.cu): argument checks and element access.
#pragma once

#include "common.cuh"
#include "host.h"

namespace flce {

// Bytes from the first to the last element of a [rows, cols] matrix.
inline int64_t span_bytes(int64_t rows, int64_t cols, int64_t ld, size_t es) {
  return rows <= 0 ? 0 : ((rows - 1) * ld + cols) * static_cast<int64_t>(es);
}

inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) &&
         y < x + static_cast<uintptr_t>(na);
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

}  // namespace flce
