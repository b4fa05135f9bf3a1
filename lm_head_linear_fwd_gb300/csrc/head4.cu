// The head with 4-bit weights and group scales: logits of a few tokens, and
// the rounding of a table to that layout.
#include <algorithm>

#include "rows.cuh"

namespace flce {

struct Head4Args {
  const void* x;
  int64_t M, D, ldx;
  const uint8_t* packed;
  int64_t ldp;
  const void* scales;
  const uint8_t* zeros;
  int group;
  int64_t V, G;
  const void* bias;
  void* y;
  int64_t ldy;
};

// Byte (from the row's start) and shift of column k in the packed layout.
__device__ __forceinline__ int64_t packed_byte(int64_t k, int* shift) {
  const int r = static_cast<int>(k & 127);
  const int w = r >> 5, t = (r >> 3) & 3, j = r & 7;
  const int p = (j >> 1) + 4 * (j & 1);
  *shift = 4 * (p & 1);
  return (k >> 7) * 64 + (4 * t + w) * 4 + (p >> 1);
}

// One warp per (token, vocabulary row).
template <typename T, typename S, typename Y>
__global__ void __launch_bounds__(256) head4_rows_kernel(Head4Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t n = a.M * a.V;
  for (int64_t o = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); o < n;
       o += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t m = o / a.V, v = o % a.V;
    const T* x = static_cast<const T*>(a.x) + m * a.ldx;
    float sum = 0.0f;
    for (int64_t k = lane; k < a.D; k += 32) {
      int shift;
      const int64_t at = packed_byte(k, &shift);
      const int q = (a.packed[v * a.ldp + at] >> shift) & 15;
      const int64_t gi = v * a.G + k / a.group;
      const int z = a.zeros != nullptr ? a.zeros[gi] & 15 : 8;
      sum += Elem<T>::load(x + k) * (static_cast<float>(q - z) *
                                     Elem<S>::load(static_cast<const S*>(a.scales) + gi));
    }
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) {
      if (a.bias != nullptr) sum += Elem<T>::load(static_cast<const T*>(a.bias) + v);
      Elem<Y>::store(static_cast<Y*>(a.y) + m * a.ldy + v, sum);
    }
  }
}

struct Quant4Args {
  const void* W;
  int64_t V, D, ldw;
  int group;
  uint8_t* packed;
  int64_t ldp;
  void* scales;
  uint8_t* zeros;
  int64_t G;
};

__device__ __forceinline__ float round_to(float v, const float*) { return v; }
__device__ __forceinline__ float round_to(float v, const __nv_bfloat16*) {
  return __bfloat162float(__float2bfloat16_rn(v));
}

// One warp per 128 columns of a row: each lane forms one 32-bit word for two
// passes of the block (words lane < 16).  The groups' extremes are found by
// the lanes that hold their columns.
template <typename T, typename S>
__global__ void __launch_bounds__(256) head4_quantize_kernel(Quant4Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t blocks = (a.D + 127) / 128;
  const int64_t n = a.V * blocks;
  for (int64_t o = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); o < n;
       o += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t v = o / blocks, b = o % blocks;
    const T* row = static_cast<const T*>(a.W) + v * a.ldw;
    // lane l < 16 holds word l of the block: columns 32 w + 8 t + j, l = 4 t + w
    const int l = lane & 15, w = l & 3, t = l >> 2;
    const int64_t k0 = b * 128 + 32 * w + 8 * t;
    float x[8], lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = k0 + j < a.D ? Elem<T>::load(row + k0 + j) : 0.0f;
      lo = fminf(lo, x[j]);
      hi = fmaxf(hi, x[j]);
    }
    // the words of one 32-column group differ in t (lane bits 2, 3); groups of
    // 64 and 128 columns also in bits 0 and 1 of w
    for (int d = 4; d <= 8; d <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
    }
    for (int d = 1; 32 * d < a.group; d <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
    }
    const bool zp = a.zeros != nullptr;
    float s = zp ? __fdiv_rn(hi - lo, 15.0f) : __fdiv_rn(fmaxf(hi, -lo), 7.0f);
    s = round_to(s, static_cast<const S*>(nullptr));
    if (s == 0.0f) s = 1.0f;
    const float z = zp ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f) : 8.0f;
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float r = rintf(__fdiv_rn(x[j], s)) + z;
      const uint32_t q = k0 + j < a.D ? static_cast<uint32_t>(fminf(fmaxf(r, 0.0f), 15.0f)) : 0u;
      word |= q << (4 * ((j >> 1) + 4 * (j & 1)));
    }
    if (lane < 16) {
      *reinterpret_cast<uint32_t*>(a.packed + v * a.ldp + b * 64 + 4 * l) = word;
      const int64_t gi = k0 / a.group;
      if (t == 0 && (32 * w) % a.group == 0 && gi < a.G) {
        Elem<S>::store(static_cast<S*>(a.scales) + v * a.G + gi, s);
        if (zp) a.zeros[v * a.G + gi] = static_cast<uint8_t>(z);
      }
    }
  }
}

static int check_head4(const void* packed, int64_t ldp, const void* scales, int dt_s, int group,
                       int64_t V, int64_t D) {
  if (!valid_dtype(dt_s)) return FLCE_EDTYPE;
  if (group != 32 && group != 64 && group != 128) return FLCE_ESHAPE;
  if (V < 1 || V >= (int64_t(1) << 31) || D < 1 || D >= (int64_t(1) << 31)) return FLCE_ESHAPE;
  if (ldp < (D + 127) / 128 * 64 || ldp >= (int64_t(1) << 31)) return FLCE_ESHAPE;
  if (packed == nullptr || scales == nullptr) return FLCE_EINVAL;
  if (ldp % 16 != 0 || !aligned(packed, 16) || !aligned(scales, dtype_size(dt_s)))
    return FLCE_EALIGN;
  return FLCE_OK;
}

}  // namespace flce

using namespace flce;

extern "C" size_t head4_workspace_bytes(int dt, int64_t M, int64_t D, int64_t V) {
  (void)dt, (void)M, (void)D, (void)V;
  return 0;
}

extern "C" int head4_logits(const void* x, int dt, int64_t M, int64_t D, int64_t ldx,
                            const uint8_t* packed, int64_t ldp, const void* scales, int dt_s,
                            const uint8_t* zeros, int group, int64_t V, const void* bias, void* y,
                            int dt_y, int64_t ldy, void* ws, size_t ws_bytes,
                            flce_stream_t stream) {
  if (!valid_dtype(dt) || !valid_dtype(dt_y)) return FLCE_EDTYPE;
  if (M < 0) return FLCE_ESHAPE;
  int rc = check_head4(packed, ldp, scales, dt_s, group, V, D);
  if (rc == FLCE_OK) rc = check_matrix(x, dt, M, D, ldx);
  if (rc == FLCE_OK) rc = check_matrix(y, dt_y, M, V, ldy);
  if (rc != FLCE_OK) return rc;
  if (!aligned(bias, dtype_size(dt))) return FLCE_EALIGN;
  const size_t need = head4_workspace_bytes(dt, M, D, V);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return FLCE_EWORKSPACE;
  if (!aligned(ws, 16)) return FLCE_EALIGN;
  if (M == 0) return FLCE_OK;
  const Head4Args a{x, M, D, ldx, packed, ldp, scales, zeros, group, V, (D + group - 1) / group,
                    bias, y, ldy};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int grid = static_cast<int>(std::min<int64_t>((M * V + 7) / 8, sm_count() * 8));
  using B = __nv_bfloat16;
#define FLCE_H4(T, S, Y) head4_rows_kernel<T, S, Y><<<grid, 256, 0, s>>>(a)
  if (dt == FLCE_BF16) {
    if (dt_s == FLCE_BF16) {
      if (dt_y == FLCE_BF16) FLCE_H4(B, B, B); else FLCE_H4(B, B, float);
    } else {
      if (dt_y == FLCE_BF16) FLCE_H4(B, float, B); else FLCE_H4(B, float, float);
    }
  } else {
    if (dt_s == FLCE_BF16) {
      if (dt_y == FLCE_BF16) FLCE_H4(float, B, B); else FLCE_H4(float, B, float);
    } else {
      if (dt_y == FLCE_BF16) FLCE_H4(float, float, B); else FLCE_H4(float, float, float);
    }
  }
#undef FLCE_H4
  return launch_status("head4_rows_kernel launch");
}

extern "C" int head4_quantize(const void* W, int dt, int64_t V, int64_t D, int64_t ldw, int group,
                              uint8_t* packed, int64_t ldp, void* scales, int dt_s, uint8_t* zeros,
                              flce_stream_t stream) {
  if (!valid_dtype(dt)) return FLCE_EDTYPE;
  int rc = check_head4(packed, ldp, scales, dt_s, group, V, D);
  if (rc == FLCE_OK) rc = check_matrix(W, dt, V, D, ldw);
  if (rc != FLCE_OK) return rc;
  const Quant4Args a{W, V, D, ldw, group, packed, ldp, scales, zeros, (D + group - 1) / group};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t blocks = (D + 127) / 128;
  const int grid = static_cast<int>(std::min<int64_t>((V * blocks + 7) / 8, sm_count() * 16));
  using B = __nv_bfloat16;
  if (dt == FLCE_BF16) {
    if (dt_s == FLCE_BF16) head4_quantize_kernel<B, B><<<grid, 256, 0, s>>>(a);
    else head4_quantize_kernel<B, float><<<grid, 256, 0, s>>>(a);
  } else {
    if (dt_s == FLCE_BF16) head4_quantize_kernel<float, B><<<grid, 256, 0, s>>>(a);
    else head4_quantize_kernel<float, float><<<grid, 256, 0, s>>>(a);
  }
  return launch_status("head4_quantize_kernel launch");
}
