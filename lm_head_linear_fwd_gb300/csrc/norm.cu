// Layer norm and RMS norm, forward and backward.
#include <algorithm>

#include "rows.cuh"

namespace flce {

constexpr int kNormThreads = 256;

// Sum over the block; every thread returns the same value.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < kNormThreads / 32; ++w) s += red[w];
  __syncthreads();
  return s;
}

struct NormArgs {
  const void* x;
  int64_t N, D, ldx;
  const void* weight;
  const void* bias;
  float eps;
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
};

template <typename T, typename U, bool kCenter>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_kernel(NormArgs a) {
  __shared__ float red[kNormThreads / 32];
  const U* w = static_cast<const U*>(a.weight);
  const U* b = static_cast<const U*>(a.bias);
  for (int64_t i = blockIdx.x; i < a.N; i += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + i * a.ldx;
    T* y = static_cast<T*>(a.y) + i * a.ldy;
    float mean = 0.0f;
    if (kCenter) {
      float s = 0.0f;
      for (int64_t j = threadIdx.x; j < a.D; j += kNormThreads) s += Elem<T>::load(x + j);
      mean = block_sum(s, red) / static_cast<float>(a.D);
    }
    float q = 0.0f;
    for (int64_t j = threadIdx.x; j < a.D; j += kNormThreads) {
      const float d = Elem<T>::load(x + j) - mean;
      q += d * d;
    }
    const float rstd = 1.0f / sqrtf(block_sum(q, red) / static_cast<float>(a.D) + a.eps);
    for (int64_t j = threadIdx.x; j < a.D; j += kNormThreads) {
      float v = (Elem<T>::load(x + j) - mean) * rstd;
      if (w != nullptr) v *= Elem<U>::load(w + j);
      if (b != nullptr) v += Elem<U>::load(b + j);
      Elem<T>::store(y + j, v);
    }
    if (threadIdx.x == 0) {
      if (kCenter && a.mean != nullptr) a.mean[i] = mean;
      if (a.rstd != nullptr) a.rstd[i] = rstd;
    }
  }
}

struct NormBwdArgs {
  const void* x;
  int64_t N, D, ldx;
  const void* dy;
  int64_t lddy;
  const void* weight;
  const float* mean;
  const float* rstd;
  void* dx;
  int64_t lddx;
  float* dw;
  float* db;
  int accumulate;
  float* part;
  int slices;
};

template <typename T, typename U, bool kCenter>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_rows_kernel(NormBwdArgs a) {
  __shared__ float red[kNormThreads / 32];
  const U* w = static_cast<const U*>(a.weight);
  for (int64_t i = blockIdx.x; i < a.N; i += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + i * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + i * a.lddy;
    T* dx = static_cast<T*>(a.dx) + i * a.lddx;
    const float mean = kCenter ? a.mean[i] : 0.0f, rstd = a.rstd[i];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t j = threadIdx.x; j < a.D; j += kNormThreads) {
      const float u = Elem<T>::load(dy + j) * (w != nullptr ? Elem<U>::load(w + j) : 1.0f);
      s1 += u;
      s2 += u * ((Elem<T>::load(x + j) - mean) * rstd);
    }
    const float c1 = kCenter ? block_sum(s1, red) / static_cast<float>(a.D) : 0.0f;
    const float c2 = block_sum(s2, red) / static_cast<float>(a.D);
    for (int64_t j = threadIdx.x; j < a.D; j += kNormThreads) {
      const float u = Elem<T>::load(dy + j) * (w != nullptr ? Elem<U>::load(w + j) : 1.0f);
      const float h = (Elem<T>::load(x + j) - mean) * rstd;
      Elem<T>::store(dx + j, rstd * (u - c1 - h * c2));
    }
  }
}

// Column sums of one slice of the rows: 256 columns per block.
template <typename T, bool kCenter>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_cols_kernel(NormBwdArgs a) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x;
  if (j >= a.D) return;
  const int64_t per = (a.N + a.slices - 1) / a.slices;
  const int64_t i0 = blockIdx.y * per, i1 = i0 + per < a.N ? i0 + per : a.N;
  float dw = 0.0f, db = 0.0f;
  for (int64_t i = i0; i < i1; ++i) {
    const float g = Elem<T>::load(static_cast<const T*>(a.dy) + i * a.lddy + j);
    const float x = Elem<T>::load(static_cast<const T*>(a.x) + i * a.ldx + j);
    dw += g * ((x - (kCenter ? a.mean[i] : 0.0f)) * a.rstd[i]);
    db += g;
  }
  a.part[(2 * static_cast<int64_t>(blockIdx.y)) * a.D + j] = dw;
  a.part[(2 * static_cast<int64_t>(blockIdx.y) + 1) * a.D + j] = db;
}

__global__ void __launch_bounds__(kNormThreads) norm_bwd_finish_kernel(NormBwdArgs a) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x;
  if (j >= a.D) return;
  float dw = 0.0f, db = 0.0f;
  for (int k = 0; k < a.slices; ++k) {
    dw += a.part[(2 * static_cast<int64_t>(k)) * a.D + j];
    db += a.part[(2 * static_cast<int64_t>(k) + 1) * a.D + j];
  }
  if (a.dw != nullptr) a.dw[j] = a.accumulate ? a.dw[j] + dw : dw;
  if (a.db != nullptr) a.db[j] = a.accumulate ? a.db[j] + db : db;
}

template <bool kCenter>
static int norm_fwd(NormArgs a, int dt, int wdt, flce_stream_t stream) {
  if (!valid_dtype(dt) || !valid_dtype(wdt)) return FLCE_EDTYPE;
  if (a.N < 0 || a.D < 1) return FLCE_ESHAPE;
  int rc = check_matrix(a.x, dt, a.N, a.D, a.ldx);
  if (rc == FLCE_OK) rc = check_matrix(a.y, dt, a.N, a.D, a.ldy);
  if (rc != FLCE_OK) return rc;
  const size_t es = dtype_size(dt);
  if (!aligned(a.weight, dtype_size(wdt)) || !aligned(a.bias, dtype_size(wdt)) ||
      !aligned(a.mean, 4) || !aligned(a.rstd, 4))
    return FLCE_EALIGN;
  if (a.x == a.y ? a.ldx != a.ldy && a.N > 1
                 : overlap(a.x, span_bytes(a.N, a.D, a.ldx, es), a.y,
                           span_bytes(a.N, a.D, a.ldy, es)))
    return FLCE_EINVAL;
  if (a.N == 0) return FLCE_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int grid = static_cast<int>(std::min<int64_t>(a.N, sm_count() * 8));
  using B = __nv_bfloat16;
  if (dt == FLCE_BF16 && wdt == FLCE_BF16)
    norm_fwd_kernel<B, B, kCenter><<<grid, kNormThreads, 0, s>>>(a);
  else if (dt == FLCE_BF16)
    norm_fwd_kernel<B, float, kCenter><<<grid, kNormThreads, 0, s>>>(a);
  else if (wdt == FLCE_BF16)
    norm_fwd_kernel<float, B, kCenter><<<grid, kNormThreads, 0, s>>>(a);
  else
    norm_fwd_kernel<float, float, kCenter><<<grid, kNormThreads, 0, s>>>(a);
  return launch_status("norm_fwd_kernel launch");
}

template <bool kCenter>
static int norm_bwd(NormBwdArgs a, int dt, int wdt, void* ws, size_t ws_bytes,
                    flce_stream_t stream) {
  if (!valid_dtype(dt) || !valid_dtype(wdt)) return FLCE_EDTYPE;
  if (a.accumulate != 0 && a.accumulate != 1) return FLCE_EINVAL;
  if (a.N < 0 || a.D < 1) return FLCE_ESHAPE;
  int rc = check_matrix(a.x, dt, a.N, a.D, a.ldx);
  if (rc == FLCE_OK) rc = check_matrix(a.dy, dt, a.N, a.D, a.lddy);
  if (rc == FLCE_OK && a.dx != nullptr) rc = check_matrix(a.dx, dt, a.N, a.D, a.lddx);
  if (rc != FLCE_OK) return rc;
  if (a.N > 0 && (a.rstd == nullptr || (kCenter && a.mean == nullptr))) return FLCE_EINVAL;
  const size_t es = dtype_size(dt);
  if (!aligned(a.weight, dtype_size(wdt)) || !aligned(a.mean, 4) || !aligned(a.rstd, 4) ||
      !aligned(a.dw, 4) || !aligned(a.db, 4))
    return FLCE_EALIGN;
  if (a.dx != nullptr) {
    const int64_t n = span_bytes(a.N, a.D, a.lddx, es);
    if (overlap(a.x, span_bytes(a.N, a.D, a.ldx, es), a.dx, n)) return FLCE_EINVAL;
    if (a.dx == a.dy ? a.lddx != a.lddy && a.N > 1
                     : overlap(a.dy, span_bytes(a.N, a.D, a.lddy, es), a.dx, n))
      return FLCE_EINVAL;
  }
  const bool cols = a.dw != nullptr || a.db != nullptr;
  if (cols) {
    const size_t need = norm_bwd_workspace_bytes(a.N, a.D);
    if (need > 0 && (ws == nullptr || ws_bytes < need)) return FLCE_EWORKSPACE;
    if (!aligned(ws, 16)) return FLCE_EALIGN;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  using B = __nv_bfloat16;
  a.part = static_cast<float*>(ws);
  a.slices = static_cast<int>(std::min<int64_t>(64, a.N));
  if (cols) {
    const unsigned nb = static_cast<unsigned>((a.D + kNormThreads - 1) / kNormThreads);
    if (a.slices > 0) {
      const dim3 g(nb, a.slices);
      if (dt == FLCE_BF16)
        norm_bwd_cols_kernel<B, kCenter><<<g, kNormThreads, 0, s>>>(a);
      else
        norm_bwd_cols_kernel<float, kCenter><<<g, kNormThreads, 0, s>>>(a);
    }
    norm_bwd_finish_kernel<<<nb, kNormThreads, 0, s>>>(a);
  }
  if (a.dx != nullptr && a.N > 0) {
    const int grid = static_cast<int>(std::min<int64_t>(a.N, sm_count() * 8));
    if (dt == FLCE_BF16 && wdt == FLCE_BF16)
      norm_bwd_rows_kernel<B, B, kCenter><<<grid, kNormThreads, 0, s>>>(a);
    else if (dt == FLCE_BF16)
      norm_bwd_rows_kernel<B, float, kCenter><<<grid, kNormThreads, 0, s>>>(a);
    else if (wdt == FLCE_BF16)
      norm_bwd_rows_kernel<float, B, kCenter><<<grid, kNormThreads, 0, s>>>(a);
    else
      norm_bwd_rows_kernel<float, float, kCenter><<<grid, kNormThreads, 0, s>>>(a);
  }
  return launch_status("norm_bwd launch");
}

}  // namespace flce

using namespace flce;

extern "C" int layer_norm_fwd(const void* x, int dt, int64_t N, int64_t D, int64_t ldx,
                              const void* weight, const void* bias, int wdt, float eps, void* y,
                              int64_t ldy, float* mean, float* rstd, flce_stream_t stream) {
  return norm_fwd<true>({x, N, D, ldx, weight, bias, eps, y, ldy, mean, rstd}, dt, wdt, stream);
}

extern "C" int rms_norm_fwd(const void* x, int dt, int64_t N, int64_t D, int64_t ldx,
                            const void* weight, int wdt, float eps, void* y, int64_t ldy,
                            float* rstd, flce_stream_t stream) {
  return norm_fwd<false>({x, N, D, ldx, weight, nullptr, eps, y, ldy, nullptr, rstd}, dt, wdt,
                         stream);
}

extern "C" size_t norm_bwd_workspace_bytes(int64_t N, int64_t D) {
  if (N < 1 || D < 1) return 0;
  return 64 * 2 * round_up(static_cast<size_t>(D) * 4, 256);
}

extern "C" int layer_norm_bwd(const void* x, int dt, int64_t N, int64_t D, int64_t ldx,
                              const void* grad_y, int64_t ldgy, const void* weight, int wdt,
                              const float* mean, const float* rstd, void* grad_x, int64_t ldgx,
                              float* grad_weight, float* grad_bias, int accumulate, void* ws,
                              size_t ws_bytes, flce_stream_t stream) {
  return norm_bwd<true>({x, N, D, ldx, grad_y, ldgy, weight, mean, rstd, grad_x, ldgx,
                         grad_weight, grad_bias, accumulate, nullptr, 0},
                        dt, wdt, ws, ws_bytes, stream);
}

extern "C" int rms_norm_bwd(const void* x, int dt, int64_t N, int64_t D, int64_t ldx,
                            const void* grad_y, int64_t ldgy, const void* weight, int wdt,
                            const float* rstd, void* grad_x, int64_t ldgx, float* grad_weight,
                            int accumulate, void* ws, size_t ws_bytes, flce_stream_t stream) {
  return norm_bwd<false>({x, N, D, ldx, grad_y, ldgy, weight, nullptr, rstd, grad_x, ldgx,
                          grad_weight, nullptr, accumulate, nullptr, 0},
                         dt, wdt, ws, ws_bytes, stream);
}
