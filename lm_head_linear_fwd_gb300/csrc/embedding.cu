// Embedding lookup and the gradient of the table.
#include <algorithm>

#include "rows.cuh"

namespace flce {

template <typename T>
__global__ void __launch_bounds__(256)
    embedding_fwd_kernel(const int64_t* __restrict__ ids, const T* __restrict__ W, int64_t N,
                         int64_t D, int64_t V, int64_t ldw, float scale, T* __restrict__ out,
                         int64_t ldo, int32_t* status) {
  for (int64_t i = blockIdx.x; i < N; i += gridDim.x) {
    const int64_t v = ids[i];
    const bool ok = label_ok(v, V);
    if (!ok && threadIdx.x == 0) set_status(status, FLCE_ELABEL);
    for (int64_t j = threadIdx.x; j < D; j += blockDim.x)
      Elem<T>::store(out + i * ldo + j, ok ? Elem<T>::load(W + v * ldw + j) * scale : 0.0f);
  }
}

// One block per table row: the block scans all ids for its row and adds the
// matching gradient rows in token order.
template <typename T, typename G>
__global__ void __launch_bounds__(256)
    embedding_bwd_scan_kernel(const int64_t* __restrict__ ids, const T* __restrict__ dy, int64_t N,
                              int64_t D, int64_t V, int64_t ldg, float scale, int64_t padding_idx,
                              G* __restrict__ grad, int64_t ldw, int accumulate, int32_t* status) {
  __shared__ uint8_t hit[256];
  for (int64_t v = blockIdx.x; v < V; v += gridDim.x) {
    for (int64_t j0 = 0; j0 < D; j0 += blockDim.x) {
      const int64_t j = j0 + threadIdx.x;
      float sum = 0.0f;
      bool any = false;
      for (int64_t i0 = 0; i0 < N; i0 += 256) {
        const int64_t i = i0 + threadIdx.x;
        const int64_t id = i < N ? ids[i] : -1;
        if (i < N && v == 0 && j0 == 0 && !label_ok(id, V)) set_status(status, FLCE_ELABEL);
        const bool h = i < N && id == v && id != padding_idx;
        hit[threadIdx.x] = h;
        if (__syncthreads_or(h)) {
          for (int k = 0; k < 256; ++k) {
            if (!hit[k]) continue;
            any = true;
            if (j < D) sum += Elem<T>::load(dy + (i0 + k) * ldg + j);
          }
          __syncthreads();
        }
      }
      if (j < D && (any || !accumulate)) {
        G* p = grad + v * ldw + j;
        Elem<G>::store(p, accumulate ? Elem<G>::load(p) + sum * scale : sum * scale);
      }
    }
  }
}

}  // namespace flce

using namespace flce;

extern "C" int embedding_fwd(const int64_t* ids, const void* W, int dt, int64_t N, int64_t D,
                             int64_t V, int64_t ldw, float scale, void* out, int64_t ldo,
                             int32_t* status, flce_stream_t stream) {
  if (!valid_dtype(dt)) return FLCE_EDTYPE;
  if (N < 0 || D < 1 || V < 1 || V >= (int64_t(1) << 31)) return FLCE_ESHAPE;
  if (status == nullptr || W == nullptr || (N > 0 && ids == nullptr)) return FLCE_EINVAL;
  int rc = check_matrix(W, dt, V, D, ldw);
  if (rc == FLCE_OK) rc = check_matrix(out, dt, N, D, ldo);
  if (rc != FLCE_OK) return rc;
  if (!aligned(ids, 8) || !aligned(status, 4)) return FLCE_EALIGN;
  const size_t es = dtype_size(dt);
  if (overlap(W, span_bytes(V, D, ldw, es), out, span_bytes(N, D, ldo, es))) return FLCE_EINVAL;
  if (N == 0) return FLCE_OK;
  const int grid = static_cast<int>(std::min<int64_t>(N, sm_count() * 8));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dt == FLCE_BF16)
    embedding_fwd_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(
        ids, static_cast<const __nv_bfloat16*>(W), N, D, V, ldw, scale,
        static_cast<__nv_bfloat16*>(out), ldo, status);
  else
    embedding_fwd_kernel<float><<<grid, 256, 0, s>>>(ids, static_cast<const float*>(W), N, D, V,
                                                     ldw, scale, static_cast<float*>(out), ldo,
                                                     status);
  return launch_status("embedding_fwd_kernel launch");
}

extern "C" size_t embedding_bwd_workspace_bytes(int64_t N, int64_t D, int64_t V) {
  (void)N, (void)D, (void)V;
  return 0;
}

extern "C" int embedding_bwd(const int64_t* ids, const void* grad_out, int dt, int64_t N,
                             int64_t D, int64_t V, int64_t ldg, float scale, int64_t padding_idx,
                             void* grad_W, int dt_grad, int64_t ldw, int accumulate_grad_W,
                             void* ws, size_t ws_bytes, int32_t* status, flce_stream_t stream) {
  if (!valid_dtype(dt) || !valid_dtype(dt_grad)) return FLCE_EDTYPE;
  if (accumulate_grad_W != 0 && accumulate_grad_W != 1) return FLCE_EINVAL;
  if (N < 0 || N >= (int64_t(1) << 31) || D < 1 || V < 1 || V >= (int64_t(1) << 31))
    return FLCE_ESHAPE;
  if (accumulate_grad_W && dt_grad != FLCE_F32) return FLCE_ENOSUP;
  if (status == nullptr || grad_W == nullptr || (N > 0 && ids == nullptr)) return FLCE_EINVAL;
  int rc = check_matrix(grad_out, dt, N, D, ldg);
  if (rc == FLCE_OK) rc = check_matrix(grad_W, dt_grad, V, D, ldw);
  if (rc != FLCE_OK) return rc;
  if (!aligned(ids, 8) || !aligned(status, 4)) return FLCE_EALIGN;
  if (overlap(grad_out, span_bytes(N, D, ldg, dtype_size(dt)), grad_W,
              span_bytes(V, D, ldw, dtype_size(dt_grad))))
    return FLCE_EINVAL;
  const size_t need = embedding_bwd_workspace_bytes(N, D, V);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return FLCE_EWORKSPACE;
  if (!aligned(ws, 16)) return FLCE_EALIGN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int grid = static_cast<int>(std::min<int64_t>(V, sm_count() * 8));
#define FLCE_BWD(T, G)                                                                     \
  embedding_bwd_scan_kernel<T, G><<<grid, 256, 0, s>>>(                                    \
      ids, static_cast<const T*>(grad_out), N, D, V, ldg, scale, padding_idx,              \
      static_cast<G*>(grad_W), ldw, accumulate_grad_W, status)
  if (dt == FLCE_BF16 && dt_grad == FLCE_BF16) FLCE_BWD(__nv_bfloat16, __nv_bfloat16);
  else if (dt == FLCE_BF16) FLCE_BWD(__nv_bfloat16, float);
  else if (dt_grad == FLCE_BF16) FLCE_BWD(float, __nv_bfloat16);
  else FLCE_BWD(float, float);
#undef FLCE_BWD
  return launch_status("embedding_bwd_scan_kernel launch");
}
