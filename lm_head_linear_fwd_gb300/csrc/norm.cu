// Layer norm and RMS norm: the calls (kernels: norm.cuh).
#include "norm.cuh"

namespace flce {

// Launches norm_fwd_kernel; returns 1 (nothing launched) when a row does not fit.
template <typename T, bool kWhole, bool kCenter, int kElems, int kRows>
static int launch_norm_fwd_k(NormArgs a, cudaStream_t s) {
  if (a.D > int64_t(kFwdThreads<T>) * kElems) return 1;
  static std::atomic<uint64_t> raised{0};
  const int rc = raise_smem(norm_fwd_kernel<T, kWhole, kCenter, kElems, kRows>, kSmemMost, raised);
  if (rc != FLCE_OK) return rc;
  const NormPlan p = norm_plan(a.N, a.D, kElems, kFwdThreads<T>);
  a.team = p.team;
  a.teams = p.teams;
  const int threads = p.team * p.teams;
  const size_t smem = weight_bytes(a.D) * (kCenter ? 2 : 1) +
                      kRows * RowCopy<T, kWhole, kElems>::bytes(threads, p.team);
  if (smem > kSmemMost) return 1;
  norm_fwd_kernel<T, kWhole, kCenter, kElems, kRows>
      <<<static_cast<unsigned>(p.blocks), threads, smem, s>>>(a);
  return launch_status("norm_fwd_kernel launch");
}

template <typename T, bool kCenter>
static int launch_norm_fwd(NormArgs a, int dt, cudaStream_t s) {
  const bool w = whole(dt, a.x, a.ldx) && whole(dt, a.y, a.ldy) && whole(dt, nullptr, a.D);
  int rc = w ? launch_norm_fwd_k<T, true, kCenter, kFwdLane, 2>(a, s)
             : launch_norm_fwd_k<T, false, kCenter, kFwdLane, 2>(a, s);
  if (rc == 1)
    rc = w ? launch_norm_fwd_k<T, true, kCenter, kFwdLaneLong, 1>(a, s)
           : launch_norm_fwd_k<T, false, kCenter, kFwdLaneLong, 1>(a, s);
  if (rc != 1) return rc;
  const int grid = static_cast<int>(std::min<int64_t>(a.N, sm_count() * 8));
  norm_fwd_long_kernel<T, kCenter><<<grid, kLongThreads, 0, s>>>(a);
  return launch_status("norm_fwd_long_kernel launch");
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
                 : overlap(Span(a.x, a.N, a.D, a.ldx, es), Span(a.y, a.N, a.D, a.ldy, es)))
    return FLCE_EINVAL;
  if (a.N == 0) return FLCE_OK;
  a.w_f32 = wdt == FLCE_F32;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dt == FLCE_BF16 ? launch_norm_fwd<__nv_bfloat16, kCenter>(a, dt, s)
                         : launch_norm_fwd<float, kCenter>(a, dt, s);
}

}  // namespace flce

using namespace flce;

extern "C" int layer_norm_fwd(const void* x, int dt, int64_t N, int64_t D, int64_t ldx,
                              const void* weight, const void* bias, int wdt, float eps, void* y,
                              int64_t ldy, float* mean, float* rstd, flce_stream_t stream) {
  NormArgs a{};
  a.x = x, a.N = N, a.D = D, a.ldx = ldx, a.weight = weight, a.bias = bias, a.eps = eps;
  a.y = y, a.ldy = ldy, a.mean = mean, a.rstd = rstd;
  return norm_fwd<true>(a, dt, wdt, stream);
}

extern "C" int rms_norm_fwd(const void* x, int dt, int64_t N, int64_t D, int64_t ldx,
                            const void* weight, int wdt, float eps, void* y, int64_t ldy,
                            float* rstd, flce_stream_t stream) {
  NormArgs a{};
  a.x = x, a.N = N, a.D = D, a.ldx = ldx, a.weight = weight, a.eps = eps;
  a.y = y, a.ldy = ldy, a.rstd = rstd;
  return norm_fwd<false>(a, dt, wdt, stream);
}

extern "C" size_t norm_bwd_workspace_bytes(int64_t N, int64_t D) {
  if (N < 1 || D < 1) return 0;
  return round_up(static_cast<size_t>(bwd_slices(N, D)) * 2 * static_cast<size_t>(D) * 4, 256);
}

extern "C" int layer_norm_bwd(const void* x, int dt, int64_t N, int64_t D, int64_t ldx,
                              const void* grad_y, int64_t ldgy, const void* weight, int wdt,
                              const float* mean, const float* rstd, void* grad_x, int64_t ldgx,
                              float* grad_weight, float* grad_bias, int accumulate, void* ws,
                              size_t ws_bytes, flce_stream_t stream) {
  NormBwdArgs a{};
  a.x = x, a.N = N, a.D = D, a.ldx = ldx, a.dy = grad_y, a.lddy = ldgy, a.weight = weight;
  a.mean = mean, a.rstd = rstd, a.dx = grad_x, a.lddx = ldgx, a.dw = grad_weight;
  a.db = grad_bias, a.accumulate = accumulate;
  return norm_bwd<true, false>(a, dt, wdt, ws, ws_bytes, stream);
}

extern "C" int rms_norm_bwd(const void* x, int dt, int64_t N, int64_t D, int64_t ldx,
                            const void* grad_y, int64_t ldgy, const void* weight, int wdt,
                            const float* rstd, void* grad_x, int64_t ldgx, float* grad_weight,
                            int accumulate, void* ws, size_t ws_bytes, flce_stream_t stream) {
  NormBwdArgs a{};
  a.x = x, a.N = N, a.D = D, a.ldx = ldx, a.dy = grad_y, a.lddy = ldgy, a.weight = weight;
  a.rstd = rstd, a.dx = grad_x, a.lddx = ldgx, a.dw = grad_weight, a.accumulate = accumulate;
  return norm_bwd<false, false>(a, dt, wdt, ws, ws_bytes, stream);
}
