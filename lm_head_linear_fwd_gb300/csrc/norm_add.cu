// The RMS norm of a residual stream: r = x + residual and y = r rstd weight in one
// pass, y in the rows' type, in 8 bits with a scale per 128 columns, or both; and
// its gradient, joined with the stream's own.
//
// Bound by the bytes of the rows.  The rows of x and of the residual are copied
// ahead to shared memory and their sum is held in registers, as in norm.cuh, by the
// same teams: vector k of thread l of a team is k * team + l.  A block of 128
// columns is thus one vector of each of 16 neighbouring lanes (bf16; 32 for fp32),
// which find its largest magnitude by shuffles; a team has at least that many.
// r is rounded to its type before it is squared: the norm is that of the row which
// the stream keeps and the backward pass reads.
#include "eight.cuh"
#include "norm.cuh"

namespace flce {

struct NormAddArgs {
  const void* x;
  int64_t N, D, ldx;
  const void* residual;  // may be null: zeros
  int64_t ldr;
  const void* weight;
  int w_f32;
  float eps;
  void* summed;  // may be null
  int64_t lds;
  void* y;  // may be null
  int64_t ldy;
  uint8_t* q;  // kQuant
  int64_t ldq;
  float* scales;
  float* rstd;  // may be null
  int team, teams;
};

// x as T holds it.
template <typename T>
__device__ __forceinline__ float rounded(float x) {
  return sizeof(T) == 2 ? __bfloat162float(__float2bfloat16_rn(x)) : x;
}

template <typename T, bool kWhole, int kElems, int kRows, bool kQuant>
__global__ void __launch_bounds__(kFwdThreads<T>) norm_add_fwd_kernel(NormAddArgs a) {
  extern __shared__ float4 weights[];  // weight, then the rows' copies
  constexpr int kPlaces = kRedPlaces<kFwdThreads<T>>;
  __shared__ __align__(16) float2 red[2 * kPlaces];
  using Copy = RowCopy<T, kWhole, kElems>;
  constexpr int VEC = Copy::VEC, NV = Copy::NV, P = VEC / 2;
  constexpr int kLanes = kBlock8 / VEC;  // that hold a block of 128 columns
  const int D = static_cast<int>(a.D);
  const int nvec = (D + VEC - 1) / VEC;
  const Team team(a.team, nvec, red, kPlaces);
  const int64_t all = static_cast<int64_t>(gridDim.x) * a.teams;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * a.teams + team.id;  // then row + all, ...
  int rows = rows_from(row, all, a.N);  // of this team, and of the warp's first one
  int turns = a.team < 32 ? __shfl_sync(0xffffffffu, rows, 0) : rows;
  const bool add = a.residual != nullptr;
  RowPtr<T, kWhole> x(a.x, row, a.ldx, all, team.l), res(a.residual, row, a.ldr, all, team.l);
  RowPtr<T, kWhole> sum(a.summed, row, a.lds, all, team.l), y(a.y, row, a.ldy, all, team.l);
  const int blocks = (D + kBlock8 - 1) / kBlock8;
  uint8_t* q = kQuant ? a.q + row * a.ldq : nullptr;
  float* scales = kQuant ? a.scales + row * blocks : nullptr;
  float* rstd_out = a.rstd != nullptr ? a.rstd + row : nullptr;
  char* places = reinterpret_cast<char*>(weights + nvec * (VEC / 4));
  const int row_bytes = Copy::bytes(blockDim.x, a.team);
  const Copy copy[2] = {Copy(places, team), Copy(places + (kRows - 1) * row_bytes, team)};
  const Copy rcopy[2] = {Copy(places + kRows * row_bytes, team),
                         Copy(places + (2 * kRows - 1) * row_bytes, team)};
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    copy[r].clear(false, team);
    rcopy[r].clear(!add, team);
    if (r < rows) {
      copy[r].start(x.p + r * x.step, D, team);
      if (add) rcopy[r].start(res.p + r * res.step, D, team);
    }
  }
  cp_async_commit();
  stage_weights<VEC>(weights, a.weight, a.w_f32, 1.0f, D);
  bool staged = false;  // the block's weights are there: needed late in the first row
  const float inv_n = 1.0f / static_cast<float>(D);
  for (int parity = 0; turns > 0; turns -= kRows, rows -= kRows, parity ^= 1) {
    float2 f[kRows][NV][P];
    cp_async_wait<0>();
    if (!kWhole) __syncwarp();  // the right neighbour's blocks
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float2 g[NV][P];
      copy[r].read(x.p + r * x.step, D, team, f[r]);
      rcopy[r].read(res.p + r * res.step, D, team, g);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 s = __fadd2_rn(f[r][k][e], g[k][e]);
          f[r][k][e] = make_float2(rounded<T>(s.x), rounded<T>(s.y));
        }
    }
    x.p += kRows * x.step;
    res.p += kRows * res.step;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (kRows + r < rows) {
        copy[r].start(x.p + r * x.step, D, team);
        if (add) rcopy[r].start(res.p + r * res.step, D, team);
      }
    cp_async_commit();
    float rstd[2] = {};
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float2 s[P];  // a chain of additions for each place in a vector
#pragma unroll
      for (int e = 0; e < P; ++e) s[e] = both(0.0f);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int e = 0; e < P; ++e) s[e] = __ffma2_rn(f[r][k][e], f[r][k][e], s[e]);
        if (a.summed != nullptr)
          store_vector<T, kWhole>(sum.p + r * sum.step, k, r < rows, D, team, f[r][k]);
      }
      rstd[r] = sum_pairs(s);
    }
    sum.p += kRows * sum.step;
    team.sum(rstd[0], rstd[1], parity);
#pragma unroll
    for (int r = 0; r < kRows; ++r) rstd[r] = rsqrtf(__fmaf_rn(rstd[r], inv_n, a.eps));
    if (!staged) __syncthreads();
    staged = true;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 w[P];
      weight_vec<VEC>(weights, nvec, min(team.at(k), nvec - 1), w);
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 v = __fmul2_rn(__fmul2_rn(f[r][k][e], both(rstd[r])), w[e]);
          f[r][k][e] = v;
          if (kQuant) m = max_nan(m, max_nan(fabsf(v.x), fabsf(v.y)));
        }
        if (a.y != nullptr)
          store_vector<T, kWhole>(y.p + r * y.step, k, r < rows, D, team, f[r][k]);
        if (!kQuant) continue;
        const Scale8 s(group_max_nan<kLanes>(m));
        const int j = team.at(k) * VEC;
        if (r >= rows || j >= D) continue;
        const int64_t at = r * all;
        if ((team.l & (kLanes - 1)) == 0) scales[at * blocks + j / kBlock8] = s.scale;
        uint32_t packed[VEC / 4];
#pragma unroll
        for (int e = 0; e < P; e += 2) {
          const float2 u = __fmul2_rn(f[r][k][e], both(s.times));
          const float2 v = __fmul2_rn(f[r][k][e + 1], both(s.times));
          packed[e / 2] = pack_e4m3x4(u.x, u.y, v.x, v.y);
        }
        uint8_t* to = q + at * a.ldq + j;
        if (j + VEC <= D) {
          if constexpr (VEC == 8)
            *reinterpret_cast<uint2*>(to) = make_uint2(packed[0], packed[1]);
          else
            *reinterpret_cast<uint32_t*>(to) = packed[0];
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (j + e < D) to[e] = static_cast<uint8_t>(packed[e / 4] >> (e % 4 * 8));
        }
      }
    }
    y.p += kRows * y.step;
    if (kQuant) {
      q += kRows * all * a.ldq;
      scales += kRows * all * blocks;
    }
    if (rstd_out != nullptr) {
      if (team.l == 0) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          if (r < rows) rstd_out[r * all] = rstd[r];
      }
      rstd_out += kRows * all;
    }
  }
  if (!staged) __syncthreads();  // warps without a row
  cp_async_wait<0>();
}

// Rows too wide to hold: one block per row, which is read again for the norm (the
// stored sum, where there is one: it may lie in x or in the residual).  A warp takes
// a block of 128 columns at a time.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) norm_add_fwd_long_kernel(NormAddArgs a) {
  __shared__ float red[kLongThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t blocks = (a.D + kBlock8 - 1) / kBlock8;
  for (int64_t i = blockIdx.x; i < a.N; i += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + i * a.ldx;
    const T* res = a.residual != nullptr ? static_cast<const T*>(a.residual) + i * a.ldr : nullptr;
    T* sum = a.summed != nullptr ? static_cast<T*>(a.summed) + i * a.lds : nullptr;
    T* y = a.y != nullptr ? static_cast<T*>(a.y) + i * a.ldy : nullptr;
    float s = 0.0f;
    for (int64_t b = warp; b < blocks; b += kLongThreads / 32)
      for (int64_t j = b * kBlock8 + lane; j < min(a.D, (b + 1) * kBlock8); j += 32) {
        float f = Elem<T>::load(x + j);
        if (res != nullptr) f = rounded<T>(f + Elem<T>::load(res + j));
        if (sum != nullptr) Elem<T>::store(sum + j, f);
        s += f * f;
      }
    const float rstd = rsqrtf(block_sum(s, red) / static_cast<float>(a.D) + a.eps);
    // the same thread as above has each element
    for (int64_t b = warp; b < blocks; b += kLongThreads / 32) {
      float v[kBlock8 / 32], m = 0.0f;
#pragma unroll
      for (int k = 0; k < kBlock8 / 32; ++k) {
        const int64_t j = b * kBlock8 + k * 32 + lane;
        v[k] = 0.0f;
        if (j < a.D) {
          float f;
          if (sum != nullptr) {
            f = Elem<T>::load(sum + j);
          } else {
            f = Elem<T>::load(x + j);
            if (res != nullptr) f = rounded<T>(f + Elem<T>::load(res + j));
          }
          v[k] = f * rstd * weight_at(a.weight, a.w_f32, j, 1.0f);
          if (y != nullptr) Elem<T>::store(y + j, v[k]);
        }
        m = max_nan(m, fabsf(v[k]));
      }
      if (a.q == nullptr) continue;
      const Scale8 sc(group_max_nan<32>(m));
      if (lane == 0) a.scales[i * blocks + b] = sc.scale;
#pragma unroll
      for (int k = 0; k < kBlock8 / 32; ++k) {
        const int64_t j = b * kBlock8 + k * 32 + lane;
        if (j < a.D)
          a.q[i * a.ldq + j] = static_cast<uint8_t>(pack_e4m3x2(__fmul_rn(v[k], sc.times), 0.0f));
      }
    }
    if (threadIdx.x == 0 && a.rstd != nullptr) a.rstd[i] = rstd;
  }
}

// Launches norm_add_fwd_kernel; returns 1 (nothing launched) when a row does not fit.
template <typename T, bool kWhole, int kElems, int kRows, bool kQuant>
static int launch_norm_add_k(NormAddArgs a, cudaStream_t s) {
  if (a.D > int64_t(kFwdThreads<T>) * kElems) return 1;
  auto* kernel = norm_add_fwd_kernel<T, kWhole, kElems, kRows, kQuant>;
  static std::atomic<uint64_t> raised{0};
  const int rc = raise_smem(kernel, kSmemMost, raised);
  if (rc != FLCE_OK) return rc;
  // (also without the 8 bits: the sums' order does not depend on the outputs asked for)
  const int least = kBlock8 * static_cast<int>(sizeof(T)) / 16;
  const NormPlan p = norm_plan(a.N, a.D, kElems, kFwdThreads<T>, least);
  a.team = p.team;
  a.teams = p.teams;
  const int threads = p.team * p.teams;
  const size_t smem =
      weight_bytes(a.D) + 2 * kRows * RowCopy<T, kWhole, kElems>::bytes(threads, p.team);
  if (smem > kSmemMost) return 1;
  kernel<<<static_cast<unsigned>(p.blocks), threads, smem, s>>>(a);
  return launch_status("norm_add_fwd_kernel launch");
}

template <typename T, bool kQuant>
static int launch_norm_add(NormAddArgs a, int dt, cudaStream_t s) {
  auto aligned_rows = [dt](const void* p, int64_t ld) { return p == nullptr || whole(dt, p, ld); };
  const bool w = aligned_rows(a.x, a.ldx) && aligned_rows(a.residual, a.ldr) &&
                 aligned_rows(a.summed, a.lds) && aligned_rows(a.y, a.ldy) &&
                 whole(dt, nullptr, a.D);
  int rc = w ? launch_norm_add_k<T, true, kFwdLane, 2, kQuant>(a, s)
             : launch_norm_add_k<T, false, kFwdLane, 2, kQuant>(a, s);
  if (rc == 1)
    rc = w ? launch_norm_add_k<T, true, kFwdLaneLong, 1, kQuant>(a, s)
           : launch_norm_add_k<T, false, kFwdLaneLong, 1, kQuant>(a, s);
  if (rc != 1) return rc;
  const int grid = static_cast<int>(std::min<int64_t>(a.N, sm_count() * 8));
  norm_add_fwd_long_kernel<T><<<grid, kLongThreads, 0, s>>>(a);
  return launch_status("norm_add_fwd_long_kernel launch");
}

// An output may be an input itself, row by row; else they must not overlap.
static bool clash(const Span& out, int64_t ld_out, const Span& in, int64_t ld_in) {
  if (out.empty() || in.empty()) return false;
  return out.p == in.p ? ld_out != ld_in && out.rows > 1 : overlap(out, in);
}

}  // namespace flce

using namespace flce;

extern "C" int rms_norm_add_fwd(const void* x, int dt, int64_t N, int64_t D, int64_t ldx,
                                const void* residual, int64_t ldr, const void* weight, int wdt,
                                float eps, void* summed, int64_t lds, void* y, int64_t ldy,
                                uint8_t* q, int64_t ldq, float* scales, float* rstd,
                                flce_stream_t stream) {
  if (!valid_dtype(dt) || !valid_dtype(wdt)) return FLCE_EDTYPE;
  if (N < 0 || D < 1) return FLCE_ESHAPE;
  int rc = check_matrix(x, dt, N, D, ldx);
  if (rc == FLCE_OK && residual != nullptr) rc = check_matrix(residual, dt, N, D, ldr);
  if (rc == FLCE_OK && summed != nullptr) rc = check_matrix(summed, dt, N, D, lds);
  if (rc == FLCE_OK && y != nullptr) rc = check_matrix(y, dt, N, D, ldy);
  if (rc == FLCE_OK && q != nullptr) rc = check_matrix8(q, N, D, ldq);
  if (rc != FLCE_OK) return rc;
  if ((q == nullptr) != (scales == nullptr) || (N > 0 && y == nullptr && q == nullptr))
    return FLCE_EINVAL;
  if (!aligned(weight, dtype_size(wdt)) || !aligned(scales, 4) || !aligned(rstd, 4))
    return FLCE_EALIGN;
  const size_t es = dtype_size(dt);
  const Span in[2] = {Span(x, N, D, ldx, es), Span(residual, N, D, ldr, es)};
  const int64_t ld_in[2] = {ldx, ldr};
  const Span s_sum(summed, N, D, lds, es), s_y(y, N, D, ldy, es), s_q(q, N, D, ldq, 1),
      s_scales(scales, N, blocks8(D), blocks8(D), 4);
  for (int i = 0; i < 2; ++i)
    if (clash(s_sum, lds, in[i], ld_in[i]) || clash(s_y, ldy, in[i], ld_in[i]) ||
        overlap(s_q, in[i]) || overlap(s_scales, in[i]))
      return FLCE_EINVAL;
  if (overlap(s_sum, s_y) || overlap(s_sum, s_q) || overlap(s_sum, s_scales) ||
      overlap(s_y, s_q) || overlap(s_y, s_scales) || overlap(s_q, s_scales))
    return FLCE_EINVAL;
  if (N == 0) return FLCE_OK;
  NormAddArgs a{};
  a.x = x, a.N = N, a.D = D, a.ldx = ldx, a.residual = residual, a.ldr = ldr;
  a.weight = weight, a.w_f32 = wdt == FLCE_F32, a.eps = eps, a.summed = summed, a.lds = lds;
  a.y = y, a.ldy = ldy, a.q = q, a.ldq = ldq, a.scales = scales, a.rstd = rstd;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dt == FLCE_BF16)
    return q != nullptr ? launch_norm_add<__nv_bfloat16, true>(a, dt, s)
                        : launch_norm_add<__nv_bfloat16, false>(a, dt, s);
  return q != nullptr ? launch_norm_add<float, true>(a, dt, s)
                      : launch_norm_add<float, false>(a, dt, s);
}

extern "C" int rms_norm_add_bwd(const void* summed, int dt, int64_t N, int64_t D, int64_t lds,
                                const void* grad_y, int64_t ldgy, const void* grad_summed,
                                int64_t ldgs, const void* weight, int wdt, const float* rstd,
                                void* grad_x, int64_t ldgx, float* grad_weight, int accumulate,
                                void* ws, size_t ws_bytes, flce_stream_t stream) {
  NormBwdArgs a{};
  a.x = summed, a.N = N, a.D = D, a.ldx = lds, a.dy = grad_y, a.lddy = ldgy;
  a.more = grad_summed, a.ldmore = ldgs, a.weight = weight, a.rstd = rstd;
  a.dx = grad_x, a.lddx = ldgx, a.dw = grad_weight, a.accumulate = accumulate;
  if (grad_x == nullptr || N == 0) a.more = nullptr;
  return a.more != nullptr ? norm_bwd<false, true>(a, dt, wdt, ws, ws_bytes, stream)
                           : norm_bwd<false, false>(a, dt, wdt, ws, ws_bytes, stream);
}
