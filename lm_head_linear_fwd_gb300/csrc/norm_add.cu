// The RMS norm of a residual stream: r = x + residual and y = r rstd weight in one
// pass, y in the rows' type, in 8 bits with a scale per 128 columns, or both; and
// its gradient, joined with the stream's own.
//
// Bound by the bytes of the rows.  The rows of x and of the residual are copied
// ahead to shared memory and their sum is held in registers, as in norm.cuh, by the
// same teams: vector k of thread l of a team is k * team + l.  A block of 128
// columns is thus one vector of each of 16 neighbouring lanes (bf16; 32 for fp32),
// which find its largest magnitude by shuffles; a team has at least that many.
// Rows that begin inside 16-byte blocks have a kernel of their own.
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

constexpr int kZeroWeights = 32;

// Rows on 16-byte boundaries.  65536 x 5120 bf16: 363 us with y in 8 bits, 415 in bf16
// (both 6.5 TB/s); 8192 x 4096 to 8 bits 43.5 us.  With two rows at a time of 16 elements
// per thread, as in norm_fwd_kernel, and two divisions per block and lane: 412, 415, 49.
template <typename T, int kElems, bool kQuant>
__global__ void __launch_bounds__(kFwdThreads<T>) norm_add_fwd_kernel(NormAddArgs a) {
  extern __shared__ float4 weights[];  // weight, then the row's copies
  constexpr int kPlaces = kRedPlaces<kFwdThreads<T>>;
  __shared__ __align__(16) float2 red[2 * kPlaces];
  using Copy = RowCopy<T, true, kElems>;
  constexpr int VEC = Copy::VEC, NV = Copy::NV, P = VEC / 2;
  constexpr int kLanes = kBlock8 / VEC;  // that hold a block of 128 columns
  const int D = static_cast<int>(a.D);
  const int nvec = D / VEC;
  const Team team(a.team, nvec, red, kPlaces);
  const int64_t all = static_cast<int64_t>(gridDim.x) * a.teams;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * a.teams + team.id;  // then row + all, ...
  int rows = rows_from(row, all, a.N);  // of this team, and of the warp's first one
  int turns = a.team < 32 ? __shfl_sync(0xffffffffu, rows, 0) : rows;
  const bool add = a.residual != nullptr;
  RowPtr<T, true> x(a.x, row, a.ldx, all, team.l), res(a.residual, row, a.ldr, all, team.l);
  RowPtr<T, true> sum(a.summed, row, a.lds, all, team.l), y(a.y, row, a.ldy, all, team.l);
  const int blocks = (D + kBlock8 - 1) / kBlock8;
  uint8_t* q = kQuant ? a.q + row * a.ldq : nullptr;
  float* scales = kQuant ? a.scales + row * blocks : nullptr;
  float* rstd_out = a.rstd != nullptr ? a.rstd + row : nullptr;
  // A vector of zeros behind the weights, for the threads' places past the row's end: 0 times
  // the last weights, if these are infinite, would be NaN in their block.  (128 bytes leave
  // the copies where they were: one vector's cost 4 of 78 us.)
  const int pitch = nvec + kZeroWeights / VEC;
  if (threadIdx.x < VEC / 4)
    weights[threadIdx.x * pitch + nvec] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  char* places = reinterpret_cast<char*>(weights + pitch * (VEC / 4));
  const Copy copy(places, team), rcopy(places + Copy::bytes(blockDim.x, a.team), team);
  copy.clear(false, team);
  rcopy.clear(!add, team);
  if (rows > 0) {
    copy.start(x.p, D, team);
    if (add) rcopy.start(res.p, D, team);
  }
  cp_async_commit();
  stage_weights<VEC>(weights, a.weight, a.w_f32, 1.0f, D, pitch);
  bool staged = false;  // the block's weights are there: needed late in the first row
  const float inv_n = 1.0f / static_cast<float>(D);
  for (int parity = 0; turns > 0; --turns, --rows, parity ^= 1) {
    float2 f[NV][P];
    cp_async_wait<0>();
    {
      float2 g[NV][P];
      copy.read(x.p, D, team, f);
      rcopy.read(res.p, D, team, g);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 s = __fadd2_rn(f[k][e], g[k][e]);
          f[k][e] = make_float2(rounded<T>(s.x), rounded<T>(s.y));
        }
    }
    x.p += x.step;
    res.p += res.step;
    if (rows > 1) {
      copy.start(x.p, D, team);
      if (add) rcopy.start(res.p, D, team);
    }
    cp_async_commit();
    float2 s[P];  // a chain of additions for each place in a vector
#pragma unroll
    for (int e = 0; e < P; ++e) s[e] = both(0.0f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int e = 0; e < P; ++e) s[e] = __ffma2_rn(f[k][e], f[k][e], s[e]);
      if (a.summed != nullptr) store_vector<T, true>(sum.p, k, rows > 0, D, team, f[k]);
    }
    sum.p += sum.step;
    float rstd = sum_pairs(s), unused = 0.0f;
    team.sum(rstd, unused, parity);
    rstd = rsqrtf(__fmaf_rn(rstd, inv_n, a.eps));
    if (!staged) __syncthreads();
    staged = true;
    float m[NV];  // the vectors' largest magnitudes
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 w[P];
      weight_vec<VEC>(weights, pitch, min(team.at(k), nvec), w);
      m[k] = 0.0f;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        f[k][e] = __fmul2_rn(__fmul2_rn(f[k][e], both(rstd)), w[e]);
        if (kQuant) m[k] = max_nan(m[k], max_nan(fabsf(f[k][e].x), fabsf(f[k][e].y)));
      }
      if (a.y != nullptr) store_vector<T, true>(y.p, k, rows > 0, D, team, f[k]);
    }
    y.p += y.step;
    if constexpr (kQuant) {
      // a lane divides for one block: the even ones form its `times`, the odd ones its scale
      constexpr int kPer = kLanes / NV;
      const float largest = max_nan(group_max_of<NV, kLanes>(m), kLeast8);
      const bool odd = (threadIdx.x & 1) != 0;
      const float mine = __fdiv_rn(odd ? largest : kMax8, odd ? kMax8 : largest);
      const int in_group = threadIdx.x & (kLanes - 1);
      const int block = (in_group / kPer * team.size + team.l - in_group) / kLanes;
      if (in_group % kPer == 1 && rows > 0 && block < blocks) scales[block] = mine;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const float times =
            __shfl_sync(0xffffffffu, mine, (threadIdx.x & 31 & ~(kLanes - 1)) + k * kPer);
        uint32_t packed[VEC / 4];
#pragma unroll
        for (int e = 0; e < P; e += 2) {
          const float2 u = __fmul2_rn(f[k][e], both(times));
          const float2 v = __fmul2_rn(f[k][e + 1], both(times));
          packed[e / 2] = pack_e4m3x4(u.x, u.y, v.x, v.y);
        }
        uint8_t* to = q + team.at(k) * VEC;
        if (rows > 0 && k < team.mine) {
          if constexpr (VEC == 8)
            *reinterpret_cast<uint2*>(to) = make_uint2(packed[0], packed[1]);
          else
            *reinterpret_cast<uint32_t*>(to) = packed[0];
        }
      }
      q += all * a.ldq;
      scales += all * blocks;
    }
    if (rstd_out != nullptr) {
      if (team.l == 0 && rows > 0) *rstd_out = rstd;
      rstd_out += all;
    }
  }
  if (!staged) __syncthreads();  // warps without a row
  cp_async_wait<0>();
}

// Rows that begin anywhere: element by element, 32 neighbouring ones to a warp's access.
// A warp has blocks of 128 columns, kAnyBlocks of them at most, in registers; `team`
// warps have a row.  Bound by the latency of a row's loads, sums and stores, one after the
// other, with what registers leave of an SM's warps (27; issue slots 54% full): 8191 x
// 1601 bf16 29 us, to 8 bits 37, fp32 44; four blocks to a warp 33, 48
// and 67 us, one 32, 42 and 43; whole 16-byte blocks shifted together, as in
// norm_fwd_kernel, 52, 55 and 75.
constexpr int kAnyThreads = 512;

template <typename T, int kAnyBlocks, bool kQuant>
__global__ void __launch_bounds__(kAnyThreads, 2) norm_add_fwd_any_kernel(NormAddArgs a) {
  __shared__ float red[2][kAnyThreads / 32];
  __shared__ uint32_t bytes[kQuant ? kAnyThreads / 32 : 1][kBlock8 / 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / a.team, w = warp - team * a.team;
  const int D = static_cast<int>(a.D), blocks = (D + kBlock8 - 1) / kBlock8;
  float wt[kAnyBlocks][4];  // the same columns of every row
#pragma unroll
  for (int b = 0; b < kAnyBlocks; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = (w + b * a.team) * kBlock8 + e * 32 + lane;
      wt[b][e] = j < D ? weight_at(a.weight, a.w_f32, j, 1.0f) : 0.0f;
    }
  const int64_t all = static_cast<int64_t>(gridDim.x) * a.teams;
  const float inv_n = 1.0f / static_cast<float>(D);
  int parity = 0;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * a.teams + team; i < a.N;
       i += all, parity ^= 1) {
    const T* x = static_cast<const T*>(a.x) + i * a.ldx;
    const T* res = a.residual != nullptr ? static_cast<const T*>(a.residual) + i * a.ldr : nullptr;
    T* sum = a.summed != nullptr ? static_cast<T*>(a.summed) + i * a.lds : nullptr;
    T* y = a.y != nullptr ? static_cast<T*>(a.y) + i * a.ldy : nullptr;
    float f[kAnyBlocks][4];
#pragma unroll
    for (int b = 0; b < kAnyBlocks; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = (w + b * a.team) * kBlock8 + e * 32 + lane;
        f[b][e] = j < D ? Elem<T>::load(x + j) : 0.0f;
      }
    if (res != nullptr) {
#pragma unroll
      for (int b = 0; b < kAnyBlocks; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = (w + b * a.team) * kBlock8 + e * 32 + lane;
          if (j < D) f[b][e] = rounded<T>(f[b][e] + Elem<T>::load(res + j));
        }
    }
    float s[4] = {};
#pragma unroll
    for (int b = 0; b < kAnyBlocks; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = (w + b * a.team) * kBlock8 + e * 32 + lane;
        s[e] = __fmaf_rn(f[b][e], f[b][e], s[e]);
        if (sum != nullptr && j < D) Elem<T>::store(sum + j, f[b][e]);
      }
    float total = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (a.team > 1) {
      if (lane == 0) red[parity][warp] = total;
      named_barrier(1 + team, a.team * 32);
      total = 0.0f;
      for (int k = 0; k < a.team; ++k) total += red[parity][team * a.team + k];
    }
    const float rstd = rsqrtf(__fmaf_rn(total, inv_n, a.eps));
    float m[kAnyBlocks];
#pragma unroll
    for (int b = 0; b < kAnyBlocks; ++b) {
      m[b] = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = (w + b * a.team) * kBlock8 + e * 32 + lane;
        f[b][e] = f[b][e] * rstd * wt[b][e];
        if (y != nullptr && j < D) Elem<T>::store(y + j, f[b][e]);
        if (kQuant) m[b] = max_nan(m[b], fabsf(f[b][e]));
      }
    }
    if constexpr (kQuant) {
      // a lane divides for one block, as above
      constexpr int kPer = 32 / kAnyBlocks;
      const float largest = max_nan(group_max_of<kAnyBlocks, 32>(m), kLeast8);
      const bool odd = (lane & 1) != 0;
      const float mine = __fdiv_rn(odd ? largest : kMax8, odd ? kMax8 : largest);
      const int mine_block = w + lane / kPer * a.team;
      if (lane % kPer == 1 && mine_block < blocks) a.scales[i * blocks + mine_block] = mine;
      uint8_t* q = a.q + i * a.ldq;
      uint8_t* own = reinterpret_cast<uint8_t*>(bytes[warp]);
#pragma unroll
      for (int b = 0; b < kAnyBlocks; ++b) {
        const float times = __shfl_sync(0xffffffffu, mine, b * kPer);
        const int j = (w + b * a.team) * kBlock8 + lane * 4;
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const uint32_t two =
              pack_e4m3x2(__fmul_rn(f[b][e], times), __fmul_rn(f[b][e + 1], times));
          own[e * 32 + lane] = static_cast<uint8_t>(two);
          own[e * 32 + 32 + lane] = static_cast<uint8_t>(two >> 8);
        }
        __syncwarp();
        if (j + 4 <= D) {
          *reinterpret_cast<uint32_t*>(q + j) = bytes[warp][lane];
        } else {
          for (int e = 0; j + e < D; ++e) q[j + e] = own[lane * 4 + e];
        }
      }
    }
    if (lane == 0 && w == 0 && a.rstd != nullptr) a.rstd[i] = rstd;
  }
}

// The gradient for rows that begin anywhere, laid out like norm_add_fwd_any_kernel with
// two blocks of 128 columns to a warp, as many rows to a block as it has warps for:
// grad_weight's sums stay in registers over all rows of a block, whose teams' are added
// at the end (then norm_bwd_finish_kernel).  8191 x 1601 bf16: 35 us, 44 by whole
// 16-byte blocks shifted together (norm_bwd_kernel).
constexpr int kAnyBwdThreads = 1024;

template <typename T>
__global__ void __launch_bounds__(kAnyBwdThreads) norm_add_bwd_any_kernel(NormBwdArgs a) {
  extern __shared__ float team_sums[];  // [teams][D]
  __shared__ float red[2][kAnyBwdThreads / 32];
  constexpr int kBlocks = 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / a.team, w = warp - team * a.team;
  const int D = static_cast<int>(a.D);
  const float inv_n = 1.0f / static_cast<float>(D);
  auto column = [&](int b, int e) { return (w + b * a.team) * kBlock8 + e * 32 + lane; };
  float wt[kBlocks][4], dw[kBlocks][4];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = column(b, e);
      wt[b][e] = j < D ? weight_at(a.weight, a.w_f32, j, 1.0f) : 0.0f;
      dw[b][e] = 0.0f;
    }
  int parity = 0;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * a.teams + team; i < a.N;
       i += static_cast<int64_t>(gridDim.x) * a.teams, parity ^= 1) {
    const T* x = static_cast<const T*>(a.x) + i * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + i * a.lddy;
    const T* more = static_cast<const T*>(a.more) + i * a.ldmore;
    T* dx = static_cast<T*>(a.dx) + i * a.lddx;
    float h[kBlocks][4], u[kBlocks][4], m[kBlocks][4];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = column(b, e);
        h[b][e] = j < D ? Elem<T>::load(x + j) : 0.0f;
        u[b][e] = j < D ? Elem<T>::load(dy + j) : 0.0f;
        m[b][e] = j < D ? Elem<T>::load(more + j) : 0.0f;
      }
    const float rstd = a.rstd[i];
    float s[4] = {};
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[b][e] *= rstd;
        dw[b][e] = __fmaf_rn(u[b][e], h[b][e], dw[b][e]);
        u[b][e] *= wt[b][e];
        s[e] = __fmaf_rn(u[b][e], h[b][e], s[e]);
      }
    float total = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (a.team > 1) {
      if (lane == 0) red[parity][warp] = total;
      named_barrier(1 + team, a.team * 32);
      total = 0.0f;
      for (int k = 0; k < a.team; ++k) total += red[parity][team * a.team + k];
    }
    const float c = total * inv_n;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = column(b, e);
        if (j < D)
          Elem<T>::store(dx + j, __fmaf_rn(__fmaf_rn(-c, h[b][e], u[b][e]), rstd, m[b][e]));
      }
  }
  if (a.part == nullptr) return;
  // the teams' sums in team order
  __syncthreads();
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int j = column(b, e);
      if (j < D) team_sums[team * D + j] = dw[b][e];
    }
  __syncthreads();
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.D;
  for (int j = threadIdx.x; j < D; j += blockDim.x) {
    float t = 0.0f;
    for (int k = 0; k < a.teams; ++k) t += team_sums[k * D + j];
    part[j] = t;
  }
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
template <typename T, bool kQuant>
static int launch_norm_add_whole(NormAddArgs a, cudaStream_t s) {
  constexpr int kElems = kFwdLaneLong;
  if (a.D > int64_t(kFwdThreads<T>) * kElems) return 1;
  auto* kernel = norm_add_fwd_kernel<T, kElems, kQuant>;
  static std::atomic<uint64_t> raised{0};
  const int rc = raise_smem(kernel, kSmemMost, raised);
  if (rc != FLCE_OK) return rc;
  // (also without the 8 bits: the sums' order does not depend on the outputs asked for)
  const int least = kBlock8 * static_cast<int>(sizeof(T)) / 16;
  const NormPlan p = norm_plan(a.N, a.D, kElems, kFwdThreads<T>, least);
  a.team = p.team;
  a.teams = p.teams;
  const int threads = p.team * p.teams;
  const size_t smem = weight_bytes(a.D + kZeroWeights) +
                      2 * RowCopy<T, true, kElems>::bytes(threads, p.team);
  if (smem > kSmemMost) return 1;
  kernel<<<static_cast<unsigned>(p.blocks), threads, smem, s>>>(a);
  return launch_status("norm_add_fwd_kernel launch");
}

template <typename T, bool kQuant>
static int launch_norm_add(NormAddArgs a, int dt, cudaStream_t s) {
  auto aligned_rows = [dt](const void* p, int64_t ld) { return p == nullptr || whole(dt, p, ld); };
  if (aligned_rows(a.x, a.ldx) && aligned_rows(a.residual, a.ldr) &&
      aligned_rows(a.summed, a.lds) && aligned_rows(a.y, a.ldy) && whole(dt, nullptr, a.D)) {
    const int rc = launch_norm_add_whole<T, kQuant>(a, s);
    if (rc != 1) return rc;
  }
  // two blocks of 128 columns to a warp, or four
  for (int per = 2; per <= 4; per += 2) {
    const int64_t warps = (blocks8(a.D) + per - 1) / per;  // of a row
    if (warps > kAnyThreads / 32) continue;
    a.team = static_cast<int>(warps);
    a.teams = std::max(1, 8 / a.team);
    const int threads = 32 * a.team * a.teams;
    // as many blocks as there is room for, rows in turn
    const int64_t grid =
        std::min<int64_t>((a.N + a.teams - 1) / a.teams, sm_count() * (1024 / threads));
    auto* kernel =
        per == 2 ? norm_add_fwd_any_kernel<T, 2, kQuant> : norm_add_fwd_any_kernel<T, 4, kQuant>;
    kernel<<<static_cast<unsigned>(grid), threads, 0, s>>>(a);
    return launch_status("norm_add_fwd_any_kernel launch");
  }
  const int grid = static_cast<int>(std::min<int64_t>(a.N, sm_count() * 8));
  norm_add_fwd_long_kernel<T><<<grid, kLongThreads, 0, s>>>(a);
  return launch_status("norm_add_fwd_long_kernel launch");
}

// All rows that norm_bwd_kernel can hold: it is not there for those off 16-byte boundaries.
static_assert(kAnyBwdThreads / 32 * 2 * kBlock8 >= kBwdThreads<16> * 16 &&
                  kBwdThreads<16> * 16 >= kBwdThreads<8> * 8,
              "rows off 16-byte boundaries are held by norm_add_bwd_any_kernel");

// Launches norm_add_bwd_any_kernel; returns 1 (nothing launched) where rows begin on
// 16-byte boundaries or are too wide.  The arguments have been checked.
template <typename T>
static int launch_norm_add_bwd_any(NormBwdArgs a, int dt, cudaStream_t s) {
  const bool w = whole(dt, a.x, a.ldx) && whole(dt, a.dy, a.lddy) && whole(dt, a.dx, a.lddx) &&
                 whole(dt, a.more, a.ldmore) && whole(dt, nullptr, a.D);
  const int64_t warps = (blocks8(a.D) + 1) / 2;  // of a row
  if (w || warps > kAnyBwdThreads / 32) return 1;
  a.team = static_cast<int>(warps);
  // (teams of several warps have a hardware barrier each, of which there are 15)
  a.teams = a.team == 1 ? kAnyBwdThreads / 32 : std::min(15, kAnyBwdThreads / 32 / a.team);
  a.slices = std::min<int64_t>({(a.N + a.teams - 1) / a.teams, sm_count(), bwd_slices(a.N, a.D)});
  norm_add_bwd_any_kernel<T><<<static_cast<unsigned>(a.slices), 32 * a.team * a.teams,
                               sizeof(float) * a.teams * a.D, s>>>(a);
  if (a.dw != nullptr)
    norm_bwd_finish_kernel<<<static_cast<unsigned>((a.D + 31) / 32), 1024, 0, s>>>(a);
  return launch_status("norm_add_bwd_any_kernel launch");
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
  if (grad_summed == nullptr || grad_x == nullptr || N == 0)
    return rms_norm_bwd(summed, dt, N, D, lds, grad_y, ldgy, weight, wdt, rstd, grad_x, ldgx,
                        grad_weight, accumulate, ws, ws_bytes, stream);
  NormBwdArgs a{};
  a.x = summed, a.N = N, a.D = D, a.ldx = lds, a.dy = grad_y, a.lddy = ldgy;
  a.more = grad_summed, a.ldmore = ldgs, a.weight = weight, a.rstd = rstd;
  a.dx = grad_x, a.lddx = ldgx, a.dw = grad_weight, a.accumulate = accumulate;
  auto any = [](NormBwdArgs b, int dtype, cudaStream_t s) {
    return dtype == FLCE_BF16 ? launch_norm_add_bwd_any<__nv_bfloat16>(b, dtype, s)
                              : launch_norm_add_bwd_any<float>(b, dtype, s);
  };
  return norm_bwd<false, true>(a, dt, wdt, ws, ws_bytes, stream, any);
}
