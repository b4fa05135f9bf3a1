// Layer norm and RMS norm, forward and backward.
//
// Both are bound by the bytes of their rows, so a row is read once and stays in
// registers: a team of threads holds it, kLane elements to a thread, loads the
// next row before it works on this one, and sums by shuffles and one shared
// word per warp.  The square sum is taken around the mean from the registers.
// The threads' columns are the same for every row: the backward pass adds up its
// columns of grad_weight and grad_bias in registers (in shared memory for the widest rows) over all rows of a block;
// one partial sum per block, which norm_bwd_finish_kernel adds in block order.
//
// Each warp holds a run of 16-byte vectors of the row, wherever the row lies, and
// the roundings are written out, so the results do not depend on strides and
// alignment.  Rows that start inside 16-byte blocks (kWhole = false) are read by
// whole blocks all the same: a vector is shifted together from two blocks, the
// second of which a neighbour has brought into the L1 cache, and written the
// other way round with the neighbour's words; only the ends of a warp's run go
// element by element.  Bytes of a block outside the row are neither used nor
// written; a block with one byte of the row lies within mapped memory as a whole.
#include <algorithm>
#include <atomic>

#include "rows.cuh"

namespace flce {

constexpr int kLane = 16;              // elements of a row per thread
constexpr int kLaneLong = 32;          // in the forward of rows too long for that
// Most threads of a block, and of an SM: what the registers allow.
template <typename T>
constexpr int kFwdThreads = sizeof(T) == 2 ? 640 : 512;
constexpr int kFwdBlock = 256;
constexpr int kBwdThreads = 512;       // with the column sums in registers
constexpr int kBwdBlock = 256;
constexpr int kBwdThreadsWide = 1024;  // with the column sums in shared memory

// How a row is spread: `team` threads to a row (a power of two up to a warp,
// then whole warps), `teams` rows at a time in a block.
struct NormPlan {
  int team, teams;
  int64_t blocks;
};

static NormPlan norm_plan(int64_t N, int64_t D, int lane, int block, int sm_threads) {
  NormPlan p;
  const int64_t need = (D + lane - 1) / lane;
  if (need <= 32) {
    p.team = 1;
    while (p.team < need) p.team *= 2;
  } else {
    p.team = static_cast<int>((need + 31) / 32 * 32);
  }
  const int sms = sm_count();
  // blocks of about `block` threads, smaller ones while there are SMs without a row
  p.teams = std::max(1, block / p.team);
  while (p.teams > 1 && p.teams * p.team > 32 && (N + p.teams - 1) / p.teams < sms) p.teams /= 2;
  const int64_t most =
      static_cast<int64_t>(sms) * std::max(1, sm_threads / std::max(64, p.team * p.teams));
  p.blocks = std::max<int64_t>(1, std::min((N + p.teams - 1) / p.teams, most));
  return p;
}

// Sums of a and of b over the team; every thread returns the same values.
// `red`: one float2 per warp of the team (an even number of places), free again
// after the next call with another.
__device__ __forceinline__ void team_sum(float& a, float& b, int team, int id, float2* red) {
  if (team < 32) {
    for (int o = team / 2; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return;
  }
  // the lower half of the warp adds up a, the upper half b
  const int lane = threadIdx.x & 31;
  const bool upper = lane >= 16;
  float s = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (team == 32) {
    const float other = __shfl_xor_sync(0xffffffffu, s, 16);
    a = upper ? other : s;
    b = upper ? s : other;
    return;
  }
  const int warps = team >> 5, warp = (threadIdx.x - id * team) >> 5;
  if ((lane & 15) == 0) reinterpret_cast<float*>(red)[2 * warp + (upper ? 1 : 0)] = s;
  named_barrier(1 + id, team);
  float2 t = make_float2(0.0f, 0.0f);
#pragma unroll 4
  for (int w = 0; w < warps; w += 2) {
    const float4 v = *reinterpret_cast<const float4*>(red + w);
    t = __fadd2_rn(t, make_float2(v.x, v.y));
    if (w + 1 < warps) t = __fadd2_rn(t, make_float2(v.z, v.w));
  }
  a = t.x;
  b = t.y;
}

// Vectors of a thread: vector k of thread l of a team is k * team + l, so that
// the team's loads of one k lie next to each other (against runs of vectors per
// warp: 215 and 291 us for the layer norm of 65536 x 5120 bf16).
struct Spread {
  int team, l;
  __device__ __forceinline__ int at(int k) const { return k * team + l; }
};

// Words [S, S + 5) of a pair of blocks, shifted right by r bits (0 or 16).
template <int S>
__device__ __forceinline__ uint4 shifted(const uint4& lo, const uint4& hi, int r) {
  const uint32_t w[9] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w, 0u};
  return make_uint4(__funnelshift_r(w[S], w[S + 1], r), __funnelshift_r(w[S + 1], w[S + 2], r),
                    __funnelshift_r(w[S + 2], w[S + 3], r),
                    __funnelshift_r(w[S + 3], w[S + 4], r));
}

// The 16 bytes from byte `from` (0..16) of a pair of blocks on.
__device__ __forceinline__ uint4 bytes_from(const uint4& lo, const uint4& hi, int from) {
  const int r = (from & 2) * 8;
  switch (from >> 2) {
    case 0: return shifted<0>(lo, hi, r);
    case 1: return shifted<1>(lo, hi, r);
    case 2: return shifted<2>(lo, hi, r);
    case 3: return shifted<3>(lo, hi, r);
    default: return hi;
  }
}

// kElems elements of a row.
template <typename T, bool kWhole, int kElems>
struct RowRegs {
  static constexpr int VEC = 16 / sizeof(T), NV = kElems / VEC;
  uint4 v[NV];       // loaded blocks; after finish(): the row's vectors
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < NV; ++k) v[k] = make_uint4(0, 0, 0, 0);
  }
  // starts the loads of a row
  __device__ __forceinline__ void load(const T* p, int D, const Spread& s) {
    const char* base = reinterpret_cast<const char*>(p);
    if (!kWhole) base -= reinterpret_cast<uintptr_t>(p) & 15;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (s.at(k) * VEC < D) v[k] = reinterpret_cast<const uint4*>(base)[s.at(k)];
  }
  // the vectors themselves, zeros past the row's end
  __device__ __forceinline__ void finish(const T* p, int D, const Spread& s) {
    if (kWhole) return;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
    const uint4* base = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) - off);
    const int last = (off + D * static_cast<int>(sizeof(T)) - 1) / 16;  // the row's last block
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int left = D - s.at(k) * VEC;
      if (off != 0 && left > 0) v[k] = bytes_from(v[k], base[min(s.at(k) + 1, last)], off);
      if (left < VEC) {
        uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (sizeof(T) == 4) {
            if (q >= left) w[q] = 0u;
          } else {
            if (2 * q >= left) w[q] = 0u;
            if (2 * q + 1 >= left) w[q] &= 0xffffu;
          }
        }
        v[k] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  // vector k as pairs (for the packed fp32 instructions)
  __device__ __forceinline__ void unpack(int k, float2 (&x)[VEC / 2]) const {
    float f[VEC];
    Elem<T>::unpack(v[k], f);
#pragma unroll
    for (int e = 0; e < VEC / 2; ++e) x[e] = make_float2(f[2 * e], f[2 * e + 1]);
  }
};

// Writes the vector at columns j.. of a row (one per lane, all lanes of the warp
// take part).  A row inside a block: each lane writes the block that begins with
// its left neighbour's last elements, where the warp holds that neighbour and the
// row fills the block; what no such block covers goes element by element.
template <typename T, bool kWhole>
__device__ __forceinline__ void store_vector(T* row, int k, int D, const Spread& s,
                                             const float2 (&pairs)[8 / sizeof(T)]) {
  constexpr int VEC = 16 / sizeof(T);
  const int j = s.at(k) * VEC;
  float x[VEC];
#pragma unroll
  for (int e = 0; e < VEC / 2; ++e) x[2 * e] = pairs[e].x, x[2 * e + 1] = pairs[e].y;
  const uint4 own = Elem<T>::pack(x);
  if (kWhole) {
    if (j < D) *reinterpret_cast<uint4*>(row + j) = own;
    return;
  }
  uint4 left_of;
  left_of.x = __shfl_up_sync(0xffffffffu, own.x, 1);
  left_of.y = __shfl_up_sync(0xffffffffu, own.y, 1);
  left_of.z = __shfl_up_sync(0xffffffffu, own.z, 1);
  left_of.w = __shfl_up_sync(0xffffffffu, own.w, 1);
  const int left = D - j;  // elements of this vector (VEC or fewer, none when <= 0)
  if (left <= 0) return;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
  const int o = off / static_cast<int>(sizeof(T));
  const int lane = threadIdx.x & 31;
  const bool begins = lane == 0 || s.l == 0, ends = lane == 31 || s.l == s.team - 1;
  const bool head = (o == 0 || !begins) && left >= VEC - o;
  const bool tail = !ends && left >= 2 * VEC - o;  // in the right neighbour's block
  if (head)
    *reinterpret_cast<uint4*>(reinterpret_cast<char*>(row + j) - off) =
        bytes_from(left_of, own, 16 - off);
  if (!head || (!tail && o > 0)) {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < left && !(e < VEC - o ? head : tail)) Elem<T>::store(row + j + e, x[e]);
  }
}

// A weight vector in shared memory as fp32: of each row vector's VEC weights
// four together, the quarters of all vectors first, so that 16-byte reads of
// neighbouring threads lie next to each other.  Zeros past the end.
template <int VEC>
__device__ __forceinline__ void stage_weights(float4* to, const void* p, int f32, float other,
                                              int D) {
  const int nvec = (D + VEC - 1) / VEC;
  const bool wide = (reinterpret_cast<uintptr_t>(p) & 15) == 0;
#pragma unroll 4
  for (int c = threadIdx.x; c < nvec * (VEC / 4); c += blockDim.x) {
    const int j = 4 * c;
    float v[4];
    if (p != nullptr && wide && j + 4 <= D) {
      if (f32)
        load_as<float, 4>(static_cast<const float*>(p) + j, v);
      else
        load_as<__nv_bfloat16, 4>(static_cast<const __nv_bfloat16*>(p) + j, v);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = j + e < D ? other : 0.0f;
        if (p != nullptr && j + e < D)
          v[e] = f32 ? static_cast<const float*>(p)[j + e]
                     : Elem<__nv_bfloat16>::load(static_cast<const __nv_bfloat16*>(p) + j + e);
      }
    }
    to[c % (VEC / 4) * nvec + c / (VEC / 4)] = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// The weights of vector i.
template <int VEC>
__device__ __forceinline__ void weight_vec(const float4* w, int nvec, int i,
                                           float2 (&pairs)[VEC / 2]) {
#pragma unroll
  for (int q = 0; q < VEC / 4; ++q) {
    const float4 v = w[q * nvec + i];
    pairs[2 * q] = make_float2(v.x, v.y);
    pairs[2 * q + 1] = make_float2(v.z, v.w);
  }
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

template <int P>
__device__ __forceinline__ float sum_pairs(const float2 (&s)[P]) {
  float2 t = s[0];
#pragma unroll
  for (int e = 1; e < P; ++e) t = __fadd2_rn(t, s[e]);
  return __fadd_rn(t.x, t.y);
}

struct NormArgs {
  const void* x;
  int64_t N, D, ldx;
  const void* weight;
  const void* bias;
  int w_f32;
  float eps;
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
  int team, teams;
};

// A team works on kRows rows at a time (two, where threads of kLane elements can
// hold a row): one read of the weights and one exchange between its warps serve
// both.
template <typename T, bool kWhole, bool kCenter, int kElems, int kRows>
__global__ void __launch_bounds__(kFwdThreads<T>) norm_fwd_kernel(NormArgs a) {
  extern __shared__ float4 weights[];  // weight, then bias
  __shared__ __align__(16) float2 red_all[2][kFwdThreads<T> / 32 + 2];
  using Row = RowRegs<T, kWhole, kElems>;
  constexpr int VEC = Row::VEC, NV = Row::NV, P = VEC / 2;
  const int team = a.team, id = threadIdx.x / team, l = threadIdx.x - id * team;
  // an even number of places for each team
  float2* red0 = red_all[0] + (team > 32 ? id * ((team + 32) / 64 * 2) : 0);
  float2* red1 = red_all[1] + (team > 32 ? id * ((team + 32) / 64 * 2) : 0);
  // teams of one warp go on together
  const int lead = team < 32 ? (threadIdx.x & ~31) / team : id;
  const int64_t all = static_cast<int64_t>(gridDim.x) * a.teams;
  int64_t first = static_cast<int64_t>(blockIdx.x) * a.teams + lead;
  int64_t row = static_cast<int64_t>(blockIdx.x) * a.teams + id;  // and row + all
  const int D = static_cast<int>(a.D);
  const Spread spread{team, l};
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  Row next[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    next[r].clear();
    if (row + r * all < a.N) next[r].load(x + (row + r * all) * a.ldx, D, spread);
  }
  const int nvec = (D + VEC - 1) / VEC;
  const float4* bias = weights + nvec * (VEC / 4);
  stage_weights<VEC>(weights, a.weight, a.w_f32, 1.0f, D);
  if (kCenter) stage_weights<VEC>(weights + nvec * (VEC / 4), a.bias, a.w_f32, 0.0f, D);
  bool staged = false;  // the block's weights are there: needed late in the first row
  const float inv_n = 1.0f / static_cast<float>(D);
  for (; first < a.N; first += kRows * all) {
    float2 f[kRows][NV][P];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (row + r * all < a.N) next[r].finish(x + (row + r * all) * a.ldx, D, spread);
#pragma unroll
      for (int k = 0; k < NV; ++k) next[r].unpack(k, f[r][k]);
    }
    const int64_t here = row;
    row += kRows * all;
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (row + r * all < a.N) next[r].load(x + (row + r * all) * a.ldx, D, spread);
    // sums: a chain of additions for each place in a vector
    float mean[kRows] = {};
    if (kCenter) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float2 s[P];
#pragma unroll
        for (int e = 0; e < P; ++e) s[e] = f[r][0][e];
#pragma unroll
        for (int k = 1; k < NV; ++k)
#pragma unroll
          for (int e = 0; e < P; ++e) s[e] = __fadd2_rn(s[e], f[r][k][e]);
        mean[r] = sum_pairs(s);
      }
      float none = 0.0f;
      team_sum(mean[0], kRows > 1 ? mean[kRows - 1] : none, team, id, red0);
#pragma unroll
      for (int r = 0; r < kRows; ++r) mean[r] = __fmul_rn(mean[r], inv_n);
    }
    float rstd[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float2 q[P];
#pragma unroll
      for (int e = 0; e < P; ++e) q[e] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int j = spread.at(k) * VEC;
#pragma unroll
        for (int e = 0; e < P; ++e) {
          if (kCenter) f[r][k][e] = __fadd2_rn(f[r][k][e], both(-mean[r]));
          // past the row's end the elements are 0, less the mean: left out
          float2 d = f[r][k][e];
          if (!kWhole && kCenter) {
            if (j + 2 * e >= D) d.x = 0.0f;
            if (j + 2 * e + 1 >= D) d.y = 0.0f;
          }
          if (!kWhole || j < D) q[e] = __ffma2_rn(d, d, q[e]);
        }
      }
      rstd[r] = sum_pairs(q);
    }
    float none = 0.0f;
    team_sum(rstd[0], kRows > 1 ? rstd[kRows - 1] : none, team, id, red1);
#pragma unroll
    for (int r = 0; r < kRows; ++r) rstd[r] = rsqrtf(__fmaf_rn(rstd[r], inv_n, a.eps));
    if (!staged) __syncthreads();
    staged = true;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (spread.at(k) * VEC < D) {
        float2 w[P], b[P];
        weight_vec<VEC>(weights, nvec, spread.at(k), w);
        if (kCenter) weight_vec<VEC>(bias, nvec, spread.at(k), b);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const float2 h = __fmul2_rn(f[r][k][e], both(rstd[r]));
            f[r][k][e] = kCenter ? __ffma2_rn(h, w[e], b[e]) : __fmul2_rn(h, w[e]);
          }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const bool in_row = here + r * all < a.N;
        store_vector<T, kWhole>(y + (in_row ? here + r * all : 0) * a.ldy, k, in_row ? D : 0,
                                spread, f[r][k]);
      }
    }
    if (l == 0) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (here + r * all >= a.N) continue;
        if (kCenter && a.mean != nullptr) a.mean[here + r * all] = mean[r];
        if (a.rstd != nullptr) a.rstd[here + r * all] = rstd[r];
      }
    }
    if (!kCenter && team > 32) named_barrier(1 + id, team);  // red1 is free again
  }
  if (!staged) __syncthreads();  // warps without a row
}

struct NormBwdArgs {
  const void* x;
  int64_t N, D, ldx;
  const void* dy;
  int64_t lddy;
  const void* weight;
  int w_f32;
  const float* mean;
  const float* rstd;
  void* dx;
  int64_t lddx;
  float* dw;
  float* db;
  int accumulate;
  float* part;  // [slices][2][D]: the blocks' column sums
  int64_t slices;
  int team, teams;
};

// kWide: the column sums in shared memory, one row at a time in a block.
template <typename T, bool kWhole, bool kCenter, bool kWide>
__global__ void __launch_bounds__(kWide ? kBwdThreadsWide : kBwdThreads)
    norm_bwd_kernel(NormBwdArgs a) {
  // weight; column sums: teams * D (kWide: D) for grad_weight, as many for grad_bias
  extern __shared__ float4 weights[];
  __shared__ __align__(16) float2 red_all[2][kBwdThreadsWide / 32 + 2];
  using Row = RowRegs<T, kWhole, kLane>;
  constexpr int VEC = Row::VEC, NV = Row::NV, P = VEC / 2;
  const int team = a.team, id = threadIdx.x / team, l = threadIdx.x - id * team;
  const int lead = team < 32 ? (threadIdx.x & ~31) / team : id;
  const int64_t step = static_cast<int64_t>(gridDim.x) * a.teams;
  int64_t first = static_cast<int64_t>(blockIdx.x) * a.teams + lead;
  int64_t row = static_cast<int64_t>(blockIdx.x) * a.teams + id;
  const int D = static_cast<int>(a.D);
  const T* xr = static_cast<const T*>(a.x) + (row < a.N ? row : 0) * a.ldx;
  const T* gr = static_cast<const T*>(a.dy) + (row < a.N ? row : 0) * a.lddy;
  const Spread spread{team, l};
  T* dxr = static_cast<T*>(a.dx) + (row < a.N ? row : 0) * a.lddx;
  const int nvec = (D + VEC - 1) / VEC;
  float* sums = reinterpret_cast<float*>(weights + nvec * (VEC / 4));
  Row nx, ng;
  float nmean = 0.0f, nrstd = 0.0f;
  nx.clear();
  ng.clear();
  auto prefetch = [&]() {
    if (row >= a.N) return;
    nx.load(xr, D, spread);
    ng.load(gr, D, spread);
    nrstd = a.rstd[row];
    if (kCenter) nmean = a.mean[row];
  };
  if (!kWide) prefetch();
  stage_weights<VEC>(weights, a.weight, a.w_f32, 1.0f, D);
  float2 dw[NV][P] = {}, db[NV][P] = {};
  if (kWide) {
    for (int j = threadIdx.x; j < (kCenter ? 2 : 1) * nvec * VEC; j += blockDim.x) sums[j] = 0.0f;
  }
  __syncthreads();
  const float inv_n = 1.0f / static_cast<float>(D);
  int parity = 0;
  for (; first < a.N; first += step) {
    if (kWide) prefetch();  // no registers for a second row
    const bool in_row = row < a.N;
    const float mean = nmean, rstd = nrstd;
    if (in_row) {
      nx.finish(xr, D, spread);
      ng.finish(gr, D, spread);
    } else {
      ng.clear();  // adds nothing to the column sums
    }
    float2 h[NV][P], u[NV][P];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      nx.unpack(k, h[k]);
      ng.unpack(k, u[k]);
    }
    row += step;
    if (row < a.N) xr += step * a.ldx, gr += step * a.lddy;
    if (!kWide) prefetch();
    float2 s1[P], s2[P];  // a chain of additions for each place in a vector
#pragma unroll
    for (int e = 0; e < P; ++e) s1[e] = s2[e] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = spread.at(k) * VEC;
      if (j >= D) continue;
      float2 w[P];
      weight_vec<VEC>(weights, nvec, spread.at(k), w);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        // past the row's end the incoming gradient is 0, and so are all sums
        if (kCenter) h[k][e] = __fadd2_rn(h[k][e], both(-mean));
        h[k][e] = __fmul2_rn(h[k][e], both(rstd));
        const float2 g = u[k][e];
        u[k][e] = __fmul2_rn(g, w[e]);
        if (kCenter) s1[e] = __fadd2_rn(s1[e], u[k][e]);
        s2[e] = __ffma2_rn(u[k][e], h[k][e], s2[e]);
        if (kWide) {
          // pairs of the vector's quarters, laid out as the weights
          float2* to = reinterpret_cast<float2*>(sums + 4 * ((e / 2) * nvec + spread.at(k))) +
                       (e & 1);
          *to = __ffma2_rn(g, h[k][e], *to);
          if (kCenter) {
            to += 2 * nvec * (VEC / 4);
            *to = __fadd2_rn(*to, g);
          }
        } else {
          dw[k][e] = __ffma2_rn(g, h[k][e], dw[k][e]);
          if (kCenter) db[k][e] = __fadd2_rn(db[k][e], g);
        }
      }
    }
    float c1 = sum_pairs(s1), c2 = sum_pairs(s2);
    team_sum(c2, c1, team, id,
             red_all[parity] + (team > 32 ? id * ((team + 32) / 64 * 2) : 0));
    parity ^= 1;
    if (a.dx == nullptr) continue;
    c1 = __fmul_rn(c1, inv_n);
    c2 = __fmul_rn(c2, inv_n);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int e = 0; e < P; ++e) {
        float2 t = u[k][e];
        if (kCenter) t = __fadd2_rn(t, both(-c1));
        t = __ffma2_rn(h[k][e], both(-c2), t);
        u[k][e] = __fmul2_rn(t, both(rstd));
      }
      store_vector<T, kWhole>(dxr, k, in_row ? D : 0, spread, u[k]);
    }
    if (row < a.N) dxr += step * a.lddx;
  }
  if (a.part == nullptr) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.D;
  if (!kWide) {
    // the teams' sums side by side, then in team order
    float* to = a.teams == 1 ? part : sums + id * D;
    const int64_t bias_at = static_cast<int64_t>(a.teams) * D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int j = spread.at(k) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (j + e >= D) continue;
        to[j + e] = (e & 1) ? dw[k][e / 2].y : dw[k][e / 2].x;
        if (kCenter) to[bias_at + j + e] = (e & 1) ? db[k][e / 2].y : db[k][e / 2].x;
      }
    }
    if (a.teams == 1) return;
  }
  __syncthreads();
  for (int64_t j = threadIdx.x; j < (kCenter ? 2 : 1) * a.D; j += blockDim.x) {
    const int64_t which = j / a.D, c = j - which * a.D;
    float s = 0.0f;
    if (kWide) {
      const int i = static_cast<int>(c) / VEC, e = static_cast<int>(c) % VEC;
      s = sums[4 * (which * nvec * (VEC / 4) + (e / 4) * nvec + i) + e % 4];
    } else {
      for (int t = 0; t < a.teams; ++t) s += sums[(which * a.teams + t) * a.D + c];
    }
    part[j] = s;
  }
}

// ------------------------------------------------------------ rows too wide to hold

constexpr int kLongThreads = 256;

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < kLongThreads / 32; ++w) s += red[w];
  __syncthreads();
  return s;
}

__device__ __forceinline__ float weight_at(const void* p, int f32, int64_t j, float other) {
  if (p == nullptr) return other;
  return f32 ? static_cast<const float*>(p)[j]
             : Elem<__nv_bfloat16>::load(static_cast<const __nv_bfloat16*>(p) + j);
}

// One block per row, the row read again for each pass.
template <typename T, bool kCenter>
__global__ void __launch_bounds__(kLongThreads) norm_fwd_long_kernel(NormArgs a) {
  __shared__ float red[kLongThreads / 32];
  for (int64_t i = blockIdx.x; i < a.N; i += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + i * a.ldx;
    T* y = static_cast<T*>(a.y) + i * a.ldy;
    float mean = 0.0f;
    if (kCenter) {
      float s = 0.0f;
      for (int64_t j = threadIdx.x; j < a.D; j += kLongThreads) s += Elem<T>::load(x + j);
      mean = block_sum(s, red) / static_cast<float>(a.D);
    }
    float q = 0.0f;
    for (int64_t j = threadIdx.x; j < a.D; j += kLongThreads) {
      const float d = Elem<T>::load(x + j) - mean;
      q += d * d;
    }
    const float rstd = 1.0f / sqrtf(block_sum(q, red) / static_cast<float>(a.D) + a.eps);
    for (int64_t j = threadIdx.x; j < a.D; j += kLongThreads) {
      float v = (Elem<T>::load(x + j) - mean) * rstd * weight_at(a.weight, a.w_f32, j, 1.0f);
      if (kCenter) v += weight_at(a.bias, a.w_f32, j, 0.0f);
      Elem<T>::store(y + j, v);
    }
    if (threadIdx.x == 0) {
      if (kCenter && a.mean != nullptr) a.mean[i] = mean;
      if (a.rstd != nullptr) a.rstd[i] = rstd;
    }
  }
}

template <typename T, bool kCenter>
__global__ void __launch_bounds__(kLongThreads) norm_bwd_long_kernel(NormBwdArgs a) {
  __shared__ float red[kLongThreads / 32];
  for (int64_t i = blockIdx.x; i < a.N; i += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + i * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + i * a.lddy;
    T* dx = static_cast<T*>(a.dx) + i * a.lddx;
    const float mean = kCenter ? a.mean[i] : 0.0f, rstd = a.rstd[i];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t j = threadIdx.x; j < a.D; j += kLongThreads) {
      const float u = Elem<T>::load(dy + j) * weight_at(a.weight, a.w_f32, j, 1.0f);
      s1 += u;
      s2 += u * ((Elem<T>::load(x + j) - mean) * rstd);
    }
    const float c1 = kCenter ? block_sum(s1, red) / static_cast<float>(a.D) : 0.0f;
    const float c2 = block_sum(s2, red) / static_cast<float>(a.D);
    for (int64_t j = threadIdx.x; j < a.D; j += kLongThreads) {
      const float u = Elem<T>::load(dy + j) * weight_at(a.weight, a.w_f32, j, 1.0f);
      const float h = (Elem<T>::load(x + j) - mean) * rstd;
      Elem<T>::store(dx + j, rstd * (u - c1 - h * c2));
    }
  }
}

// Column sums of one slice of the rows, 256 columns per block; before
// norm_bwd_long_kernel, which may overwrite dy.
template <typename T, bool kCenter>
__global__ void __launch_bounds__(kLongThreads) norm_bwd_long_cols_kernel(NormBwdArgs a) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kLongThreads + threadIdx.x;
  if (j >= a.D) return;
  const int64_t per = (a.N + a.slices - 1) / a.slices;
  const int64_t i0 = min(a.N, blockIdx.y * per), i1 = min(a.N, i0 + per);
  float dw = 0.0f, db = 0.0f;
  for (int64_t i = i0; i < i1; ++i) {
    const float g = Elem<T>::load(static_cast<const T*>(a.dy) + i * a.lddy + j);
    const float x = Elem<T>::load(static_cast<const T*>(a.x) + i * a.ldx + j);
    dw += g * ((x - (kCenter ? a.mean[i] : 0.0f)) * a.rstd[i]);
    db += g;
  }
  a.part[(2 * static_cast<int64_t>(blockIdx.y)) * a.D + j] = dw;
  if (kCenter) a.part[(2 * static_cast<int64_t>(blockIdx.y) + 1) * a.D + j] = db;
}

// ---------------------------------------------------------------- column sums

// 32 columns per block: 32 warps add up every 32nd slice, then the warps' sums
// in warp order.  blockIdx.y: grad_weight, grad_bias.
__global__ void __launch_bounds__(1024) norm_bwd_finish_kernel(NormBwdArgs a) {
  __shared__ float red[32][33];
  float* out = blockIdx.y == 0 ? a.dw : a.db;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (j < a.D) {
#pragma unroll 8
    for (int64_t k = warp; k < a.slices; k += 32) s += a.part[(2 * k + blockIdx.y) * a.D + j];
  }
  red[warp][lane] = s;
  __syncthreads();
  // warp w: the 32 sums of column w
  s = red[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane == 0 && c < a.D) out[c] = a.accumulate ? out[c] + s : s;
}

// ------------------------------------------------------------------------ host

// Whether the rows of a matrix start on 16-byte boundaries.
static bool whole(int dt, const void* p, int64_t ld) {
  return aligned(p, 16) && ld % (dt == FLCE_BF16 ? 8 : 4) == 0;
}

// A weight vector in shared memory, to whole row vectors.
static size_t weight_bytes(int64_t D) { return round_up(static_cast<size_t>(D), 8) * 4; }

constexpr int kSmemMost = 224 * 1024;

// Allows a kernel kSmemMost bytes of shared memory, once per device.
template <typename K>
static int raise_smem(K kern, std::atomic<uint64_t>& raised) {
  int dev = 0;
  int rc = cuda_status(cudaGetDevice(&dev), "cudaGetDevice");
  if (rc != FLCE_OK) return rc;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(raised.load() & bit)) {
    rc = cuda_status(
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost),
        "cudaFuncSetAttribute(norm kernel)");
    if (rc == FLCE_OK) raised.fetch_or(bit);
  }
  return rc;
}

template <typename T, bool kWhole, bool kCenter, int kElems, int kRows>
static int launch_norm_fwd_k(NormArgs a, cudaStream_t s) {
  static std::atomic<uint64_t> raised{0};
  const int rc = raise_smem(norm_fwd_kernel<T, kWhole, kCenter, kElems, kRows>, raised);
  if (rc != FLCE_OK) return rc;
  const NormPlan p = norm_plan(a.N, a.D, kElems, kFwdBlock, kFwdThreads<T>);
  a.team = p.team;
  a.teams = p.teams;
  const size_t smem = weight_bytes(a.D) * (kCenter ? 2 : 1);
  norm_fwd_kernel<T, kWhole, kCenter, kElems, kRows>
      <<<static_cast<unsigned>(p.blocks), p.team * p.teams, smem, s>>>(a);
  return launch_status("norm_fwd_kernel launch");
}

template <typename T, bool kCenter>
static int launch_norm_fwd(NormArgs a, int dt, cudaStream_t s) {
  const bool w = whole(dt, a.x, a.ldx) && whole(dt, a.y, a.ldy) && whole(dt, nullptr, a.D);
  if (a.D <= int64_t(kFwdThreads<T>) * kLane)
    return w ? launch_norm_fwd_k<T, true, kCenter, kLane, 2>(a, s)
             : launch_norm_fwd_k<T, false, kCenter, kLane, 2>(a, s);
  if (a.D <= int64_t(kFwdThreads<T>) * kLaneLong)
    return w ? launch_norm_fwd_k<T, true, kCenter, kLaneLong, 1>(a, s)
             : launch_norm_fwd_k<T, false, kCenter, kLaneLong, 1>(a, s);
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
                 : overlap(a.x, span_bytes(a.N, a.D, a.ldx, es), a.y,
                           span_bytes(a.N, a.D, a.ldy, es)))
    return FLCE_EINVAL;
  if (a.N == 0) return FLCE_OK;
  a.w_f32 = wdt == FLCE_F32;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dt == FLCE_BF16 ? launch_norm_fwd<__nv_bfloat16, kCenter>(a, dt, s)
                         : launch_norm_fwd<float, kCenter>(a, dt, s);
}

// Column sums in registers, in shared memory, or by kernels of their own.
static bool bwd_narrow(int64_t D) { return D <= int64_t(kBwdThreads) * kLane; }
static bool bwd_held(int64_t D) { return D <= int64_t(kBwdThreadsWide) * kLane; }

static int64_t bwd_slices(int64_t N, int64_t D) {
  if (bwd_held(D)) return norm_plan(N, D, kLane, kBwdBlock, kBwdThreads).blocks;
  return std::min<int64_t>(64, N);
}

template <typename T, bool kWhole, bool kCenter>
static int launch_norm_bwd_held(NormBwdArgs a, cudaStream_t s) {
  const NormPlan p = norm_plan(a.N, a.D, kLane, kBwdBlock, kBwdThreads);
  a.team = p.team;
  a.teams = p.teams;
  const unsigned grid = static_cast<unsigned>(p.blocks);
  const int threads = p.team * p.teams;
  const size_t per = static_cast<size_t>(a.D) * sizeof(float) * (kCenter ? 2 : 1);
  const size_t w = weight_bytes(a.D);
  if (bwd_narrow(a.D)) {
    static std::atomic<uint64_t> raised{0};
    const int rc = raise_smem(norm_bwd_kernel<T, kWhole, kCenter, false>, raised);
    if (rc != FLCE_OK) return rc;
    const size_t smem = w + (p.teams > 1 ? p.teams * per : 0);
    norm_bwd_kernel<T, kWhole, kCenter, false><<<grid, threads, smem, s>>>(a);
  } else {
    static std::atomic<uint64_t> raised{0};
    const int rc = raise_smem(norm_bwd_kernel<T, kWhole, kCenter, true>, raised);
    if (rc != FLCE_OK) return rc;
    norm_bwd_kernel<T, kWhole, kCenter, true>
        <<<grid, threads, w * (kCenter ? 3 : 2), s>>>(a);
  }
  return launch_status("norm_bwd_kernel launch");
}

template <typename T, bool kCenter>
static int launch_norm_bwd(NormBwdArgs a, int dt, cudaStream_t s) {
  if (a.N > 0 && bwd_held(a.D)) {
    const bool w = whole(dt, a.x, a.ldx) && whole(dt, a.dy, a.lddy) &&
                   whole(dt, a.dx, a.dx != nullptr ? a.lddx : 0) && whole(dt, nullptr, a.D);
    const int rc = w ? launch_norm_bwd_held<T, true, kCenter>(a, s)
                     : launch_norm_bwd_held<T, false, kCenter>(a, s);
    if (rc != FLCE_OK) return rc;
  } else if (a.N > 0) {
    if (a.part != nullptr) {
      const dim3 g(static_cast<unsigned>((a.D + kLongThreads - 1) / kLongThreads),
                   static_cast<unsigned>(a.slices));
      norm_bwd_long_cols_kernel<T, kCenter><<<g, kLongThreads, 0, s>>>(a);
    }
    if (a.dx != nullptr) {
      const int grid = static_cast<int>(std::min<int64_t>(a.N, sm_count() * 8));
      norm_bwd_long_kernel<T, kCenter><<<grid, kLongThreads, 0, s>>>(a);
    }
  }
  if (a.dw != nullptr || a.db != nullptr) {
    const dim3 g(static_cast<unsigned>((a.D + 31) / 32), a.db != nullptr ? 2 : 1);
    norm_bwd_finish_kernel<<<g, 1024, 0, s>>>(a);
  }
  return launch_status("norm_bwd launch");
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
  a.part = cols ? static_cast<float*>(ws) : nullptr;
  a.slices = a.N > 0 ? bwd_slices(a.N, a.D) : 0;
  a.w_f32 = wdt == FLCE_F32;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dt == FLCE_BF16 ? launch_norm_bwd<__nv_bfloat16, kCenter>(a, dt, s)
                         : launch_norm_bwd<float, kCenter>(a, dt, s);
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
  return norm_bwd<true>(a, dt, wdt, ws, ws_bytes, stream);
}

extern "C" int rms_norm_bwd(const void* x, int dt, int64_t N, int64_t D, int64_t ldx,
                            const void* grad_y, int64_t ldgy, const void* weight, int wdt,
                            const float* rstd, void* grad_x, int64_t ldgx, float* grad_weight,
                            int accumulate, void* ws, size_t ws_bytes, flce_stream_t stream) {
  NormBwdArgs a{};
  a.x = x, a.N = N, a.D = D, a.ldx = ldx, a.dy = grad_y, a.lddy = ldgy, a.weight = weight;
  a.rstd = rstd, a.dx = grad_x, a.lddx = ldgx, a.dw = grad_weight, a.accumulate = accumulate;
  return norm_bwd<false>(a, dt, wdt, ws, ws_bytes, stream);
}
