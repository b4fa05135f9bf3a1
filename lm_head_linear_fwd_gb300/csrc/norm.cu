// Layer norm and RMS norm, forward and backward.
//
// Both are bound by the bytes of their rows, so a row is read once and stays in
// registers: a team of threads holds it, a few 16-byte vectors to a thread, and
// sums by shuffles and one shared word per warp.  The square sum is taken around
// the mean from the registers.  What the memory needs is bytes in flight: each
// thread copies its own vectors of the next rows to shared memory (cp.async, no
// barrier: it reads back what it copied), which costs no registers.  A thread's
// columns are the same for every row: the backward pass adds up its columns of
// grad_weight and grad_bias in registers over all rows of a block; one partial
// sum per block, which norm_bwd_finish_kernel adds in block order.
//
// Vector k of thread l of a team is k * team + l, wherever the row lies, and the
// roundings are written out, so the results do not depend on strides and
// alignment.  Rows that start inside 16-byte blocks (kWhole = false) are read by
// whole blocks all the same: a vector is shifted together from its own block and
// its right neighbour's, and written the other way round with the left
// neighbour's words; only the ends of a warp's vectors go element by element.
// Bytes of a block outside the row are neither used nor written; a block with one
// byte of the row lies within mapped memory as a whole.
#include <algorithm>

#include "rows.cuh"

namespace flce {

// Elements of a row per thread in the forward, where two rows at a time or one
// fit the registers.
constexpr int kFwdLane = 16, kFwdLaneLong = 32;
constexpr int kBlock = 512;      // threads of a block, where a team is not larger
// Most threads of a block, and of an SM: what registers and shared memory allow.
template <typename T>
constexpr int kFwdThreads = sizeof(T) == 2 ? 640 : 512;
template <int kElems>
constexpr int kBwdThreads = kElems == 8 ? 640 : 512;
constexpr int kSmemMost = 224 * 1024;  // beside the static sums of a team

// How a row is spread: `team` threads to a row (a power of two up to a warp,
// then whole warps), `teams` rows at a time in a block.
struct NormPlan {
  int team, teams;
  int64_t blocks;
};

static NormPlan norm_plan(int64_t N, int64_t D, int lane, int sm_threads) {
  NormPlan p;
  const int64_t need = (D + lane - 1) / lane;
  if (need <= 32) {
    p.team = 1;
    while (p.team < need) p.team *= 2;
  } else {
    p.team = static_cast<int>((need + 31) / 32 * 32);
  }
  const int sms = sm_count();
  // blocks of about kBlock threads, smaller ones while there are SMs without a row
  p.teams = std::max(1, kBlock / p.team);
  while (p.teams > 1 && p.teams * p.team > 32 && (N + p.teams - 1) / p.teams < sms) p.teams /= 2;
  const int64_t most =
      static_cast<int64_t>(sms) * std::max(1, sm_threads / std::max(64, p.team * p.teams));
  p.blocks = std::max<int64_t>(1, std::min((N + p.teams - 1) / p.teams, most));
  return p;
}

// The threads that hold a row, and this thread's place among them.
struct Team {
  int size, id, l;     // threads; which team of the block; which thread of it
  int mine;            // how many of the thread's vectors begin within the row
  bool first, last;    // no left, no right neighbour within the warp
  float2* red[2];      // a pair of sums for each warp, places to a multiple of eight
  int warp;
  __device__ __forceinline__ Team(int size, int nvec, float2* pairs, int kind)
      : size(size), id(threadIdx.x / size), l(threadIdx.x - id * size) {
    mine = (nvec - l + size - 1) / size;
    first = l == 0 || (threadIdx.x & 31) == 0;
    last = l == size - 1 || (threadIdx.x & 31) == 31;
    warp = l >> 5;
    const int warps = size >> 5, places = (warps + 7) / 8 * 8;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      red[q] = pairs + q * kind + (size > 32 ? id * places : 0);
      if (size > 32)
        for (int w = warps + l; w < places; w += size) red[q][w] = make_float2(0.0f, 0.0f);
    }
  }
  // Vector k of the thread is vector at(k) of the row: the team's vectors of one k
  // lie next to each other (against runs of vectors per warp: 215 and 291 us for
  // the layer norm of 65536 x 5120 bf16).
  __device__ __forceinline__ int at(int k) const { return k * size + l; }

  // Sums of a and of b over the team; every thread returns the same.  Two calls
  // in a row use different q.
  __device__ __forceinline__ void sum(float& a, float& b, int q) const {
    if (size < 32) {
      for (int o = size / 2; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
      }
      return;
    }
    // the lower half of the warp adds up a, the upper half b
    const bool upper = (threadIdx.x & 16) != 0;
    float s = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (size == 32) {
      const float other = __shfl_xor_sync(0xffffffffu, s, 16);
      a = upper ? other : s;
      b = upper ? s : other;
      return;
    }
    float2* r = red[q];
    if ((threadIdx.x & 15) == 0) reinterpret_cast<float*>(r + warp)[upper ? 1 : 0] = s;
    named_barrier(1 + id, size);
    float2 t = make_float2(0.0f, 0.0f);
    for (int w = 0; w < size; w += 256, r += 8) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float4 v = *reinterpret_cast<const float4*>(r + k);
        t = __fadd2_rn(t, make_float2(v.x, v.y));
        t = __fadd2_rn(t, make_float2(v.z, v.w));
      }
    }
    a = t.x;
    b = t.y;
  }
};

// Places of all teams of a block: teams of two warps or more take eight each.
template <int kThreads>
constexpr int kRedPlaces = kThreads / 64 * 8 + 8;

// How many of the rows first, first + step, ... there are.
__device__ __forceinline__ int rows_from(int64_t first, int64_t step, int64_t N) {
  return static_cast<int>(max(int64_t(0), N - first + step - 1) / step);
}

// A row pointer that a thread moves on by a fixed step.  Whole rows: at the
// thread's first vector, others: at the row.  The step is kept in registers (it
// would be multiplied out again for every row).
template <typename T, bool kWhole>
struct RowPtr {
  char* p;
  int64_t step;
  __device__ __forceinline__ RowPtr(const void* base, int64_t row, int64_t ld, int64_t rows, int l)
      : p(static_cast<char*>(const_cast<void*>(base)) +
          row * ld * static_cast<int64_t>(sizeof(T)) + (kWhole ? 16 * l : 0)),
        step(rows * ld * static_cast<int64_t>(sizeof(T))) {
    asm volatile("" : "+l"(step));
  }
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

// A thread's places for one row in shared memory: vector k at k * blockDim * 16;
// kWhole = false: after them, for each thread without a right neighbour in its
// warp, the blocks after its own.
template <typename T, bool kWhole, int kElems>
struct RowCopy {
  static constexpr int VEC = 16 / sizeof(T), NV = kElems / VEC;
  // threads of a block without a right neighbour in their warp
  static __host__ __device__ __forceinline__ int ends(int threads, int team) {
    return threads / (team < 32 ? team : 32);
  }
  static __host__ __device__ __forceinline__ int bytes(int threads, int team) {
    return NV * 16 * (threads + (kWhole ? 0 : ends(threads, team)));
  }
  char* own;
  char* end;
  int pitch, end_pitch;
  __device__ __forceinline__ RowCopy(char* place, const Team& t)
      : own(place + threadIdx.x * 16),
        end(place + NV * blockDim.x * 16 + threadIdx.x / (t.size < 32 ? t.size : 32) * 16),
        pitch(blockDim.x * 16),
        end_pitch(ends(blockDim.x, t.size) * 16) {}
  // starts the copies of the row at p (see RowPtr)
  __device__ __forceinline__ void start(const char* p, int D, const Team& t) const {
    const uint32_t to = smem_u32(own);
    if (kWhole) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (k < t.mine) cp_async16(to + k * pitch, p + k * t.size * 16);
    } else {
      const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
      const int last = (off + D * static_cast<int>(sizeof(T)) - 1) / 16;  // the row's last block
      const char* from = p - off + 16 * t.l;
      const uint32_t to_end = smem_u32(end);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (t.at(k) <= last) cp_async16(to + k * pitch, from + k * t.size * 16);
        if (t.last && t.at(k) < last)
          cp_async16(to_end + k * end_pitch, from + k * t.size * 16 + 16);
      }
    }
  }
  // zeros in the place of a row, or where no row is copied to
  __device__ __forceinline__ void clear(bool row, const Team& t) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (row || (kWhole && k >= t.mine))
        *reinterpret_cast<uint4*>(own + k * pitch) = make_uint4(0, 0, 0, 0);
      if (!kWhole && row && t.last)
        *reinterpret_cast<uint4*>(end + k * end_pitch) = make_uint4(0, 0, 0, 0);
    }
  }
  // the row's vectors as pairs (for the packed fp32 instructions), zeros past its end
  __device__ __forceinline__ void read(const char* p, int D, const Team& t,
                                       float2 (&x)[NV][VEC / 2]) const {
    const int off = kWhole ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      // (whole rows: places past the row's end were cleared and are never written)
      uint4 v = *reinterpret_cast<const uint4*>(own + k * pitch);
      if (!kWhole) {
        const uint4 right = *reinterpret_cast<const uint4*>(
            t.last ? end + k * end_pitch : own + k * pitch + 16);
        v = bytes_from(v, right, off);
        const int left = D - t.at(k) * VEC;
        if (left < VEC) {
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (sizeof(T) == 4) {
              if (q >= left) w[q] = 0u;
            } else {
              if (2 * q >= left) w[q] = 0u;
              if (2 * q + 1 >= left) w[q] &= 0xffffu;
            }
          }
          v = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      float f[VEC];
      Elem<T>::unpack(v, f);
#pragma unroll
      for (int e = 0; e < VEC / 2; ++e) x[k][e] = make_float2(f[2 * e], f[2 * e + 1]);
    }
  }
};

// Writes the vector k of a row (one per lane, all lanes of the warp take part).  A
// row inside a block: each lane writes the block that begins with its left
// neighbour's last elements, where the warp holds that neighbour and the row
// fills the block; what no such block covers goes element by element.
template <typename T, bool kWhole>
__device__ __forceinline__ void store_vector(char* p, int k, bool in_row, int D, const Team& t,
                                             const float2 (&pairs)[8 / sizeof(T)]) {
  constexpr int VEC = 16 / sizeof(T);
  float x[VEC];
#pragma unroll
  for (int e = 0; e < VEC / 2; ++e) x[2 * e] = pairs[e].x, x[2 * e + 1] = pairs[e].y;
  const uint4 own = Elem<T>::pack(x);
  if (kWhole) {
    if (in_row && k < t.mine) *reinterpret_cast<uint4*>(p + k * t.size * 16) = own;
    return;
  }
  uint4 left_of;
  left_of.x = __shfl_up_sync(0xffffffffu, own.x, 1);
  left_of.y = __shfl_up_sync(0xffffffffu, own.y, 1);
  left_of.z = __shfl_up_sync(0xffffffffu, own.z, 1);
  left_of.w = __shfl_up_sync(0xffffffffu, own.w, 1);
  T* row = reinterpret_cast<T*>(p);
  const int j = t.at(k) * VEC;
  const int left = in_row ? D - j : 0;  // elements of this vector (VEC or fewer)
  if (left <= 0) return;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
  const int o = off / static_cast<int>(sizeof(T));
  const bool head = (o == 0 || !t.first) && left >= VEC - o;
  const bool tail = !t.last && left >= 2 * VEC - o;  // in the right neighbour's block
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

// A team works on kRows rows at a time (two, where threads of kFwdLane
// elements can hold a row): one read of the weights and one exchange between its warps serve
// both.  Layer norm 65536 x 5120 bf16: 209 us (6.4 TB/s); RMS norm 8192 x 4096 fp32:
// 44 us (6.0 TB/s); rows of 1601 that start inside blocks, 8191 of them: 28 us, of 1600 14.
template <typename T, bool kWhole, bool kCenter, int kElems, int kRows>
__global__ void __launch_bounds__(kFwdThreads<T>) norm_fwd_kernel(NormArgs a) {
  extern __shared__ float4 weights[];  // weight, then bias, then the rows' copies
  constexpr int kPlaces = kRedPlaces<kFwdThreads<T>>;
  __shared__ __align__(16) float2 red[2 * kPlaces];
  using Copy = RowCopy<T, kWhole, kElems>;
  constexpr int VEC = Copy::VEC, NV = Copy::NV, P = VEC / 2;
  const int D = static_cast<int>(a.D);
  const int nvec = (D + VEC - 1) / VEC;
  const Team team(a.team, nvec, red, kPlaces);
  const int64_t all = static_cast<int64_t>(gridDim.x) * a.teams;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * a.teams + team.id;  // then row + all, ...
  int rows = rows_from(row, all, a.N);  // of this team, and of the warp's first one
  int turns = a.team < 32 ? __shfl_sync(0xffffffffu, rows, 0) : rows;
  RowPtr<T, kWhole> x(a.x, row, a.ldx, all, team.l), y(a.y, row, a.ldy, all, team.l);
  float* mean_out = a.mean != nullptr ? a.mean + row : nullptr;
  float* rstd_out = a.rstd != nullptr ? a.rstd + row : nullptr;
  char* places = reinterpret_cast<char*>(weights + (kCenter ? 2 : 1) * nvec * (VEC / 4));
  const int row_bytes = Copy::bytes(blockDim.x, a.team);
  const Copy copy[2] = {Copy(places, team), Copy(places + (kRows - 1) * row_bytes, team)};
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    copy[r].clear(false, team);
    if (r < rows) copy[r].start(x.p + r * x.step, D, team);
  }
  cp_async_commit();
  const float4* bias = weights + nvec * (VEC / 4);
  stage_weights<VEC>(weights, a.weight, a.w_f32, 1.0f, D);
  if (kCenter) stage_weights<VEC>(weights + nvec * (VEC / 4), a.bias, a.w_f32, 0.0f, D);
  bool staged = false;  // the block's weights are there: needed late in the first row
  const float inv_n = 1.0f / static_cast<float>(D);
  for (; turns > 0; turns -= kRows, rows -= kRows) {
    float2 f[kRows][NV][P];
    cp_async_wait<0>();
    if (!kWhole) __syncwarp();  // the right neighbour's blocks
#pragma unroll
    for (int r = 0; r < kRows; ++r) copy[r].read(x.p + r * x.step, D, team, f[r]);
    x.p += kRows * x.step;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (kRows + r < rows) copy[r].start(x.p + r * x.step, D, team);
    cp_async_commit();
    // sums: a chain of additions for each place in a vector
    float mean[2] = {};
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
      team.sum(mean[0], mean[1], 0);
#pragma unroll
      for (int r = 0; r < kRows; ++r) mean[r] = __fmul_rn(mean[r], inv_n);
    }
    float rstd[2] = {};
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float2 q[P];
#pragma unroll
      for (int e = 0; e < P; ++e) q[e] = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int j = team.at(k) * VEC;
#pragma unroll
        for (int e = 0; e < P; ++e) {
          if (kCenter) f[r][k][e] = __fadd2_rn(f[r][k][e], both(-mean[r]));
          // past the row's end the elements are 0, less the mean: left out
          float2 d = f[r][k][e];
          if (!kWhole && kCenter) {
            if (j + 2 * e >= D) d.x = 0.0f;
            if (j + 2 * e + 1 >= D) d.y = 0.0f;
          }
          if (!kWhole || k < team.mine) q[e] = __ffma2_rn(d, d, q[e]);
        }
      }
      rstd[r] = sum_pairs(q);
    }
    team.sum(rstd[0], rstd[1], 1);
#pragma unroll
    for (int r = 0; r < kRows; ++r) rstd[r] = rsqrtf(__fmaf_rn(rstd[r], inv_n, a.eps));
    if (!staged) __syncthreads();
    staged = true;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float2 w[P], b[P];
      const int i = min(team.at(k), nvec - 1);  // past the row's end: not written
      weight_vec<VEC>(weights, nvec, i, w);
      if (kCenter) weight_vec<VEC>(bias, nvec, i, b);
#pragma unroll
      for (int r = 0; r < kRows; ++r)
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 h = __fmul2_rn(f[r][k][e], both(rstd[r]));
          f[r][k][e] = kCenter ? __ffma2_rn(h, w[e], b[e]) : __fmul2_rn(h, w[e]);
        }
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        store_vector<T, kWhole>(y.p + r * y.step, k, r < rows, D, team, f[r][k]);
    }
    y.p += kRows * y.step;
    if (team.l == 0) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (kCenter && r < rows && mean_out != nullptr) mean_out[r * all] = mean[r];
        if (r < rows && rstd_out != nullptr) rstd_out[r * all] = rstd[r];
      }
      if (kCenter && mean_out != nullptr) mean_out += kRows * all;
      if (rstd_out != nullptr) rstd_out += kRows * all;
    }
    if (!kCenter && a.team > 32) named_barrier(1 + team.id, a.team);  // the sums' places
  }
  if (!staged) __syncthreads();  // warps without a row
  cp_async_wait<0>();
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

// kAhead: rows copied ahead.  Bound by the latency from a row's loads over its sums to
// its stores (16 warps of 126 registers to an SM).  RMS norm 8192 x 4096 bf16: 38.6 us
// with norm_bwd_finish_kernel (5.2 TB/s); layer norm 8191 x 1600: 30 us, x 1601: 39.
template <typename T, bool kWhole, bool kCenter, int kElems, int kAhead>
__global__ void __launch_bounds__(kBwdThreads<kElems>) norm_bwd_kernel(NormBwdArgs a) {
  // weight; the rows' copies (at the end: the teams' column sums)
  extern __shared__ float4 weights[];
  constexpr int kPlaces = kRedPlaces<kBwdThreads<kElems>>;
  __shared__ __align__(16) float2 red[2 * kPlaces];
  using Copy = RowCopy<T, kWhole, kElems>;
  constexpr int VEC = Copy::VEC, NV = Copy::NV, P = VEC / 2;
  const int D = static_cast<int>(a.D);
  const int nvec = (D + VEC - 1) / VEC;
  const Team team(a.team, nvec, red, kPlaces);
  const int64_t all = static_cast<int64_t>(gridDim.x) * a.teams;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * a.teams + team.id;  // then row + all, ...
  int rows = rows_from(row, all, a.N);  // of this team, and of the warp's first one
  int turns = a.team < 32 ? __shfl_sync(0xffffffffu, rows, 0) : rows;
  RowPtr<T, kWhole> x(a.x, row, a.ldx, all, team.l), dy(a.dy, row, a.lddy, all, team.l);
  RowPtr<T, kWhole> dx(a.dx, row, a.lddx, all, team.l);
  char* places = reinterpret_cast<char*>(weights + nvec * (VEC / 4));
  const int row_bytes = Copy::bytes(blockDim.x, a.team);
  const float* mean_in = kCenter ? a.mean + row : nullptr;
  const float* rstd_in = a.rstd + row;
  // rows in even and odd turns, each in places of its own
  struct Ahead {
    Copy x, g;
    float mean, rstd;
  };
  Ahead even{Copy(places, team), Copy(places + row_bytes, team), 0.0f, 0.0f};
  Ahead odd{Copy(places + 2 * (kAhead - 1) * row_bytes, team),
            Copy(places + (2 * kAhead - 1) * row_bytes, team), 0.0f, 0.0f};
  auto fetch = [&](Ahead& f, int ahead) {  // the row `ahead` of x.p
    if (ahead < rows) {
      f.x.start(x.p + ahead * x.step, D, team);
      f.g.start(dy.p + ahead * dy.step, D, team);
      f.rstd = rstd_in[ahead * all];
      if (kCenter) f.mean = mean_in[ahead * all];
    } else {
      // a warp whose other teams go on: a row of zeros adds nothing
      f.x.clear(true, team);
      f.g.clear(true, team);
      f.rstd = f.mean = 0.0f;
    }
    cp_async_commit();
  };
  even.x.clear(false, team);
  even.g.clear(false, team);
  fetch(even, 0);
  if (kAhead == 2) {
    odd.x.clear(false, team);
    odd.g.clear(false, team);
    fetch(odd, 1);
  }
  stage_weights<VEC>(weights, a.weight, a.w_f32, 1.0f, D);
  float2 dw[NV][P] = {}, db[NV][P] = {};
  __syncthreads();
  const float inv_n = 1.0f / static_cast<float>(D);
  auto turn = [&](Ahead& f, int parity) {
    const float mean = f.mean, rstd = f.rstd;
    float2 h[NV][P], u[NV][P];
    cp_async_wait<kAhead - 1>();
    if (!kWhole) __syncwarp();  // the right neighbour's blocks
    f.x.read(x.p, D, team, h);
    f.g.read(dy.p, D, team, u);
    __syncwarp();
    fetch(f, kAhead);
    x.p += x.step;
    dy.p += dy.step;
    rstd_in += all;
    if (kCenter) mean_in += all;
    float2 s1[P], s2[P];  // a chain of additions for each place in a vector
#pragma unroll
    for (int e = 0; e < P; ++e) s1[e] = s2[e] = both(0.0f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      // past the row's end the incoming gradient is 0, and so are all sums
      float2 w[P];
      weight_vec<VEC>(weights, nvec, min(team.at(k), nvec - 1), w);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        if (kCenter) h[k][e] = __fadd2_rn(h[k][e], both(-mean));
        h[k][e] = __fmul2_rn(h[k][e], both(rstd));
        const float2 g = u[k][e];
        u[k][e] = __fmul2_rn(g, w[e]);
        if (kCenter) s1[e] = __fadd2_rn(s1[e], u[k][e]);
        s2[e] = __ffma2_rn(u[k][e], h[k][e], s2[e]);
        dw[k][e] = __ffma2_rn(g, h[k][e], dw[k][e]);
        if (kCenter) db[k][e] = __fadd2_rn(db[k][e], g);
      }
    }
    float c1 = kCenter ? sum_pairs(s1) : 0.0f, c2 = sum_pairs(s2);
    team.sum(c2, c1, parity);
    if (a.dx == nullptr) return;
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
      store_vector<T, kWhole>(dx.p, k, rows > 0, D, team, u[k]);
    }
    dx.p += dx.step;
  };
  if (kAhead == 2) {
    for (; turns > 0; turns -= 2) {
      turn(even, 0);
      --rows;
      if (turns > 1) turn(odd, 1);
      --rows;
    }
  } else {
    for (; turns > 0; --turns, --rows) turn(even, turns & 1);
  }
  cp_async_wait<0>();
  if (a.part == nullptr) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.D;
  // the teams' sums side by side, then in team order
  float* sums = reinterpret_cast<float*>(places);
  float* to = a.teams == 1 ? part : sums + team.id * D;
  const int64_t bias_at = static_cast<int64_t>(a.teams) * D;
  __syncthreads();  // the copies are no longer needed
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int j = team.at(k) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (j + e >= D) continue;
      to[j + e] = (e & 1) ? dw[k][e / 2].y : dw[k][e / 2].x;
      if (kCenter) to[bias_at + j + e] = (e & 1) ? db[k][e / 2].y : db[k][e / 2].x;
    }
  }
  if (a.teams == 1) return;
  __syncthreads();
  for (int j = threadIdx.x; j < (kCenter ? 2 : 1) * D; j += blockDim.x) {
    const int which = j / D, c = j - which * D;
    float s = 0.0f;
    for (int t = 0; t < a.teams; ++t) s += sums[(which * a.teams + t) * D + c];
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
// in warp order.  Bound by latency: about 3 us for 152 slices of 4096 columns.  blockIdx.y: grad_weight, grad_bias.
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

// Elements per thread in norm_bwd_kernel (0: rows too long for it).  Eight where
// only one team of sixteen fits an SM (layer norm 65536 x 5120 bf16: 412 against
// 511 us), and for fp32, whose rows copied ahead take the registers (RMS norm
// 8192 x 4096: 65 against 77 us); else sixteen (bf16: 39 against 48 us).  The same
// for all strides and alignments: the order of the sums depends on it.
static int bwd_elems(int64_t D, bool f32) {
  if (D > int64_t(kBwdThreads<16>) * 16) return 0;
  const bool fits8 = D <= int64_t(kBwdThreads<8>) * 8;
  return fits8 && (f32 || D > int64_t(kBwdThreads<16>) / 2 * 16) ? 8 : 16;
}

static NormPlan bwd_plan(int64_t N, int64_t D, int elems) {
  return norm_plan(N, D, elems, elems == 8 ? kBwdThreads<8> : kBwdThreads<16>);
}

// Most partial sums: the workspace does not depend on the type.
static int64_t bwd_slices(int64_t N, int64_t D) {
  int64_t n = std::min<int64_t>(64, N);
  if (bwd_elems(D, false) > 0) n = std::max(n, bwd_plan(N, D, bwd_elems(D, false)).blocks);
  if (bwd_elems(D, true) > 0) n = std::max(n, bwd_plan(N, D, bwd_elems(D, true)).blocks);
  return n;
}

template <typename T, bool kWhole, bool kCenter, int kElems, int kAhead>
static int launch_norm_bwd_k(NormBwdArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> raised{0};
  const int rc = raise_smem(norm_bwd_kernel<T, kWhole, kCenter, kElems, kAhead>, kSmemMost, raised);
  if (rc != FLCE_OK) return rc;
  const NormPlan p = bwd_plan(a.N, a.D, kElems);
  a.team = p.team;
  a.teams = p.teams;
  a.slices = p.blocks;
  const int threads = p.team * p.teams;
  const size_t sums = p.teams > 1 ? 2 * p.teams * static_cast<size_t>(a.D) * sizeof(float) : 0;
  const size_t copies = 2 * kAhead * RowCopy<T, kWhole, kElems>::bytes(threads, p.team);
  norm_bwd_kernel<T, kWhole, kCenter, kElems, kAhead>
      <<<static_cast<unsigned>(p.blocks), threads, weight_bytes(a.D) + std::max(sums, copies),
         s>>>(a);
  return launch_status("norm_bwd_kernel launch");
}

template <typename T, bool kCenter>
static int launch_norm_bwd_held(NormBwdArgs& a, int elems, bool whole, cudaStream_t s) {
  constexpr int kAhead16 = sizeof(T) == 2 ? 2 : 1;
  if (whole)
    return elems == 8 ? launch_norm_bwd_k<T, true, kCenter, 8, 2>(a, s)
                      : launch_norm_bwd_k<T, true, kCenter, 16, kAhead16>(a, s);
  return elems == 8 ? launch_norm_bwd_k<T, false, kCenter, 8, 2>(a, s)
                    : launch_norm_bwd_k<T, false, kCenter, 16, 1>(a, s);
}

template <typename T, bool kCenter>
static int launch_norm_bwd(NormBwdArgs a, int dt, cudaStream_t s) {
  const bool w = whole(dt, a.x, a.ldx) && whole(dt, a.dy, a.lddy) &&
                 whole(dt, a.dx, a.dx != nullptr ? a.lddx : 0) && whole(dt, nullptr, a.D);
  const int elems = bwd_elems(a.D, dt == FLCE_F32);
  if (a.N > 0 && elems > 0) {
    const int rc = launch_norm_bwd_held<T, kCenter>(a, elems, w, s);
    if (rc != FLCE_OK) return rc;
  } else if (a.N > 0) {
    a.slices = std::min<int64_t>(64, a.N);
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
    const Span dx(a.dx, a.N, a.D, a.lddx, es);
    if (overlap(Span(a.x, a.N, a.D, a.ldx, es), dx)) return FLCE_EINVAL;
    if (a.dx == a.dy ? a.lddx != a.lddy && a.N > 1
                     : overlap(Span(a.dy, a.N, a.D, a.lddy, es), dx))
      return FLCE_EINVAL;
  }
  const bool cols = a.dw != nullptr || a.db != nullptr;
  if (cols) {
    const size_t need = norm_bwd_workspace_bytes(a.N, a.D);
    if (need > 0 && (ws == nullptr || ws_bytes < need)) return FLCE_EWORKSPACE;
    if (!aligned(ws, 16)) return FLCE_EALIGN;
  }
  a.part = cols ? static_cast<float*>(ws) : nullptr;
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
