// Rounding a matrix to 8 bits (eight.cuh), by rows, by square blocks, and
// transposed: what the three products of a layer's training pass read.
//
// A block of 256 threads takes 128 x 128 elements, each read once and held in registers: a
// warp has 16 rows, a lane 8 (bf16) or 4 (fp32) columns of each, rows in runs of eight, so
// that a column's eight numbers of one thread are eight bytes of the transposed matrix.
// These go through shared memory, whose 8-byte units are permuted by column so that a
// warp's lie in different banks.
//
// Alone near the bytes' time: 65536 x 5120 bf16 155 us (148 at the copy rate).  With the
// transpose bound by the latency of a block's loads, reductions and stores, one after the
// other in each block, at two blocks to an SM by rows (102 registers; issue slots 53%
// full) and three by squares: 283 and 218 us (198), 8192 x 4096 34.1 and 27.0 (19.8), of
// fp32 43.4 and 36.6 (29.7).
#include "eight.cuh"

namespace flce {

constexpr int kQThreads = 256;
constexpr int kQWarps = kQThreads / 32;

struct Quantize8Args {
  const void* x;
  int64_t R, C, ldx;
  uint8_t* q;  // [R, ldq], may be null
  int64_t ldq;
  float* scales;
  uint8_t* qt;  // [C, ldqt], may be null
  int64_t ldqt;
  float* scales_t;
};

// The 8-byte unit u of column c in shared memory.
template <int VEC>
__device__ __forceinline__ int unit8(int c, int u) {
  return c * 16 + (u ^ ((c / VEC) & 15));
}

// kSquare: one scale for the whole 128 x 128 block; else one per row (and, for the
// transposed matrix, per column).
template <typename T, bool kWhole, bool kSquare, bool kT>
__global__ void __launch_bounds__(kQThreads) quantize8_kernel(Quantize8Args a) {
  constexpr int VEC = 16 / sizeof(T);
  constexpr int kLanes = kBlock8 / VEC;  // of a row
  constexpr int kRuns = sizeof(T) / 2;   // runs of eight rows of a lane
  __shared__ float tops[kSquare ? kQWarps : 16 / kRuns][kSquare ? 1 : kBlock8];
  __shared__ __align__(16) uint2 bytes[kT ? kBlock8 * 16 : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t bc = (a.C + kBlock8 - 1) / kBlock8;
  const int64_t tr = blockIdx.x / bc, tc = blockIdx.x % bc;
  const int64_t r0 = tr * kBlock8, c0 = tc * kBlock8;
  const int rows = static_cast<int>(min(int64_t(kBlock8), a.R - r0));
  const int cols = static_cast<int>(min(int64_t(kBlock8), a.C - c0));
  const int col = lane % kLanes * VEC;                         // the lane's first
  const int first = warp * 16 + lane / kLanes * 8;             // its first row
  const T* x = static_cast<const T*>(a.x) + r0 * a.ldx + c0 + col;

  RawVec<T, VEC> raw[kRuns * 8];
#pragma unroll
  for (int i = 0; i < kRuns * 8; ++i) {
    const int r = first + i;
#pragma unroll
    for (int w = 0; w < 4; ++w) raw[i].w[w] = 0u;
    if (r >= rows) continue;
    const T* p = x + static_cast<int64_t>(r) * a.ldx;
    if (kWhole && col + VEC <= cols) {
      raw[i].load(p);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (col + e < cols) {
          if constexpr (sizeof(T) == 4)
            raw[i].w[e] = __float_as_uint(p[e]);
          else
            raw[i].w[e / 2] |= static_cast<uint32_t>(__bfloat16_as_ushort(p[e])) << (e % 2 * 16);
        }
    }
  }

  float down[VEC];  // largest of the lane's columns
#pragma unroll
  for (int e = 0; e < VEC; ++e) down[e] = 0.0f;
  float block_times = 0.0f;
  if (kSquare) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kRuns * 8; ++i) {
      float v[VEC];
      raw[i].unpack(v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) m = max_nan(m, fabsf(v[e]));
    }
    m = group_max_nan<32>(m);
    if (lane == 0) tops[warp][0] = m;
    __syncthreads();
    m = 0.0f;
#pragma unroll
    for (int w = 0; w < kQWarps; ++w) m = max_nan(m, tops[w][0]);
    const Scale8 s(m);
    block_times = s.times;
    if (threadIdx.x == 0) {
      if (a.q != nullptr) a.scales[tr * bc + tc] = s.scale;
      if (kT) a.scales_t[tc * ((a.R + kBlock8 - 1) / kBlock8) + tr] = s.scale;
    }
  }

  // by rows
  float row_times = block_times;  // !kSquare: of row i in lane i * kPer of the row's lanes
  constexpr int kRows = kRuns * 8, kPer = kLanes / kRows;
  if (!kSquare) {
    float m[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float v[VEC];
      raw[i].unpack(v);
      m[i] = 0.0f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        m[i] = max_nan(m[i], fabsf(v[e]));
        if (kT) down[e] = max_nan(down[e], fabsf(v[e]));
      }
    }
    if (a.q != nullptr) {
      // a lane divides for one row: the even ones form its `times`, the odd ones its scale
      const float largest = max_nan(group_max_of<kRows, kLanes>(m), kLeast8);
      const bool odd = (lane & 1) != 0;
      row_times = __fdiv_rn(odd ? largest : kMax8, odd ? kMax8 : largest);
      const int r = first + lane % kLanes / kPer;
      if (odd && r < rows) a.scales[(r0 + r) * bc + tc] = row_times;
    }
  }
  if (a.q != nullptr) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const float times =
          kSquare ? block_times
                  : __shfl_sync(0xffffffffu, row_times, (lane & ~(kLanes - 1)) + i * kPer);
      if (first + i >= rows) continue;
      float v[VEC];
      raw[i].unpack(v);
      uint32_t packed[VEC / 4];
#pragma unroll
      for (int e = 0; e < VEC; e += 4)
        packed[e / 4] =
            pack_e4m3x4(__fmul_rn(v[e], times), __fmul_rn(v[e + 1], times),
                        __fmul_rn(v[e + 2], times), __fmul_rn(v[e + 3], times));
      uint8_t* to = a.q + (r0 + first + i) * a.ldq + c0 + col;
      if (col + VEC <= cols) {
        if constexpr (VEC == 8)
          *reinterpret_cast<uint2*>(to) = make_uint2(packed[0], packed[1]);
        else
          *reinterpret_cast<uint32_t*>(to) = packed[0];
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (col + e < cols) to[e] = static_cast<uint8_t>(packed[e / 4] >> (e % 4 * 8));
      }
    }
  }
  if constexpr (kT) {
    // transposed
    float times[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) times[e] = block_times;
    if (!kSquare) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) tops[first / (8 * kRuns)][col + e] = down[e];
      __syncthreads();
      {
        // two threads to a column: one forms its `times`, the other its scale
        static_assert(kQThreads == 2 * kBlock8, "a pair of threads to a column");
        const int c = threadIdx.x / 2;
        const bool odd = (threadIdx.x & 1) != 0;
        float m = kLeast8;
#pragma unroll
        for (int w = 0; w < 16 / kRuns; ++w) m = max_nan(m, tops[w][c]);
        const float mine = __fdiv_rn(odd ? m : kMax8, odd ? kMax8 : m);
        __syncwarp();  // the pair has read its column
        if (!odd)
          tops[0][c] = mine;
        else if (c < cols)
          a.scales_t[(c0 + c) * ((a.R + kBlock8 - 1) / kBlock8) + tr] = mine;
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < VEC; ++e) times[e] = tops[0][col + e];
    }
#pragma unroll
    for (int run = 0; run < kRuns; ++run) {
      float v[8][VEC];
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[run * 8 + i].unpack(v[i]);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = pack_e4m3x4(__fmul_rn(v[4 * h][e], times[e]), __fmul_rn(v[4 * h + 1][e], times[e]),
                             __fmul_rn(v[4 * h + 2][e], times[e]),
                             __fmul_rn(v[4 * h + 3][e], times[e]));
        bytes[unit8<VEC>(col + e, first / 8 + run)] = make_uint2(w[0], w[1]);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kBlock8 * 8; i += kQThreads) {
      const int c = i / 8, u = i % 8 * 2;  // two units: 16 rows
      if (c >= cols || u * 8 >= rows) continue;
      const uint2 lo = bytes[unit8<VEC>(c, u)], hi = bytes[unit8<VEC>(c, u + 1)];
      uint8_t* to = a.qt + (c0 + c) * a.ldqt + r0 + u * 8;
      if (u * 8 + 16 <= rows) {
        *reinterpret_cast<uint4*>(to) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      } else {
        const uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (u * 8 + k < rows) to[k] = static_cast<uint8_t>(w[k / 4] >> (k % 4 * 8));
      }
    }
  }
}

template <typename T, bool kWhole, bool kSquare>
static int launch_quantize8(const Quantize8Args& a, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(blocks8(a.R) * blocks8(a.C));
  if (a.qt != nullptr)
    quantize8_kernel<T, kWhole, kSquare, true><<<grid, kQThreads, 0, s>>>(a);
  else
    quantize8_kernel<T, kWhole, kSquare, false><<<grid, kQThreads, 0, s>>>(a);
  return launch_status("quantize8_kernel launch");
}

template <typename T>
static int launch_quantize8(const Quantize8Args& a, bool square, cudaStream_t s) {
  const bool w = aligned(a.x, 16) && a.ldx % (16 / static_cast<int64_t>(sizeof(T))) == 0;
  if (square) return w ? launch_quantize8<T, true, true>(a, s) : launch_quantize8<T, false, true>(a, s);
  return w ? launch_quantize8<T, true, false>(a, s) : launch_quantize8<T, false, false>(a, s);
}

}  // namespace flce

using namespace flce;

extern "C" int quantize8(const void* x, int dt, int64_t R, int64_t C, int64_t ldx, int rows,
                         uint8_t* q, int64_t ldq, float* scales, uint8_t* qt, int64_t ldqt,
                         float* scales_t, flce_stream_t stream) {
  if (!valid_dtype(dt)) return FLCE_EDTYPE;
  if (rows != 1 && rows != kBlock8) return FLCE_EINVAL;
  if (R < 0 || C < 1) return FLCE_ESHAPE;
  int rc = check_matrix(x, dt, R, C, ldx);
  if (rc == FLCE_OK && q != nullptr) rc = check_matrix8(q, R, C, ldq);
  if (rc == FLCE_OK && qt != nullptr) rc = check_matrix8(qt, C, R, ldqt);
  if (rc != FLCE_OK) return rc;
  if (blocks8(R) > ((int64_t(1) << 31) - 1) / blocks8(C)) return FLCE_ESHAPE;
  if ((q == nullptr) != (scales == nullptr) || (qt == nullptr) != (scales_t == nullptr) ||
      (R > 0 && q == nullptr && qt == nullptr))
    return FLCE_EINVAL;
  if (!aligned(scales, 4) || !aligned(scales_t, 4)) return FLCE_EALIGN;
  const int64_t sr = rows == 1 ? R : blocks8(R), sc = rows == 1 ? C : blocks8(C);
  const Span all[5] = {Span(x, R, C, ldx, dtype_size(dt)), Span(q, R, C, ldq, 1),
                       Span(qt, C, R, ldqt, 1), Span(scales, sr, blocks8(C), blocks8(C), 4),
                       Span(scales_t, sc, blocks8(R), blocks8(R), 4)};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(all[i], all[j])) return FLCE_EINVAL;
  if (R == 0) return FLCE_OK;
  Quantize8Args a{x, R, C, ldx, q, ldq, scales, qt, ldqt, scales_t};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dt == FLCE_BF16 ? launch_quantize8<__nv_bfloat16>(a, rows == kBlock8, s)
                         : launch_quantize8<float>(a, rows == kBlock8, s);
}
