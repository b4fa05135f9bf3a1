// The head with 4-bit weights and group scales: logits of a few tokens, and
// the rounding of a table to that layout.
#include <algorithm>

#include "head4_few.cuh"
#include "head4_many.cuh"

namespace flce {

constexpr int kSmemMost = 226 * 1024;  // beside a few static words

// Tiles of `rows` rows, and how many of a block's `units` share one; at most `fit`
// stages of the tokens stand in shared memory.
static int plan_head4(Head4Args& a, int rows, int units, int64_t fit) {
  const int64_t stages = std::min((a.D + kStageCols - 1) / kStageCols, fit);
  a.chunk = stages * kStageCols;
  a.tiles = (a.V + rows - 1) / rows;
  const int sms = sm_count();
  a.wk = 1;
  while (a.wk < units && 2 * a.wk <= stages && a.tiles * 2 * a.wk <= int64_t(sms) * units)
    a.wk *= 2;
  return static_cast<int>(std::min<int64_t>(a.tiles, sms));
}

template <int G32, typename ST, int NT>
static int launch_few(Head4Args a, cudaStream_t s) {
  static std::atomic<uint64_t> raised{0};
  const int rc = raise_smem(head4_few_kernel<G32, ST, NT>, kSmemMost, raised);
  if (rc != FLCE_OK) return rc;
  const int64_t fit = ((kSmemMost - kRing) / a.cols - kXPad) / (2 * kStageCols);
  const int grid = plan_head4(a, 32, kWarps, fit);
  const int64_t smem = kRing + a.cols * (a.chunk * 2 + kXPad);
  head4_few_kernel<G32, ST, NT><<<grid, 32 * kWarps, static_cast<size_t>(smem), s>>>(a);
  return launch_status("head4_few_kernel launch");
}

template <int G32, typename ST>
static int launch_many(Head4Args a, cudaStream_t s) {
  static std::atomic<uint64_t> raised{0};
  const int rc = raise_smem(head4_many_kernel<G32, ST>, kSmemMost, raised);
  if (rc != FLCE_OK) return rc;
  constexpr int kStageX = kManyCols * kStageCols * 2;
  const int grid = plan_head4(a, 128, kWarps / 4, (kSmemMost - kRing - 1024) / kStageX);
  const int64_t smem = kRing + a.chunk / kStageCols * kStageX + 1024;  // 1 KB to align
  head4_many_kernel<G32, ST><<<grid, 32 * kWarps, static_cast<size_t>(smem), s>>>(a);
  return launch_status("head4_many_kernel launch");
}

// Above 16 token columns the tcgen05 kernel, whose time hardly depends on their
// number: 121 us for 20 tokens on 128256 x 4096 and 132 for 32, where mma.sync takes
// 192; with 16 columns mma.sync takes 100.  Groups of 32 stay with mma.sync (219 us
// for 32 tokens): A and four sums of 32 columns would take 192 tensor memory columns,
// and a warpgroup has 128.
template <int G32, typename ST>
static int launch_head4(const Head4Args& a, cudaStream_t s) {
  if constexpr (G32 > 1) {
    if (a.cols > 16) return launch_many<G32, ST>(a, s);
  } else {
    if (a.cols > 16) return launch_few<G32, ST, 4>(a, s);
  }
  if (a.cols > 8) return launch_few<G32, ST, 2>(a, s);
  return launch_few<G32, ST, 1>(a, s);
}

template <typename ST>
static int launch_group(int group, const Head4Args& a, cudaStream_t s) {
  return group == 32   ? launch_head4<1, ST>(a, s)
         : group == 64 ? launch_head4<2, ST>(a, s)
                       : launch_head4<4, ST>(a, s);
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

// A lane's sixteen columns from k0 on of a row as they lie in memory, zeros from D on;
// kWide: in 16-byte loads where they are all there, else one word per element.
template <typename T, bool kWide>
struct QuantWords {
  static constexpr int kWords = kWide ? 4 * sizeof(T) : 16;
  uint32_t w[kWords];
  static __device__ __forceinline__ uint32_t element(const T* p) {
    if constexpr (sizeof(T) == 4)
      return *reinterpret_cast<const uint32_t*>(p);
    else
      return *reinterpret_cast<const uint16_t*>(p);
  }
  __device__ __forceinline__ void load(const T* row, int64_t k0, int64_t D) {
    if constexpr (kWide) {
      if (k0 + 16 <= D) {
#pragma unroll
        for (int q = 0; q < kWords; q += 4) {
          const uint4 v = __ldcs(reinterpret_cast<const uint4*>(row + k0) + q / 4);
          w[q] = v.x, w[q + 1] = v.y, w[q + 2] = v.z, w[q + 3] = v.w;
        }
        return;
      }
    }
#pragma unroll
    for (int q = 0; q < kWords; ++q) w[q] = 0u;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      constexpr int kPer = 16 / kWords;  // elements of a word
      if (k0 + e < D) w[e / kPer] |= element(row + k0 + e) << (16 * (e % kPer));
    }
  }
  __device__ __forceinline__ void unpack(float (&x)[16]) const {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if constexpr (sizeof(T) == 4)
        x[e] = __uint_as_float(w[e]);
      else if constexpr (kWide)
        x[e] = (e & 1) ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
      else
        x[e] = bf16_lo(w[e]);
    }
  }
};

// Eight lanes per 128 columns of a row, sixteen columns (two words) to a lane.  The
// groups' extremes are found by the lanes that hold their columns; the next block's
// columns are loaded before this one's are used.
//
// Bound by issue, so a quotient is the product with 1 / s, corrected once by its exact
// remainder (P. Markstein, IBM J. Res. Dev. 34, 1990), which is what a division gives.
// It is rounded by adding 1.5 * 2^23, which leaves the nibble in the sum's lowest bits.
// 128256 x 4096 in groups of 128: bf16 333 us (a copy's rate: 196), fp32 367 (353); a
// division for every element, half of a warp idle and loads of one element: 1713 us.
template <typename T, typename S, bool kWide>
__global__ void __launch_bounds__(256) head4_quantize_kernel(Quant4Args a) {
  const int lane = threadIdx.x & 31;
  const int64_t blocks = (a.D + 127) / 128;
  const int64_t n = a.V * blocks;
  // columns 32 w + 16 h + (0..15) of the block: its words 8 h + w and 8 h + 4 + w
  const int w = lane & 3, h = lane >> 2 & 1;
  const bool zp = a.zeros != nullptr;
  const int group_bits = a.group == 32 ? 5 : a.group == 64 ? 6 : 7;
  const bool writes_group = h == 0 && ((32 * w) & (a.group - 1)) == 0;
  // this lane's block and the step to its next one as rows and blocks (divisions in
  // the loop would cost more than all else in it); the warp's first block decides on
  // the end, as all lanes take part in the shuffles
  const int64_t step = static_cast<int64_t>(gridDim.x) * 32, step_v = step / blocks;
  const int64_t step_b = step - step_v * blocks;
  int64_t first = (static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5)) * 4;
  int64_t at_v = (first + (lane >> 3)) / blocks, b = first + (lane >> 3) - at_v * blocks;
  const T* W = static_cast<const T*>(a.W);
  const int k_lane = 32 * w + 16 * h;
  QuantWords<T, kWide> ahead = {};
  if (at_v < a.V) ahead.load(W + at_v * a.ldw, b * 128 + k_lane, a.D);
  while (first < n) {
    const int64_t v = at_v, block = b;
    float x[16], lo = 0.0f, hi = 0.0f;
    ahead.unpack(x);
    first += step;
    at_v += step_v;
    b += step_b;
    if (b >= blocks) {
      b -= blocks;
      ++at_v;
    }
    if (at_v < a.V) ahead.load(W + at_v * a.ldw, b * 128 + k_lane, a.D);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      lo = fminf(lo, x[j]);
      hi = fmaxf(hi, x[j]);
    }
    // a group of 32 columns: two lanes; of 64 and 128 also their neighbours in w
    float s, z = 8.0f;
    if (zp) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, 4));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, 4));
      for (int d = 1; 32 * d < a.group; d <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
      }
      // (the range itself may pass fp32's; half of it does not)
      const float range = __fadd_rn(hi, -lo);
      s = range <= 3.40282347e38f ? __fdiv_rn(range, 15.0f)
                                  : __fdiv_rn(__fadd_rn(0.5f * hi, -0.5f * lo), 7.5f);
      s = round_to(s, static_cast<const S*>(nullptr));
      if (s == 0.0f) s = 1.0f;
      z = fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.0f), 15.0f);
    } else {
      hi = fmaxf(hi, -lo);
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, 4));
      for (int d = 1; 32 * d < a.group; d <<= 1)
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
      s = round_to(__fdiv_rn(hi, 7.0f), static_cast<const S*>(nullptr));
      if (s == 0.0f) s = 1.0f;
    }
    const float inv = __fdiv_rn(1.0f, s), low = -z, high = 15.0f - z;
    const float whole = 12582912.0f + z;
    // a quotient within the nibble's range, rounded before z is added (halves go to even)
    auto nibble = [&](float q) {
      q = __fadd_rn(__fadd_rn(fminf(fmaxf(q, low), high), 12582912.0f), -12582912.0f);
      return __fadd_rn(q, whole);
    };
    if (s > 0x1p-100f && s < 0x1p100f) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float q = __fmul_rn(x[j], inv);
        x[j] = nibble(__fmaf_rn(__fmaf_rn(-q, s, x[j]), inv, q));
      }
    } else {  // where a step above could leave the normal numbers
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = nibble(__fdiv_rn(x[j], s));
    }
    if (v < a.V) {
      uint32_t* to = reinterpret_cast<uint32_t*>(a.packed + v * a.ldp + block * 64) + 8 * h + w;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        // the numbers stand above 0x4b400000: what that adds up to is taken off
        uint32_t word = 0, extra = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t place = 1u << (4 * ((j >> 1) + 4 * (j & 1)));
          word += __float_as_uint(x[8 * half + j]) * place;
          extra += 0x4b400000u * place;
        }
        word -= extra;
        const int64_t left = a.D - (block * 128 + k_lane + 8 * half);
        if (left < 8) {  // columns past the end: 0
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j >= left) word &= ~(15u << (4 * ((j >> 1) + 4 * (j & 1))));
        }
        to[4 * half] = word;
      }
      const int64_t gi = (block * 128 + k_lane) >> group_bits;
      if (writes_group && gi < a.G) {
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

// The parts of a head: what head4_logits reads and head4_quantize writes.
struct HeadSpans {
  Span packed, scales, zeros;
  HeadSpans(const void* packed, int64_t ldp, const void* scales, int dt_s, const void* zeros,
            int group, int64_t V, int64_t D)
      : packed(packed, V, (D + 127) / 128 * 64, ldp, 1),
        scales(scales, 1, V * ((D + group - 1) / group), 0, dtype_size(dt_s)),
        zeros(zeros, 1, V * ((D + group - 1) / group), 0, 1) {}
  bool meet(const Span& s) const {
    return overlap(packed, s) || overlap(scales, s) || overlap(zeros, s);
  }
};

}  // namespace flce

using namespace flce;

extern "C" int head4_logits(const void* x, int dt, int64_t M, int64_t D, int64_t ldx,
                            const uint8_t* packed, int64_t ldp, const void* scales, int dt_s,
                            const uint8_t* zeros, int group, int64_t V, const void* bias, void* y,
                            int dt_y, int64_t ldy, int32_t* status, flce_stream_t stream) {
  if (!valid_dtype(dt) || !valid_dtype(dt_y)) return FLCE_EDTYPE;
  if (M < 0) return FLCE_ESHAPE;
  int rc = check_head4(packed, ldp, scales, dt_s, group, V, D);
  if (rc == FLCE_OK) rc = check_matrix(x, dt, M, D, ldx);
  if (rc == FLCE_OK) rc = check_matrix(y, dt_y, M, V, ldy);
  if (rc != FLCE_OK) return rc;
  if (!aligned(bias, dtype_size(dt)) || !aligned(status, 4)) return FLCE_EALIGN;
  const Span out(y, M, V, ldy, dtype_size(dt_y));
  if (HeadSpans(packed, ldp, scales, dt_s, zeros, group, V, D).meet(out) ||
      overlap(Span(x, M, D, ldx, dtype_size(dt)), out) ||
      overlap(Span(bias, 1, V, 0, dtype_size(dt)), out))
    return FLCE_EINVAL;
  if (M == 0) return FLCE_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Head4Args a{};
  a.x_f32 = dt == FLCE_F32;
  a.D = D;
  a.ldx = ldx;
  a.packed = packed;
  a.ldp = ldp;
  a.scales = scales;
  a.zeros = zeros;
  a.V = V;
  a.G = (D + group - 1) / group;
  a.bias = bias;
  a.y_f32 = dt_y == FLCE_F32;
  a.status = status;
  a.ldy = ldy;
  const int64_t most = a.x_f32 ? 10 : 32;
  for (int64_t m0 = 0; m0 < M && rc == FLCE_OK; m0 += most) {
    a.M = static_cast<int>(std::min(most, M - m0));
    a.cols = a.x_f32 ? 3 * a.M : a.M;
    a.x = static_cast<const char*>(x) + m0 * ldx * static_cast<int64_t>(dtype_size(dt));
    a.y = static_cast<char*>(y) + m0 * ldy * static_cast<int64_t>(dtype_size(dt_y));
    if (dt_s == FLCE_BF16)
      rc = launch_group<__nv_bfloat16>(group, a, s);
    else
      rc = launch_group<float>(group, a, s);
  }
  return rc;
}

extern "C" int head4_quantize(const void* W, int dt, int64_t V, int64_t D, int64_t ldw, int group,
                              uint8_t* packed, int64_t ldp, void* scales, int dt_s, uint8_t* zeros,
                              flce_stream_t stream) {
  if (!valid_dtype(dt)) return FLCE_EDTYPE;
  int rc = check_head4(packed, ldp, scales, dt_s, group, V, D);
  if (rc == FLCE_OK) rc = check_matrix(W, dt, V, D, ldw);
  if (rc != FLCE_OK) return rc;
  const HeadSpans to(packed, ldp, scales, dt_s, zeros, group, V, D);
  if (to.meet(Span(W, V, D, ldw, dtype_size(dt))) || overlap(to.packed, to.scales) ||
      overlap(to.packed, to.zeros) || overlap(to.scales, to.zeros))
    return FLCE_EINVAL;
  const Quant4Args a{W, V, D, ldw, group, packed, ldp, scales, zeros, (D + group - 1) / group};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t blocks = (D + 127) / 128;
  const int grid = static_cast<int>(std::min<int64_t>((V * blocks + 31) / 32, sm_count() * 24));
  const bool wide = aligned(W, 16) && ldw % (dt == FLCE_BF16 ? 8 : 4) == 0;
  using B = __nv_bfloat16;
#define HEAD4_QUANTIZE(T, S)                                            \
  if (wide) head4_quantize_kernel<T, S, true><<<grid, 256, 0, s>>>(a);  \
  else head4_quantize_kernel<T, S, false><<<grid, 256, 0, s>>>(a)
  if (dt == FLCE_BF16) {
    if (dt_s == FLCE_BF16) {
      HEAD4_QUANTIZE(B, B);
    } else {
      HEAD4_QUANTIZE(B, float);
    }
  } else {
    if (dt_s == FLCE_BF16) {
      HEAD4_QUANTIZE(float, B);
    } else {
      HEAD4_QUANTIZE(float, float);
    }
  }
#undef HEAD4_QUANTIZE
  return launch_status("head4_quantize_kernel launch");
}

extern "C" int head4_wait_selftest(float* y, int32_t* status, uint64_t limit_ns,
                                   flce_stream_t stream) {
  if (y == nullptr || status == nullptr) return FLCE_EINVAL;
  if (!aligned(y, 4) || !aligned(status, 4)) return FLCE_EALIGN;
  if (limit_ns > 2000000000ull) return FLCE_ESHAPE;
  head4_wait_selftest_kernel<<<1, 32 * kWarps, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      y, status, limit_ns);
  return launch_status("head4_wait_selftest_kernel launch");
}
