// The head with 4-bit weights and group scales: logits of a few tokens, and
// the rounding of a table to that layout.
#include <algorithm>
#include <atomic>

#include "head4_few.cuh"
#include "head4_many.cuh"

namespace flce {

constexpr int kSmemMost = 226 * 1024;

// The kernel's limit on shared memory, raised once per device and kernel.
template <typename K>
static int raise_smem(K* kernel, std::atomic<uint64_t>& raised) {
  int dev = 0;
  int rc = cuda_status(cudaGetDevice(&dev), "cudaGetDevice");
  if (rc != FLCE_OK) return rc;
  const uint64_t bit = 1ull << (dev & 63);
  if (raised.load() & bit) return FLCE_OK;
  rc = cuda_status(
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost),
      "cudaFuncSetAttribute(head4 kernel)");
  if (rc == FLCE_OK) raised.fetch_or(bit);
  return rc;
}

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
  const int rc = raise_smem(head4_few_kernel<G32, ST, NT>, raised);
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
  const int rc = raise_smem(head4_many_kernel<G32, ST>, raised);
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
