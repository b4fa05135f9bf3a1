// The product of matrices in 8 bits: the kernel for few tokens and the calls (gemm8.cuh
// has the formula, gemm8_pair.cuh the kernel for many).
//
// The weights are the 128 rows of the instruction's first operand and the tokens its
// columns, 16 to 64 of them: for a few tokens the weights stream once through a deep
// ring, and what is formed per thread is a row of weights, so that neighbouring
// lanes write neighbouring elements of y.  Bound by the weights' bytes and a start of
// some 8 us: 1 x 4096 x 128256 85 us (6.2 TB/s), 32 x 5120 x 151936 132 us (6.0).
// Issuing several blocks' copies together, for longer runs of a row, changed nothing.
#include <algorithm>

#include "gemm8.cuh"
#include "gemm8_pair.cuh"

namespace flce {

constexpr int kG8Rows = 128;     // rows of weights of a tile
constexpr int kG8Ahead = 8;      // blocks whose scales are loaded together

template <int BN>
struct Gemm8Geo {
  static constexpr int kStageA = kG8Rows * 128;
  static constexpr int kStageBytes = kStageA + BN * 128;
  static constexpr int kStages = BN == 64 ? 8 : 10;
  static constexpr int kBufs = 4;  // of a block's sums in tensor memory
  static constexpr int kTmemCols = kBufs * BN;
  static constexpr int kScaleBytes = 2 * kG8Ahead * BN * 4;
  static constexpr int kSmemBytes = kStages * kStageBytes + kScaleBytes + 1024;
  // Warps that add up: each of two sets of four has half of the columns where they are
  // many
  static constexpr int kSets = BN == 64 ? 2 : 1;
  static constexpr int kCols = BN / kSets;  // of a thread
  static constexpr int kAdders = 128 * kSets;
  static constexpr int kThreads = 64 + kAdders;  // and copies, and products
  static constexpr int kLoad = BN == 16 ? 16 : 32;  // columns read back at a time
};

// The scales of kG8Ahead blocks from block k on, of one row; 0 past the last block
// and for rows that are not there.
__device__ __forceinline__ void load_scales(const float* row, int k, int end,
                                            float (&s)[kG8Ahead]) {
#pragma unroll
  for (int i = 0; i < kG8Ahead; ++i) s[i] = row != nullptr && k + i < end ? row[k + i] : 0.0f;
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

template <int BN>
__global__ void __launch_bounds__(Gemm8Geo<BN>::kThreads, 1)
    gemm8_kernel(const __grid_constant__ CUtensorMap map_b,
                 const __grid_constant__ CUtensorMap map_a, const Gemm8Args g) {
  using G = Gemm8Geo<BN>;
  constexpr int S = G::kStages, kBufs = G::kBufs;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[S], empty_bar[S], sum_bar[kBufs], read_bar[kBufs], drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* col_scales = reinterpret_cast<float*>(smem + S * G::kStageBytes);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  volatile int* abort_flag = &abort_sh;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&sum_bar[i], 1);
      mbar_init(&read_bar[i], 4 * G::kSets);
    }
    mbar_init(&drain_bar, 1);
    // checked builds: the ring and the scales fit the launch's shared memory
    abort_sh = smem_in_range(0, G::kSmemBytes, g.status) ? 0 : 1;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&map_b);
    tma_prefetch_map(&map_a);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, G::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_sh;
  // this CTA's share of a tile's blocks, and its tiles
  const int rank = g.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int k0 = static_cast<int>(static_cast<int64_t>(g.blocks) * rank / g.split);
  const int k1 = static_cast<int>(static_cast<int64_t>(g.blocks) * (rank + 1) / g.split);
  const int64_t tiles = g.tiles_m * g.tiles_n;
  const int64_t first = blockIdx.x / g.split, step = gridDim.x / g.split;
  auto fail = [&]() {
    *abort_flag = 1;
    set_status(g.status, FLCE_ETIMEOUT);
  };

  if (warp == 0) {
    if (lane == 0) {
      // copies
      uint32_t stage = 0, phase = 0;
      int issued = 0;
      bool ok = true;
      for (int64_t t = first; t < tiles && ok; t += step) {
        const int m0 = static_cast<int>(t % g.tiles_m) * BN;
        const int n0 = static_cast<int>(t / g.tiles_m) * kG8Rows;
        for (int k = k0; k < k1; ++k) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* to = smem + stage * G::kStageBytes;
          mbar_arrive_expect_tx(&full_bar[stage], G::kStageBytes);
          tma_load_2d(to, &map_b, &full_bar[stage], k * 128, n0);
          tma_load_2d(to + G::kStageA, &map_a, &full_bar[stage], k * 128, m0);
          ++issued;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        fail();
        // let the copies already in flight land before the CTA exits
        for (int i = 0; i < S && i < issued; ++i) {
          if (stage == 0) {
            stage = S;
            phase ^= 1u;
          }
          --stage;
          const uint64_t t0 = global_ns();
          while (!mbar_try_wait(smem_u32(&full_bar[stage]), phase) &&
                 global_ns() - t0 < kWaitLimitNs) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // products: the sums of one block after the other
    constexpr uint32_t idesc = make_idesc(0, kG8Rows, BN, false, false);  // 0: e4m3
    const uint64_t desc = smem_desc_sw128(smem_u32(smem), 16, 1024);
    uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
    bool ok = true;
    for (int64_t t = first; t < tiles && ok; t += step) {
      for (int k = k0; k < k1; ++k) {
        ok = mbar_wait(&read_bar[buf], buf_phase ^ 1u, abort_flag) &&
             mbar_wait(&full_bar[stage], phase, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t da = desc + stage * (G::kStageBytes / 16), db = da + G::kStageA / 16;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_8bit(tmem_base + buf * BN, da + 2 * j, db + 2 * j, idesc, j > 0 ? 1u : 0u);
          mma_commit(&empty_bar[stage]);
          mma_commit(&sum_bar[buf]);
        }
        __syncwarp();
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
        if (++buf == kBufs) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) fail();
    // wait (bounded) until every product issued above has finished
    if (elect_one()) mma_commit(&drain_bar);
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(smem_u32(&drain_bar), 0) && global_ns() - t0 < kWaitLimitNs) {
    }
    __syncwarp();
  } else {
    // sums: a thread has kCols columns (tokens) of one row of weights
    const int quad = warp & 3;  // the tensor memory lanes this warp may access
    const int c0 = (warp - 2) / 4 * G::kCols;
    const int row = quad * 32 + lane, t0 = threadIdx.x - 64;
    const uint32_t lanes =
        tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(c0);
    uint32_t buf = 0, buf_phase = 0;
    int half = 0;
    float acc[G::kCols];
    int64_t m0 = 0, n = 0;
    // y[m0 + j, n] of the thread's row
    auto store = [&](int j, float v) {
      if (n >= g.N || m0 + j >= g.M) return;
      v += bias_at(g, n);
      const int64_t at = (m0 + j) * g.ldy + n;
      if (g.y_f32) {
        float* y = static_cast<float*>(g.y) + at;
        *y = g.accumulate ? *y + v : v;
      } else {
        Elem<__nv_bfloat16>::store(static_cast<__nv_bfloat16*>(g.y) + at, v);
      }
    };
    for (int64_t t = first; t < tiles; t += step) {
      m0 = t % g.tiles_m * BN;
      n = t / g.tiles_m * kG8Rows + row;
      const float* row_scale =
          n < g.N ? g.b_scales + (g.b_rows == 1 ? n : n / kBlock8) * g.blocks : nullptr;
      const float* col_scale =
          t0 < BN && m0 + t0 < g.M ? g.a_scales + (m0 + t0) * g.blocks : nullptr;
#pragma unroll
      for (int j = 0; j < G::kCols; ++j) acc[j] = 0.0f;
      float rs[kG8Ahead], cs[kG8Ahead], rs_next[kG8Ahead];
      load_scales(row_scale, k0, k1, rs_next);
      load_scales(col_scale, k0, k1, cs);
      bool good = true;
      for (int k = k0; k < k1; k += kG8Ahead, half ^= 1) {
        float* shared_scales = col_scales + half * kG8Ahead * BN;
        if (t0 < BN) {
#pragma unroll
          for (int i = 0; i < kG8Ahead; ++i) shared_scales[i * BN + t0] = cs[i];
        }
#pragma unroll
        for (int i = 0; i < kG8Ahead; ++i) rs[i] = rs_next[i];
        load_scales(row_scale, k + kG8Ahead, k1, rs_next);
        load_scales(col_scale, k + kG8Ahead, k1, cs);
        named_barrier(1, G::kAdders);
#pragma unroll
        for (int i = 0; i < kG8Ahead; ++i) {
          if (k + i >= k1) break;
          good &= mbar_wait(&sum_bar[buf], buf_phase, abort_flag);
          __syncwarp();
          tc_fence_after();
          const float4* s4 = reinterpret_cast<const float4*>(shared_scales + i * BN + c0);
#pragma unroll
          for (int j = 0; j < G::kCols; j += G::kLoad) {
            float v[G::kLoad];
            tmem_ld(lanes + buf * BN + j, v);
#pragma unroll
            for (int e = 0; e < G::kLoad; e += 4) {
              // the scales' product first: a sum times one of them may leave fp32's range
              const float4 s = s4[(j + e) / 4];
              acc[j + e] = __fmaf_rn(v[e], __fmul_rn(s.x, rs[i]), acc[j + e]);
              acc[j + e + 1] = __fmaf_rn(v[e + 1], __fmul_rn(s.y, rs[i]), acc[j + e + 1]);
              acc[j + e + 2] = __fmaf_rn(v[e + 2], __fmul_rn(s.z, rs[i]), acc[j + e + 2]);
              acc[j + e + 3] = __fmaf_rn(v[e + 3], __fmul_rn(s.w, rs[i]), acc[j + e + 3]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&read_bar[buf]);
          if (++buf == kBufs) {
            buf = 0;
            buf_phase ^= 1u;
          }
        }
      }
      if (!good) {  // a wait gave up: its elements are not a number
        fail();
#pragma unroll
        for (int j = 0; j < G::kCols; ++j) acc[j] = __int_as_float(0x7fffffff);
      }
      if (g.split == 1) {
#pragma unroll
        for (int j = 0; j < G::kCols; ++j) store(c0 + j, acc[j]);
      }
    }
    if (g.split > 1) {
      // One tile per cluster: each CTA adds up all shares of its part of the columns, in
      // the order of the ranks.  The ring is free in every CTA (its blocks' sums are
      // read), and takes the shares as [from][column][row].
      const int part = BN / g.split;
      __syncwarp();  // (one lane arrives and reports: the barrier wants whole warps)
      cluster_sync();
      const uint32_t mine =
          smem_u32(smem) + static_cast<uint32_t>((rank * part * kG8Rows + row) * 4);
#pragma unroll
      for (int j = 0; j < G::kCols; ++j) {
        const int c = c0 + j;
        st_cluster_f32(mapa_shared(mine + static_cast<uint32_t>(c % part * kG8Rows * 4),
                                   static_cast<uint32_t>(c / part)), acc[j]);
      }
      cluster_sync();
      const float* shares = reinterpret_cast<const float*>(smem);
      for (int c = (warp - 2) / 4; c < part; c += G::kSets) {
        float v = 0.0f;
        for (int r = 0; r < g.split; ++r) v += shares[(r * part + c) * kG8Rows + row];
        store(rank * part + c, v);
      }
    }
  }
  if (g.split > 1 && warp < 2) {
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, G::kTmemCols);
  }
}

// ------------------------------------------------------------------------ host

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
typedef CUresult (*CurrentFn)(CUcontext*);

template <typename F>
static F driver_entry(const char* name) {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion(name, &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<F>(p);
}

// The map's encoding needs a current context: a thread that has none bound (an
// autograd worker) gets the current device's.
static int with_context() {
  static const CurrentFn current = driver_entry<CurrentFn>("cuCtxGetCurrent");
  CUcontext ctx = nullptr;
  if (current != nullptr && current(&ctx) == CUDA_SUCCESS && ctx != nullptr) return FLCE_OK;
  int dev = 0;
  const int rc = cuda_status(cudaGetDevice(&dev), "cudaGetDevice");
  return rc != FLCE_OK ? rc : cuda_status(cudaSetDevice(dev), "cudaSetDevice");
}

// A map of a [rows, cols] matrix in boxes of 128 bytes of `box` rows, 128-byte swizzle,
// zeros outside.
static int map8(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, int box,
                CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT8, int es = 1) {
  static const EncodeFn encode = driver_entry<EncodeFn>("cuTensorMapEncodeTiled");
  if (encode == nullptr) {
    record_cuda_error(cudaErrorUnknown, "cuTensorMapEncodeTiled entry point");
    return FLCE_ECUDA;
  }
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(ld * es)};
  const cuuint32_t boxes[2] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(box)};
  const cuuint32_t one[2] = {1, 1};
  if (encode(m, type, 2, const_cast<void*>(p), dims, stride, boxes, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
    record_cuda_error(cudaErrorUnknown, "cuTensorMapEncodeTiled of a product's matrix");
    return FLCE_ECUDA;
  }
  return FLCE_OK;
}

// Few tiles: a cluster of CTAs to each, while there are SMs and each has two blocks (1 x
// 4096 x 4096: 16.6 us with a CTA to each of the 32 tiles, 7.2 in a captured graph with
// four).
static int split_of(int64_t tiles, int64_t blocks) {
  int split = 1;
  while (split < 8 && tiles * split * 2 <= sm_count() && blocks >= 4 * split) split *= 2;
  return split;
}

// Tokens of a tile (0: a tile of gemm8_pair_kernel).  Up to 64 tokens one tile has them
// all, and the weights are read once.  More than that go by 64 where this makes one
// round of the SMs at most, and else to the pairs (M x N x 4096 in captured graphs: 200
// x 4096 15.5 us, on pairs 17.3; 300 x 4096 27.1 and 17.4; 128 x 128256 172 and 114; 160 x
// 128256 242 and 115).  Smaller tiles where all these CTAs fill less than half of the SMs
// (77 x 768 x 1601: 6.3 us by 16, 7.9 by 32, 8.7 by 64).
static int tile_tokens(int64_t M, int64_t N, int64_t blocks) {
  const int64_t tiles_n = (N + kG8Rows - 1) / kG8Rows, sms = sm_count();
  int bn = M <= 16 ? 16 : M <= 32 ? 32 : 64;
  if (M > 64 && (M + 63) / 64 * tiles_n > sms) return 0;
  for (; bn > 16; bn /= 2) {
    const int64_t tiles = (M + bn - 1) / bn * tiles_n;
    if (2 * tiles * split_of(tiles, blocks) >= sms) break;
  }
  return bn;
}

template <int BN>
static int launch_gemm8(Gemm8Args g, const uint8_t* a, int64_t lda, const uint8_t* b, int64_t ldb,
                        int64_t K, cudaStream_t s) {
  using G = Gemm8Geo<BN>;
  CUtensorMap ma, mb;
  int rc = map8(&mb, b, g.N, K, ldb, kG8Rows);
  if (rc == FLCE_OK) rc = map8(&ma, a, g.M, K, lda, BN);
  static std::atomic<uint64_t> raised{0};
  if (rc == FLCE_OK) rc = raise_smem(gemm8_kernel<BN>, G::kSmemBytes, raised);
  if (rc != FLCE_OK) return rc;
  g.tiles_m = (g.M + BN - 1) / BN;
  g.tiles_n = (g.N + kG8Rows - 1) / kG8Rows;
  const int64_t tiles = g.tiles_m * g.tiles_n;
  g.split = split_of(tiles, g.blocks);
  if (g.split == 1) {
    gemm8_kernel<BN><<<static_cast<unsigned>(std::min<int64_t>(tiles, sm_count())), G::kThreads,
                       G::kSmemBytes, s>>>(mb, ma, g);
    return launch_status("gemm8_kernel launch");
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(g.split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * g.split), 1, 1);
  cfg.blockDim = dim3(G::kThreads, 1, 1);
  cfg.dynamicSmemBytes = G::kSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, gemm8_kernel<BN>, mb, ma, g),
                     "cudaLaunchKernelEx(gemm8_kernel)");
}

// A lone CTA cannot run half of a pair: as many pairs as can be resident at once.
template <bool kCols, bool kTma>
static int launch_gemm8_pair(Gemm8Args g, const uint8_t* a, int64_t lda, const uint8_t* b,
                             int64_t ldb, int64_t K, cudaStream_t s) {
  using G = Gemm8Pair<kCols>;
  auto* kernel = gemm8_pair_kernel<kCols, kTma>;
  CUtensorMap ma, mb, my;
  int rc = map8(&ma, a, g.M, K, lda, 128);
  if (rc == FLCE_OK) rc = map8(&mb, b, g.N, K, ldb, 64);
  my = ma;  // not used without kTma
  if (rc == FLCE_OK && kTma)
    rc = map8(&my, g.y, g.M, g.N, g.ldy, 32,
              g.y_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              g.y_f32 ? 4 : 2);
  static std::atomic<uint64_t> raised{0};
  if (rc == FLCE_OK) rc = raise_smem(kernel, G::kSmemBytes, raised);
  if (rc != FLCE_OK) return rc;
  g.tiles_m = (g.M + G::kTile - 1) / G::kTile;
  g.tiles_n = (g.N + G::kTile - 1) / G::kTile;
  const int64_t tiles = g.tiles_m * g.tiles_n;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(G::kThreads, 1, 1);
  cfg.dynamicSmemBytes = G::kSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static std::atomic<int> resident[64];
  int dev = 0;
  rc = cuda_status(cudaGetDevice(&dev), "cudaGetDevice");
  if (rc != FLCE_OK) return rc;
  int pairs = resident[dev & 63].load();
  if (pairs <= 0) {
    cfg.gridDim = dim3(2 * static_cast<unsigned>(std::max(1, sm_count() / 2)), 1, 1);
    rc = cuda_status(cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg),
                     "cudaOccupancyMaxActiveClusters");
    if (rc != FLCE_OK) return rc;
    if (pairs < 1) return FLCE_ENOSUP;
    resident[dev & 63].store(pairs);
  }
  cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<int64_t>(tiles, pairs)), 1, 1);
  const int group_m = static_cast<int>(std::min<int64_t>(8, g.tiles_m));
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, ma, mb, my, g, group_m),
                     "cudaLaunchKernelEx(gemm8_pair_kernel)");
}

}  // namespace flce

using namespace flce;

extern "C" int gemm8(const uint8_t* a, int64_t lda, const float* a_scales, int64_t M,
                     const uint8_t* b, int64_t ldb, const float* b_scales, int b_rows, int64_t N,
                     int64_t K, const void* bias, int dt_bias, void* y, int dt_y, int64_t ldy,
                     int accumulate, int32_t* status, flce_stream_t stream) {
  if (!valid_dtype(dt_y) || !valid_dtype(dt_bias)) return FLCE_EDTYPE;
  if ((b_rows != 1 && b_rows != kBlock8) || (accumulate != 0 && accumulate != 1))
    return FLCE_EINVAL;
  // row numbers are the 32-bit coordinates of a copy
  if (M < 0 || N < 1 || K < 1 || M > 0x7fffff00 || N > 0x7fffff00 || K > 0x7fffff00)
    return FLCE_ESHAPE;
  int rc = check_matrix8(a, M, K, lda);
  if (rc == FLCE_OK) rc = check_matrix8(b, N, K, ldb);
  if (rc == FLCE_OK) rc = check_matrix(y, dt_y, M, N, ldy);
  if (rc != FLCE_OK) return rc;
  if ((M > 0 && a_scales == nullptr) || b_scales == nullptr) return FLCE_EINVAL;
  if (!aligned(a_scales, 4) || !aligned(b_scales, 4) || !aligned(bias, dtype_size(dt_bias)) ||
      !aligned(status, 4))
    return FLCE_EALIGN;
  if (accumulate && dt_y != FLCE_F32) return FLCE_ENOSUP;
  const int64_t blocks = blocks8(K);
  const Span out(y, M, N, ldy, dtype_size(dt_y));
  if (overlap(out, Span(a, M, K, lda, 1)) || overlap(out, Span(b, N, K, ldb, 1)) ||
      overlap(out, Span(a_scales, M, blocks, blocks, 4)) ||
      overlap(out, Span(b_scales, b_rows == 1 ? N : blocks8(N), blocks, blocks, 4)) ||
      overlap(out, Span(bias, 1, N, N, dtype_size(dt_bias))))
    return FLCE_EINVAL;
  if (M == 0) return FLCE_OK;
  if (blocks8(M) > 0x7fffffff / blocks8(N)) return FLCE_ESHAPE;  // tiles are counted in 32 bits
  rc = with_context();
  if (rc != FLCE_OK) return rc;
  Gemm8Args g{};
  g.M = M, g.N = N, g.blocks = static_cast<int>(blocks);
  g.a_scales = a_scales, g.b_scales = b_scales, g.b_rows = b_rows;
  g.bias = bias, g.bias_f32 = dt_bias == FLCE_F32;
  g.y = y, g.ldy = ldy, g.y_f32 = dt_y == FLCE_F32, g.accumulate = accumulate, g.status = status;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (tile_tokens(M, N, blocks)) {
    case 16: return launch_gemm8<16>(g, a, lda, b, ldb, K, s);
    case 32: return launch_gemm8<32>(g, a, lda, b, ldb, K, s);
    case 64: return launch_gemm8<64>(g, a, lda, b, ldb, K, s);
    default: break;
  }
  const int es = g.y_f32 ? 4 : 2;
  const bool tma = aligned(y, 16) && ldy * es % 16 == 0 && ldy * es < (int64_t(1) << 40);
  auto* pairs = b_rows == 1 ? tma ? launch_gemm8_pair<true, true> : launch_gemm8_pair<true, false>
                : tma       ? launch_gemm8_pair<false, true>
                            : launch_gemm8_pair<false, false>;
  return pairs(g, a, lda, b, ldb, K, s);
}
