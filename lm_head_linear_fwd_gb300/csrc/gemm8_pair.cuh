// gemm8 for many tokens: 256 x 256 tiles on pairs of CTAs.
//
// The pair's two SMs form one tile with tcgen05.mma.cta_group::2: each loads its 128
// rows of a and 128 of the tile's 256 rows of b, and has 128 rows of the sums in its
// tensor memory, a block's in one half of the 512 columns while the next block's are
// formed in the other.  Eight warps add them up, a thread 128 columns of one row, so
// that a's scale is one number per thread, and b's, where it is for 128 rows, one per
// warp: one multiply-add per element and block.  Two more warps load the scales, a few
// blocks ahead, to shared memory.
//
// Barriers as in the pair kernel of tc_gemm.cuh:
//   full[s]   leader: both CTAs' copies have landed     empty[s]  both: stage was read
//   sum[i]    both: a block's sums are there            read[i]   leader: 16 warps have
//                                                       read them
//   scaled[r] both: kAhead blocks' scales are there     used[r]   both: they were used
#pragma once

#include "gemm8.cuh"
#include "tc_gemm.cuh"

namespace flce {

struct Gemm8Pair {
  // A warpgroup for copies and products, two that add up.  The registers of 384 threads
  // at launch, 168 each (65536 / 384, down to a multiple of eight), are dealt anew: 56
  // and 224, the same sum, 4 x 56 + 8 x 224 = 12 x 168.
  static constexpr int kThreads = 384;
  static constexpr int kTile = 256;     // rows of a, and of b, of a pair's tile
  static constexpr int kStageA = 128 * 128;
  static constexpr int kStageBytes = 2 * kStageA;
  static constexpr int kStages = 5;
  static constexpr int kAhead = 4;  // blocks whose scales are loaded together
  static constexpr int kRing = 3;   // of these
  static constexpr int kScales = 128 + 256;  // a block's: of the rows, and of the columns
  static constexpr int kScaleBytes = kRing * kAhead * kScales * 4;
  static constexpr int kStaging = 8 * 4096;
  static constexpr int kSmemBytes = kStages * kStageBytes + kStaging + kScaleBytes + 1024;
};

__device__ __forceinline__ void mma_8bit_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 columns of this thread's lane, to be waited for.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Waits for all loads of this thread; r are those of the last one (so that no use of
// them comes before).
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ float2 pair_of(const uint32_t (&r)[32], int p) {
  return make_float2(__uint_as_float(r[2 * p]), __uint_as_float(r[2 * p + 1]));
}

// Arrive on a barrier of another CTA of the cluster for tensor memory that was read:
// the loads have been waited for and no other memory is handed over, so that no wider
// fence is needed than a barrier's own.
__device__ __forceinline__ void mbar_arrive_read(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// The scales of four blocks from k on of a row (null: 0), each to its block's place.
__device__ __forceinline__ void stage_scales(const float* row, int k, int blocks, bool wide,
                                             float* to) {
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (row != nullptr) {
    if (wide) {  // all four are there, on a 16-byte boundary
      v = *reinterpret_cast<const float4*>(row + k);
    } else {
      v.x = row[k];
      if (k + 1 < blocks) v.y = row[k + 1];
      if (k + 2 < blocks) v.z = row[k + 2];
      if (k + 3 < blocks) v.w = row[k + 3];
    }
  }
  to[0] = v.x;
  to[Gemm8Pair::kScales] = v.y;
  to[2 * Gemm8Pair::kScales] = v.z;
  to[3 * Gemm8Pair::kScales] = v.w;
}

// kCols: b has a scale for each of its rows (the tile's columns); else one for 128.
template <bool kCols>
__global__ void __launch_bounds__(Gemm8Pair::kThreads, 1)
    gemm8_pair_kernel(const __grid_constant__ CUtensorMap map_a,
                      const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ CUtensorMap map_y, const Gemm8Args g,
                      const int group_m, const int tma_store) {
  using G = Gemm8Pair;
  constexpr int S = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[S], empty_bar[S], sum_bar[2], read_bar[2], drain_bar;
  __shared__ uint64_t scaled_bar[G::kRing], used_bar[G::kRing];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  float* scale_ring = reinterpret_cast<float*>(smem + S * G::kStageBytes + G::kStaging);
  volatile int* abort_flag = &abort_sh;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sum_bar[i], 1);
      mbar_init(&read_bar[i], 16);
    }
    for (int i = 0; i < G::kRing; ++i) {
      mbar_init(&scaled_bar[i], 2);
      mbar_init(&used_bar[i], 8);
    }
    mbar_init(&drain_bar, 1);
    // checked builds: everything fits the launch's shared memory
    abort_sh = smem_in_range(0, G::kSmemBytes, g.status) ? 0 : 1;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  if (warp == 1) {
    tmem_alloc_pair(&tmem_base_sh, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs initialised; tensor memory allocated in both
  tc_fence_after();
  const uint32_t tmem_base = tmem_base_sh;
  const int nm = static_cast<int>(g.tiles_m), nn = static_cast<int>(g.tiles_n);
  const int tiles = nm * nn, first = static_cast<int>(blockIdx.x >> 1);
  const int step = static_cast<int>(gridDim.x >> 1);
  const uint32_t full_leader = mapa_shared(smem_u32(&full_bar[0]), 0);
  const uint32_t read_leader = mapa_shared(smem_u32(&read_bar[0]), 0);
  auto fail = [&]() {
    *abort_flag = 1;
    set_status(g.status, FLCE_ETIMEOUT);
  };

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  if (warp == 0) {
    if (lane == 0) {
      // copies
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        int mt, nt;
        tile_coords(t, nm, nn, group_m, mt, nt);
        const int arow = mt * G::kTile + static_cast<int>(rank) * 128;
        const int brow = nt * G::kTile + static_cast<int>(rank) * 128;
        for (int k = 0; k < g.blocks; ++k) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * G::kStageBytes);
          uint8_t* to = smem + stage * G::kStageBytes;
          const uint32_t bar = full_leader + stage * 8u;
          tma_load_2d_pair(to, &map_a, bar, k * 128, arow);
          tma_load_2d_pair(to + G::kStageA, &map_b, bar, k * 128, brow);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        fail();
        // copies in flight complete on the leader's barrier; give them time to land
        const uint64_t t0 = global_ns();
        while (global_ns() - t0 < 20000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    if (leader && lane == 0) {
      // products: the sums of one block after the other
      constexpr uint32_t idesc = make_idesc(0, 256, G::kTile, false, false);  // 0: e4m3
      uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        for (int k = 0; k < g.blocks; ++k) {
          if (!mbar_wait(&read_bar[buf], buf_phase ^ 1u, abort_flag) ||
              !mbar_wait(&full_bar[stage], phase, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + stage * G::kStageBytes);
          const uint32_t sb = sa + G::kStageA;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_8bit_pair(tmem_base + buf * G::kTile, smem_desc_sw128(sa + j * 32, 16, 1024),
                          smem_desc_sw128(sb + j * 32, 16, 1024), idesc, j > 0 ? 1u : 0u);
          mma_commit_pair(&empty_bar[stage], 0x3);
          mma_commit_pair(&sum_bar[buf], 0x3);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
          buf ^= 1u;
          if (buf == 0) buf_phase ^= 1u;
        }
      }
      if (!ok) fail();
      mma_commit_pair(&drain_bar, 0x1);
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(smem_u32(&drain_bar), 0) && global_ns() - t0 < kWaitLimitNs) {
      }
    }
  } else if (warp < 4) {
    // scales: warp 2 those of the rows, warp 3 those of the columns
    const bool wide = g.blocks % G::kAhead == 0 &&
                      ((reinterpret_cast<uintptr_t>(g.a_scales) |
                        reinterpret_cast<uintptr_t>(g.b_scales)) & 15) == 0;
    uint32_t slot = 0, phase = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      int mt, nt;
      tile_coords(t, nm, nn, group_m, mt, nt);
      const int64_t m0 = static_cast<int64_t>(mt) * G::kTile + rank * 128;
      const int64_t n0 = static_cast<int64_t>(nt) * G::kTile;
      for (int k = 0; k < g.blocks; k += G::kAhead) {
        ok = mbar_wait(&used_bar[slot], phase ^ 1u, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0) fail();
          ok = false;
          break;
        }
        float* to = scale_ring + slot * G::kAhead * G::kScales;
        if (warp == 2) {
#pragma unroll
          for (int i = lane; i < 128; i += 32)
            stage_scales(m0 + i < g.M ? g.a_scales + (m0 + i) * g.blocks : nullptr, k, g.blocks,
                         wide, to + i);
        } else if (kCols) {
#pragma unroll
          for (int i = lane; i < 256; i += 32)
            stage_scales(n0 + i < g.N ? g.b_scales + (n0 + i) * g.blocks : nullptr, k, g.blocks,
                         wide, to + 128 + i);
        } else if (lane < 2) {
          const int64_t n = n0 + lane * 128;
          stage_scales(n < g.N ? g.b_scales + n / kBlock8 * g.blocks : nullptr, k, g.blocks, wide,
                       to + 128 + lane);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&scaled_bar[slot]);
        if (++slot == G::kRing) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // sums: a thread has 128 columns of one row
    const int quad = warp & 3;         // the tensor memory lanes this warp may access
    const int half = (warp - 4) >> 2;  // its half of the columns
    const uint32_t lanes =
        tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(half * 128);
    uint8_t* slab = smem + S * G::kStageBytes + (warp - 4) * 4096;
    uint32_t buf = 0, buf_phase = 0, slot = 0, slot_phase = 0;
    for (int t = first; t < tiles; t += step) {
      int mt, nt;
      tile_coords(t, nm, nn, group_m, mt, nt);
      float2 acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = make_float2(0.0f, 0.0f);
      bool good = true;
      for (int k = 0; k < g.blocks; ++k) {
        const int at = k & (G::kAhead - 1);
        if (at == 0) good &= mbar_wait(&scaled_bar[slot], slot_phase, abort_flag);
        const float* scales = scale_ring + (slot * G::kAhead + at) * G::kScales;
        float s = scales[quad * 32 + lane];
        if (!kCols) s = __fmul_rn(s, scales[128 + half]);
        const float4* c4 = reinterpret_cast<const float4*>(scales + 128 + half * 128);
        good &= mbar_wait(&sum_bar[buf], buf_phase, abort_flag);
        __syncwarp();
        tc_fence_after();
        const uint32_t from = lanes + buf * G::kTile;
        uint32_t r[2][32];
        tmem_ld32_start(from, r[0]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          tmem_ld32_wait(r[j & 1]);
          if (j < 3) {
            tmem_ld32_start(from + 32 * (j + 1), r[(j + 1) & 1]);
          } else {
            // the last columns are here: the next block but one may be formed
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_read(read_leader + buf * 8u);
          }
#pragma unroll
          for (int p = 0; p < 16; p += 2) {
            float2 a = pair_of(r[j & 1], p), b = pair_of(r[j & 1], p + 1);
            if (kCols) {
              const float4 c = c4[j * 8 + p / 2];
              a = __fmul2_rn(a, make_float2(c.x, c.y));
              b = __fmul2_rn(b, make_float2(c.z, c.w));
            }
            acc[j * 16 + p] = __ffma2_rn(a, make_float2(s, s), acc[j * 16 + p]);
            acc[j * 16 + p + 1] = __ffma2_rn(b, make_float2(s, s), acc[j * 16 + p + 1]);
          }
        }
        buf ^= 1u;
        if (buf == 0) buf_phase ^= 1u;
        if (at == G::kAhead - 1 || k == g.blocks - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&used_bar[slot]);
          if (++slot == G::kRing) {
            slot = 0;
            slot_phase ^= 1u;
          }
        }
      }
      const int64_t m_first = static_cast<int64_t>(mt) * G::kTile + rank * 128 + quad * 32;
      const int64_t n0 = static_cast<int64_t>(nt) * G::kTile + half * 128;
      if (!good) fail();
      if (!good) {  // a wait gave up: its elements are not a number
#pragma unroll
        for (int j = 0; j < 64; ++j) acc[j] = both_nan();
      }
      if (g.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < 64; ++j) {
          acc[j].x += bias_at(g, n0 + 2 * j);
          acc[j].y += bias_at(g, n0 + 2 * j + 1);
        }
      }
      // out through shared memory, 32 rows of 128 bytes at a time, 16-byte units
      // permuted by row
      const int slab_cols = g.y_f32 ? 32 : 64;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (!g.y_f32 && c >= 2) break;
        const int64_t n = n0 + c * slab_cols;
        if (n >= g.N || m_first >= g.M) break;
        if (tma_store) {
          if (lane == 0) bulk_wait_read_all();  // the last store has read the slab
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint4 u;
          if (g.y_f32) {
            const float2 a = acc[c * 16 + 2 * j], b = acc[c * 16 + 2 * j + 1];
            u = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                           __float_as_uint(b.y));
          } else {
            const int at = (c & 1) * 32 + 4 * j;
            u = make_uint4(pack_bf16x2(acc[at].x, acc[at].y),
                           pack_bf16x2(acc[at + 1].x, acc[at + 1].y),
                           pack_bf16x2(acc[at + 2].x, acc[at + 2].y),
                           pack_bf16x2(acc[at + 3].x, acc[at + 3].y));
          }
          *reinterpret_cast<uint4*>(slab + lane * 128 + ((j ^ (lane & 7)) << 4)) = u;
        }
        if (tma_store) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (g.accumulate)
              tma_reduce_add_2d(&map_y, slab, static_cast<int>(n), static_cast<int>(m_first));
            else
              tma_store_2d(&map_y, slab, static_cast<int>(n), static_cast<int>(m_first));
            bulk_commit();
          }
        } else {
          // rows that a copy cannot start in: element by element, lanes along a row
          __syncwarp();
          const int rows = static_cast<int>(min(int64_t(32), g.M - m_first));
          const int width = static_cast<int>(min(static_cast<int64_t>(slab_cols), g.N - n));
          for (int r = 0; r < rows; ++r) {
            const int64_t at = (m_first + r) * g.ldy + n;
            for (int e = lane; e < width; e += 32) {
              const int byte = e * (g.y_f32 ? 4 : 2);
              const uint8_t* from = slab + r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15);
              if (g.y_f32) {
                float* y = static_cast<float*>(g.y) + at + e;
                const float v = *reinterpret_cast<const float*>(from);
                *y = g.accumulate ? *y + v : v;
              } else {
                static_cast<uint16_t*>(g.y)[at + e] = *reinterpret_cast<const uint16_t*>(from);
              }
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync();  // both CTAs done with the pair's tensor memory and shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace flce
