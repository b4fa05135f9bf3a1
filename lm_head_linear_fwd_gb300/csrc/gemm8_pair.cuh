// gemm8 for many tokens: 256 x 256 tiles on pairs of CTAs.
//
// The pair's two SMs form one tile with tcgen05.mma.cta_group::2: each loads its 128
// rows of a and 128 of the tile's 256 rows of b, and has 128 rows of the sums in its
// tensor memory.  Eight warps add them up, a thread 128 columns of one row, so that
// a's scale is one number per thread, and b's, where it is for 128 rows, one per warp:
// one multiply-add per element and block.  The two halves of the columns are apart: a
// thread of its own issues each half's products, into one of the half's two places in
// tensor memory while its four warps read the other, so that one half's waits fall
// into the other's additions.  A warp loads the scales, a few blocks ahead, to shared
// memory.
//
// Bound by the way of a block's sums from the tensor cores through the registers: of
// about 800 cycles per block the products take 512 and the additions 256 (packed fp32
// at half rate); the rest are the waits between them, which two warps to a scheduler
// (their sums fill the registers) hide in part.  8192 x 4096 x 16384, scales of b for
// 128 rows: 373 us, 2.9 PFLOP/s; for each row, twice the arithmetic, 531 us (519 with the
// sum times one scale formed first, which leaves fp32's range where the other scale would
// bring it back; the scales' products formed while the sums are on their way 564).  The
// scales loaded by the adding threads took 723 us (they spill), handed over for four
// blocks at a time 385 and 529; tensor memory read without a load ahead 438; one lane in
// the issuing warp's loop 446; sixteen adding warps of 64 columns 414.
//
// Barriers as in the pair kernel of tc_gemm.cuh:
//   full[s]   leader: both CTAs' copies have landed     empty[s]  both: both halves' were read
//   sum[i]    both: a half block's sums are there       read[i]   leader: its 8 warps have
//                                                       read them
//   scaled[r] both: kAhead blocks' scales are there     used[r]   both: they were used
#pragma once

#include "gemm8.cuh"
#include "tc_gemm.cuh"

namespace flce {

// kCols: b has a scale for each of its rows (the tile's columns); else one for 128.
template <bool kCols>
struct Gemm8Pair {
  // A warpgroup for copies and products, two that add up.  The registers of 384 threads
  // at launch, 168 each (65536 / 384, down to a multiple of eight), are dealt anew: 56
  // and 224, the same sum, 4 x 56 + 8 x 224 = 12 x 168.
  static constexpr int kThreads = 384;
  static constexpr int kTile = 256;     // rows of a, and of b, of a pair's tile
  static constexpr int kStageA = 128 * 128;
  static constexpr int kStageBytes = 2 * kStageA;
  static constexpr int kStages = 4;
  static constexpr int kAhead = 8;  // blocks whose scales are handed over together
  static constexpr int kRing = 2;   // of these
  static constexpr int kScales = 128 + (kCols ? 256 : 4);  // a block's: rows, then columns
  static constexpr int kScaleBytes = kRing * kAhead * kScales * 4;
  static constexpr int kStaging = 8 * 2 * 4096;
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

// 16 columns of fp32 of this thread's lane of tensor memory, to be waited for; and the
// wait for all loads of this thread, which gives the last one's values as pairs.
__device__ __forceinline__ void tmem_ld_start(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(const uint32_t (&r)[16], uint64_t (&v)[8]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;\n\t"
      "mov.b64 %0, {%8, %9};\n\t"
      "mov.b64 %1, {%10, %11};\n\t"
      "mov.b64 %2, {%12, %13};\n\t"
      "mov.b64 %3, {%14, %15};\n\t"
      "mov.b64 %4, {%16, %17};\n\t"
      "mov.b64 %5, {%18, %19};\n\t"
      "mov.b64 %6, {%20, %21};\n\t"
      "mov.b64 %7, {%22, %23};\n\t"
      : "=l"(v[0]), "=l"(v[1]), "=l"(v[2]), "=l"(v[3]), "=l"(v[4]), "=l"(v[5]), "=l"(v[6]),
        "=l"(v[7])
      : "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
      : "memory");
}
// Packed fp32 arithmetic on pairs.
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 both_of(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void fma_pair(uint64_t a, uint64_t b, uint64_t& c) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}

// Arrive on a barrier of another CTA of the cluster for tensor memory that was read:
// the loads have been waited for and no other memory is handed over, so that no wider
// fence is needed than a barrier's own.
__device__ __forceinline__ void mbar_arrive_read(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Two pairs from shared memory, here and no earlier (volatile): loaded ahead, the
// columns' scales take the registers that the sums need (675 against 580 us then).
__device__ __forceinline__ void lds_pairs(uint32_t addr, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr));
}

// The scales of four blocks from k on, of 128 rows from `first` on: each to its block's
// place, kScales further.  All loads are under way before the first is waited for.
template <int kScales>
__device__ __forceinline__ void stage_scales(const float* scales, int64_t first, int64_t rows,
                                             int k, int blocks, bool wide, int lane, float* to) {
  float4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // past the last row the last one's: their sums are not stored
    const float* row = scales + min(first + 32 * i + lane, rows - 1) * blocks;
    if (wide) {  // all four are there, on a 16-byte boundary
      v[i] = *reinterpret_cast<const float4*>(row + k);
    } else {
      const int last = blocks - 1;
      v[i].x = row[k];
      v[i].y = row[min(k + 1, last)];
      v[i].z = row[min(k + 2, last)];
      v[i].w = row[min(k + 3, last)];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float* at = to + 32 * i + lane;
    at[0] = v[i].x;
    at[kScales] = v[i].y;
    at[2 * kScales] = v[i].z;
    at[3 * kScales] = v[i].w;
  }
}

// kTma: the rows of y can be stored by copies (16-byte addresses and strides).
template <bool kCols, bool kTma>
__global__ void __launch_bounds__(Gemm8Pair<kCols>::kThreads, 1)
    gemm8_pair_kernel(const __grid_constant__ CUtensorMap map_a,
                      const __grid_constant__ CUtensorMap map_b,
                      const __grid_constant__ CUtensorMap map_y, const Gemm8Args g,
                      const int group_m) {
  using G = Gemm8Pair<kCols>;
  constexpr int S = G::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full_bar[S], empty_bar[S], sum_bar[4], read_bar[4], drain_bar[2];
  __shared__ uint64_t scaled_bar[G::kRing], used_bar[G::kRing];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  float* scale_ring = reinterpret_cast<float*>(smem + S * G::kStageBytes + G::kStaging);
  volatile int* abort_flag = &abort_sh;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sum_bar[i], 1);
      mbar_init(&read_bar[i], 8);
    }
    for (int i = 0; i < G::kRing; ++i) {
      mbar_init(&scaled_bar[i], 1);
      mbar_init(&used_bar[i], 8);
    }
    mbar_init(&drain_bar[0], 1);
    mbar_init(&drain_bar[1], 1);
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
        const int brow = nt * G::kTile + static_cast<int>(rank) * 64;
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
          tma_load_2d_pair(to + G::kStageA + G::kStageA / 2, &map_b, bar, k * 128, brow + 128);
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
    __syncwarp();  // one lane has copied: the barrier at the end wants whole warps
  } else if (warp <= 2) {
    if (leader) {
      // products of one half of the tile's columns: the sums of one block after the other
      const int h = warp - 1;
      constexpr uint32_t idesc = make_idesc(0, 256, 128, false, false);  // 0: e4m3
      const uint64_t desc = smem_desc_sw128(smem_u32(smem), 16, 1024);
      uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        for (int k = 0; k < g.blocks; ++k) {
          ok = mbar_wait(&read_bar[2 * h + buf], buf_phase ^ 1u, abort_flag) &&
               mbar_wait(&full_bar[stage], phase, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t da = desc + stage * (G::kStageBytes / 16);
            const uint64_t db = da + (G::kStageA + h * (G::kStageA / 2)) / 16;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_8bit_pair(tmem_base + h * G::kTile + buf * 128, da + 2 * j, db + 2 * j, idesc,
                            j > 0 ? 1u : 0u);
            mma_commit_pair(&empty_bar[stage], 0x3);
            mma_commit_pair(&sum_bar[2 * h + buf], 0x3);
          }
          __syncwarp();
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
          buf ^= 1u;
          if (buf == 0) buf_phase ^= 1u;
        }
      }
      if (!ok && lane == 0) fail();
      if (elect_one()) mma_commit_pair(&drain_bar[h], 0x1);
      const uint64_t t0 = global_ns();
      while (!mbar_try_wait(smem_u32(&drain_bar[h]), 0) && global_ns() - t0 < kWaitLimitNs) {
      }
      __syncwarp();
    }
  } else if (warp < 4) {
    // scales
    const bool wide = g.blocks % 4 == 0 &&
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
        // the rows' and, each 128, the columns'
#pragma unroll 1
        for (int part = 0; part < (kCols ? 3 : 1); ++part) {
          const float* scales = part == 0 ? g.a_scales : g.b_scales;
          const int64_t from = part == 0 ? m0 : n0 + (part - 1) * 128;
          const int64_t rows = part == 0 ? g.M : g.N;
#pragma unroll 1
          for (int c = k; c < min(k + G::kAhead, g.blocks); c += 4)
            stage_scales<G::kScales>(scales, from, rows, c, g.blocks, wide, lane,
                                     to + (c - k) * G::kScales + part * 128);
        }
        if (!kCols && lane < 2 * G::kAhead) {
          const int64_t n = min(n0 / kBlock8 + lane % 2, (g.N - 1) / kBlock8);
          const int at = lane / 2;
          to[at * G::kScales + 128 + lane % 2] =
              g.b_scales[n * g.blocks + min(k + at, g.blocks - 1)];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&scaled_bar[slot]);
        if (++slot == G::kRing) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // sums: a thread has 128 columns of one row
    const int quad = warp & 3;         // the tensor memory lanes this warp may access
    const int half = (warp - 4) >> 2;  // its half of the columns
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) +
                           static_cast<uint32_t>(half * G::kTile);
    uint8_t* slabs = smem + S * G::kStageBytes + (warp - 4) * 8192;
    uint32_t buf = 0, buf_phase = 0, slot = 0, slot_phase = 0;
    int next_slab = 0;
    for (int t = first; t < tiles; t += step) {
      int mt, nt;
      tile_coords(t, nm, nn, group_m, mt, nt);
      uint64_t sums[64];  // pairs of columns
#pragma unroll
      for (int j = 0; j < 64; ++j) sums[j] = 0;
      // the next block's scale is asked for while this one's columns are added
      bool good = mbar_wait(&scaled_bar[slot], slot_phase, abort_flag);
      const float* scales = scale_ring + slot * G::kAhead * G::kScales;
      float row_s = scales[quad * 32 + lane], col_s = kCols ? 1.0f : scales[128 + half];
      for (int k = 0; k < g.blocks; ++k) {
        const int at = k & (G::kAhead - 1);
        const bool last = k + 1 == g.blocks, slot_done = last || at == G::kAhead - 1;
        const float s = kCols ? row_s : __fmul_rn(row_s, col_s);
        const uint64_t s2 = pair_of(s, s);
        good &= mbar_wait(&sum_bar[2 * half + buf], buf_phase, abort_flag);
        __syncwarp();
        tc_fence_after();
        const uint32_t from = lanes + buf * 128;
        // !kCols: kLoad columns are on their way while those before them are added (438
        // against 385 us; kCols the other way round, 511 and 534)
        constexpr int kLoad = 16, kLast = 128 / kLoad - 1;
        uint32_t r[2][kLoad];
        if (!kCols) tmem_ld_start(from, r[0]);
#pragma unroll
        for (int j = 0; j <= kLast; ++j) {
          uint64_t v[kLoad / 2];
          if (kCols) tmem_ld_start(from + kLoad * j, r[j & 1]);
          tmem_ld_wait(r[j & 1], v);
          if (!kCols && j < kLast) tmem_ld_start(from + kLoad * (j + 1), r[(j + 1) & 1]);
          if (j == kLast / 2 && !last && !slot_done) {
            row_s = scales[G::kScales + quad * 32 + lane];
            if (!kCols) col_s = scales[G::kScales + 128 + half];
          }
          if (j == kLast) {
            // the last columns are here: the next block but one may be formed
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_read(read_leader + (2 * half + buf) * 8u);
          }
          if constexpr (kCols) {
            const uint32_t at_cols = smem_u32(scales + 128 + half * 128 + j * kLoad);
#pragma unroll
            for (int p = 0; p < kLoad / 2; p += 4) {
              uint64_t c[4];
              lds_pairs(at_cols + p * 8, c[0], c[1]);
              lds_pairs(at_cols + p * 8 + 16, c[2], c[3]);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                // the scales' product first: a sum times one of them may leave fp32's range
                fma_pair(v[p + q], mul_pair(c[q], s2), sums[j * (kLoad / 2) + p + q]);
              }
            }
          } else {
#pragma unroll
            for (int p = 0; p < kLoad / 2; ++p) fma_pair(v[p], s2, sums[j * (kLoad / 2) + p]);
          }
        }
        buf_phase ^= buf;
        buf ^= 1u;
        scales += G::kScales;
        if (slot_done) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&used_bar[slot]);
          if (++slot == G::kRing) {
            slot = 0;
            slot_phase ^= 1u;
          }
          if (!last) {
            good &= mbar_wait(&scaled_bar[slot], slot_phase, abort_flag);
            scales = scale_ring + slot * G::kAhead * G::kScales;
            row_s = scales[quad * 32 + lane];
            if (!kCols) col_s = scales[128 + half];
          }
        }
      }
      const int64_t m_first = static_cast<int64_t>(mt) * G::kTile + rank * 128 + quad * 32;
      const int64_t n0 = static_cast<int64_t>(nt) * G::kTile + half * 128;
      if (!good) fail();
      float2 acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = both_of(sums[j]);
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
        uint8_t* slab = slabs + next_slab * 4096;
        next_slab ^= 1;
        // a copy writes whole 16-byte units, also past the last column
        const bool copy = kTma && n + slab_cols <= g.N;
        if (kTma && lane == 0) bulk_wait_read_le1();  // the slab's last store has read it
        __syncwarp();
        if constexpr (kTma) {
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
          if (copy) {
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
            // element by element, lanes along a row
            if (lane == 0) bulk_commit();  // the slabs' stores are counted
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
        } else {
          const int rows = static_cast<int>(min(int64_t(32), g.M - m_first));
          const int width = static_cast<int>(min(static_cast<int64_t>(slab_cols), g.N - n));
          const int64_t first_at = m_first * g.ldy + n;
          // bf16: pairs from the row's first 4-byte boundary on
          const int64_t row0 =
              static_cast<int64_t>(reinterpret_cast<uintptr_t>(g.y) >> 1) + first_at;
          const bool shift = !g.y_f32 && ((row0 + lane * g.ldy) & 1) != 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint4 u;
            if (g.y_f32) {
              const float2 a = acc[c * 16 + 2 * j], b = acc[c * 16 + 2 * j + 1];
              u = make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                             __float_as_uint(b.y));
            } else {
              const float2* v = acc + (c & 1) * 32;
              uint32_t w[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int i = 4 * j + q;
                w[q] = pack_bf16x2(v[i].x, v[i].y);
                const float next = i < 31 ? v[i + 1 < 32 ? i + 1 : 31].x : 0.0f;
                if (shift) w[q] = pack_bf16x2(v[i].y, next);
              }
              u = make_uint4(w[0], w[1], w[2], w[3]);
            }
            *reinterpret_cast<uint4*>(slab + lane * 128 + ((j ^ (lane & 7)) << 4)) = u;
          }
          // word by word, lanes along a row
          if (shift && lane < rows)
            Elem<__nv_bfloat16>::store(
                static_cast<__nv_bfloat16*>(g.y) + first_at + lane * g.ldy, acc[(c & 1) * 32].x);
          __syncwarp();
#pragma unroll 4
          for (int r = 0; r < rows; ++r) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(
                slab + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
            const int64_t at = first_at + r * g.ldy;
            if (g.y_f32) {
              float* y = static_cast<float*>(g.y) + at + lane;
              if (lane < width) *y = g.accumulate ? *y + __uint_as_float(w) : __uint_as_float(w);
            } else {
              const int e = 2 * lane + static_cast<int>((row0 + r * g.ldy) & 1);
              uint16_t* y = static_cast<uint16_t*>(g.y) + at + e;
              if (e + 1 < width)
                *reinterpret_cast<uint32_t*>(y) = w;
              else if (e < width)
                *y = static_cast<uint16_t>(w);
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
