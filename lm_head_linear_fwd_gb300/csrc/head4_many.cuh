// The 4-bit head for more than 16 token columns: tcgen05.
//
// A warpgroup streams tiles of 128 vocabulary rows, a thread to a row.  In steps of
// 128 columns the thread unpacks its row, 32 registers at a time, and stores it to
// tensor memory: the row is a row of the A operand of tcgen05.mma (128 rows x 16
// columns), the tokens are B, and each scale group has its own sum D in tensor
// memory, read back by the row's thread, which owns the row's scales.  Where there
// are fewer tiles than warpgroups, wk of them split the columns of a tile and add up
// their sums in order.
//
// Bound by the chain of a step (unpack, store, barrier, products, sums), which the
// other three warpgroups of the SM fill in part: 133 us for 32 tokens on 128256 x
// 4096 with groups of 128 (2.0 TB/s of weights), 185 us on 151936 x 5120 with groups
// of 64.  So it waits rarely and keeps to the 128 registers that 512 threads have, but
// for 12 to 20 bytes that the compiler spills: steps of 64 columns with two A's took
// 140 and 211 us, the sums read after the next step's first unpacking (which spills
// much more) 154 and 234, the products issued one step late, with no barrier but an
// mbarrier, 151 and 252; the wait below without the warp's vote 133 and 199.
#pragma once

#include "head4.cuh"

namespace flce {

constexpr int kManyCols = 32;  // token columns

// D (+)= A B^T with A (128 x 16 bf16) in tensor memory and B in shared memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}

// 32 words to 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// acc += s * 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_add32(uint32_t taddr, float s, float (&acc)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i] += s * __uint_as_float(r[i]);
}

// Waits for a phase by a whole warp, converged again afterwards (the tensor memory
// instructions that follow are the warp's).  A wait that gives up says so in *failed
// and leaves NaN in the sums, which stays there: no logit is wrong in silence.
template <int N>
__device__ __forceinline__ void wait_or_nan(uint64_t* bar, uint32_t parity, volatile int* failed,
                                            float (&acc)[N], uint64_t limit_ns = kWaitLimitNs) {
  const bool ok = mbar_wait(bar, parity, failed, limit_ns);
  if (!__all_sync(0xffffffffu, ok)) {
    *failed = 1;
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = __uint_as_float(0x7fffffffu);
  }
}

// Whether a wait of any warp of the block gave up; for all threads, after their last
// wait.
__device__ __forceinline__ bool some_wait_failed(volatile int* failed) {
  __syncthreads();
  return *failed != 0;
}

// G32: 32-column pieces per group; ST: the scales' type.
template <int G32, typename ST>
__global__ void __launch_bounds__(32 * kWarps, 1)
    head4_many_kernel(const __grid_constant__ Head4Args a) {
  using Rows = RowStream<G32, ST, 128>;
  constexpr int SW = Rows::SW, ZW = Rows::ZW;
  constexpr int kGroups = kWarps / 4;   // warpgroups
  constexpr int N = kManyCols;          // columns of D
  constexpr int kCols = 512 / kGroups;  // tensor memory columns of a warpgroup
  constexpr int kSums = 4 / G32;        // groups in 128 columns
  static_assert(64 + kSums * N <= kCols, "A and its sums");
  extern __shared__ char smem_raw[];
  char* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;  // the swizzle's atoms
  __shared__ uint32_t tmem_base_sh;
  __shared__ __align__(8) uint64_t done[kGroups];  // a warpgroup's MMAs
  __shared__ int failed_sh;
  volatile int* failed = &failed_sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp >> 2, quarter = warp & 3;
  const uint32_t ring = smem_u32(smem) + warp * (kRingStages * kWarpStage);
  const char* ring_p = smem + warp * (kRingStages * kWarpStage);
  char* xs = smem + kRing;

  Rows rows(a, ring, group, kGroups, 32 * quarter);
  const int stages = rows.stages, wk = rows.wk, kw = rows.kw;
  const int chunk_stages = static_cast<int>(a.chunk / kStageCols);
  const int chunks = (stages + chunk_stages - 1) / chunk_stages;
  rows.fetch(0);
  uint32_t sc[SW], zp[ZW];
  rows.fetch_scales(sc, zp);
  // the tokens as the B operand: 64 columns after another, K-major with the 128-byte
  // swizzle
  auto place = [&](int row, int j) {
    return reinterpret_cast<uint4*>(xs + (j >> 3) * (N * 128) + (row >> 3) * 1024 +
                                    (row & 7) * 128 + (((j & 7) ^ (row & 7)) * 16));
  };
  if (warp == 0) {
    tmem_alloc(&tmem_base_sh, 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    failed_sh = 0;
    for (int g = 0; g < kGroups; ++g) mbar_init(&done[g], 1);
    fence_barrier_init();
  }
  if (chunks == 1) stage_tokens(a, 0, place);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh + group * kCols;
  const uint32_t my_lanes = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t tm_a = tmem, tm_d = tmem + 64;
  const uint32_t xs_a = smem_u32(xs);
  constexpr uint32_t idesc = make_idesc(1, 128, N, false, false);

  int slot = 0;
  uint32_t used = 0;    // steps of 128 columns so far
  float acc[N];
  float later[kSums];   // scales of the sums that are still to be read
  // waits for the MMAs of the step before and adds up its sums
  auto add_sums = [&]() {
    wait_or_nan(&done[group], (used - 1) & 1, failed, acc);
    tc_fence_after();
#pragma unroll
    for (int d = 0; d < kSums; ++d) tmem_add32(tm_d + d * N + my_lanes, later[d], acc);
  };
  for (int round = 0; round < rows.rounds; ++round) {
    __syncwarp();
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
    const bool real = rows.first_row(round) < a.V;  // the same for the warpgroup
    int stage = kw;
    for (int c = 0; c < chunks; ++c) {
      if (chunks > 1) {
        __syncthreads();  // everyone is done with the last chunk
        stage_tokens(a, c * a.chunk, place);
        fence_proxy_async_smem();
        __syncthreads();
      }
      const int end = min(stages, (c + 1) * chunk_stages);
      bool pending = false;  // the sums of the step before are still to be read
      for (; stage < end; stage += wk) {
        rows.fetch(slot ^ 1);
        uint32_t next_sc[SW], next_zp[ZW];
        rows.fetch_scales(next_sc, next_zp);
        cp_async_wait<1>();
        __syncwarp();
        if (real) {
          const char* row = ring_p + slot * kWarpStage + lane * kStageBytes;
          const uint32_t x0 = xs_a + (stage - c * chunk_stages) * (4 * N * 128);
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // steps of 128 columns
            // A is free once the MMAs that read it last are done
            if (pending) add_sums();
            uint4 word[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
              word[t] = *reinterpret_cast<const uint4*>(
                  row + (((h * 4 + t) ^ Rows::swizzle(lane)) * 16));
#pragma unroll
            for (int q = 0; q < 2; ++q) {  // 64 columns
              uint32_t r[32];
#pragma unroll
              for (int w2 = 0; w2 < 2; ++w2) {
                const int gi = (h * 4 + q * 2 + w2) / G32;
                uint32_t mz = 0xbd88bd88u;
                if (a.zeros != nullptr)
                  mz = ((zp[gi / 4] >> (8 * (gi % 4))) & 15u) * 0x10001u | 0xbd80bd80u;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                  const uint32_t w = q == 0 ? (w2 == 0 ? word[t].x : word[t].y)
                                            : (w2 == 0 ? word[t].z : word[t].w);
                  const int at = (w2 * 4 + t) * 4;
                  r[at] = unpack_pair<0>(w, mz);
                  r[at + 1] = unpack_pair<1>(w, mz);
                  r[at + 2] = unpack_pair<2>(w, mz);
                  r[at + 3] = unpack_pair<3>(w, mz);
                }
              }
              tmem_st32(tm_a + q * 32 + my_lanes, r);
            }
            tmem_wait_st();
            tc_fence_before();
            named_barrier(1 + group, 128);
            if (quarter == 0 && lane == 0) {
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint64_t b = smem_desc_sw128(x0 + (h * 2 + (k >> 2)) * (N * 128), 16, 1024);
                mma_ts(tm_d + k / (2 * G32) * N, tm_a + k * 8, b + (k & 3) * 2, idesc,
                       k % (2 * G32) > 0);
              }
              mma_commit(&done[group]);
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < kSums; ++k) later[k] = Rows::scale_of(sc, h * kSums + k);
            ++used;
            pending = true;
          }
        }
        __syncwarp();  // the slot may be filled again
        slot ^= 1;
#pragma unroll
        for (int k = 0; k < SW; ++k) sc[k] = next_sc[k];
#pragma unroll
        for (int k = 0; k < ZW; ++k) zp[k] = next_zp[k];
      }
      if (pending) add_sums();
    }
    if (wk > 1) {
      // one round: the ring is no longer needed
      cp_async_wait<0>();
      __syncthreads();
      float* red = reinterpret_cast<float*>(smem);
      const int mine = threadIdx.x & 127;
      if (kw > 0) {
#pragma unroll
        for (int e = 0; e < N; ++e) red[(group * N + e) * 128 + mine] = acc[e];
      }
      __syncthreads();
      if (kw > 0) continue;
      for (int k = 1; k < wk; ++k) {
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] += red[((group + k) * N + e) * 128 + mine];
      }
    }
    const int64_t v = rows.first_row(round) + 32 * quarter + lane;
    if (v >= a.V) continue;
    const float bias = head4_bias(a, v);
    auto put = [&](int m, float sum) {
      if (m < a.M) head4_put(a, v, m, sum, 2048.0f, bias);
    };
    if (!a.x_f32) {
#pragma unroll
      for (int m = 0; m < N; ++m) put(m, acc[m]);
    } else {
#pragma unroll
      for (int m = 0; m < N / 3; ++m)  // the smallest part first
        put(m, acc[3 * m + 2] + acc[3 * m + 1] + acc[3 * m]);
    }
  }
  cp_async_wait<0>();
  tc_fence_before();
  if (some_wait_failed(failed)) {
    // once more for the MMAs still under way, which read the memory freed below
    if (used > 0) mbar_wait(&done[group], (used - 1) & 1, nullptr);
    __syncthreads();
    if (threadIdx.x == 0) set_status(a.status, FLCE_ETIMEOUT);
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_base_sh, 512);
  }
}

// The same wait and report with an mbarrier per warpgroup, of which nothing completes
// the last one's.  y[g] is what warpgroup g holds afterwards: 1, the last one NaN.
__global__ void __launch_bounds__(32 * kWarps) head4_wait_selftest_kernel(float* y,
                                                                          int32_t* status,
                                                                          uint64_t limit_ns) {
  constexpr int kGroups = kWarps / 4;
  __shared__ __align__(8) uint64_t done[kGroups];
  __shared__ int failed_sh;
  volatile int* failed = &failed_sh;
  const int group = threadIdx.x >> 7, in_group = threadIdx.x & 127;
  if (threadIdx.x == 0) {
    failed_sh = 0;
    for (int g = 0; g < kGroups; ++g) mbar_init(&done[g], 1);
    fence_barrier_init();
  }
  __syncthreads();
  if (in_group == 0 && group + 1 < kGroups) mbar_arrive(&done[group]);
  __syncwarp();
  float acc[1] = {1.0f};
  wait_or_nan(&done[group], 0, failed, acc, limit_ns);
  if (in_group == 0) y[group] = acc[0];
  if (some_wait_failed(failed) && threadIdx.x == 0) set_status(status, FLCE_ETIMEOUT);
}

}  // namespace flce
