// The 4-bit head for up to 16 token columns, and 32 with groups of 32: mma.sync.
//
// Bound by the weights' bytes (V D / 2) for a few tokens.  Every weight is read once,
// unpacked in registers and multiplied by instructions whose 16 rows are vocabulary
// rows and whose 8 columns are tokens, so up to 8 tokens cost the same instructions
// as one.  Where there are fewer tiles of 32 rows than warps, wk warps split the
// columns of a tile and add up their sums in warp order.
//
// In a stage a lane holds, for rows g and g + 8 of an instruction (g = lane / 4), the
// 32-bit words w = 0..3 of its t = lane % 4: word w of the four lanes covers the
// columns 32 w .. 32 w + 31, so each pair of instructions stays within 32 columns and
// any group of 32, 64 or 128 columns can be scaled on its own.
//
// One token on 128256 x 4096 with groups of 128 takes 58.5 us (4.6 TB/s of weights),
// with groups of 32 and zero points 76; two instructions' rows to each of 16 warps
// (four to each of 8: 61 and 102).  The instruction's rate bounds more columns: 8
// token columns cost about 45 us there, 16 tokens take 99 us and 32 would take 192.
// At 128 registers 16 columns spill 8 to 40 bytes, 8 with groups of 32 8 to 24, and 32
// with groups of 32 208 to 216.
#pragma once

#include "head4.cuh"

namespace flce {

constexpr int kXPad = 64;  // bytes after a token's row: eight lanes' reads in 32 banks

// c (+)= a b for 16 rows x 16 columns by 16 x 8, bf16 with fp32 sums; `fresh`
// starts from zero.
__device__ __forceinline__ void mma_bf16(float (&c)[4], bool fresh, uint32_t a0, uint32_t a1,
                                         uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  const float z0 = fresh ? 0.0f : c[0], z1 = fresh ? 0.0f : c[1];
  const float z2 = fresh ? 0.0f : c[2], z3 = fresh ? 0.0f : c[3];
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z0), "f"(z1), "f"(z2), "f"(z3));
}


// G32: 32-column pieces per group; ST: the scales' type; NT: instructions'
// widths of 8 token columns.
template <int G32, typename ST, int NT>
__global__ void __launch_bounds__(32 * kWarps, 1)
    head4_few_kernel(const __grid_constant__ Head4Args a) {
  using Rows = RowStream<G32, ST, 32>;
  constexpr int SPW = Rows::SPW, SW = Rows::SW, ZW = Rows::ZW;
  constexpr int R = 2;  // the instruction's 16 rows in a warp's 32
  // The scales times a power of two that cannot overflow, where the product makes for
  // better code: 16 tokens on 128256 x 4096 in groups of 128 take 99.3 us with it and
  // 103.3 without, 32 in groups of 32 219.8 and 222; one in groups of 32 with zero
  // points 80.3 and 75.9.
  constexpr float kHalf = NT > 1 ? 0.5f : 1.0f;
  extern __shared__ __align__(128) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * (kRingStages * kWarpStage);
  char* xs = smem + kRing;
  const char* ring_p = smem + warp * (kRingStages * kWarpStage);
  const uint32_t xstride = static_cast<uint32_t>(a.chunk * 2 + kXPad);

  Rows rows(a, ring, warp, kWarps, 0);
  const int stages = rows.stages, wk = rows.wk, kw = rows.kw;
  const int chunk_stages = static_cast<int>(a.chunk / kStageCols);
  const int chunks = (stages + chunk_stages - 1) / chunk_stages;
  rows.fetch(0);
  uint32_t sc[SW], zp[ZW];
  rows.fetch_scales(sc, zp);
  auto place = [&](int row, int j) { return reinterpret_cast<uint4*>(xs + row * xstride + 16 * j); };
  if (chunks == 1) {
    stage_tokens(a, 0, place);
    __syncthreads();
  }
  uint32_t xrow[NT];  // this lane's token column (beyond the last: its result is not used)
#pragma unroll
  for (int n = 0; n < NT; ++n) xrow[n] = min(n * 8 + g, a.cols - 1) * xstride + t * 16;
  int slot = 0;
  float acc[R][NT][4];
  for (int round = 0; round < rows.rounds; ++round) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][n][e] = 0.0f;
    const bool real = rows.first_row(round) < a.V;
    int stage = kw;
    for (int c = 0; c < chunks; ++c) {
      if (chunks > 1) {
        __syncthreads();  // everyone is done with the last chunk
        stage_tokens(a, c * a.chunk, place);
        __syncthreads();
      }
      const int end = min(stages, (c + 1) * chunk_stages);
      for (; stage < end; stage += wk) {
        rows.fetch(slot ^ 1);
        uint32_t next_sc[SW], next_zp[ZW];
        rows.fetch_scales(next_sc, next_zp);
        cp_async_wait<1>();
        __syncwarp();
        if (real) {
          const uint32_t x0 = (stage - c * chunk_stages) * (kStageCols * 2);
          const char* w0 = ring_p + slot * kWarpStage + g * kStageBytes;
          uint32_t s_lo[R], s_hi[R], z_lo[R], z_hi[R];  // rows g and g + 8 of each tile
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // blocks of 128 columns
            uint4 lo[R], hi[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const char* at = w0 + r * 16 * kStageBytes + (((h * 4 + t) ^ Rows::swizzle(g)) * 16);
              lo[r] = *reinterpret_cast<const uint4*>(at);
              hi[r] = *reinterpret_cast<const uint4*>(at + 8 * kStageBytes);
            }
            float part[R][NT][4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const int gi = (h * 4 + w) / G32;
              uint4 b[NT];
#pragma unroll
              for (int n = 0; n < NT; ++n)
                b[n] = *reinterpret_cast<const uint4*>(xs + xrow[n] + x0 + (h * 4 + w) * 64);
#pragma unroll
              for (int r = 0; r < R; ++r) {
                const int src = r * 16 + g;
                uint32_t zl = 0xbd88bd88u, zh = 0xbd88bd88u;
                if (a.zeros != nullptr) {
                  if (w % G32 == 0 && gi % 4 == 0) {
                    z_lo[r] = __shfl_sync(0xffffffffu, zp[gi / 4], src);
                    z_hi[r] = __shfl_sync(0xffffffffu, zp[gi / 4], src + 8);
                  }
                  zl = ((z_lo[r] >> (8 * (gi % 4))) & 15u) * 0x10001u | 0xbd80bd80u;
                  zh = ((z_hi[r] >> (8 * (gi % 4))) & 15u) * 0x10001u | 0xbd80bd80u;
                }
                const uint32_t wl = w == 0 ? lo[r].x : w == 1 ? lo[r].y : w == 2 ? lo[r].z : lo[r].w;
                const uint32_t wh = w == 0 ? hi[r].x : w == 1 ? hi[r].y : w == 2 ? hi[r].z : hi[r].w;
                {
                  const uint32_t a0 = unpack_pair<0>(wl, zl), a1 = unpack_pair<0>(wh, zh);
                  const uint32_t a2 = unpack_pair<1>(wl, zl), a3 = unpack_pair<1>(wh, zh);
#pragma unroll
                  for (int n = 0; n < NT; ++n)
                    mma_bf16(part[r][n], w % G32 == 0, a0, a1, a2, a3, b[n].x, b[n].y);
                }
                {
                  const uint32_t a0 = unpack_pair<2>(wl, zl), a1 = unpack_pair<2>(wh, zh);
                  const uint32_t a2 = unpack_pair<3>(wl, zl), a3 = unpack_pair<3>(wh, zh);
#pragma unroll
                  for (int n = 0; n < NT; ++n)
                    mma_bf16(part[r][n], false, a0, a1, a2, a3, b[n].z, b[n].w);
                }
                if (w % G32 == G32 - 1) {
                  if (gi % SPW == 0) {
                    s_lo[r] = __shfl_sync(0xffffffffu, sc[gi / SPW], src);
                    s_hi[r] = __shfl_sync(0xffffffffu, sc[gi / SPW], src + 8);
                  }
                  float sl, sh;
                  if constexpr (SPW == 1) {
                    sl = __uint_as_float(s_lo[r]), sh = __uint_as_float(s_hi[r]);
                  } else if (gi & 1) {
                    sl = bf16_hi(s_lo[r]), sh = bf16_hi(s_hi[r]);
                  } else {
                    sl = bf16_lo(s_lo[r]), sh = bf16_lo(s_hi[r]);
                  }
                  sl *= kHalf;
                  sh *= kHalf;
#pragma unroll
                  for (int n = 0; n < NT; ++n) {
                    acc[r][n][0] += part[r][n][0] * sl;
                    acc[r][n][1] += part[r][n][1] * sl;
                    acc[r][n][2] += part[r][n][2] * sh;
                    acc[r][n][3] += part[r][n][3] * sh;
                  }
                }
              }
            }
          }
        }
        __syncwarp();  // the slot may be filled again
        slot ^= 1;
#pragma unroll
        for (int k = 0; k < SW; ++k) sc[k] = next_sc[k];
#pragma unroll
        for (int k = 0; k < ZW; ++k) zp[k] = next_zp[k];
      }
    }
    if (wk > 1) {
      // one round: the ring is no longer needed
      cp_async_wait<0>();
      __syncthreads();
      float* red = reinterpret_cast<float*>(smem);
      constexpr int kAcc = R * NT * 4;
      const float* f = &acc[0][0][0];
      if (kw > 0) {
#pragma unroll
        for (int e = 0; e < kAcc; ++e) red[(warp * kAcc + e) * 32 + lane] = f[e];
      }
      __syncthreads();
      if (kw > 0) continue;
      for (int k = 1; k < wk; ++k) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[r][n][e] += red[((warp + k) * kAcc + (r * NT + n) * 4 + e) * 32 + lane];
      }
    }
    if (!real) continue;
    auto put = [&](int64_t v, int m, float sum) {
      if (v < a.V && m < a.M) head4_put(a, v, m, sum, 2048.0f / kHalf, head4_bias(a, v));
    };
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t v = rows.first_row(round) + r * 16 + g;
      if (!a.x_f32) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          put(v, n * 8 + 2 * t, acc[r][n][0]);
          put(v, n * 8 + 2 * t + 1, acc[r][n][1]);
          put(v + 8, n * 8 + 2 * t, acc[r][n][2]);
          put(v + 8, n * 8 + 2 * t + 1, acc[r][n][3]);
        }
      } else {
        // token m's three columns lie in the lanes and registers of their number
#pragma unroll
        for (int m = 0; m < (8 * NT) / 3; ++m) {
          float lo = 0.0f, hi = 0.0f;
#pragma unroll
          for (int part = 2; part >= 0; --part) {  // the smallest first
            const int col = 3 * m + part;
            const int src = (lane & 28) | ((col & 7) >> 1);
            lo += __shfl_sync(0xffffffffu, acc[r][col / 8][col & 1], src);
            hi += __shfl_sync(0xffffffffu, acc[r][col / 8][2 + (col & 1)], src);
          }
          if (t == (m & 3)) {
            put(v, m, lo);
            put(v + 8, m, hi);
          }
        }
      }
    }
  }
  cp_async_wait<0>();
}

}  // namespace flce
