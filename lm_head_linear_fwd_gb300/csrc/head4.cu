// The head with 4-bit weights and group scales: logits of a few tokens, and
// the rounding of a table to that layout.
#include <algorithm>
#include <atomic>

#include "rows.cuh"

namespace flce {

// Logits.  Bound by the weights' bytes (V D / 2) for a few tokens.  Every weight
// is read once, unpacked in registers and multiplied by tensor-core instructions
// whose 16 rows are vocabulary rows and whose 8 columns are tokens, so up to 8
// tokens cost the same instructions as one.
//
// A persistent block per SM keeps the tokens in shared memory as bf16 (all
// columns, or a chunk of them at a time) and W warps that share nothing else:
// each streams its own R tiles of 16 rows through a ring of S stages of 256
// columns (128 bytes of each row, cp.async) without waiting for other warps.
// Where there are fewer tiles than warps, WK warps split the columns of a tile
// and add up their sums in warp order.
//
// In a stage a lane holds, for rows g and g + 8 of a tile (g = lane / 4), the
// 32-bit words w = 0..3 of its t = lane % 4: word w of the four lanes covers the
// columns 32 w .. 32 w + 31, so each pair of instructions stays within 32
// columns and any group of 32, 64 or 128 columns can be scaled on its own.  A
// word's nibble pairs (p, p + 4) become bf16 pairs by putting the nibble into the
// mantissa of 128: 128 + q, and one fused multiply-add to (q - z) 2^-11, both
// exact.  The power of two keeps a group's sum (up to 128 * 15 |x|) within fp32
// for any x; the scales carry its inverse.

constexpr int kStageCols = 256;
constexpr int kStageBytes = kStageCols / 2;
constexpr int kXPad = 64;  // bytes after a token's row: eight lanes' reads in 32 banks

struct Head4Args {
  const void* x;
  int x_f32, M;          // tokens of this launch
  int64_t D, ldx;
  const uint8_t* packed;
  int64_t ldp;
  const void* scales;
  const uint8_t* zeros;
  int64_t V, G;
  const void* bias;
  void* y;
  int y_f32;
  int64_t ldy;
  int cols;              // token columns: M, or 3 M for fp32 tokens
  int64_t chunk;         // columns of x in shared memory (a multiple of kStageCols)
  int wk;                // warps that share a tile's columns
  int64_t tiles;         // of 16 R rows
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;  // the rest is filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

// (q - z) 2^-11 of nibbles P and P + 4 as a bf16 pair; minus_z = -(128 + z) 2^-11
// in both halves.
template <int P>
__device__ __forceinline__ uint32_t unpack_pair(uint32_t word, uint32_t minus_z) {
  uint32_t v, r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;"  // (a & b) | c
      : "=r"(v)
      : "r"(word >> (4 * P)), "r"(0x000f000fu), "r"(0x43004300u));
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0x3a003a00u), "r"(minus_z));
  return r;
}

// Columns [k0, k0 + chunk) of the tokens to shared memory as bf16, zeros from D
// on.  An fp32 value becomes three rows: its upper 16 bits, the upper 16 bits of
// what is left, and the rest (each at most 8 significant bits: exact).
__device__ void stage_tokens(const Head4Args& a, int64_t k0, char* xs, int64_t stride) {
  const int per = static_cast<int>(a.chunk / 8);
  const bool wide = !a.x_f32 && a.ldx % 8 == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0;
  for (int i = threadIdx.x; i < a.M * per; i += blockDim.x) {
    const int m = i / per, j = i - m * per;
    const int64_t k = k0 + 8 * j;
    if (!a.x_f32) {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.x) + m * a.ldx + k;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (wide && k + 8 <= a.D) {
        v = *reinterpret_cast<const uint4*>(p);
      } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (k + e < a.D)
            w[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[e])
                        << (16 * (e & 1));
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      *reinterpret_cast<uint4*>(xs + m * stride + 16 * j) = v;
    } else {
      const float* p = static_cast<const float*>(a.x) + m * a.ldx + k;
      uint32_t w[3][4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v = k + e < a.D ? p[e] : 0.0f;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const uint32_t top = (__float_as_uint(v) >> 16) | (v != v ? 0x40u : 0u);
          w[part][e / 2] = (e & 1) ? w[part][e / 2] | (top << 16) : top;
          const float head = __uint_as_float(top << 16);
          // an infinity or NaN stands in the first part alone
          v = fabsf(head) <= 3.4e38f ? v - head : 0.0f;
        }
      }
#pragma unroll
      for (int part = 0; part < 3; ++part)
        *reinterpret_cast<uint4*>(xs + (3 * m + part) * stride + 16 * j) =
            make_uint4(w[part][0], w[part][1], w[part][2], w[part][3]);
    }
  }
}

// G32: 32-column pieces per group; ST: the scales' type; NT: instructions'
// widths of 8 token columns.
template <int G32, typename ST, int NT, int R, int W, int S>
__global__ void __launch_bounds__(32 * W, 1) head4_kernel(const __grid_constant__ Head4Args a) {
  extern __shared__ __align__(128) char smem[];
  constexpr int kRows = 16 * R;
  constexpr int kSlot = kRows * kStageBytes;
  constexpr int GP = 8 / G32;        // groups of a row in a stage
  constexpr int RR = kRows / 32;     // rows whose scales a lane fetches
  constexpr int SPW = 4 / sizeof(ST);  // scales per word
  constexpr int SW = GP / SPW;         // words of a row's scales in a stage
  constexpr int ZW = (GP + 3) / 4;     // words of its zero points
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * (S * kSlot);
  char* xs = smem + W * S * kSlot;
  const char* ring_p = smem + warp * (S * kSlot);
  const uint32_t xstride = static_cast<uint32_t>(a.chunk * 2 + kXPad);

  const int wk = a.wk, wr = warp / wk, kw = warp - wr * wk;
  const int per_round = W / wk;
  const int64_t span = static_cast<int64_t>(per_round) * gridDim.x;
  const int rounds = static_cast<int>((a.tiles + span - 1) / span);
  const int stages = static_cast<int>((a.D + kStageCols - 1) / kStageCols);
  const int chunk_stages = static_cast<int>(a.chunk / kStageCols);
  const int chunks = (stages + chunk_stages - 1) / chunk_stages;
  const int64_t row_bytes = (a.D + 127) / 128 * 64;

  // the warp's stages in order: round by round, within each its columns
  auto first_row = [&](int round) {
    return ((static_cast<int64_t>(round) * per_round + wr) * gridDim.x + blockIdx.x) * kRows;
  };
  // One cursor for the weights, S - 1 stages ahead, and one for the scales, one
  // stage ahead.  Rows past the last one read it again; a round without rows
  // reads nothing.
  struct Cursor {
    int round, stage;
    bool real;
  };
  const int sub = lane >> 3;                                    // row within four
  const uint32_t dst0 = ring + sub * kStageBytes + (((lane & 7) ^ ((sub & 1) * 4)) * 16);
  const int64_t step4 = 4 * a.ldp;
  const uint8_t* wp = nullptr;  // this lane's 16 bytes of stage 0 in its first row
  bool wp_last = false;         // the tile holds rows past the last
  auto enter_weights = [&](Cursor& p) {
    const int64_t row0 = first_row(p.round);
    p.real = p.round < rounds && row0 < a.V;
    wp_last = row0 + kRows > a.V;
    wp = a.packed + min(row0 + sub, a.V - 1) * a.ldp + (lane & 7) * 16;
  };
  auto fetch = [&](Cursor& p, int slot) {
    if (p.real) {
      const int at = p.stage * kStageBytes;
      const bool valid = at + (lane & 7) * 16 < row_bytes;
      const uint8_t* src = valid ? wp + at : wp - (lane & 7) * 16;
      const uint32_t dst = dst0 + slot * kSlot;
      if (!wp_last) {
#pragma unroll
        for (int i = 0; i < kRows / 4; ++i) {
          cp_async16(dst + i * 4 * kStageBytes, src, valid);
          src += step4;
        }
      } else {
        const int64_t row0 = first_row(p.round);
#pragma unroll
        for (int i = 0; i < kRows / 4; ++i) {
          const int64_t row = min(row0 + sub + 4 * i, a.V - 1);
          cp_async16(dst + i * 4 * kStageBytes,
                     a.packed + row * a.ldp + (valid ? at + (lane & 7) * 16 : 0), valid);
        }
      }
    }
    cp_async_commit();
    p.stage += wk;
    if (p.stage >= stages) {
      p.stage = kw;
      ++p.round;
      enter_weights(p);
    }
  };
  // scales (and zero points) of a stage: lane l fetches rows l, l + 32
  int64_t sp[RR];  // index of the row's first group
  auto enter_scales = [&](Cursor& p) {
    const int64_t row0 = first_row(p.round);
    p.real = p.round < rounds && row0 < a.V;
#pragma unroll
    for (int q = 0; q < RR; ++q) sp[q] = min(row0 + lane + 32 * q, a.V - 1) * a.G;
  };
  // Words as loaded (a conversion here would wait for the load), in one access
  // where rows of groups are aligned to it.
  const ST* scales = static_cast<const ST*>(a.scales);
  const bool wide_s = a.G % GP == 0 && reinterpret_cast<uintptr_t>(scales) % 16 == 0 &&
                      reinterpret_cast<uintptr_t>(a.zeros) % 8 == 0;
  auto fetch_scales = [&](Cursor& p, uint32_t (&sc)[RR][SW], uint32_t (&zp)[RR][ZW]) {
    const int g0 = p.stage * GP;
#pragma unroll
    for (int q = 0; q < RR; ++q) {
#pragma unroll
      for (int k = 0; k < SW; ++k) sc[q][k] = 0u;
#pragma unroll
      for (int k = 0; k < ZW; ++k) zp[q][k] = 0u;
      if (!p.real) continue;
      const ST* from = scales + sp[q] + g0;
      const uint8_t* zfrom = a.zeros + sp[q] + g0;
      if (wide_s) {
        if (g0 < a.G) {
#pragma unroll
          for (int k = 0; k < SW; k += 4) {
            const uint32_t* f = reinterpret_cast<const uint32_t*>(from) + k;
            if constexpr (SW == 1) {
              sc[q][0] = f[0];
            } else if constexpr (SW == 2) {
              const uint2 v = *reinterpret_cast<const uint2*>(f);
              sc[q][0] = v.x, sc[q][1] = v.y;
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(f);
              sc[q][k] = v.x, sc[q][k + 1] = v.y, sc[q][k + 2] = v.z, sc[q][k + 3] = v.w;
            }
          }
          if (a.zeros != nullptr) {
            if constexpr (GP == 2) {
              zp[q][0] = *reinterpret_cast<const uint16_t*>(zfrom);
            } else if constexpr (GP == 4) {
              zp[q][0] = *reinterpret_cast<const uint32_t*>(zfrom);
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(zfrom);
              zp[q][0] = v.x, zp[q][ZW - 1] = v.y;
            }
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < GP; ++k) {
          if (g0 + k >= a.G) continue;
          if constexpr (SPW == 1)
            sc[q][k] = reinterpret_cast<const uint32_t*>(from)[k];
          else
            sc[q][k / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(from)[k])
                            << (16 * (k & 1));
          if (a.zeros != nullptr) zp[q][k / 4] |= static_cast<uint32_t>(zfrom[k]) << (8 * (k & 3));
        }
      }
    }
    p.stage += wk;
    if (p.stage >= stages) {
      p.stage = kw;
      ++p.round;
      enter_scales(p);
    }
  };

  Cursor weights{0, kw, false}, scale{0, kw, false};
  enter_weights(weights);
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(weights, s);
  uint32_t sc[RR][SW], zp[RR][ZW];
  enter_scales(scale);
  fetch_scales(scale, sc, zp);
  if (chunks == 1) {
    stage_tokens(a, 0, xs, xstride);
    __syncthreads();
  }
  uint32_t xrow[NT];  // this lane's token column (beyond the last: its result is not used)
#pragma unroll
  for (int n = 0; n < NT; ++n) xrow[n] = min(n * 8 + g, a.cols - 1) * xstride + t * 16;
  int slot = 0;
  float acc[R][NT][4];
  for (int round = 0; round < rounds; ++round) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][n][e] = 0.0f;
    const bool real = first_row(round) < a.V;
    int stage = kw;
    for (int c = 0; c < chunks; ++c) {
      if (chunks > 1) {
        __syncthreads();  // everyone is done with the last chunk
        stage_tokens(a, c * a.chunk, xs, xstride);
        __syncthreads();
      }
      const int end = min(stages, (c + 1) * chunk_stages);
      for (; stage < end; stage += wk) {
        fetch(weights, slot + S - 1 < S ? slot + S - 1 : slot - 1);
        uint32_t next_sc[RR][SW], next_zp[RR][ZW];
        fetch_scales(scale, next_sc, next_zp);
        cp_async_wait<S - 1>();
        __syncwarp();
        if (real) {
          const uint32_t x0 = (stage - c * chunk_stages) * (kStageCols * 2);
          const char* w0 = ring_p + slot * kSlot + g * kStageBytes;
          uint32_t s_lo[R], s_hi[R], z_lo[R], z_hi[R];  // rows g and g + 8 of each tile
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // blocks of 128 columns
            uint4 lo[R], hi[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const char* at = w0 + r * 16 * kStageBytes + (((h * 4 + t) ^ ((g & 1) * 4)) * 16);
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
                const int src = (r & 1) * 16 + g;
                uint32_t zl = 0xbd88bd88u, zh = 0xbd88bd88u;
                if (a.zeros != nullptr) {
                  if (w % G32 == 0 && gi % 4 == 0) {
                    z_lo[r] = __shfl_sync(0xffffffffu, zp[r / 2][gi / 4], src);
                    z_hi[r] = __shfl_sync(0xffffffffu, zp[r / 2][gi / 4], src + 8);
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
                    s_lo[r] = __shfl_sync(0xffffffffu, sc[r / 2][gi / SPW], src);
                    s_hi[r] = __shfl_sync(0xffffffffu, sc[r / 2][gi / SPW], src + 8);
                  }
                  float sl, sh;
                  if constexpr (SPW == 1) {
                    sl = __uint_as_float(s_lo[r]), sh = __uint_as_float(s_hi[r]);
                  } else if (gi & 1) {
                    sl = bf16_hi(s_lo[r]), sh = bf16_hi(s_hi[r]);
                  } else {
                    sl = bf16_lo(s_lo[r]), sh = bf16_lo(s_hi[r]);
                  }
                  sl *= 2048.0f;
                  sh *= 2048.0f;
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
        slot = slot + 1 < S ? slot + 1 : 0;
#pragma unroll
        for (int q = 0; q < RR; ++q) {
#pragma unroll
          for (int k = 0; k < SW; ++k) sc[q][k] = next_sc[q][k];
#pragma unroll
          for (int k = 0; k < ZW; ++k) zp[q][k] = next_zp[q][k];
        }
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
    auto put = [&](int64_t v, int m, float val) {
      if (v >= a.V || m >= a.M) return;
      if (a.bias != nullptr)
        val += a.x_f32 ? static_cast<const float*>(a.bias)[v]
                       : Elem<__nv_bfloat16>::load(static_cast<const __nv_bfloat16*>(a.bias) + v);
      const int64_t at = m * a.ldy + v;
      if (a.y_f32)
        static_cast<float*>(a.y)[at] = val;
      else
        Elem<__nv_bfloat16>::store(static_cast<__nv_bfloat16*>(a.y) + at, val);
    };
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t v = first_row(round) + r * 16 + g;
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

constexpr int kSmemMost = 227 * 1024;

template <int G32, typename ST, int NT, int R, int W, int S>
static int launch_head4_k(Head4Args a, cudaStream_t s) {
  constexpr int kRing = W * S * 16 * R * kStageBytes;
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  int rc = cuda_status(cudaGetDevice(&dev), "cudaGetDevice");
  if (rc != FLCE_OK) return rc;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(raised.load() & bit)) {
    rc = cuda_status(cudaFuncSetAttribute(head4_kernel<G32, ST, NT, R, W, S>,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost),
                     "cudaFuncSetAttribute(head4_kernel)");
    if (rc != FLCE_OK) return rc;
    raised.fetch_or(bit);
  }
  const int64_t stages = (a.D + kStageCols - 1) / kStageCols;
  const int64_t fit = ((kSmemMost - kRing) / a.cols - kXPad) / (2 * kStageCols);
  a.chunk = std::min(stages, fit) * kStageCols;
  a.tiles = (a.V + 16 * R - 1) / (16 * R);
  const int sms = sm_count();
  a.wk = 1;
  while (a.wk < W && 2 * a.wk <= std::min(stages, fit) && a.tiles * 2 * a.wk <= int64_t(sms) * W)
    a.wk *= 2;
  const int64_t smem = kRing + a.cols * (a.chunk * 2 + kXPad);
  const int grid = static_cast<int>(std::min<int64_t>(a.tiles, sms));
  head4_kernel<G32, ST, NT, R, W, S><<<grid, 32 * W, static_cast<size_t>(smem), s>>>(a);
  return launch_status("head4_kernel launch");
}

// Two tiles to each of 16 warps; from 17 token columns on four to each of 8, so
// that the tokens read from shared memory serve twice the weights.  A third
// stage where the tokens leave room for it.
template <int G32, typename ST>
static int launch_head4(const Head4Args& a, cudaStream_t s) {
  if (a.cols > 16) return launch_head4_k<G32, ST, 4, 4, 8, 2>(a, s);
  if (a.cols > 8) return launch_head4_k<G32, ST, 2, 2, 16, 2>(a, s);
  const int64_t stages = (a.D + kStageCols - 1) / kStageCols;
  const int64_t x = a.cols * (stages * kStageCols * 2 + kXPad);
  if (x <= kSmemMost - 16 * 3 * 32 * kStageBytes) return launch_head4_k<G32, ST, 1, 2, 16, 3>(a, s);
  return launch_head4_k<G32, ST, 1, 2, 16, 2>(a, s);
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
                            int dt_y, int64_t ldy, flce_stream_t stream) {
  if (!valid_dtype(dt) || !valid_dtype(dt_y)) return FLCE_EDTYPE;
  if (M < 0) return FLCE_ESHAPE;
  int rc = check_head4(packed, ldp, scales, dt_s, group, V, D);
  if (rc == FLCE_OK) rc = check_matrix(x, dt, M, D, ldx);
  if (rc == FLCE_OK) rc = check_matrix(y, dt_y, M, V, ldy);
  if (rc != FLCE_OK) return rc;
  if (!aligned(bias, dtype_size(dt))) return FLCE_EALIGN;
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
