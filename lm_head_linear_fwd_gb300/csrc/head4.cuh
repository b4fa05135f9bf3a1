// The 4-bit head: what its two kernels share.
//
// A persistent block per SM keeps the tokens in shared memory as bf16 (all
// columns, or a chunk of them at a time).  Each warp streams 32 vocabulary rows at
// a time, 256 columns a stage (128 bytes of each row), through a ring of two stages
// of its own (cp.async), without waiting for other warps.
//
// A word's nibble pairs (p, p + 4) become bf16 pairs by putting the nibble into the
// mantissa of 128: 128 + q, and one fused multiply-add to (q - z) 2^-11, both
// exact.  The power of two keeps a group's sum (up to 128 * 15 |x|) within fp32
// for any x.  Its inverse comes last, with the bias: a scale times 2^11 could pass
// fp32's range.  (Logits below 2^-115 keep their bits down to 2^-138.)
#pragma once

#include "rows.cuh"

namespace flce {

constexpr int kStageCols = 256;
constexpr int kStageBytes = kStageCols / 2;
constexpr int kWarps = 16;
constexpr int kRingStages = 2;                // a third: 102 against 81 us for one token on
                                              // 128256 x 4096 with groups of 32
constexpr int kWarpStage = 32 * kStageBytes;  // bytes of a warp's stage
constexpr int kRing = kWarps * kRingStages * kWarpStage;

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
  int wk;                // warps (warpgroups) that share a tile's columns
  int64_t tiles;         // of 32 (128) rows
  int32_t* status;
};

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


// Columns [k0, k0 + chunk) of the tokens to shared memory as bf16, zeros from D on:
// columns 8 j .. 8 j + 7 of a row to *place(row, j).  An fp32 value becomes three
// rows: its upper 16 bits, the upper 16 bits of what is left, and the rest (each at
// most 8 significant bits: exact where the last part's are above 2^-133, so for |x|
// from 2^-110 on; the bits below are cut).
template <typename Place>
__device__ __forceinline__ void stage_tokens(const Head4Args& a, int64_t k0, const Place& place) {
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
      *place(m, j) = v;
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
        *place(3 * m + part, j) =
            make_uint4(w[part][0], w[part][1], w[part][2], w[part][3]);
    }
  }
}

// A warp's rows: where it is among the stages, its copies ahead and its scales.
// G32: 32-column pieces per group; ST: the scales' type; TILE: rows of a tile, of
// which the warp streams 32 from `off` on.
template <int G32, typename ST, int TILE>
struct RowStream {
  static constexpr int GP = 8 / G32;        // groups of a row in a stage
  static constexpr int SPW = 4 / sizeof(ST);  // scales per word
  static constexpr int SW = GP / SPW;         // words of a row's scales in a stage
  static constexpr int ZW = (GP + 3) / 4;     // words of its zero points

  // One cursor for the weights, a stage ahead, and one for the scales.  Rows past
  // the last one read it again; a round without rows reads nothing.
  struct Cursor {
    int round, stage;
    bool real;
  };
  const Head4Args& a;
  const int wk, kw, wr, off, per_round, rounds, stages;
  const bool wide_s;      // a stage's scales in one access
  uint32_t dst0;          // of this lane's first 16 bytes in slot 0
  Cursor weights, scale;
  const uint8_t* wp;      // this lane's 16 bytes of stage 0 in its first row
  bool wp_last;           // the tile holds rows past the last
  int64_t sp;             // index of this lane's row's first group

  // `unit` of `units` warps or warpgroups with tiles of their own
  __device__ __forceinline__ RowStream(const Head4Args& args, uint32_t ring, int unit, int units,
                                       int offset)
      : a(args),
        wk(args.wk),
        kw(unit % args.wk),
        wr(unit / args.wk),
        off(offset),
        per_round(units / args.wk),
        rounds(static_cast<int>((args.tiles + static_cast<int64_t>(per_round) * gridDim.x - 1) /
                                (static_cast<int64_t>(per_round) * gridDim.x))),
        stages(static_cast<int>((args.D + kStageCols - 1) / kStageCols)),
        wide_s(args.G % GP == 0 && reinterpret_cast<uintptr_t>(args.scales) % 16 == 0 &&
               reinterpret_cast<uintptr_t>(args.zeros) % 8 == 0),
        weights{0, kw, false},
        scale{0, kw, false} {
    const int lane = threadIdx.x & 31, sub = lane >> 3;
    dst0 = ring + sub * kStageBytes + (((lane & 7) ^ swizzle(sub)) * 16);
    enter_weights();
    enter_scales();
  }
  // A row's 16-byte pieces stand in the order c ^ swizzle(row): neither a thread per
  // row nor four threads on each of two rows meet in a bank.
  static __device__ __forceinline__ int swizzle(int row) {
    return ((row & 1) << 2) | ((row >> 1) & 3);
  }
  // the tile's first row, in the round
  __device__ __forceinline__ int64_t first_row(int round) const {
    return ((static_cast<int64_t>(round) * per_round + wr) * gridDim.x + blockIdx.x) * TILE;
  }
  __device__ __forceinline__ void enter_weights() {
    const int lane = threadIdx.x & 31;
    const int64_t row0 = first_row(weights.round);
    weights.real = weights.round < rounds && row0 < a.V;
    wp_last = row0 + TILE > a.V;
    wp = a.packed + min(row0 + off + (lane >> 3), a.V - 1) * a.ldp + (lane & 7) * 16;
  }
  // starts the copy of the next stage (an empty group of copies after the last)
  __device__ __forceinline__ void fetch(int slot) {
    const int lane = threadIdx.x & 31;
    if (weights.real) {
      const int at = weights.stage * kStageBytes;
      const bool valid = at + (lane & 7) * 16 < (a.D + 127) / 128 * 64;
      const uint32_t dst = dst0 + slot * kWarpStage;
      if (!wp_last) {
        const uint8_t* src = valid ? wp + at : wp - (lane & 7) * 16;
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // row sub + 4 i: swizzle(sub) ^ 2 (i & 1)
          cp_async16((dst ^ ((i & 1) * 32)) + i * 4 * kStageBytes, src, valid);
          src += 4 * a.ldp;
        }
      } else {
        const int64_t row0 = first_row(weights.round) + off + (lane >> 3);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          cp_async16((dst ^ ((i & 1) * 32)) + i * 4 * kStageBytes,
                     a.packed + min(row0 + 4 * i, a.V - 1) * a.ldp +
                         (valid ? at + (lane & 7) * 16 : 0),
                     valid);
      }
    }
    cp_async_commit();
    weights.stage += wk;
    if (weights.stage >= stages) {
      weights.stage = kw;
      ++weights.round;
      enter_weights();
    }
  }
  __device__ __forceinline__ void enter_scales() {
    const int64_t row0 = first_row(scale.round);
    scale.real = scale.round < rounds && row0 < a.V;
    sp = min(row0 + off + (threadIdx.x & 31), a.V - 1) * a.G;
  }
  // This lane's row's scales and zero points of the next stage, as words as loaded
  // (a conversion here would wait for the load), in one access where rows of groups
  // are aligned to it.
  __device__ __forceinline__ void fetch_scales(uint32_t (&sc)[SW], uint32_t (&zp)[ZW]) {
    const int g0 = scale.stage * GP;
#pragma unroll
    for (int k = 0; k < SW; ++k) sc[k] = 0u;
#pragma unroll
    for (int k = 0; k < ZW; ++k) zp[k] = 0u;
    if (scale.real) {
      const ST* from = static_cast<const ST*>(a.scales) + sp + g0;
      const uint8_t* zfrom = a.zeros + sp + g0;
      if (wide_s) {
        if (g0 < a.G) {
          const uint32_t* f = reinterpret_cast<const uint32_t*>(from);
          if constexpr (SW == 1) {
            sc[0] = f[0];
          } else if constexpr (SW == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(f);
            sc[0] = v.x, sc[1] = v.y;
          } else {
#pragma unroll
            for (int k = 0; k < SW; k += 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(f + k);
              sc[k] = v.x, sc[k + 1] = v.y, sc[k + 2] = v.z, sc[k + 3] = v.w;
            }
          }
          if (a.zeros != nullptr) {
            if constexpr (GP == 2) {
              zp[0] = *reinterpret_cast<const uint16_t*>(zfrom);
            } else if constexpr (GP == 4) {
              zp[0] = *reinterpret_cast<const uint32_t*>(zfrom);
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(zfrom);
              zp[0] = v.x, zp[ZW - 1] = v.y;
            }
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < GP; ++k) {
          if (g0 + k >= a.G) continue;
          if constexpr (SPW == 1)
            sc[k] = reinterpret_cast<const uint32_t*>(from)[k];
          else
            sc[k / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(from)[k])
                         << (16 * (k & 1));
          if (a.zeros != nullptr) zp[k / 4] |= static_cast<uint32_t>(zfrom[k]) << (8 * (k & 3));
        }
      }
    }
    scale.stage += wk;
    if (scale.stage >= stages) {
      scale.stage = kw;
      ++scale.round;
      enter_scales();
    }
  }
  // the scale of group gi of the stage
  static __device__ __forceinline__ float scale_of(const uint32_t (&sc)[SW], int gi) {
    if constexpr (SPW == 1) return __uint_as_float(sc[gi]);
    return (gi & 1) ? bf16_hi(sc[gi / 2]) : bf16_lo(sc[gi / 2]);
  }
};

// The bias of row v; the logit of token m and row v: its sum times `unit`, and the bias.
__device__ __forceinline__ float head4_bias(const Head4Args& a, int64_t v) {
  if (a.bias == nullptr) return 0.0f;
  return a.x_f32 ? static_cast<const float*>(a.bias)[v]
                 : Elem<__nv_bfloat16>::load(static_cast<const __nv_bfloat16*>(a.bias) + v);
}
__device__ __forceinline__ void head4_put(const Head4Args& a, int64_t v, int m, float sum,
                                          float unit, float bias) {
  const float logit = __fmaf_rn(sum, unit, bias);
  const int64_t at = m * a.ldy + v;
  if (a.y_f32)
    static_cast<float*>(a.y)[at] = logit;
  else
    Elem<__nv_bfloat16>::store(static_cast<__nv_bfloat16*>(a.y) + at, logit);
}

}  // namespace flce
