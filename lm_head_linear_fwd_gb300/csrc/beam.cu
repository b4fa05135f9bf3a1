// Beam search on the head's logits: the best continuations over beams and
// vocabulary, and the beams' states put in their order.
//
// A request has K beams.  Beam k with score s_k and logits z_k goes on with token v
// at s_k + z_k[v] - lse(z_k); the `num` best of its K V continuations are wanted,
// best first, of equal ones the one with the lowest k V + v.  Within a beam that
// order is the logits' own, so the selection splits:
//   beam_rows_kernel    a block takes a chunk of a row, reads it once (twice where its
//                       logits rise), and leaves the chunk's maximum and sum of
//                       exponentials and its `num` best tokens, as 64-bit keys: the
//                       logit's bits in an order-keeping form, then the token's
//                       complement, so that keys differ and the larger one comes first;
//   beam_merge_kernel   a block takes a request: every row's lse and best `num` keys
//                       from its chunks', then the request's from its rows'.
// Bound by latency: of a block's steps for many rows, of the two launches for few.
//
// beam_reorder_kernel moves rows of caches and histories.  Their order is a map that
// repeats some beams and drops others, in place: a thread owns 16 bytes of each of a
// request's rows, copies the rows that move to shared memory, and writes them back.
// Rows that stay where they are are not touched.  Bound by bytes.
#include <algorithm>

#include "rows.cuh"

namespace flce {

constexpr int kBeamThreads = 256;
constexpr int kBeamLong = 32, kBeamShort = 8;  // elements of a thread in a tile
constexpr int kBeamMost = 64;                  // beams of a request, and `num`
constexpr int kBeamFew = 16;                   // `num` up to which threads go by fours
// Keys that a chunk writes down under one bound: 300 are expected of 4 tiles at the largest
// `num`; ranking costs their square.
constexpr int kBeamOnce = 512;
constexpr int64_t kBeamVocab = int64_t(1) << 20;
constexpr int kBeamMergeThreads = 512;

// Order-keeping bits of a float (not NaN): larger floats, larger numbers.
__device__ __forceinline__ uint32_t ordered(float z) {
  const uint32_t u = __float_as_uint(z);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t beam_key(float z, uint32_t token) {
  // the two zeros are equal
  return static_cast<uint64_t>(ordered(z + 0.0f)) << 32 | (0xffffffffu - token);
}
__device__ __forceinline__ uint32_t key_token(uint64_t key) {
  return 0xffffffffu - static_cast<uint32_t>(key);
}
__device__ __forceinline__ float key_logit(uint64_t key) {
  return unordered(static_cast<uint32_t>(key >> 32));
}

struct BeamArgs {
  const void* logits;
  int64_t V, ld;
  const float* scores;      // [B K]
  const uint8_t* finished;  // [B K] or null
  int64_t pad;
  int K, num, chunks, tiles;
  uint64_t* keys;  // [B K, chunks, num]
  float2* sums;    // [B K, chunks]: maximum, sum of exp(z - maximum)
  float* out_scores;
  int64_t* out_tokens;
  int64_t* out_parents;
};

// A row whose logits count: its beam goes on and has a score.
__device__ __forceinline__ bool row_counts(const BeamArgs& a, int64_t row) {
  const float s = a.scores[row];
  return !(a.finished != nullptr && a.finished[row] != 0) && s > -INFINITY && s < INFINITY;
}

// A block has `tiles` tiles of ELEMS elements to a thread, one after the other.
// The block's threads, four together where `num` is at most kBeamFew, are groups; the
// num-th largest of the groups' largest keys of a tile is a bound that the tile's best
// num keys reach, and at most num groups have keys that do.  The first tile's bound
// serves the whole chunk: what reaches it is written down without a wait, some num
// keys to a tile, and ranked at the end.  Where that overflows (rows that rise) the
// chunk is read again, with a bound and the best num so far for each tile.  Bound by the
// latency of a block's loads, bound and ranking at four blocks to an SM (28 warps, issue
// slots 47% full with some 14 instructions per logit): 320 x 151936 fp32 34 of 42 us with
// the merge (5.7 TB/s; the bytes take 28.7), 128 x 128256 bf16 26 to 27 us (4.8: half the
// bytes, the same instructions, and 768 blocks for 608 places of which 128 have less than a
// tile).  With a bound for every tile, of one to a block, 52 of 61 and 31; eight tiles to a
// block 43 and 24.  The fp32 rows with their first half masked take 72 us, all equal 60,
// sorted upwards 115.
template <typename T, int ELEMS>
struct BeamTile {
  static constexpr int VEC = 16 / sizeof(T), NV = ELEMS / VEC;
  static constexpr int kSize = kBeamThreads * ELEMS, kStep = kBeamThreads * VEC;
  // keys that reach a tile's own bound, at most
  static constexpr int kRoom = kBeamMost * ELEMS > kBeamFew * 4 * ELEMS ? kBeamMost * ELEMS
                                                                        : kBeamFew * 4 * ELEMS;
  float v[ELEMS];
  int first;    // the thread's first place; -infinity outside the row
  bool inside;  // the tile lies within the row
  __device__ __forceinline__ int place(int i) const { return first + i / VEC * kStep + i % VEC; }
  // begins on a 16-byte boundary
  __device__ __forceinline__ void load(const T* z, int begin, int V) {
    first = begin + static_cast<int>(threadIdx.x) * VEC;
    inside = begin >= 0 && begin + kSize <= V;
    if (inside) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float f[VEC];
        Elem<T>::unpack(__ldcs(reinterpret_cast<const uint4*>(z + first + k * kStep)), f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[k * VEC + e] = f[e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < ELEMS; ++i) {
        const int j = place(i);
        v[i] = j >= 0 && j < V ? Elem<T>::load(z + j) : -INFINITY;
      }
    }
  }
  __device__ __forceinline__ float largest() const {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < ELEMS; ++i) m = fmaxf(m, v[i]);
    return m;
  }
  // The tile's bound (see above): the same for every thread; 0, which every key reaches,
  // where fewer than num groups have an element.  Two barriers.
  __device__ __forceinline__ uint64_t bound(float m, int V, int num, uint64_t* tops,
                                            uint64_t* bound_sh) const {
    // the thread's largest key (0, below every key, without an element): the largest
    // logit, of equal ones the first
    int at = -1;
    if (inside) {
#pragma unroll
      for (int i = ELEMS - 1; i >= 0; --i)
        if (v[i] == m) at = i / VEC * kStep + i % VEC;
      if (at >= 0) at += first;  // (all NaN: none)
    } else {
#pragma unroll
      for (int i = ELEMS - 1; i >= 0; --i) {
        const int j = place(i);
        if (v[i] == m && j >= 0 && j < V) at = j;
      }
    }
    uint64_t top = at >= 0 ? beam_key(m, static_cast<uint32_t>(at)) : 0;
    const bool by_four = num <= kBeamFew;
    if (by_four) {
#pragma unroll
      for (int o = 1; o < 4; o *= 2) {
        const uint64_t other = __shfl_xor_sync(0xffffffffu, top, o);
        top = other > top ? other : top;
      }
      if ((threadIdx.x & 3) == 0) tops[threadIdx.x / 4] = top;
    } else {
      tops[threadIdx.x] = top;
    }
    __syncthreads();
    // a group's rank: how many are larger.  By four each of its threads looks at a quarter.
    const int looked = by_four ? kBeamThreads / 16 : kBeamThreads;
    const uint64_t* at_tops = tops + (by_four ? (threadIdx.x & 3) * looked : 0);
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < looked; ++i) rank += at_tops[i] > top ? 1 : 0;
    if (by_four) {
      rank += __shfl_xor_sync(0xffffffffu, rank, 1);
      rank += __shfl_xor_sync(0xffffffffu, rank, 2);
    }
    if (rank < num && top == 0) *bound_sh = 0;
    if (rank == num - 1 && top != 0) *bound_sh = top;
    __syncthreads();
    return *bound_sh;
  }
  // Writes down the keys that reach `least`.  *count passes `room` where one finds no
  // room; the rest are then left, for the chunk is read again.
  __device__ __forceinline__ void collect(float m, uint64_t least, int V, uint64_t* keys,
                                          int room, int* count) const {
    const float z_least = least != 0 ? key_logit(least) : -INFINITY;
    if (!(m >= z_least)) return;
    uint32_t reach = 0;  // elements that may
#pragma unroll
    for (int i = 0; i < ELEMS; ++i) reach |= v[i] >= z_least ? 1u << i : 0u;
    if ((reach & (reach - 1)) != 0) {
      // Equal logits reach it up to its token.  Masked and constant tiles are equal all
      // over: not by the loop below, an element at a time.
      const uint32_t last = key_token(least);
#pragma unroll
      for (int i = 0; i < ELEMS; ++i)
        if (v[i] == z_least && static_cast<uint32_t>(place(i)) > last) reach &= ~(1u << i);
    }
    while (reach != 0) {
      const int i = __ffs(reach) - 1;
      reach &= reach - 1;
      float x = v[0];
#pragma unroll
      for (int q = 1; q < ELEMS; ++q) x = q == i ? v[q] : x;
      const int j = place(i);
      const uint64_t key = beam_key(x, static_cast<uint32_t>(j));
      if (key < least || j < 0 || j >= V) continue;
      const int slot = atomicAdd(count, 1);
      if (slot >= room) return;
      keys[slot] = key;
    }
  }
};

// The best num of n keys to `out`, largest first.
__device__ __forceinline__ void rank_keys(const uint64_t* keys, int n, int num, uint64_t* out) {
  for (int i = threadIdx.x; i < n; i += kBeamThreads) {
    const uint64_t key = keys[i];
    int r = 0;
    for (int k = 0; k < n; ++k) r += keys[k] > key ? 1 : 0;
    if (r < num) out[r] = key;
  }
}

template <typename T, int ELEMS>
__global__ void __launch_bounds__(kBeamThreads, 4) beam_rows_kernel(BeamArgs a) {
  using Tile = BeamTile<T, ELEMS>;
  constexpr int kWarps = kBeamThreads / 32;
  __shared__ uint64_t tops[kBeamThreads];
  __shared__ uint64_t found[kBeamMost + Tile::kRoom];
  static_assert(kBeamOnce <= kBeamMost + Tile::kRoom, "the first reading's keys fit");
  __shared__ uint64_t kept[kBeamMost];
  __shared__ float2 red[kWarps];
  __shared__ uint64_t bound_sh;
  __shared__ int count;
  const int64_t row = blockIdx.x / a.chunks;
  const int chunk = static_cast<int>(blockIdx.x - row * a.chunks);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (!row_counts(a, row)) return;
  const T* z = static_cast<const T*>(a.logits) + row * a.ld;
  // chunks begin on 16-byte boundaries, `off` elements before the row for the first
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T);
  const int V = static_cast<int>(a.V);
  const int begin = chunk * a.tiles * Tile::kSize - off;
  const int end = min(V, begin + a.tiles * Tile::kSize);
  if (threadIdx.x == 0) count = 0;
  Tile tile;
  // the sum of exponentials relative to the largest logit of the thread: NaN and
  // +infinity make it NaN, nothing but -infinity 0
  float m = -INFINITY, s = 0.0f;
  uint64_t least = 0;
  for (int at = begin; at < end || at == begin; at += Tile::kSize) {
    tile.load(z, at, V);
    const float tm = tile.largest();
    if (tm > m) {
      if (m > -INFINITY) s *= ex2((m - tm) * kLog2e);
      m = tm;
    }
    if (m > -INFINITY) {
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < ELEMS; ++i) t += ex2((tile.v[i] - m) * kLog2e);
      s += t;
    } else {
#pragma unroll
      for (int i = 0; i < ELEMS; ++i)
        if (tile.v[i] != tile.v[i]) s = tile.v[i];
    }
    if (at == begin) least = tile.bound(tm, V, a.num, tops, &bound_sh);
    tile.collect(tm, least, V, found, kBeamOnce, &count);
  }
  float wm = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
  if (m > -INFINITY) s *= ex2((m - wm) * kLog2e);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) red[warp] = make_float2(wm, s);
  __syncthreads();
  if (threadIdx.x == kBeamThreads - 1) {
    float bm = red[0].x, bs = 0.0f;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) bm = fmaxf(bm, red[w].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      bs += red[w].x > -INFINITY ? red[w].y * ex2((red[w].x - bm) * kLog2e) : red[w].y;
    a.sums[row * a.chunks + chunk] = make_float2(bm, bs);
  }
  uint64_t* out = a.keys + (row * a.chunks + chunk) * a.num;
  int n = count;
  if (n <= kBeamOnce) {
    rank_keys(found, n, a.num, out);
  } else {
    // again, tile by tile, the best num so far first in `found`
    n = 0;
    for (int at = begin; at < end; at += Tile::kSize) {
      tile.load(z, at, V);
      const float tm = tile.largest();
      uint64_t reach = tile.bound(tm, V, a.num, tops, &bound_sh);
      if (n == a.num && found[n - 1] > reach) reach = found[n - 1];
      if (threadIdx.x == 0) count = n;
      __syncthreads();
      tile.collect(tm, reach, V, found, kBeamMost + Tile::kRoom, &count);
      __syncthreads();
      rank_keys(found, count, a.num, kept);
      n = min(count, a.num);
      __syncthreads();
      for (int i = threadIdx.x; i < n; i += kBeamThreads) found[i] = kept[i];
      __syncthreads();
    }
    for (int i = threadIdx.x; i < n; i += kBeamThreads) out[i] = found[i];
  }
  for (int i = n + threadIdx.x; i < a.num; i += kBeamThreads) out[i] = 0;
}

// log(x) for x >= 1, off by an fp32 step of a number below 1, however large x is
// (double-precision log takes longer than all else here).
__device__ __forceinline__ double log_of_sum(float x) {
  const uint32_t u = __float_as_uint(x);
  const int e = static_cast<int>(u >> 23) - 127;
  return static_cast<double>(e) * 0.69314718055994531 +
         static_cast<double>(logf(__uint_as_float((u & 0x7fffffu) | 0x3f800000u)));
}

// The lowest num tokens, all at -infinity, but one that goes first.
__device__ __forceinline__ uint32_t nth_token(int i, bool first_set, int64_t first) {
  if (!first_set) return static_cast<uint32_t>(i);
  if (i == 0) return static_cast<uint32_t>(first);
  return static_cast<uint32_t>(i - 1 < first ? i - 1 : i);
}

__global__ void __launch_bounds__(kBeamMergeThreads) beam_merge_kernel(BeamArgs a) {
  extern __shared__ uint64_t staged[];  // [warps][chunks * num], then the beams' best
  const int64_t b = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int num = a.num, all = a.chunks * num;
  const int per = static_cast<int>(min(static_cast<int64_t>(num), a.V));  // of a beam
  uint64_t* keys = staged + warp * all;
  double* score = reinterpret_cast<double*>(staged + warps * all);   // [K][num]
  uint32_t* token = reinterpret_cast<uint32_t*>(score + a.K * num);  // [K][num]
  for (int k = warp; k < a.K; k += warps) {
    const int64_t row = b * a.K + k;
    const float s = a.scores[row];
    const bool done = a.finished != nullptr && a.finished[row] != 0;
    double base = -INFINITY;  // score - lse
    const uint64_t* from = a.keys + row * all;
    uint64_t least = 1;  // (a short chunk's places hold 0)
    if (row_counts(a, row)) {
      float m = -INFINITY, sum = 0.0f;
      for (int c = lane; c < a.chunks; c += 32) {
        const float2 p = a.sums[row * a.chunks + c];
        // a chunk's last key is a bound: its num keys reach it
        const uint64_t last = from[c * num + num - 1];
        least = last > least ? last : least;
        const float to = fmaxf(m, p.x);
        if (m > -INFINITY) sum *= ex2((m - to) * kLog2e);
        sum += p.x > -INFINITY ? p.y * ex2((p.x - to) * kLog2e) : p.y;
        m = to;
      }
      float wm = m;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, o));
      if (m > -INFINITY) sum *= ex2((m - wm) * kLog2e);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const uint64_t other = __shfl_xor_sync(0xffffffffu, least, o);
        least = other > least ? other : least;
      }
      // a NaN or +infinity among the logits, or nothing but -infinity: no distribution
      if (wm > -INFINITY && wm < INFINITY && sum >= 1.0f && sum < INFINITY)
        base = static_cast<double>(s) - (static_cast<double>(wm) + log_of_sum(sum));
    }
    const bool live = base > -INFINITY;
    if (!live) {
      const bool ended = done && s > -INFINITY && s < INFINITY;
      for (int i = lane; i < per; i += 32) {
        score[k * num + i] = ended && i == 0 ? static_cast<double>(s) : -INFINITY;
        token[k * num + i] = nth_token(i, ended, a.pad);
      }
    } else {
      // the keys that reach the largest bound are moved together, and counted off
      // against each other
      int n = 0;
      for (int i = lane; i - lane < all; i += 32) {
        const uint64_t key = i < all ? from[i] : 0;
        const unsigned in = __ballot_sync(0xffffffffu, key >= least);
        if (key >= least) keys[n + __popc(in & ((1u << lane) - 1))] = key;
        n += __popc(in);
      }
      __syncwarp();
      for (int i = lane; i < n; i += 32) {
        const uint64_t key = keys[i];
        int rank = 0;
        for (int o = 0; o < n; ++o) rank += keys[o] > key ? 1 : 0;
        if (rank < num) {
          score[k * num + rank] = base + static_cast<double>(key_logit(key));
          token[k * num + rank] = key_token(key);
        }
      }
      __syncwarp();
    }
  }
  __syncthreads();
  // a beam's continuations come best first: one of all beams' comes after all those
  // before it in its own, and those of each other beam that are better
  for (int i = threadIdx.x; i < a.K * per; i += blockDim.x) {
    const int k = i / per, p = i - k * per;
    const double s = score[k * num + p];
    int rank = p;
    for (int o = 0; o < a.K && rank < num; ++o) {
      if (o == k) continue;
      int lo = 0, hi = per;  // of equal ones the lower beam's come first
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        const double t = score[o * num + mid];
        if (o < k ? t >= s : t > s)
          lo = mid + 1;
        else
          hi = mid;
      }
      rank += lo;
    }
    if (rank >= num) continue;
    a.out_scores[b * num + rank] = static_cast<float>(s);
    a.out_tokens[b * num + rank] = token[k * num + p];
    a.out_parents[b * num + rank] = k;
  }
}

// ---------------------------------------------------------------- reordering

constexpr int kReorderThreads = 128;
constexpr int kReorderStates = 64;  // of a launch

struct ReorderState {
  char* data;
  int64_t row_stride, outer_stride, units;  // bytes; units of one row
  int64_t inner;                            // units of an inner run
  int64_t first;                            // the state's first block
};

struct ReorderArgs {
  ReorderState state[kReorderStates];
  int states, K;
  int64_t B;
  const int64_t* parents;
  int32_t* status;
};

__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// U: a unit, the largest power of two up to 16 that all addresses are multiples of.
template <typename U>
__global__ void __launch_bounds__(kReorderThreads)
    beam_reorder_kernel(const __grid_constant__ ReorderArgs a) {
  extern __shared__ uint4 moved_raw[];
  U* moved = reinterpret_cast<U*>(moved_raw);  // [K][threads]
  __shared__ int from[kBeamMost];
  int t = 0;
  while (t + 1 < a.states && static_cast<int64_t>(blockIdx.x) >= a.state[t + 1].first) ++t;
  const ReorderState& st = a.state[t];
  const int64_t block = blockIdx.x - st.first;
  const int64_t per_row = (st.units + kReorderThreads - 1) / kReorderThreads;  // blocks
  const int64_t b = block / per_row;
  const int64_t u = block % per_row * kReorderThreads + threadIdx.x;
  for (int k = threadIdx.x; k < a.K; k += kReorderThreads) {
    int64_t p = a.parents[b * a.K + k];
    if (p < 0 || p >= a.K) {  // no such beam: the row stays as it is
      set_status(a.status, FLCE_ELABEL);
      p = k;
    }
    from[k] = static_cast<int>(p);
  }
  __syncthreads();
  if (u >= st.units) return;
  const int64_t outer = u / st.inner;
  char* p = st.data + b * a.K * st.row_stride + outer * st.outer_stride +
            (u - outer * st.inner) * static_cast<int64_t>(sizeof(U));
  for (int k = 0; k < a.K; ++k) {
    if (from[k] == k) continue;
    const char* src = p + from[k] * st.row_stride;
    U* to = moved + k * kReorderThreads + threadIdx.x;
    if constexpr (sizeof(U) == 16)
      cp_async16(smem_u32(to), src);
    else if constexpr (sizeof(U) == 8)
      cp_async8(smem_u32(to), src);
    else if constexpr (sizeof(U) == 4)
      cp_async4(smem_u32(to), src);
    else
      *to = *reinterpret_cast<const U*>(src);
  }
  cp_async_commit();
  cp_async_wait<0>();
  for (int k = 0; k < a.K; ++k)
    if (from[k] != k)
      *reinterpret_cast<U*>(p + k * st.row_stride) = moved[k * kReorderThreads + threadIdx.x];
}

// ------------------------------------------------------------------------ host

// How rows are cut: elements of a thread in a tile, tiles of a chunk.  Long tiles where
// they fill half of the places for blocks, several to a chunk where there are more; else
// short ones (4 x 50257 fp32: 8.8 against 9.3 us.  A long vocabulary pays for them in the
// merge, whose block has the chunks of all rows of a request: 8 x 128256 bf16 of one
// request 27.7 against 14.8).
struct BeamPlan {
  int elems, tiles;
  int64_t chunks;
};

static BeamPlan beam_plan(int64_t R, int64_t V) {
  const int64_t room = static_cast<int64_t>(sm_count()) * 4;  // blocks at a time
  BeamPlan p{kBeamLong, 1, 0};
  const int64_t tiles = R * (V / (kBeamThreads * kBeamLong));
  if (tiles < room / 2 && V <= kBeamVocab / 2)  // (the merge holds a row's keys)
    p.elems = kBeamShort;
  else
    p.tiles = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(4, tiles / room)));
  // a row may begin inside a 16-byte block: its first chunk is up to 7 elements short
  const int64_t chunk = static_cast<int64_t>(kBeamThreads) * p.elems * p.tiles;
  p.chunks = (V + 7 + chunk - 1) / chunk;
  return p;
}

static bool beam_sizes(int64_t B, int64_t K, int64_t V, int64_t num) {
  constexpr int64_t kChunk = kBeamThreads * kBeamShort;  // of the most blocks (beam_plan)
  return B >= 0 && B <= 0x7fffffff / kBeamMost && K >= 1 && K <= kBeamMost && V >= 1 &&
         V <= kBeamVocab && num >= 1 && num <= kBeamMost && num <= K * V &&
         B * K * ((V + 7 + kChunk - 1) / kChunk) <= 0x7fffffff;
}

template <typename U>
static int launch_reorder(const ReorderArgs& a, int64_t blocks, cudaStream_t s) {
  static std::atomic<uint64_t> raised{0};
  const int rc = raise_smem(beam_reorder_kernel<U>, kBeamMost * kReorderThreads * 16, raised);
  if (rc != FLCE_OK) return rc;
  beam_reorder_kernel<U><<<static_cast<unsigned>(blocks), kReorderThreads,
                           a.K * kReorderThreads * sizeof(U), s>>>(a);
  return launch_status("beam_reorder_kernel launch");
}

// The largest power of two up to 16 that a state's address, runs and strides are
// multiples of.
static int reorder_unit(const flce_beam_state_t& t, int64_t R) {
  uint64_t bits = reinterpret_cast<uintptr_t>(t.data) | static_cast<uint64_t>(t.inner) | 16u;
  if (R > 1) bits |= static_cast<uint64_t>(t.row_stride);
  if (t.outer > 1) bits |= static_cast<uint64_t>(t.outer_stride);
  return static_cast<int>(bits & (~bits + 1));
}

static int64_t reorder_blocks(const flce_beam_state_t& t, int64_t B, int unit) {
  const int64_t units = t.outer * (t.inner / unit);
  const int64_t per_row = (units + kReorderThreads - 1) / kReorderThreads;
  return per_row > 0x7fffffff ? per_row : per_row * B;
}

// A state's bytes and more: whole rows from their first byte to their last,
static Span whole_rows(const flce_beam_state_t& t, int64_t R) {
  return Span(t.data, R, (t.outer - 1) * t.outer_stride + t.inner, t.row_stride, 1);
}

// or lines of `inner` bytes one pitch apart, where both strides allow it.  States that
// are apart in either way are apart.
static Span lines(const flce_beam_state_t& t, int64_t R) {
  if (t.outer == 1) return Span(t.data, R, t.inner, t.row_stride, 1);
  if (R == 1) return Span(t.data, t.outer, t.inner, t.outer_stride, 1);
  if (t.row_stride % t.outer_stride == 0)
    return Span(t.data, (R - 1) * (t.row_stride / t.outer_stride) + t.outer, t.inner,
                t.outer_stride, 1);
  if (t.outer_stride % t.row_stride == 0)
    return Span(t.data, (t.outer - 1) * (t.outer_stride / t.row_stride) + R, t.inner,
                t.row_stride, 1);
  const int64_t end = (R - 1) * t.row_stride + (t.outer - 1) * t.outer_stride + t.inner;
  return Span(t.data, 1, end, end, 1);
}

static bool meet(const flce_beam_state_t& a, const flce_beam_state_t& b, int64_t R) {
  if (a.outer == 0 || a.inner == 0 || b.outer == 0 || b.inner == 0) return false;
  return overlap(whole_rows(a, R), whole_rows(b, R)) && overlap(lines(a, R), lines(b, R));
}
// Whether a state shares a byte with consecutive ones.  The runs of the shorter stride lie
// within a step of the longer one, and bytes as long as that step hold a run: the steps
// that begin near them are looked at, three at most before one is found or all are passed.
static bool meet(const flce_beam_state_t& t, const Span& bytes, int64_t R) {
  if (t.outer == 0 || t.inner == 0 || bytes.empty()) return false;
  const bool by_row = t.outer == 1 || (R > 1 && t.row_stride >= t.outer_stride);
  const int64_t steps = by_row ? R : t.outer, step = by_row ? t.row_stride : t.outer_stride;
  const int64_t runs = by_row ? t.outer : R, stride = by_row ? t.outer_stride : t.row_stride;
  const uintptr_t data = reinterpret_cast<uintptr_t>(t.data);
  int64_t i = steps > 1 && bytes.p > data ? static_cast<int64_t>(bytes.p - data) / step : 0;
  for (; i < steps && data + static_cast<uintptr_t>(i * step) < bytes.end(); ++i)
    if (overlap(Span(static_cast<char*>(t.data) + i * step, runs, t.inner, stride, 1), bytes))
      return true;
  return false;
}

}  // namespace flce

using namespace flce;

extern "C" size_t beam_select_workspace_bytes(int64_t B, int64_t K, int64_t V, int64_t num) {
  if (!beam_sizes(B, K, V, num) || B == 0) return 0;
  const size_t lists = static_cast<size_t>(B * K * beam_plan(B * K, V).chunks);
  return round_up(lists * (num * sizeof(uint64_t) + sizeof(float2)), 256);
}

extern "C" int beam_select(const void* logits, int dt, int64_t B, int64_t K, int64_t V, int64_t ld,
                           const float* scores, const uint8_t* finished, int64_t pad_id,
                           int64_t num, float* out_scores, int64_t* out_tokens,
                           int64_t* out_parents, void* ws, size_t ws_bytes,
                           flce_stream_t stream) {
  if (!valid_dtype(dt)) return FLCE_EDTYPE;
  if (!beam_sizes(B, K, V, num)) return FLCE_ESHAPE;
  if (finished != nullptr && (pad_id < 0 || pad_id >= V)) return FLCE_EINVAL;
  const int rc = check_matrix(logits, dt, B * K, V, ld);
  if (rc != FLCE_OK) return rc;
  if (B == 0) return FLCE_OK;
  if (scores == nullptr || out_scores == nullptr || out_tokens == nullptr ||
      out_parents == nullptr)
    return FLCE_EINVAL;
  if (!aligned(scores, 4) || !aligned(out_scores, 4) || !aligned(out_tokens, 8) ||
      !aligned(out_parents, 8) || !aligned(ws, 16))
    return FLCE_EALIGN;
  if (ws == nullptr || ws_bytes < beam_select_workspace_bytes(B, K, V, num))
    return FLCE_EWORKSPACE;
  const int64_t R = B * K, n = B * num;
  const Span in[3] = {Span(logits, R, V, ld, dtype_size(dt)), Span(scores, 1, R, R, 4),
                      Span(finished, 1, R, R, 1)};
  const Span out[4] = {Span(out_scores, 1, n, n, 4), Span(out_tokens, 1, n, n, 8),
                       Span(out_parents, 1, n, n, 8),
                       Span(ws, 1, static_cast<int64_t>(ws_bytes), 0, 1)};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 3; ++j)
      if (overlap(out[i], in[j])) return FLCE_EINVAL;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return FLCE_EINVAL;
  }
  BeamArgs a{};
  a.logits = logits, a.V = V, a.ld = ld, a.scores = scores, a.finished = finished;
  a.pad = pad_id, a.K = static_cast<int>(K), a.num = static_cast<int>(num);
  const BeamPlan plan = beam_plan(R, V);
  a.chunks = static_cast<int>(plan.chunks);
  a.tiles = plan.tiles;
  a.keys = static_cast<uint64_t*>(ws);
  a.sums = reinterpret_cast<float2*>(a.keys + R * a.chunks * num);
  a.out_scores = out_scores, a.out_tokens = out_tokens, a.out_parents = out_parents;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(a.chunks * R);
  const bool longer = plan.elems == kBeamLong;
  auto* rows = dt == FLCE_BF16 ? longer ? beam_rows_kernel<__nv_bfloat16, kBeamLong>
                                        : beam_rows_kernel<__nv_bfloat16, kBeamShort>
               : longer        ? beam_rows_kernel<float, kBeamLong>
                               : beam_rows_kernel<float, kBeamShort>;
  rows<<<grid, kBeamThreads, 0, s>>>(a);
  // a warp for each beam, where their keys fit shared memory together
  const int64_t list = static_cast<int64_t>(a.chunks) * num * 8, best = K * num * 12;
  constexpr int64_t kMost = 200 * 1024;  // at least 257 chunks of 64 and 4096 best: 176 KB
  const int warps = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>({kBeamMergeThreads / 32, K, (kMost - best) / list})));
  static std::atomic<uint64_t> raised{0};
  const int rc2 = raise_smem(beam_merge_kernel, kMost, raised);
  if (rc2 != FLCE_OK) return rc2;
  beam_merge_kernel<<<static_cast<unsigned>(B), 32 * warps, warps * list + best, s>>>(a);
  return launch_status("beam_merge_kernel launch");
}

extern "C" int beam_reorder(const flce_beam_state_t* states, int n, int64_t B, int64_t K,
                            const int64_t* parents, int32_t* status, flce_stream_t stream) {
  if (n < 0 || B < 0 || K < 1 || K > kBeamMost || B > 0x7fffffff / kBeamMost) return FLCE_ESHAPE;
  if (n > 0 && states == nullptr) return FLCE_EINVAL;
  if (n > 0 && B > 0 && parents == nullptr) return FLCE_EINVAL;
  if (!aligned(parents, 8) || !aligned(status, 4)) return FLCE_EALIGN;
  const int64_t R = B * K;
  constexpr int64_t kFar = int64_t(1) << 60;
  for (int i = 0; i < n; ++i) {
    const flce_beam_state_t& t = states[i];
    if (t.outer < 0 || t.inner < 0 || t.row_stride < 0 || t.outer_stride < 0) return FLCE_ESHAPE;
    if (t.outer == 0 || t.inner == 0 || R == 0) continue;
    if (t.inner > kFar / t.outer || t.outer_stride > kFar / t.outer || t.row_stride > kFar / R)
      return FLCE_ESHAPE;
    if (t.data == nullptr) return FLCE_EINVAL;
    // runs that do not meet: one row's within the row's stride, or all rows' within one
    // step of the outer stride
    const int64_t row = (t.outer - 1) * t.outer_stride + t.inner;
    const bool steps = t.outer == 1 || t.outer_stride >= t.inner;
    const bool rows = R == 1 || t.row_stride >= row ||
                      (t.row_stride >= t.inner &&
                       t.outer_stride >= (R - 1) * t.row_stride + t.inner);
    if (!steps || !rows) return FLCE_ESHAPE;
    if (reorder_blocks(t, B, reorder_unit(t, R)) > 0x7fffffff) return FLCE_ESHAPE;
  }
  if (R == 0) return FLCE_OK;
  // blocks read the parents, and report, while others already write
  const Span order(parents, 1, R, R, 8), word(status, 1, 1, 1, 4);
  if (overlap(order, word)) return FLCE_EINVAL;
  for (int i = 0; i < n; ++i) {
    if (meet(states[i], order, R) || meet(states[i], word, R)) return FLCE_EINVAL;
    for (int j = 0; j < i; ++j)
      if (meet(states[i], states[j], R)) return FLCE_EINVAL;
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // one launch for the states of each unit
  for (int unit = 16; unit > 0; unit /= 2) {
    ReorderArgs a{};
    a.K = static_cast<int>(K), a.B = B, a.parents = parents, a.status = status;
    int64_t blocks = 0;
    auto launch = [&]() {
      int rc = FLCE_OK;
      if (a.states > 0)
        rc = unit == 16  ? launch_reorder<uint4>(a, blocks, s)
             : unit == 8 ? launch_reorder<uint2>(a, blocks, s)
             : unit == 4 ? launch_reorder<uint32_t>(a, blocks, s)
             : unit == 2 ? launch_reorder<uint16_t>(a, blocks, s)
                         : launch_reorder<uint8_t>(a, blocks, s);
      a.states = 0;
      blocks = 0;
      return rc;
    };
    for (int i = 0; i < n; ++i) {
      const flce_beam_state_t& t = states[i];
      if (t.outer == 0 || t.inner == 0) continue;
      if (reorder_unit(t, R) != unit) continue;
      ReorderState& d = a.state[a.states];
      d.data = static_cast<char*>(t.data);
      d.row_stride = t.row_stride, d.outer_stride = t.outer_stride;
      d.inner = t.inner / unit;
      d.units = t.outer * d.inner;
      const int64_t need = reorder_blocks(t, B, unit);
      if (a.states > 0 && blocks + need > 0x7fffffff) {
        const ReorderState keep = d;
        const int rc = launch();
        if (rc != FLCE_OK) return rc;
        a.state[0] = keep;
      }
      a.state[a.states++].first = blocks;
      blocks += need;
      if (a.states == kReorderStates) {
        const int rc = launch();
        if (rc != FLCE_OK) return rc;
      }
    }
    const int rc = launch();
    if (rc != FLCE_OK) return rc;
  }
  return FLCE_OK;
}
