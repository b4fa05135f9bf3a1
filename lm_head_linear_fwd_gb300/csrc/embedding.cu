// Embedding lookup and the gradient of the table.
#include <algorithm>
#include <atomic>

#include "rows.cuh"

namespace flce {

// p[k] += x[k] at the memory, without waiting for the old values.  Each element
// of a gradient is added to once per call, so the result does not depend on the
// order of the adds.
template <int VEC>
__device__ __forceinline__ void add_to(float* p, const float (&x)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int k = 0; k < VEC; k += 4)
      asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p + k), "f"(x[k]),
                   "f"(x[k + 1]), "f"(x[k + 2]), "f"(x[k + 3])
                   : "memory");
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) atomicAdd(p + k, x[k]);
  }
}

// Elements per access that two row matrices allow: base addresses, row strides
// and, where the kernel has no tail, the columns (else D = 0) are multiples of it.
static int vec_width(int64_t D, const void* p, int dt, int64_t ld, const void* q, int dtq,
                     int64_t ldq) {
  const int most = dt == FLCE_BF16 ? 8 : 4;
  for (int v = most; v > 1; v = v == 8 ? 2 : 1) {
    // an access to q of v elements is split into 16-byte ones
    const size_t a = dtype_size(dt) * v, b = std::min<size_t>(dtype_size(dtq) * v, 16);
    if (D % v == 0 && aligned(p, a) && ld % v == 0 && aligned(q, b) && ldq % v == 0) return v;
  }
  return 1;
}

// ---------------------------------------------------------------------- lookup

constexpr int kLookupThreads = 128;
constexpr int kLookupLane = 32;  // elements of a row per lane and task

// One warp copies 32 * kLookupLane elements of one row at a time, all its loads
// in flight together.  Bound by memory: 65536 rows of 5120 bf16 take 130 us (6.3 TB/s
// with each table row counted once).
template <typename T, int VEC>
__global__ void __launch_bounds__(kLookupThreads)
    embedding_fwd_kernel(const int64_t* __restrict__ ids, const T* __restrict__ W, int64_t N,
                         int64_t D, int64_t V, int64_t ldw, float scale, T* __restrict__ out,
                         int64_t ldo, int64_t pieces, int32_t* status) {
  constexpr int U = kLookupLane / VEC;
  const int lane = threadIdx.x & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kLookupThreads / 32);
  const int64_t n = N * pieces;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kLookupThreads / 32) + (threadIdx.x >> 5);
       t < n; t += step) {
    const int64_t i = t / pieces;
    const int64_t j0 = (t - i * pieces) * (32 * kLookupLane) + lane * VEC;
    const int64_t v = ids[i];
    T* o = out + i * ldo;
    if (!label_ok(v, V)) {
      if (lane == 0) set_status(status, FLCE_ELABEL);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int64_t j = j0 + u * 32 * VEC + e;
          if (j < D) Elem<T>::store(o + j, 0.0f);
        }
      continue;
    }
    const T* w = W + v * ldw;
    if (j0 - lane * VEC + 32 * kLookupLane <= D) {
      Vec<T, VEC> r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) r[u].load(w + j0 + u * 32 * VEC);
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) r[u].x[e] *= scale;
        r[u].store(o + j0 + u * 32 * VEC);
      }
    } else {
      Vec<T, VEC> r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t j = j0 + u * 32 * VEC;
        if (j + VEC <= D) {
          r[u].load(w + j);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) r[u].x[e] = j + e < D ? Elem<T>::load(w + j + e) : 0.0f;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t j = j0 + u * 32 * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) r[u].x[e] *= scale;
        if (j + VEC <= D) {
          r[u].store(o + j);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (j + e < D) Elem<T>::store(o + j + e, r[u].x[e]);
        }
      }
    }
  }
}

template <typename T, int VEC>
static void launch_fwd(const int64_t* ids, const void* W, int64_t N, int64_t D, int64_t V,
                       int64_t ldw, float scale, void* out, int64_t ldo, int32_t* status,
                       cudaStream_t s) {
  const int64_t pieces = (D + 32 * kLookupLane - 1) / (32 * kLookupLane);
  constexpr int kWarps = kLookupThreads / 32;
  const int64_t need = (N * pieces + kWarps - 1) / kWarps;
  const int grid = static_cast<int>(std::min<int64_t>(need, int64_t(1) << 30));
  embedding_fwd_kernel<T, VEC><<<grid, kLookupThreads, 0, s>>>(
      ids, static_cast<const T*>(W), N, D, V, ldw, scale, static_cast<T*>(out), ldo, pieces,
      status);
}

// -------------------------------------------------------------------- gradient
//
// grad_W[v] (+)= scale * sum over the tokens i of id v of dy[i].
//
// 1. embedding_sort_kernel: one cluster of CTAs sorts the tokens by id (least
//    significant digit first, stable, so a row's tokens stay in token order and
//    the sums do not depend on timing).  Tokens that contribute nothing (the
//    padding id, ids out of range) get the key V and come last.  Meanwhile the
//    other CTAs write zeros to the rows that no token names: each finds them by
//    marking the ids that fall into its rows.
// 2. embedding_reduce_kernel: the sorted tokens are cut into chunks of equal
//    length, whatever the ids, so a frequent id costs no more than rare ones.
//    A CTA adds up a chunk's rows over a tile of columns and writes the rows
//    whose tokens all lie in its chunk.  A run of equal ids over several chunks
//    leaves one partial sum per chunk; the last CTA to arrive (an integer
//    ticket) adds the partial sums in chunk order and writes the row.
//
// Bound by the gradient's stores where it is written whole (8192 x 4096 tokens into
// 128256 rows of fp32: 336 us, 6.5 TB/s), else by the two steps in a row.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigitBits = 9;
constexpr int kFillRows = 1 << 16;  // rows marked at a time (one bit each)
constexpr int kMaxSortCtas = 8;
constexpr int kSortAhead = 4;       // tokens per lane loaded together

struct SortPlan {
  int passes, bits;  // digits of `bits` bits
};

static SortPlan sort_plan(int64_t V) {  // keys 0..V
  int total = 1;
  while (total < 32 && (V >> total) != 0) ++total;
  const int passes = (total + kMaxDigitBits - 1) / kMaxDigitBits;
  return {passes, (total + passes - 1) / passes};
}

static int sort_ctas(int64_t N) {
  int c = 1;
  while (c < kMaxSortCtas && N > int64_t(kSortThreads) * c) c *= 2;
  return c;
}

struct SortArgs {
  const int64_t* ids;
  int64_t N, V, padding_idx;
  uint2* buf0;     // (key, token) pairs, written by the passes in turn
  uint2* buf1;
  int passes, bits;
  int32_t* ticket;  // zeroed here for the reduction
  int64_t tickets;
  void* grad;       // null: nothing to fill
  int64_t D, ldw;
  int grad_es;
  int32_t* status;
};

// The key a token is sorted by: its id, or V (after every id) when it
// contributes nothing.
__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, int64_t id, bool* ok) {
  *ok = label_ok(id, a.V);
  return static_cast<uint32_t>(*ok && id != a.padding_idx ? id : a.V);
}

// Bitmap of the rows of [v0, v1) that some token names.
__device__ __forceinline__ void mark_row(uint32_t* mark, int64_t v0, int64_t v1, uint32_t key) {
  if (key >= v0 && key < v1) atomicOr(&mark[(key - v0) >> 5], 1u << ((key - v0) & 31));
}

__device__ void mark_rows(const SortArgs& a, int64_t v0, int64_t v1, uint32_t* mark) {
  for (int k = threadIdx.x; k < (v1 - v0 + 31) / 32; k += kSortThreads) mark[k] = 0;
  __syncthreads();
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < a.N; i += kSortThreads) {
    bool ok;
    mark_row(mark, v0, v1, sort_key(a, a.ids[i], &ok));
  }
  __syncthreads();
}

// Zeros for the rows of [v0, v1) that are not marked.  A warp takes the next
// rows from *next (shared, 0 at the start), so warps may join at any time.
__device__ void zero_rows(const SortArgs& a, int64_t v0, int64_t v1, const uint32_t* mark,
                          int* next) {
  const int lane = threadIdx.x & 31;
  const int n = static_cast<int>(v1 - v0);
  const int64_t row_bytes = a.D * a.grad_es;
  const int64_t ld_bytes = a.ldw * a.grad_es;
  char* g = static_cast<char*>(a.grad) + v0 * ld_bytes;
  // at least 4 KB at a time
  const int take = static_cast<int>(max(int64_t(1), min(int64_t(64), 4096 / row_bytes)));
  while (true) {
    int r0 = 0;
    if (lane == 0) r0 = atomicAdd(next, take);
    r0 = __shfl_sync(0xffffffffu, r0, 0);
    if (r0 >= n) return;
    const int r1 = min(n, r0 + take);
    for (int r = r0; r < r1; ++r) {
      if ((mark[r >> 5] >> (r & 31)) & 1u) continue;
      // whole 16-byte blocks, and the elements before and after them
      char* p = g + r * ld_bytes;
      const int64_t head = min(
          row_bytes, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15));
      char* end = p + row_bytes;
      char* first = p + head;
      char* last = first + (row_bytes - head) / 16 * 16;
      for (char* q = first + 16 * lane; q < last; q += 512)
        __stcs(reinterpret_cast<uint4*>(q), make_uint4(0, 0, 0, 0));
      const int edge = lane < 8 ? lane : lane - 8;
      char* q = (lane < 8 ? p : last) + edge * a.grad_es;
      if (lane < 16 && q < (lane < 8 ? first : end)) {
        if (a.grad_es == 4)
          *reinterpret_cast<uint32_t*>(q) = 0u;
        else
          *reinterpret_cast<uint16_t*>(q) = 0;
      }
    }
  }
}

__global__ void __launch_bounds__(kSortThreads) embedding_sort_kernel(SortArgs a) {
  extern __shared__ uint32_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int next_row;
  const int C = static_cast<int>(cluster_nctarank());
  const int rank = static_cast<int>(cluster_ctarank());
  if (blockIdx.x >= static_cast<unsigned>(C)) {
    // rows of this CTA, a bitmap's worth at a time
    const int64_t parts = static_cast<int64_t>(gridDim.x) - C;
    const int64_t me = static_cast<int64_t>(blockIdx.x) - C;
    const int64_t per = (a.V + parts - 1) / parts;
    const int64_t end = min(a.V, (me + 1) * per);
    for (int64_t v = me * per; v < end; v += kFillRows) {
      if (tid == 0) next_row = 0;
      mark_rows(a, v, min(end, v + kFillRows), smem);
      zero_rows(a, v, min(end, v + kFillRows), smem, &next_row);
      __syncthreads();
    }
    return;
  }
  // the other CTAs' shared memory may be written once all of them have started
  cluster_sync();
  for (int64_t k = rank * kSortThreads + tid; k < a.tickets; k += C * kSortThreads)
    a.ticket[k] = 0;
  const int R = 1 << a.bits;
  const int S = R + 1;                       // a digit's counts of all warps in 32 banks
  uint32_t* count = smem;                    // [kSortWarps][S]
  uint32_t* total = smem + kSortWarps * S;   // [kMaxSortCtas][R], written by every CTA
  uint32_t* start = total + kMaxSortCtas * R;  // [R]
  __shared__ uint32_t warp_sum[kSortWarps];
  // this warp's share of the tokens, a multiple of 32 except at the end
  const int64_t share = ((a.N + C * kSortWarps - 1) / (C * kSortWarps) + 31) / 32 * 32;
  const int64_t i0 = min(a.N, (static_cast<int64_t>(rank) * kSortWarps + warp) * share);
  const int64_t i1 = min(a.N, i0 + share);
  for (int pass = 0; pass < a.passes; ++pass) {
    const uint2* src = (pass & 1) ? a.buf0 : a.buf1;
    uint2* dst = (pass & 1) ? a.buf1 : a.buf0;
    const int shift = pass * a.bits;
    auto fetch = [&](int64_t i) -> uint2 {
      if (pass > 0) return __ldcg(src + i);
      bool ok;
      const uint32_t key = sort_key(a, a.ids[i], &ok);
      if (!ok) set_status(a.status, FLCE_ELABEL);
      return make_uint2(key, static_cast<uint32_t>(i));
    };
    for (int k = tid; k < kSortWarps * S; k += kSortThreads) count[k] = 0;
    __syncthreads();
    uint32_t* mine = count + warp * S;
    // kSortAhead loads in flight per lane, here and where the tokens are placed
    for (int64_t i = i0 + lane; i < i1; i += 32 * kSortAhead) {
      uint2 e[kSortAhead];
#pragma unroll
      for (int k = 0; k < kSortAhead; ++k)
        if (i + 32 * k < i1) e[k] = fetch(i + 32 * k);
#pragma unroll
      for (int k = 0; k < kSortAhead; ++k)
        if (i + 32 * k < i1) atomicAdd(&mine[(e[k].x >> shift) & (R - 1)], 1u);
    }
    __syncthreads();
    // per digit: exclusive sums over this CTA's warps, and the CTA's total,
    // handed to every CTA of the cluster
    for (int d = warp; d < R; d += kSortWarps) {
      const uint32_t c = count[lane * S + d];
      uint32_t s = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
      }
      count[lane * S + d] = s - c;
      const uint32_t sum = __shfl_sync(0xffffffffu, s, 31);
      if (lane < C) {
        const uint32_t at = mapa_shared(smem_u32(total + rank * R + d), lane);
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(sum) : "memory");
      }
    }
    cluster_sync();
    // first place of each digit: all smaller digits, then the CTAs before this
    // one (R <= kSortThreads: one digit per thread)
    uint32_t all = 0, before = 0;
    if (tid < R) {
      for (int c = 0; c < C; ++c) {
        const uint32_t t = total[c * R + tid];
        if (c < rank) before += t;
        all += t;
      }
    }
    uint32_t s = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += t;
    }
    if (lane == 31) warp_sum[warp] = s;
    __syncthreads();
    uint32_t base = 0;
    for (int w = 0; w < warp; ++w) base += warp_sum[w];
    if (tid < R) start[tid] = base + s - all + before;
    __syncthreads();
    // each warp places its tokens in order; lanes of one digit by lane
    for (int64_t i = i0 + lane; i - lane < i1; i += 32 * kSortAhead) {
      uint2 e[kSortAhead];
#pragma unroll
      for (int k = 0; k < kSortAhead; ++k)
        e[k] = i + 32 * k < i1 ? fetch(i + 32 * k) : make_uint2(0, 0);
#pragma unroll
      for (int k = 0; k < kSortAhead; ++k) {
        const bool in = i + 32 * k < i1;
        const uint32_t digit = in ? (e[k].x >> shift) & (R - 1) : R;
        const uint32_t same = __match_any_sync(0xffffffffu, digit);
        const int before_me = __popc(same & ((1u << lane) - 1u));
        if (in) {
          const uint32_t at = start[digit] + mine[digit] + before_me;
          if (in_range(at, a.N, a.status)) __stcg(dst + at, e[k]);
        }
        __syncwarp();
        if (in && before_me == 0) mine[digit] += __popc(same);
        __syncwarp();
      }
    }
    cluster_sync();
  }
}

// The sort of up to kRankShare tokens per SM: every CTA finds the places of its
// share of the tokens by itself.  It orders its share, then runs over all ids
// and looks up by bisection how many of its tokens come after each; the running
// sum of these counts is the number of tokens before each of its own.  Indices
// outside the share lie all before or all after it, so keys alone decide.
// No passes, and no CTA waits for another.  Where rows are to be filled, half of
// the warps start on that at once and the others join them.
// Bound by the look-ups' instructions on every SM: 8192 tokens take 8 us.  The work
// grows with N times the bisection's steps, the cluster's sort with N alone but it
// starts higher: gradients (added) of 8192 x 4096 with this 43.8 us, with the sort
// 56.2; of 16384 x 1024 33.6 and 37.9; of 32768 x 1024 56.7 and 52.8.
constexpr int kRankShare = 128;
constexpr int kRankAhead = 4;  // ids a thread looks up together

__global__ void __launch_bounds__(kSortThreads) embedding_rank_kernel(SortArgs a) {
  __shared__ uint64_t own[kRankShare];
  __shared__ uint32_t ordered[2 * kRankShare], token[kRankShare];  // own keys in order
  __shared__ uint32_t before[kRankShare + 1];
  __shared__ uint32_t mark[kFillRows / 32];
  __shared__ int next_row;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int64_t k = blockIdx.x * int64_t(kSortThreads) + tid; k < a.tickets;
       k += gridDim.x * int64_t(kSortThreads))
    a.ticket[k] = 0;
  const int64_t rows = (a.V + gridDim.x - 1) / gridDim.x;
  const int64_t v0 = min(a.V, blockIdx.x * rows), v_end = min(a.V, v0 + rows);
  const int64_t v1 = min(v_end, v0 + kFillRows);
  const bool fill = a.grad != nullptr;
  int team = kSortThreads;  // threads that sort
  if (fill) {
    if (tid == 0) next_row = 0;
    mark_rows(a, v0, v1, mark);
    team = kSortThreads / 2;
  }
  if (tid < team) {
    const int64_t share = (a.N + gridDim.x - 1) / gridDim.x;
    const int64_t t0 = blockIdx.x * share;
    const int m = static_cast<int>(max(int64_t(0), min(share, a.N - t0)));
    if (tid <= kRankShare) before[tid] = 0;
    // a token as one number: by key, then by index
    if (tid < m) {
      bool ok;
      const uint32_t key = sort_key(a, a.ids[t0 + tid], &ok);
      if (!ok) set_status(a.status, FLCE_ELABEL);
      own[tid] = static_cast<uint64_t>(key) << 32 | static_cast<uint64_t>(t0 + tid);
    }
    if (tid >= m && tid < 2 * kRankShare) ordered[tid] = 0xffffffffu;  // above every key
    named_barrier(1, team);
    // the order of the own tokens, a warp to a token
    for (int i = warp; i < m; i += team / 32) {
      const uint64_t e = own[i];
      int r = 0;
      for (int j = lane; j < m; j += 32) r += own[j] < e;
      r = __reduce_add_sync(0xffffffffu, r);
      if (lane == 0) {
        ordered[r] = static_cast<uint32_t>(e >> 32);
        token[r] = static_cast<uint32_t>(e);
      }
    }
    named_barrier(1, team);
    if (m > 0) {
      int top = 1;
      while (2 * top <= m) top *= 2;
      for (int64_t i0 = tid; i0 < a.N; i0 += kRankAhead * team) {
        uint32_t bound[kRankAhead];
        int lo[kRankAhead];
#pragma unroll
        for (int k = 0; k < kRankAhead; ++k) {
          // own tokens before token i: those of smaller keys, and the equal ones where
          // all own tokens come first (past the end: i = N - 1 again, not counted)
          const int64_t i = min(i0 + k * team, a.N - 1);
          bool ok;
          bound[k] = sort_key(a, a.ids[i], &ok) + (i > t0 ? 1u : 0u);
          lo[k] = 0;
        }
        for (int step = top; step > 0; step >>= 1)
#pragma unroll
          for (int k = 0; k < kRankAhead; ++k)
            if (ordered[lo[k] + step - 1] < bound[k]) lo[k] += step;
#pragma unroll
        for (int k = 0; k < kRankAhead; ++k) {
          const int64_t i = i0 + k * team;
          if (i < a.N && (i < t0 || i >= t0 + m) && lo[k] < m) atomicAdd(&before[lo[k]], 1u);
        }
      }
    }
    named_barrier(1, team);
    // a warp to 32 own tokens: the counts up to each, and it itself
    if (warp * 32 < m) {
      uint32_t s = before[tid];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
      }
      for (int w = 0; w < warp; ++w) s += __reduce_add_sync(0xffffffffu, before[w * 32 + lane]);
      s += static_cast<uint32_t>(tid);
      if (tid < m && in_range(s, a.N, a.status)) a.buf0[s] = make_uint2(ordered[tid], token[tid]);
    }
  }
  if (!fill) return;
  zero_rows(a, v0, v1, mark, &next_row);
  for (int64_t v = v1; v < v_end; v += kFillRows) {
    __syncthreads();
    if (tid == 0) next_row = 0;
    mark_rows(a, v, min(v_end, v + kFillRows), mark);
    zero_rows(a, v, min(v_end, v + kFillRows), mark, &next_row);
  }
}

constexpr int kReduceLane = 8;  // columns per thread
constexpr int kMinChunk = 16, kMaxChunk = 128;
constexpr int kReduceAhead = 8;  // token rows loaded together

struct ReducePlan {
  int chunk;        // tokens per chunk, a multiple of kReduceAhead
  int64_t chunks, tiles;
};

// Threads of a block: one warp for rows it can hold alone.
static int reduce_threads(int64_t D) { return D <= 32 * kReduceLane ? 32 : 128; }

// One wave of blocks (24 warps to an SM) while a chunk stays within kMaxChunk
// tokens, and no chunk shorter than sqrt(N / 8) tokens while that is within
// kMaxChunk too: up to 131072 tokens a run over an eighth of them is joined from no
// more partial sums than a chunk has tokens, beyond that from N / 1024.
static ReducePlan reduce_plan(int64_t N, int64_t D) {
  const int64_t tile = reduce_threads(D) * kReduceLane;
  const int64_t tiles = (D + tile - 1) / tile;
  const int64_t wave = int64_t(sm_count()) * 24 * 32 / reduce_threads(D);
  int64_t chunk = std::max<int64_t>(kMinChunk, (N * tiles + wave - 1) / wave);
  while (chunk < kMaxChunk && chunk * chunk < N / 8) ++chunk;
  chunk = std::min<int64_t>(kMaxChunk, (chunk + kReduceAhead - 1) / kReduceAhead * kReduceAhead);
  return {static_cast<int>(chunk), (N + chunk - 1) / chunk, tiles};
}

struct ReduceArgs {
  const uint2* sorted;
  const void* dy;
  int64_t N, D, V, ldg;
  float scale;
  void* grad;
  int64_t ldw;
  int accumulate;
  int chunk;
  int64_t chunks, tiles;
  float* part;      // [chunks][2][tiles][threads of a block][kReduceLane]
  int32_t* ticket;  // [chunks][tiles]
};

// First chunk of the run of id v that chunk c begins inside (the one whose
// predecessor ends in another id), by one warp.  `word` is the lane's first
// candidate, the id that ends chunk c - 2 - lane.
__device__ __forceinline__ int64_t run_first_chunk(const ReduceArgs& a, int64_t c, uint32_t v,
                                                   uint32_t word) {
  for (int64_t b = c - 1;; b -= 32) {
    const int64_t q = b - (threadIdx.x & 31);
    if (b != c - 1 && q > 0) word = a.sorted[q * a.chunk - 1].x;
    const uint32_t m = __ballot_sync(0xffffffffu, q <= 0 || word != v);
    if (m) return b - (__ffs(m) - 1);
  }
}

// Last chunk of the run of id v that chunk c ends in or holds; `word` is the id
// that begins chunk c + 1 + lane.
__device__ __forceinline__ int64_t run_last_chunk(const ReduceArgs& a, int64_t c, uint32_t v,
                                                  uint32_t word) {
  for (int64_t b = c;; b += 32) {
    const int64_t at = (b + (threadIdx.x & 31) + 1) * a.chunk;
    if (b != c && at < a.N) word = a.sorted[at].x;
    const uint32_t m = __ballot_sync(0xffffffffu, at >= a.N || word != v);
    if (m) return b + __ffs(m) - 1;
  }
}

template <typename T, typename G, int VEC, int kThreads>
__global__ void __launch_bounds__(kThreads, VEC == 8 ? 24 * 32 / kThreads : 1)
    embedding_reduce_kernel(ReduceArgs a) {
  constexpr int U = kReduceLane / VEC;
  constexpr int kTile = kThreads * kReduceLane;
  __shared__ uint2 tok[kMaxChunk];
  __shared__ int64_t run_first[2], run_last[2];
  __shared__ int last[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* dy = static_cast<const T*>(a.dy);
  const uint32_t V = static_cast<uint32_t>(a.V);
  const int64_t items = a.chunks * a.tiles;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t c = item / a.tiles, tile = item - c * a.tiles;
    const int64_t col0 = tile * kTile + tid * VEC;
    const int64_t t0 = c * a.chunk;
    const int n = static_cast<int>(min(static_cast<int64_t>(a.chunk), a.N - t0));
    __syncthreads();  // tok and the run's words are free again
    for (int k = tid; k < n; k += kThreads) tok[k] = a.sorted[t0 + k];
    const uint32_t none = 0xffffffffu;
    const uint32_t before = t0 > 0 ? a.sorted[t0 - 1].x : none;
    const uint32_t after = t0 + n < a.N ? a.sorted[t0 + n].x : none;
    // the ends of the chunks next to this one, for runs that leave it
    const int64_t prev_at = (c - 1 - lane) * a.chunk - 1, next_at = (c + 1 + lane) * a.chunk;
    const uint32_t prev_word = prev_at >= 0 ? a.sorted[prev_at].x : none;
    const uint32_t next_word = next_at < a.N ? a.sorted[next_at].x : none;
    __syncthreads();

    auto out_row = [&](uint32_t v, const float (&acc)[U][VEC]) {
      G* g = static_cast<G*>(a.grad) + static_cast<int64_t>(v) * a.ldw;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t j = col0 + u * kThreads * VEC;
        if (j >= a.D) break;  // D is a multiple of VEC
        float r[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) r[e] = acc[u][e] * a.scale;
        if (a.accumulate)
          add_to<VEC>(reinterpret_cast<float*>(g + j), r);
        else
          store_as<G, VEC>(g + j, r);
      }
    };
    // this thread's eight columns of a chunk's partial sum, next to each other
    auto part_of = [&](int64_t chunk, int slot) {
      return reinterpret_cast<float4*>(
          a.part + (((chunk * 2 + slot) * a.tiles + tile) * kThreads + tid) * kReduceLane);
    };

    float acc[U][VEC] = {};
    uint32_t key = tok[0].x;
    bool first = true;  // in the run that the chunk begins with
    int slots = 0;      // bit 0: partial of a run from before, bit 1: of one that goes on
    auto flush = [&](bool goes_on) {
      if (key == V) return;
      const bool from_before = first && key == before;
      if (!from_before && !goes_on) {
        out_row(key, acc);
      } else {
        const int slot = from_before ? 0 : 1;
        const float* f = &acc[0][0];
        float4* p = part_of(c, slot);
        __stcg(p, make_float4(f[0], f[1], f[2], f[3]));
        __stcg(p + 1, make_float4(f[4], f[5], f[6], f[7]));
        slots |= 1 << slot;
      }
    };
    for (int k0 = 0; k0 < n; k0 += kReduceAhead) {
      // loads without conditions: past the chunk's end its last token again, past
      // the last column the last ones again (neither is used), and the rows of
      // tokens that contribute nothing (their run, the key V, is never written)
      RawVec<T, VEC> r[kReduceAhead][U];
#pragma unroll
      for (int k = 0; k < kReduceAhead; ++k) {
        const T* row = dy + static_cast<int64_t>(tok[min(k0 + k, n - 1)].y) * a.ldg;
#pragma unroll
        for (int u = 0; u < U; ++u) r[k][u].load(row + min(col0 + u * kThreads * VEC, a.D - VEC));
      }
#pragma unroll
      for (int k = 0; k < kReduceAhead; ++k) {
        if (k0 + k < n) {
          const uint32_t next = tok[k0 + k].x;
          if (next != key) {
            flush(false);
            first = false;
            key = next;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int e = 0; e < VEC; ++e) acc[u][e] = 0.0f;
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float x[VEC];
            r[k][u].unpack(x);
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[u][e] += x[e];
          }
        }
      }
    }
    flush(key == after);

    // runs over several chunks: the last CTA to arrive adds the partial sums
    if (slots == 0) continue;  // the same for all threads
    __threadfence();
    __syncthreads();
    // one warp for each of the two runs, or one for both
#pragma unroll
    for (int slot = 0; slot < 2; ++slot) {
      if (warp != (kThreads > 32 ? slot : 0) || !(slots >> slot & 1)) continue;
      const uint32_t v = slot == 0 ? before : key;
      const int64_t lo = slot == 0 ? run_first_chunk(a, c, v, prev_word) : c;
      const int64_t hi = run_last_chunk(a, c, v, next_word);
      if (lane == 0) {
        run_first[slot] = lo;
        run_last[slot] = hi;
        last[slot] = atomicAdd(a.ticket + lo * a.tiles + tile, 1) == static_cast<int>(hi - lo);
      }
    }
    __syncthreads();
#pragma unroll
    for (int slot = 0; slot < 2; ++slot) {
      if (!(slots >> slot & 1) || !last[slot]) continue;
      __threadfence();
      float sum[U][VEC] = {};
      float* f = &sum[0][0];
      constexpr int kAhead = 8;
      for (int64_t q0 = run_first[slot]; q0 <= run_last[slot]; q0 += kAhead) {
        float4 lo4[kAhead], hi4[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int64_t q = q0 + k;
          lo4[k] = hi4[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (q <= run_last[slot]) {
            const float4* p = part_of(q, q == run_first[slot] ? 1 : 0);
            lo4[k] = __ldcg(p);
            hi4[k] = __ldcg(p + 1);
          }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          f[0] += lo4[k].x, f[1] += lo4[k].y, f[2] += lo4[k].z, f[3] += lo4[k].w;
          f[4] += hi4[k].x, f[5] += hi4[k].y, f[6] += hi4[k].z, f[7] += hi4[k].w;
        }
      }
      out_row(slot == 0 ? before : key, sum);
    }
  }
}

template <typename T, typename G, int VEC, int kThreads>
static int launch_reduce_k(const ReduceArgs& a, cudaStream_t s) {
  const unsigned grid =
      static_cast<unsigned>(std::min<int64_t>(a.chunks * a.tiles, int64_t(1) << 30));
  embedding_reduce_kernel<T, G, VEC, kThreads><<<grid, kThreads, 0, s>>>(a);
  return launch_status("embedding_reduce_kernel launch");
}

template <typename T, typename G>
static int launch_reduce(const ReduceArgs& a, int vec, cudaStream_t s) {
  constexpr int V16 = Elem<T>::kPerVec, V4 = sizeof(T) == 2 ? 2 : 1;
  const bool narrow = reduce_threads(a.D) == 32;
  if (vec == V16)
    return narrow ? launch_reduce_k<T, G, V16, 32>(a, s) : launch_reduce_k<T, G, V16, 128>(a, s);
  if (vec == 2)
    return narrow ? launch_reduce_k<T, G, V4, 32>(a, s) : launch_reduce_k<T, G, V4, 128>(a, s);
  return narrow ? launch_reduce_k<T, G, 1, 32>(a, s) : launch_reduce_k<T, G, 1, 128>(a, s);
}

static size_t sort_smem(int bits) {
  const size_t R = size_t(1) << bits;
  const size_t sort = sizeof(uint32_t) * ((R + 1) * kSortWarps + R * (kMaxSortCtas + 1));
  return std::max<size_t>(sort, kFillRows / 8);
}

// Clusters of the sort's launch that run at once on the current device.
static int sort_clusters(cudaLaunchConfig_t cfg, int* clusters) {
  static std::atomic<int> cache[64][4][kMaxDigitBits + 1];
  int dev = 0;
  int rc = cuda_status(cudaGetDevice(&dev), "cudaGetDevice");
  if (rc != FLCE_OK) return rc;
  int c = 0, bits = 1;
  while ((2 << c) <= static_cast<int>(cfg.attrs[0].val.clusterDim.x)) ++c;
  while (bits < kMaxDigitBits && sort_smem(bits) < cfg.dynamicSmemBytes) ++bits;
  std::atomic<int>& known = cache[dev & 63][c][bits];
  if (known.load() == 0) {
    rc = cuda_status(cudaFuncSetAttribute(embedding_sort_kernel,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(sort_smem(kMaxDigitBits))),
                     "cudaFuncSetAttribute(embedding_sort_kernel)");
    if (rc != FLCE_OK) return rc;
    int n = 0;
    rc = cuda_status(cudaOccupancyMaxActiveClusters(&n, embedding_sort_kernel, &cfg),
                     "cudaOccupancyMaxActiveClusters(embedding_sort_kernel)");
    if (rc != FLCE_OK) return rc;
    known.store(std::max(n, 2));
  }
  *clusters = known.load();
  return FLCE_OK;
}

static int launch_sort(const SortArgs& a, cudaStream_t s) {
  const int C = sort_ctas(a.N);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(C);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(C), 1, 1);
  cfg.blockDim = dim3(kSortThreads, 1, 1);
  cfg.dynamicSmemBytes = sort_smem(a.bits);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 1;
  const int rc = sort_clusters(cfg, &clusters);
  if (rc != FLCE_OK) return rc;
  if (a.grad != nullptr) cfg.gridDim.x = static_cast<unsigned>(C * clusters);
  return cuda_status(cudaLaunchKernelEx(&cfg, embedding_sort_kernel, a),
                     "cudaLaunchKernelEx(embedding_sort_kernel)");
}

struct BwdWorkspace {
  size_t buf, ticket, part, total;
};

static BwdWorkspace bwd_workspace(int64_t N, int64_t D) {
  const ReducePlan r = reduce_plan(N, D);
  BwdWorkspace w;
  w.buf = round_up(static_cast<size_t>(N) * sizeof(uint2), 256);
  w.ticket = round_up(static_cast<size_t>(r.chunks * r.tiles) * sizeof(int32_t), 256);
  w.part = static_cast<size_t>(r.chunks * r.tiles) * 2 * reduce_threads(D) * kReduceLane *
           sizeof(float);
  w.total = 2 * w.buf + w.ticket + w.part;
  return w;
}

}  // namespace flce

using namespace flce;

extern "C" int embedding_fwd(const int64_t* ids, const void* W, int dt, int64_t N, int64_t D,
                             int64_t V, int64_t ldw, float scale, void* out, int64_t ldo,
                             int32_t* status, flce_stream_t stream) {
  if (!valid_dtype(dt)) return FLCE_EDTYPE;
  if (N < 0 || D < 1 || V < 1 || V >= (int64_t(1) << 31)) return FLCE_ESHAPE;
  if (status == nullptr || W == nullptr || (N > 0 && ids == nullptr)) return FLCE_EINVAL;
  int rc = check_matrix(W, dt, V, D, ldw);
  if (rc == FLCE_OK) rc = check_matrix(out, dt, N, D, ldo);
  if (rc != FLCE_OK) return rc;
  if (!aligned(ids, 8) || !aligned(status, 4)) return FLCE_EALIGN;
  const size_t es = dtype_size(dt);
  if (overlap(Span(W, V, D, ldw, es), Span(out, N, D, ldo, es))) return FLCE_EINVAL;
  if (N == 0) return FLCE_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int vec = vec_width(0, W, dt, ldw, out, dt, ldo);
#define FLCE_FWD(T, VEC) launch_fwd<T, VEC>(ids, W, N, D, V, ldw, scale, out, ldo, status, s)
  if (dt == FLCE_BF16) {
    if (vec == 8) FLCE_FWD(__nv_bfloat16, 8);
    else if (vec == 2) FLCE_FWD(__nv_bfloat16, 2);
    else FLCE_FWD(__nv_bfloat16, 1);
  } else {
    if (vec == 4) FLCE_FWD(float, 4);
    else FLCE_FWD(float, 1);
  }
#undef FLCE_FWD
  return launch_status("embedding_fwd_kernel launch");
}

extern "C" size_t embedding_bwd_workspace_bytes(int64_t N, int64_t D, int64_t V) {
  if (N < 1 || N >= (int64_t(1) << 31) || D < 1 || V < 1) return 0;
  return bwd_workspace(N, D).total;
}

extern "C" int embedding_bwd(const int64_t* ids, const void* grad_out, int dt, int64_t N,
                             int64_t D, int64_t V, int64_t ldg, float scale, int64_t padding_idx,
                             void* grad_W, int dt_grad, int64_t ldw, int accumulate_grad_W,
                             void* ws, size_t ws_bytes, int32_t* status, flce_stream_t stream) {
  if (!valid_dtype(dt) || !valid_dtype(dt_grad)) return FLCE_EDTYPE;
  if (accumulate_grad_W != 0 && accumulate_grad_W != 1) return FLCE_EINVAL;
  if (N < 0 || N >= (int64_t(1) << 31) || D < 1 || V < 1 || V >= (int64_t(1) << 31))
    return FLCE_ESHAPE;
  if (accumulate_grad_W && dt_grad != FLCE_F32) return FLCE_ENOSUP;
  if (status == nullptr || grad_W == nullptr || (N > 0 && ids == nullptr)) return FLCE_EINVAL;
  int rc = check_matrix(grad_out, dt, N, D, ldg);
  if (rc == FLCE_OK) rc = check_matrix(grad_W, dt_grad, V, D, ldw);
  if (rc != FLCE_OK) return rc;
  if (!aligned(ids, 8) || !aligned(status, 4)) return FLCE_EALIGN;
  if (overlap(Span(grad_out, N, D, ldg, dtype_size(dt)),
              Span(grad_W, V, D, ldw, dtype_size(dt_grad))))
    return FLCE_EINVAL;
  const size_t need = embedding_bwd_workspace_bytes(N, D, V);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return FLCE_EWORKSPACE;
  if (!aligned(ws, 16)) return FLCE_EALIGN;
  if (N == 0 && accumulate_grad_W) return FLCE_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

  const BwdWorkspace w = bwd_workspace(N, D);
  const ReducePlan plan = reduce_plan(N, D);
  const SortPlan sp = sort_plan(V);
  char* base = static_cast<char*>(ws);
  SortArgs sa{};
  sa.ids = ids;
  sa.N = N;
  sa.V = V;
  sa.padding_idx = padding_idx;
  sa.buf0 = reinterpret_cast<uint2*>(base);
  sa.buf1 = reinterpret_cast<uint2*>(base + w.buf);
  sa.passes = sp.passes;
  sa.bits = sp.bits;
  sa.ticket = reinterpret_cast<int32_t*>(base + 2 * w.buf);
  sa.tickets = plan.chunks * plan.tiles;
  sa.grad = accumulate_grad_W ? nullptr : grad_W;
  sa.D = D;
  sa.ldw = ldw;
  sa.grad_es = static_cast<int>(dtype_size(dt_grad));
  sa.status = status;
  const bool rank = N <= int64_t(kRankShare) * sm_count();
  if (rank) {
    embedding_rank_kernel<<<sm_count(), kSortThreads, 0, s>>>(sa);
    rc = launch_status("embedding_rank_kernel launch");
  } else {
    rc = launch_sort(sa, s);
  }
  if (rc != FLCE_OK || N == 0) return rc;

  ReduceArgs ra{};
  ra.sorted = rank || (sp.passes & 1) ? sa.buf0 : sa.buf1;
  ra.dy = grad_out;
  ra.N = N;
  ra.D = D;
  ra.V = V;
  ra.ldg = ldg;
  ra.scale = scale;
  ra.grad = grad_W;
  ra.ldw = ldw;
  ra.accumulate = accumulate_grad_W;
  ra.chunk = plan.chunk;
  ra.chunks = plan.chunks;
  ra.tiles = plan.tiles;
  ra.ticket = sa.ticket;
  ra.part = reinterpret_cast<float*>(base + 2 * w.buf + w.ticket);
  const int vec = vec_width(D, grad_out, dt, ldg, grad_W, dt_grad, ldw);
  using B = __nv_bfloat16;
  if (dt == FLCE_BF16)
    return dt_grad == FLCE_BF16 ? launch_reduce<B, B>(ra, vec, s) : launch_reduce<B, float>(ra, vec, s);
  return dt_grad == FLCE_BF16 ? launch_reduce<float, B>(ra, vec, s)
                              : launch_reduce<float, float>(ra, vec, s);
}
