// Tokens sorted by expert and back: the stable order of the (token, rank)
// pairs, the rows gathered into it, the rows combined with their weights, and
// the gradients of both.
//
//   gather            xs[position[t][r]] = x[t]
//   its gradient      gx[t] = sum_r gxs[position[t][r]]
//   combine           y[t] = sum_r w[t][r] ys[position[t][r]]
//   its gradient      gys[position[t][r]] = w[t][r] gy[t],  gw[t][r] = <gy[t], ys[position[t][r]]>
//
// All sums are fp32 in rank order: no atomics on values, so the results do not
// depend on the order in which blocks run. Rows of dropped pairs (position -1)
// are left out; places behind the kept pairs become zero rows.
#include "host.hpp"
#include "mxfp4.cuh"
#include "sort.cuh"

namespace si {

// ---------------------------------------------------------------------------
// Sort: one block per expert (and one for the dropped pairs), one launch.
// Every block counts all ids into shared memory, so it knows where its expert
// starts without waiting for another block, and keeps one bit per id for its
// own matches; a scan over the words of 32 ids then gives every match its
// place. More ids than kSortChunk go through the bits in chunks, read again.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortWords = 2048;                    // bit words in shared memory
constexpr int64_t kSortChunk = kSortWords * 32;     // ids they hold

// The ids of one chunk: match bits of expert `me`, and all ids counted if COUNT.
template <bool COUNT>
SI_DEV void sort_scan(const SortArgs &a, int64_t c0, int me, int *s_hist, uint32_t *s_bits) {
  constexpr int U = 8;                              // loads in flight per thread
  const int E = a.n_experts, lane = threadIdx.x & 31;
  const int64_t c1 = c0 + kSortChunk < a.pairs ? c0 + kSortChunk : a.pairs;
  for (int64_t b = c0 + (threadIdx.x & ~31) * U; b < c1; b += kSortThreads * U) {
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = b + u * 32 + lane;
      id[u] = i < c1 ? __ldcg(a.ids + i) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = b + u * 32 + lane;
      const int e = id[u] >= 0 && id[u] < E ? id[u] : E;
      if (COUNT && i < c1) atomicAdd(&s_hist[e], 1);
      const uint32_t m = __ballot_sync(0xffffffffu, i < c1 && e == me);
      if (lane == 0 && b + u * 32 < c1) s_bits[(b - c0) / 32 + u] = m;
    }
  }
}

__global__ void __launch_bounds__(kSortThreads) sort_pairs_kernel(SortArgs a) {
  __shared__ int s_hist[kSortMaxExperts + 1];
  __shared__ uint32_t s_bits[kSortWords];
  __shared__ int s_red[2][kSortWarps];
  grid_dep_wait();
  grid_dep_launch();
  const int E = a.n_experts, me = blockIdx.x;     // me == E: the dropped pairs
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i <= E; i += kSortThreads) s_hist[i] = 0;
  __syncthreads();
  for (int64_t c0 = 0; c0 < a.pairs; c0 += kSortChunk) sort_scan<true>(a, c0, me, s_hist, s_bits);
  __syncthreads();
  // places and tiles before this expert
  int before = 0, tiles = 0;
  for (int e = tid; e < me; e += kSortThreads) {
    before += s_hist[e];
    if (a.tile_rows > 0) tiles += (s_hist[e] + a.tile_rows - 1) / a.tile_rows;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  tiles = __reduce_add_sync(0xffffffffu, tiles);
  if (lane == 0) {
    s_red[0][warp] = before;
    s_red[1][warp] = tiles;
  }
  __syncthreads();
  before = tiles = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    before += s_red[0][w];
    tiles += s_red[1][w];
  }
  int place = a.tile_rows > 0 ? tiles * a.tile_rows : before;
  const int count = s_hist[me];
  if (tid == 0) {
    if (a.offsets) a.offsets[me] = place;
    if (me == E && a.n_tiles) *a.n_tiles = tiles;
  }
  if (me < E && a.tile_rows > 0) {
    const int n = (count + a.tile_rows - 1) / a.tile_rows;
    for (int i = tid; i < n; i += kSortThreads) {
      a.tile_expert[tiles + i] = me;
      a.tile_count[tiles + i] = min(a.tile_rows, count - i * a.tile_rows);
    }
  }
  if (count == 0) return;
  for (int64_t c0 = 0; c0 < a.pairs; c0 += kSortChunk) {
    if (a.pairs > kSortChunk) {
      __syncthreads();                              // the chunk before is written out
      sort_scan<false>(a, c0, me, s_hist, s_bits);
    }
    const int64_t ids = a.pairs - c0 < kSortChunk ? a.pairs - c0 : kSortChunk;
    const int words = static_cast<int>((ids + 31) / 32);
    // each thread owns `per` consecutive words
    const int per = (words + kSortThreads - 1) / kSortThreads;
    const int w0 = min(tid * per, words), w1 = min(w0 + per, words);
    __syncthreads();
    int mine = 0;
    for (int w = w0; w < w1; ++w) mine += __popc(s_bits[w]);
    int at = mine;                                  // inclusive scan over the warp, then the warps
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, at, m);
      if (lane >= m) at += o;
    }
    if (lane == 31) s_red[0][warp] = at;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) at += s_red[0][w];
      sum += s_red[0][w];
    }
    int p = place + at - mine;
    for (int w = w0; w < w1; ++w) {
      for (uint32_t m = s_bits[w]; m; m &= m - 1, ++p) {
        const int64_t i = c0 + static_cast<int64_t>(w) * 32 + __ffs(m) - 1;
        if (a.position) a.position[i] = me < E ? p : -1;
        if (a.order) a.order[p] = me < E ? static_cast<int32_t>(i) : -1;
      }
    }
    place += sum;
  }
}

cudaError_t sort_launch(const SortArgs &a, cudaStream_t s) {
  return launch_pdl(sort_pairs_kernel, dim3(a.n_experts + 1), dim3(kSortThreads), 0, s, a);
}


// ---------------------------------------------------------------------------
// Rows. One block per token; a thread owns the same 16 bytes (or, for rows that
// do not start on 16-byte boundaries, the same value) of the token's row and of
// its pairs' rows, so each row is read or written once, in 16-byte pieces.
// ---------------------------------------------------------------------------
constexpr int kRowMaxK = 8;

// A piece of a row: V = 16 bytes' worth of T, or 1 value.
template <typename T, int V> SI_DEV void row_load(const T *p, float v[V]) {
  if constexpr (V == 1) {
    v[0] = to_f32<T>(*p);
  } else {
    unpack16<T>(__ldcg(reinterpret_cast<const uint4 *>(p)), v);
  }
}
template <typename T, int V> SI_DEV void row_store(T *p, const float v[V]) {
  if constexpr (V == 1) {
    *p = from_f32<T>(v[0]);
  } else {
    *reinterpret_cast<uint4 *>(p) = pack16<T>(v);
  }
}

struct RowArgs {
  int k;
  int64_t hidden, rows;      // rows: of the sorted side
  const int32_t *position;   // [tokens][k]
  const int32_t *n_kept;     // offsets + E
};
// Row of pair (t, r), -1 for a dropped pair, a missing rank, or a place that
// is no row: nothing outside the buffers is touched.
SI_DEV int row_of(const RowArgs &a, int64_t t, int r) {
  if (r >= a.k) return -1;
  const int p = __ldcg(a.position + t * a.k + r);
  return p >= 0 && p < a.rows ? p : -1;
}

// Zero rows behind the kept pairs: block t takes rows t * k .. t * k + k - 1.
template <typename T, int V> SI_DEV void zero_tail(const RowArgs &a, T *rows) {
  const int64_t kept = __ldcg(a.n_kept);
  const float z[V] = {};
  for (int r = 0; r < a.k; ++r) {
    const int64_t p = static_cast<int64_t>(blockIdx.x) * a.k + r;
    if (p < kept) continue;
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < a.hidden; c += static_cast<int64_t>(blockDim.x) * V)
      row_store<T, V>(rows + p * a.hidden + c, z);
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(256) gather_rows_kernel(RowArgs a, const T *__restrict__ x, T *__restrict__ xs) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t = blockIdx.x;
  int p[kRowMaxK];
#pragma unroll
  for (int r = 0; r < kRowMaxK; ++r) p[r] = row_of(a, t, r);
  for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < a.hidden; c += static_cast<int64_t>(blockDim.x) * V) {
    float v[V];
    row_load<T, V>(x + t * a.hidden + c, v);
#pragma unroll
    for (int r = 0; r < kRowMaxK; ++r)
      if (p[r] >= 0) row_store<T, V>(xs + p[r] * a.hidden + c, v);
  }
  zero_tail<T, V>(a, xs);
}

// y[t] = sum_r w[t][r] rows[position[t][r]]; w NULL: a plain sum.
template <typename T, int V>
__global__ void __launch_bounds__(256)
    combine_rows_kernel(RowArgs a, const T *__restrict__ rows, const float *__restrict__ w, T *__restrict__ y) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t = blockIdx.x;
  int p[kRowMaxK];
  float g[kRowMaxK];
#pragma unroll
  for (int r = 0; r < kRowMaxK; ++r) {
    p[r] = row_of(a, t, r);
    g[r] = w && p[r] >= 0 ? __ldcg(w + t * a.k + r) : 1.f;
  }
  for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < a.hidden; c += static_cast<int64_t>(blockDim.x) * V) {
    float v[kRowMaxK][V];
#pragma unroll
    for (int r = 0; r < kRowMaxK; ++r)
      if (p[r] >= 0) row_load<T, V>(rows + p[r] * a.hidden + c, v[r]);
    float acc[V] = {};
#pragma unroll
    for (int r = 0; r < kRowMaxK; ++r)
      if (p[r] >= 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(g[r], v[r][i], acc[i]);
      }
    row_store<T, V>(y + t * a.hidden + c, acc);
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(256)
    combine_backward_kernel(RowArgs a, const T *__restrict__ gy, const T *__restrict__ ys,
                            const float *__restrict__ w, T *__restrict__ gys, float *__restrict__ gw) {
  __shared__ float s_dot[kRowMaxK][8];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int p[kRowMaxK];
  float g[kRowMaxK], dot[kRowMaxK];
#pragma unroll
  for (int r = 0; r < kRowMaxK; ++r) {
    p[r] = row_of(a, t, r);
    g[r] = p[r] >= 0 ? __ldcg(w + t * a.k + r) : 0.f;
    dot[r] = 0.f;
  }
  for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < a.hidden; c += static_cast<int64_t>(blockDim.x) * V) {
    float q[V], v[kRowMaxK][V];
    row_load<T, V>(gy + t * a.hidden + c, q);
#pragma unroll
    for (int r = 0; r < kRowMaxK; ++r)
      if (p[r] >= 0) row_load<T, V>(ys + p[r] * a.hidden + c, v[r]);
#pragma unroll
    for (int r = 0; r < kRowMaxK; ++r)
      if (p[r] >= 0) {
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          dot[r] = fmaf(q[i], v[r][i], dot[r]);
          o[i] = g[r] * q[i];
        }
        row_store<T, V>(gys + p[r] * a.hidden + c, o);
      }
  }
#pragma unroll
  for (int r = 0; r < kRowMaxK; ++r) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) dot[r] += __shfl_xor_sync(0xffffffffu, dot[r], m);
    if (lane == 0) s_dot[r][warp] = dot[r];
  }
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < a.k) {
    float s = 0.f;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) s += s_dot[threadIdx.x][i];
    gw[t * a.k + threadIdx.x] = s;
  }
  zero_tail<T, V>(a, gys);
}

// ---- host ------------------------------------------------------------------

static si_status rows_check(int n_tokens, int top_k, int64_t hidden, si_dtype type, const void *position) {
  if (n_tokens < 1 || top_k < 1 || top_k > kRowMaxK || hidden < 1 || hidden > (int64_t(1) << 24) || !position ||
      (reinterpret_cast<uintptr_t>(position) & 3u))
    return SI_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n_tokens) * top_k > 0x7FFFFFFF) return SI_ERR_INVALID_ARG;
  if (type != SI_F32 && type != SI_F16 && type != SI_BF16) return SI_ERR_UNSUPPORTED;
  return SI_OK;
}
static bool whole(const void *p, int size) { return p && reinterpret_cast<uintptr_t>(p) % size == 0; }

// Threads for a row of `pieces` pieces: whole warps, at most 256.
static unsigned row_threads(int64_t pieces) {
  return static_cast<unsigned>(pieces >= 256 ? 256 : (pieces + 31) / 32 * 32);
}

// fn(T{}, V): T the type's element, V the pieces' values.
template <typename F> static cudaError_t by_type(si_dtype type, bool vec, F fn) {
  using std::integral_constant;
  if (type == SI_F32)
    return vec ? fn(float{}, integral_constant<int, 4>{}) : fn(float{}, integral_constant<int, 1>{});
  if (type == SI_BF16)
    return vec ? fn(__nv_bfloat16{}, integral_constant<int, 8>{}) : fn(__nv_bfloat16{}, integral_constant<int, 1>{});
  return vec ? fn(__half{}, integral_constant<int, 8>{}) : fn(__half{}, integral_constant<int, 1>{});
}

cudaError_t combine_launch(const void *rows, int64_t n_rows, int n_tokens, int top_k, int64_t hidden,
                           const int32_t *position, const float *w, void *y, cudaStream_t s) {
  const RowArgs a{top_k, hidden, n_rows, position, nullptr};
  return launch_pdl(combine_rows_kernel<__nv_bfloat16, 8>, dim3(n_tokens), dim3(row_threads(hidden / 8)), 0, s, a,
                    static_cast<const __nv_bfloat16 *>(rows), w, static_cast<__nv_bfloat16 *>(y));
}

}  // namespace si

using namespace si;

extern "C" si_status si_moe_sort(const int32_t *topk_ids, int n_tokens, int top_k, int n_experts, int32_t *order,
                                 int32_t *position, int32_t *offsets, void *stream) {
  if (!whole(topk_ids, 4) || !whole(order, 4) || !whole(position, 4) || !whole(offsets, 4)) return SI_ERR_INVALID_ARG;
  if (n_tokens < 1 || top_k < 1 || top_k > kRowMaxK || n_experts < 1 || n_experts > kSortMaxExperts ||
      static_cast<int64_t>(n_tokens) * top_k > 0x7FFFFFFF)
    return SI_ERR_INVALID_ARG;
  SortArgs a{};
  a.ids = topk_ids;
  a.pairs = static_cast<int64_t>(n_tokens) * top_k;
  a.n_experts = n_experts;
  a.order = order;
  a.position = position;
  a.offsets = offsets;
  return cuda_status(sort_launch(a, static_cast<cudaStream_t>(stream)));
}

extern "C" si_status si_moe_gather(const void *x, si_dtype type, int n_tokens, int top_k, int64_t hidden,
                                   const int32_t *position, const int32_t *n_kept, void *xs, void *stream) {
  const si_status st = rows_check(n_tokens, top_k, hidden, type, position);
  if (st != SI_OK) return st;
  const int size = type == SI_F32 ? 4 : 2;
  if (!whole(x, size) || !whole(xs, size) || !whole(n_kept, 4)) return SI_ERR_INVALID_ARG;
  const bool vec = hidden * size % 16 == 0 && aligned16(x) && aligned16(xs);
  const RowArgs a{top_k, hidden, static_cast<int64_t>(n_tokens) * top_k, position, n_kept};
  return cuda_status(by_type(type, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value;
    return launch_pdl(gather_rows_kernel<T, V>, dim3(n_tokens), dim3(row_threads(hidden / V)), 0,
                      static_cast<cudaStream_t>(stream), a, static_cast<const T *>(x), static_cast<T *>(xs));
  }));
}

static si_status combine_enqueue(const void *rows, si_dtype type, int n_tokens, int top_k, int64_t hidden,
                                 const int32_t *position, const float *w, void *y, void *stream) {
  const si_status st = rows_check(n_tokens, top_k, hidden, type, position);
  if (st != SI_OK) return st;
  const int size = type == SI_F32 ? 4 : 2;
  if (!whole(rows, size) || !whole(y, size)) return SI_ERR_INVALID_ARG;
  const bool vec = hidden * size % 16 == 0 && aligned16(rows) && aligned16(y);
  const RowArgs a{top_k, hidden, static_cast<int64_t>(n_tokens) * top_k, position, nullptr};
  return cuda_status(by_type(type, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value;
    return launch_pdl(combine_rows_kernel<T, V>, dim3(n_tokens), dim3(row_threads(hidden / V)), 0,
                      static_cast<cudaStream_t>(stream), a, static_cast<const T *>(rows), w, static_cast<T *>(y));
  }));
}

extern "C" si_status si_moe_combine(const void *ys, si_dtype type, int n_tokens, int top_k, int64_t hidden,
                                    const int32_t *position, const float *topk_w, void *y, void *stream) {
  if (!whole(topk_w, 4)) return SI_ERR_INVALID_ARG;
  return combine_enqueue(ys, type, n_tokens, top_k, hidden, position, topk_w, y, stream);
}

extern "C" si_status si_moe_gather_backward(const void *gxs, si_dtype type, int n_tokens, int top_k, int64_t hidden,
                                            const int32_t *position, void *gx, void *stream) {
  return combine_enqueue(gxs, type, n_tokens, top_k, hidden, position, nullptr, gx, stream);
}

extern "C" si_status si_moe_combine_backward(const void *gy, const void *ys, si_dtype type, int n_tokens, int top_k,
                                             int64_t hidden, const int32_t *position, const int32_t *n_kept,
                                             const float *topk_w, void *gys, float *gw, void *stream) {
  const si_status st = rows_check(n_tokens, top_k, hidden, type, position);
  if (st != SI_OK) return st;
  const int size = type == SI_F32 ? 4 : 2;
  if (!whole(gy, size) || !whole(ys, size) || !whole(gys, size) || !whole(n_kept, 4) || !whole(topk_w, 4) ||
      !whole(gw, 4))
    return SI_ERR_INVALID_ARG;
  const bool vec = hidden * size % 16 == 0 && aligned16(gy) && aligned16(ys) && aligned16(gys);
  const RowArgs a{top_k, hidden, static_cast<int64_t>(n_tokens) * top_k, position, n_kept};
  return cuda_status(by_type(type, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value;
    return launch_pdl(combine_backward_kernel<T, V>, dim3(n_tokens), dim3(row_threads(hidden / V)), 0,
                      static_cast<cudaStream_t>(stream), a, static_cast<const T *>(gy), static_cast<const T *>(ys),
                      topk_w, static_cast<T *>(gys), gw);
  }));
}
