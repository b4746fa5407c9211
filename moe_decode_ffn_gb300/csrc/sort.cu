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
// Sort of few pairs: one block per expert (and one for the dropped pairs), one
// launch. Every block counts all ids into shared memory, so it knows where its
// expert starts without waiting for another block, and keeps one bit per id for
// its own matches; a scan over the words of 32 bits gives every match its place.
// Latency bounds it: 3.0 us for 64 x 8 pairs over 128 experts, 5.5 us for 512 x 8.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;

SI_DEV void sort_place(const SortArgs &a, int64_t i, int e, int p) {
  if (a.position) a.position[i] = e < a.n_experts ? p : -1;
  if (a.order) a.order[p] = e < a.n_experts ? static_cast<int32_t>(i) : -1;
}

__global__ void __launch_bounds__(kSortThreads) sort_pairs_kernel(SortArgs a) {
  __shared__ int s_hist[kSortMaxExperts + 1];
  __shared__ uint32_t s_bits[kSortFewPairs / 32];
  __shared__ int s_red[2][kSortWarps];
  grid_dep_wait();
  grid_dep_launch();
  const int E = a.n_experts, me = blockIdx.x, n = static_cast<int>(a.pairs);   // me == E: the dropped pairs
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i <= E; i += kSortThreads) s_hist[i] = 0;
  __syncthreads();
  for (int b = tid & ~31; b < n; b += kSortThreads) {
    const int i = b + lane;
    const int e = i < n ? sort_expert(a, i) : -1;
    if (e >= 0) atomicAdd(&s_hist[e], 1);
    const uint32_t m = __ballot_sync(0xffffffffu, e == me);
    if (lane == 0) s_bits[b >> 5] = m;
  }
  __syncthreads();
  // pairs and tiles before this expert
  int before = 0, tiles = 0;
  for (int e = tid; e < me; e += kSortThreads) {
    before += s_hist[e];
    tiles += sort_tiles(a, s_hist[e]);
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
  const int place = a.tile_rows > 0 ? tiles * a.tile_rows : before;
  if (tid == 0) {
    if (a.offsets) a.offsets[me] = place;
    if (me == E && a.n_tiles) *a.n_tiles = tiles;
  }
  if (me < E && a.tile_rows > 0) sort_list(a, me, s_hist[me], tiles, tid, kSortThreads);
  // a thread's word: the matches before it are those of the words before
  for (int w = warp; w * 32 < n; w += kSortWarps) {
    const uint32_t m = s_bits[w];
    if (m == 0) continue;
    int at = 0;
    for (int j = lane; j < w; j += 32) at += __popc(s_bits[j]);
    at = __reduce_add_sync(0xffffffffu, at);
    if (m >> lane & 1u) sort_place(a, w * 32 + lane, me, place + at + __popc(m & ((1u << lane) - 1u)));
  }
}

// ---------------------------------------------------------------------------
// Sort of many pairs, two launches over at most kSortChunks chunks of ids: the
// first counts every chunk's ids by expert; a block of the second sums the
// counts of the chunks before its own and of the experts before each expert, and
// places its ids in rounds of kSortRound: a warp ranks its ids with match.any,
// a scan over the warps' counts does the rest. 1024 x 8 pairs 5.9 us, 8192 x 8 over
// 256 experts 9.4 us; with a block per expert that reads all ids, 20 us.
// ---------------------------------------------------------------------------
constexpr int kSortIds = 2;                                // ids per thread and round
constexpr int kSortRound = kSortThreads * kSortIds;

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a) {
  __shared__ int s_hist[kSortMaxExperts + 1];
  grid_dep_wait();
  grid_dep_launch();
  for (int i = threadIdx.x; i <= a.n_experts; i += kSortThreads) s_hist[i] = 0;
  __syncthreads();
  const int64_t c0 = a.chunk * blockIdx.x, c1 = min(c0 + a.chunk, a.pairs);
  for (int64_t i = c0 + threadIdx.x; i < c1; i += kSortRound) {
#pragma unroll
    for (int u = 0; u < kSortIds; ++u)
      if (i + u * kSortThreads < c1) atomicAdd(&s_hist[sort_expert(a, i + u * kSortThreads)], 1);
  }
  __syncthreads();
  int32_t *row = a.counts + static_cast<size_t>(blockIdx.x) * (a.n_experts + 1);
  for (int i = threadIdx.x; i <= a.n_experts; i += kSortThreads) row[i] = s_hist[i];
}

// Exclusive sums of v over the threads of the block (s_red: one word a warp).
SI_DEV int block_scan(int v, int *s_red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int at = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, at, m);
    if (lane >= m) at += o;
  }
  __syncthreads();                                         // s_red may still be read
  if (lane == 31) s_red[warp] = at;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w)
    if (w < warp) at += s_red[w];
  return at - v;
}

__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortArgs a) {
  extern __shared__ int s_warp[];                          // [kSortWarps][E + 1]
  __shared__ int s_next[kSortMaxExperts + 1];              // next place of an expert in this chunk
  __shared__ int s_red[kSortWarps];
  const int E = a.n_experts, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_wait();
  grid_dep_launch();
  const int64_t c0 = a.chunk * blockIdx.x, c1 = min(c0 + a.chunk, a.pairs);
  // experts in runs of `per` consecutive ones a thread
  const int per = (E + kSortThreads) / kSortThreads;
  const int e0 = min(tid * per, E + 1), e1 = min(e0 + per, E + 1);
  int mine = 0, my_tiles = 0;
  for (int e = e0; e < e1; ++e) {
    int total = 0, before = 0;
    for (int c0 = 0; c0 < static_cast<int>(gridDim.x); c0 += 16) {
      int n[16];
#pragma unroll
      for (int u = 0; u < 16; ++u)
        n[u] = c0 + u < static_cast<int>(gridDim.x) ? __ldcg(a.counts + static_cast<size_t>(c0 + u) * (E + 1) + e) : 0;
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        if (c0 + u < static_cast<int>(blockIdx.x)) before += n[u];
        total += n[u];
      }
    }
    s_next[e] = before;
    s_warp[e] = total;
    mine += total;
    if (e < E) my_tiles += sort_tiles(a, total);
  }
  int at = block_scan(mine, s_red), tile = a.tile_rows > 0 ? block_scan(my_tiles, s_red) : 0;
  for (int e = e0; e < e1; ++e) {
    const int total = s_warp[e], place = a.tile_rows > 0 ? tile * a.tile_rows : at;
    s_next[e] += place;
    if (blockIdx.x == 0) {
      if (a.offsets) a.offsets[e] = place;
      if (e == E && a.n_tiles) *a.n_tiles = tile;
    }
    // every block lists the tiles of some experts
    if (e < E && a.tile_rows > 0 && e % gridDim.x == blockIdx.x) sort_list(a, e, total, tile, 0, 1);
    at += total;
    if (e < E) tile += sort_tiles(a, total);
  }
  int *counts = s_warp + warp * (E + 1);
  for (int64_t b = c0; b < c1; b += kSortRound) {
    __syncthreads();
    for (int i = lane; i <= E; i += 32) counts[i] = 0;
    __syncwarp();
    int e[kSortIds], rank[kSortIds];
    const int64_t i0 = b + warp * (32 * kSortIds) + lane;
#pragma unroll
    for (int u = 0; u < kSortIds; ++u) e[u] = i0 + u * 32 < c1 ? sort_expert(a, i0 + u * 32) : -1;
#pragma unroll
    for (int u = 0; u < kSortIds; ++u) {
      const uint32_t same = __match_any_sync(0xffffffffu, e[u]);
      rank[u] = __popc(same & ((1u << lane) - 1u));
      if (e[u] >= 0) rank[u] += counts[e[u]];
      __syncwarp();
      if (e[u] >= 0 && lane == 31 - __clz(same)) counts[e[u]] = rank[u] + 1;
      __syncwarp();
    }
    __syncthreads();
    for (int x = tid; x <= E; x += kSortThreads) {
      int next = s_next[x];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const int n = s_warp[w * (E + 1) + x];
        s_warp[w * (E + 1) + x] = next;
        next += n;
      }
      s_next[x] = next;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kSortIds; ++u)
      if (e[u] >= 0) sort_place(a, i0 + u * 32, e[u], counts[e[u]] + rank[u]);
  }
}

size_t sort_workspace_bytes(int64_t pairs, int n_experts) {
  return pairs <= kSortFewPairs ? 0 : static_cast<size_t>(kSortChunks) * (n_experts + 1) * sizeof(int32_t);
}

cudaError_t sort_launch(SortArgs a, cudaStream_t s) {
  if (a.pairs <= kSortFewPairs)
    return launch_pdl(sort_pairs_kernel, dim3(a.n_experts + 1), dim3(kSortThreads), 0, s, a);
  // whole rounds, at most kSortChunks chunks
  a.chunk = (a.pairs + kSortChunks * int64_t(kSortRound) - 1) / (kSortChunks * int64_t(kSortRound)) * kSortRound;
  const dim3 grid(static_cast<unsigned>((a.pairs + a.chunk - 1) / a.chunk));
  cudaError_t e = launch_pdl(sort_count_kernel, grid, dim3(kSortThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  const size_t smem = static_cast<size_t>(kSortWarps) * (a.n_experts + 1) * sizeof(int);
  e = allow_smem(sort_place_kernel, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(sort_place_kernel, grid, dim3(kSortThreads), smem, s, a);
}

// ---------------------------------------------------------------------------
// Rows. A block walks over tokens; a thread owns the same 16 bytes (or, for rows
// that do not start on 16-byte boundaries, the same value) of the token's row
// and of its pairs' rows, so each row is read or written once, in 16-byte
// pieces. Lane r of every warp holds the place and the weight of rank r, read
// one token ahead; a token's rows are requested together and stay packed in
// registers until they are summed.
// ---------------------------------------------------------------------------
constexpr int kRowMaxK = 8;
constexpr int kRowThreads = 256;

// A piece of a row: V = 16 bytes' worth of T as it lies in memory, or 1 value.
template <typename T, int V> struct Piece {
  uint4 u;
  SI_DEV void load(const T *p) { u = __ldcg(reinterpret_cast<const uint4 *>(p)); }
  SI_DEV void store(T *p) const { *reinterpret_cast<uint4 *>(p) = u; }
  SI_DEV void unpack(float v[V]) const { unpack16<T>(u, v); }
  SI_DEV void pack(const float v[V]) { u = pack16<T>(v); }
};
template <typename T> struct Piece<T, 1> {
  T u;
  SI_DEV void load(const T *p) { u = *p; }
  SI_DEV void store(T *p) const { *p = u; }
  SI_DEV void unpack(float v[1]) const { v[0] = to_f32<T>(u); }
  SI_DEV void pack(const float v[1]) { u = from_f32<T>(v[0]); }
};

struct RowArgs {
  int64_t tokens;
  int k;
  int64_t hidden, rows;      // rows: of the sorted side
  const int32_t *position;   // [tokens][k]
  const float *w;            // [tokens][k], or NULL for ones
  const int32_t *n_kept;     // offsets + E
};
// Rank `lane` of token t: its row, -1 for a dropped pair, a missing rank, or a
// place that is no row (nothing outside the buffers is touched), and its weight.
struct Pair {
  int p;
  float w;
};
SI_DEV Pair pair_of(const RowArgs &a, int64_t t, int lane) {
  Pair q = {-1, 1.f};
  if (t < a.tokens && lane < a.k) {
    q.p = __ldcg(a.position + t * a.k + lane);
    if (a.w) q.w = __ldcg(a.w + t * a.k + lane);
    if (q.p < 0 || q.p >= a.rows) q.p = -1;
  }
  return q;
}

// Zero rows behind the kept pairs: token t stands for rows t * k .. t * k + k - 1.
template <typename T, int V> SI_DEV void zero_tail(const RowArgs &a, int64_t t, int64_t kept, T *rows) {
  const float z[V] = {};
  Piece<T, V> o;
  o.pack(z);
  for (int64_t p = t * a.k < kept ? kept : t * a.k; p < (t + 1) * a.k; ++p)
    for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < a.hidden; c += static_cast<int64_t>(blockDim.x) * V)
      o.store(rows + p * a.hidden + c);
}

// One block per token: the rows written, 8 of 9, need no pipeline, and blocks
// that walk over tokens measured slower (55.1 against 46.3 us, 6.5 TB/s, for
// 8192 x 8 rows of 4 KB).
template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) gather_rows_kernel(RowArgs a, const T *__restrict__ x, T *__restrict__ xs) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  int64_t kept = __ldcg(a.n_kept);
  if (kept < 0) kept = 0;
  const Pair now = pair_of(a, t, lane);
  int p[kRowMaxK];
#pragma unroll
  for (int r = 0; r < kRowMaxK; ++r) p[r] = __shfl_sync(0xffffffffu, now.p, r);
  for (int64_t c = static_cast<int64_t>(threadIdx.x) * V; c < a.hidden; c += static_cast<int64_t>(blockDim.x) * V) {
    Piece<T, V> v;
    v.load(x + t * a.hidden + c);
#pragma unroll
    for (int r = 0; r < kRowMaxK; ++r)
      if (p[r] >= 0) v.store(xs + p[r] * a.hidden + c);
  }
  zero_tail<T, V>(a, t, kept, xs);
}

// y[t] = sum_r w[t][r] rows[position[t][r]]. Three blocks an SM: 53.6 us for 8192
// x 8 rows of 4 KB (5.6 TB/s); four 58.2, two with the next token's rows in
// flight as well 63.5, rows asked into the L2 a token ahead 64.2.
// TO: the sums' type; the MXFP4 experts' rows are fp32 and their sums bf16 (4096 x 8
// rows of 8 KB 49.2 us, 5.8 TB/s).
template <typename T, int V, typename TO = T>
__global__ void __launch_bounds__(kRowThreads, 3)
    combine_rows_kernel(RowArgs a, const T *__restrict__ rows, TO *__restrict__ y) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  Pair next = pair_of(a, blockIdx.x, lane);
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const Pair now = next;
    next = pair_of(a, t + gridDim.x, lane);
    for (int64_t c0 = static_cast<int64_t>(threadIdx.x) * V; c0 - lane * V < a.hidden;
         c0 += static_cast<int64_t>(blockDim.x) * V) {
      const bool in = c0 < a.hidden;
      const int64_t c = in ? c0 : 0;               // the warp's lanes stay together for the shuffles
      Piece<T, V> v[kRowMaxK];
#pragma unroll
      for (int r = 0; r < kRowMaxK; ++r) {
        const int p = __shfl_sync(0xffffffffu, now.p, r);
        if (p >= 0) v[r].load(rows + p * a.hidden + c);
      }
      float acc[V] = {};
#pragma unroll
      for (int r = 0; r < kRowMaxK; ++r) {
        const int p = __shfl_sync(0xffffffffu, now.p, r);
        const float g = __shfl_sync(0xffffffffu, now.w, r);
        if (p < 0) continue;
        float f[V];
        v[r].unpack(f);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(g, f[i], acc[i]);
      }
      if constexpr (std::is_same_v<T, TO>) {
        Piece<T, V> o;
        o.pack(acc);
        if (in) o.store(y + t * a.hidden + c);
      } else {
        static_assert(V == 4 && std::is_same_v<TO, __nv_bfloat16>, "fp32 rows to bf16");
        const uint2 o = make_uint2(bf16_bits(acc[0]) | (static_cast<uint32_t>(bf16_bits(acc[1])) << 16),
                                   bf16_bits(acc[2]) | (static_cast<uint32_t>(bf16_bits(acc[3])) << 16));
        if (in) *reinterpret_cast<uint2 *>(y + t * a.hidden + c) = o;
      }
    }
  }
}

// The rows of the next token on their way into the L2: lane r asks for row r.
// It pays where rows are written as well: 107.8 -> 99.0 us (5.8 TB/s) for 8192 x 8
// rows of 4 KB.
template <typename T, int V> SI_DEV void prefetch_rows(const RowArgs &a, const Pair &next, const T *rows) {
  if constexpr (V > 1) {
    if (threadIdx.x < 32 && next.p >= 0)
      bulk_prefetch_l2(rows + next.p * a.hidden, static_cast<uint32_t>(a.hidden * sizeof(T)));
  }
}

// Sums of 8 values over the warp, each lane handing half of its values on at
// every step: value (lane / 4) on lanes 4i (9 shuffles instead of 40).
SI_DEV float reduce8(float v[8], int lane) {
#pragma unroll
  for (int n = 4, m = 16; n > 0; n >>= 1, m >>= 1) {
    const bool up = (lane & m) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
    }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads, 3)
    combine_backward_kernel(RowArgs a, const T *__restrict__ gy, const T *__restrict__ ys, T *__restrict__ gys,
                            float *__restrict__ gw) {
  __shared__ float s_dot[2][kRowMaxK][kRowThreads / 32];   // by the token's parity: one barrier a token
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t kept = __ldcg(a.n_kept);
  if (kept < 0) kept = 0;
  Pair next = pair_of(a, blockIdx.x, lane);
  int par = 0;
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x, par ^= 1) {
    const Pair now = next;
    next = pair_of(a, t + gridDim.x, lane);
    prefetch_rows<T, V>(a, next, ys);
    float dot[kRowMaxK] = {};
    for (int64_t c0 = static_cast<int64_t>(threadIdx.x) * V; c0 - lane * V < a.hidden;
         c0 += static_cast<int64_t>(blockDim.x) * V) {
      const bool in = c0 < a.hidden;
      const int64_t c = in ? c0 : 0;
      Piece<T, V> q, v[kRowMaxK];
      q.load(gy + t * a.hidden + c);
#pragma unroll
      for (int r = 0; r < kRowMaxK; ++r) {
        const int p = __shfl_sync(0xffffffffu, now.p, r);
        if (p >= 0) v[r].load(ys + p * a.hidden + c);
      }
      float g[V];
      q.unpack(g);
      if (!in) {
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = 0.f;
      }
#pragma unroll
      for (int r = 0; r < kRowMaxK; ++r) {
        const int p = __shfl_sync(0xffffffffu, now.p, r);
        const float w = __shfl_sync(0xffffffffu, now.w, r);
        if (p < 0) continue;
        float f[V], o[V];
        v[r].unpack(f);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (in) dot[r] = fmaf(g[i], f[i], dot[r]);
          o[i] = w * g[i];
        }
        Piece<T, V> ov;
        ov.pack(o);
        if (in) ov.store(gys + p * a.hidden + c);
      }
    }
    const float sum = reduce8(dot, lane);
    if ((lane & 3) == 0) s_dot[par][lane >> 2][warp] = sum;
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < a.k) {
      float s = 0.f;
      for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) s += s_dot[par][threadIdx.x][i];
      gw[t * a.k + threadIdx.x] = s;
    }
    zero_tail<T, V>(a, t, kept, gys);
  }
}

// ---- host ------------------------------------------------------------------

// Threads for a row of `pieces` pieces: whole warps, at most kRowThreads.
static unsigned row_threads(int64_t pieces) {
  return static_cast<unsigned>(pieces >= kRowThreads ? kRowThreads : (pieces + 31) / 32 * 32);
}
// Blocks: as many tokens as stay resident at once, for `per_sm` threads an SM.
static unsigned row_blocks(int64_t tokens, unsigned threads, int per_sm) {
  const int64_t most = static_cast<int64_t>(sm_count()) * (per_sm / threads);
  return static_cast<unsigned>(tokens < most ? tokens : most);
}

static si_status rows_check(int n_tokens, int top_k, int64_t hidden, si_dtype type, const void *position) {
  if (n_tokens < 1 || top_k < 1 || top_k > kRowMaxK || hidden < 1 || hidden > (int64_t(1) << 24) || !position ||
      (reinterpret_cast<uintptr_t>(position) & 3u))
    return SI_ERR_INVALID_ARG;
  if (static_cast<int64_t>(n_tokens) * top_k > 0x7FFFFFFF) return SI_ERR_INVALID_ARG;
  if (type != SI_F32 && type != SI_F16 && type != SI_BF16) return SI_ERR_UNSUPPORTED;
  return SI_OK;
}
static bool whole(const void *p, int size) { return p && reinterpret_cast<uintptr_t>(p) % size == 0; }

// fn(T{}, V): T the type's element, V the pieces' values.
template <typename F> static cudaError_t by_type(si_dtype type, bool vec, F fn) {
  using std::integral_constant;
  if (type == SI_F32)
    return vec ? fn(float{}, integral_constant<int, 4>{}) : fn(float{}, integral_constant<int, 1>{});
  if (type == SI_BF16)
    return vec ? fn(__nv_bfloat16{}, integral_constant<int, 8>{}) : fn(__nv_bfloat16{}, integral_constant<int, 1>{});
  return vec ? fn(__half{}, integral_constant<int, 8>{}) : fn(__half{}, integral_constant<int, 1>{});
}

static cudaError_t combine_rows(const RowArgs &a, si_dtype type, bool vec, const void *rows, void *y, cudaStream_t s) {
  return by_type(type, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value;
    const unsigned threads = row_threads(a.hidden / V);
    return launch_pdl(combine_rows_kernel<T, V>, dim3(row_blocks(a.tokens, threads, 3 * kRowThreads)), dim3(threads),
                      0, s, a, static_cast<const T *>(rows), static_cast<T *>(y));
  });
}

cudaError_t combine_launch(const float *rows, int64_t n_rows, int n_tokens, int top_k, int64_t hidden,
                           const int32_t *position, const float *w, void *y, cudaStream_t s) {
  const RowArgs a{n_tokens, top_k, hidden, n_rows, position, w, nullptr};
  const unsigned threads = row_threads(hidden / 4);
  return launch_pdl(combine_rows_kernel<float, 4, __nv_bfloat16>, dim3(row_blocks(n_tokens, threads, 3 * kRowThreads)),
                    dim3(threads), 0, s, a, rows, static_cast<__nv_bfloat16 *>(y));
}

}  // namespace si

using namespace si;

static bool sort_shape_ok(int n_tokens, int top_k, int n_experts) {
  return n_tokens >= 1 && top_k >= 1 && top_k <= kRowMaxK && n_experts >= 1 && n_experts <= kSortMaxExperts &&
         static_cast<int64_t>(n_tokens) * top_k <= 0x7FFFFFFF;
}

extern "C" size_t si_moe_sort_workspace_bytes(int n_tokens, int top_k, int n_experts) {
  if (!sort_shape_ok(n_tokens, top_k, n_experts)) return 0;
  const size_t need = sort_workspace_bytes(static_cast<int64_t>(n_tokens) * top_k, n_experts);
  return need ? round_up(need, 256) : 0;
}

extern "C" si_status si_moe_sort(const int32_t *topk_ids, int n_tokens, int top_k, int n_experts, int32_t *order,
                                 int32_t *position, int32_t *offsets, void *workspace, size_t workspace_bytes,
                                 void *stream) {
  if (!whole(topk_ids, 4) || !whole(order, 4) || !whole(position, 4) || !whole(offsets, 4)) return SI_ERR_INVALID_ARG;
  if (!sort_shape_ok(n_tokens, top_k, n_experts)) return SI_ERR_INVALID_ARG;
  const size_t need = si_moe_sort_workspace_bytes(n_tokens, top_k, n_experts);
  if (need && (!workspace || !aligned256(workspace) || workspace_bytes < need)) return SI_ERR_WORKSPACE;
  SortArgs a{};
  a.ids = topk_ids;
  a.pairs = static_cast<int64_t>(n_tokens) * top_k;
  a.n_experts = n_experts;
  a.order = order;
  a.position = position;
  a.offsets = offsets;
  a.counts = static_cast<int32_t *>(workspace);
  return cuda_status(sort_launch(a, static_cast<cudaStream_t>(stream)));
}

extern "C" si_status si_moe_gather(const void *x, si_dtype type, int n_tokens, int top_k, int64_t hidden,
                                   const int32_t *position, const int32_t *n_kept, void *xs, void *stream) {
  const si_status st = rows_check(n_tokens, top_k, hidden, type, position);
  if (st != SI_OK) return st;
  const int size = type == SI_F32 ? 4 : 2;
  if (!whole(x, size) || !whole(xs, size) || !whole(n_kept, 4)) return SI_ERR_INVALID_ARG;
  const bool vec = hidden * size % 16 == 0 && aligned16(x) && aligned16(xs);
  const RowArgs a{n_tokens, top_k, hidden, static_cast<int64_t>(n_tokens) * top_k, position, nullptr, n_kept};
  return cuda_status(by_type(type, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value;
    const unsigned threads = row_threads(hidden / V);
    return launch_pdl(gather_rows_kernel<T, V>, dim3(n_tokens), dim3(threads), 0,
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
  const RowArgs a{n_tokens, top_k, hidden, static_cast<int64_t>(n_tokens) * top_k, position, w, nullptr};
  return cuda_status(combine_rows(a, type, vec, rows, y, static_cast<cudaStream_t>(stream)));
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
  const RowArgs a{n_tokens, top_k, hidden, static_cast<int64_t>(n_tokens) * top_k, position, topk_w, n_kept};
  return cuda_status(by_type(type, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value;
    const unsigned threads = row_threads(hidden / V);
    return launch_pdl(combine_backward_kernel<T, V>, dim3(row_blocks(n_tokens, threads, 3 * kRowThreads)),
                      dim3(threads), 0, static_cast<cudaStream_t>(stream), a, static_cast<const T *>(gy),
                      static_cast<const T *>(ys), static_cast<T *>(gys), gw);
  }));
}
