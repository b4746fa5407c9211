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
// Sort: one block per expert (and one for the dropped pairs), one launch. Every
// block compares all ids with its expert and keeps one bit per id; a scan over
// the words of 32 bits then gives every match its place. Where its expert
// starts follows from a count of all ids, which it takes itself or, for long
// batches, shares with the blocks of its cluster (each counts a part into its
// shared memory and reads the other parts): no block waits for more than that.
// More ids than kSortChunk go through the bits in chunks, read again.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortWords = 2048;                    // bit words in shared memory
constexpr int64_t kSortChunk = kSortWords * 32;     // ids they hold
constexpr int kSortCluster = 8;

SI_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n barrier.cluster.wait.aligned;" ::: "memory");
}
// 32 bits of shared memory of block `rank` of this cluster, at our own address p.
SI_DEV int ld_cluster(const int *p, uint32_t rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// The ids of one chunk: match bits of expert `me`; COUNT: the ids of every
// `of`-th round of the block counted, from round `part` on. A thread takes 8
// consecutive ids, a byte of the bits.
template <bool COUNT>
SI_DEV void sort_scan(const SortArgs &a, int64_t c0, uint32_t me, int part, int of, int *s_hist, uint8_t *s_bits) {
  constexpr int U = 2;                              // bytes per thread in flight
  const uint32_t E = a.n_experts;
  const int64_t c1 = c0 + kSortChunk < a.pairs ? c0 + kSortChunk : a.pairs;
  int round = 0;
  for (int64_t b0 = c0; b0 < c1; b0 += kSortThreads * 8 * U) {
    uint32_t id[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t b = b0 + (u * kSortThreads + threadIdx.x) * 8;
      if (a.vec && b + 8 <= c1) {
        const uint4 lo = __ldcg(reinterpret_cast<const uint4 *>(a.ids + b));
        const uint4 hi = __ldcg(reinterpret_cast<const uint4 *>(a.ids + b) + 1);
        id[u][0] = lo.x; id[u][1] = lo.y; id[u][2] = lo.z; id[u][3] = lo.w;
        id[u][4] = hi.x; id[u][5] = hi.y; id[u][6] = hi.z; id[u][7] = hi.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) id[u][i] = b + i < c1 ? static_cast<uint32_t>(__ldcg(a.ids + b + i)) : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u, ++round) {
      const int64_t b = b0 + (u * kSortThreads + threadIdx.x) * 8;
      if (b >= c1) break;
      uint32_t bits = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t e = min(id[u][i], E);        // negative ids are large unsigned ones
        bits |= (e == me ? 1u : 0u) << i;
        if (COUNT && round % of == part && b + i < c1) atomicAdd(&s_hist[e], 1);
      }
      if (c1 - b < 8) bits &= (1u << (c1 - b)) - 1u;
      s_bits[(b - c0) / 8] = static_cast<uint8_t>(bits);
    }
  }
}

template <bool SHARED>
__global__ void __launch_bounds__(kSortThreads) sort_pairs_kernel(SortArgs a) {
  __shared__ int s_hist[kSortMaxExperts + 1];
  __shared__ uint32_t s_bits[kSortWords];
  __shared__ int s_red[2][kSortWarps];
  __shared__ int s_count;
  grid_dep_wait();
  grid_dep_launch();
  const int E = a.n_experts, me = blockIdx.x;     // me == E: the dropped pairs; beyond: only counting
  const int part = SHARED ? static_cast<int>(blockIdx.x) % kSortCluster : 0;
  constexpr int of = SHARED ? kSortCluster : 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i <= E; i += kSortThreads) s_hist[i] = 0;
  // whole words for the scan: bytes behind the last id are 0
  if (tid < 4) reinterpret_cast<uint8_t *>(s_bits)[min((a.pairs - 1) % kSortChunk / 8 + 1 + tid, kSortChunk / 8 - 1)] = 0;
  __syncthreads();
  for (int64_t c0 = 0; c0 < a.pairs; c0 += kSortChunk)
    sort_scan<true>(a, c0, me, part, of, s_hist, reinterpret_cast<uint8_t *>(s_bits));
  if constexpr (SHARED) cluster_sync();
  else __syncthreads();
  // pairs and tiles before this expert, and its own pairs
  int before = 0, tiles = 0;
  for (int e = tid; e <= min(me, E); e += kSortThreads) {
    int n = 0;
    if constexpr (SHARED) {
#pragma unroll
      for (int r = 0; r < kSortCluster; ++r) n += ld_cluster(s_hist + e, r);
    } else {
      n = s_hist[e];
    }
    if (e < me) {
      before += n;
      if (a.tile_rows > 0) tiles += (n + a.tile_rows - 1) / a.tile_rows;
    } else {
      s_count = n;
    }
  }
  before = __reduce_add_sync(0xffffffffu, before);
  tiles = __reduce_add_sync(0xffffffffu, tiles);
  if (lane == 0) {
    s_red[0][warp] = before;
    s_red[1][warp] = tiles;
  }
  if constexpr (SHARED) cluster_sync();             // every part has been read
  else __syncthreads();
  if (me > E) return;
  before = tiles = 0;
#pragma unroll
  for (int w = 0; w < kSortWarps; ++w) {
    before += s_red[0][w];
    tiles += s_red[1][w];
  }
  const int count = s_count;
  int place = a.tile_rows > 0 ? tiles * a.tile_rows : before;
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
      if (tid < 4 && c0 + kSortChunk >= a.pairs)
        reinterpret_cast<uint8_t *>(s_bits)[min((a.pairs - 1) % kSortChunk / 8 + 1 + tid, kSortChunk / 8 - 1)] = 0;
      __syncthreads();
      sort_scan<false>(a, c0, me, 0, 1, s_hist, reinterpret_cast<uint8_t *>(s_bits));
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

cudaError_t sort_launch(SortArgs a, cudaStream_t s) {
  a.vec = (reinterpret_cast<uintptr_t>(a.ids) & 15u) == 0;
  // the shared count pays from a few thousand pairs on
  if (a.pairs < kSortSharePairs) return launch_pdl(sort_pairs_kernel<false>, dim3(a.n_experts + 1), dim3(kSortThreads), 0, s, a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.n_experts + kSortCluster) / kSortCluster * kSortCluster);
  cfg.blockDim = dim3(kSortThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kSortCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sort_pairs_kernel<true>, a);
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

template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads) gather_rows_kernel(RowArgs a, const T *__restrict__ x, T *__restrict__ xs) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  int64_t kept = __ldcg(a.n_kept);
  if (kept < 0) kept = 0;
  Pair next = pair_of(a, blockIdx.x, lane);
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const Pair now = next;
    next = pair_of(a, t + gridDim.x, lane);
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
}

// y[t] = sum_r w[t][r] rows[position[t][r]]
template <typename T, int V>
__global__ void __launch_bounds__(kRowThreads, 4)
    combine_rows_kernel(RowArgs a, const T *__restrict__ rows, T *__restrict__ y) {
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
      Piece<T, V> o;
      o.pack(acc);
      if (in) o.store(y + t * a.hidden + c);
    }
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
    return launch_pdl(combine_rows_kernel<T, V>, dim3(row_blocks(a.tokens, threads, 4 * kRowThreads)), dim3(threads),
                      0, s, a, static_cast<const T *>(rows), static_cast<T *>(y));
  });
}

cudaError_t combine_launch(const void *rows, int64_t n_rows, int n_tokens, int top_k, int64_t hidden,
                           const int32_t *position, const float *w, void *y, cudaStream_t s) {
  const RowArgs a{n_tokens, top_k, hidden, n_rows, position, w, nullptr};
  return combine_rows(a, SI_BF16, true, rows, y, s);
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
  const RowArgs a{n_tokens, top_k, hidden, static_cast<int64_t>(n_tokens) * top_k, position, nullptr, n_kept};
  return cuda_status(by_type(type, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr int V = decltype(v)::value;
    const unsigned threads = row_threads(hidden / V);
    return launch_pdl(gather_rows_kernel<T, V>, dim3(row_blocks(n_tokens, threads, 6 * kRowThreads)), dim3(threads), 0,
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
