// Products of sorted rows with their experts' matrices on the tensor cores.
//
//   y[r] = W[e(r)] x[r]                              (si_moe_matmul)
//   gx[r] = W[e(r)]^T gy[r]                          (the same, matrices by columns)
//   gW[e] = sum of gy[r] x[r]^T over e's rows        (si_moe_matmul_grad_w)
//   h = silu(G x) * (U x), g and u kept in 8 bits    (si_moe_gateup)
//
// bf16 or fp16 operands, fp32 sums in tensor memory (tcgen05.mma kind::f16), rounded
// once. The experts' rows follow one another without padding: expert e has rows
// offsets[e] .. offsets[e + 1]. Three forms of one kernel:
//  - kGmTokens: 128 rows of an expert on the lanes of tensor memory, 256 of its
//    features as the N operand;
//  - kGmFew: 128 features on the lanes, NT rows as the N operand, where an expert has
//    few rows: the matrices then pass through the tensor cores once;
//  - kGmGrad: 128 x 256 of an expert's gradient, summed over its rows.
// An operand whose summed index is contiguous in memory lies in shared memory row
// by row (K-major), the others as they are, 64 values of 64 summed indices a piece
// (MN-major): nothing is transposed on the way.
//
// A tile of rows may reach behind its expert's: the rows of the next expert that it
// then holds give rows of tensor memory that are not written. In kGmGrad they would
// enter the sums, so the MMA warp clears them in shared memory.
//
// A block: a thread of warp 0 keeps operand A of a ring of stages (64 summed
// indices) coming by tensor TMA, one of the last warp operand B, warp 1 issues the
// MMAs, the others read the accumulators and write. Blocks are persistent; two accumulators,
// so that the MMAs of a tile run beside the epilogue of the one before.
#include <algorithm>

#include "host.hpp"
#include "mxint8.cuh"
#include "sort.cuh"
#include "tma.cuh"

namespace si {

constexpr int kGmK = 64;              // summed indices of a stage: 128 bytes
constexpr int kGmPiece = 8192;        // 64 x 64 values of an MN-major operand
constexpr int kGmGroups = kSortMaxExperts + 2;

enum GmOp { kGmTokens, kGmFew, kGmGrad };
enum GmOut { kGmBf16, kGmF16, kGmF32 };
template <int OUT> constexpr int kGmSize = OUT == kGmF32 ? 4 : 2;

template <int OP, int NT, bool SWIGLU> struct GmCfg {
  static constexpr int MA = OP == kGmFew && SWIGLU ? 2 : 1;   // 128-row A tiles: gate and up
  static constexpr int kN = OP == kGmFew ? NT : 256;
  static constexpr int kEpiWarps = OP == kGmFew ? 4 : 8;
  static constexpr int kThreads = 32 * (3 + kEpiWarps);
  static constexpr int kABytes = MA * 128 * 128, kBBytes = kN * 128, kStage = kABytes + kBBytes;
  static constexpr int kList = OP == kGmGrad ? 0 : (kGmGroups + 1) * 8;
  static constexpr int kFit = (227 * 1024 - kList - 1536) / kStage;
  static constexpr int kStages = kFit < 12 ? kFit : 12;
  static constexpr int kAccCols = MA * kN;       // of one accumulator; two of them
  static constexpr int kCols = 2 * kAccCols <= 32 ? 32 : 2 * kAccCols <= 64 ? 64 : 2 * kAccCols <= 128 ? 128 : 2 * kAccCols <= 256 ? 256 : 512;
  static_assert(2 * kAccCols <= 512, "tensor memory has 512 columns");
  static constexpr int kBars = 2 * kStages + 5;
  static_assert(8 * kBars + 4 <= 512, "barriers");
  static constexpr int kSmem = kStages * kStage + 512 + kList + 1024;
};

struct GmParams {
  CUtensorMap a, b;
  const int32_t *offsets;
  int n_experts;
  int rows;              // sorted rows
  int n, k;              // features (of y; rows of gW) and summed columns (of x; columns of gW)
  int n_rt, n_ct;        // tiles along n; kGmGrad: along k
  void *out;
  int64_t ld, mat;       // distances of rows; kGmGrad: of matrices, in values
  int wide, codes_wide;  // rows of `out` and blocks of codes on 32-byte boundaries
  uint8_t *codes, *scales;   // SWIGLU: [rows][2 n], [rows][2 mi_blocks(n)]
  uint32_t fmt;          // input type in the instruction descriptor
  uint32_t *status;
};

// ---- tiles -------------------------------------------------------------------

// Sorted rows in groups: 0 the rows before offsets[0], 1 + e expert e's, n_experts + 1
// the rows behind the last; the first and the last are written as zeros. Bounds
// outside the rows are moved inside, and a bound below an earlier one to that one.
struct GmList {
  int row[kGmGroups + 1], tile[kGmGroups + 1];
};
struct GmTile {
  int e, row0, count;    // expert (-1: zeros), first row, rows
  int rt, ct;
};

// The list, by all threads of the block.
template <int M> SI_DEV void gm_list(const GmParams &p, GmList &l) {
  const int E = p.n_experts;
  for (int i = threadIdx.x; i <= E; i += blockDim.x) l.tile[i] = min(max(__ldcg(p.offsets + i), 0), p.rows);
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int most = 0;
    for (int i0 = 0; i0 <= E; i0 += 32) {        // running maximum of the bounds
      int v = i0 + lane <= E ? l.tile[i0 + lane] : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v = max(v, o);
      }
      v = max(v, most);
      most = __shfl_sync(0xffffffffu, v, 31);
      if (i0 + lane <= E) l.row[i0 + lane + 1] = v;
    }
    if (lane == 0) {
      l.row[0] = 0;
      l.row[E + 2] = p.rows;
    }
    __syncwarp();
    int at = 0;
    for (int i0 = 0; i0 < E + 2; i0 += 32) {
      const int i = i0 + lane;
      const int own = i < E + 2 ? (l.row[i + 1] - l.row[i] + M - 1) / M * p.n_rt : 0;
      int v = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
      }
      if (i < E + 2) l.tile[i] = at + v - own;
      at += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) l.tile[E + 2] = at;
  }
  __syncthreads();
}
// Tile w: the tiles of a group's rows lie side by side for the same features.
template <int M> SI_DEV GmTile gm_tile(const GmParams &p, const GmList &l, int w) {
  int lo = 0, hi = p.n_experts + 1;              // the last group whose first tile is at most w
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.tile[mid] <= w) lo = mid;
    else hi = mid - 1;
  }
  const int r0 = l.row[lo], r1 = l.row[lo + 1], mts = (r1 - r0 + M - 1) / M, i = w - l.tile[lo];
  GmTile t;
  t.rt = i / mts;
  t.ct = 0;
  t.row0 = r0 + (i - t.rt * mts) * M;
  t.count = min(M, r1 - t.row0);
  t.e = lo <= p.n_experts ? lo - 1 : -1;
  return t;
}
SI_DEV GmTile gm_tile_grad(const GmParams &p, int w) {
  GmTile t;
  t.ct = w % p.n_ct;
  const int r = w / p.n_ct;
  t.rt = r % p.n_rt;
  t.e = r / p.n_rt;
  const int r0 = min(max(__ldcg(p.offsets + t.e), 0), p.rows), r1 = min(max(__ldcg(p.offsets + t.e + 1), 0), p.rows);
  t.row0 = r0;
  t.count = max(r1 - r0, 0);
  return t;
}
// Stages of a tile.
template <int OP> SI_DEV int gm_steps(const GmParams &p, const GmTile &t) {
  return OP == kGmGrad ? (t.count + kGmK - 1) / kGmK : t.e < 0 ? 0 : (p.k + kGmK - 1) / kGmK;
}

// ---- tensor core -----------------------------------------------------------------

// Shared-memory matrix descriptors: 128-byte swizzle (layout 2), version 1; 8-row
// groups (8 summed indices, MN-major) 1024 bytes apart, and MN-major the next 64
// values kGmPiece bytes on. The high word is the same for both.
constexpr uint32_t kGmDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
template <bool MN> SI_DEV uint32_t gm_desc_lo(uint32_t addr) {
  return (addr >> 4) | ((MN ? kGmPiece >> 4 : 1u) << 16);
}
template <bool MN> constexpr uint32_t kGmK16 = (MN ? 16 * 128 : 32) / 16;   // 16 summed indices on
SI_DEV void gm_mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kGmDescHi)
      : "memory");
}

// ---- epilogues ---------------------------------------------------------------

template <int OUT> SI_DEV uint32_t gm_pack(uint32_t lo, uint32_t hi) {
  uint32_t w;
  if constexpr (OUT == kGmBf16)
    asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(w) : "f"(__uint_as_float(lo)), "f"(__uint_as_float(hi)));
  else
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(w) : "f"(__uint_as_float(lo)), "f"(__uint_as_float(hi)));
  return w;
}
// `bytes` (a multiple of 16, at most 4 N) of w to p, 32 at a time where rows allow it.
template <int N> SI_DEV void gm_store(uint8_t *p, const uint32_t *w, int bytes, bool wide) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    if (4 * i >= bytes) break;
    if (wide && 4 * i + 32 <= bytes) {
      st_global32(p + 4 * i, w + i);
    } else {
      *reinterpret_cast<uint4 *>(p + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
      if (4 * i + 32 <= bytes)
        *reinterpret_cast<uint4 *>(p + 4 * i + 16) = make_uint4(w[i + 4], w[i + 5], w[i + 6], w[i + 7]);
    }
  }
}

// 128 columns of the accumulator to this lane's row: `cols` of them are inside it.
template <int OUT, typename Release>
SI_DEV void gm_write_row(uint8_t *out, int cols, bool wide, bool valid, bool zero, uint32_t acc, Release release) {
  constexpr int kWords = 8 * kGmSize<OUT>;       // of 32 values
#pragma unroll
  for (int c = 0; c < 128; c += 32) {
    uint32_t r[32], w[kWords];
    if (zero) {
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = 0;
    } else {
      if (c < cols) {
        tmem_ld32(acc + c, r);
        tmem_wait_ld();
      }
      if (c == 96) release();
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (OUT == kGmF32) w[i] = r[i];
      else w[i] = gm_pack<OUT>(r[2 * i], r[2 * i + 1]);
    }
    if (valid && c < cols) gm_store<kWords>(out + c * kGmSize<OUT>, w, min(32, cols - c) * kGmSize<OUT>, wide);
  }
}

// silu(g) u; g below -87 (|silu(g)| < 2^-119) gives 0: the reciprocal is below the
// normal range. ex2 and rcp of the hardware, each within 2 units in the last place.
SI_DEV float gm_silu_mul(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return g * r * u;
}

// 32 values to their MXINT8 block: 8 words of codes, the scale.
SI_DEV uint32_t gm_encode32(const uint32_t *v, uint32_t w[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) top = max(top, v[i] & 0x7FFFFFFFu);
  const uint32_t s = mi_scale_of(top);
  const float up = mi_inv_scale(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = mi_code(__uint_as_float(v[4 * i + j]) * up);
    w[i] = s == 255u ? 0u : mi_pack4(c[0], c[1], c[2], c[3]);
  }
  return s;
}
// `bytes` (a multiple of 8, at most 32) of codes.
SI_DEV void gm_store_codes(uint8_t *p, const uint32_t w[8], int bytes, bool wide) {
  if (wide && bytes == 32) {
    st_global32(p, w);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (8 * i < bytes) *reinterpret_cast<uint2 *>(p + 8 * i) = make_uint2(w[2 * i], w[2 * i + 1]);
}

// 64 features (from f0) of this lane's row: h, and the blocks of g and u.
template <int OUT, typename Release>
SI_DEV void gm_write_swiglu_row(const GmParams &p, int f0, int64_t row, bool valid, bool zero, uint32_t acc_g,
                                uint32_t acc_u, Release release) {
  const int64_t blocks = mi_blocks(p.n);
#pragma unroll
  for (int c = 0; c < 64; c += 32) {
    const int f = f0 + c, left = min(32, p.n - f);
    uint32_t g[32], u[32], w[16];
    if (left > 0 && !zero) {
      tmem_ld32(acc_g + c, g);
      tmem_ld32(acc_u + c, u);
      tmem_wait_ld();
    }
    if (c == 32 && !zero) release();
    if (left <= 0) continue;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (zero || i >= left) g[i] = u[i] = 0;    // behind the last feature
#pragma unroll
    for (int i = 0; i < 16; ++i)
      w[i] = gm_pack<OUT>(__float_as_uint(gm_silu_mul(__uint_as_float(g[2 * i]), __uint_as_float(u[2 * i]))),
                          __float_as_uint(gm_silu_mul(__uint_as_float(g[2 * i + 1]), __uint_as_float(u[2 * i + 1]))));
    if (valid) gm_store<16>(static_cast<uint8_t *>(p.out) + (row * p.ld + f) * 2, w, 2 * left, p.wide);
    if (!p.codes) continue;
    uint32_t q[8];
    uint8_t *codes = p.codes + row * 2 * p.n + f, *scales = p.scales + row * 2 * blocks + (f >> 5);
    const uint32_t sg = gm_encode32(g, q);
    if (valid) gm_store_codes(codes, q, left, p.codes_wide);
    const uint32_t su = gm_encode32(u, q);
    if (valid) {
      gm_store_codes(codes + p.n, q, left, p.codes_wide);
      scales[0] = static_cast<uint8_t>(sg);
      scales[blocks] = static_cast<uint8_t>(su);
    }
  }
}

template <int OUT> SI_DEV void gm_store1(void *out, int64_t at, float v) {
  if constexpr (OUT == kGmBf16) static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
  else if constexpr (OUT == kGmF16) static_cast<__half *>(out)[at] = __float2half_rn(v);
  else static_cast<float *>(out)[at] = v;
}
// This lane's feature f of `count` rows from row0, the accumulator's columns.
template <int OUT, int NT>
SI_DEV void gm_write_few(const GmParams &p, int f, int64_t row0, int count, bool zero, uint32_t acc) {
#pragma unroll
  for (int j0 = 0; j0 < NT; j0 += 16) {
    if (j0 >= count) break;
    uint32_t r[16];
    if (!zero) {
      tmem_ld16(acc + j0, r);
      tmem_wait_ld();
    }
    if (f < p.n) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j0 + j < count) gm_store1<OUT>(p.out, (row0 + j0 + j) * p.ld + f, zero ? 0.f : __uint_as_float(r[j]));
    }
  }
}
// The same of h, g and u: the warp's 32 lanes are one block of every row.
template <int OUT, int NT>
SI_DEV void gm_write_swiglu_few(const GmParams &p, int f, int64_t row0, int count, bool zero, uint32_t acc_g,
                                uint32_t acc_u, int lane) {
  const int64_t blocks = mi_blocks(p.n);
  const bool in = f < p.n;
  if (f - lane >= p.n) return;                   // the whole warp
#pragma unroll 1
  for (int j0 = 0; j0 < NT; j0 += 16) {
    if (j0 >= count) break;
    uint32_t g[16], u[16];
    if (!zero) {
      tmem_ld16(acc_g + j0, g);
      tmem_ld16(acc_u + j0, u);
      tmem_wait_ld();
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (j0 + j >= count) break;
      if (zero || !in) g[j] = u[j] = 0;
      const int64_t row = row0 + j0 + j;
      if (in) gm_store1<OUT>(p.out, row * p.ld + f, gm_silu_mul(__uint_as_float(g[j]), __uint_as_float(u[j])));
      if (!p.codes) continue;
      const uint32_t sg = mi_scale_of(__reduce_max_sync(0xffffffffu, g[j] & 0x7FFFFFFFu));
      const uint32_t su = mi_scale_of(__reduce_max_sync(0xffffffffu, u[j] & 0x7FFFFFFFu));
      const uint32_t cg = sg == 255u ? 0u : mi_code(__uint_as_float(g[j]) * mi_inv_scale(sg));
      const uint32_t cu = su == 255u ? 0u : mi_code(__uint_as_float(u[j]) * mi_inv_scale(su));
      uint8_t *codes = p.codes + row * 2 * p.n + f, *scales = p.scales + row * 2 * blocks + (f >> 5);
      if (in) {
        codes[0] = static_cast<uint8_t>(cg);
        codes[p.n] = static_cast<uint8_t>(cu);
      }
      if (lane == 0) {
        scales[0] = static_cast<uint8_t>(sg);
        scales[blocks] = static_cast<uint8_t>(su);
      }
    }
  }
}

// ---- the kernel ----------------------------------------------------------------

// WMN: the matrices lie by columns (features contiguous).
template <int OP, bool WMN, int NT, bool SWIGLU, int OUT>
__global__ void __launch_bounds__(GmCfg<OP, NT, SWIGLU>::kThreads, 1)
    moe_mm_kernel(const __grid_constant__ GmParams p) {
  using C = GmCfg<OP, NT, SWIGLU>;
  constexpr int S = C::kStages, M = OP == kGmFew ? NT : 128;
  constexpr bool kAMn = OP == kGmGrad || (OP == kGmFew && WMN), kBMn = OP == kGmGrad || (OP == kGmTokens && WMN);
  static_assert(!(SWIGLU && (WMN || OP == kGmGrad || OUT == kGmF32)), "gate and up lie row by row");
  extern __shared__ uint8_t gm_smem[];
  uint8_t *base = gm_smem + ((1024u - (smem_addr(gm_smem) & 1023u)) & 1023u);
  uint64_t *full = reinterpret_cast<uint64_t *>(base + S * C::kStage);
  uint64_t *empty = full + S, *acc_full = empty + S, *acc_empty = acc_full + 2, *drain = acc_empty + 2;
  uint32_t *s_taddr = reinterpret_cast<uint32_t *>(drain + 1);
  GmList &list = *reinterpret_cast<GmList *>(base + S * C::kStage + 512);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(full + i, 2);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, C::kEpiWarps);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  grid_dep_wait();
  if (warp == 1) {
    // before the next kernel may start: its blocks take tensor memory too
    tmem_alloc(s_taddr, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  if constexpr (OP != kGmGrad) gm_list<M>(p, list);
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *s_taddr, 0);
  const int total = OP == kGmGrad ? p.n_experts * p.n_rt * p.n_ct : list.tile[p.n_experts + 2];
  const int step = gridDim.x;
  auto tile = [&](int w) {
    if constexpr (OP == kGmGrad) return gm_tile_grad(p, w);
    else return gm_tile<M>(p, list, w);
  };

  if (warp == 0 || warp == 2 + C::kEpiWarps) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int w = blockIdx.x; ok && w < total; w += step) {
        const GmTile t = tile(w);
        const int nk = gm_steps<OP>(p, t);
        for (int ks = 0; ks < nk; ++ks, ++it) {
          const int s = it % S;
          if (!mbar_wait_bounded(empty + s, ((it / S) & 1) ^ 1, p.status)) {
            ok = false;
            break;
          }
          uint8_t *st = base + s * C::kStage;
          const int c = ks * kGmK;
          if (warp == 0) {
            mbar_arrive_expect_tx(full + s, C::kABytes);
            if constexpr (OP == kGmTokens) {
              tma_load3(st, &p.a, c, t.row0, 0, full + s);
            } else if constexpr (OP == kGmGrad) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                tma_load3(st + i * kGmPiece, &p.a, t.rt * 128 + i * 64, t.row0 + c, 0, full + s);
            } else if constexpr (WMN) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                tma_load3(st + i * kGmPiece, &p.a, t.rt * 128 + i * 64, c, t.e, full + s);
            } else {
#pragma unroll
              for (int i = 0; i < C::MA; ++i)
                tma_load3(st + i * 128 * 128, &p.a, c, t.rt * 128 + i * p.n, t.e, full + s);
            }
          } else {
            st += C::kABytes;
            mbar_arrive_expect_tx(full + s, C::kBBytes);
            if constexpr (OP == kGmFew) {
              tma_load3(st, &p.b, c, t.row0, 0, full + s);
            } else if constexpr (OP == kGmGrad) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                tma_load3(st + i * kGmPiece, &p.b, t.ct * 256 + i * 64, t.row0 + c, 0, full + s);
            } else if constexpr (WMN) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                tma_load3(st + i * kGmPiece, &p.b, t.rt * 256 + i * 64, c, t.e, full + s);
            } else if constexpr (SWIGLU) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                tma_load3(st + i * 128 * 128, &p.b, c, t.rt * 128 + i * p.n, t.e, full + s);
            } else {
              tma_load3(st, &p.b, c, t.rt * 256, t.e, full + s);
            }
          }
        }
      }
      if (!ok) {   // copies in flight land before the block's memory goes
        const uint32_t n = it < static_cast<uint32_t>(S) ? it : S;
        for (uint32_t i = it - n; i < it; ++i) mbar_wait_bounded(full + i % S, (i / S) & 1, p.status);
      }
    }
  } else if (warp == 1) {
    // the warp walks over the stages together, the leader alone waits and issues
    const bool leader = elect_lane();
    const uint32_t smem0 = smem_addr(base);
    uint32_t n = 0;                  // accumulators taken so far
    int s = 0;                       // stage and its parity
    uint32_t parity = 0;
    bool ok = true;
    for (int w = blockIdx.x; w < total; w += step) {
      const GmTile t = tile(w);
      const int nk = gm_steps<OP>(p, t);
      if (nk == 0) continue;         // zeros: no accumulator
      const uint32_t u = n & 1, d = tmem + u * C::kAccCols;
      if (leader && ok) ok = mbar_wait_bounded(acc_empty + u, ((n >> 1) & 1) ^ 1, p.status);
      const int cols = OP == kGmFew ? (t.count + 15) & ~15 : 256;
      const uint32_t idesc = (1u << 4) | p.fmt | (kAMn ? 1u << 15 : 0u) | (kBMn ? 1u << 16 : 0u) |
                             (static_cast<uint32_t>(cols >> 3) << 17) | ((128u >> 4) << 24);
      const int last = OP == kGmGrad ? t.count : p.k;   // summed indices
      for (int ks = 0; ks < nk; ++ks) {
        const int left = min(kGmK, last - ks * kGmK), n16 = (left + 15) >> 4;
        const uint32_t st = smem0 + s * C::kStage;
        if constexpr (OP == kGmGrad) {
          if (left & 15) {           // the rows behind the expert's in the last 16: cleared
            ok = __all_sync(0xffffffffu, ok || !leader) != 0;
            if (ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(full + s, parity, p.status)) != 0;
            uint8_t *q = base + s * C::kStage;
            for (int r = left; ok && r < n16 * 16; ++r)
              for (int i = lane; i < C::kStage / kGmPiece * 8; i += 32)
                *reinterpret_cast<uint4 *>(q + (i >> 3) * kGmPiece + r * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_async_smem();
            __syncwarp();
          }
        }
        if (leader && ok) ok = mbar_wait_bounded(full + s, parity, p.status);
        if (leader && ok) {
          tc_fence_after();
          const uint32_t la = gm_desc_lo<kAMn>(st), lb = gm_desc_lo<kBMn>(st + C::kABytes);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i >= n16) break;
#pragma unroll
            for (int a = 0; a < C::MA; ++a)
              gm_mma(d + a * C::kN, la + a * (128 * 128 / 16) + i * kGmK16<kAMn>, lb + i * kGmK16<kBMn>, idesc,
                     i > 0 || ks > 0);
          }
          umma_commit(empty + s);
        }
        if (++s == S) {
          s = 0;
          parity ^= 1;
        }
      }
      if (leader && ok) umma_commit(acc_full + u);
      ++n;
    }
    if (leader && !ok) {   // MMAs in flight end before the tensor memory goes
      umma_commit(drain);
      mbar_wait_bounded(drain, 0, p.status);
    }
    __syncwarp();
  } else {
    const int q = warp & 3, part = (warp - 2) >> 2;   // the 32 lanes of tensor memory this warp may read
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
    uint32_t n = 0;
    for (int w = blockIdx.x; w < total; w += step) {
      const GmTile t = tile(w);
      const bool zero = gm_steps<OP>(p, t) == 0;
      uint32_t acc = 0;
      if (!zero) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(acc_full + (n & 1), (n >> 1) & 1, p.status))) break;
        tc_fence_after();
        acc = lanes + (n & 1) * C::kAccCols;
      }
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + (n & 1));
      };
      if constexpr (OP == kGmFew) {
        const int f = t.rt * 128 + q * 32 + lane;
        if constexpr (SWIGLU) gm_write_swiglu_few<OUT, NT>(p, f, t.row0, t.count, zero, acc, acc + NT, lane);
        else gm_write_few<OUT, NT>(p, f, t.row0, t.count, zero, acc);
        if (!zero) release();
      } else if constexpr (SWIGLU) {
        const int j = q * 32 + lane;
        gm_write_swiglu_row<OUT>(p, t.rt * 128 + part * 64, static_cast<int64_t>(t.row0) + j, j < t.count, zero,
                                 acc + part * 64, acc + 128 + part * 64, release);
      } else {
        const int j = q * 32 + lane;
        int64_t row;
        int col, cols;
        bool valid;
        if constexpr (OP == kGmGrad) {
          row = t.rt * 128 + j;
          valid = row < p.n;
          col = t.ct * 256 + part * 128;
          cols = p.k - col;
        } else {
          row = static_cast<int64_t>(t.row0) + j;
          valid = j < t.count;
          col = t.rt * 256 + part * 128;
          cols = p.n - col;
        }
        uint8_t *out = static_cast<uint8_t *>(p.out) +
                       ((OP == kGmGrad ? t.e * p.mat : 0) + row * p.ld + col) * kGmSize<OUT>;
        gm_write_row<OUT>(out, min(cols, 128), p.wide, valid, zero, acc + part * 128, release);
      }
      if (!zero) ++n;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, C::kCols);
  }
}

// ---- host ------------------------------------------------------------------

// 16-bit values [mats][rows][cols], boxes of box_rows rows x 64 values in the 128-byte
// swizzle; what lies outside reads as zero.
static bool gm_map(CUtensorMap *m, const void *v, bool bf16, int64_t mats, int64_t rows, int64_t cols, int64_t ld,
                   int64_t mat, int box_rows) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(mats)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * 2), static_cast<cuuint64_t>(mats > 1 ? mat * 2 : ld * 2)};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  return encode_map(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, v, 3, dims, strides,
                    box);
}

template <int OP, bool WMN, int NT, bool SWIGLU, int OUT>
static cudaError_t gm_launch(const GmParams &p, int64_t most, cudaStream_t s) {
  using C = GmCfg<OP, NT, SWIGLU>;
  const cudaError_t e = allow_smem(moe_mm_kernel<OP, WMN, NT, SWIGLU, OUT>, C::kSmem);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(most, sm_count()));
  return launch_pdl(moe_mm_kernel<OP, WMN, NT, SWIGLU, OUT>, dim3(grid), dim3(C::kThreads), C::kSmem, s, p);
}
template <typename F> static cudaError_t gm_by_out(si_dtype t, F f) {
  using std::integral_constant;
  return t == SI_BF16  ? f(integral_constant<int, kGmBf16>{})
         : t == SI_F16 ? f(integral_constant<int, kGmF16>{})
                       : f(integral_constant<int, kGmF32>{});
}

static bool gm_type(si_dtype t) { return t == SI_BF16 || t == SI_F16; }
static uint32_t gm_fmt(si_dtype t) { return t == SI_BF16 ? (1u << 7) | (1u << 10) : 0u; }
static bool gm_width(int64_t n) { return n >= 8 && n % 8 == 0 && n <= (int64_t(1) << 20); }
static bool gm_rows(int64_t rows, int n_experts) {
  return rows >= 0 && rows <= 0x7FFFFFFF - 256 && n_experts >= 1 && n_experts <= kSortMaxExperts;
}
// Rows at 16-byte boundaries, at least `cols` values apart.
static bool gm_ld(int64_t ld, int64_t cols, int size) {
  return ld >= cols && ld * size % 16 == 0 && ld <= (int64_t(1) << 36);
}
static bool gm_wide(const void *p, int64_t ld, int size) {
  return ld * size % 32 == 0 && (reinterpret_cast<uintptr_t>(p) & 31u) == 0;
}

// Rows of an expert on average up to which its features go on the lanes.
static bool gm_few(int64_t rows, int n_experts) { return rows <= 16 * static_cast<int64_t>(n_experts); }

// Tiles of the sorted rows in M rows each, at most: 0 if they pass 2^30.
static int64_t gm_tiles(int64_t rows, int n_experts, int m, int64_t n_rt) {
  const int64_t t = (rows / m + std::min<int64_t>(n_experts + 2, rows)) * n_rt;
  return t <= (int64_t(1) << 30) ? t : 0;
}

}  // namespace si

using namespace si;

extern "C" size_t si_moe_matmul_workspace_bytes(void) { return sizeof(WsHeader); }

extern "C" si_status si_moe_matmul(const void *x, si_dtype type, int64_t rows, int64_t ldx, const void *w,
                                   int n_experts, int64_t n, int64_t k, int64_t ldw, int64_t matw, int by_columns,
                                   const int32_t *offsets, void *out, si_dtype out_type, int64_t ldo, void *workspace,
                                   size_t workspace_bytes, void *stream) {
  if (!gm_rows(rows, n_experts) || !gm_width(n) || !gm_width(k)) return SI_ERR_INVALID_ARG;
  if (!gm_type(type) || (out_type != SI_F32 && out_type != type)) return SI_ERR_UNSUPPORTED;
  const int size = out_type == SI_F32 ? 4 : 2;
  if (rows == 0) return SI_OK;
  if (!x || !w || !offsets || !out || !aligned16(x) || !aligned16(w) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(offsets) & 3u) || !gm_ld(ldx, k, 2) || !gm_ld(ldo, n, size) ||
      !gm_ld(ldw, by_columns ? n : k, 2) || (n_experts > 1 && !gm_ld(matw, ldw * (by_columns ? k : n) - (ldw - (by_columns ? n : k)), 2)))
    return SI_ERR_INVALID_ARG;
  if (workspace && (!aligned256(workspace) || workspace_bytes < sizeof(WsHeader))) return SI_ERR_WORKSPACE;
  const bool few = gm_few(rows, n_experts), cols = by_columns != 0, bf16 = type == SI_BF16;
  GmParams p{};
  p.n_rt = static_cast<int>(few ? (n + 127) / 128 : (n + 255) / 256);
  const int64_t most = gm_tiles(rows, n_experts, few ? 16 : 128, p.n_rt);
  if (!most) return SI_ERR_UNSUPPORTED;
  CUtensorMap &mx = few ? p.b : p.a, &mw = few ? p.a : p.b;
  if (!gm_map(&mx, x, bf16, 1, rows, k, ldx, 0, few ? 16 : 128) ||
      !gm_map(&mw, w, bf16, n_experts, cols ? k : n, cols ? n : k, ldw, matw, cols ? 64 : few ? 128 : 256))
    return SI_ERR_CUDA;
  p.offsets = offsets;
  p.n_experts = n_experts;
  p.rows = static_cast<int>(rows);
  p.n = static_cast<int>(n);
  p.k = static_cast<int>(k);
  p.out = out;
  p.ld = ldo;
  p.wide = gm_wide(out, ldo, size);
  p.fmt = gm_fmt(type);
  p.status = static_cast<uint32_t *>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(gm_by_out(out_type, [&](auto o) {
    constexpr int O = decltype(o)::value;
    if (few)
      return cols ? gm_launch<kGmFew, true, 16, false, O>(p, most, s) : gm_launch<kGmFew, false, 16, false, O>(p, most, s);
    return cols ? gm_launch<kGmTokens, true, 0, false, O>(p, most, s)
                : gm_launch<kGmTokens, false, 0, false, O>(p, most, s);
  }));
}

extern "C" si_status si_moe_matmul_grad_w(const void *gy, int64_t ldg, const void *x, int64_t ldx, si_dtype type,
                                          int64_t rows, int n_experts, int64_t n, int64_t k, const int32_t *offsets,
                                          void *gw, si_dtype gw_type, void *workspace, size_t workspace_bytes,
                                          void *stream) {
  if (!gm_rows(rows, n_experts) || !gm_width(n) || !gm_width(k)) return SI_ERR_INVALID_ARG;
  if (!gm_type(type) || (gw_type != SI_F32 && gw_type != type)) return SI_ERR_UNSUPPORTED;
  const int size = gw_type == SI_F32 ? 4 : 2;
  if (!gw || !aligned16(gw)) return SI_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) return cuda_status(cudaMemsetAsync(gw, 0, static_cast<size_t>(n_experts) * n * k * size, s));
  if (!gy || !x || !offsets || !aligned16(gy) || !aligned16(x) || (reinterpret_cast<uintptr_t>(offsets) & 3u) ||
      !gm_ld(ldg, n, 2) || !gm_ld(ldx, k, 2))
    return SI_ERR_INVALID_ARG;
  if (workspace && (!aligned256(workspace) || workspace_bytes < sizeof(WsHeader))) return SI_ERR_WORKSPACE;
  GmParams p{};
  p.n_rt = static_cast<int>((n + 127) / 128);
  p.n_ct = static_cast<int>((k + 255) / 256);
  const int64_t most = static_cast<int64_t>(n_experts) * p.n_rt * p.n_ct;
  if (most > (int64_t(1) << 30)) return SI_ERR_UNSUPPORTED;
  const bool bf16 = type == SI_BF16;
  if (!gm_map(&p.a, gy, bf16, 1, rows, n, ldg, 0, kGmK) || !gm_map(&p.b, x, bf16, 1, rows, k, ldx, 0, kGmK))
    return SI_ERR_CUDA;
  p.offsets = offsets;
  p.n_experts = n_experts;
  p.rows = static_cast<int>(rows);
  p.n = static_cast<int>(n);
  p.k = static_cast<int>(k);
  p.out = gw;
  p.ld = k;
  p.mat = n * k;
  p.wide = gm_wide(gw, k, size);
  p.fmt = gm_fmt(type);
  p.status = static_cast<uint32_t *>(workspace);
  return cuda_status(
      gm_by_out(gw_type, [&](auto o) { return gm_launch<kGmGrad, false, 0, false, decltype(o)::value>(p, most, s); }));
}

extern "C" si_status si_moe_gateup(const void *x, si_dtype type, int64_t rows, int64_t ldx, const void *gate_up,
                                   int n_experts, int64_t inter, int64_t hidden, const int32_t *offsets, void *h,
                                   void *codes, void *scales, void *workspace, size_t workspace_bytes, void *stream) {
  if (!gm_rows(rows, n_experts) || !gm_width(inter) || !gm_width(hidden)) return SI_ERR_INVALID_ARG;
  if (!gm_type(type)) return SI_ERR_UNSUPPORTED;
  if (rows == 0) return SI_OK;
  if (!x || !gate_up || !offsets || !h || !aligned16(x) || !aligned16(gate_up) || !aligned16(h) || !aligned16(codes) ||
      (reinterpret_cast<uintptr_t>(offsets) & 3u) || !gm_ld(ldx, hidden, 2) || !codes != !scales)
    return SI_ERR_INVALID_ARG;
  if (workspace && (!aligned256(workspace) || workspace_bytes < sizeof(WsHeader))) return SI_ERR_WORKSPACE;
  const bool few = gm_few(rows, n_experts), bf16 = type == SI_BF16;
  GmParams p{};
  p.n_rt = static_cast<int>((inter + 127) / 128);
  const int64_t most = gm_tiles(rows, n_experts, few ? 16 : 128, p.n_rt);
  if (!most) return SI_ERR_UNSUPPORTED;
  CUtensorMap &mx = few ? p.b : p.a, &mw = few ? p.a : p.b;
  if (!gm_map(&mx, x, bf16, 1, rows, hidden, ldx, 0, few ? 16 : 128) ||
      !gm_map(&mw, gate_up, bf16, n_experts, 2 * inter, hidden, hidden, 2 * inter * hidden, 128))
    return SI_ERR_CUDA;
  p.offsets = offsets;
  p.n_experts = n_experts;
  p.rows = static_cast<int>(rows);
  p.n = static_cast<int>(inter);
  p.k = static_cast<int>(hidden);
  p.out = h;
  p.ld = inter;
  p.wide = gm_wide(h, inter, 2);
  p.codes_wide = gm_wide(codes, inter, 1);
  p.codes = static_cast<uint8_t *>(codes);
  p.scales = static_cast<uint8_t *>(scales);
  p.fmt = gm_fmt(type);
  p.status = static_cast<uint32_t *>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (type == SI_BF16)
    return cuda_status(few ? gm_launch<kGmFew, false, 16, true, kGmBf16>(p, most, s)
                           : gm_launch<kGmTokens, false, 0, true, kGmBf16>(p, most, s));
  return cuda_status(few ? gm_launch<kGmFew, false, 16, true, kGmF16>(p, most, s)
                         : gm_launch<kGmTokens, false, 0, true, kGmF16>(p, most, s));
}
