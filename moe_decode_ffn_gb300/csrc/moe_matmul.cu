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
//  - kGmWide: 256 features on the lanes of tensor memory, 128 in each of two neighbouring
//    SMs (cta_group::2), up to 256 rows of an expert as the N operand, half of them in
//    each SM: a tile's N is its own number of rows, to the next 32, so that ragged
//    experts cost no more than they hold, and every SM brings in half of each operand;
//  - kGmFew: the same in one SM with 16 rows, where an expert has few: a deep ring of
//    its matrix' pieces and nothing else;
//  - kGmGrad: 256 x 256 of an expert's gradient, summed over its rows, in two SMs.
// An operand whose summed index is contiguous in memory lies in shared memory row
// by row (K-major), the others as they are, 64 values of 64 summed indices a piece
// (MN-major): nothing is transposed on the way.
//
// A tile of rows may reach behind its expert's: the rows of the next expert that it
// then holds give columns of tensor memory that are not written. In kGmGrad they would
// enter the sums: an expert's rows behind its last whole 16 come into a buffer of their own,
// where a warp of each SM clears what is behind them while the other stages are on
// their way (cleared in the last stage, on the MMAs' way, they made 500 rows an expert 381 us
// instead of 290).
//
// A block: a thread of warp 0 keeps operand A of a ring of stages (64 summed
// indices) coming by tensor TMA, one of another warp operand B, warp 1 (of the first SM
// of a pair) issues the MMAs, the others read the accumulators and write. Blocks are
// persistent; two accumulators, so that the MMAs of a tile run beside the epilogue of
// the one before.
//
// What bounds it, on a GB300. Few rows: HBM (64 tokens, top-8 of 128 experts of 2048 x 768, of
// which about 108 have rows, 56.7 us, 6.0 TB/s; all 128 with 4 rows each 66 us, 6.1 TB/s). Where there are
// fewer tiles than SMs (one token, 96 tiles, 13.7 us) the way of a stage: of its 709 cycles (502 with
// matrices that lie in the L2) the MMA warp waits 54 % (37 %) for the copies, the rest goes to issuing four
// MMAs and their commit; the tensor pipe is active for 4.5 %. Many rows: the tensor cores
// (16384 rows over 8 experts of 4096 x 4096 308 to 340 us, 1.6 to 1.8 PFLOP/s, by the clock that
// the power limit leaves). Between them, 256 ragged rows an expert over 128 experts: the
// loads, 188 us for 1536 x 2048 (5.0 TB/s from HBM, 10.8 TB/s from the L2; the MMA warp waits for
// a stage for 47 % of the time, tensor pipe active 54 %); the gradients 216 to 221 us (805 MB
// written, 4.8 TB/s with what is read; waits for stages 18 %, for last rows 11 %, for accumulators 8 %), in fp32
// 314 us (1.61 GB written, 5.9 TB/s).
#include <algorithm>
#include <atomic>

#include "host.hpp"
#include "mxint8.cuh"
#include "sort.cuh"
#include "tma.cuh"

namespace si {

constexpr int kGmK = 64;              // summed indices of a stage: 128 bytes
constexpr int kGmPiece = 8192;        // 64 x 64 values of an MN-major operand
constexpr int kGmTail = 2 * 16 * 128;  // 128 values of 16 summed indices
constexpr int kGmGroups = kSortMaxExperts + 2;

enum GmOp { kGmWide, kGmFew, kGmGrad };
// What becomes of the sums: written, SwiGLU of gate and up (kGmSwigluParts: summed in parts, see
// kGmChunk), the gradients of SwiGLU.
enum GmMode { kGmPlain, kGmSwiglu, kGmSwigluParts, kGmSwigluBack };
template <int MODE> constexpr bool kGmForward = MODE == kGmSwiglu || MODE == kGmSwigluParts;
enum GmOut { kGmBf16, kGmF16, kGmF32 };
template <int OUT> constexpr int kGmSize = OUT == kGmF32 ? 4 : 2;

template <int OP, int MODE, int OUT> struct GmCfg {
  static constexpr int CG = OP == kGmFew ? 1 : 2;                    // SMs of a tile
  static constexpr int MA = OP == kGmFew && kGmForward<MODE> ? 2 : 1;   // 128-row A tiles: gate and up
  static constexpr int kN = OP == kGmFew ? 16 : 256;                 // columns of an accumulator
  // fp32 outputs are summed up in registers: 64 columns a warp instead of 128; and what SwiGLU
  // asks for goes faster with more warps to take turns
  static constexpr int kEpiWarps = OP == kGmFew ? 4 : OUT == kGmF32 || MODE != kGmPlain ? 16 : 8;
  static constexpr int kBWarp = 2 + kEpiWarps, kTailWarp = OP == kGmGrad ? kBWarp + 1 : -1;
  static constexpr int kThreads = 32 * (kBWarp + 1 + (OP == kGmGrad));
  static constexpr int kABytes = MA * 128 * 128, kBBytes = kN / CG * 128, kStage = kABytes + kBBytes;
  static constexpr int kList = OP == kGmGrad ? 0 : (kGmGroups + 1) * 8;
  static constexpr int kBox = OP == kGmGrad ? 2048 : 1024;           // a warp's rows on their way out
  static constexpr int kOut = kEpiWarps * kBox;
  // the last rows of an expert, of both operands, twice
  static constexpr int kTail = OP == kGmGrad ? 2 * 2 * kGmTail : 0;
  static constexpr int kFit = (227 * 1024 - kList - kOut - kTail - 1536) / kStage;
  static constexpr int kStages = kFit < 12 ? kFit : 12;
  static constexpr int kAccCols = MA * kN;       // of one accumulator; two of them
  static constexpr int kCols = 2 * kAccCols <= 32 ? 32 : 2 * kAccCols <= 64 ? 64 : 512;
  static_assert(2 * kAccCols <= kCols, "tensor memory has 512 columns");
  static constexpr int kBars = 2 * kStages + 11;
  static_assert(8 * kBars + 4 <= 512, "barriers");
  static constexpr int kSmem = kStages * kStage + kTail + kOut + 512 + kList + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct GmParams {
  CUtensorMap a, b[4];   // b, kGmWide: by boxes of 32, 64, 96 and 128 rows
  CUtensorMap o, ta, tb; // kGmGrad: the gradient, boxes of 32 rows x 64 bytes; a and b by 16 rows
  const int32_t *offsets;
  int n_experts;
  int rows;              // sorted rows
  int n, k;              // features (of y; rows of gW) and summed columns (of x; columns of gW)
  int n_rt, n_ct;        // tiles along n; kGmGrad: along k
  int whole_a, whole_b;  // MN-major operands: whole pieces of 64 values, two in a box
  void *out;             // y; h; kGmSwigluBack: ggu
  int64_t ld;            // distance of its rows in values
  uint8_t *codes, *scales;   // kGmSwiglu[Back]: [rows][2 n], [rows][2 mi_blocks(n)]
  // kGmSwigluBack: row weights by pair, the pair of a row, c h, partial sums of gw [rows][parts]
  const float *c;
  const int32_t *order;
  void *wh;
  float *part;
  int parts;
  uint32_t fmt;          // input type in the instruction descriptor
  uint32_t *status;
};

// ---- tiles -------------------------------------------------------------------

// Sorted rows in groups: 0 the rows before offsets[0], 1 + e expert e's, n_experts + 1
// the rows behind the last; the first and the last are written as zeros. Bounds
// outside the rows are moved inside, and a bound below an earlier one to that one.
// Tiles are dealt out to the pairs of SMs in turn. (Dealt out by their cost, the largest
// first or large and small by turns, measured the same.)
struct GmList {
  int row[kGmGroups + 1], tile[kGmGroups + 1];   // first row and first tile of a group
};
struct GmTile {
  int e, row0, count;    // expert (-1: zeros), first row, rows
  int rt, ct;
};

// A group's rows in tiles: of 16, or kGmWide in as many even parts as parts of 256 would be,
// each to the next 32 rows.
template <int OP> SI_DEV int gm_parts(int rows) { return OP == kGmFew ? (rows + 15) >> 4 : (rows + 255) >> 8; }
template <int OP> SI_DEV int gm_per(int rows, int parts) {
  return OP == kGmFew ? 16 : min(256, ((rows + parts - 1) / parts + 31) & ~31);
}
SI_DEV int gm_scan_add(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// The list, by all threads of the block; of its first warp a lane has some neighbouring
// bounds and groups, so that one scan over the lanes does for each.
template <int OP> SI_DEV void gm_list(const GmParams &p, GmList &l) {
  const int E = p.n_experts;
  for (int i = threadIdx.x; i <= E; i += blockDim.x) l.row[i + 1] = min(max(__ldcg(p.offsets + i), 0), p.rows);
  if (threadIdx.x == 0) {
    l.row[0] = 0;
    l.row[E + 2] = p.rows;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, n = (E + 32) >> 5;   // of E + 1 bounds, then of E + 2 groups
    const int b0 = 1 + min(lane * n, E + 1), b1 = 1 + min((lane + 1) * n, E + 1);
    int most = 0;
    for (int i = b0; i < b1; ++i) most = max(most, l.row[i]);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {           // running maximum
      const int o = __shfl_up_sync(0xffffffffu, most, d);
      if (lane >= d) most = max(most, o);
    }
    most = __shfl_up_sync(0xffffffffu, most, 1);
    if (lane == 0) most = 0;
    for (int i = b0; i < b1; ++i) l.row[i] = most = max(most, l.row[i]);
    __syncwarp();
    const int m = (E + 33) >> 5, g0 = min(lane * m, E + 2), g1 = min((lane + 1) * m, E + 2);
    auto tiles = [&](int i) { return gm_parts<OP>(l.row[i + 1] - l.row[i]) * p.n_rt; };
    int sum = 0;
    for (int i = g0; i < g1; ++i) sum += tiles(i);
    const int upto = gm_scan_add(sum, lane);
    int at = upto - sum;
    for (int i = g0; i < g1; ++i) {
      l.tile[i] = at;
      at += tiles(i);
    }
    if (lane == 31) l.tile[E + 2] = upto;
  }
  __syncthreads();
}
// Tile w: the tiles of a group's rows lie side by side for the same features. kGmGrad reads
// its expert's bounds through the L1: from the L2, where all blocks' warps ask for the same
// few lines, 128 rows an expert took 185 us instead of 163.
template <int OP> SI_DEV GmTile gm_tile(const GmParams &p, const GmList &l, int w) {
  GmTile t;
  if constexpr (OP == kGmGrad) {
    t.ct = w % p.n_ct;
    const int r = w / p.n_ct;
    t.rt = r % p.n_rt;
    t.e = r / p.n_rt;
    t.row0 = min(max(__ldg(p.offsets + t.e), 0), p.rows);
    t.count = max(min(max(__ldg(p.offsets + t.e + 1), 0), p.rows) - t.row0, 0);
  } else {
    int lo = 0, hi = p.n_experts + 1;            // the last group whose first tile is at most w
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (l.tile[mid] <= w) lo = mid;
      else hi = mid - 1;
    }
    const int rows = l.row[lo + 1] - l.row[lo], i = w - l.tile[lo];
    const int parts = gm_parts<OP>(rows), per = gm_per<OP>(rows, parts);
    t.rt = i / parts;
    t.ct = 0;
    const int r = (i - t.rt * parts) * per;
    t.row0 = l.row[lo] + r;
    t.count = min(per, rows - r);
    t.e = lo <= p.n_experts ? lo - 1 : -1;
  }
  return t;
}
// Stages of a tile; for kGmGrad of its expert's whole 16 rows, up to 15 more are the tail.
template <int OP> SI_DEV int gm_steps(const GmParams &p, const GmTile &t) {
  return OP == kGmGrad ? ((t.count & ~15) + kGmK - 1) / kGmK : t.e < 0 ? 0 : (p.k + kGmK - 1) / kGmK;
}

// ---- tensor core -----------------------------------------------------------------

// Shared-memory matrix descriptors: 128-byte swizzle (layout 2), version 1; 8-row
// groups (8 summed indices, MN-major) 1024 bytes apart, and MN-major the next 64
// values kGmPiece bytes on. The high word is the same for both.
constexpr uint32_t kGmDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
template <bool MN> SI_DEV uint32_t gm_desc_lo(uint32_t addr, uint32_t piece = kGmPiece) {
  return (addr >> 4) | ((MN ? piece >> 4 : 1u) << 16);
}
template <bool MN> constexpr uint32_t kGmK16 = (MN ? 16 * 128 : 32) / 16;   // 16 summed indices on
template <int CG> SI_DEV void gm_mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kGmDescHi)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 da, db;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
        " setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "n"(kGmDescHi)
        : "memory");
}
// Arrive on `bar` (of both blocks of a pair) once the MMAs issued so far are complete.
template <int CG> SI_DEV void gm_commit(uint64_t *bar) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    umma_commit(bar);
}
template <int CG> SI_DEV void gm_tmem_alloc(uint32_t *dst, uint32_t cols) {   // a whole warp (of each block)
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, cols);
    tmem_relinquish();
  }
}
template <int CG> SI_DEV void gm_tmem_free(uint32_t addr, uint32_t cols) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
  else
    tmem_dealloc(addr, cols);
}

// 8 columns of this warp's lanes; tcgen05.wait::st before they are read.
SI_DEV void gm_tmem_st8(uint32_t addr, const float v[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}

// ---- epilogues ---------------------------------------------------------------

template <int OUT> SI_DEV uint32_t gm_pack(float lo, float hi) {
  uint32_t w;
  if constexpr (OUT == kGmBf16) asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(w) : "f"(lo), "f"(hi));
  else asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(w) : "f"(lo), "f"(hi));
  return w;
}
template <int OUT> SI_DEV void gm_store1(void *out, int64_t at, float v) {
  if constexpr (OUT == kGmBf16) static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
  else if constexpr (OUT == kGmF16) static_cast<__half *>(out)[at] = __float2half_rn(v);
  else static_cast<float *>(out)[at] = v;
}

// The largest magnitude over the warp of each of 16 values, cut to 16 bits (which hold
// its exponent): lane j gets value (j & 15)'s, in the low half for even ones. A lane hands
// half of its words on at every step, so 10 shuffles do (redux.sync for each value made gate
// and up of 512 rows an expert, kept, 528 us instead of 363; 284 with what is said at
// gm_keep16 and in the kernel).
SI_DEV uint32_t gm_top16(const float v[16], int lane) {
  uint32_t top[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    top[i] = __byte_perm(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]), 0x7632) & 0x7FFF7FFFu;
#pragma unroll
  for (int n = 4, m = 16; n > 0; n >>= 1, m >>= 1) {
    const bool up = (lane & m) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const uint32_t give = up ? top[i] : top[i + n], keep = up ? top[i + n] : top[i];
      top[i] = __vmaxu2(keep, __shfl_xor_sync(0xffffffffu, give, m));
    }
  }
  uint32_t t = top[0];                           // word lane / 4
  t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, 2));
  t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, 1));
  return __shfl_sync(0xffffffffu, t, (lane & 14) * 2) & 0x7FFF7FFFu;
}

// The tokens of a tile, 16 columns of the accumulator at a time, dealt out to the
// parts of the epilogue: piece i of a part.
template <int PARTS> SI_DEV int gm_piece(int i, int part) { return (i * PARTS + part) * 16; }

// This lane's feature f of 16 rows from row0, `left` of them in the tile: fp32 rows
// straight from the registers (128 bytes of a row a store), others in 16-byte words
// through `box` (1024 bytes of the warp's own).
template <int OUT, int ROWS = 16>
SI_DEV void gm_write16(const GmParams &p, void *out, int64_t ld, int f, int lane, int64_t row0, int left,
                       const float *v, uint8_t *box) {
  if constexpr (OUT == kGmF32) {
    if (f >= p.n) return;
    float *o = static_cast<float *>(out) + row0 * ld + f;
#pragma unroll
    for (int j = 0; j < 16; ++j, o += ld)
      if (j < left) *o = v[j];
  } else {
    __syncwarp();                                // the box has been read
#pragma unroll
    for (int j = 0; j < ROWS; ++j) gm_store1<OUT>(box + j * 64, lane, v[j]);
    __syncwarp();
    const int f0 = f - lane + (lane & 3) * 8;
#pragma unroll
    for (int h = 0; h < ROWS / 8; ++h) {
      const int j = h * 8 + (lane >> 2);
      const uint4 w = *reinterpret_cast<const uint4 *>(box + j * 64 + (lane & 3) * 16);
      if (j < left && f0 < p.n) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + (row0 + j) * ld + f0) = w;
    }
  }
}
// The 8-bit blocks of 16 rows at this warp's 32 values (side 0: g, 1: u) from feature
// f - lane, through `box` (512 bytes of the warp's own) so that rows leave in 16-byte
// words. Lane j finds the scale of row j and its inverse, which the others fetch.
SI_DEV void gm_keep16(const GmParams &p, int f, int lane, int64_t row0, int left, const float v[16], int side,
                      uint8_t *box) {
  const uint32_t pair = gm_top16(v, lane), top = lane & 1 ? pair & 0xFFFF0000u : pair << 16, s = mi_scale_of(top);
  const bool far = mi_far(top);
  const float up = far ? 0.f : mi_inv_step(s);
  __syncwarp();                                  // the box has been read
  if (!__any_sync(0xffffffffu, far)) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      box[j * 32 + lane] = static_cast<uint8_t>(mi_code_near(v[j], __shfl_sync(0xffffffffu, up, j)));
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t sj = __shfl_sync(0xffffffffu, s, j);
      box[j * 32 + lane] = static_cast<uint8_t>(sj == 255u ? 0u : mi_code(v[j] * mi_inv_scale(sj)));
    }
  }
  __syncwarp();
  const int f0 = f - lane, j = lane >> 1, c = (lane & 1) * 16;
  const int64_t blocks = mi_blocks(p.n);
  if (j < left) {
    uint8_t *to = p.codes + (row0 + j) * 2 * p.n + side * static_cast<int64_t>(p.n) + f0 + c;
    const uint4 w = *reinterpret_cast<const uint4 *>(box + lane * 16);
    if (f0 + c + 16 <= p.n && (p.n & 15) == 0) {
      *reinterpret_cast<uint4 *>(to) = w;
    } else {                                     // n is a multiple of 8
      if (f0 + c < p.n) *reinterpret_cast<uint2 *>(to) = make_uint2(w.x, w.y);
      if (f0 + c + 8 < p.n) *reinterpret_cast<uint2 *>(to + 8) = make_uint2(w.z, w.w);
    }
  }
  if (lane < 16 && lane < left) p.scales[(row0 + lane) * 2 * blocks + side * blocks + (f0 >> 5)] = static_cast<uint8_t>(s);
}

// Sums of 16 values over the warp: value (lane / 2) on even lanes, each lane handing
// half of its values on at every step.
SI_DEV float gm_reduce16(float v[16], int lane) {
#pragma unroll
  for (int n = 8, m = 16; n > 0; n >>= 1, m >>= 1) {
    const bool up = (lane & m) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// What 16 rows need beside gh, as it comes from memory: 16 codes of g and of u of row
// lane / 2, lane j's and 16 + j's scales of row j's, lane j's weight of row j, and which rows
// are a pair's.
struct GmKept {
  uint4 g, u;
  uint32_t s, live;
  float c;
};
SI_DEV GmKept gm_load_kept(const GmParams &p, int f, int lane, int64_t row0, int left) {
  GmKept k;
  k.g = k.u = make_uint4(0, 0, 0, 0);
  const int64_t blocks = mi_blocks(p.n);
  const int f0 = f - lane + (lane & 1) * 16, r = lane >> 1, j = lane & 15;
  if (r < left) {
    const uint8_t *at = p.codes + (row0 + r) * 2 * p.n + f0;
    if (f0 + 16 <= p.n && (p.n & 15) == 0) {
      k.g = __ldg(reinterpret_cast<const uint4 *>(at));
      k.u = __ldg(reinterpret_cast<const uint4 *>(at + p.n));
    } else {                                     // n is a multiple of 8
      uint2 w[4] = {};
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (f0 + 8 * i < p.n) {
          w[i] = __ldg(reinterpret_cast<const uint2 *>(at + 8 * i));
          w[2 + i] = __ldg(reinterpret_cast<const uint2 *>(at + p.n + 8 * i));
        }
      k.g = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
      k.u = make_uint4(w[2].x, w[2].y, w[3].x, w[3].y);
    }
  }
  k.s = 0;
  k.c = 0.f;
  bool live = false;
  if (j < left) {
    if (f - lane < p.n) k.s = __ldg(p.scales + (row0 + j) * 2 * blocks + (lane >> 4) * blocks + ((f - lane) >> 5));
    const int64_t pair = p.order ? __ldg(p.order + row0 + j) : row0 + j;
    live = pair >= 0 && pair < p.rows;
    if (live) k.c = p.c ? __ldg(p.c + pair) : 1.f;
  }
  k.live = __ballot_sync(0xffffffffu, live);
  return k;
}
// The gradients of h = silu(g) u in 16 rows: gh comes from the accumulator. The codes go
// to the lanes of their features through `box` (1024 bytes of the warp's own), g's and u's
// side by side; the results leave through it 8 rows at a time.
template <int OUT>
SI_DEV void gm_swiglu_back16(const GmParams &p, int f, int lane, int64_t row0, int left, const GmKept &k, float gh[16],
                             int slot, uint8_t *box) {
  __syncwarp();                                  // the box has been read
  const uint32_t g4[4] = {k.g.x, k.g.y, k.g.z, k.g.w}, u4[4] = {k.u.x, k.u.y, k.u.z, k.u.w};
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {                  // code + 128, as mi_values4 has it
    w[2 * i] = __byte_perm(g4[i], u4[i], 0x5140) ^ 0x80808080u;
    w[2 * i + 1] = __byte_perm(g4[i], u4[i], 0x7362) ^ 0x80808080u;
  }
  *reinterpret_cast<uint4 *>(box + lane * 32) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4 *>(box + lane * 32 + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  __syncwarp();
  uint32_t q[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) q[j] = *reinterpret_cast<const uint16_t *>(box + (j * 32 + lane) * 2);
  const float step = mi_step(k.s);               // lane j: of row j's g, lane 16 + j: of its u
  const int64_t ld = 2 * static_cast<int64_t>(p.n);
#pragma unroll
  for (int h = 0; h < 16; h += 8) {
    float ch[8];
    __syncwarp();                                // the box has been read
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = h + i;
      const float g = (__uint_as_float(__byte_perm(q[j], 0x4B000000u, 0x7540)) - 8388736.f) * __shfl_sync(0xffffffffu, step, j);
      const float u = (__uint_as_float(__byte_perm(q[j], 0x4B000000u, 0x7541)) - 8388736.f) * __shfl_sync(0xffffffffu, step, 16 + j);
      const float c = __shfl_sync(0xffffffffu, k.c, j), l = mi_logistic(g), si = g * l, hv = si * u, cd = c * gh[j];
      float gg = cd * u * fmaf(si, 1.f - l, l), gu = cd * si;   // s (1 + g (1 - s))
      ch[i] = c * hv;
      gh[j] *= hv;
      if (!((k.live >> j) & 1u)) gg = gu = ch[i] = gh[j] = 0.f;   // a row of no pair, the same for the warp
      gm_store1<OUT>(box + i * 64, lane, gg);
      gm_store1<OUT>(box + 512 + i * 64, lane, gu);
    }
    __syncwarp();
    const int r = lane >> 2, f0 = f - lane + (lane & 3) * 8;
    const bool out = h + r < left && f0 < p.n;
    const uint4 a = *reinterpret_cast<const uint4 *>(box + lane * 16), b = *reinterpret_cast<const uint4 *>(box + 512 + lane * 16);
    if (out) {
      uint16_t *to = static_cast<uint16_t *>(p.out) + (row0 + h + r) * ld + f0;
      *reinterpret_cast<uint4 *>(to) = a;
      *reinterpret_cast<uint4 *>(to + p.n) = b;
    }
    if (p.wh) gm_write16<OUT, 8>(p, p.wh, p.n, f, lane, row0 + h, left - h, ch, box);
  }
  if (!p.part) return;
  if (f >= p.n) {
#pragma unroll
    for (int j = 0; j < 16; ++j) gh[j] = 0.f;
  }
  const float sum = gm_reduce16(gh, lane);
  const int j = lane >> 1;
  if (!(lane & 1) && j < left) p.part[(row0 + j) * p.parts + slot] = sum;
}

// ---- the kernel ----------------------------------------------------------------

// Stages that one accumulator takes up. The tensor cores' additions truncate: with
// fp32 outputs the sums of 512 terms are added up in registers instead, rounded to
// nearest (1448 terms were off by 1.8e-6 relative, now 6e-7; fp32 sums in turn 7e-7).
// kGmSwigluParts: so are fp16's gate and up, whose errors turn 8-bit codes (of 4096 terms
// 1.5e-4 of them, in parts 2.7e-5, as fp32 products do; beside bf16's own rounding they do not
// show). A pair of SMs adds the first 1024 terms up in one: its accumulator is held while the
// 8-bit blocks before are made, and the MMAs get one part ahead (256 rows an expert, 2048
// terms, kept 200 us, 217 in parts so, 237 in parts of 512; in one SM, 4 rows an expert, 122
// and in parts of 512 124).
template <int MODE, int OUT> constexpr int kGmChunk = OUT == kGmF32 || MODE == kGmSwigluParts ? 8 : 1 << 30;
template <int OP, int MODE, int OUT>
constexpr int kGmFirst = MODE == kGmSwigluParts && OP == kGmWide ? 16 : kGmChunk<MODE, OUT>;
template <int OP, int MODE, int OUT> SI_DEV int gm_next(int k0) {
  return k0 == 0 ? kGmFirst<OP, MODE, OUT> : k0 + kGmChunk<MODE, OUT>;
}

// WMN: the matrices lie by columns (features contiguous).
template <int OP, int MODE, bool WMN, int OUT>
__global__ void __launch_bounds__(GmCfg<OP, MODE, OUT>::kThreads, 1) moe_mm_kernel(const __grid_constant__ GmParams p) {
  using C = GmCfg<OP, MODE, OUT>;
  constexpr int S = C::kStages, CG = C::CG, PARTS = C::kEpiWarps / 4, PIECES = C::kN / 16 / PARTS;
  constexpr bool kAMn = OP == kGmGrad || WMN, kBMn = OP == kGmGrad;
  static_assert(MODE == kGmPlain || (OP != kGmGrad && OUT != kGmF32 && !(kGmForward<MODE> && WMN)), "forms");
  extern __shared__ uint8_t gm_smem[];
  uint8_t *base = gm_smem + ((1024u - (smem_addr(gm_smem) & 1023u)) & 1023u);
  uint8_t *tails = base + S * C::kStage, *outs = tails + C::kTail;
  uint64_t *full = reinterpret_cast<uint64_t *>(outs + C::kOut);
  uint64_t *empty = full + S, *acc_full = empty + S, *acc_empty = acc_full + 2, *drain = acc_empty + 2;
  // tails: landed in this block, cleared in both, read by their MMA
  uint64_t *tail_full = drain + 1, *tail_ready = tail_full + 2, *tail_empty = tail_ready + 2;
  uint32_t *s_taddr = reinterpret_cast<uint32_t *>(tail_empty + 2);
  GmList &list = *reinterpret_cast<GmList *>(outs + C::kOut + 512);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? static_cast<int>(cluster_rank()) : 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(full + i, 2);            // the producers; of a pair, the first block's
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, C::kEpiWarps * CG);   // of the first block
    }
    mbar_init(drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(tail_full + i, 2);
      mbar_init(tail_ready + i, CG);
      mbar_init(tail_empty + i, 1);
    }
    fence_mbar_init();
  }
  if (threadIdx.x == 32) {           // the maps on their way
    prefetch_map(&p.a);
    prefetch_map(p.b);
  }
  grid_dep_wait();
  // before the next kernel may start: its blocks take tensor memory too
  if (warp == C::kBWarp) gm_tmem_alloc<CG>(s_taddr, C::kCols);
  tc_fence_before();
  if constexpr (OP != kGmGrad) gm_list<OP>(p, list);
  if constexpr (CG == 2) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *s_taddr, 0);
  const int total = OP == kGmGrad ? p.n_experts * p.n_rt * p.n_ct : list.tile[p.n_experts + 2];
  const int first = blockIdx.x / CG, step = gridDim.x / CG;
  auto tile = [&](int w) { return gm_tile<OP>(p, list, w); };
  // a tile's columns of the accumulator: its rows, to the next 32 (16 in one SM)
  auto columns = [&](const GmTile &t) { return OP == kGmGrad ? 256 : (t.count + 16 * CG - 1) & -(16 * CG); };
  // rows of the tail, behind an expert's whole 16
  auto tail_rows = [&](const GmTile &t) { return OP == kGmGrad ? t.count & 15 : 0; };
  const uint32_t full0 = CG == 2 ? cluster_addr(smem_addr(full), 0) : smem_addr(full);

  if (warp == 0 || warp == C::kBWarp) {
    if (lane == 0) {
      uint32_t it = 0, cuts = 0;
      bool ok = true;
      auto load = [&](void *to, const CUtensorMap *m, int c0, int c1, int c2, int c3, uint32_t bar) {
        tma_load4<CG == 2>(to, m, c0, c1, c2, c3, bar);
      };
      // 128 values, from v, of some summed indices of an MN-major operand: pieces of 64 values
      auto load_mn = [&](uint8_t *to, int piece, const CUtensorMap *m, int whole, int v, int c1, int c3, uint32_t bar) {
        if (whole) {
          load(to, m, 0, c1, v >> 6, c3, bar);
        } else {
          load(to, m, v, c1, 0, c3, bar);
          load(to + piece, m, v + 64, c1, 0, c3, bar);
        }
      };
      for (int w = first; ok && w < total; w += step) {
        const GmTile t = tile(w);
        const int nk = gm_steps<OP>(p, t), half = columns(t) / CG;
        if constexpr (OP == kGmGrad) {
          // the tail first: it is cleared while the stages are on their way
          if (tail_rows(t)) {
            const uint32_t u = cuts & 1;
            if (!mbar_wait_bounded(tail_empty + u, ((cuts >> 1) & 1) ^ 1, p.status)) {
              ok = false;
              break;
            }
            uint8_t *to = tails + (u * 2 + (warp != 0)) * kGmTail;
            const int r = t.row0 + (t.count & ~15);
            mbar_arrive_expect_tx(tail_full + u, kGmTail);
            if (warp == 0)
              load_mn(to, kGmTail / 2, &p.ta, p.whole_a, t.rt * 256 + rank * 128, r, 0, smem_addr(tail_full + u));
            else
              load_mn(to, kGmTail / 2, &p.tb, p.whole_b, t.ct * 256 + rank * 128, r, 0, smem_addr(tail_full + u));
            ++cuts;
          }
        }
        for (int ks = 0; ks < nk; ++ks, ++it) {
          const int s = it % S;
          if (!mbar_wait_bounded(empty + s, ((it / S) & 1) ^ 1, p.status)) {
            ok = false;
            break;
          }
          uint8_t *st = base + s * C::kStage + (warp == 0 ? 0 : C::kABytes);
          const int c = ks * kGmK;
          // The copies of both blocks count at the first one's barrier of the stage, which its
          // producers arrive at for both. One copy a stage and thread: two or three of them,
          // at a few hundred cycles each, bound the stage (320 rows an expert in three boxes
          // of 32 a stage 302 us, in one 231).
          const uint32_t bar = full0 + s * 8;
          auto expect = [&](uint32_t bytes) {
            if (rank == 0) mbar_arrive_expect_tx(full + s, bytes * CG);
          };
          if (warp == 0) {
            expect(C::kABytes);
            if constexpr (OP == kGmGrad)
              load_mn(st, kGmPiece, &p.a, p.whole_a, t.rt * 256 + rank * 128, t.row0 + c, 0, bar);
            else if constexpr (kGmForward<MODE>)    // gate and up
              load(st, &p.a, c, t.rt * 128 + rank * 64, 0, t.e, bar);
            else if constexpr (WMN)
              load_mn(st, kGmPiece, &p.a, p.whole_a, (t.rt * CG + rank) * 128, c, t.e, bar);
            else
              load(st, &p.a, c, (t.rt * CG + rank) * 128, 0, t.e, bar);
          } else if constexpr (OP == kGmGrad) {
            expect(C::kBBytes);
            load_mn(st, kGmPiece, p.b, p.whole_b, t.ct * 256 + rank * 128, t.row0 + c, 0, bar);
          } else if constexpr (OP == kGmFew) {
            expect(C::kBBytes);
            load(st, p.b, c, t.row0, 0, 0, bar);
          } else {                   // no more rows than the next 32: they come from the L2
            const int n = (half - 1) >> 5;
            expect((n + 1) * 32 * 128);
            load(st, p.b + n, c, t.row0 + rank * half, 0, 0, bar);
          }
        }
      }
      if (!ok) {   // copies in flight land before the block's memory goes
        if constexpr (CG == 1) {
          const uint32_t n = it < static_cast<uint32_t>(S) ? it : S;
          for (uint32_t i = it - n; i < it; ++i) mbar_wait_bounded(full + i % S, (i / S) & 1, p.status);
        } else {   // their barrier may be the other block's: 10 ms are a thousand times their way
          const uint64_t t0 = now_ns();
          while (now_ns() - t0 < 10000000u) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // the warp walks over the stages together, the leader alone waits and issues
    const bool leader = elect_lane();
    const uint32_t smem0 = smem_addr(base);
    uint32_t n = 0, cuts = 0;        // accumulators and tails taken so far
    int s = 0;                       // stage and its parity
    uint32_t parity = 0;
    bool ok = true;
    for (int w = rank == 0 ? first : total; w < total; w += step) {
      const GmTile t = tile(w);
      const int nk = gm_steps<OP>(p, t);
      const uint32_t idesc = (1u << 4) | p.fmt | (kAMn ? 1u << 15 : 0u) | (kBMn ? 1u << 16 : 0u) |
                             (static_cast<uint32_t>(columns(t) >> 3) << 17) | ((CG * 128u >> 4) << 24);
      const int last = OP == kGmGrad ? t.count & ~15 : p.k, cut = tail_rows(t);   // summed indices
      for (int k0 = 0; k0 < nk || (k0 == 0 && cut); k0 = gm_next<OP, MODE, OUT>(k0), ++n) {
        const uint32_t u = n & 1, d = tmem + u * C::kAccCols;
        if (leader && ok) {          // (the fence behind it is the stages' and the tail's)
          const uint32_t free = ((n >> 1) & 1) ^ 1;
          ok = CG == 2 ? mbar_wait_cluster(acc_empty + u, free, p.status) : mbar_wait_bounded(acc_empty + u, free, p.status);
        }
        const int k1 = min(nk, gm_next<OP, MODE, OUT>(k0));
        for (int ks = k0; ks < k1; ++ks) {
          const int n16 = (min(kGmK, last - ks * kGmK) + 15) >> 4;
          const uint32_t st = smem0 + s * C::kStage;
          if (leader && ok) ok = mbar_wait_bounded(full + s, parity, p.status);
          if (leader && ok) {
            tc_fence_after();
            const uint32_t la = gm_desc_lo<kAMn>(st), lb = gm_desc_lo<kBMn>(st + C::kABytes);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i >= n16) break;
#pragma unroll
              for (int a = 0; a < C::MA; ++a)
                gm_mma<CG>(d + a * C::kN, la + a * (128 * 128 / 16) + i * kGmK16<kAMn>, lb + i * kGmK16<kBMn>, idesc,
                           i > 0 || ks > k0);
            }
            gm_commit<CG>(empty + s);
          }
          if (++s == S) {
            s = 0;
            parity ^= 1;
          }
        }
        if constexpr (OP == kGmGrad) {
          if (cut && k1 == nk) {
            const uint32_t v = cuts & 1, at = smem_addr(tails) + v * 2 * kGmTail;
            if (leader && ok) ok = mbar_wait_cluster(tail_ready + v, (cuts >> 1) & 1, p.status);
            if (leader && ok) {
              tc_fence_after();
              gm_mma<CG>(d, gm_desc_lo<true>(at, kGmTail / 2), gm_desc_lo<true>(at + kGmTail, kGmTail / 2), idesc, k1 > k0);
              gm_commit<CG>(tail_empty + v);
            }
            ++cuts;
          }
        }
        if (leader && ok) gm_commit<CG>(acc_full + u);
      }
    }
    if (leader && !ok) {   // MMAs in flight end before the tensor memory goes
      gm_commit<CG>(drain);
      mbar_wait_bounded(drain, 0, p.status);
    }
    __syncwarp();
  } else if (warp == C::kTailWarp) {
    // the rows behind the expert's in its tail: cleared, in both operands
    const uint32_t ready0 = cluster_addr(smem_addr(tail_ready), 0);
    uint32_t cuts = 0;
    for (int w = first; w < total; w += step) {
      const int left = tail_rows(tile(w));
      if (left == 0) continue;
      const uint32_t u = cuts & 1;
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(tail_full + u, (cuts >> 1) & 1, p.status))) break;
      ++cuts;
      uint8_t *to = tails + u * 2 * kGmTail + (lane >> 3) * (kGmTail / 2) + (lane & 7) * 16;
      for (int r = left; r < 16; ++r) *reinterpret_cast<uint4 *>(to + r * 128) = make_uint4(0, 0, 0, 0);
      fence_async_smem();
      __syncwarp();
      // written here, read by the MMA that a thread of the first block issues for both
      if (lane == 0) mbar_arrive_cluster(ready0 + u * 8);
    }
  } else {
    const int q = warp & 3, part = (warp - 2) >> 2;   // the 32 lanes of tensor memory this warp may read
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t free0 = CG == 2 ? cluster_addr(smem_addr(acc_empty), 0) : smem_addr(acc_empty);
    uint8_t *stage = outs + (warp - 2) * C::kBox;
    uint32_t n = 0;
    bool ok = true;
    auto wait_acc = [&] {            // its address; n goes on with release()
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(acc_full + (n & 1), (n >> 1) & 1, p.status));
      tc_fence_after();
      return lanes + (n & 1) * C::kAccCols;
    };
    auto release = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) mbar_arrive_cluster_relaxed(free0 + (n & 1) * 8);   // what was read is in registers
        else mbar_arrive(acc_empty + (n & 1));
      }
      ++n;
    };
    // after a wait that ran out nothing is waited for any more: zeros, so that warps that
    // meet at a barrier all come there
    for (int w = first; w < total; w += step) {
      const GmTile t = tile(w);
      const int steps = gm_steps<OP>(p, t), nk = !ok ? 0 : steps == 0 && tail_rows(t) ? 1 : steps;
      bool zero = nk == 0;
      if constexpr (OP == kGmGrad) {
        // lane = row of the gradient; a part's columns, 64 bytes of them at a time through shared
        // memory (boxes of 128 bytes would take the room of a stage)
        constexpr int kPer = 64 / kGmSize<OUT>, kMine = 256 / PARTS;   // columns of a box, of a part
        const int row = t.rt * 256 + rank * 128 + q * 32, col = t.ct * 256 + part * kMine;
        float sum[OUT == kGmF32 ? kMine : 1] = {};
        uint32_t acc = 0;
        if constexpr (OUT == kGmF32) {
          for (int k0 = 0; ok && k0 < nk; k0 += kGmChunk<MODE, OUT>) {
            acc = wait_acc();
            if (!ok) break;
#pragma unroll
            for (int c = 0; c < kMine; c += 8) {
              float r[8];
              tmem_ld8(acc + part * kMine + c, r);
#pragma unroll
              for (int i = 0; i < 8; ++i) sum[c + i] += r[i];
            }
            release();
          }
        } else if (!zero) {
          acc = wait_acc();
        }
        zero |= !ok;
#pragma unroll
        for (int c = 0; c < kMine; c += kPer) {
          uint32_t v[16];            // 64 bytes of the row
          if (OUT != kGmF32 && zero) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0;
          } else if constexpr (OUT == kGmF32) {   // zeros where there was nothing to add
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(sum[c + i]);
          } else {
            uint32_t r[32];
            tmem_ld32(acc + part * kMine + c, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = gm_pack<OUT>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
            if (c + kPer == kMine) release();
          }
          if (lane == 0) tma_store_wait_read();        // the box before has been read
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4 *>(stage + lane * 64 + ((i ^ (lane >> 1 & 3)) * 16)) =
                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          fence_async_smem();
          __syncwarp();
          if (lane == 0 && row < p.n && col + c < p.k) tma_store4(&p.o, stage, col + c, row, 0, t.e);
        }
      } else {
        // lane = feature; 16 rows at a time
        const int tf = kGmForward<MODE> && OP == kGmWide ? t.rt * 128 + rank * 64 + (q & 1) * 32
                                                          : (t.rt * CG + rank) * 128 + q * 32;
        const int f = tf + lane;
        auto read16 = [&](uint32_t addr, float v[16]) {
          uint32_t r[16];
          tmem_ld16(addr, r);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
        };
        auto zeros = [&](float v[16]) {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = 0.f;
        };
        // the last piece of this part, behind which the accumulator is free
        const int mine = t.count > part * 16 ? (t.count - part * 16 + 16 * PARTS - 1) / (16 * PARTS) : 0;
        uint32_t acc = 0;
        if constexpr (OUT == kGmF32) {
          float sum[PIECES][16] = {};
          for (int k0 = 0; ok && k0 < nk; k0 += kGmChunk<MODE, OUT>) {
            acc = wait_acc();
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
              if (i >= mine) break;
#pragma unroll
              for (int h = 0; h < 16; h += 8) {
                float r[8];
                tmem_ld8(acc + gm_piece<PARTS>(i, part) + h, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[i][h + j] += r[j];
              }
            }
            release();
          }
#pragma unroll
          for (int i = 0; i < PIECES; ++i) {
            if (i >= mine) break;
            const int j0 = gm_piece<PARTS>(i, part);
            gm_write16<OUT>(p, p.out, p.ld, f, lane, static_cast<int64_t>(t.row0) + j0, t.count - j0, sum[i], stage);
          }
        } else {
          if constexpr (MODE != kGmSwigluBack) {
            constexpr bool kParts = MODE == kGmSwigluParts;
            constexpr int HALVES = kParts && OP == kGmFew ? 2 : 1;
            float sum[kParts ? HALVES * PIECES : 1][16] = {};
            auto each = [&](auto f) {            // 8 columns of each piece
#pragma unroll
              for (int i = 0; i < HALVES * PIECES; ++i) {
                if (i % PIECES >= mine) continue;
#pragma unroll
                for (int h = 0; h < 16; h += 8) f(acc + i / PIECES * C::kN + gm_piece<PARTS>(i % PIECES, part) + h, sum[i] + h);
              }
            };
            if constexpr (kParts) {
              for (int k0 = 0; ok && gm_next<OP, MODE, OUT>(k0) < nk; k0 = gm_next<OP, MODE, OUT>(k0)) {   // but the last
                acc = wait_acc();
                if (!ok) break;
                each([&](uint32_t at, float *to) {
                  float r[8];
                  tmem_ld8(at, r);
#pragma unroll
                  for (int j = 0; j < 8; ++j) to[j] += r[j];
                });
                release();
              }
            }
            if (!zero && ok) acc = wait_acc();
            zero |= !ok;
            if constexpr (kParts) {
              if (!zero && nk > kGmFirst<OP, MODE, OUT>) {   // into the last one's place
                each([&](uint32_t at, float *to) {
                  float r[8];
                  tmem_ld8(at, r);
#pragma unroll
                  for (int j = 0; j < 8; ++j) r[j] += to[j];
                  gm_tmem_st8(at, r);
                });
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
              }
            }
            if (!zero && mine == 0) release();
          }
          bool have = MODE != kGmSwigluBack;     // the accumulator has been waited for
          GmKept next;                           // of the piece to come
          if constexpr (MODE == kGmSwigluBack)
            next = gm_load_kept(p, f, lane, static_cast<int64_t>(t.row0) + part * 16, zero ? 0 : t.count - part * 16);
          for (int i = 0; i < mine; ++i) {
            const int j0 = gm_piece<PARTS>(i, part), left = t.count - j0;
            const int64_t row0 = static_cast<int64_t>(t.row0) + j0;
            float v[16];
            if constexpr (MODE == kGmPlain) {
              if (zero) zeros(v);
              else read16(acc + j0, v);
              if (!zero && i == mine - 1) release();
              gm_write16<OUT>(p, p.out, p.ld, f, lane, row0, left, v, stage);
            } else if constexpr (MODE == kGmSwigluBack) {
              const GmKept kept = next;
              next = gm_load_kept(p, f, lane, row0 + 16 * PARTS, zero || i == mine - 1 ? 0 : left - 16 * PARTS);
              if (!zero && !have) {
                acc = wait_acc();
                zero = !ok;
                have = true;
              }
              if (zero) zeros(v);
              else read16(acc + j0, v);
              if (!zero && i == mine - 1) release();
              gm_swiglu_back16<OUT>(p, f, lane, row0, left, kept, v, (t.rt * CG + rank) * 4 + q, stage);
            } else if constexpr (OP == kGmFew) {
              float u[16];
              if (zero) {
                zeros(v);
                zeros(u);
              } else {
                read16(acc + j0, v);
                read16(acc + C::kN + j0, u);
                if (i == mine - 1) release();
              }
              if (tf < p.n && p.codes) {
                gm_keep16(p, f, lane, row0, left, v, 0, stage);
                gm_keep16(p, f, lane, row0, left, u, 1, stage);
              }
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = v[j] * mi_logistic(v[j]) * u[j];
              gm_write16<OUT>(p, p.out, p.ld, f, lane, row0, left, v, stage);
            } else {
              // lanes 0-63 hold g, 64-127 u of the same features: a pair of warps exchanges
              // halves of its rows through their boxes, g's takes the first 8, u's the last
              const int side = q >> 1, pair = 1 + part * 2 + (q & 1);
              if (zero) zeros(v);
              else read16(acc + j0, v);
              if (!zero && i == mine - 1) release();
              float *own = reinterpret_cast<float *>(stage);
              // (warps 2 and 3 of four read lanes 64-127)
              const float *other = reinterpret_cast<const float *>(stage + (side ? 2 : -2) * C::kBox);
              __syncwarp();          // the box has been read
#pragma unroll
              for (int j = 0; j < 8; ++j) own[j * 32 + lane] = side ? v[j] : v[8 + j];
              asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
              float h[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float o = other[j * 32 + lane], g = side ? o : v[j], u = side ? v[8 + j] : o;
                h[j] = g * mi_logistic(g) * u;
              }
              asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
              gm_write16<OUT, 8>(p, p.out, p.ld, f, lane, row0 + side * 8, left - side * 8, h, stage);
              if (tf < p.n && p.codes) gm_keep16(p, f, lane, row0, left, v, side, stage);
            }
          }
          if constexpr (MODE == kGmSwigluBack) {
            if (!zero && !have) {                // no rows of this part
              wait_acc();
              if (ok) release();
            }
          }
        }
      }
    }
    if (OP == kGmGrad && lane == 0) tma_store_wait_read();
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync();         // the other block's MMAs and arrivals are over too
  else __syncthreads();
  tc_fence_after();
  if (warp == C::kBWarp) {
    __syncwarp();
    gm_tmem_free<CG>(tmem, C::kCols);
  }
}

// gw of a row's pair: the sum of its partial sums, in their order.
__global__ void __launch_bounds__(256) gm_sum_kernel(const float *part, int n, int rows, const int32_t *order, float *gw) {
  grid_dep_wait();
  grid_dep_launch();
  const int row = blockIdx.x * 256 + threadIdx.x;
  if (row >= rows) return;
  const int64_t pair = order ? __ldg(order + row) : row;
  if (pair < 0 || pair >= rows) return;
  float sum = 0.f;
  for (int i = 0; i < n; i += 4) {               // n is a multiple of 4
    const float4 v = __ldcg(reinterpret_cast<const float4 *>(part + static_cast<int64_t>(row) * n + i));
    sum += v.x;
    sum += v.y;
    sum += v.z;
    sum += v.w;
  }
  gw[pair] = sum;
}

// ---- host ------------------------------------------------------------------

// Values of 2 or 4 bytes in four dimensions, the inner one contiguous, the others `stride`
// values apart, boxes of `inner` (128 or 64) bytes x b1 x b2 in the swizzle of that size; what lies outside
// reads as zero and is not written.
struct GmDims {
  int64_t d0, d1, s1, d2, s2, d3, s3;
};
static bool gm_map(CUtensorMap *m, const void *v, si_dtype type, const GmDims &g, int b1, int b2 = 1, int inner = 128) {
  const int64_t size = type == SI_F32 ? 4 : 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(g.d0), static_cast<cuuint64_t>(g.d1),
                              static_cast<cuuint64_t>(g.d2), static_cast<cuuint64_t>(g.d3)};
  // a dimension of one has a stride all the same: any that is allowed
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(g.s1 * size),
                                 static_cast<cuuint64_t>((g.d2 > 1 ? g.s2 : g.s1) * size),
                                 static_cast<cuuint64_t>((g.d3 > 1 ? g.s3 : g.s1) * size)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(inner / size), static_cast<cuuint32_t>(b1),
                             static_cast<cuuint32_t>(b2), 1};
  return encode_map(m, type == SI_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                       : type == SI_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                    v, 4, dims, strides, box, inner == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}
// Rows [rows][cols], ld apart, in boxes of `box` of them.
static bool gm_map_rows(CUtensorMap *m, const void *v, si_dtype type, int64_t rows, int64_t cols, int64_t ld, int box) {
  return gm_map(m, v, type, {cols, rows, ld, 1, 0, 1, 0}, box);
}
// The same (of each of `mats` matrices) as an MN-major operand: `box` rows x 64 columns, two such
// pieces side by side where the columns are whole pieces.
static bool gm_map_mn(CUtensorMap *m, int *whole, const void *v, si_dtype type, int64_t mats, int64_t rows,
                      int64_t cols, int64_t ld, int64_t mat, int box = kGmK) {
  *whole = cols % 64 == 0;
  return *whole ? gm_map(m, v, type, {64, rows, ld, cols / 64, 64, mats, mat}, box, 2)
                : gm_map(m, v, type, {cols, rows, ld, 1, 0, mats, mat}, box);
}

// Pairs of blocks that are resident at once, on the current device: fewer than half of
// the SMs where a part of the chip has an odd number of them.
template <typename C, typename K> static cudaError_t gm_pairs(K kernel, int *pairs) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (*pairs = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sm_count() & ~1));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(pairs, kernel, &cfg);
  if (e == cudaSuccess && *pairs < 1) e = cudaErrorInvalidConfiguration;
  if (e == cudaSuccess && dev < 64) known[dev].store(*pairs, std::memory_order_relaxed);
  return e;
}

template <int OP, int MODE, bool WMN, int OUT>
static cudaError_t gm_launch(const GmParams &p, int64_t most, cudaStream_t s) {
  using C = GmCfg<OP, MODE, OUT>;
  const auto kernel = moe_mm_kernel<OP, MODE, WMN, OUT>;
  cudaError_t e = allow_smem(kernel, C::kSmem);
  if (e != cudaSuccess) return e;
  int units = sm_count();
  if (C::CG == 2) {
    e = gm_pairs<C>(kernel, &units);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(most, units)) * C::CG);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C::CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C::CG == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}
template <typename F> static cudaError_t gm_by_out(si_dtype t, F f) {
  using std::integral_constant;
  return t == SI_BF16  ? f(integral_constant<int, kGmBf16>{})
         : t == SI_F16 ? f(integral_constant<int, kGmF16>{})
                       : f(integral_constant<int, kGmF32>{});
}
template <typename F> static cudaError_t gm_by_half(si_dtype t, F f) {
  using std::integral_constant;
  return t == SI_BF16 ? f(integral_constant<int, kGmBf16>{}) : f(integral_constant<int, kGmF16>{});
}

static bool gm_type(si_dtype t) { return t == SI_BF16 || t == SI_F16; }
static uint32_t gm_fmt(si_dtype t) { return t == SI_BF16 ? (1u << 7) | (1u << 10) : 0u; }
static bool gm_width(int64_t n, int64_t most = int64_t(1) << 20) { return n >= 8 && n % 8 == 0 && n <= most; }
constexpr int64_t kGmBoth = int64_t(1) << 21;    // g's and u's features side by side, where a gradient needs them
static bool gm_rows(int64_t rows, int n_experts) {
  return rows >= 0 && rows <= 0x7FFFFFFF - 256 && n_experts >= 1 && n_experts <= kSortMaxExperts;
}
// Rows at 16-byte boundaries, at least `cols` values apart.
static bool gm_ld(int64_t ld, int64_t cols, int size) {
  return ld >= cols && ld * size % 16 == 0 && ld <= (int64_t(1) << 36);
}
static bool gm_whole(const void *p, int size) { return p && reinterpret_cast<uintptr_t>(p) % size == 0; }

// Rows of an expert on average up to which a tile is one SM's, with 16 rows. The host does not know
// how many of the rows are an expert's: those of none count too. Measured with every row an expert's, in
// one SM against two, rows dealt out at random: 128 experts 1536 x 2048, 8 / 12 / 16 / 20 rows 125 /
// 126 / 128 / 150 us against 136 / 137 / 138 / 138; 2048 x 768 67 / 67 / 80 / 93 against 71 / 71 / 72 / 72;
// 256 of 512 x 2048 88 / 88 / 90 / 106 against 93 / 94 / 95 / 96; 16 of 4096 x 1024, 8 / 12 / 16 rows
// 27.4 / 26.1 / 32.0 against 28.9 / 29.4 / 29.5. Behind 16 rows an expert's second tile reads its matrix again.
static bool gm_few(int64_t rows, int n_experts) { return rows <= 12 * static_cast<int64_t>(n_experts); }

// What the products of sorted rows share: the rows' operand and the list. `tile`: features
// of a tile. Returns the number of tiles at most, 0 if they pass 2^30, -1 without a map.
static int64_t gm_forward(GmParams &p, bool few, const void *x, si_dtype type, int64_t rows, int64_t k, int64_t ldx,
                          int n_experts, int64_t n, int tile, const int32_t *offsets, void *workspace) {
  p.n_rt = static_cast<int>((n + tile - 1) / tile);
  const int m = few ? 16 : 256;
  const int64_t most = (rows / m + std::min<int64_t>(n_experts + 2, rows)) * p.n_rt;
  if (most > (int64_t(1) << 30)) return 0;
  for (int i = 0; i < (few ? 1 : 4); ++i)
    if (!gm_map_rows(p.b + i, x, type, rows, k, ldx, few ? 16 : 32 * (i + 1))) return -1;
  p.offsets = offsets;
  p.n_experts = n_experts;
  p.rows = static_cast<int>(rows);
  p.n = static_cast<int>(n);
  p.k = static_cast<int>(k);
  p.fmt = gm_fmt(type);
  p.status = static_cast<uint32_t *>(workspace);
  return most;
}

}  // namespace si

using namespace si;

extern "C" size_t si_moe_matmul_workspace_bytes(void) { return sizeof(WsHeader); }

extern "C" si_status si_moe_matmul(const void *x, si_dtype type, int64_t rows, int64_t ldx, const void *w,
                                   int n_experts, int64_t n, int64_t k, int64_t ldw, int64_t matw, int by_columns,
                                   const int32_t *offsets, void *out, si_dtype out_type, int64_t ldo, void *workspace,
                                   size_t workspace_bytes, void *stream) {
  if (!gm_rows(rows, n_experts) || !gm_width(n) || !gm_width(k, kGmBoth)) return SI_ERR_INVALID_ARG;
  if (!gm_type(type) || (out_type != SI_F32 && out_type != type)) return SI_ERR_UNSUPPORTED;
  if (rows == 0) return SI_OK;
  const bool few = gm_few(rows, n_experts), cols = by_columns != 0;
  const int64_t inner = cols ? n : k, outer = cols ? k : n;
  if (!x || !w || !offsets || !out || !aligned16(x) || !aligned16(w) || !aligned16(out) || !gm_whole(offsets, 4) ||
      !gm_ld(ldx, k, 2) || !gm_ld(ldo, n, out_type == SI_F32 ? 4 : 2) || !gm_ld(ldw, inner, 2) ||
      (n_experts > 1 && !gm_ld(matw, ldw * (outer - 1) + inner, 2)))
    return SI_ERR_INVALID_ARG;
  if (workspace && (!aligned256(workspace) || workspace_bytes < sizeof(WsHeader))) return SI_ERR_WORKSPACE;
  GmParams p{};
  const int64_t most = gm_forward(p, few, x, type, rows, k, ldx, n_experts, n, few ? 128 : 256, offsets, workspace);
  if (most == 0) return SI_ERR_UNSUPPORTED;
  if (most < 0 || !(cols ? gm_map_mn(&p.a, &p.whole_a, w, type, n_experts, k, n, ldw, matw)
                         : gm_map(&p.a, w, type, {k, n, ldw, 1, 0, n_experts, matw}, 128)))
    return SI_ERR_CUDA;
  p.out = out;
  p.ld = ldo;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(gm_by_out(out_type, [&](auto o) {
    constexpr int O = decltype(o)::value;
    if (few)
      return cols ? gm_launch<kGmFew, kGmPlain, true, O>(p, most, s) : gm_launch<kGmFew, kGmPlain, false, O>(p, most, s);
    return cols ? gm_launch<kGmWide, kGmPlain, true, O>(p, most, s) : gm_launch<kGmWide, kGmPlain, false, O>(p, most, s);
  }));
}

extern "C" si_status si_moe_matmul_grad_w(const void *gy, int64_t ldg, const void *x, int64_t ldx, si_dtype type,
                                          int64_t rows, int n_experts, int64_t n, int64_t k, const int32_t *offsets,
                                          void *gw, si_dtype gw_type, void *workspace, size_t workspace_bytes,
                                          void *stream) {
  if (!gm_rows(rows, n_experts) || !gm_width(n, kGmBoth) || !gm_width(k)) return SI_ERR_INVALID_ARG;
  if (!gm_type(type) || (gw_type != SI_F32 && gw_type != type)) return SI_ERR_UNSUPPORTED;
  const int size = gw_type == SI_F32 ? 4 : 2;
  if (!gw || !aligned16(gw)) return SI_ERR_INVALID_ARG;
  GmParams p{};
  p.n_rt = static_cast<int>((n + 255) / 256);
  p.n_ct = static_cast<int>((k + 255) / 256);
  const int64_t most = static_cast<int64_t>(n_experts) * p.n_rt * p.n_ct;
  if (most > (int64_t(1) << 30)) return SI_ERR_UNSUPPORTED;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) return cuda_status(cudaMemsetAsync(gw, 0, static_cast<size_t>(n_experts) * n * k * size, s));
  if (!gy || !x || !aligned16(gy) || !aligned16(x) || !gm_whole(offsets, 4) || !gm_ld(ldg, n, 2) || !gm_ld(ldx, k, 2))
    return SI_ERR_INVALID_ARG;
  if (workspace && (!aligned256(workspace) || workspace_bytes < sizeof(WsHeader))) return SI_ERR_WORKSPACE;
  if (!gm_map_mn(&p.a, &p.whole_a, gy, type, 1, rows, n, ldg, 0) ||
      !gm_map_mn(p.b, &p.whole_b, x, type, 1, rows, k, ldx, 0) ||
      !gm_map_mn(&p.ta, &p.whole_a, gy, type, 1, rows, n, ldg, 0, 16) ||
      !gm_map_mn(&p.tb, &p.whole_b, x, type, 1, rows, k, ldx, 0, 16) ||
      !gm_map(&p.o, gw, gw_type, {k, n, k, 1, 0, n_experts, n * k}, 32, 1, 64))
    return SI_ERR_CUDA;
  p.offsets = offsets;
  p.n_experts = n_experts;
  p.rows = static_cast<int>(rows);
  p.n = static_cast<int>(n);
  p.k = static_cast<int>(k);
  p.fmt = gm_fmt(type);
  p.status = static_cast<uint32_t *>(workspace);
  return cuda_status(gm_by_out(
      gw_type, [&](auto o) { return gm_launch<kGmGrad, kGmPlain, false, decltype(o)::value>(p, most, s); }));
}

extern "C" si_status si_moe_gateup(const void *x, si_dtype type, int64_t rows, int64_t ldx, const void *gate_up,
                                   int n_experts, int64_t inter, int64_t hidden, const int32_t *offsets, void *h,
                                   void *codes, void *scales, void *workspace, size_t workspace_bytes, void *stream) {
  if (!gm_rows(rows, n_experts) || !gm_width(inter) || !gm_width(hidden)) return SI_ERR_INVALID_ARG;
  if (!gm_type(type)) return SI_ERR_UNSUPPORTED;
  if (rows == 0) return SI_OK;
  if (!x || !gate_up || !h || !aligned16(x) || !aligned16(gate_up) || !aligned16(h) || !gm_whole(offsets, 4) ||
      !gm_ld(ldx, hidden, 2) || !codes != !scales || !aligned16(codes))
    return SI_ERR_INVALID_ARG;
  if (workspace && (!aligned256(workspace) || workspace_bytes < sizeof(WsHeader))) return SI_ERR_WORKSPACE;
  const bool few = gm_few(rows, n_experts);
  GmParams p{};
  const int64_t most = gm_forward(p, few, x, type, rows, hidden, ldx, n_experts, inter, 128, offsets, workspace);
  if (most == 0) return SI_ERR_UNSUPPORTED;
  if (most < 0 ||
      !gm_map(&p.a, gate_up, type, {hidden, inter, hidden, 2, inter * hidden, n_experts, 2 * inter * hidden},
              few ? 128 : 64, 2))
    return SI_ERR_CUDA;
  p.out = h;
  p.ld = inter;
  p.codes = static_cast<uint8_t *>(codes);
  p.scales = static_cast<uint8_t *>(scales);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(gm_by_half(type, [&](auto o) {
    constexpr int O = decltype(o)::value;
    // more terms than the first part's (512 rows an expert, 512 terms, kept, took 43 us with the parts' code, 37 without)
    if constexpr (O == kGmF16) {
      if (hidden > (few ? kGmFirst<kGmFew, kGmSwigluParts, O> : kGmFirst<kGmWide, kGmSwigluParts, O>) * kGmK)
        return few ? gm_launch<kGmFew, kGmSwigluParts, false, O>(p, most, s)
                   : gm_launch<kGmWide, kGmSwigluParts, false, O>(p, most, s);
    }
    return few ? gm_launch<kGmFew, kGmSwiglu, false, O>(p, most, s) : gm_launch<kGmWide, kGmSwiglu, false, O>(p, most, s);
  }));
}

// Partial sums of a row's gw: one of 32 features each, in whole tiles.
static int64_t gm_sums(int64_t rows, int n_experts, int64_t inter) {
  return gm_few(rows, n_experts) ? (inter + 127) / 128 * 4 : (inter + 255) / 256 * 8;
}

extern "C" size_t si_moe_down_backward_workspace_bytes(int64_t rows, int n_experts, int64_t inter) {
  if (!gm_rows(rows, n_experts) || !gm_width(inter)) return 0;
  return round_up(sizeof(WsHeader) + static_cast<size_t>(rows) * gm_sums(rows, n_experts, inter) * 4, 256);
}

extern "C" si_status si_moe_down_backward(const void *gy, si_dtype type, int64_t rows, int64_t ldg, const void *down,
                                          int n_experts, int64_t hidden, int64_t inter, const int32_t *offsets,
                                          const void *codes, const void *scales, const float *row_w,
                                          const int32_t *order, void *ggu, void *wh, float *gw, void *workspace,
                                          size_t workspace_bytes, void *stream) {
  if (!gm_rows(rows, n_experts) || !gm_width(inter) || !gm_width(hidden)) return SI_ERR_INVALID_ARG;
  if (!gm_type(type)) return SI_ERR_UNSUPPORTED;
  if (rows == 0) return SI_OK;
  if (!gy || !down || !codes || !scales || !ggu || !aligned16(gy) || !aligned16(down) || !gm_whole(offsets, 4) ||
      !aligned16(codes) || !aligned16(ggu) || !aligned16(wh) || (row_w && !gm_whole(row_w, 4)) ||
      (order && !gm_whole(order, 4)) || (gw && !gm_whole(gw, 4)) || !gm_ld(ldg, hidden, 2))
    return SI_ERR_INVALID_ARG;
  if ((gw && !workspace) ||
      (workspace && (!aligned256(workspace) ||
                     workspace_bytes < (gw ? si_moe_down_backward_workspace_bytes(rows, n_experts, inter) : sizeof(WsHeader)))))
    return SI_ERR_WORKSPACE;
  const bool few = gm_few(rows, n_experts);
  GmParams p{};
  const int64_t most = gm_forward(p, few, gy, type, rows, hidden, ldg, n_experts, inter, few ? 128 : 256, offsets, workspace);
  if (most == 0) return SI_ERR_UNSUPPORTED;
  if (most < 0 || !gm_map_mn(&p.a, &p.whole_a, down, type, n_experts, hidden, inter, inter, hidden * inter)) return SI_ERR_CUDA;
  p.out = ggu;
  p.codes = static_cast<uint8_t *>(const_cast<void *>(codes));
  p.scales = static_cast<uint8_t *>(const_cast<void *>(scales));
  p.c = row_w;
  p.order = order;
  p.wh = wh;
  p.parts = static_cast<int>(gm_sums(rows, n_experts, inter));
  p.part = gw ? reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + sizeof(WsHeader)) : nullptr;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = gm_by_half(type, [&](auto o) {
    constexpr int O = decltype(o)::value;
    return few ? gm_launch<kGmFew, kGmSwigluBack, true, O>(p, most, s) : gm_launch<kGmWide, kGmSwigluBack, true, O>(p, most, s);
  });
  if (e != cudaSuccess || !gw) return cuda_status(e);
  if (order && cudaMemsetAsync(gw, 0, static_cast<size_t>(rows) * sizeof(float), s) != cudaSuccess) return SI_ERR_CUDA;
  return cuda_status(launch_pdl(gm_sum_kernel, dim3(static_cast<unsigned>((rows + 255) / 256)), dim3(256), 0, s,
                                static_cast<const float *>(p.part), p.parts, p.rows, order, gw));
}
