// Products of MXFP4 matrices on the tensor cores: the plain product and the
// expert FFN of a routed batch.
//
//   out[m][n] = sum_k a[m][k] w[n][k]            (si_mxfp4_matmul)
//   h = silu(G x) * (U x), y = D h per pair      (si_moe_ffn_mxfp4)
//
// Both are one kernel: tcgen05.mma kind::mxf4 with block scales. Products of two
// E2M1 values are exact and the accumulators fp32. It has two orientations:
//  - few tokens: 128 (or gate 128 and up 128) weight rows on the lanes of tensor
//    memory, a tile of NT tokens as the N operand, so that a small batch wastes
//    no tensor rows;
//  - many tokens (TOK): 128 tokens on the lanes and 256 weight rows (gate 128 and
//    up 128, or 256 neighbours) as the N operand. An MMA of N <= 128 takes about
//    90 cycles whatever its N, one of N = 256 about 128, so this orientation does
//    the same products in 4 MMAs a stage instead of 8; and a lane holds whole
//    32-value blocks of its token, which quantises h without any exchange.
//
// A block: a thread of warp 0 keeps the tokens of a ring of stages coming (256
// columns: codes by tensor TMA in the 128-byte swizzle, scale tiles by plain bulk
// copies), a thread of each of the last warps the same of one weight operand; one
// thread of warp 1 moves the scales into tensor memory (tcgen05.cp) and issues the
// MMAs, warps 2.. read the accumulators and write the outputs (4 of them cover the
// 128 lanes of tensor memory; each group of 4 takes a part of the columns).
// Blocks are persistent: tile i of block b is b + i * gridDim. With the weights on the
// lanes the accumulators are a ring of two tiles, so that the MMAs of a tile run beside
// the epilogue of the one before. With the tokens on the lanes tensor memory holds one
// accumulator of 256 columns beside the scales: the next tile's MMAs wait until the
// epilogue has read it and run beside its packing and stores only.
//
// What bounds it. Few tokens: the weights' way from HBM; 64 tokens over 128 experts
// (H 2048, I 768) read 181.5 MB for gate and up in 34 us and 90.4 MB for down in
// 23 us. Many tokens: shared memory, into which a stage brings 51 KB while its MMAs
// read 48 KB (690 cycles, 512 of them the MMAs'; a third less to load or a quarter of
// the MMAs takes only 4 or 5 us off 53, both 11), the reads of the accumulator, which
// hold up the MMAs, and the stores, which hold up the loads of the next tile (11 us):
// 8192 x 4096 x 4096 takes 52 us (5.3 PFLOP/s; tensor pipe active 63 % of cycles; its
// 65536 MMAs alone 27 us), gate/up of 4096 x 8 pairs 64 us, down 70 us, of it the
// fp32 rows' 268 MB. A plain bulk copy holds its thread for about 270 cycles, so the
// copies of a stage are spread over threads.
#include <cuda.h>

#include <algorithm>

#include "host.hpp"
#include "mxfp4.cuh"
#include "sort.cuh"
#include "tc.cuh"

namespace si {

constexpr int kMmStageK = 256;         // columns of a stage: 128 bytes of codes per row
constexpr int kMmABytes = 128 * 128;   // 128 weight rows of a stage

enum MmMode {
  kMmPlain = 0,
  kMmGateUp = 1,
  kMmStaged = 2,   // TOK: plain, its stores through shared memory (mm_launch_tok)
};

// MA: 128-row weight tiles of a block's tile (gate and up, or two neighbours).
// NT: tokens of a tile. TOK: the tokens on the lanes (NT = 128).
template <int MODE, int MA, int NT, bool TOK> struct MmCfg {
  static_assert(!TOK || (MA == 2 && NT == 128), "128 tokens by 256 weight rows");
  static_assert(MODE != kMmGateUp || TOK || NT == 16, "the SwiGLU epilogue takes 16 tokens");
  static_assert(MODE != kMmStaged || TOK, "weights on the lanes: kMmPlain stages its 2-byte outputs itself");
  // epilogue warps: 4 for the lanes, times the parts of the columns. TOK: a part
  // is 64 columns, which fit into registers, so that the accumulator is free
  // before it is written; otherwise parts of the tokens.
  static constexpr int kParts = TOK ? 4 : NT >= 32 ? 2 : 1;
  static constexpr int kEpiWarps = 4 * kParts;
  static constexpr int kWeightWarp = 2 + kEpiWarps;
  static constexpr int kThreads = 32 * (kWeightWarp + MA);   // TOK: 20 warps, which leave 96 registers a thread
  static constexpr int kBBytes = NT * 128;
  static constexpr int kSfBytes = 2 * kMxTileBytes;               // per operand tile and stage
  static constexpr int kStage = MA * kMmABytes + kBBytes + (MA + 1) * kSfBytes;
  // 16-token groups of an epilogue warp's part, all read at once; staging for
  // two of them at a time (16 tokens x 32 features of 2 bytes each)
  static constexpr int kGroups = NT < 16 * kParts ? 1 : NT / 16 / kParts;
  static constexpr int kEpiBytes = MODE == kMmStaged ? 1024 : MODE == kMmGateUp || TOK ? 0 : kGroups == 1 ? 1024 : 2048;
  static constexpr int kMaxSmem = 227 * 1024 - kEpiWarps * kEpiBytes - 1536;   // less alignment and barriers
  static constexpr int kStages = kMaxSmem / kStage < 8 ? kMaxSmem / kStage : 8;
  // tensor memory: accumulators (a tile takes one of 256 columns, of which one fits, or
  // MA of NT columns, a ring of two tiles), then the scales of every stage (a column holds 4 blocks of 32
  // rows: 128 rows x 8 blocks take 8 columns)
  static constexpr int kAccCols = TOK ? 256 : NT;
  static constexpr int kTileAccs = TOK ? 1 : MA;
  static constexpr int kSfCols = 8 * (MA + 1);
  static constexpr int kFit = (512 - kStages * kSfCols) / kAccCols;
  static constexpr int kAccs = kFit < 2 * kTileAccs ? kFit : 2 * kTileAccs;
  static constexpr int kUsed = kAccs * kAccCols + kStages * kSfCols;
  static constexpr int kCols = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  static_assert(kAccs >= kTileAccs && kUsed <= 512, "tensor memory has 512 columns");
  static_assert(TOK ? kAccs == 1 : kAccs == 2 * MA, "one tile with the tokens on the lanes, else two");
  static constexpr int kBars = 2 * kStages + 2 * kAccs + 1;
  static constexpr int kSmem = kStages * kStage + kEpiWarps * kEpiBytes + 1024 + 512;
  static_assert(8 * kBars + 4 <= 512, "barriers");
};

struct MmParams {
  CUtensorMap a0, a1, b;               // weight rows [mats][rows][K / 2], token rows [..][K / 2]
  const uint8_t *sa0, *sa1, *sb;       // their scale tiles
  int rows, row_tiles;                 // weight rows of a matrix; its 128-row scale tiles
  int n_rt;                            // tiles along the weight rows
  int K, kt;                           // columns; scale tiles along them
  // tokens: a dense batch of `tokens`, or the tiles of a sorted one
  int64_t tokens;
  const int32_t *tile_expert, *tile_count, *n_tiles;
  // plain: out[token][feature]
  void *out;
  int64_t ld;
  int wide;                            // rows of whole 32-byte words
  // gate/up: the MXFP4 rows of h
  uint8_t *h_codes, *h_scales;
  int h_kt;
  uint32_t *status;
  int early;                           // the tile list and the weights are complete before the wait
};

struct MmTile {
  int rt, tt, mat, count;
};

SI_DEV int mm_total(const MmParams &p, int nt) {
  const int n_tt = p.n_tiles ? __ldcg(p.n_tiles) : static_cast<int>((p.tokens + nt - 1) / nt);
  return n_tt * p.n_rt;
}
SI_DEV MmTile mm_tile(const MmParams &p, int w, int nt) {
  MmTile t;
  t.rt = w % p.n_rt;
  t.tt = w / p.n_rt;
  if (p.n_tiles) {
    t.mat = __ldcg(p.tile_expert + t.tt);
    t.count = __ldcg(p.tile_count + t.tt);
  } else {
    const int64_t left = p.tokens - static_cast<int64_t>(t.tt) * nt;
    t.mat = 0;
    t.count = left < nt ? static_cast<int>(left) : nt;
  }
  return t;
}

SI_DEV void tma_load3(void *dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_addr(bar))
      : "memory");
}
SI_DEV void mbar_arrive(uint64_t *bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Shared-memory matrix descriptors (bits as in umma_desc_kmajor): low words,
// with the address, and the high words, which are constants.
//  - codes: K-major, 128-byte swizzle (layout 2), rows of 128 bytes, 8-row
//    groups 1024 bytes apart;
//  - a scale tile: no swizzle, 32 rows of 16 bytes, 8-row groups 128 bytes apart.
constexpr uint32_t kMmCodesHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kMmScaleHi = (128u >> 4) | (1u << 14);
SI_DEV uint32_t mm_codes_lo(uint32_t addr) { return (addr >> 4) | (1u << 16); }
SI_DEV uint32_t mm_scale_lo(uint32_t addr) { return addr >> 4; }
// One lane of a converged warp. The MMA warp runs its loops together and only
// this lane issues: the operands then are uniform values, which the tensor
// instructions take as they are (a single-lane loop converts each of them for
// each instruction and cannot feed the tensor core).
SI_DEV bool elect_lane() {
  uint32_t is;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(is));
  return is != 0;
}
// 512 bytes of scales to 4 columns of tensor memory, on all four 32-lane quarters.
SI_DEV void mm_copy_sf(uint32_t taddr, uint32_t lo) {
  asm volatile("{\n .reg .b64 d;\n mov.b64 d, {%1, %2};\n"
               " tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d;\n}\n" ::"r"(taddr),
               "r"(lo), "n"(kMmScaleHi)
               : "memory");
}
// Instruction descriptor, kind::mxf4: E2M1 operands (bits [7,10), [10,12)),
// K-major, N >> 3 in [17,23), E8M0 scales (bit 23), M >> 4 in [24,29); the scale
// pair of a 4-byte column (blocks 0-1 or 2-3) in [29,31) for A and [4,6) for B.
SI_DEV uint32_t mm_idesc(int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | ((128u >> 4) << 24);
}
// D[tmem] (+)= A B^T over 64 columns, one thread.
SI_DEV void mm_mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n mov.b64 da, {%1, %7};\n mov.b64 db, {%2, %7};\n"
      " setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], da, db, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc), "n"(kMmCodesHi)
      : "memory");
}
// 16 consecutive fp32 columns of this warp's 32 lanes; the wait is separate so
// that two loads can be in flight.
SI_DEV void tmem_ld16(uint32_t taddr, uint32_t r[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
SI_DEV void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---- epilogues ---------------------------------------------------------------

// Outputs whose rows start on 16-byte boundaries leave in 16-byte words (2-byte
// types: VEC); other rows value by value, lane = feature.
enum MmOut { kMmBf16, kMmF16, kMmF32, kMmBf16Vec, kMmF16Vec, kMmF32Vec };

template <int OUT> SI_DEV void mm_store(void *out, int64_t at, float v) {
  if constexpr (OUT == kMmBf16) static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
  else if constexpr (OUT == kMmF32) static_cast<float *>(out)[at] = v;
  else static_cast<__half *>(out)[at] = __float2half_rn(v);
}
template <int OUT> SI_DEV uint32_t mm_pack(uint32_t lo, uint32_t hi) {
  uint32_t w;
  if constexpr (OUT == kMmBf16Vec)
    asm("cvt.rn.bf16x2.f32 %0, %2, %1;" : "=r"(w) : "f"(__uint_as_float(lo)), "f"(__uint_as_float(hi)));
  else
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(w) : "f"(__uint_as_float(lo)), "f"(__uint_as_float(hi)));
  return w;
}
// 16 lanes x 16 columns of tensor memory in the fragment order of an 8 x 8
// matrix store: register 4c + 2h + i of lane l is row 8h + l / 4, column
// 8c + 2 (l % 4) + i.
SI_DEV void tmem_ld_frag(uint32_t taddr, uint32_t r[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

// One accumulator (128 features x count tokens) of this warp's 32 features, the
// warp's part of the tokens. release() once everything is in registers.
template <int OUT, typename C, typename Release>
SI_DEV void mm_write_plain(const MmParams &p, int f0, int64_t row0, int count, uint32_t acc, int part, int lane,
                           uint8_t *stage, Release release) {
  constexpr int G = C::kGroups;
  const int j0 = 16 * G * part;
  const int left = f0 < p.rows ? count - j0 : 0;        // of this warp's tokens
  if constexpr (OUT == kMmBf16Vec || OUT == kMmF16Vec) {
    // 8 x 8 blocks transposed through shared memory: a token's 32 features are
    // 64 bytes, its four 16-byte words permuted by the token so that neither
    // side of the staging meets a bank twice
    uint32_t lo[G][8], hi[G][8];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (16 * i >= left) break;
      tmem_ld_frag(acc + j0 + 16 * i, lo[i]);
      tmem_ld_frag(acc + (16u << 16) + j0 + 16 * i, hi[i]);
    }
    tmem_wait_ld();
    release();
    const int wj = lane & 7, wc = lane >> 3;            // this lane's row address: token wj, word wc
    const int rj = lane >> 2, rc = lane & 3;            // the word that it writes out
    const uint32_t put = smem_addr(stage + wj * 64 + ((wc ^ ((wj >> 1) & 3)) * 16));
    const uint8_t *get = stage + rj * 64 + ((rc ^ ((rj >> 1) & 3)) * 16);
    uint16_t *out = static_cast<uint16_t *>(p.out) + (row0 + j0 + rj) * p.ld + f0 + 8 * rc;
    const bool in = f0 + 8 * rc < p.rows;               // rows % 8 == 0: a word is whole or absent
#pragma unroll
    for (int i0 = 0; i0 < G; i0 += 2) {
      if (16 * i0 >= left) break;
      constexpr int kN = G == 1 ? 2 : 4;                // 8-token blocks of a round
      __syncwarp();                                     // the staging has been read
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        const int i = i0 + c / 2;
        if (i >= G) break;
        const uint32_t *l = lo[i] + 4 * (c & 1), *h = hi[i] + 4 * (c & 1);
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(put + c * 512),
                     "r"(mm_pack<OUT>(l[0], l[1])), "r"(mm_pack<OUT>(l[2], l[3])), "r"(mm_pack<OUT>(h[0], h[1])),
                     "r"(mm_pack<OUT>(h[2], h[3]))
                     : "memory");
      }
      __syncwarp();
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        if (i0 + c / 2 >= G) break;
        const int j = 16 * i0 + 8 * c;
        const uint4 v = *reinterpret_cast<const uint4 *>(get + c * 512);
        if (in && j + rj < left) *reinterpret_cast<uint4 *>(out + j * p.ld) = v;
      }
    }
  } else {
    uint32_t r[G][16];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      if (16 * i >= left) break;
      tmem_ld16(acc + j0 + 16 * i, r[i]);
    }
    tmem_wait_ld();
    release();
    if (f0 + lane < p.rows) {
#pragma unroll
      for (int j = 0; j < 16 * G; ++j)
        if (j < left) mm_store<OUT>(p.out, (row0 + j0 + j) * p.ld + f0 + lane, __uint_as_float(r[j / 16][j % 16]));
    }
  }
}

// 8 x 8 nibbles over 8 consecutive lanes: nibble c of lane r to nibble r of lane c.
SI_DEV uint32_t transpose_nibbles(uint32_t w, int lane) {
  uint32_t o = __shfl_xor_sync(0xffffffffu, w, 4);
  w = lane & 4 ? (w & 0xFFFF0000u) | (o >> 16) : (w & 0x0000FFFFu) | (o << 16);
  o = __shfl_xor_sync(0xffffffffu, w, 2);
  w = lane & 2 ? (w & 0xFF00FF00u) | ((o >> 8) & 0x00FF00FFu) : (w & 0x00FF00FFu) | ((o & 0x00FF00FFu) << 8);
  o = __shfl_xor_sync(0xffffffffu, w, 1);
  return lane & 1 ? (w & 0xF0F0F0F0u) | ((o >> 4) & 0x0F0F0F0Fu) : (w & 0x0F0F0F0Fu) | ((o & 0x0F0F0F0Fu) << 4);
}

// silu(g) u: ex2 and rcp of the hardware, each within 2 units in the last place.
// g below -87 (|silu(g)| < 2^-119): the reciprocal, below the normal range, is 0.
SI_DEV float mm_silu_mul(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return g * r * u;
}

// h = silu(g) u of a lane's feature for up to 16 tokens, then MXFP4: the 32 lanes
// of the warp are one block of every token, so its scale is a warp maximum. Lane j
// keeps the scale of token j and its multiplier, which the others fetch.
SI_DEV void mm_write_h(const MmParams &p, const MmTile &t, uint32_t acc_g, uint32_t acc_u, int q, int lane) {
  const int64_t row0 = static_cast<int64_t>(t.tt) * 16;
  const int blk = t.rt * 4 + q;                 // this warp's block of 32 features
  const size_t row_bytes = static_cast<size_t>(p.rows) / 2;
  uint8_t *sf = p.h_scales + (static_cast<size_t>(t.tt) * p.h_kt + t.rt) * kMxTileBytes;
  const bool mine = lane < 16 && lane < t.count;
  if (blk * 32 >= p.rows) {                     // behind the last feature (rows % 32 == 0): scales that multiply zeros
    if (mine) sf[mx_scale_byte(lane, blk)] = 0;
    return;
  }
  uint32_t g[16], u[16];
  tmem_ld16(acc_g, g);
  tmem_ld16(acc_u, u);
  tmem_wait_ld();
  float h[16];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    h[j] = mm_silu_mul(__uint_as_float(g[j]), __uint_as_float(u[j]));
    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(h[j]) & 0x7FFFFFFFu);
    if ((lane & 15) == j) top = m;
  }
  const uint32_t s = mx_scale_of(top);
  const float up = mx_inv_scale(s);
  const uint32_t bad = __ballot_sync(0xffffffffu, s == 255u);   // tokens with an infinity or a NaN
  if (mine) sf[mx_scale_byte(lane, blk)] = static_cast<uint8_t>(s);
#pragma unroll
  for (int j = 0; j < 16; ++j) h[j] *= __shfl_sync(0xffffffffu, up, j);
#pragma unroll
  for (int h8 = 0; h8 < 16; h8 += 8) {
    uint32_t w = mx_codes8(h + h8);
    if (bad) {                                  // their codes are 0
      for (int j = 0; j < 8; ++j)
        if (bad >> (h8 + j) & 1u) w &= ~(15u << (4 * j));
    }
    w = transpose_nibbles(w, lane);
    const int j = h8 + (lane & 7);
    if (j < t.count)
      *reinterpret_cast<uint32_t *>(p.h_codes + (row0 + j) * row_bytes + blk * 16 + (lane >> 3) * 4) = w;
  }
}

// ---- epilogues, tokens on the lanes ---------------------------------------------

SI_DEV void tmem_ld32(uint32_t taddr, uint32_t r[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// 32 bytes of a row: one sector, one store (mm_launch_tok says when). Not kept in
// the L1, which the ring of stages shares: 8192 x 4096 x 4096 with its quantisation
// 73.0 -> 72.1 us.
SI_DEV void st_global32(void *p, const uint32_t w[8]) {
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 64 features (from f0) of this lane's token `j`, 32 at a time; 2-byte
// outputs wait, packed, until all are read.
template <int OUT, typename Release>
SI_DEV void mm_write_tokens(const MmParams &p, int f0, int64_t row0, int j, bool valid, uint32_t acc, Release release) {
  constexpr int kSize = OUT == kMmF32Vec ? 4 : 2;
  constexpr int kPer = 32 / kSize;               // values of a 32-byte word
  constexpr int kWords = 8 * kSize;              // words of 32 features
  const bool any = f0 < p.rows;
  uint8_t *out = static_cast<uint8_t *>(p.out) + ((row0 + j) * p.ld + f0) * kSize;
  auto write = [&](int c0, const uint32_t *w) {  // features f0 + c0 .. + 31
#pragma unroll
    for (int c = 0; c < 32; c += kPer, w += 8) {
      if (f0 + c0 + c >= p.rows) break;
      uint8_t *o = out + (c0 + c) * kSize;
      const bool whole = f0 + c0 + c + kPer <= p.rows;
      if (p.wide && whole) {
        st_global32(o, w);
      } else {                                   // rows of 16-byte words
        *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
        if (whole) *reinterpret_cast<uint4 *>(o + 16) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  };
  uint32_t w[2][kWords];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (any) {
      uint32_t r[32];
      tmem_ld32(acc + 32 * h, r);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (OUT == kMmF32Vec) w[h][i] = r[i];
        else w[h][i] = mm_pack<OUT>(r[2 * i], r[2 * i + 1]);
      }
    }
    if (h == 1) release();
    if (OUT == kMmF32Vec && any && valid) write(32 * h, w[h]);
  }
  if (OUT != kMmF32Vec && any && valid) {
    write(0, w[0]);
    write(32, w[1]);
  }
}

// 64 features (from f0) of the warp's 32 tokens (lane = token, from row0, `left`
// of them in the batch), 32 at a time; 2-byte outputs wait, packed, until all are
// read. 128 bytes of 8 tokens at a time go through the warp's staging (words
// permuted by the token: no bank met twice), so that a store writes 4 whole
// 128-byte pieces of rows.
template <int OUT, typename Release>
SI_DEV void mm_write_tokens_staged(const MmParams &p, int f0, int64_t row0, int left, uint32_t acc, int lane,
                                   uint8_t *stage, Release release) {
  constexpr int kSize = OUT == kMmF32Vec ? 4 : 2;
  constexpr int kWords = 8 * kSize;              // words of 32 features
  const bool any = f0 < p.rows && left > 0;
  auto write = [&](int c0, const uint32_t *w) {  // features f0 + c0 .. + 128 / kSize - 1
    const int r = lane >> 3, c = lane & 7;       // the word that this lane writes out, of tokens r and r + 4
    const bool in = f0 + c0 + c * (16 / kSize) < p.rows;   // whole words (rows * kSize % 16 == 0)
    uint8_t *out = static_cast<uint8_t *>(p.out) + ((row0 + r) * p.ld + f0 + c0) * kSize + c * 16;
#pragma unroll
    for (int t = 0; t < 32; t += 8) {
      if (t >= left) break;
      __syncwarp();                              // the staging has been read
      if ((lane & 24) == t) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4 *>(stage + c * 128 + ((i ^ c) * 16)) =
              make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(stage + (r + i) * 128 + ((c ^ (r + i)) * 16));
        if (in && t + i + r < left) *reinterpret_cast<uint4 *>(out + (t + i) * p.ld * kSize) = v;
      }
    }
  };
  uint32_t w[2 * kWords];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (any) {
      uint32_t r[32];
      tmem_ld32(acc + 32 * h, r);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (OUT == kMmF32Vec) w[h * kWords + i] = r[i];
        else w[h * kWords + i] = mm_pack<OUT>(r[2 * i], r[2 * i + 1]);
      }
    }
    if (h == 1) release();
    if (OUT == kMmF32Vec && any) write(32 * h, w + h * kWords);
  }
  if (OUT != kMmF32Vec && any) write(0, w);
}

// h = silu(g) u of one block of 32 features of this lane's token, as MXFP4: the
// block lies in this lane's registers.
template <typename Release>
SI_DEV void mm_write_h_tokens(const MmParams &p, const MmTile &t, int blk, int j, bool valid, uint32_t acc_g,
                              uint32_t acc_u, Release release) {
  const bool live = blk * 32 < p.rows;           // rows % 32 == 0
  float h[32];
  uint32_t top = 0;
  if (live) {
#pragma unroll
    for (int i0 = 0; i0 < 32; i0 += 16) {
      uint32_t g[16], u[16];
      tmem_ld16(acc_g + i0, g);
      tmem_ld16(acc_u + i0, u);
      tmem_wait_ld();
      if (i0 == 16) release();                   // the next tile's MMAs run beside the rest
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        h[i0 + i] = mm_silu_mul(__uint_as_float(g[i]), __uint_as_float(u[i]));
        top = max(top, __float_as_uint(h[i0 + i]) & 0x7FFFFFFFu);
      }
    }
  }
  if (!live) release();
  if (!valid) return;
  uint8_t *sf = p.h_scales + (static_cast<size_t>(t.tt) * p.h_kt + t.rt) * kMxTileBytes + mx_scale_byte(j, blk);
  if (!live) {                                   // behind the last feature: a scale that multiplies zeros
    *sf = 0;
    return;
  }
  const uint32_t s = mx_scale_of(top);
  const float up = mx_inv_scale(s);
#pragma unroll
  for (int i = 0; i < 32; ++i) h[i] *= up;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = s == 255u ? 0u : mx_codes8(h + 8 * i);
  *reinterpret_cast<uint4 *>(p.h_codes + (static_cast<size_t>(t.tt) * 128 + j) * (static_cast<size_t>(p.rows) / 2) +
                             blk * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  *sf = static_cast<uint8_t>(s);
}

// ---- the kernel ----------------------------------------------------------------

// The tiles of weight rows that tile t of the list reads, and of them the ones
// inside the matrix.
template <int MODE, int MA> SI_DEV int mm_operands(const MmParams &p, const MmTile &t) {
  return MODE == kMmGateUp || MA == 1 || t.rt * MA * 128 + 128 < p.rows ? MA : 1;
}

template <int MODE, int MA, int NT, bool TOK, int OUT>
__global__ void __launch_bounds__(MmCfg<MODE, MA, NT, TOK>::kThreads, 1)
    mxfp4_mm_kernel(const __grid_constant__ MmParams p) {
  using C = MmCfg<MODE, MA, NT, TOK>;
  constexpr int S = C::kStages, U = C::kAccs;
  extern __shared__ uint8_t mm_smem[];
  uint8_t *base = mm_smem + ((1024u - (smem_addr(mm_smem) & 1023u)) & 1023u);
  uint8_t *staging = base + S * C::kStage;
  uint64_t *full = reinterpret_cast<uint64_t *>(staging + C::kEpiWarps * C::kEpiBytes);
  uint64_t *empty = full + S, *acc_full = empty + S, *acc_empty = acc_full + U, *drain = acc_empty + U;
  uint32_t *s_taddr = reinterpret_cast<uint32_t *>(drain + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_ks = (p.K + kMmStageK - 1) / kMmStageK;
  // the weight operand that this warp brings
  const int operand = warp - C::kWeightWarp;

  // the copies of stage ks of a tile, codes and scales: a thread for the tokens and
  // one for each weight operand, which all arrive at the full barrier of the stage
  auto load_tokens = [&](const MmTile &t, int ks, int s) {
    uint8_t *sb = base + s * C::kStage + MA * kMmABytes;
    const uint32_t bytes = min(2, p.kt - 2 * ks) * kMxTileBytes;
    mbar_arrive_expect_tx(full + s, C::kBBytes + bytes);
    tma_load3(sb, &p.b, ks * 128, t.tt * NT, 0, full + s);
    bulk_g2s(sb + C::kBBytes + MA * C::kSfBytes, p.sb + (static_cast<size_t>(t.tt) * p.kt + 2 * ks) * kMxTileBytes,
             bytes, full + s);
  };
  auto load_weights = [&](const MmTile &t, int na, int ks, int s) {   // of this warp's operand
    if (operand >= na) {
      mbar_arrive(full + s);         // no such weights in this tile
      return;
    }
    const bool up = MODE == kMmGateUp && operand == 1;
    const int rt = MODE == kMmGateUp ? t.rt : t.rt * MA + operand;
    const uint32_t bytes = min(2, p.kt - 2 * ks) * kMxTileBytes;
    uint8_t *st = base + s * C::kStage;
    mbar_arrive_expect_tx(full + s, kMmABytes + bytes);
    tma_load3(st + operand * kMmABytes, up ? &p.a1 : &p.a0, ks * 128, rt * 128, t.mat, full + s);
    bulk_g2s(st + MA * kMmABytes + C::kBBytes + operand * C::kSfBytes,
             (up ? p.sa1 : p.sa0) + (static_cast<size_t>(t.mat * p.row_tiles + rt) * p.kt + 2 * ks) * kMxTileBytes,
             bytes, full + s);
  };

  int ahead = 0;                     // stages whose weights were requested before the wait
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(full + i, 1 + MA);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < U; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, C::kEpiWarps);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (p.early) {                     // uniform over the grid
    __syncthreads();
    if (lane == 0 && operand >= 0 && static_cast<int>(blockIdx.x) < mm_total(p, NT)) {
      const MmTile t = mm_tile(p, blockIdx.x, NT);
      const int na = mm_operands<MODE, MA>(p, t);
      for (; ahead < S && ahead < n_ks; ++ahead) load_weights(t, na, ahead, ahead);
    }
  }
  grid_dep_wait();
  if (warp == 1) {
    // before the next kernel may start: its blocks take tensor memory too
    tmem_alloc(s_taddr, C::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *s_taddr, 0);
  const int total = mm_total(p, NT);

  // every role reads a tile's entry of the list one tile ahead
  const int step = gridDim.x;
  const MmTile none = {0, 0, 0, 0};
  MmTile nx = static_cast<int>(blockIdx.x) < total ? mm_tile(p, blockIdx.x, NT) : none;
  auto next_tile = [&](int w) {
    const MmTile t = nx;
    if (w + step < total) nx = mm_tile(p, w + step, NT);
    return t;
  };

  if (warp == 0 || operand >= 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int w = blockIdx.x; ok && w < total; w += step) {
        const MmTile t = next_tile(w);
        const int na = mm_operands<MODE, MA>(p, t);
        for (int ks = 0; ks < n_ks; ++ks, ++it) {
          const int s = it % S;
          const bool fresh = static_cast<int>(it) >= ahead;
          if (fresh && !mbar_wait_bounded(empty + s, ((it / S) & 1) ^ 1, p.status)) {
            ok = false;
            break;
          }
          if (warp == 0) load_tokens(t, ks, s);
          else if (fresh) load_weights(t, na, ks, s);
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
      const MmTile t = next_tile(w);
      const int na = mm_operands<MODE, MA>(p, t);
      const int nu = TOK ? 1 : na;   // accumulators of this tile
      uint32_t d[C::kTileAccs];
#pragma unroll
      for (int a = 0; a < C::kTileAccs; ++a) {
        const uint32_t u = (n + a) % U;
        d[a] = tmem + u * C::kAccCols;
        if (leader && a < nu && ok) ok = mbar_wait_bounded(acc_empty + u, (((n + a) / U) & 1) ^ 1, p.status);
      }
      const uint32_t idesc = mm_idesc(TOK ? 128 * na : (t.count + 15) & ~15);
      for (int ks = 0; ks < n_ks; ++ks) {
        const int n64 = min(4, (p.K - ks * kMmStageK + 63) / 64);
        const uint32_t st = smem0 + s * C::kStage;
        const uint32_t sf = mm_scale_lo(st + MA * kMmABytes + C::kBBytes);
        const uint32_t ca = mm_codes_lo(st), cb = mm_codes_lo(st + MA * kMmABytes);
        const uint32_t tsf = tmem + U * C::kAccCols + s * C::kSfCols;
        const uint32_t more = ks > 0;
        // columns of operand a's scales: TOK keeps the two weight tiles of a 128-column
        // piece side by side, the 256 rows of one operand
        auto sf_cols = [&](int kt, int a) { return TOK && a < MA ? tsf + kt * 8 + a * 4 : tsf + a * 8 + kt * 4; };
        auto copy_sf = [&](int kt, int a) {
          mm_copy_sf(sf_cols(kt, a), sf + (a * C::kSfBytes + kt * kMxTileBytes) / 16);
        };
        auto mma = [&](int i, int a) {
          const uint32_t id = idesc | (static_cast<uint32_t>(i & 1) * 2u << 29) | (static_cast<uint32_t>(i & 1) * 2u << 4);
          const uint32_t acc = i > 0 ? 1u : more;
          if constexpr (TOK)
            mm_mma(d[0], cb + i * 32 / 16, ca + i * 32 / 16, id, sf_cols(i >> 1, MA), sf_cols(i >> 1, 0), acc);
          else
            mm_mma(d[a], ca + (a * kMmABytes + i * 32) / 16, cb + i * 32 / 16, id, sf_cols(i >> 1, a),
                   sf_cols(i >> 1, MA), acc);
        };
        if (leader && ok) ok = mbar_wait_bounded(full + s, parity, p.status);
        if (leader && ok) {
          tc_fence_after();
          if (n64 == 4 && na == MA) {
#pragma unroll
            for (int i = 0; i < 2 * (MA + 1); ++i) copy_sf(i / (MA + 1), i % (MA + 1));
#pragma unroll
            for (int i = 0; i < 4 * C::kTileAccs; ++i) mma(i / C::kTileAccs, i % C::kTileAccs);
          } else {                   // the last columns, or the last rows of an odd number of tiles
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
              if (2 * kt >= n64) break;
#pragma unroll
              for (int a = 0; a <= MA; ++a)
                if (a < na || a == MA) copy_sf(kt, a);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i >= n64) break;
#pragma unroll
              for (int a = 0; a < C::kTileAccs; ++a)
                if (a < nu) mma(i, a);
            }
          }
          umma_commit(empty + s);
        }
        if (++s == S) {
          s = 0;
          parity ^= 1;
        }
      }
      if (leader && ok)
        for (int a = 0; a < nu; ++a) umma_commit(acc_full + (n + a) % U);
      n += nu;
    }
    if (leader && !ok) {   // MMAs in flight end before the tensor memory goes
      umma_commit(drain);
      mbar_wait_bounded(drain, 0, p.status);
    }
    __syncwarp();
  } else {
    const int q = warp & 3, part = (warp - 2) >> 2;   // the 32 lanes of tensor memory this warp may read
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
    uint8_t *stage = staging + (warp - 2) * C::kEpiBytes;
    uint32_t n = 0;
    bool ok = true;
    auto wait_acc = [&](uint32_t i) {
      ok = __all_sync(0xffffffffu, mbar_wait_bounded(acc_full + i % U, (i / U) & 1, p.status));
      tc_fence_after();
      return lanes + (i % U) * C::kAccCols;
    };
    auto free_acc = [&](uint32_t i) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty + i % U);
    };
    for (int w = blockIdx.x; ok && w < total; w += step) {
      const MmTile t = next_tile(w);
      if constexpr (TOK) {
        const uint32_t acc = wait_acc(n);
        if (!ok) break;
        const int j = q * 32 + lane;
        auto release = [&] { free_acc(n); };
        if constexpr (MODE == kMmGateUp)
          mm_write_h_tokens(p, t, t.rt * 4 + part, j, j < t.count, acc + part * 32, acc + 128 + part * 32, release);
        else if constexpr (MODE == kMmStaged)
          mm_write_tokens_staged<OUT>(p, t.rt * 256 + part * 64, static_cast<int64_t>(t.tt) * NT + q * 32,
                                      t.count - q * 32, acc + part * 64, lane, stage, release);
        else
          mm_write_tokens<OUT>(p, t.rt * 256 + part * 64, static_cast<int64_t>(t.tt) * NT, j, j < t.count,
                               acc + part * 64, release);
        ++n;
      } else if constexpr (MODE == kMmGateUp) {
        const uint32_t g = wait_acc(n);
        if (!ok) break;
        const uint32_t u = wait_acc(n + 1);
        if (!ok) break;
        mm_write_h(p, t, g, u, q, lane);
        free_acc(n);
        free_acc(n + 1);
        n += 2;
      } else {
        const int na = mm_operands<MODE, MA>(p, t);
        for (int a = 0; a < na; ++a, ++n) {
          const uint32_t acc = wait_acc(n);
          if (!ok) break;
          mm_write_plain<OUT, C>(p, (t.rt * MA + a) * 128 + q * 32, static_cast<int64_t>(t.tt) * NT, t.count, acc, part,
                                 lane, stage, [&] { free_acc(n); });
        }
      }
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

// ---------------------------------------------------------------------------
// x to MXFP4 rows at the sorted places: one block per token quantises its row
// once and writes it to its kept places. Scale tiles belong to one token tile
// each (NT of their 128 rows).
// ---------------------------------------------------------------------------
struct ScatterArgs {
  const __nv_bfloat16 *x;
  int k, H, kt, nt;
  const int32_t *position;
  uint8_t *codes, *scales;
};
struct ScatterRows {
  uint8_t *code[8], *scale[8];   // rows of the token's kept pairs
  int n;
};
// Place p (-1: dropped) of pair `lane` of the token to the list; one whole warp.
SI_DEV void scatter_list(const ScatterArgs &a, int p, int lane, ScatterRows &out) {
  const uint32_t kept = __ballot_sync(0xffffffffu, p >= 0);
  const int at = __popc(kept & ((1u << lane) - 1u));
  if (p >= 0) {
    out.code[at] = a.codes + static_cast<size_t>(p) * a.H / 2;
    out.scale[at] = a.scales + static_cast<size_t>(p / a.nt) * a.kt * kMxTileBytes + mx_scale_byte(p % a.nt, 0);
  }
  if (lane == 0) out.n = __popc(kept);
}
SI_DEV void scatter_row(const ScatterArgs &a, int64_t t, const ScatterRows &to) {
  const int lane = threadIdx.x & 31, n = to.n;
  // whole scale tiles (128 columns, 16 lanes): the blocks behind H get scale 0
  for (int c0 = (threadIdx.x & ~31) * 8; c0 < a.kt * 128; c0 += blockDim.x * 8) {
    const int c = c0 + lane * 8;
    Raw8<__nv_bfloat16> v;
    if (c < a.H) v.load16(a.x + t * a.H + c);
    else v.zero();
    uint32_t s;
    const uint32_t w = mx_encode_4lanes(v, s);
    uint32_t s4 = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) s4 |= __shfl_sync(0xffffffffu, s, (lane & 16) + 4 * b) << (8 * b);
    for (int r = 0; r < n; ++r) {
      if (c < a.H) *reinterpret_cast<uint32_t *>(to.code[r] + c / 2) = w;
      if ((lane & 15) == 0 && c < a.kt * 128) *reinterpret_cast<uint32_t *>(to.scale[r] + c / 128 * kMxTileBytes) = s4;
    }
  }
}
__global__ void __launch_bounds__(256) quantize_scatter_kernel(ScatterArgs a) {
  __shared__ ScatterRows s_rows;
  grid_dep_wait();
  grid_dep_launch();
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) scatter_list(a, lane < a.k ? __ldcg(a.position + t * a.k + lane) : -1, lane, s_rows);
  __syncthreads();
  scatter_row(a, t, s_rows);
}

// At most 32 pairs: the sort too, in the same launch, by one warp of every block
// (a lane per pair); block 0 writes the tile list. The launch that this saves
// counts more there than the weights that gate/up could request before its wait
// with the sort two launches back. In a graph, 1 / 4 tokens: 128 experts, H 2048, I 768,
// top-8 14.6 / 23.9 us against 16.3 / 24.4 with two launches; 256, 2048, 512, top-8 14.8 / 16.8
// against 16.8 / 19.3; 8, 4096, 2048, top-2 19.8 / 26.4 against 20.8 / 27.5. With more pairs it
// turns (128 pairs on the first layer 44.0 against 43.2), and a lane holds one pair.
constexpr int kFewPairs = 32;
__global__ void __launch_bounds__(256) sort_scatter_kernel(SortArgs so, ScatterArgs a) {
  __shared__ ScatterRows s_rows;
  grid_dep_wait();
  grid_dep_launch();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, first = blockIdx.x * a.k;   // this token's pairs: first .. first + k - 1
    const int e = lane < static_cast<int>(so.pairs) ? sort_expert(so, lane) : 0x7FFFFFFF;
    const bool kept = e < so.n_experts;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    const int tiles = kept && rank == 0 ? sort_tiles(so, __popc(same)) : 0;
    int tile = 0;                                             // tiles of the experts before e
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const int ej = __shfl_sync(0xffffffffu, e, j), n = __shfl_sync(0xffffffffu, tiles, j);
      if (ej < e) tile += n;
    }
    const int total = __reduce_add_sync(0xffffffffu, tiles);
    if (blockIdx.x == 0) {
      if (tiles > 0) sort_list(so, e, __popc(same), tile, 0, 1);
      if (lane == 0) *so.n_tiles = total;
    }
    int p = __shfl_sync(0xffffffffu, kept ? tile * so.tile_rows + rank : -1, (first + lane) & 31);
    if (lane < a.k) so.position[first + lane] = p;
    else p = -1;
    scatter_list(a, p, lane, s_rows);
  }
  __syncthreads();
  scatter_row(a, blockIdx.x, s_rows);
}

// ---- host ------------------------------------------------------------------

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
static EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// Codes [mats][rows][cols / 2], boxes of box_rows rows x 128 bytes; what lies
// outside reads as zero.
static bool codes_map(CUtensorMap *m, const void *codes, int64_t mats, int64_t rows, int64_t cols, int box_rows) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols / 2), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(mats)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols / 2), static_cast<cuuint64_t>(cols / 2 * rows)};
  const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(box_rows), 1}, one[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(codes), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int MA, int NT, bool TOK, int OUT>
static cudaError_t mm_launch_as(const MmParams &p, int64_t max_tiles, cudaStream_t s) {
  using C = MmCfg<MODE, MA, NT, TOK>;
  const cudaError_t e = allow_smem(mxfp4_mm_kernel<MODE, MA, NT, TOK, OUT>, C::kSmem);
  if (e != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(max_tiles, sm_count()));
  return launch_pdl(mxfp4_mm_kernel<MODE, MA, NT, TOK, OUT>, dim3(grid), dim3(C::kThreads), C::kSmem, s, p);
}
// The tokens on the lanes. While a tile's columns fit into the ring of stages, the
// next tile's loads are all on their way when the stores come, and these bound
// it: whole 128-byte pieces of rows (16384 x 4096 x 1024 bf16 39.3 against 42.3 us,
// fp32 62.1 against 69.5; x 256: 31.2 against 33.8). With more columns the stores
// stand in the way of the loads, and 32 bytes a lane, straight from the registers,
// do so less (x 1152: 47.9 against 51.8, x 4096: 102.0 against 106.2).
template <int OUT> static cudaError_t mm_launch_tok(const MmParams &p, int64_t max_tiles, cudaStream_t s) {
  return p.K <= MmCfg<kMmStaged, 2, 128, true>::kStages * kMmStageK
             ? mm_launch_as<kMmStaged, 2, 128, true, OUT>(p, max_tiles, s)
             : mm_launch_as<kMmPlain, 2, 128, true, OUT>(p, max_tiles, s);
}
template <int OUT>
static cudaError_t mm_launch_dense(int nt, const MmParams &p, int64_t max_tiles, cudaStream_t s) {
  return nt == 16   ? mm_launch_as<kMmPlain, 1, 16, false, OUT>(p, max_tiles, s)
         : nt == 32 ? mm_launch_as<kMmPlain, 1, 32, false, OUT>(p, max_tiles, s)
         : nt == 64 ? mm_launch_as<kMmPlain, 1, 64, false, OUT>(p, max_tiles, s)
                    : mm_launch_as<kMmPlain, 1, 128, false, OUT>(p, max_tiles, s);
}
static cudaError_t mm_launch_gateup(int nt, const MmParams &p, int64_t max_tiles, cudaStream_t s) {
  return nt == 16 ? mm_launch_as<kMmGateUp, 2, 16, false, 0>(p, max_tiles, s)
                  : mm_launch_as<kMmGateUp, 2, 128, true, 0>(p, max_tiles, s);
}
// 256 rows a tile for few tokens: fewer loads for the same bytes (128 tokens, with
// rows of bf16, 66.2 -> 63.5 us).
// y stays fp32 until the ranks are summed, so that a token's output is rounded once
// (with bf16 rows its error against 64 bits is 0.0024 relative, not 0.0017). Twice
// the bytes: 58.2 against 57.5 us at 64 tokens, 104 against 90 at 1024, 213 against
// 161 at 4096 (128 experts, H 2048, I 768, top-8).
static cudaError_t mm_launch_down(int nt, const MmParams &p, int64_t max_tiles, cudaStream_t s) {
  return nt == 16 ? mm_launch_as<kMmPlain, 2, 16, false, kMmF32>(p, max_tiles, s)
                  : mm_launch_tok<kMmF32Vec>(p, max_tiles, s);
}

// ---- expert FFN: workspace ---------------------------------------------------
struct FfnMxGeom {
  int nt;                   // tokens of a tile
  int64_t pairs, max_tiles, rows;
  int kt_x, kt_h;
  size_t off_position, off_counts, off_expert, off_count, off_n, off_xc, off_xs, off_hc, off_hs, off_y, bytes;
};
static FfnMxGeom ffn_mx_geom(const si_mxfp4_experts &L, int n_tokens, int top_k) {
  FfnMxGeom g{};
  g.pairs = static_cast<int64_t>(n_tokens) * top_k;
  // tiles of 16 tokens while an expert has 8 pairs on average, so that few experts
  // need a second tile; else the tokens on the lanes. In a graph at averages of
  // 8 / 24, tiles of 16 against 128: E 128, H 2048, I 768, top-8 66.3 / 82.0 against 73.4 / 81.7
  // us; 256, 2048, 512, top-8 91.5 / 119.3 against 94.2 / 114.4; 64, 1024, 4096, top-2
  // 78.5 / 98.0 against 81.8 / 88.5; 32, 2880, 1440, top-4 48.6 / 64.0 against 56.7 / 60.0; 8, 4096,
  // 2048, top-2 32.1 / 35.9 against 33.6 / 34.8. In between the layers differ (at 16 the
  // first four still gain 1 to 7 % with tiles of 16, the last loses 6 %).
  const int64_t avg = (g.pairs + L.n_experts - 1) / L.n_experts;
  g.nt = avg <= 8 ? 16 : 128;
  const int64_t with = std::min<int64_t>(L.n_experts, g.pairs);   // experts that can hold pairs
  g.max_tiles = (g.pairs + with * (g.nt - 1)) / g.nt;
  g.rows = g.max_tiles * g.nt;
  g.kt_x = (L.hidden + 127) / 128;
  g.kt_h = (L.inter + 127) / 128;
  size_t off = sizeof(WsHeader);
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = round_up(off + bytes, 256);
    return at;
  };
  g.off_position = take(g.pairs * 4);
  g.off_counts = take(sort_workspace_bytes(g.pairs, L.n_experts));
  g.off_expert = take(g.max_tiles * 4);
  g.off_count = take(g.max_tiles * 4);
  g.off_n = take(4);
  g.off_xc = take(static_cast<size_t>(g.rows) * L.hidden / 2);
  g.off_xs = take(static_cast<size_t>(g.max_tiles) * g.kt_x * kMxTileBytes);
  g.off_hc = take(static_cast<size_t>(g.rows) * L.inter / 2);
  g.off_hs = take(static_cast<size_t>(g.max_tiles) * g.kt_h * kMxTileBytes);
  g.off_y = take(static_cast<size_t>(g.rows) * L.hidden * 4);
  g.bytes = off;
  return g;
}
static bool ffn_mx_shape_ok(const si_mxfp4_experts *L, int n_tokens, int top_k) {
  return L && L->hidden > 0 && L->hidden % 32 == 0 && L->hidden <= 65536 && L->inter > 0 && L->inter % 32 == 0 &&
         L->inter <= 65536 && L->n_experts >= 1 && L->n_experts <= kSortMaxExperts && top_k >= 1 && top_k <= 8 &&
         n_tokens >= 1 && static_cast<int64_t>(n_tokens) * top_k <= (int64_t(1) << 24);
}

}  // namespace si

using namespace si;

extern "C" size_t si_mxfp4_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (m < 1 || n < 1 || k < 32 || k % 32 || m > (int64_t(1) << 30) || n > (int64_t(1) << 30) ||
      k > (int64_t(1) << 20))
    return 0;
  return sizeof(WsHeader);
}

extern "C" si_status si_mxfp4_matmul(const void *a_codes, const void *a_scales, int64_t m, const void *w_codes,
                                     const void *w_scales, int64_t n, int64_t k, void *out, si_dtype out_type,
                                     int64_t ld_out, void *workspace, size_t workspace_bytes, void *stream) {
  const size_t need = si_mxfp4_matmul_workspace_bytes(m, n, k);
  if (!need || !a_codes || !a_scales || !w_codes || !w_scales || !out || ld_out < n || ld_out > (int64_t(1) << 40))
    return SI_ERR_INVALID_ARG;
  if (out_type != SI_F32 && out_type != SI_F16 && out_type != SI_BF16) return SI_ERR_UNSUPPORTED;
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(w_codes) || !aligned16(w_scales) ||
      reinterpret_cast<uintptr_t>(out) % (out_type == SI_F32 ? 4 : 2))
    return SI_ERR_INVALID_ARG;
  if (workspace && (!aligned256(workspace) || workspace_bytes < need)) return SI_ERR_WORKSPACE;
  MmParams p{};
  const int nt = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128;
  const int64_t n_tt = (m + nt - 1) / nt, row_tiles = (n + 127) / 128;
  const int size = out_type == SI_F32 ? 4 : 2;
  const bool vec = n * size % 16 == 0 && ld_out * size % 16 == 0 && aligned16(out);
  // the tokens on the lanes when tiles of 128 x 128 take more than one round of
  // the SMs (k 4096, n 4096: m 1024 10.2 us against 12.9, but m 512 10.0 against
  // 8.1) and the rows can be written in whole words
  const bool tok = nt == 128 && vec && n_tt * row_tiles > sm_count();
  const int ma = tok ? 2 : 1;
  const int64_t n_rt = (row_tiles + ma - 1) / ma;
  if (n_tt * n_rt > (int64_t(1) << 30)) return SI_ERR_UNSUPPORTED;
  if (!codes_map(&p.a0, w_codes, 1, n, k, 128) || !codes_map(&p.b, a_codes, 1, m, k, nt)) return SI_ERR_CUDA;
  p.a1 = p.a0;
  p.sa0 = p.sa1 = static_cast<const uint8_t *>(w_scales);
  p.sb = static_cast<const uint8_t *>(a_scales);
  p.rows = static_cast<int>(n);
  p.row_tiles = static_cast<int>(row_tiles);
  p.n_rt = static_cast<int>(n_rt);
  p.K = static_cast<int>(k);
  p.kt = static_cast<int>((k + 127) / 128);
  p.tokens = m;
  p.out = out;
  p.ld = ld_out;
  p.status = static_cast<uint32_t *>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.wide = ld_out * size % 32 == 0 && (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  const int64_t tiles = n_tt * n_rt;
  if (tok)
    return cuda_status(out_type == SI_F32    ? mm_launch_tok<kMmF32Vec>(p, tiles, s)
                       : out_type == SI_BF16 ? mm_launch_tok<kMmBf16Vec>(p, tiles, s)
                                             : mm_launch_tok<kMmF16Vec>(p, tiles, s));
  return cuda_status(out_type == SI_F32 ? mm_launch_dense<kMmF32>(nt, p, tiles, s)
                     : out_type == SI_BF16
                         ? (vec ? mm_launch_dense<kMmBf16Vec>(nt, p, tiles, s) : mm_launch_dense<kMmBf16>(nt, p, tiles, s))
                         : (vec ? mm_launch_dense<kMmF16Vec>(nt, p, tiles, s) : mm_launch_dense<kMmF16>(nt, p, tiles, s)));
}

extern "C" size_t si_moe_ffn_mxfp4_workspace_bytes(const si_mxfp4_experts *L, int n_tokens, int top_k) {
  return ffn_mx_shape_ok(L, n_tokens, top_k) ? ffn_mx_geom(*L, n_tokens, top_k).bytes : 0;
}

extern "C" si_status si_moe_ffn_mxfp4(const si_mxfp4_experts *L, int n_tokens, int top_k, const void *x,
                                      const int32_t *topk_ids, const float *topk_w, void *routed_out,
                                      void *workspace, size_t workspace_bytes, void *stream) {
  if (!ffn_mx_shape_ok(L, n_tokens, top_k) || !x || !topk_ids || !topk_w || !routed_out) return SI_ERR_INVALID_ARG;
  const void *ws[6] = {L->gate_codes, L->gate_scales, L->up_codes, L->up_scales, L->down_codes, L->down_scales};
  for (const void *w : ws)
    if (!w || !aligned16(w)) return SI_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(routed_out) || (reinterpret_cast<uintptr_t>(topk_ids) & 3u) ||
      (reinterpret_cast<uintptr_t>(topk_w) & 3u))
    return SI_ERR_INVALID_ARG;
  const FfnMxGeom g = ffn_mx_geom(*L, n_tokens, top_k);
  if (!workspace || !aligned256(workspace) || workspace_bytes < g.bytes) return SI_ERR_WORKSPACE;
  if (g.rows > 0x7FFFFFFF) return SI_ERR_UNSUPPORTED;
  uint8_t *base = static_cast<uint8_t *>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int H = L->hidden, I = L->inter, E = L->n_experts;

  MmParams gu{}, dn{};
  if (!codes_map(&gu.a0, L->gate_codes, E, I, H, 128) || !codes_map(&gu.a1, L->up_codes, E, I, H, 128) ||
      !codes_map(&gu.b, base + g.off_xc, 1, g.rows, H, g.nt) || !codes_map(&dn.a0, L->down_codes, E, H, I, 128) ||
      !codes_map(&dn.b, base + g.off_hc, 1, g.rows, I, g.nt))
    return SI_ERR_CUDA;

  SortArgs so{};
  so.ids = topk_ids;
  so.pairs = g.pairs;
  so.n_experts = E;
  so.position = reinterpret_cast<int32_t *>(base + g.off_position);
  so.counts = reinterpret_cast<int32_t *>(base + g.off_counts);
  so.tile_rows = g.nt;
  so.tile_expert = reinterpret_cast<int32_t *>(base + g.off_expert);
  so.tile_count = reinterpret_cast<int32_t *>(base + g.off_count);
  so.n_tiles = reinterpret_cast<int32_t *>(base + g.off_n);
  const ScatterArgs sc{static_cast<const __nv_bfloat16 *>(x), top_k, H, g.kt_x, g.nt, so.position, base + g.off_xc,
                       base + g.off_xs};
  const bool few = g.pairs <= kFewPairs;
  cudaError_t e;
  if (few) {
    e = launch_pdl(sort_scatter_kernel, dim3(n_tokens), dim3(256), 0, s, so, sc);
  } else {
    e = sort_launch(so, s);
    if (e != cudaSuccess) return SI_ERR_CUDA;
    e = launch_pdl(quantize_scatter_kernel, dim3(n_tokens), dim3(256), 0, s, sc);
  }
  if (e != cudaSuccess) return SI_ERR_CUDA;

  gu.sa0 = static_cast<const uint8_t *>(L->gate_scales);
  gu.sa1 = static_cast<const uint8_t *>(L->up_scales);
  gu.sb = base + g.off_xs;
  gu.rows = I;
  gu.row_tiles = gu.n_rt = (I + 127) / 128;
  gu.K = H;
  gu.kt = g.kt_x;
  gu.tile_expert = so.tile_expert;
  gu.tile_count = so.tile_count;
  gu.n_tiles = so.n_tiles;
  gu.h_codes = base + g.off_hc;
  gu.h_scales = base + g.off_hs;
  gu.h_kt = g.kt_h;
  gu.status = reinterpret_cast<uint32_t *>(base);
  // the sort is two launches back: complete when the blocks of its successor have
  // passed their wait, before which this launch does not start
  gu.early = few ? 0 : 1;
  e = mm_launch_gateup(g.nt, gu, g.max_tiles * gu.n_rt, s);
  if (e != cudaSuccess) return SI_ERR_CUDA;

  dn.a1 = dn.a0;
  dn.sa0 = dn.sa1 = static_cast<const uint8_t *>(L->down_scales);
  dn.sb = base + g.off_hs;
  dn.rows = H;
  dn.row_tiles = (H + 127) / 128;
  dn.n_rt = (dn.row_tiles + 1) / 2;
  dn.K = I;
  dn.kt = g.kt_h;
  dn.tile_expert = so.tile_expert;
  dn.tile_count = so.tile_count;
  dn.n_tiles = so.n_tiles;
  dn.out = base + g.off_y;
  dn.ld = H;
  dn.wide = 1;                       // rows of H * 4 bytes, H % 32 == 0
  dn.status = reinterpret_cast<uint32_t *>(base);
  dn.early = 1;
  e = mm_launch_down(g.nt, dn, g.max_tiles * dn.n_rt, s);
  if (e != cudaSuccess) return SI_ERR_CUDA;
  return cuda_status(combine_launch(reinterpret_cast<const float *>(base + g.off_y), g.rows, n_tokens, top_k, H,
                                    so.position, topk_w, routed_out, s));
}
