// Activations kept in 8 bits (MXINT8, mxint8.cuh) for the backward pass, and SwiGLU,
// which keeps its inputs so.
//
//   h = silu(g) u, with s = 1 / (1 + exp(-g)):  silu(g) = g s
//   backwards, from the kept g and u, for rows of weight c (h enters a sum as c h):
//     gg = c gh u s (1 + g (1 - s)),  gu = c gh g s,  ch = c g s u,  gc = <gh, g s u>
//
// All in fp32, rounded once to the rows' type. The row sum gc is formed lane by lane,
// then over the warp, then over the warps of the row in their order: it does not
// depend on how blocks run. A warp takes 256 columns of a row, 8 a lane; 4 lanes hold
// a block of 32 values. All of it is bound by HBM.
#include <algorithm>

#include "host.hpp"
#include "mxint8.cuh"

namespace si {

constexpr int kActThreads = 256;
constexpr int kActCols = 256;        // of a warp's pass
constexpr int kActInFlight = 4;      // passes whose loads are on their way together

// ---- 8 values of a row, of which `n` (0..8) lie inside -----------------------------

template <bool VEC, typename T> SI_DEV void act_load(Raw8<T> &v, const T *p, int n) {
  v.zero();
  if constexpr (VEC) {
    if (n > 0) v.load16(p);
  } else if (n >= 8) {
    v.load(p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i >= n) break;
      if constexpr (sizeof(T) == 4) v.w[i] = __float_as_uint(p[i]);
      else v.w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[i]) << (16 * (i & 1));
    }
  }
}
template <bool VEC, typename T> SI_DEV void act_store(T *p, const float v[8], int n) {
  if constexpr (VEC) {
    if (n <= 0) return;
#pragma unroll
    for (int i = 0; i < 8; i += kVecOf<T>) *reinterpret_cast<uint4 *>(p + i) = pack16<T>(v + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}
template <bool VEC> SI_DEV uint2 act_load_codes(const uint8_t *p, int n) {
  uint2 q = make_uint2(0, 0);
  if constexpr (VEC) {
    if (n > 0) q = __ldg(reinterpret_cast<const uint2 *>(p));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) (i < 4 ? q.x : q.y) |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  }
  return q;
}
template <bool VEC> SI_DEV void act_store_codes(uint8_t *p, uint2 q, int n) {
  if constexpr (VEC) {
    if (n > 0) *reinterpret_cast<uint2 *>(p) = q;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
  }
}
SI_DEV int act_inside(int64_t c, int64_t cols) {
  return static_cast<int>(min(max(cols - c, static_cast<int64_t>(0)), static_cast<int64_t>(8)));
}

// Codes of 8 values of a block that 4 neighbouring lanes hold; every lane of the warp.
template <typename T> SI_DEV uint2 act_encode(const Raw8<T> &x, uint32_t &s) {
  const uint32_t top = mx_top_4lanes(x);
  s = mi_scale_of(top);
  float v[8];
  x.unpack(v);
  uint32_t c[8];
  if (!mi_far(top)) {
    const float up = mi_inv_step(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = mi_code_near(v[i], up);
  } else {
    const float up = mi_inv_scale(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = s == 255u ? 0u : mi_code(v[i] * up);
  }
  return make_uint2(mi_pack4(c[0], c[1], c[2], c[3]), mi_pack4(c[4], c[5], c[6], c[7]));
}
SI_DEV void act_decode(uint2 q, uint32_t s, float v[8]) {
  const float step = mi_step(s);
  mi_values4(q.x, v);
  mi_values4(q.y, v + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= step;
}

// ---- rows to 8 bits and back -------------------------------------------------------

struct ActShape {
  int64_t rows, cols, ld;   // of the float rows, in values
  int64_t passes, units;    // passes of a row; rows * passes
};
struct ActAt {
  int64_t row, c;
  int n;                    // of this lane's 8 columns
};
SI_DEV ActAt act_at(const ActShape &sh, int64_t unit, int lane) {
  ActAt a;
  if (sh.rows == 1) {
    a.row = 0;
    a.c = unit * kActCols + lane * 8;
  } else {
    a.row = (sh.units >> 32) == 0 ? static_cast<uint32_t>(unit) / static_cast<uint32_t>(sh.passes) : unit / sh.passes;
    a.c = (unit - a.row * sh.passes) * kActCols + lane * 8;
  }
  a.n = unit < sh.units ? act_inside(a.c, sh.cols) : 0;
  return a;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kActThreads)
    quantize_mxint8_kernel(const T *__restrict__ x, ActShape sh, uint8_t *__restrict__ codes,
                           uint8_t *__restrict__ scales) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t u0 = (static_cast<int64_t>(blockIdx.x) * (kActThreads / 32) + (threadIdx.x >> 5)) * kActInFlight;
  const int64_t blocks = mi_blocks(sh.cols);
  Raw8<T> v[kActInFlight];
  ActAt a[kActInFlight];
#pragma unroll
  for (int i = 0; i < kActInFlight; ++i) {
    a[i] = act_at(sh, u0 + i, lane);
    act_load<VEC>(v[i], x + a[i].row * sh.ld + a[i].c, a[i].n);
  }
  // the scales of all passes leave together: lane 8 i + b has block b's of pass i
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < kActInFlight; ++i) {
    uint32_t s;
    const uint2 q = act_encode(v[i], s);
    act_store_codes<VEC>(codes + a[i].row * sh.cols + a[i].c, q, a[i].n);
    s = __shfl_sync(0xffffffffu, s, (lane & 7) * 4);
    if (lane >> 3 == i) mine = s;
  }
  static_assert(kActInFlight == 4 && kActCols == 256, "a lane for each block");
  const ActAt at = act_at(sh, u0 + (lane >> 3), (lane & 7) * 4);
  if (at.n > 0) scales[at.row * blocks + (at.c >> 5)] = static_cast<uint8_t>(mine);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kActThreads)
    dequantize_mxint8_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, ActShape sh,
                             T *__restrict__ y) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t u0 = (static_cast<int64_t>(blockIdx.x) * (kActThreads / 32) + (threadIdx.x >> 5)) * kActInFlight;
  const int64_t blocks = mi_blocks(sh.cols);
  uint2 q[kActInFlight];
  uint32_t s[kActInFlight];
  ActAt a[kActInFlight];
#pragma unroll
  for (int i = 0; i < kActInFlight; ++i) {
    a[i] = act_at(sh, u0 + i, lane);
    q[i] = act_load_codes<VEC>(codes + a[i].row * sh.cols + a[i].c, a[i].n);
    s[i] = a[i].n > 0 ? __ldg(scales + a[i].row * blocks + (a[i].c >> 5)) : 0u;
  }
#pragma unroll
  for (int i = 0; i < kActInFlight; ++i) {
    float v[8];
    act_decode(q[i], s[i], v);
    act_store<VEC>(y + a[i].row * sh.ld + a[i].c, v, a[i].n);
  }
}

// ---- SwiGLU ------------------------------------------------------------------------

// A block of (32, warps of a row, rows) threads, which walks over rows; a warp of a row has
// 256 columns of it, or with ONE false (rows of more than 2048) every blockDim.y-th such
// piece. Addresses move by a fixed step from row to row: reckoned anew for each row they
// were 250 of the 440 instructions that a warp spent on a piece. With ONE the next
// row's loads are on their way while a row is worked on. 32768 rows of 768 bf16: forward,
// kept, 33.9 us (6.0 TB/s), backward 44.7 (5.7 TB/s); with a block for each group of rows,
// which waits for its loads and goes, 37.4 and 65.5.
struct ActRow {
  int64_t row, walk;         // the first row; from a row to the next
  int first, step;           // this lane's first column; from a piece of this warp's to its next
};
SI_DEV ActRow act_row() {
  return {static_cast<int64_t>(blockIdx.x) * blockDim.z + threadIdx.z, static_cast<int64_t>(gridDim.x) * blockDim.z,
          static_cast<int>(threadIdx.y * kActCols + threadIdx.x * 8), static_cast<int>(blockDim.y * kActCols)};
}
SI_DEV int act_left(int c, int cols) { return min(max(cols - c, 0), 8); }

constexpr int kActForward = 4, kActBackward = 3;   // blocks of kActThreads on an SM

// KEEP: the codes and scales of g and of u beside h.
template <typename T, bool VEC, bool KEEP, bool ONE>
__global__ void __launch_bounds__(kActThreads, kActForward)
    swiglu_kernel(const T *__restrict__ gu, int64_t rows, int I, int64_t ld, T *__restrict__ h,
                  uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
  grid_dep_wait();
  grid_dep_launch();
  const ActRow a = act_row();
  const int lane = threadIdx.x, blocks = (I + 31) >> 5, b0 = a.first >> 5;
  gu += a.row * ld + a.first;
  h += a.row * I + a.first;
  codes += a.row * 2 * I + a.first;
  scales += a.row * 2 * blocks + b0;
  if (a.first - lane * 8 >= I) return;           // no columns for this warp
  auto piece = [&](Raw8<T> g, Raw8<T> u, int d, int n) {   // from column first + d
    float fg[8], fu[8];
    g.unpack(fg);
    u.unpack(fu);
#pragma unroll
    for (int i = 0; i < 8; ++i) fu[i] *= fg[i] * mi_logistic(fg[i]);
    act_store<VEC>(h + d, fu, n);
    if constexpr (KEEP) {
      uint32_t sg, su;
      const uint2 qg = act_encode(g, sg), qu = act_encode(u, su);
      act_store_codes<VEC>(codes + d, qg, n);
      act_store_codes<VEC>(codes + I + d, qu, n);
      if ((lane & 3) == 0 && n > 0) {
        scales[d >> 5] = static_cast<uint8_t>(sg);
        scales[blocks + (d >> 5)] = static_cast<uint8_t>(su);
      }
    }
  };
  const int64_t in = a.walk * ld, out = a.walk * I;
  const int n = act_left(a.first, I);
  Raw8<T> g, u;
  if constexpr (ONE) {
    act_load<VEC>(g, gu, a.row < rows ? n : 0);
    act_load<VEC>(u, gu + I, a.row < rows ? n : 0);
  }
  for (int64_t row = a.row; row < rows; row += a.walk) {
    gu += in;
    if constexpr (ONE) {
      const Raw8<T> g0 = g, u0 = u;
      const int m = row + a.walk < rows ? n : 0;
      act_load<VEC>(g, gu, m);
      act_load<VEC>(u, gu + I, m);
      piece(g0, u0, 0, n);
    } else {
      for (int d = 0; a.first - lane * 8 + d < I; d += a.step) {
        const int m = act_left(a.first + d, I);
        act_load<VEC>(g, gu - in + d, m);
        act_load<VEC>(u, gu - in + I + d, m);
        piece(g, u, d, m);
      }
    }
    h += out;
    codes += 2 * out;
    scales += a.walk * 2 * blocks;
  }
}

struct SwigluBack {
  int64_t rows;
  int inter;
  const uint8_t *codes, *scales;
  const float *c;            // row weights or NULL: 1
  const int32_t *order;      // row r is pair order[r] of c and gc, or NULL: pair r
  float *gc;
};
// What a lane reads of a row's piece; zeros behind the row's last column add nothing.
template <typename T> struct SwigluPiece {
  Raw8<T> gh;
  uint2 g, u;
  uint32_t sg, su;
};

template <typename T, bool VEC, bool ONE>
__global__ void __launch_bounds__(kActThreads, kActBackward)
    swiglu_backward_kernel(SwigluBack p, const T *__restrict__ gh, T *__restrict__ ggu, T *__restrict__ ch) {
  __shared__ float s_sum[2][kActThreads / 32];   // by the row's parity: one barrier a row
  grid_dep_wait();
  grid_dep_launch();
  const ActRow a = act_row();
  const int lane = threadIdx.x, I = p.inter, blocks = (I + 31) >> 5, warp = threadIdx.z * blockDim.y + threadIdx.y;
  const bool works = a.first - lane * 8 < I;     // the warp has columns
  const uint8_t *codes = p.codes + a.row * 2 * I + a.first, *scales = p.scales + a.row * 2 * blocks + (a.first >> 5);
  gh += a.row * I + a.first;
  ggu += a.row * 2 * I + a.first;
  const int64_t step = a.walk * I;
  T *wh = ch ? ch + a.row * I + a.first : nullptr;
  auto pair_of = [&](int64_t row) {
    return row >= p.rows ? -1 : p.order ? __ldg(p.order + row) : static_cast<int32_t>(row);
  };
  auto weight_of = [&](int32_t pair) { return pair < 0 || pair >= p.rows ? 0.f : p.c ? __ldg(p.c + pair) : 1.f; };
  auto load = [&](int d, int n) {
    SwigluPiece<T> v;
    act_load<VEC>(v.gh, gh + d, n);
    v.g = act_load_codes<VEC>(codes + d, n);
    v.u = act_load_codes<VEC>(codes + I + d, n);
    v.sg = n > 0 ? __ldg(scales + (d >> 5)) : 0u;
    v.su = n > 0 ? __ldg(scales + blocks + (d >> 5)) : 0u;
    return v;
  };
  const int n = act_left(a.first, I);
  int32_t pair = pair_of(a.row), next_pair = pair_of(a.row + a.walk);
  float c = weight_of(pair);
  SwigluPiece<T> next;
  if constexpr (ONE) next = load(0, a.row < p.rows ? n : 0);
  int par = 0;
  for (int64_t row = a.row; row - threadIdx.z < p.rows; row += a.walk, par ^= 1) {   // together over the block
    const bool live = pair >= 0 && pair < p.rows;  // else a row of no pair: zeros
    const float next_c = weight_of(next_pair);
    const int32_t after = pair_of(row + 2 * a.walk);
    float sum = 0.f;
    auto piece = [&](const SwigluPiece<T> &v, int d0, int m) {
      float g[8], u[8], d[8];
      act_decode(v.g, v.sg, g);
      act_decode(v.u, v.su, u);
      v.gh.unpack(d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float l = mi_logistic(g[i]), si = g[i] * l, h = si * u[i];
        sum = fmaf(d[i], h, sum);
        d[i] *= c;
        g[i] = d[i] * u[i] * fmaf(si, 1.f - l, l);   // s (1 + g (1 - s))
        d[i] *= si;
        u[i] = c * h;
      }
      if (!live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = d[i] = u[i] = 0.f;
      }
      act_store<VEC>(ggu + d0, g, m);
      act_store<VEC>(ggu + I + d0, d, m);
      if (ch) act_store<VEC>(wh + d0, u, m);
    };
    if constexpr (ONE) {
      const SwigluPiece<T> v = next;
      gh += step;
      codes += 2 * step;
      scales += a.walk * 2 * blocks;
      next = load(0, row + a.walk < p.rows ? n : 0);
      if (works) piece(v, 0, row < p.rows ? n : 0);
    } else {
      for (int d = 0; works && row < p.rows && a.first - lane * 8 + d < I; d += a.step) {
        const int m = act_left(a.first + d, I);
        piece(load(d, m), d, m);
      }
      gh += step;
      codes += 2 * step;
      scales += a.walk * 2 * blocks;
    }
    ggu += 2 * step;
    if (ch) wh += step;
    if (p.gc) {                      // uniform over the grid
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      if (lane == 0) s_sum[par][warp] = sum;
      __syncthreads();
      if (lane == 0 && threadIdx.y == 0 && live) {
        for (int i = 1; i < static_cast<int>(blockDim.y); ++i) sum += s_sum[par][warp + i];
        p.gc[pair] = sum;
      }
    }
    pair = next_pair;
    next_pair = after;
    c = next_c;
  }
}

// ---- host ------------------------------------------------------------------

template <typename F> static cudaError_t act_by_type(si_dtype type, bool vec, F fn) {
  using std::integral_constant;
  if (type == SI_F32) return vec ? fn(float{}, integral_constant<bool, true>{}) : fn(float{}, integral_constant<bool, false>{});
  if (type == SI_BF16)
    return vec ? fn(__nv_bfloat16{}, integral_constant<bool, true>{}) : fn(__nv_bfloat16{}, integral_constant<bool, false>{});
  return vec ? fn(__half{}, integral_constant<bool, true>{}) : fn(__half{}, integral_constant<bool, false>{});
}
static bool act_type(si_dtype t) { return t == SI_F32 || t == SI_F16 || t == SI_BF16; }
static int act_size(si_dtype t) { return t == SI_F32 ? 4 : 2; }
static bool act_whole(const void *p, int size) { return p && reinterpret_cast<uintptr_t>(p) % size == 0; }
static bool act_limits(int64_t rows, int64_t cols) {
  return rows >= 0 && cols >= 1 && cols <= (int64_t(1) << 40) && rows <= (int64_t(1) << 40) &&
         (rows == 0 || cols <= (int64_t(1) << 40) / rows);
}
// A row's columns count in 32 bits.
static bool act_width(int64_t inter) { return inter >= 1 && inter <= (int64_t(1) << 24); }
// Rows of whole blocks that follow one another are one row.
static ActShape act_shape(int64_t rows, int64_t cols, int64_t ld) {
  ActShape s{rows, cols, ld, 0, 0};
  if (ld == cols && cols % 32 == 0) {
    s.cols = s.ld = rows * cols;
    s.rows = 1;
  }
  s.passes = (s.cols + kActCols - 1) / kActCols;
  s.units = s.rows * s.passes;
  return s;
}
// A warp for each 256 columns of a row, at most a block of them; as many rows as fit.
static dim3 act_block(int64_t cols) {
  const int64_t pieces = (cols + kActCols - 1) / kActCols, warps = pieces < kActThreads / 32 ? pieces : kActThreads / 32;
  return dim3(32, static_cast<unsigned>(warps), static_cast<unsigned>(kActThreads / 32 / warps));
}
// Blocks of it: as many as are resident at once, for `resident` of kActThreads on an SM.
static dim3 act_walk(int64_t rows, dim3 block, int resident) {
  const int64_t groups = (rows + block.z - 1) / block.z;
  const int64_t most = static_cast<int64_t>(sm_count()) * (resident * kActThreads / (block.x * block.y * block.z));
  return dim3(static_cast<unsigned>(std::min(groups, most)));
}
static int64_t act_grid(int64_t units) {
  const int64_t b = static_cast<int64_t>(kActThreads / 32) * kActInFlight;
  return (units + b - 1) / b;
}

}  // namespace si

using namespace si;

extern "C" si_status si_quantize_mxint8(const void *x, si_dtype x_type, int64_t rows, int64_t cols, int64_t row_stride,
                                        void *codes, void *scales, void *stream) {
  if (!act_limits(rows, cols) || row_stride < cols || row_stride > (int64_t(1) << 40)) return SI_ERR_INVALID_ARG;
  if (!act_type(x_type)) return SI_ERR_UNSUPPORTED;
  if (rows == 0) return SI_OK;
  const int size = act_size(x_type);
  if (!act_whole(x, size) || !codes || !scales) return SI_ERR_INVALID_ARG;
  const ActShape sh = act_shape(rows, cols, row_stride);
  const bool vec = sh.cols % 8 == 0 && sh.ld * size % 16 == 0 && aligned16(x) && act_whole(codes, 8);
  const int64_t grid = act_grid(sh.units);
  if (grid > 0x7FFFFFFF) return SI_ERR_UNSUPPORTED;
  return cuda_status(act_by_type(x_type, vec, [&](auto t, auto v) {
    using T = decltype(t);
    return launch_pdl(quantize_mxint8_kernel<T, decltype(v)::value>, dim3(static_cast<unsigned>(grid)),
                      dim3(kActThreads), 0, static_cast<cudaStream_t>(stream), static_cast<const T *>(x), sh,
                      static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales));
  }));
}

extern "C" si_status si_dequantize_mxint8(const void *codes, const void *scales, int64_t rows, int64_t cols, void *y,
                                          si_dtype y_type, int64_t row_stride, void *stream) {
  if (!act_limits(rows, cols) || row_stride < cols || row_stride > (int64_t(1) << 40)) return SI_ERR_INVALID_ARG;
  if (!act_type(y_type)) return SI_ERR_UNSUPPORTED;
  if (rows == 0) return SI_OK;
  const int size = act_size(y_type);
  if (!act_whole(y, size) || !codes || !scales) return SI_ERR_INVALID_ARG;
  const ActShape sh = act_shape(rows, cols, row_stride);
  const bool vec = sh.cols % 8 == 0 && sh.ld * size % 16 == 0 && aligned16(y) && act_whole(codes, 8);
  const int64_t grid = act_grid(sh.units);
  if (grid > 0x7FFFFFFF) return SI_ERR_UNSUPPORTED;
  return cuda_status(act_by_type(y_type, vec, [&](auto t, auto v) {
    using T = decltype(t);
    return launch_pdl(dequantize_mxint8_kernel<T, decltype(v)::value>, dim3(static_cast<unsigned>(grid)),
                      dim3(kActThreads), 0, static_cast<cudaStream_t>(stream), static_cast<const uint8_t *>(codes),
                      static_cast<const uint8_t *>(scales), sh, static_cast<T *>(y));
  }));
}

extern "C" si_status si_swiglu(const void *gu, si_dtype type, int64_t rows, int64_t inter, int64_t row_stride, void *h,
                               void *codes, void *scales, void *stream) {
  if (!act_width(inter) || !act_limits(rows, 2 * inter) || row_stride < 2 * inter || row_stride > (int64_t(1) << 40))
    return SI_ERR_INVALID_ARG;
  if (!act_type(type)) return SI_ERR_UNSUPPORTED;
  if (rows == 0) return SI_OK;
  const int size = act_size(type);
  if (!act_whole(gu, size) || !act_whole(h, size) || !codes != !scales) return SI_ERR_INVALID_ARG;
  const bool vec = inter % 8 == 0 && row_stride * size % 16 == 0 && aligned16(gu) && aligned16(h) &&
                   (reinterpret_cast<uintptr_t>(codes) & 7u) == 0;
  const dim3 block = act_block(inter), grid = act_walk(rows, block, kActForward);
  const bool one = inter <= kActThreads / 32 * kActCols;
  return cuda_status(act_by_type(type, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr bool V = decltype(v)::value;
    const auto kernel = codes ? (one ? swiglu_kernel<T, V, true, true> : swiglu_kernel<T, V, true, false>)
                              : (one ? swiglu_kernel<T, V, false, true> : swiglu_kernel<T, V, false, false>);
    return launch_pdl(kernel, grid, block, 0, static_cast<cudaStream_t>(stream), static_cast<const T *>(gu), rows,
                      static_cast<int>(inter), row_stride, static_cast<T *>(h), static_cast<uint8_t *>(codes),
                      static_cast<uint8_t *>(scales));
  }));
}

extern "C" si_status si_swiglu_backward(const void *gh, si_dtype type, int64_t rows, int64_t inter, const void *codes,
                                        const void *scales, const float *row_w, const int32_t *order, void *ggu,
                                        void *wh, float *gw, void *stream) {
  if (!act_width(inter) || !act_limits(rows, 2 * inter) || rows > 0x7FFFFFFF) return SI_ERR_INVALID_ARG;
  if (!act_type(type)) return SI_ERR_UNSUPPORTED;
  if (rows == 0) return SI_OK;
  const int size = act_size(type);
  if (!act_whole(gh, size) || !act_whole(ggu, size) || !codes || !scales || (wh && !act_whole(wh, size)) ||
      (row_w && !act_whole(row_w, 4)) || (order && !act_whole(order, 4)) || (gw && !act_whole(gw, 4)))
    return SI_ERR_INVALID_ARG;
  const bool vec = inter % 8 == 0 && aligned16(gh) && aligned16(ggu) && aligned16(wh) && act_whole(codes, 8);
  const SwigluBack p{rows, static_cast<int>(inter), static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), row_w,
                     order, gw};
  const dim3 block = act_block(inter), grid = act_walk(rows, block, kActBackward);
  if (gw && order) {                 // of the pairs without a row too
    const cudaError_t e = cudaMemsetAsync(gw, 0, static_cast<size_t>(rows) * sizeof(float), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return SI_ERR_CUDA;
  }
  const bool one = inter <= kActThreads / 32 * kActCols;
  return cuda_status(act_by_type(type, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr bool V = decltype(v)::value;
    return launch_pdl(one ? swiglu_backward_kernel<T, V, true> : swiglu_backward_kernel<T, V, false>, grid, block, 0,
                      static_cast<cudaStream_t>(stream), p, static_cast<const T *>(gh), static_cast<T *>(ggu),
                      static_cast<T *>(wh));
  }));
}
