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
  s = mi_scale_of(mx_top_4lanes(x));
  const float up = mi_inv_scale(s);
  float v[8];
  x.unpack(v);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = mi_code(v[i] * up);
  const uint2 q = make_uint2(mi_pack4(c[0], c[1], c[2], c[3]), mi_pack4(c[4], c[5], c[6], c[7]));
  return s == 255u ? make_uint2(0, 0) : q;
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
    a.row = unit / sh.passes;
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
#pragma unroll
  for (int i = 0; i < kActInFlight; ++i) {
    uint32_t s;
    const uint2 q = act_encode(v[i], s);
    act_store_codes<VEC>(codes + a[i].row * sh.cols + a[i].c, q, a[i].n);
    if ((lane & 3) == 0 && a[i].n > 0) scales[a[i].row * blocks + (a[i].c >> 5)] = static_cast<uint8_t>(s);
  }
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

// The logistic function; exp and the reciprocal in fp32 (1 / inf is 0).
SI_DEV float act_logistic(float g) { return __frcp_rn(1.f + __expf(-g)); }

// KEEP: the codes and scales of g and of u beside h.
template <typename T, bool VEC, bool KEEP>
__global__ void __launch_bounds__(kActThreads)
    swiglu_kernel(const T *__restrict__ gu, ActShape sh, T *__restrict__ h, uint8_t *__restrict__ codes,
                  uint8_t *__restrict__ scales) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kActThreads / 32) + (threadIdx.x >> 5);
  const int64_t I = sh.cols, blocks = mi_blocks(I);
  const ActAt a = act_at(sh, unit, lane);
  Raw8<T> g, u;
  const T *src = gu + a.row * sh.ld + a.c;
  act_load<VEC>(g, src, a.n);
  act_load<VEC>(u, src + I, a.n);
  float fg[8], fu[8];
  g.unpack(fg);
  u.unpack(fu);
#pragma unroll
  for (int i = 0; i < 8; ++i) fu[i] *= fg[i] * act_logistic(fg[i]);
  act_store<VEC>(h + a.row * I + a.c, fu, a.n);
  if constexpr (KEEP) {
    uint32_t sg, su;
    const uint2 qg = act_encode(g, sg), qu = act_encode(u, su);
    uint8_t *c = codes + a.row * 2 * I + a.c, *s = scales + a.row * 2 * blocks + (a.c >> 5);
    act_store_codes<VEC>(c, qg, a.n);
    act_store_codes<VEC>(c + I, qu, a.n);
    if ((lane & 3) == 0 && a.n > 0) {
      s[0] = static_cast<uint8_t>(sg);
      s[blocks] = static_cast<uint8_t>(su);
    }
  }
}

struct SwigluBack {
  int64_t rows, inter;
  int warps, per_block;      // warps of a row, rows of a block
  const uint8_t *codes, *scales;
  const float *c;            // row weights or NULL: 1
  const int32_t *order;      // row r is pair order[r] of c and gc, or NULL: pair r
  float *gc;
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kActThreads)
    swiglu_backward_kernel(SwigluBack p, const T *__restrict__ gh, T *__restrict__ ggu, T *__restrict__ ch) {
  __shared__ float s_sum[kActThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp % p.warps;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * p.per_block + warp / p.warps;
  const int64_t I = p.inter, blocks = mi_blocks(I);
  int64_t pair = row;
  if (p.order && row < p.rows) pair = __ldg(p.order + row);
  const bool live = row < p.rows && pair >= 0 && pair < p.rows;   // a row of no pair: zeros
  const float c = !live ? 0.f : p.c ? __ldg(p.c + pair) : 1.f;
  float sum = 0.f;
  if (row < p.rows) {
    for (int64_t c0 = static_cast<int64_t>(mine) * kActCols; c0 < I; c0 += static_cast<int64_t>(p.warps) * kActCols) {
      const int64_t at = c0 + lane * 8;
      const int n = act_inside(at, I);
      float o1[8] = {}, o2[8] = {}, o3[8] = {};
      if (live) {
        Raw8<T> v;
        act_load<VEC>(v, gh + row * I + at, n);
        const uint8_t *q = p.codes + row * 2 * I + at, *s = p.scales + row * 2 * blocks + (at >> 5);
        const uint2 qg = act_load_codes<VEC>(q, n), qu = act_load_codes<VEC>(q + I, n);
        const uint32_t sg = n > 0 ? __ldg(s) : 0u, su = n > 0 ? __ldg(s + blocks) : 0u;
        float g[8], u[8], d[8];
        act_decode(qg, sg, g);
        act_decode(qu, su, u);
        v.unpack(d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float l = act_logistic(g[i]), si = g[i] * l, hv = si * u[i];
          if (i < n) sum = fmaf(d[i], hv, sum);
          const float cd = c * d[i];
          o1[i] = cd * u[i] * (l * fmaf(g[i], 1.f - l, 1.f));
          o2[i] = cd * si;
          o3[i] = c * hv;
        }
      }
      T *to = ggu + row * 2 * I + at;
      act_store<VEC>(to, o1, n);
      act_store<VEC>(to + I, o2, n);
      if (ch) act_store<VEC>(ch + row * I + at, o3, n);
    }
  }
  if (!p.gc) return;                 // uniform over the grid
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  if (lane == 0 && mine == 0 && live) {
    for (int i = 1; i < p.warps; ++i) sum += s_sum[warp + i];
    p.gc[pair] = sum;
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
// Rows of whole blocks that follow one another are one row.
static ActShape act_shape(int64_t rows, int64_t cols, int64_t ld, bool flat) {
  ActShape s{rows, cols, ld, 0, 0};
  if (flat && ld == cols && cols % 32 == 0) {
    s.cols = s.ld = rows * cols;
    s.rows = 1;
  }
  s.passes = (s.cols + kActCols - 1) / kActCols;
  s.units = s.rows * s.passes;
  return s;
}
static int64_t act_grid(int64_t units, int per_warp) {
  const int64_t b = static_cast<int64_t>(kActThreads / 32) * per_warp;
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
  const ActShape sh = act_shape(rows, cols, row_stride, true);
  const bool vec = sh.cols % 8 == 0 && sh.ld * size % 16 == 0 && aligned16(x) && act_whole(codes, 8);
  const int64_t grid = act_grid(sh.units, kActInFlight);
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
  const ActShape sh = act_shape(rows, cols, row_stride, true);
  const bool vec = sh.cols % 8 == 0 && sh.ld * size % 16 == 0 && aligned16(y) && act_whole(codes, 8);
  const int64_t grid = act_grid(sh.units, kActInFlight);
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
  if (!act_limits(rows, 2 * inter) || inter < 1 || row_stride < 2 * inter || row_stride > (int64_t(1) << 40))
    return SI_ERR_INVALID_ARG;
  if (!act_type(type)) return SI_ERR_UNSUPPORTED;
  if (rows == 0) return SI_OK;
  const int size = act_size(type);
  if (!act_whole(gu, size) || !act_whole(h, size) || !codes != !scales) return SI_ERR_INVALID_ARG;
  const ActShape sh = act_shape(rows, inter, row_stride, false);
  const bool vec = inter % 8 == 0 && row_stride * size % 16 == 0 && aligned16(gu) && aligned16(h) &&
                   (reinterpret_cast<uintptr_t>(codes) & 7u) == 0;
  const int64_t grid = act_grid(sh.units, 1);
  if (grid > 0x7FFFFFFF) return SI_ERR_UNSUPPORTED;
  return cuda_status(act_by_type(type, vec, [&](auto t, auto v) {
    using T = decltype(t);
    constexpr bool V = decltype(v)::value;
    return launch_pdl(codes ? swiglu_kernel<T, V, true> : swiglu_kernel<T, V, false>, dim3(static_cast<unsigned>(grid)),
                      dim3(kActThreads), 0, static_cast<cudaStream_t>(stream), static_cast<const T *>(gu), sh,
                      static_cast<T *>(h), static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales));
  }));
}

extern "C" si_status si_swiglu_backward(const void *gh, si_dtype type, int64_t rows, int64_t inter, const void *codes,
                                        const void *scales, const float *row_w, const int32_t *order, void *ggu,
                                        void *wh, float *gw, void *stream) {
  if (!act_limits(rows, 2 * inter) || inter < 1 || rows > 0x7FFFFFFF) return SI_ERR_INVALID_ARG;
  if (!act_type(type)) return SI_ERR_UNSUPPORTED;
  if (rows == 0) return SI_OK;
  const int size = act_size(type);
  if (!act_whole(gh, size) || !act_whole(ggu, size) || !codes || !scales || (wh && !act_whole(wh, size)) ||
      (row_w && !act_whole(row_w, 4)) || (order && !act_whole(order, 4)) || (gw && !act_whole(gw, 4)))
    return SI_ERR_INVALID_ARG;
  const bool vec = inter % 8 == 0 && aligned16(gh) && aligned16(ggu) && aligned16(wh) && act_whole(codes, 8);
  const int64_t passes = (inter + kActCols - 1) / kActCols;
  SwigluBack p{rows, inter, 0, 0, static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), row_w,
               order, gw};
  p.warps = static_cast<int>(passes < kActThreads / 32 ? passes : kActThreads / 32);
  p.per_block = kActThreads / 32 / p.warps;
  const int64_t grid = (rows + p.per_block - 1) / p.per_block;
  return cuda_status(act_by_type(type, vec, [&](auto t, auto v) {
    using T = decltype(t);
    return launch_pdl(swiglu_backward_kernel<T, decltype(v)::value>, dim3(static_cast<unsigned>(grid)),
                      dim3(32 * p.warps * p.per_block), 0, static_cast<cudaStream_t>(stream), p,
                      static_cast<const T *>(gh), static_cast<T *>(ggu), static_cast<T *>(wh));
  }));
}
