// MXFP4 quantisation and dequantisation of matrices (mxfp4.cuh has the format).
//
// Both kernels give a block of 256 threads one scale tile: 128 rows x 128
// columns. 16 consecutive lanes take a row (8 values, 16 or 32 bytes each), so
// every access of a warp covers whole 32-byte sectors, and the tile's 512
// scale bytes are assembled in shared memory and move as one piece. Both are
// bound by HBM: 98304 x 2048 bf16 values are quantised in 75.2 us and decoded in
// 76.9 us (6.8 and 6.6 TB/s; a copy of them reaches 6.7); before the largest value
// of a block was found two values at a time the quantiser issued for 89 us.
#include "host.hpp"
#include "mxfp4.cuh"

namespace si {

constexpr int kMxThreads = 256;
constexpr int kMxRowsPerPass = kMxThreads / 16;   // 16 rows of 128 columns
constexpr int kMxPasses = 128 / kMxRowsPerPass;   // 8
constexpr int kMxInFlight = 4;                    // rows loaded by a thread before the first encode

struct MxShape {
  int64_t rows, cols, row_stride, mat_stride;     // of the float matrix, in values
  int row_tiles, col_tiles;
};

// Tile blockIdx.x: matrix, row tile, column tile (columns fastest).
struct MxTile {
  int64_t mat;
  int rt, ct;
};
SI_DEV MxTile mx_tile(const MxShape &s) {
  MxTile t;
  const uint32_t b = blockIdx.x;
  t.ct = static_cast<int>(b % s.col_tiles);
  const uint32_t r = b / s.col_tiles;
  t.rt = static_cast<int>(r % s.row_tiles);
  t.mat = r / s.row_tiles;
  return t;
}

// VEC: the 8 values of a lane are loaded or stored as 16-byte words (every row
// starts on a 16-byte boundary); otherwise one by one.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kMxThreads)
    quantize_mxfp4_kernel(const T *__restrict__ x, MxShape sh, uint8_t *__restrict__ codes,
                          uint8_t *__restrict__ scales) {
  __shared__ __align__(16) uint8_t s_tile[kMxTileBytes];
  grid_dep_wait();
  grid_dep_launch();
  const MxTile t = mx_tile(sh);
  const int l16 = threadIdx.x & 15, r16 = threadIdx.x >> 4;
  const int64_t c = static_cast<int64_t>(t.ct) * 128 + l16 * 8;
  const int64_t r0 = static_cast<int64_t>(t.rt) * 128 + r16;
  const T *src = x + t.mat * sh.mat_stride + c;
  uint8_t *dst = codes + (t.mat * sh.rows * sh.cols + c) / 2;
  const bool in_col = c < sh.cols;                // cols % 32 == 0: 8 values are in or out together
#pragma unroll
  for (int p0 = 0; p0 < kMxPasses; p0 += kMxInFlight) {
    Raw8<T> v[kMxInFlight];
#pragma unroll
    for (int u = 0; u < kMxInFlight; ++u) {
      const int64_t r = r0 + (p0 + u) * kMxRowsPerPass;
      if (!in_col || r >= sh.rows) v[u].zero();
      else if constexpr (VEC) v[u].load16(src + r * sh.row_stride);
      else v[u].load(src + r * sh.row_stride);
    }
#pragma unroll
    for (int u = 0; u < kMxInFlight; ++u) {
      const int lr = r16 + (p0 + u) * kMxRowsPerPass;
      const int64_t r = r0 + (p0 + u) * kMxRowsPerPass;
      uint32_t s;
      const uint32_t w = mx_encode_4lanes(v[u], s);
      if (in_col && r < sh.rows) *reinterpret_cast<uint32_t *>(dst + r * (sh.cols / 2)) = w;
      if ((l16 & 3) == 0) s_tile[mx_scale_byte(lr, l16 >> 2)] = static_cast<uint8_t>(s);   // rows and blocks outside: 0
    }
  }
  __syncthreads();
  if (threadIdx.x < kMxTileBytes / 16)
    reinterpret_cast<uint4 *>(scales + static_cast<size_t>(blockIdx.x) * kMxTileBytes)[threadIdx.x] =
        reinterpret_cast<const uint4 *>(s_tile)[threadIdx.x];
}

// 6 blocks an SM: 77.0 us for 98304 x 2048 bf16 values, against 86.2 with the 5
// that the registers otherwise leave.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kMxThreads, 6)
    dequantize_mxfp4_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                            MxShape sh, T *__restrict__ y) {
  __shared__ __align__(16) uint8_t s_tile[kMxTileBytes];
  grid_dep_wait();
  grid_dep_launch();
  const MxTile t = mx_tile(sh);
  const int l16 = threadIdx.x & 15, r16 = threadIdx.x >> 4;
  const int64_t c = static_cast<int64_t>(t.ct) * 128 + l16 * 8;
  const int64_t r0 = static_cast<int64_t>(t.rt) * 128 + r16;
  const uint8_t *src = codes + (t.mat * sh.rows * sh.cols + c) / 2;
  T *dst = y + t.mat * sh.mat_stride + c;
  const bool in_col = c < sh.cols;
  uint32_t w[kMxPasses];
#pragma unroll
  for (int p = 0; p < kMxPasses; ++p) {
    const int64_t r = r0 + p * kMxRowsPerPass;
    w[p] = in_col && r < sh.rows ? __ldg(reinterpret_cast<const uint32_t *>(src + r * (sh.cols / 2))) : 0u;
  }
  if (threadIdx.x < kMxTileBytes / 16)
    reinterpret_cast<uint4 *>(s_tile)[threadIdx.x] =
        __ldg(reinterpret_cast<const uint4 *>(scales + static_cast<size_t>(blockIdx.x) * kMxTileBytes) + threadIdx.x);
  __syncthreads();
#pragma unroll
  for (int p = 0; p < kMxPasses; ++p) {
    const int64_t r = r0 + p * kMxRowsPerPass;
    if (!in_col || r >= sh.rows) continue;
    const float d = mx_scale_value(s_tile[mx_scale_byte(r16 + p * kMxRowsPerPass, l16 >> 2)]);
    float v[8];
    mx_values8(w[p], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= d;
    T *o = dst + r * sh.row_stride;
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < 8 / kVecOf<T>; ++i) reinterpret_cast<uint4 *>(o)[i] = pack16<T>(v + i * kVecOf<T>);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = from_f32<T>(v[i]);
    }
  }
}

static bool float_size(si_dtype t, int &size) {
  if (t == SI_F32) size = 4;
  else if (t == SI_F16 || t == SI_BF16) size = 2;
  else return false;
  return true;
}

// Shapes of both calls; SI_OK with tiles = 0 where there is nothing to do.
static si_status mx_check(const void *f, si_dtype type, const void *codes, const void *scales,
                          int64_t n_mats, int64_t rows, int64_t cols, int64_t row_stride,
                          int64_t mat_stride, MxShape &sh, int64_t &tiles, bool &vec) {
  constexpr int64_t kMax = int64_t(1) << 31;
  tiles = 0;
  if (n_mats < 0 || rows < 0 || cols <= 0 || cols % kMxBlock || n_mats >= kMax || rows >= kMax || cols >= kMax)
    return SI_ERR_INVALID_ARG;
  int size = 0;
  if (!float_size(type, size)) return SI_ERR_UNSUPPORTED;
  if (n_mats == 0 || rows == 0) return SI_OK;
  if (!f || !codes || !scales || !aligned16(codes) || !aligned16(scales) ||
      (reinterpret_cast<uintptr_t>(f) % size))
    return SI_ERR_INVALID_ARG;
  // rows that overlap or run backwards are refused, for reading too: matrices lie
  // one behind the other, or row by row in turn
  if (row_stride < 0 || row_stride > (int64_t(1) << 40) || mat_stride < 0 || mat_stride > (int64_t(1) << 50) ||
      (rows > 1 && row_stride < cols) || (n_mats > 1 && mat_stride < cols))
    return SI_ERR_INVALID_ARG;
  const int64_t rows_end = rows > 1 ? (rows - 1) * row_stride + cols : cols;
  const int64_t mats_end = n_mats > 1 && mat_stride <= (int64_t(1) << 40) / n_mats ? (n_mats - 1) * mat_stride + cols : 0;
  if (n_mats > 1 && mat_stride < rows_end && (rows == 1 || mats_end == 0 || row_stride < mats_end))
    return SI_ERR_INVALID_ARG;
  sh.rows = rows;
  sh.cols = cols;
  sh.row_stride = row_stride;
  sh.mat_stride = mat_stride;
  sh.row_tiles = static_cast<int>((rows + 127) / 128);
  sh.col_tiles = static_cast<int>((cols + 127) / 128);
  const int64_t per_mat = static_cast<int64_t>(sh.row_tiles) * sh.col_tiles;
  if (per_mat > 0x7FFFFFFF || n_mats > 0x7FFFFFFF / per_mat) return SI_ERR_UNSUPPORTED;
  tiles = n_mats * per_mat;
  vec = aligned16(f) && (rows == 1 || row_stride * size % 16 == 0) && (n_mats == 1 || mat_stride * size % 16 == 0);
  return SI_OK;
}

template <typename T>
static cudaError_t quantize_launch(const void *x, const MxShape &sh, int64_t tiles, bool vec, void *codes,
                                   void *scales, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(tiles)), block(kMxThreads);
  const T *xt = static_cast<const T *>(x);
  uint8_t *c = static_cast<uint8_t *>(codes), *sc = static_cast<uint8_t *>(scales);
  return vec ? launch_pdl(quantize_mxfp4_kernel<T, true>, grid, block, 0, s, xt, sh, c, sc)
             : launch_pdl(quantize_mxfp4_kernel<T, false>, grid, block, 0, s, xt, sh, c, sc);
}
template <typename T>
static cudaError_t dequantize_launch(const void *codes, const void *scales, const MxShape &sh, int64_t tiles,
                                     bool vec, void *y, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(tiles)), block(kMxThreads);
  T *yt = static_cast<T *>(y);
  const uint8_t *c = static_cast<const uint8_t *>(codes), *sc = static_cast<const uint8_t *>(scales);
  return vec ? launch_pdl(dequantize_mxfp4_kernel<T, true>, grid, block, 0, s, c, sc, sh, yt)
             : launch_pdl(dequantize_mxfp4_kernel<T, false>, grid, block, 0, s, c, sc, sh, yt);
}

}  // namespace si

using namespace si;

extern "C" size_t si_mxfp4_scale_bytes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0 || cols % kMxBlock || rows >= (int64_t(1) << 31) || cols >= (int64_t(1) << 31)) return 0;
  return static_cast<size_t>((rows + 127) / 128) * static_cast<size_t>((cols + 127) / 128) * kMxTileBytes;
}

extern "C" si_status si_quantize_mxfp4(const void *x, si_dtype x_type, int64_t n_mats, int64_t rows,
                                       int64_t cols, int64_t row_stride, int64_t mat_stride, void *codes,
                                       void *scales, void *stream) {
  MxShape sh{};
  int64_t tiles = 0;
  bool vec = false;
  const si_status st =
      mx_check(x, x_type, codes, scales, n_mats, rows, cols, row_stride, mat_stride, sh, tiles, vec);
  if (st != SI_OK || tiles == 0) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(x_type == SI_F32    ? quantize_launch<float>(x, sh, tiles, vec, codes, scales, s)
                     : x_type == SI_BF16 ? quantize_launch<__nv_bfloat16>(x, sh, tiles, vec, codes, scales, s)
                                         : quantize_launch<__half>(x, sh, tiles, vec, codes, scales, s));
}

extern "C" si_status si_dequantize_mxfp4(const void *codes, const void *scales, int64_t n_mats, int64_t rows,
                                         int64_t cols, void *y, si_dtype y_type, int64_t row_stride,
                                         int64_t mat_stride, void *stream) {
  MxShape sh{};
  int64_t tiles = 0;
  bool vec = false;
  const si_status st =
      mx_check(y, y_type, codes, scales, n_mats, rows, cols, row_stride, mat_stride, sh, tiles, vec);
  if (st != SI_OK || tiles == 0) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(y_type == SI_F32    ? dequantize_launch<float>(codes, scales, sh, tiles, vec, y, s)
                     : y_type == SI_BF16 ? dequantize_launch<__nv_bfloat16>(codes, scales, sh, tiles, vec, y, s)
                                         : dequantize_launch<__half>(codes, scales, sh, tiles, vec, y, s));
}
