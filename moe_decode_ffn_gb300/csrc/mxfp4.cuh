// MXFP4 (OCP microscaling, E2M1 elements, E8M0 scales) on the device.
//
// 32 consecutive values of a row share the power of two 2^(s - 127) with
//   s = max(exponent field of max |x| - 2, 0)            (fp32 exponent field)
// so that the largest element lands in [4, 8); every value is x * 2^(127 - s)
// rounded to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to even, larger
// ones to 6). A block that holds an infinity or a NaN gets s = 255 (the E8M0
// NaN) and codes 0.
//
// Codes: two per byte, the even column in the low nibble, rows contiguous.
// Scales: tiles of 128 rows x 4 blocks (128 columns) of 512 bytes, byte
// (row % 32) * 16 + (row % 128) / 32 * 4 + block % 4, the order in which
// tcgen05.cp lays the scale factors of a 128-row operand into tensor memory.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace si {

constexpr int kMxBlock = 32;         // values that share a scale
constexpr int kMxTileBytes = 512;    // one scale tile: 128 rows x 4 blocks

SI_DEV uint32_t mx_scale_byte(uint32_t row, uint32_t blk) {   // within a tile
  return (row & 31u) * 16u + ((row >> 5) & 3u) * 4u + (blk & 3u);
}
// s from the largest |x| of the block, as bits (they order like the values,
// NaN above infinity above every finite value).
SI_DEV uint32_t mx_scale_of(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(127 - s): the exact multiplier into the element range (s = 255: 0, so
// that finite values get code 0; see mx_codes8 for the others).
SI_DEV float mx_inv_scale(uint32_t s) {
  return s == 255u ? 0.f : __uint_as_float((254u - s) << 23);
}
SI_DEV float mx_scale_value(uint32_t s) {   // 2^(s - 127), NaN for 255
  return __uint_as_float(s == 255u ? 0x7FC00000u : (s == 0u ? 0x00400000u : s << 23));
}
// Eight values to eight codes, value i in nibble i (round to nearest even,
// saturating).
SI_DEV uint32_t mx_codes8(const float v[8]) {
  uint32_t w;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w;
}
// Eight codes to their values (E2M1 values are exact in fp16).
SI_DEV void mx_values8(uint32_t w, float v[8]) {
  uint32_t h[4];
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = half_bits_to_float(static_cast<uint16_t>(h[i] & 0xFFFFu));
    v[2 * i + 1] = half_bits_to_float(static_cast<uint16_t>(h[i] >> 16));
  }
}
// ---- rows of bf16, fp16 or fp32 ------------------------------------------------
template <typename T> SI_DEV float to_f32(T v);
template <> SI_DEV float to_f32<float>(float v) { return v; }
template <> SI_DEV float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> SI_DEV float to_f32<__half>(__half v) { return __half2float(v); }
template <typename T> SI_DEV T from_f32(float v);
template <> SI_DEV float from_f32<float>(float v) { return v; }
template <> SI_DEV __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> SI_DEV __half from_f32<__half>(float v) { return __float2half_rn(v); }

// kVec values of T in 16 bytes.
template <typename T> constexpr int kVecOf = 16 / static_cast<int>(sizeof(T));
template <typename T> SI_DEV void unpack16(uint4 u, float *v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    } else {
      v[2 * i] = half_bits_to_float(static_cast<uint16_t>(w[i] & 0xFFFFu));
      v[2 * i + 1] = half_bits_to_float(static_cast<uint16_t>(w[i] >> 16));
    }
  }
}
template <typename T> SI_DEV uint4 pack16(const float *v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      w[i] = __float_as_uint(v[i]);
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      w[i] = bf16_bits(v[2 * i]) | (static_cast<uint32_t>(bf16_bits(v[2 * i + 1])) << 16);
    } else {
      w[i] = float_to_half_bits(v[2 * i]) | (static_cast<uint32_t>(float_to_half_bits(v[2 * i + 1])) << 16);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight consecutive values of a row as they lie in memory.
template <typename T> struct Raw8 {
  static constexpr int kWords = 2 * static_cast<int>(sizeof(T));
  uint32_t w[kWords];
  SI_DEV void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  SI_DEV void load16(const T *p) {               // p on a 16-byte boundary
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p) + i);
      w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
    }
  }
  SI_DEV void load(const T *p) {                 // value by value
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(p[i]);
    } else {
      const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = q[2 * i] | (static_cast<uint32_t>(q[2 * i + 1]) << 16);
    }
  }
  SI_DEV void unpack(float v[8]) const {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      unpack16<T>(make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]), v + i * kVecOf<T>);
  }
};

// Quantise 8 values of a 32-value block held by 4 consecutive lanes (8 each):
// the codes of this lane's values; s is the same on the four lanes. Every lane
// of the warp takes part. Magnitudes order like their bits, so the largest of a
// 16-bit type is found two values at a time.
template <typename T> SI_DEV uint32_t mx_encode_4lanes(const Raw8<T> &x, uint32_t &s) {
  uint32_t top;
  if constexpr (sizeof(T) == 4) {
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, x.w[i] & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  } else {
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    uint32_t m = __vimax3_u16x2(x.w[0] & kAbs, x.w[1] & kAbs, x.w[2] & kAbs);
    m = __vimax3_u16x2(m, x.w[3] & kAbs, __shfl_xor_sync(0xffffffffu, __vmaxu2(m, x.w[3] & kAbs), 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = max(m >> 16, m & 0xFFFFu);
    if constexpr (std::is_same_v<T, __nv_bfloat16>) top = m << 16;
    else top = __float_as_uint(half_bits_to_float(static_cast<uint16_t>(m)));
  }
  s = mx_scale_of(top);
  const float up = mx_inv_scale(s);
  float q[8];
  x.unpack(q);
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] *= up;
  const uint32_t w = mx_codes8(q);
  return s == 255u ? 0u : w;
}

}  // namespace si
