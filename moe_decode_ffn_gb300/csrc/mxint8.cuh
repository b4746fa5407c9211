// MXINT8 (OCP microscaling, 8-bit integer elements, E8M0 scales) on the device.
//
// 32 consecutive values of a row share the power of two X = 2^(s - 127) with s the
// exponent field of max |x| in fp32, so that the largest lies in [X, 2X); every
// value is code * X / 64, code = x / X * 64 rounded to nearest even and kept within
// +-127. A block that holds an infinity or a NaN gets s = 255 (the E8M0 NaN) and
// codes 0.
#pragma once

#include "mxfp4.cuh"

namespace si {

// s from the largest |x| of the block, as bits.
SI_DEV uint32_t mi_scale_of(uint32_t amax_bits) { return amax_bits >> 23; }
// 2^(127 - s), exact; s = 255: 0.
SI_DEV float mi_inv_scale(uint32_t s) {
  return s >= 254u ? (s == 254u ? __uint_as_float(1u << 22) : 0.f) : __uint_as_float((254u - s) << 23);
}
// 2^(s - 133), the value of code 1 (exact, subnormal below s = 7); NaN for 255.
SI_DEV float mi_step(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7FC00000u : s > 6u ? (s - 6u) << 23 : 1u << (s + 16u));
}
// A value, times 2^(127 - s), to its code in the low byte: within +-127/64, then
// rounded to a multiple of 1/64 by the addition to 1.5 * 2^23.
SI_DEV uint32_t mi_code(float v) {
  return __float_as_uint(fmaf(fminf(fmaxf(v, -127.f / 64.f), 127.f / 64.f), 64.f, 12582912.f));
}
// Nearly every block needs less: one multiplication and addition by 64 / X. Not the ones that
// mi_far() names: X below 2^-121, where 64 / X passes fp32; an infinity or a NaN; and a
// largest magnitude from 127.5 / 64 X on (all seven leading bits of the mantissa), which
// has to be kept within 127. `top`: at least its upper 16 bits.
SI_DEV bool mi_far(uint32_t top) { return top < (6u << 23) || top >= (255u << 23) || (~top & 0x7F0000u) == 0; }
SI_DEV float mi_inv_step(uint32_t s) { return __uint_as_float((260u - s) << 23); }
SI_DEV uint32_t mi_code_near(float v, float inv_step) { return __float_as_uint(fmaf(v, inv_step, 12582912.f)); }
SI_DEV uint32_t mi_pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// Four codes to their integers as fp32: code + 128 becomes the low byte of 2^23 + (code + 128).
SI_DEV void mi_values4(uint32_t w, float v[4]) {
  w ^= 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 + i)) - 8388736.f;
}
// The logistic function; g below -87 gives 0 where the reciprocal is below the normal
// range (s < 2^-125). ex2 and rcp of the hardware, each within 2 units in the last place; the
// argument's rounding adds about |g| units to exp(-g), which counts where g is well below 0.
SI_DEV float mi_logistic(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
// Scales of a row of `cols` values.
__host__ __device__ constexpr int64_t mi_blocks(int64_t cols) { return (cols + 31) / 32; }

}  // namespace si
