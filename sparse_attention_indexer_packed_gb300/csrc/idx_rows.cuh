// Rows of 128 held by 16 lanes, eight elements a lane, and their quantisation: what the
// store and the norm, rotation and store pass have in common; and the NVFP4 rule.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>
#include <string.h>

#include "idx_internal.cuh"
#include "idx_ops.cuh"

namespace idx {

// The NVFP4 rule, per group of 16: scale s = E4M3(amax / 6), codes e2m1(x / s).
//
// The codes come from the hardware e2m1 conversion (round to nearest, ties to
// the even code, saturating at 6, the sign kept) of a quotient q2 that equals
// x / s where that is on the e2m1 grid's midpoints and is within two ulps of it
// elsewhere: q1 = x * r with r = 1 / s, the residual e = x - q1 * s (exact in
// one fma), q2 = q1 + e * r (one correction step of a reciprocal-based
// quotient, after Markstein, "IA-64 and Elementary Functions", 2000).  This is
// enough: every midpoint t of the grid has at most three significant bits and
// s at most four, so t * s is a bf16 value, and a bf16 x either equals t * s
// (then the residual is exact and q2 = t) or lies a bf16 spacing away from it,
// far beyond the quotient's error, on the same side as fl(x / s).  (An fp32 x, as of a
// key that was normed and rotated, may get the code of a neighbour two ulps away.)
// Value of an E4M3 byte with the sign bit clear (scales are never negative):
// exponent field 0 -> m * 2^-9; otherwise (8 + m) * 2^(e - 10).
__device__ __forceinline__ float e4m3_magnitude(uint32_t b) {
  const uint32_t e = (b >> 3) & 0xfu, m = b & 7u;
  if (e == 0) return (float)m * 0.001953125f;
  return __uint_as_float(((e + 120u) << 23) | (m << 20));
}

__device__ __forceinline__ __nv_bfloat162 as_bf16x2(uint32_t u) {
  __nv_bfloat162 v;
  memcpy(&v, &u, sizeof(v));
  return v;
}

// x / s on the e2m1 midpoints, within two ulps elsewhere (see above), with
// x's sign (the fma steps would turn -0 into +0).
__device__ __forceinline__ float grid_quotient(float x, float s, float r) {
  const float q1 = x * r;
  return copysignf(fmaf(fmaf(-q1, s, x), r, q1), x);
}

// Byte of two e2m1 codes: the code of lo in the low nibble, of hi in the high.
__device__ __forceinline__ uint32_t e2m1x2_byte(float lo, float hi) {
  uint32_t d;
  asm("{\n\t.reg .b8 t;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
      "cvt.u32.u8 %0, t;\n\t}"
      : "=r"(d)
      : "f"(hi), "f"(lo));
  return d;
}

// One row to a plane of format KF, eight fp32 values x a lane (16 lanes a row, every lane
// of the warp takes part).  up: 1 / outer scale (NVFP4; a power of two, so the product is
// exact).  `write` is the same in the row's lanes.
//  e4m3: one fp32 scale a row, the rule in idx_ops.cuh; a NaN makes scale and codes NaN.
//  NVFP4: a NaN makes its group's scale NaN; an infinity, and what lies past 6 * 448, is
//  held as 6 * 448.
template <int KF>
__device__ __forceinline__ void put_row(float (&x)[8], float up, uint8_t* payload, void* scale,
                                        unsigned long long row, int lane, bool write) {
  if (KF == kBf16) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      memcpy(&w[e], &v, 4);
    }
    if (write) reinterpret_cast<uint4*>(payload + row * 256)[lane] = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
  float m = 0.f;
  if (KF == kNvfp4) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= up;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmax_nan(m, fabsf(x[e]));
#pragma unroll
  for (int o = KF == kFp8 ? 8 : 1; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (KF == kFp8) {
    const float amax = fmax_nan(m, kAmaxFloor), f = e4m3_up(amax);
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = e4m3x2(__fmul_rn(x[2 * e], f), __fmul_rn(x[2 * e + 1], f));
    if (write) {
      reinterpret_cast<uint2*>(payload + row * 128)[lane] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      if (lane == 0) static_cast<float*>(scale)[row] = __fdiv_rn(amax, kE4m3Max);
    }
    return;
  }
  const uint32_t s_code = e4m3x2(__fdiv_rn(m, 6.0f), 0.f) & 0x7fu;
  const float s = e4m3_magnitude(s_code);
  uint32_t c = 0;
  if (s > 0.f && m == m) {
    const float r = __frcp_rn(s);
    if (m > 0x1p120f) {   // no quotient of it is finite
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaxf(fminf(x[e], 0x1p120f), -0x1p120f);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c |= e2m1x2_byte(grid_quotient(x[2 * e], s, r), grid_quotient(x[2 * e + 1], s, r)) << (8 * e);
  }
  // the row's eight scales in its first lane
  uint2 all;
  {
    uint32_t b = s_code << (8 * ((lane >> 1) & 3));
    if (lane & 1) b = 0;
    b |= __shfl_xor_sync(0xffffffffu, b, 2);
    b |= __shfl_xor_sync(0xffffffffu, b, 4);
    all = make_uint2(b, __shfl_xor_sync(0xffffffffu, b, 8));
  }
  if (write) {
    reinterpret_cast<uint32_t*>(payload + row * 64)[lane] = c;
    if (lane == 0) reinterpret_cast<uint2*>(scale)[row] = all;
  }
}

__device__ __forceinline__ void bf16x8_to_f32(uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

}  // namespace idx
