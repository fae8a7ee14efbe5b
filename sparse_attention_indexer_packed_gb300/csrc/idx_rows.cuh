// Rows of 128 held by 16 lanes, eight elements a lane, and their quantisation: what the
// store and the norm, rotation and store pass have in common; and the NVFP4 rule.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>
#include <string.h>

#include "idx_internal.cuh"
#include "idx_ops.cuh"
#include "idx_ptx.cuh"

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

// x / s on the e2m1 midpoints, within two ulps elsewhere (see above), of two elements from
// -x: q1 = (-x) (-r), the residual q1 s - x, q2 = q1 - residual r.  In this form a zero keeps
// its sign.  nr = -1 / s.
__device__ __forceinline__ float2 grid_quotient(float2 neg_x, float s, float nr) {
  const float2 r2 = make_float2(nr, nr), q1 = fmul2_rn(neg_x, r2);
  return ffma2_rn(ffma2_rn(q1, make_float2(s, s), neg_x), r2, q1);
}

// Eight e2m1 codes (half to even, saturating, the sign kept), the first in the low nibble.
__device__ __forceinline__ uint32_t e2m1x8(float2 a, float2 b, float2 c, float2 d) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return w;
}

// The scale code of a group whose largest magnitude is m, in units of the outer scale; NaN
// (0x7f) for a NaN.
__device__ __forceinline__ uint32_t nvfp4_scale(float m) { return e4m3x2(__fdiv_rn(m, 6.0f), 0.f) & 0x7fu; }

// Codes of 2 N elements of a group, given as -x; s_code as above, m > 2^120: an element's
// quotient may not be finite.  The outer scale goes with the group's scale: a power of two,
// it changes no quotient.
template <int N>
__device__ __forceinline__ void nvfp4_codes(float2 (&neg_x)[N], uint32_t s_code, float m, float outer, float up,
                                            uint32_t (&c)[N / 4]) {
  const float s0 = e4m3_magnitude(s_code);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) c[i] = 0u;
  if (!(s0 > 0.f && m == m)) return;
  const float s = s0 * outer, nr = -__frcp_rn(s0) * up;
  if (m > 0x1p120f) {
    const float most = fminf(0x1p120f * outer, 0x1p126f);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      neg_x[e].x = fmaxf(fminf(neg_x[e].x, most), -most);
      neg_x[e].y = fmaxf(fminf(neg_x[e].y, most), -most);
    }
  }
#pragma unroll
  for (int e = 0; e < N; ++e) neg_x[e] = grid_quotient(neg_x[e], s, nr);
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    c[i] = e2m1x8(neg_x[4 * i], neg_x[4 * i + 1], neg_x[4 * i + 2], neg_x[4 * i + 3]);
}

// Two bf16 as -x.
__device__ __forceinline__ float2 neg_bf16x2(uint32_t w) {
  w ^= 0x80008000u;
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// One row to a plane of format KF, eight fp32 values x a lane (16 lanes a row, every lane
// of the warp takes part).  up: 1 / outer scale (NVFP4).  `write` is the same in the row's
// lanes.
//  e4m3: one fp32 scale a row, the rule in idx_ops.cuh; a NaN makes scale and codes NaN.
//  NVFP4: a NaN makes its group's scale NaN; an infinity, and what lies past 6 * 448, is
//  held as 6 * 448.
template <int KF>
__device__ __forceinline__ void put_row(float (&x)[8], float outer, float up, uint8_t* payload, void* scale,
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
  m *= up;
  const uint32_t s_code = nvfp4_scale(m);
  uint32_t c[1];
  float2 neg_x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) neg_x[e] = make_float2(-x[2 * e], -x[2 * e + 1]);
  nvfp4_codes(neg_x, s_code, m, outer, up, c);
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
    reinterpret_cast<uint32_t*>(payload + row * 64)[lane] = c[0];
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
