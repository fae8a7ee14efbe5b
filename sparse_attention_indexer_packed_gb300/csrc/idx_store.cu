// NVFP4 quantize-store of staged bf16 keys into the paged pool planes.
//
// What it computes (ROCm/ATOM #2745, Summary, "Store" and "Write"): each key of
// D = 128 is quantised per group of 16 elements with scale = E4M3(amax / 6) and
// e2m1 codes rounded half-to-even that saturate at 6, with a unit outer scale;
// two codes per byte, the even element in the low nibble; the payload (64 B) and
// the scale byte of each group (8 B) go to the key's real slot in two planes.
//
// Readings of the points the page leaves open: amax and amax/6 in fp32 with a
// correctly rounded division; the scale rounds half-to-even and saturates at
// 448; a zero scale writes all-zero codes; codes are those of the correctly
// rounded fp32 quotient x / scale; a negative value that rounds to zero keeps
// its sign.  An infinity counts as the largest finite value of its sign; a NaN is left out of
// amax and takes the code of 6 (the conversion's).
//
// (How the codes are found without a division each: idx_rows.cuh.)
//
// One thread per (key, group of 16): eight threads cover a key, a warp four.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "idx_internal.cuh"
#include "idx_rows.cuh"

namespace idx {

namespace {

// Two bf16 with infinities as the largest finite value of their sign; a NaN stays.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w) {
  const __nv_bfloat162 v = __hmax2_nan(__hmin2_nan(as_bf16x2(w), as_bf16x2(0x7f7f7f7fu)), as_bf16x2(0xff7fff7fu));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Quantise one group (its 16 bf16 values in w) and write it.
__device__ __forceinline__ void store_group(const uint32_t (&w)[8], int64_t row, int grp,
                                            uint8_t* payload, uint8_t* scale) {
  // amax of the 16 magnitudes (a max is exact in any order)
  __nv_bfloat162 m2 = as_bf16x2(w[0] & 0x7fff7fffu);
#pragma unroll
  for (int e = 1; e < 8; ++e) m2 = __hmax2(m2, as_bf16x2(w[e] & 0x7fff7fffu));
  const float amax = fmaxf(__low2float(m2), __high2float(m2));
  const float s_f = __fdiv_rn(amax, 6.0f);
  const uint32_t s_code =
      (uint32_t)__nv_cvt_float_to_fp8(s_f, __NV_SATFINITE, __NV_E4M3) & 0x7fu;
  const float s = e4m3_magnitude(s_code);
  uint32_t lo = 0, hi = 0;
  if (s > 0.f) {
    const float nr = -__frcp_rn(s);
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = w[e];
    if (amax == INFINITY) {   // an infinity's residual would be inf - inf: the largest finite value saturates too
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = finite_bf16x2(v[e]);
    }
    float2 q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = grid_quotient(neg_bf16x2(v[e]), s, nr);
    lo = e2m1x8(q[0], q[1], q[2], q[3]);
    hi = e2m1x8(q[4], q[5], q[6], q[7]);
  }
  *reinterpret_cast<uint2*>(payload + row * 64 + grp * 8) = make_uint2(lo, hi);
  scale[row * 8 + grp] = (uint8_t)s_code;
}

// Each thread quantises kGroups groups, blockDim apart (each load instruction
// of a warp covers 1 KB of consecutive keys); all their loads go out before
// any of them is used.
constexpr int kGroups = 2;

__global__ void __launch_bounds__(256) store_nvfp4_kernel(const uint16_t* __restrict__ src,
                                                          const int64_t* __restrict__ slot_mapping,
                                                          int64_t num_tokens, uint8_t* payload,
                                                          uint8_t* scale, int64_t num_rows) {
  const int64_t base = (int64_t)blockIdx.x * blockDim.x * kGroups + threadIdx.x;
  uint4 u[kGroups][2];
  int64_t row[kGroups];
#pragma unroll
  for (int j = 0; j < kGroups; ++j) {
    const int64_t gid = base + (int64_t)j * blockDim.x;
    const int64_t tok = gid >> 3;
    row[j] = -1;
    if (tok < num_tokens) {
      // the key's bytes do not depend on its slot: the loads go out together
      const uint4* p = reinterpret_cast<const uint4*>(src + tok * kDim + (gid & 7) * 16);
      row[j] = __ldg(slot_mapping + tok);
      u[j][0] = __ldcs(p);
      u[j][1] = __ldcs(p + 1);
    }
  }
#pragma unroll
  for (int j = 0; j < kGroups; ++j) {
    if (row[j] < 0 || row[j] >= num_rows) continue;
    const uint32_t w[8] = {u[j][0].x, u[j][0].y, u[j][0].z, u[j][0].w,
                           u[j][1].x, u[j][1].y, u[j][1].z, u[j][1].w};
    store_group(w, row[j], (int)((base + (int64_t)j * blockDim.x) & 7), payload, scale);
  }
}

}  // namespace

cudaError_t launch_store_nvfp4(const uint16_t* src, const int64_t* slot_mapping, int64_t num_tokens,
                               uint8_t* payload, uint8_t* scale, int64_t num_rows,
                               cudaStream_t stream) {
  if (num_tokens <= 0) return cudaSuccess;
  const int64_t groups = num_tokens * 8;
  const int64_t blocks = (groups + 256 * kGroups - 1) / (256 * kGroups);
  store_nvfp4_kernel<<<(unsigned)blocks, 256, 0, stream>>>(src, slot_mapping, num_tokens, payload,
                                                         scale, num_rows);
  return cudaGetLastError();
}

}  // namespace idx
