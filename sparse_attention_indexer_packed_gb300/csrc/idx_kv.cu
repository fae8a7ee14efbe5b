// Store of new keys and values into the paged cache.
//
// What it computes: token i of head h goes to plane row
// (slot / 64 * heads + h) * 64 + slot % 64 of the keys' and the values' plane.
// bf16 planes take the bits; e4m3 planes take codes and one fp32 scale a row
// (the rule in idx_ops.cuh; the reciprocal and the products are single fp32
// roundings, so the stored bytes are the same wherever they are computed).
//
// What bounds it: 256 bytes in and 256 (or 132) out a row: HBM, and for a decode
// step's few rows the launch.  16 lanes hold a row (one 16-byte load a lane), so
// a warp's loads cover two whole rows and the row maximum is four shuffles.
#include <stdint.h>

#include "idx_internal.cuh"
#include "idx_ops.cuh"

namespace idx {

namespace {

template <int KF>
__global__ void __launch_bounds__(256) store_kv_kernel(const StoreArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long rows = a.tokens * a.heads;
  const long long item = (long long)blockIdx.x * (blockDim.x / 16) + threadIdx.x / 16;
  const int lane = threadIdx.x & 15;
  const int plane = item >= rows;
  const long long k = item - (plane ? rows : 0);
  const bool live = k < rows && plane < a.planes;
  long long slot = -1;
  uint4 u = make_uint4(0, 0, 0, 0);
  long long tok = 0;
  int h = 0;
  if (live) {
    tok = k / a.heads;
    h = (int)(k - tok * a.heads);
    slot = __ldg(reinterpret_cast<const long long*>(a.slots) + tok);
    const uint16_t* src = plane ? a.src[1] + tok * a.stride[1] : a.src[0] + tok * a.stride[0];
    u = __ldg(reinterpret_cast<const uint4*>(src + h * kDim) + lane);
  }
  const bool write = slot >= 0 && slot < a.num_slots;
  const long long row = (slot / kPage * a.heads + h) * kPage + slot % kPage;
  uint8_t* payload = plane ? a.payload[1] : a.payload[0];
  if (KF == kBf16) {
    if (write) reinterpret_cast<uint4*>(payload + row * 256)[lane] = u;
    return;
  }
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  float x[8], m = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(w[e] << 16);
    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    m = fmax_nan(m, fmax_nan(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float amax = fmax_nan(m, kAmaxFloor), up = e4m3_up(amax);
  if (!write) return;
  const uint32_t lo = e4m3x2(__fmul_rn(x[0], up), __fmul_rn(x[1], up)) |
                      (e4m3x2(__fmul_rn(x[2], up), __fmul_rn(x[3], up)) << 16);
  const uint32_t hi = e4m3x2(__fmul_rn(x[4], up), __fmul_rn(x[5], up)) |
                      (e4m3x2(__fmul_rn(x[6], up), __fmul_rn(x[7], up)) << 16);
  reinterpret_cast<uint2*>(payload + row * 128)[lane] = make_uint2(lo, hi);
  if (lane == 0) (plane ? a.scale[1] : a.scale[0])[row] = __fdiv_rn(amax, kE4m3Max);
}

}  // namespace

cudaError_t launch_store_kv(int key_format, const StoreArgs& a, cudaStream_t stream) {
  const long long items = a.tokens * a.heads * a.planes;
  const int grid = (int)((items + 15) / 16);
  cudaError_t e = key_format == kBf16 ? launch_pdl(store_kv_kernel<kBf16>, grid, 256, 0, stream, a)
                                      : launch_pdl(store_kv_kernel<kFp8>, grid, 256, 0, stream, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace idx
