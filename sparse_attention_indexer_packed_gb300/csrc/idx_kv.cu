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
// the row maximum is four shuffles.  A CTA takes consecutive tokens of one head
// and one plane, whose rows and scales lie side by side in the cache: their writes
// fill whole sectors (one row a half warp, heads of a token side by side: 26.6 us
// instead of 18.8 on 32K tokens x 4 heads to e4m3).
// Measured: that store 18.1 us, 5.6 TB/s, 0.83 of the copy peak (issue slots 84%
// used); 32K x 4 heads bf16 22.1 us, 0.90; 50,001 index keys bf16 4.1 us.
#include <cuda_bf16.h>
#include <stdint.h>

#include "idx_internal.cuh"
#include "idx_ops.cuh"

namespace idx {

namespace {

constexpr int kRowsAtOnce = 16;   // rows of a 256-thread CTA at a time

__device__ __forceinline__ __nv_bfloat162 magnitudes(uint32_t w) {
  w &= 0x7fff7fffu;
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}

// Each 16 lanes store kTokens rows, kRowsAtOnce tokens apart; their loads all go
// out before any is used.
template <int KF, int kTokens>
__global__ void __launch_bounds__(256) store_kv_kernel(const StoreArgs a, int chunks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int hp = blockIdx.x / chunks, chunk = blockIdx.x - hp * chunks;
  const int plane = hp >= a.heads, h = hp - (plane ? a.heads : 0);
  const int lane = threadIdx.x & 15;
  const uint16_t* src = (plane ? a.src[1] : a.src[0]) + h * kDim;
  const long long stride = plane ? a.stride[1] : a.stride[0];
  uint8_t* payload = plane ? a.payload[1] : a.payload[0];
  const long long tok0 = (long long)chunk * (kRowsAtOnce * kTokens) + threadIdx.x / 16;
  uint4 u[kTokens];
  long long row[kTokens];
#pragma unroll
  for (int j = 0; j < kTokens; ++j) {
    const long long tok = tok0 + j * kRowsAtOnce;
    u[j] = make_uint4(0, 0, 0, 0);
    row[j] = -1;
    if (tok < a.tokens) {
      u[j] = __ldcs(reinterpret_cast<const uint4*>(src + tok * stride) + lane);
      row[j] = __ldg(reinterpret_cast<const long long*>(a.slots) + tok);
    }
  }
#pragma unroll
  for (int j = 0; j < kTokens; ++j) {
    const unsigned long long slot = (unsigned long long)row[j];   // negative: past every slot
    const bool write = slot < (unsigned long long)a.num_slots;
    const unsigned long long r = ((slot >> 6) * a.heads + h) * kPage + (slot & (kPage - 1));
    if (KF == kBf16) {
      if (write) reinterpret_cast<uint4*>(payload + r * 256)[lane] = u[j];
      continue;
    }
    const uint32_t w[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
    // the row's largest magnitude on bf16 pairs, a NaN kept
    __nv_bfloat162 m2 = __hmax2_nan(__hmax2_nan(magnitudes(w[0]), magnitudes(w[1])),
                                    __hmax2_nan(magnitudes(w[2]), magnitudes(w[3])));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m2 = __hmax2_nan(m2, __shfl_xor_sync(0xffffffffu, m2, o));
    const float m = fmax_nan(__low2float(m2), __high2float(m2));
    const float amax = fmax_nan(m, kAmaxFloor), up = e4m3_up(amax);
    if (!write) continue;
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c[e] = e4m3x2(__fmul_rn(__uint_as_float(w[e] << 16), up),
                    __fmul_rn(__uint_as_float(w[e] & 0xffff0000u), up));
    reinterpret_cast<uint2*>(payload + r * 128)[lane] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    if (lane == 0) (plane ? a.scale[1] : a.scale[0])[r] = __fdiv_rn(amax, kE4m3Max);
  }
}

template <int KF>
cudaError_t launch(const StoreArgs& a, cudaStream_t stream) {
  // four rows a thread once that still gives every SM a CTA or two
  const bool many = a.tokens * a.heads * a.planes >= 16384;
  const int per = kRowsAtOnce * (many ? 4 : 1);
  const int chunks = (int)((a.tokens + per - 1) / per);
  const int grid = chunks * a.heads * a.planes;
  return many ? launch_pdl(store_kv_kernel<KF, 4>, grid, 256, 0, stream, a, chunks)
              : launch_pdl(store_kv_kernel<KF, 1>, grid, 256, 0, stream, a, chunks);
}

}  // namespace

cudaError_t launch_store_kv(int key_format, const StoreArgs& a, cudaStream_t stream) {
  const cudaError_t e = key_format == kBf16 ? launch<kBf16>(a, stream) : launch<kFp8>(a, stream);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace idx
