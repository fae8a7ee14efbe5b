// Residual addition + root-mean-square norm with an e4m3 result.
//
// What it computes, per row of n elements (fp32 throughout):
//   h = x + residual;  residual' = bf16(h);  y = h / sqrt(mean(h^2) + eps) * weight;
//   per group (128 elements, or the whole row): a = max(max |y|, 2^-96),
//   scale = a / 448, code = e4m3(y * (448 * (1 / a))), round to nearest even, saturating.
// The norm is taken of the unrounded sum h.  The maximum passes a NaN on, so a
// row that holds one gets NaN scales and codes instead of finite nonsense.
//
// What bounds it: 7 bytes an element (x, residual in; residual, codes out)
// against ~6 flop, so HBM; a few rows are a matter of latency.
//
// How: a row stays in registers between the two passes over it (sum of squares,
// then maximum and codes), so every byte crosses HBM once.  Rows of a multiple of 8
// elements on 16-byte boundaries take 16-byte accesses: a row of up to 128 elements
// belongs to 16 lanes, up to 512 to a warp (neither needs a barrier), a longer one
// to a CTA.  Any other row goes element by element through shared memory.
//
// Measured: 16000 x 5120 with one scale a row 87.4 to 88.1 us, 6.5 TB/s, 0.96 of the copy
// peak (89.7 a call, back to back); 9000 x 8192 in groups 79 us, 0.97; 16000 x 1024 19.3 us, 0.88; 16000 x 128 3.1
// us (from L2); 64 x 6144 2.6 us, latency.  Element by element 16000 x 1001 takes 64
// us, 0.26 (a warp a row with the elements in registers: 89).
#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

#include "idx_internal.cuh"
#include "idx_ops.cuh"

namespace idx {

namespace {

constexpr int kGroup = 128;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int kLanes>
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x = fmax_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// Sum (or NaN-keeping maximum) over the block; `buf` holds one float a warp and
// is free again after the next block-wide barrier.
template <bool kMax>
__device__ __forceinline__ float block_reduce(float x, float* buf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  x = kMax ? lanes_max<32>(x) : warp_sum(x);
  if (lane == 0) buf[warp] = x;
  __syncthreads();
  float v = lane < warps ? buf[lane] : 0.f;
  return kMax ? lanes_max<32>(v) : warp_sum(v);
}

__device__ __forceinline__ float2 unpack(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Sum (or maximum) over the threads of a row: kLanes of a warp, or (0) the block.
template <bool kMax, int kLanes>
__device__ __forceinline__ float row_reduce(float x, float* buf) {
  if constexpr (kLanes == 0) {
    return block_reduce<kMax>(x, buf);
  } else {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, x, o);
      x = kMax ? fmax_nan(x, y) : x + y;
    }
    return x;
  }
}

// kVec 16-byte pieces a thread.  kLanes: threads of a row (16 or 32, 256 threads of
// them a CTA), or 0: a CTA a row.
template <int kVec, int kLanes>
__global__ void __launch_bounds__(kLanes ? 256 : 1024) norm_vec_kernel(const NormArgs a) {
  __shared__ float buf[2][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int nt = kLanes ? kLanes : blockDim.x, t = kLanes ? threadIdx.x % kLanes : threadIdx.x;
  constexpr int kRows = kLanes ? 256 / (kLanes ? kLanes : 1) : 1;   // of a CTA
  const long long want = (long long)blockIdx.x * kRows + (kLanes ? threadIdx.x / (256 / kRows) : 0);
  const bool live = want < a.rows;       // lanes past the last row only take part in the shuffles
  const long long row = live ? want : 0;
  const int nv = live ? a.dim / 8 : 0;
  const uint4* x = reinterpret_cast<const uint4*>(a.x + row * a.x_stride);
  const uint4* res = a.residual ? reinterpret_cast<const uint4*>(a.residual + row * a.residual_stride) : nullptr;
  const uint4* w = reinterpret_cast<const uint4*>(a.weight);
  float h[kVec][8];
  uint4 ux[kVec], ur[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int v = t + j * nt;
    ux[j] = ur[j] = make_uint4(0, 0, 0, 0);
    if (v < nv) {
      ux[j] = __ldcs(x + v);
      if (res) ur[j] = __ldcs(res + v);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int v = t + j * nt;
    const uint32_t wx[4] = {ux[j].x, ux[j].y, ux[j].z, ux[j].w};
    const uint32_t wr[4] = {ur[j].x, ur[j].y, ur[j].z, ur[j].w};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 p = unpack(wx[e]), q = unpack(wr[e]);
      // without a residual the sum is x itself (x + 0 would turn -0 into +0)
      const float s0 = res ? p.x + q.x : p.x, s1 = res ? p.y + q.y : p.y;
      h[j][2 * e] = s0, h[j][2 * e + 1] = s1;
      sum = fmaf(s0, s0, fmaf(s1, s1, sum));
      o[e] = pack(s0, s1);
    }
    if (a.out_residual && v < nv)
      __stcs(reinterpret_cast<uint4*>(a.out_residual + row * a.dim) + v, make_uint4(o[0], o[1], o[2], o[3]));
  }
  const float rstd = rsqrtf(row_reduce<false, kLanes>(sum, buf[0]) / (float)a.dim + a.eps);
  float top = 0.f, group_top[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int v = t + j * nt;
    float m = 0.f;
    if (v < nv) {
      const uint4 u = __ldg(w + v);
      const uint32_t ww[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack(ww[e]);
        h[j][2 * e] = h[j][2 * e] * rstd * f.x;
        h[j][2 * e + 1] = h[j][2 * e + 1] * rstd * f.y;
        m = fmax_nan(m, fmax_nan(fabsf(h[j][2 * e]), fabsf(h[j][2 * e + 1])));
      }
    }
    group_top[j] = m;
    top = fmax_nan(top, m);
  }
  if (!a.group) top = row_reduce<true, kLanes>(top, buf[1]);
  const int groups = a.group ? (a.dim + kGroup - 1) / kGroup : 1;
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const int v = t + j * nt;
    // a group of 128 is 16 lanes' pieces
    const float m = a.group ? lanes_max<16>(group_top[j]) : top;
    const float amax = fmax_nan(m, kAmaxFloor), up = e4m3_up(amax);
    if (v < nv) {
      const uint32_t lo = e4m3x2(h[j][0] * up, h[j][1] * up) | (e4m3x2(h[j][2] * up, h[j][3] * up) << 16);
      const uint32_t hi = e4m3x2(h[j][4] * up, h[j][5] * up) | (e4m3x2(h[j][6] * up, h[j][7] * up) << 16);
      __stcs(reinterpret_cast<uint2*>(a.out + row * a.dim) + v, make_uint2(lo, hi));
      if (a.group ? (v & 15) == 0 : v == 0)
        a.out_scale[row * groups + (a.group ? v / 16 : 0)] = __fdiv_rn(amax, kE4m3Max);
    }
  }
}

// Any length and alignment: the row's sums, then its products, in shared memory.
__global__ void __launch_bounds__(256) norm_any_kernel(const NormArgs a) {
  extern __shared__ float hs[];
  __shared__ float buf[2][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long row = blockIdx.x;
  const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(a.x) + row * a.x_stride;
  const __nv_bfloat16* res = a.residual ? reinterpret_cast<const __nv_bfloat16*>(a.residual) + row * a.residual_stride : nullptr;
  const __nv_bfloat16* w = reinterpret_cast<const __nv_bfloat16*>(a.weight);
  __nv_bfloat16* out_res = reinterpret_cast<__nv_bfloat16*>(a.out_residual) + row * a.dim;
  float sum = 0.f;
  for (int d = threadIdx.x; d < a.dim; d += blockDim.x) {
    float h = __bfloat162float(x[d]);
    if (res) h += __bfloat162float(res[d]);
    hs[d] = h;
    sum = fmaf(h, h, sum);
    if (a.out_residual) out_res[d] = __float2bfloat16_rn(h);
  }
  const float rstd = rsqrtf(block_reduce<false>(sum, buf[0]) / (float)a.dim + a.eps);
  float top = 0.f;
  for (int d = threadIdx.x; d < a.dim; d += blockDim.x) {   // each thread's own elements
    hs[d] = hs[d] * rstd * __bfloat162float(w[d]);
    top = fmax_nan(top, fabsf(hs[d]));
  }
  if (!a.group) top = block_reduce<true>(top, buf[1]);
  __syncthreads();
  const int group = a.group ? kGroup : a.dim, groups = (a.dim + group - 1) / group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  // a warp a group of 128, or all warps over the whole row
  for (int gi = a.group ? warp : 0; gi < groups; gi += a.group ? warps : 1) {
    const int d0 = gi * group, d1 = min(a.dim, d0 + group);
    float m = top;
    if (a.group) {
      m = 0.f;
      for (int d = d0 + lane; d < d1; d += 32) m = fmax_nan(m, fabsf(hs[d]));
      m = lanes_max<32>(m);
    }
    const float amax = fmax_nan(m, kAmaxFloor), up = e4m3_up(amax);
    const int first = a.group ? lane : threadIdx.x, step = a.group ? 32 : (int)blockDim.x;
    for (int d = d0 + first; d < d1; d += step)
      a.out[row * a.dim + d] = (uint8_t)(e4m3x2(hs[d] * up, 0.f) & 0xffu);
    if (first == 0) a.out_scale[row * groups + gi] = __fdiv_rn(amax, kE4m3Max);
  }
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t stream) {
  auto on16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool vec = a.dim % 8 == 0 && a.x_stride % 8 == 0 && a.residual_stride % 8 == 0 &&
                   on16(a.x) && on16(a.residual) && on16(a.weight) && on16(a.out_residual) &&
                   (reinterpret_cast<uintptr_t>(a.out) & 7) == 0;
  cudaError_t e;
  const int nv = a.dim / 8;
  auto grid_of = [&](int rows) { return (int)((a.rows + rows - 1) / rows); };
  if (vec && nv <= 16) {
    e = launch_pdl(norm_vec_kernel<1, 16>, grid_of(16), 256, 0, stream, a);
  } else if (vec && nv <= 64) {
    e = nv <= 32 ? launch_pdl(norm_vec_kernel<1, 32>, grid_of(8), 256, 0, stream, a)
                 : launch_pdl(norm_vec_kernel<2, 32>, grid_of(8), 256, 0, stream, a);
  } else if (vec) {
    // two pieces a thread; four for many long rows: more CTAs an SM then overlap
    // one row's passes with another's loads (9000 x 8192: 91 -> 79 us, 6000 x 12288:
    // 112 -> 81; but 64 x 6144 2.6 -> 3.4)
    const int per = (nv > 640 && a.rows >= 1024) || nv > 2048 ? 4 : 2;
    int threads = ((nv + per - 1) / per + 31) / 32 * 32;
    threads = threads < 64 ? 64 : threads;
    e = per == 2 ? launch_pdl(norm_vec_kernel<2, 0>, grid_of(1), threads, 0, stream, a)
                 : launch_pdl(norm_vec_kernel<4, 0>, grid_of(1), threads, 0, stream, a);
  } else {
    static std::atomic<unsigned long long> attr_done{0};
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = smem_limit_once(norm_any_kernel, kMaxNormDim * (int)sizeof(float), dev, attr_done);
    if (e == cudaSuccess) e = launch_pdl(norm_any_kernel, grid_of(1), 256, (size_t)a.dim * sizeof(float), stream, a);
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace idx
