// Queries, keys and values of new tokens from the layer's projection to where the attention
// takes them from: norm head by head, rotation by position, the keys and values into the
// paged cache.
//
// What it computes, in fp32, per token and head of 128 elements x:
//   y = x / sqrt(mean(x^2) + eps) * weight       (queries and keys; without a weight y = x)
//   pair (a, b) of the first rotary_dim elements, pair i at position p of its axis:
//     a' = a cos - b sin,  b' = b cos + a sin    with (cos, sin) = table[p][i]
//   queries: rounded to bf16, or e4m3 codes with one fp32 scale a row; keys: rounded once
//   into the cache's type, as the values, which are neither normed nor rotated.
// A position outside the table gives NaN.
//
// What bounds it: 256 bytes in and 256, 132 or 72 out a row: HBM, and for a decode step's
// few rows the launch.  16 lanes hold a row, so a row's sum is four shuffles and its
// pairs' other halves (rotary_dim / 2 elements away) one shuffle an element.
#include <cuda_bf16.h>
#include <stdint.h>

#include "idx_internal.cuh"
#include "idx_ops.cuh"
#include "idx_rows.cuh"

namespace idx {

namespace {

constexpr int kTokens = 16;   // of a 256-thread CTA, a half warp each

// kRows rows of a token a half warp: their loads all go out before any is used, and the
// token's cosines and sines are loaded once for them.
template <int KF, int kRows>
__global__ void __launch_bounds__(256) norm_rope_store_kernel(const RopeArgs a, int chunks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int chunk = blockIdx.x % chunks, lane = threadIdx.x & 15;
  const long long want = (long long)(blockIdx.x / chunks) * kTokens + threadIdx.x / 16;
  const bool live = want < a.tokens;     // lanes past the last token only take part in the shuffles
  const long long tok = live ? want : a.tokens - 1;
  const int first = chunk * kRows;
  uint4 u[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int row = first + j;
    u[j] = make_uint4(0, 0, 0, 0);
    if (row < a.rows) {
      const int kind = row < a.q_heads ? 0 : row < a.q_heads + a.kv_heads ? 1 : 2;
      const int head = row - (kind == 0 ? 0 : kind == 1 ? a.q_heads : a.q_heads + a.kv_heads);
      const uint16_t* src = kind == 0 ? a.src[0] : kind == 1 ? a.src[1] : a.src[2];
      const long long stride = kind == 0 ? a.stride[0] : kind == 1 ? a.stride[1] : a.stride[2];
      u[j] = __ldcs(reinterpret_cast<const uint4*>(src + tok * stride + head * kDim) + lane);
    }
  }
  unsigned long long slot = ~0ull;
  if (first + kRows > a.q_heads) slot = (unsigned long long)__ldg(reinterpret_cast<const long long*>(a.slots) + tok);

  // cos and sin of the lane's eight elements; the sine negative for a pair's first
  float c[8], s[8];
  const int half = a.rotary_dim / 2;
  const bool turned = lane * 8 < a.rotary_dim && first < a.q_heads + a.kv_heads;
  int other = lane;                      // the lane with the other halves of the lane's pairs
  if (turned) {
    const bool second = !a.interleaved && lane * 8 >= half;
    const int pair0 = a.interleaved ? lane * 4 : lane * 8 - (second ? half : 0);
    if (!a.interleaved) other = second ? lane - half / 8 : lane + half / 8;
    const float nan = __int_as_float(0x7fffffff);
    const int n = a.interleaved ? 4 : 8;
    // axes of the lane's pairs, two bits each (pair0 is a multiple of four, or of eight)
    const uint32_t axes = a.axes > 1 ? a.pair_axis[pair0 / 16] >> (2 * (pair0 % 16)) : 0u;
    const uint32_t same = (axes & 3u) * 0x5555u;
    const uint32_t mask = n == 8 ? 0xffffu : 0xffu;
    float cs[8], sn[8];
    if (((axes ^ same) & mask) == 0u) {
      const int p = __ldg(a.positions + (long long)(axes & 3u) * a.tokens + tok);
      const bool ok = p >= 0 && p < a.num_positions;
      const float* t = a.table + (long long)(ok ? p : 0) * a.rotary_dim + pair0;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        if (e >= n) break;
        const float4 x = __ldg(reinterpret_cast<const float4*>(t + e));
        const float4 z = __ldg(reinterpret_cast<const float4*>(t + half + e));
        cs[e] = ok ? x.x : nan, cs[e + 1] = ok ? x.y : nan, cs[e + 2] = ok ? x.z : nan, cs[e + 3] = ok ? x.w : nan;
        sn[e] = z.x, sn[e + 1] = z.y, sn[e + 2] = z.z, sn[e + 3] = z.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= n) break;
        const int p = __ldg(a.positions + (long long)((axes >> (2 * e)) & 3u) * a.tokens + tok);
        const bool ok = p >= 0 && p < a.num_positions;
        const float* t = a.table + (long long)(ok ? p : 0) * a.rotary_dim + pair0 + e;
        cs[e] = ok ? __ldg(t) : nan;
        sn[e] = __ldg(t + half);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[e] = a.interleaved ? cs[e / 2] : cs[e];
      s[e] = a.interleaved ? ((e & 1) ? sn[e / 2] : -sn[e / 2]) : second ? sn[e] : -sn[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = 1.f, s[e] = 0.f;
  }

#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int row = first + j;
    if (row >= a.rows) break;
    const int kind = row < a.q_heads ? 0 : row < a.q_heads + a.kv_heads ? 1 : 2;
    const int head = row - (kind == 0 ? 0 : kind == 1 ? a.q_heads : a.q_heads + a.kv_heads);
    float x[8];
    bf16x8_to_f32(u[j], x);
    if (kind < 2) {
      const uint16_t* weight = kind ? a.weight[1] : a.weight[0];
      if (weight) {
        float w[8], sum = 0.f;
        bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(weight) + lane), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float rstd = rsqrtf(sum / (float)kDim + a.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * rstd * w[e];
      }
      if (a.table) {
        float y[8];
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], other, 16);
        }
        if (turned) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = fmaf(x[e], c[e], y[e] * s[e]);
        }
      }
    }
    if (kind == 0) {
      const unsigned long long at = (unsigned long long)tok * a.q_heads + head;
      if (a.out_q_scale)
        put_row<kFp8>(x, 1.f, static_cast<uint8_t*>(a.out_q), a.out_q_scale, at, lane, live);
      else
        put_row<kBf16>(x, 1.f, static_cast<uint8_t*>(a.out_q), nullptr, at, lane, live);
    } else {
      const bool write = live && slot < (unsigned long long)a.num_slots;   // negative: past every slot
      const unsigned long long at = ((slot >> 6) * a.kv_heads + head) * kPage + (slot & (kPage - 1));
      put_row<KF>(x, kind == 1 ? a.up[0] : a.up[1], kind == 1 ? a.payload[0] : a.payload[1],
                  kind == 1 ? a.scale[0] : a.scale[1], at, lane, write);
    }
  }
}

template <int KF>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
  // four rows a half warp once that still gives every SM a CTA or two
  const long long groups = (a.tokens + kTokens - 1) / kTokens;
  const bool many = groups * a.rows >= 152 * 8;
  const int per = many ? 4 : 1, chunks = (a.rows + per - 1) / per;
  const int grid = (int)(groups * chunks);
  return many ? launch_pdl(norm_rope_store_kernel<KF, 4>, grid, 256, 0, stream, a, chunks)
              : launch_pdl(norm_rope_store_kernel<KF, 1>, grid, 256, 0, stream, a, chunks);
}

}  // namespace

cudaError_t launch_norm_rope_store(int key_format, const RopeArgs& a, cudaStream_t stream) {
  const cudaError_t e = key_format == kBf16   ? launch<kBf16>(a, stream)
                        : key_format == kFp8 ? launch<kFp8>(a, stream)
                                             : launch<kNvfp4>(a, stream);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace idx
