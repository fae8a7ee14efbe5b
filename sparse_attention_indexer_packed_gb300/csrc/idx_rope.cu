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
//
// Measured (one GB300): 16K tokens of 32 query, 4 key and 4 value heads 60.8 us, 0.83 of the
// copy peak (78.3 with a row at a time, 71.8 with cos and sin times the weights made once for
// four rows; long chunks loaded a batch ahead the rest); 64 tokens 2.3 us.
#include <cuda_bf16.h>
#include <stdint.h>

#include "idx_internal.cuh"
#include "idx_ops.cuh"
#include "idx_rows.cuh"

namespace idx {

namespace {

constexpr int kTokens = 16;   // of a 256-thread CTA, a half warp each

// The rows of a token in chunks of `rows` of one kind: the queries', the keys', the values'.
struct Chunks {
  int q, k, all, rows;
};

// A chunk of a token a half warp, kRows rows at a time: their loads all go out before any is
// used; kMore: the chunk may have more than kRows, loaded under the arithmetic before.  What the
// rows are multiplied by, cos and sin times the norm's weights, is made once for the chunk:
// out = rstd (x A + y B), y the other half of x's pair.
template <int KF, int kRows, bool kMore>
__global__ void __launch_bounds__(256, kMore ? 3 : 4) norm_rope_store_kernel(const RopeArgs a, Chunks chunks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int chunk = blockIdx.x % chunks.all;
  const int lane = threadIdx.x & 15;
  const long long want = (long long)(blockIdx.x / chunks.all) * kTokens + threadIdx.x / 16;
  const bool live = want < a.tokens;     // lanes past the last token only take part in the shuffles
  const long long tok = live ? want : a.tokens - 1;
  const int kind = chunk < chunks.q ? 0 : chunk < chunks.k ? 1 : 2;
  chunk -= kind == 0 ? 0 : kind == 1 ? chunks.q : chunks.k;
  const int first = chunk * chunks.rows;
  const int rows = min((kind ? a.kv_heads : a.q_heads) - first, chunks.rows);
  const uint16_t* src = (kind == 0 ? a.src[0] + tok * a.stride[0]
                         : kind == 1 ? a.src[1] + tok * a.stride[1] : a.src[2] + tok * a.stride[2]) + first * kDim;
  uint4 u[kRows];
  auto load = [&](uint4(&v)[kRows], int j0) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      v[j] = make_uint4(0, 0, 0, 0);
      if (j0 + j < rows) v[j] = __ldcs(reinterpret_cast<const uint4*>(src + (j0 + j) * kDim) + lane);
    }
  };
  load(u, 0);
  unsigned long long at0, at_step;       // output row of the chunk's first row; to the next
  bool write = live;
  if (kind == 0) {
    at0 = (unsigned long long)tok * a.q_heads + first;
    at_step = 1;
  } else {
    const unsigned long long slot = (unsigned long long)__ldg(reinterpret_cast<const long long*>(a.slots) + tok);
    write = live && slot < (unsigned long long)a.num_slots;   // negative: past every slot
    at0 = ((slot >> 6) * a.kv_heads + first) * kPage + (slot & (kPage - 1));
    at_step = kPage;
  }
  uint8_t* payload = kind == 1 ? a.payload[0] : a.payload[1];
  void* scale = kind == 1 ? a.scale[0] : a.scale[1];
  const float outer = kind == 1 ? a.outer[0] : a.outer[1], up = kind == 1 ? a.up[0] : a.up[1];
  // f(row of the chunk, its words) for each row
  auto each = [&](auto&& f) {
    if constexpr (kMore) {
      for (int j0 = 0; j0 < rows; j0 += kRows) {
        uint4 next[kRows];
        load(next, j0 + kRows);
#pragma unroll
        for (int j = 0; j < kRows; ++j)
          if (j0 + j < rows) f(j0 + j, u[j]);
#pragma unroll
        for (int j = 0; j < kRows; ++j) u[j] = next[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (j < rows) f(j, u[j]);
    }
  };
  if (kind == 2) {
    each([&](int j, uint4 v) {
      if (KF == kBf16) {
        if (write) reinterpret_cast<uint4*>(payload + (at0 + j * at_step) * 256)[lane] = v;
        return;
      }
      float x[8];
      bf16x8_to_f32(v, x);
      put_row<KF>(x, outer, up, payload, scale, at0 + j * at_step, lane, write);
    });
    return;
  }

  // A and B of the lane's eight elements
  const uint16_t* weight = kind ? a.weight[1] : a.weight[0];
  const int half = a.rotary_dim / 2;
  const bool turned = lane * 8 < a.rotary_dim;
  const bool second = !a.interleaved && lane * 8 >= half;
  // the lane with the other halves of the lane's pairs
  const int other = !turned || a.interleaved ? lane : second ? lane - half / 8 : lane + half / 8;
  float A[8], B[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) A[e] = 1.f, B[e] = 0.f;
  if (turned) {
    const int pair0 = a.interleaved ? lane * 4 : lane * 8 - (second ? half : 0);
    const float nan = __int_as_float(0x7fffffff);
    // axes of the lane's pairs, two bits each (pair0 is a multiple of four, or of eight)
    const uint32_t axes = a.axes > 1 ? a.pair_axis[pair0 / 16] >> (2 * (pair0 % 16)) : 0u;
    const uint32_t mask = a.interleaved ? 0xffu : 0xffffu;
    float cs[8], sn[8];
    if (((axes ^ ((axes & 3u) * 0x5555u)) & mask) == 0u) {
      const int p = __ldg(a.positions + (long long)(axes & 3u) * a.tokens + tok);
      const bool ok = p >= 0 && p < a.num_positions;
      const float* t = a.table + (long long)(ok ? p : 0) * a.rotary_dim + pair0;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        if (e == 4 && a.interleaved) break;
        const float4 x = __ldg(reinterpret_cast<const float4*>(t + e));
        const float4 z = __ldg(reinterpret_cast<const float4*>(t + half + e));
        cs[e] = ok ? x.x : nan, cs[e + 1] = ok ? x.y : nan, cs[e + 2] = ok ? x.z : nan, cs[e + 3] = ok ? x.w : nan;
        sn[e] = z.x, sn[e + 1] = z.y, sn[e + 2] = z.z, sn[e + 3] = z.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e == 4 && a.interleaved) break;
        const int p = __ldg(a.positions + (long long)((axes >> (2 * e)) & 3u) * a.tokens + tok);
        const bool ok = p >= 0 && p < a.num_positions;
        const float* t = a.table + (long long)(ok ? p : 0) * a.rotary_dim + pair0 + e;
        cs[e] = ok ? __ldg(t) : nan;
        sn[e] = __ldg(t + half);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      A[e] = a.interleaved ? cs[e / 2] : cs[e];
      B[e] = a.interleaved ? ((e & 1) ? sn[e / 2] : -sn[e / 2]) : second ? sn[e] : -sn[e];
    }
  }
  if (weight) {
    float w[8], v[8];
    bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(weight) + lane), w);
    bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(weight) + other), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) A[e] *= w[e], B[e] *= a.interleaved ? w[e ^ 1] : v[e];
  }

  each([&](int j, uint4 words) {
    float x[8];
    bf16x8_to_f32(words, x);
    float rstd = 1.f;
    if (weight) {
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 8; e += 2) sum = ffma2_rn(make_float2(x[e], x[e + 1]), make_float2(x[e], x[e + 1]), sum);
      float all = sum.x + sum.y;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      rstd = rsqrtf(fmaf(all, 1.f / kDim, a.eps));
    }
    float y[8];
    if (a.table) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = a.interleaved ? x[e ^ 1] : __shfl_sync(0xffffffffu, x[e], other, 16);
    }
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      float2 z = fmul2_rn(make_float2(x[e], x[e + 1]), make_float2(A[e], A[e + 1]));
      if (turned) z = ffma2_rn(make_float2(y[e], y[e + 1]), make_float2(B[e], B[e + 1]), z);
      z = fmul2_rn(z, make_float2(rstd, rstd));
      x[e] = z.x, x[e + 1] = z.y;
    }
    const unsigned long long at = at0 + j * at_step;
    if (kind == 1)
      put_row<KF>(x, outer, up, payload, scale, at, lane, write);
    else if (a.out_q_scale)
      put_row<kFp8>(x, 1.f, 1.f, static_cast<uint8_t*>(a.out_q), a.out_q_scale, at, lane, write);
    else
      put_row<kBf16>(x, 1.f, 1.f, static_cast<uint8_t*>(a.out_q), nullptr, at, lane, write);
  });
}

template <int KF, int kRows, bool kMore>
cudaError_t launch_rows(const RopeArgs& a, int rows, cudaStream_t stream) {
  auto chunks_of = [&](int heads) { return (heads + rows - 1) / rows; };
  Chunks c;
  c.q = chunks_of(a.q_heads);
  c.k = c.q + chunks_of(a.kv_heads);
  c.all = c.k + (a.src[2] ? chunks_of(a.kv_heads) : 0);
  c.rows = rows;
  const int grid = (int)((a.tokens + kTokens - 1) / kTokens * c.all);
  return launch_pdl(norm_rope_store_kernel<KF, kRows, kMore>, grid, 256, 0, stream, a, c);
}

template <int KF>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream) {
  // Few rows: a CTA more for each, so that they start side by side; many: cos and sin made for
  // more of them.  40 heads to bf16, us with chunks of 1 / 4 / 16 rows: 256 tokens 3.25 / 3.15 / 6.35,
  // 480 4.7 / 3.35 / 6.4, 2000 15.0 / 9.7 / 10.3, 3800 29.8 / 19.5 / 18.4, 8000 59.5 / 37.3 / 32.7.
  const long long rows = (a.tokens + kTokens - 1) / kTokens * a.rows;
  if (rows < 152 * 4) return launch_rows<KF, 1, false>(a, 1, stream);
  if (rows < 152 * 48) return launch_rows<KF, 4, false>(a, 4, stream);
  return launch_rows<KF, 4, true>(a, 16, stream);
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
