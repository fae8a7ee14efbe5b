// Attention of the newest tokens over the paged cache: the whole cache, or the
// 128-token blocks of the index step's lists.
//
// What it computes: for packed row i of a unit (idx_attn.cuh), with query q_i
// and visible tokens T_i = { t < the row's length [, t / 128 in the row's list] },
//   s_t = scale * q_i . k_t,   lse = ln sum_T e^{s_t},   out = sum_T e^{s_t - lse} v_t
// in one pass over the keys and values, with the running maximum m and sum l of
// the softmax: a token piece with maximum m' rescales what was summed so far by
// e^{m - max(m, m')}.  A row with no visible token gives out = 0, lse = -inf.
//
// What bounds it: the cache's bytes.  16 rows cost 16 flop a byte of a bf16
// cache (32 of an e4m3 one), far below the ridge, so the tiles of a unit are
// read once for all of its rows and the work is the stream from HBM.
//
// How (sm_103a):
//  * a persistent grid, one CTA per SM; every CTA takes an equal stretch of the
//    units' 32-token pieces (idx_attn.cuh), so one long request is split over
//    many CTAs and many short ones share a CTA;
//  * where the units are many and of like lengths they are not cut: teams of 1, 2, 4
//    or 8 warps take whole units in turn, so that the cost of a unit's end (3 us for
//    a CTA) is paid by several at a time.  The host picks the team from the units'
//    number, every CTA finds from the lengths whether to deal or to cut (Cost).
//    Cut / dealt, us: bf16 64 x 8 heads x 256 tokens 26.1 / 18.1, x 1K 53.4 / 46.2,
//    x 8K 300 / 297; 256 x 8 x 100 61.7 / 26.8; 1 x 200 8.7 / 7.5; e4m3 64 x 8 x 256
//    30.3 / 13.8, x 1K 54.2 / 31.7, 256 x 8 x 100 78.7 / 22.2.  Lists: bf16 128 x 4
//    lists of 16 blocks 92.1 / 71.9, 60 x 4 of 12 38.9 / 31.7, e4m3 72.3 / 54.4 and
//    35.4 / 26.2 (the host decides; no join kernel runs).  The second way in
//    the kernel costs calls that cut 1 to 6% (1 x 1K 9.1 -> 9.4), those of e4m3 with
//    more units than SMs 9%;
//  * a warp owns one shared-memory stage of one piece (keys and values, by TMA
//    through the page table) and refills it as soon as it has been used; no
//    stage is shared between warps, so there is no "empty" barrier;
//  * a piece is two chains of m16n8k16 products on the registers: scores from
//    ldmatrix'ed keys, then the weights, still in the accumulators' layout,
//    against transposed-ldmatrix values.  An e4m3 piece is decoded to exact f16
//    in registers;
//  * warps keep softmax states of their own; they are joined through shared
//    memory at a unit's end.  A unit inside one CTA is written at once; of one
//    that was cut each CTA leaves (m, l, out) in the workspace for a join kernel.
//    (Joined in this kernel by the CTA that comes last, through tagged counters:
//    measured slower on small calls, 1 x 1K 9.4 -> 10.5 us and blocks 1 x 32K
//    11.5 -> 14.7, the fences and counter round trips costing more than the
//    second launch);
//  * every wait is bounded, as in the score kernels.
//
// Measured (one GB300, calls back to back): bf16 16 x 131K, 16 rows: 152 us, 6.49
// TB/s of cache, 0.96 of the copy peak.  e4m3 16 x 131K: 96 us, 5.3 TB/s, 0.78: the
// products' operands are decoded in registers, 8 warps of 255 registers leave the
// issue slots 34% used and the warps waiting on their own chains (12 warps of 168
// registers spill: 117 us).  Lists, 16 x 131K, 4 x 4 rows, 64 blocks: 65 us for 369 MB
// of joined blocks, 5.7 TB/s.  Short calls are latency: 1 x 1K 9.4 us (request table
// 0.9, first page id 2, first tile 4.3, output 5.7, join 8.7), 48 ragged requests
// 25 us (first tiles 5 to 8, last output 21, join 25; e4m3 29).
// Tried and slower: two e4m3 query terms on m16n8k32 (113 -> 134 us, one stage a
// warp); the next piece's scores under this one's weights with stages of their own
// for keys and values (96 -> 108); 4 warps of 2 stages for bf16 (1 x 1K 8.9 -> 8.4,
// lists 65.9 -> 68.2); units never cut when they have at most 40 pieces (1 x 1K
// 9.0 -> 10.8).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "idx_attn.cuh"
#include "idx_attn_rows.cuh"
#include "idx_ptx.cuh"

namespace idx {

namespace {

using namespace attn;

constexpr int kTile = 16;                              // packed rows of a group here
constexpr int kItem = 32;                              // tokens of a piece
constexpr int kMergeStride = kDim + 8;                 // floats: keeps row writes off one bank

template <int KF>
struct ACfg;
template <>
struct ACfg<kBf16> {
  static constexpr int kRowBytes = 256;
  static constexpr int kWarps = 8;
  static constexpr int kDepth = 1;
};
template <>
struct ACfg<kFp8> {
  static constexpr int kRowBytes = 128;
  static constexpr int kWarps = 8;
  static constexpr int kDepth = 2;
};

template <int KF>
struct ALayout {
  static constexpr int NW = ACfg<KF>::kWarps;
  static constexpr int D = ACfg<KF>::kDepth;       // stages of a warp
  static constexpr int kThreads = 32 * NW;
  static constexpr int kTileBytes = kItem * ACfg<KF>::kRowBytes;  // keys or values of a piece
  static constexpr int kStage = 2 * kTileBytes;
  static constexpr int kScaleBytes = KF == kFp8 ? 2 * kItem * 4 : 0;
  static constexpr int kScaleOff = NW * D * kStage;
  static constexpr int kMergeOff = kScaleOff + NW * D * kScaleBytes;
  static constexpr int kMlOff = kMergeOff + NW / 2 * kTile * kMergeStride * 4;
  static constexpr int kBarOff = kMlOff + NW / 2 * kTile * 8;
  static constexpr int kCtlOff = kBarOff + (NW * D + 1) * 8;       // flags, longest unit, one int a warp
  static constexpr int kPreOff = (kCtlOff + 8 + NW * 4 + 15) & ~15;
  static constexpr int kListOff = kPreOff + kRequestsBytes;
  static constexpr int kBytes = kListOff + kMaxList * 4;
  // the block bits are only held while a list is joined: in the merge area,
  // which is free between two units
  static constexpr int kBitsOff = kMergeOff;
  static constexpr int kSmem = kBytes + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t& r0, uint32_t& r1,
                                                  uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

// The 16 query rows in A-fragment order.
//  bf16: a[ks] = {row g: d 16ks+2t,+1; row g+8: same; row g: +8,+9; row g+8: +8,+9}
//  e4m3 keys: the queries as f16, scaled a row by the power of two that brings
//  the row's largest magnitude into [2^7, 2^8) (exact for every element within
//  2^21 of it, undone by post): e4m3 values are exact in f16, so each product is
//  exact.  k order: step c takes d = 16c + 4t + {0,1} and + {2,3}, the order in
//  which a lane's four bytes of an ldmatrix'ed key arrive.  (Two e4m3 query terms
//  on m16n8k32 would spare the keys' conversion; measured on the 16 x 131K decode
//  134 us against 113: the warp-level e4m3 product is the slower one here.)
template <int KF>
struct QRows {
  uint32_t a[8][4];
  float post0, post1;
  // the rows' words as they lie in memory: the loads go out, nothing waits
  __device__ __forceinline__ void load(const uint16_t* r0, const uint16_t* r1) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (KF == kBf16) {
        const int o = 16 * c + 2 * t;
        a[c][0] = r0 ? __ldg(reinterpret_cast<const uint32_t*>(r0 + o)) : 0u;
        a[c][1] = r1 ? __ldg(reinterpret_cast<const uint32_t*>(r1 + o)) : 0u;
        a[c][2] = r0 ? __ldg(reinterpret_cast<const uint32_t*>(r0 + o + 8)) : 0u;
        a[c][3] = r1 ? __ldg(reinterpret_cast<const uint32_t*>(r1 + o + 8)) : 0u;
      } else {
        const int o = 16 * c + 4 * t;
        const uint2 u = r0 ? __ldg(reinterpret_cast<const uint2*>(r0 + o)) : make_uint2(0, 0);
        const uint2 v = r1 ? __ldg(reinterpret_cast<const uint2*>(r1 + o)) : make_uint2(0, 0);
        a[c][0] = u.x, a[c][2] = u.y, a[c][1] = v.x, a[c][3] = v.y;
      }
    }
  }
  // what the scores are to be multiplied by; e4m3 keys: the rows to scaled f16
  __device__ __forceinline__ void finish(float scale_log2) {
    post0 = post1 = scale_log2;
    if (KF == kFp8) {
      post0 = fmaxf(post0 * to_f16(0), kLeastPost);
      post1 = fmaxf(post1 * to_f16(1), kLeastPost);
    }
  }
  __device__ __forceinline__ float to_f16(int half) {
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int e = half; e < 4; e += 2)
        amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(a[c][e])), fabsf(bf16_hi(a[c][e]))));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int x = to_2_7(amax);
    const float up = ldexpf(1.f, x);
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int e = half; e < 4; e += 2)
        a[c][e] = pack_f16(bf16_lo(a[c][e]) * up, bf16_hi(a[c][e]) * up);
    return ldexpf(1.f, -x);
  }
};

// Softmax state of the two rows a lane holds (g and g + 8), and its part of the
// unnormalised output.  m in log2 units, the same in the four lanes of a row;
// l is the lane's own part of the sum.  e4m3 values: o is held in units of 2^n0 and
// 2^n1 (n absolute, as m), so that weight times value scale fits f16; see raise_unit.
// (l is not: a unit far from the weights would flush what was summed before.)
struct State {
  float m0, m1, l0, l1, n0, n1;
  float o[16][4];
  __device__ __forceinline__ void reset() {
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
    n0 = n1 = -INFINITY;
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  }
};

// One 32-token piece.  kMask: some token of the piece lies outside some row
// (len0, len1: the rows' visible lengths, 0 for a row that does not list the
// block) or at or past glen, where the cache holds anything: such values are
// dropped by selection, not by a product with zero.
template <int KF, bool kMask>
__device__ __forceinline__ void piece(const QRows<KF>& q, State& st, uint32_t stage,
                                      const float* scales, int lane, int tb, int len0, int len1,
                                      int glen) {
  const int t = lane & 3, m = lane >> 3, rr = lane & 7;
  constexpr int TB = ALayout<KF>::kTileBytes;
  // the four token tiles' chains side by side
  float s[4][4];
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
  const uint32_t krow = stage + (uint32_t)(rr * 128);
#pragma unroll
  for (int c = 0; c < (KF == kBf16 ? 4 : 2); ++c) {
    const int ch = 4 * c + m;
    const uint32_t at = krow + (KF == kBf16 ? (uint32_t)((ch >> 3) * (TB / 2)) : 0u) + (uint32_t)(((ch ^ rr) & 7) << 4);
    uint32_t w[4][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) ldmatrix_x4(at + nt * 1024, w[nt][0], w[nt][1], w[nt][2], w[nt][3]);
    if (KF == kBf16) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) mma_bf16_16816(s[nt], q.a[2 * c + e], w[nt][2 * e], w[nt][2 * e + 1]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          uint32_t lo, hi;
          e4m3x4_to_f16x2x2(w[nt][e], lo, hi);
          mma_f16_16816(s[nt], q.a[4 * c + e], lo, hi);
        }
    }
  }
  // y: the scores before the rows' factor, two tokens of a row at a time; their
  // row maxima (post is positive, so it keeps the order)
  float2 y0[4], y1[4];
  float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) {
    y0[nt] = make_float2(s[nt][0], s[nt][1]);
    y1[nt] = make_float2(s[nt][2], s[nt][3]);
    if (KF == kFp8) {
      const float2 ks = *reinterpret_cast<const float2*>(scales + nt * 8 + 2 * t);
      y0[nt] = fmul2_rn(y0[nt], ks);
      y1[nt] = fmul2_rn(y1[nt], ks);
    }
    if (kMask) {
      const int t0 = tb + nt * 8 + 2 * t;
      if (t0 >= len0) y0[nt].x = -INFINITY;
      if (t0 + 1 >= len0) y0[nt].y = -INFINITY;
      if (t0 >= len1) y1[nt].x = -INFINITY;
      if (t0 + 1 >= len1) y1[nt].y = -INFINITY;
    }
    mx0 = fmaxf(mx0, fmaxf(y0[nt].x, y0[nt].y));
    mx1 = fmaxf(mx1, fmaxf(y1[nt].x, y1[nt].y));
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
  }
  const float mn0 = fmaxf(st.m0, mx0 * q.post0), mn1 = fmaxf(st.m1, mx1 * q.post1);
  const float ref0 = mn0 == -INFINITY ? 0.f : mn0, ref1 = mn1 == -INFINITY ? 0.f : mn1;
  const float c0 = ex2_approx(st.m0 - ref0), c1 = ex2_approx(st.m1 - ref1);
  float co0 = c0, co1 = c1;   // what the output gathered so far is multiplied by
  st.m0 = mn0, st.m1 = mn1;
  const float2 p0 = make_float2(q.post0, q.post0), p1 = make_float2(q.post1, q.post1);
  const float2 r0 = make_float2(-ref0, -ref0), r1 = make_float2(-ref1, -ref1);
  float f0 = 1.f, f1 = 1.f;   // weights to the output's unit
  float2 vs[4];
  if (KF == kFp8) {
    // what the weights times scales of the tokens that a row sees are at most
    float top0 = 0.f, top1 = 0.f;
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      vs[nt] = *reinterpret_cast<const float2*>(scales + kItem + nt * 8 + 2 * t);
      const float x = fabsf(vs[nt].x), y = fabsf(vs[nt].y);
      if (kMask) {
        const int t0 = tb + nt * 8 + 2 * t;
        top0 = fmaxf(top0, fmaxf(t0 < len0 ? x : 0.f, t0 + 1 < len0 ? y : 0.f));
        top1 = fmaxf(top1, fmaxf(t0 < len1 ? x : 0.f, t0 + 1 < len1 ? y : 0.f));
      } else {
        top0 = fmaxf(top0, fmaxf(x, y));
      }
    }
    if (!kMask) top1 = top0;
    co0 = co1 = 1.f;          // the unit does not move with the maximum
    f0 = to_unit(mn0, st.n0), f1 = to_unit(mn1, st.n1);
    if (__any_sync(0xffffffffu, past_unit(top0, f0) || past_unit(top1, f1))) {
      top0 = top1 = 0.f;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const float2 u = ffma2_rn(y0[nt], p0, r0), w = ffma2_rn(y1[nt], p1, r1);
        top0 = fmaxf(top0, fmaxf(fabsf(ex2_approx(u.x) * vs[nt].x), fabsf(ex2_approx(u.y) * vs[nt].y)));
        top1 = fmaxf(top1, fmaxf(fabsf(ex2_approx(w.x) * vs[nt].x), fabsf(ex2_approx(w.y) * vs[nt].y)));
      }
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {
        top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, o));
        top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, o));
      }
      co0 = raise_unit(top0, mn0, st.n0);
      co1 = raise_unit(top1, mn1, st.n1);
      f0 = to_unit(mn0, st.n0), f1 = to_unit(mn1, st.n1);
    }
  }
  float2 l0 = make_float2(0.f, 0.f), l1 = l0;
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) {
    y0[nt] = ffma2_rn(y0[nt], p0, r0);
    y1[nt] = ffma2_rn(y1[nt], p1, r1);
    y0[nt].x = ex2_approx(y0[nt].x), y0[nt].y = ex2_approx(y0[nt].y);
    y1[nt].x = ex2_approx(y1[nt].x), y1[nt].y = ex2_approx(y1[nt].y);
    l0 = fadd2_rn(l0, y0[nt]);
    l1 = fadd2_rn(l1, y1[nt]);
    if (KF == kFp8) {
      // (scale times factor is infinite where the weight is next to nothing and the unit
      // far below the scale; the row is then recomputed token by token)
      y0[nt] = fmul2_rn(y0[nt], fmul2_rn(vs[nt], make_float2(f0, f0)));
      y1[nt] = fmul2_rn(y1[nt], fmul2_rn(vs[nt], make_float2(f1, f1)));
      if (kMask) {   // a masked token's scale may be anything
        const int t0 = tb + nt * 8 + 2 * t;
        if (t0 >= len0) y0[nt].x = 0.f;
        if (t0 + 1 >= len0) y0[nt].y = 0.f;
        if (t0 >= len1) y1[nt].x = 0.f;
        if (t0 + 1 >= len1) y1[nt].y = 0.f;
      }
    }
  }
  st.l0 = fmaf(st.l0, c0, l0.x + l0.y);
  st.l1 = fmaf(st.l1, c1, l1.x + l1.y);
  if (__any_sync(0xffffffffu, co0 != 1.f || co1 != 1.f)) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      st.o[j][0] *= co0, st.o[j][1] *= co0;
      st.o[j][2] *= co1, st.o[j][3] *= co1;
    }
  }
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    uint32_t p[4], plo[4];
    const float2 w[4] = {y0[2 * ks], y1[2 * ks], y0[2 * ks + 1], y1[2 * ks + 1]};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (KF == kBf16) {
        // a weight as the sum of two bf16 (together 16 bits): rounded to one, the
        // weights would cost as much precision as the result's own rounding
        p[e] = pack_bf16(w[e].x, w[e].y);
        plo[e] = pack_bf16(w[e].x - bf16_lo(p[e]), w[e].y - bf16_hi(p[e]));
      } else {
        p[e] = pack_f16(w[e].x, w[e].y);
      }
    }
    uint32_t k0 = 0xffffffffu, k1 = 0xffffffffu;   // which of the lane's tokens exist
    if (kMask) {
      const int t0 = tb + ks * 16 + 2 * t;
      k0 = (t0 < glen ? 0xffffu : 0u) | (t0 + 1 < glen ? 0xffff0000u : 0u);
      k1 = (t0 + 8 < glen ? 0xffffu : 0u) | (t0 + 9 < glen ? 0xffff0000u : 0u);
    }
    const uint32_t row = stage + TB + (uint32_t)((ks * 16 + (m & 1) * 8 + rr) * 128);
#pragma unroll
    for (int j = 0; j < (KF == kBf16 ? 8 : 4); ++j) {
      const int ch = 2 * j + (m >> 1);
      uint32_t v0, v1, v2, v3;
      ldmatrix_x4_trans(row + (KF == kBf16 ? (uint32_t)((ch >> 3) * (TB / 2)) : 0u) +
                            (uint32_t)(((ch ^ rr) & 7) << 4),
                        v0, v1, v2, v3);
      if (kMask) v0 &= k0, v1 &= k1, v2 &= k0, v3 &= k1;
      if (KF == kBf16) {
        mma_bf16_16816(st.o[2 * j], p, v0, v1);
        mma_bf16_16816(st.o[2 * j + 1], p, v2, v3);
        mma_bf16_16816(st.o[2 * j], plo, v0, v1);
        mma_bf16_16816(st.o[2 * j + 1], plo, v2, v3);
      } else {
        // a register holds two dims (even, odd) of two tokens: the even dims'
        // bytes first, then the odd ones', each pair one operand register
        uint32_t e0, o0, e1, o1;
        e4m3x4_to_f16x2x2(prmt(v0, 0u, 0x3120), e0, o0);
        e4m3x4_to_f16x2x2(prmt(v1, 0u, 0x3120), e1, o1);
        mma_f16_16816(st.o[4 * j], p, e0, e1);
        mma_f16_16816(st.o[4 * j + 1], p, o0, o1);
        e4m3x4_to_f16x2x2(prmt(v2, 0u, 0x3120), e0, o0);
        e4m3x4_to_f16x2x2(prmt(v3, 0u, 0x3120), e1, o1);
        mma_f16_16816(st.o[4 * j + 2], p, e0, e1);
        mma_f16_16816(st.o[4 * j + 3], p, o0, o1);
      }
    }
  }
}

// A part of a shared unit's row: (running max, sum) and the unnormalised output.
__device__ __forceinline__ void put_part(const AttnArgs& a, int slot, int i, float m, float l,
                                         float4 o, int lane) {
  const size_t at = (size_t)slot * kTile + i;
  if (lane == 0) a.part_ml[at] = make_float2(m, l);
  reinterpret_cast<float4*>(a.part_o + at * kDim)[lane] = o;
}

// What the estimates below count in: the time in which an SM at its full rate takes a
// piece (bf16 0.38 us, HBM's share; e4m3 0.23, the warps' own).  A warp alone needs
// kAlone of it for a piece; kEnd and kEndAlone are a team's and a warp's cost of a unit
// beside its pieces, kStretch that of another stretch of the line, kCut of the first
// one and the join.
template <int KF, bool kBlocks>
struct Cost {
  static constexpr float kAlone = 5.f, kList = !kBlocks ? 0.f : KF == kBf16 ? 6.f : 9.f;
  static constexpr float kEnd = (KF == kBf16 ? 6.f : 12.f) + kList;
  static constexpr float kEndAlone = KF == kBf16 ? 3.f : 6.f;
  static constexpr float kStretch = (KF == kBf16 ? 7.f : 14.f) + kList;
  static constexpr float kCut = (KF == kBf16 ? 9.6f : 13.f) + kList;
};

// Words of a team's joined list.
__host__ __device__ constexpr int team_list_words(int tw) { return kMaxList / (kLeast / tw); }

// Whether the units of the call are dealt whole to teams of TW warps rather than cut
// along the line: the estimate of both, the first from what the host knows (Dealt).
// Every CTA comes to the same answer.
template <int KF, int TW>
__device__ __forceinline__ bool whole_units(const AttnArgs& a, const Requests& rq, int longest, int C) {
  using K = Cost<KF, false>;
  if (a.shift > 0) return false;
  const int per = (int)a.by_per.d;
  const float units = (float)(a.R * per), each = __fdividef(1.f, (float)C);
  const float total = (float)((rq.pre[a.R] - a.R * a.unit_cost) * per), mean = __fdividef(total, units);
  const float whole = a.dealt_ends + fmaxf(mean, (float)TW) * a.dealt_piece +
                      ((float)longest - mean) * (K::kAlone / TW);
  const float cut = fmaxf(total * each, K::kAlone) + K::kStretch * units * each + K::kCut;
  return whole <= cut;
}

// The rows of a unit that one warp has (g and g + 8 of every lane, i0 and i1 their
// places in out).
template <int KF, bool kBlocks>
__device__ __forceinline__ void write_rows(const AttnArgs& a, const Items& it, const uint32_t* list,
                                           const State& st, int r, int row_first, int nrows, int p0,
                                           bool has0, bool has1, size_t i0, size_t i1, int lane) {
  const int t = lane & 3;
  const bool see0 = st.m0 != -INFINITY, see1 = st.m1 != -INFINITY;
  const float f0 = see0 ? 1.f / st.l0 : 0.f, f1 = see1 ? 1.f / st.l1 : 0.f;
  bool odd0 = false, odd1 = false;   // something not finite: nothing visible is 0, not 0 * NaN
  uint16_t* o0 = a.out + i0 * kDim;
  uint16_t* o1 = a.out + i1 * kDim;
#pragma unroll
  for (int j = 0; j < 16; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      odd0 |= see0 && !(fabsf(st.o[j][e]) < INFINITY);
      odd1 |= see1 && !(fabsf(st.o[j][e + 2]) < INFINITY);
    }
  auto two = [](bool see, float x, float y, float f) { return see ? pack_bf16(x * f, y * f) : 0u; };
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float* x = st.o[2 * j];
    const float* y = st.o[2 * j + 1];
    if (KF == kBf16) {
      if (has0) {
        *reinterpret_cast<uint32_t*>(o0 + 16 * j + 2 * t) = two(see0, x[0], x[1], f0);
        *reinterpret_cast<uint32_t*>(o0 + 16 * j + 8 + 2 * t) = two(see0, y[0], y[1], f0);
      }
      if (has1) {
        *reinterpret_cast<uint32_t*>(o1 + 16 * j + 2 * t) = two(see1, x[2], x[3], f1);
        *reinterpret_cast<uint32_t*>(o1 + 16 * j + 8 + 2 * t) = two(see1, y[2], y[3], f1);
      }
    } else {
      if (has0)
        *reinterpret_cast<uint2*>(o0 + 16 * j + 4 * t) =
            make_uint2(two(see0, x[0], y[0], f0), two(see0, x[1], y[1], f0));
      if (has1)
        *reinterpret_cast<uint2*>(o1 + 16 * j + 4 * t) =
            make_uint2(two(see1, x[2], y[2], f1), two(see1, x[3], y[3], f1));
    }
  }
  if (a.lse && t == 0) {
    if (has0) a.lse[i0] = see0 ? (st.m0 + log2f(st.l0)) * kLn2 : st.m0;
    if (has1) a.lse[i1] = see1 ? (st.m1 + log2f(st.l1)) * kLn2 : st.m1;
  }
  const uint32_t odds = __ballot_sync(0xffffffffu, odd0), more = __ballot_sync(0xffffffffu, odd1);
  for (int i = 0; (odds | more) != 0u && i < nrows; ++i) {
    if (((i < 8 ? odds : more) >> (4 * (i & 7)) & 0xfu) == 0u) continue;
    const int pk = row_first + i, p = a.by_nq.div(pk);
    const size_t at = ((size_t)r * a.P + p) * a.q_heads + it.head * a.nq + (pk - p * a.nq);
    float m, l;
    float4 o;
    __syncwarp();
    careful_row<KF, kItem, kBlocks>(a, it, list, a.q + at * kDim, it.glen > 0 ? row_len(a, r, p) : 0,
                                    p - p0, lane, m, l, o);
    write_row(a, at, m, l, o, lane);
  }
}

// The CTA's units, TW warps a unit: its stretch of the line (kCut, TW = NW), or whole
// units dealt in turn to the teams of all CTAs (kWhole), or the one that `whole` says.
// record: the unit the CTA started and did not end.
// (One body for either needs less code but a branch and a register here and there.
// bf16, teams of 8: two bodies 1 x 400 8.74, 8 x 1000 13.66; one 8.92, 14.3.  e4m3: the
// second body of a kernel comes out 8 to 20% slower, one body 1 to 5%.)
enum class Deal { kCut, kWhole, kEither };
template <int KF, bool kBlocks, int TW, Deal kDeal>
__device__ __forceinline__ void run_units(const AttnArgs& a, const CUtensorMap& k_map,
                                          const CUtensorMap& v_map, uint8_t* smem, int W, int C,
                                          bool whole, SplitRecord& record) {
  using L = ALayout<KF>;
  constexpr int NW = L::NW;
  const uint32_t sbase = smem_u32(smem);
  unsigned int* cta_flags = reinterpret_cast<unsigned int*>(smem + L::kCtlOff);
  const Requests rq = requests_at(smem + L::kPreOff);
  constexpr int kTeams = NW / TW;
  uint32_t* list = reinterpret_cast<uint32_t*>(smem + L::kListOff) + team_list_words(TW) * (threadIdx.x / (32 * TW));
  // a team's block bits lie where its parts will
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem + L::kBitsOff) +
                   (L::kMlOff - L::kMergeOff) / 4 / kTeams * (threadIdx.x / (32 * TW));
  static_assert(!kBlocks || 2 * kMaxBlockWords * 4 * kTeams <= L::kMlOff - L::kMergeOff, "block bits");
  float* merge = reinterpret_cast<float*>(smem + L::kMergeOff);
  float2* ml = reinterpret_cast<float2*>(smem + L::kMlOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int c = blockIdx.x;
  const bool cut = kDeal == Deal::kCut || (kDeal == Deal::kEither && !whole);
  const int team = warp / TW, member = warp % TW;
  auto team_sync = [&]() {
    if (TW == NW)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(TW * 32) : "memory");
  };

  // ---- this warp's feed: items member, member + TW, ... of each stretch ---------
  // The page id is loaded here and looked at when the copy is issued, a piece
  // later, so nothing waits for it.
  struct Next {
    int unit;      // -1: nothing left
    int tb;
    uint32_t members;
    int page, kv_head;
  };
  Walk walk, fwalk;
  if (cut)
    walk.begin(a, rq.pre, c < C ? W * c / C : 0, c < C ? W * (c + 1) / C : 0);
  else
    walk.begin_units(a, team * (int)gridDim.x + c, (NW / TW) * (int)gridDim.x);
  fwalk = walk;
  Items fit = {};
  int funit = -1, fi = 0;
  bool dead = false;
  auto feed = [&]() -> Next {
    Next n = {-1, 0, 0u, 0, 0};
    while (!dead) {
      if (fi >= fit.i1) {
        if (kBlocks || !fwalk.more()) break;
        const Segment s = cut ? fwalk.next(a, rq.pre) : fwalk.next_unit(a, rq.pre);
        if (!s.live) continue;
        fit = make_items<kItem, kBlocks>(a, rq, s, 0);
        funit = s.unit;
        fi = fit.i0 + member;
        continue;
      }
      const int i = fi;
      fi += TW;
      if (!item_tokens<kItem, kBlocks>(fit, list, i, n.tb, n.members)) continue;
      n.page = __ldg(a.page_table + (size_t)fit.slot * a.max_pages + n.tb / kPage);
      n.kv_head = fit.kv_head;
      n.unit = funit;
      break;
    }
    return n;
  };
  // The warp's D stages are used in turn: its k-th piece lies in stage k % D.
  constexpr int D = L::D;
  auto stage_of = [&](int k) { return sbase + (warp * D + k % D) * L::kStage; };
  auto scales_of = [&](int k) { return L::kScaleOff + (warp * D + k % D) * L::kScaleBytes; };
  auto bar_of = [&](int k) { return sbase + L::kBarOff + (warp * D + k % D) * 8; };
  const Next none = {-1, 0, 0u, 0, 0};
  Next fl[D], nxt = none;     // pieces in flight, oldest first; the one after them
#pragma unroll
  for (int d = 0; d < D; ++d) fl[d] = none;
  int issued = 0;
  // ask for the copies of the next piece whose page exists
  auto fetch = [&]() -> Next {
    Next n = nxt;
    while (n.unit >= 0 && (n.page < 0 || n.page >= a.num_pages)) {
      if (lane == 0) atomicOr(cta_flags, kErrBadPage);
      n = feed();
    }
    if (n.unit < 0) return nxt = n;
    if (lane == 0) {
      const int row = (n.page * a.kv_heads + n.kv_head) * kPage + n.tb % kPage;
      const uint32_t stage = stage_of(issued), bar = bar_of(issued);
      mbar_arrive_expect_tx(bar, L::kStage + L::kScaleBytes);
      if (KF == kBf16) {
        tma_load_2d(stage, &k_map, 0, row, bar);
        tma_load_2d(stage + L::kTileBytes / 2, &k_map, 64, row, bar);
        tma_load_2d(stage + L::kTileBytes, &v_map, 0, row, bar);
        tma_load_2d(stage + L::kTileBytes + L::kTileBytes / 2, &v_map, 64, row, bar);
      } else {
        const uint32_t sc = sbase + scales_of(issued);
        tma_load_2d(stage, &k_map, 0, row, bar);
        bulk_load(sc, a.k_scale + row, kItem * 4, bar);
        tma_load_2d(stage + L::kTileBytes, &v_map, 0, row, bar);
        bulk_load(sc + kItem * 4, a.v_scale + row, kItem * 4, bar);
      }
    }
    ++issued;
    nxt = feed();
    return n;
  };

  int used = 0;           // pieces this warp has waited for
  bool primed = false;
  while (walk.more()) {
    const Segment s = cut ? walk.next(a, rq.pre) : walk.next_unit(a, rq.pre);
    if (!s.live) continue;
    const int row_first = s.group * kTile;
    const int nrows = min(kTile, a.P * a.nq - row_first);
    const int p0 = a.by_nq.div(row_first);
    int n_items = 0;
    if (kBlocks) {
      n_items = join_lists(a, rq, s, p0, (row_first + nrows - 1) / a.nq, list, bits,
                           threadIdx.x % (32 * TW), 32 * TW, team_sync) *
                (kBlock / kItem);
      fit = make_items<kItem, kBlocks>(a, rq, s, n_items);
      funit = s.unit;
      fi = fit.i0 + member;
      primed = false;
    }
    // the first page id, the queries and the first copies overlap
    const bool prime = !primed;
    if (prime) {
      primed = true;
      nxt = feed();
    }
    const Items it = kBlocks ? fit : make_items<kItem, kBlocks>(a, rq, s, 0);
    // ---- the unit's rows ----------------------------------------------------
    auto q_index = [&](int pk, int p) {   // packed row pk of the unit head, draft row p = pk / nq
      return ((size_t)s.r * a.P + p) * a.q_heads + s.head * a.nq + (pk - p * a.nq);
    };
    const int pk0 = row_first + g, pd0 = a.by_nq.div(pk0), pk1 = pk0 + 8, pd1 = a.by_nq.div(pk1);
    const bool has0 = g < nrows, has1 = g + 8 < nrows;
    // with one draft row the request's longest row is the row
    const int L0 = !has0 || it.glen == 0 ? 0 : a.P == 1 ? it.glen : row_len(a, s.r, pd0);
    const int L1 = !has1 || it.glen == 0 ? 0 : a.P == 1 ? it.glen : row_len(a, s.r, pd1);
    QRows<KF> q;
    q.load(has0 ? a.q + q_index(pk0, pd0) * kDim : nullptr,
           has1 ? a.q + q_index(pk1, pd1) * kDim : nullptr);
    if (prime) {
#pragma unroll
      for (int d = 0; d < D; ++d) fl[d] = fetch();
    }
    q.finish(a.scale_log2);
    State st;
    st.reset();
    // ---- its pieces -----------------------------------------------------------
    while (fl[0].unit == s.unit) {
      const Next cur = fl[0];
      const bool stall = a.stall_test && warp == 0 && used == 0;
      if (!mbar_wait_bounded(stall ? sbase + L::kBarOff + NW * D * 8 : bar_of(used),
                             stall ? 0u : (uint32_t)((used / D) & 1), a.wait_ns)) {
        if (lane == 0) atomicOr(cta_flags, kErrTimeout);
        dead = true;
      }
      dead = __any_sync(0xffffffffu, dead);
      if (dead) break;
      const int e0 = has0 && (!kBlocks || (cur.members >> (pd0 - p0)) & 1u) ? L0 : 0;
      const int e1 = has1 && (!kBlocks || (cur.members >> (pd1 - p0)) & 1u) ? L1 : 0;
      const bool whole = __all_sync(0xffffffffu, (!has0 || cur.tb + kItem <= e0) &&
                                                     (!has1 || cur.tb + kItem <= e1));
      const uint32_t stage = stage_of(used);
      const float* scales = reinterpret_cast<const float*>(smem + scales_of(used));
      if (whole)
        piece<KF, false>(q, st, stage, scales, lane, cur.tb, e0, e1, it.glen);
      else
        piece<KF, true>(q, st, stage, scales, lane, cur.tb, e0, e1, it.glen);
      ++used;
      // every lane's reads of the stage come before the copies that refill it
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
#pragma unroll
      for (int d = 0; d + 1 < D; ++d) fl[d] = fl[d + 1];
      fl[D - 1] = fetch();
    }
    if (dead) {
      // let the copies in flight land, take no more
      for (; used < issued; ++used)
        if (lane == 0) (void)mbar_wait_bounded(bar_of(used), (uint32_t)((used / D) & 1), 200000000ull);
#pragma unroll
      for (int d = 0; d < D; ++d) fl[d] = none;
      nxt = none;
    }
    // ---- join the warps: the upper half into the lower, then those by rows -----
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
      st.l0 += __shfl_xor_sync(0xffffffffu, st.l0, o);
      st.l1 += __shfl_xor_sync(0xffffffffu, st.l1, o);
    }
    st.m0 = not_empty(st.m0, st.l0);
    st.m1 = not_empty(st.m1, st.l1);
    if (KF == kFp8) {
      // the output in the maximum's unit, as the sum
      const float u0 = ex2_approx(st.n0 - st.m0), u1 = ex2_approx(st.n1 - st.m1);
#pragma unroll
      for (int j = 0; j < 16; ++j) st.o[j][0] *= u0, st.o[j][1] *= u0, st.o[j][2] *= u1, st.o[j][3] *= u1;
    }
    if constexpr (TW == 1) {
      // one warp has the whole unit: its rows are written from the registers
      write_rows<KF, kBlocks>(a, it, list, st, s.r, row_first, nrows, p0, has0, has1,
                              q_index(pk0, pd0), q_index(pk1, pd1), lane);
      continue;
    }
    constexpr int nh = TW > 1 ? TW / 2 : 1;
    const int first = team * nh, place = first + (member < nh ? member : member - nh);
    float* w0 = merge + (size_t)(place * kTile + g) * kMergeStride;
    float* w1 = w0 + 8 * kMergeStride;
    float2* ml0 = ml + place * kTile + g;
    auto put = [&]() {
      if (t == 0) {
        ml0[0] = make_float2(st.m0, st.l0);
        ml0[8] = make_float2(st.m1, st.l1);
      }
      if (KF == kBf16) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          *reinterpret_cast<float2*>(w0 + 8 * j + 2 * t) = make_float2(st.o[j][0], st.o[j][1]);
          *reinterpret_cast<float2*>(w1 + 8 * j + 2 * t) = make_float2(st.o[j][2], st.o[j][3]);
        }
      } else {
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const float* e = st.o[2 * ch];
          const float* d = st.o[2 * ch + 1];
          *reinterpret_cast<float4*>(w0 + 16 * ch + 4 * t) = make_float4(e[0], d[0], e[1], d[1]);
          *reinterpret_cast<float4*>(w1 + 16 * ch + 4 * t) = make_float4(e[2], d[2], e[3], d[3]);
        }
      }
    };
    if (member >= nh) put();
    team_sync();
    if (member < nh) {
      const float2 x0 = ml0[0], x1 = ml0[8];
      const float n0 = fmaxf(st.m0, x0.x), n1 = fmaxf(st.m1, x1.x);
      const float r0 = n0 == -INFINITY ? 0.f : n0, r1 = n1 == -INFINITY ? 0.f : n1;
      // a half with nothing visible in the row holds zeros (or 0 * NaN: dropped)
      const bool has_a0 = st.m0 != -INFINITY, has_a1 = st.m1 != -INFINITY;
      const bool has_b0 = x0.x != -INFINITY, has_b1 = x1.x != -INFINITY;
      const float a0 = ex2_approx(st.m0 - r0), a1 = ex2_approx(st.m1 - r1);
      const float b0 = ex2_approx(x0.x - r0), b1 = ex2_approx(x1.x - r1);
      st.l0 = (has_a0 ? st.l0 * a0 : 0.f) + (has_b0 ? x0.y * b0 : 0.f);
      st.l1 = (has_a1 ? st.l1 * a1 : 0.f) + (has_b1 ? x1.y * b1 : 0.f);
      st.m0 = n0, st.m1 = n1;
      auto fold = [](bool ha, float a, float fa, bool hb, float b, float fb) {
        return (ha ? a * fa : 0.f) + (hb ? b * fb : 0.f);
      };
      if (KF == kBf16) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float2 y0 = *reinterpret_cast<const float2*>(w0 + 8 * j + 2 * t);
          const float2 y1 = *reinterpret_cast<const float2*>(w1 + 8 * j + 2 * t);
          st.o[j][0] = fold(has_a0, st.o[j][0], a0, has_b0, y0.x, b0);
          st.o[j][1] = fold(has_a0, st.o[j][1], a0, has_b0, y0.y, b0);
          st.o[j][2] = fold(has_a1, st.o[j][2], a1, has_b1, y1.x, b1);
          st.o[j][3] = fold(has_a1, st.o[j][3], a1, has_b1, y1.y, b1);
        }
      } else {
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const float4 y0 = *reinterpret_cast<const float4*>(w0 + 16 * ch + 4 * t);
          const float4 y1 = *reinterpret_cast<const float4*>(w1 + 16 * ch + 4 * t);
          float* e = st.o[2 * ch];
          float* d = st.o[2 * ch + 1];
          e[0] = fold(has_a0, e[0], a0, has_b0, y0.x, b0);
          d[0] = fold(has_a0, d[0], a0, has_b0, y0.y, b0);
          e[1] = fold(has_a0, e[1], a0, has_b0, y0.z, b0);
          d[1] = fold(has_a0, d[1], a0, has_b0, y0.w, b0);
          e[2] = fold(has_a1, e[2], a1, has_b1, y1.x, b1);
          d[2] = fold(has_a1, d[2], a1, has_b1, y1.y, b1);
          e[3] = fold(has_a1, e[3], a1, has_b1, y1.z, b1);
          d[3] = fold(has_a1, d[3], a1, has_b1, y1.w, b1);
        }
      }
      __syncwarp();
      put();
    }
    team_sync();
    const bool complete = !cut || (s.o0 == 0 && s.o1 == s.cap);
    const int slot_out = 2 * c + (s.o0 == 0 ? 1 : 0);
    if (s.o0 == 0 && !complete) {
      record.unit = s.unit;
      record.splits = owner(s.start + s.cap - 1, W, C) - c + 1;
    }
    for (int i = member; i < nrows; i += TW) {
      const int pk = row_first + i, p = a.by_nq.div(pk);
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < NW / 2; ++w)
        if (w < nh) m = fmaxf(m, ml[(first + w) * kTile + i].x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (m != -INFINITY) {
#pragma unroll
        for (int w = 0; w < NW / 2; ++w) {
          if (w >= nh) break;
          const float2 x = ml[(first + w) * kTile + i];
          const float f = ex2_approx(x.x - m);
          if (x.x == -INFINITY) continue;   // a warp with nothing visible in the row
          const float4 v = *reinterpret_cast<const float4*>(merge + (size_t)((first + w) * kTile + i) * kMergeStride + 4 * lane);
          l = fmaf(x.y, f, l);
          o = make_float4(fmaf(v.x, f, o.x), fmaf(v.y, f, o.y), fmaf(v.z, f, o.z), fmaf(v.w, f, o.w));
        }
      }
      if (__any_sync(0xffffffffu, !finite4(o)))
        careful_row<KF, kItem, kBlocks>(a, it, list, a.q + q_index(pk, p) * kDim,
                                        it.glen > 0 ? row_len(a, s.r, p) : 0, p - p0, lane, m, l, o);
      if (complete)
        write_row(a, q_index(pk, p), m, l, o, lane);
      else
        put_part(a, slot_out, i, m, l, o, lane);
    }
    team_sync();
  }
  if (!cut) __syncthreads();
}

template <int KF, bool kBlocks, int TW, Deal kDeal>
__global__ void __launch_bounds__(ALayout<KF>::kThreads, 1)
    attn_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                const __grid_constant__ CUtensorMap v_map) {
  using L = ALayout<KF>;
  constexpr int NW = L::NW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  unsigned int* cta_flags = reinterpret_cast<unsigned int*>(smem + L::kCtlOff);
  const Requests rq = requests_at(smem + L::kPreOff);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) {
    for (int d = 0; d < L::D; ++d) mbar_init(sbase + L::kBarOff + (warp * L::D + d) * 8, 1);
    if (warp == 0) mbar_init(sbase + L::kBarOff + NW * L::D * 8, 1);  // the stall test's barrier
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  build_requests<kItem, kBlocks, false>(a, rq, reinterpret_cast<int*>(cta_flags + 2), cta_flags);

  const int W = rq.pre[a.R] * (int)a.by_per.d;
  // no CTA takes less than about one piece a warp
  static_assert(NW == kLeast, "positions a CTA takes at least");
  const int C = min((W + kLeast - 1) / kLeast, (int)gridDim.x);
  SplitRecord record = {-1, 0};
  if constexpr (kDeal != Deal::kEither) {
    run_units<KF, kBlocks, TW, kDeal>(a, k_map, v_map, smem, W, C, false, record);
  } else {
    const bool whole = whole_units<KF, TW>(a, rq, (int)cta_flags[1], C);
    if constexpr (KF == kFp8 && TW == NW)
      run_units<KF, kBlocks, NW, Deal::kEither>(a, k_map, v_map, smem, W, C, whole, record);
    else if (whole)
      run_units<KF, kBlocks, TW, Deal::kWhole>(a, k_map, v_map, smem, W, C, true, record);
    else
      run_units<KF, kBlocks, NW, Deal::kCut>(a, k_map, v_map, smem, W, C, false, record);
  }
  if (threadIdx.x == 0) {
    a.records[blockIdx.x] = record;
    a.err_bytes[blockIdx.x] = (uint8_t)*cta_flags;
    if (blockIdx.x == 0) *a.err_count = gridDim.x;
  }
}

// ---------------------------------------------------------------------------
// The join of units that several CTAs shared.  The parts of the unit that CTA c
// started and did not end are CTA c's second slot and the first slots of the CTAs
// behind it; a row's maxima and sums are read at once, one a lane, then its
// outputs are added in a fixed order, so the result does not depend on timing.
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 4, kJoinThreads = 32 * kJoinWarps;

__device__ __forceinline__ size_t part_at(const AttnArgs& a, int c, int s, int i) {
  return (size_t)(s == 0 ? 2 * c + 1 : 2 * (c + s)) * a.group_rows + i;
}

// Output row and packed row of row i of the unit; false past the unit's rows.
__device__ __forceinline__ bool joined_row(const AttnArgs& a, int unit, int i, size_t& row) {
  const int r = a.by_per.div(unit), k = unit - r * (int)a.by_per.d;
  const int head = a.by_groups.div(k), pk = (k - head * a.groups) * a.group_rows + i;
  if (pk >= a.P * a.nq) return false;
  const int p = a.by_nq.div(pk);
  row = ((size_t)r * a.P + p) * a.q_heads + head * a.nq + (pk - p * a.nq);
  return true;
}

__device__ __forceinline__ void add_scaled(float4& o, const float4& v, float f) {
  o = make_float4(fmaf(v.x, f, o.x), fmaf(v.y, f, o.y), fmaf(v.z, f, o.z), fmaf(v.w, f, o.w));
}

// One warp a row, block (c, rows / 4).
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quads = (min(a.group_rows, a.P * a.nq) + kJoinWarps - 1) / kJoinWarps;
  const int c = blockIdx.x / quads, i = (blockIdx.x - c * quads) * kJoinWarps + warp;
  const SplitRecord rec = a.records[c];
  size_t row;
  if (rec.unit < 0 || !joined_row(a, rec.unit, i, row)) return;
  constexpr int kPer = (kMaxCtas + 31) / 32;
  float2 x[kPer];
  float m = -INFINITY;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int s = lane + 32 * e;
    x[e] = make_float2(-INFINITY, 0.f);
    if (s < rec.splits) x[e] = a.part_ml[part_at(a, c, s, i)];
    m = fmaxf(m, x[e].x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  float l = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    // a part with nothing visible in the row is not read: factor -1 says so
    const float f = x[e].x == -INFINITY ? -1.f : ex2_approx(x[e].x - m);
    if (x[e].x != -INFINITY) l = fmaf(x[e].y, f, l);
    x[e].x = f;
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    for (int s0 = 32 * e; s0 < min(rec.splits, 32 * e + 32); s0 += 8) {
      float4 v[8];
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {   // eight parts' loads in flight
        f[k] = __shfl_sync(0xffffffffu, x[e].x, (s0 + k) & 31);
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (f[k] != -1.f)
          v[k] = reinterpret_cast<const float4*>(a.part_o + part_at(a, c, s0 + k, i) * kDim)[lane];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (f[k] != -1.f) add_scaled(o, v[k], f[k]);
    }
  }
  write_row(a, row, m, l, o, lane);
}

// A call of few units may have 100 parts a row: four blocks a row, 32 dims each,
// and a block for every unit, which looks its CTA up (1 x 131K: 30.2 -> 23.7 us a
// call, four draft rows 36.0 -> 27.4; but 1 x 1K 8.9 -> 9.3, so only where a unit
// may have over 32 parts).
constexpr int kFewSplit = 4;
__global__ void __launch_bounds__(kJoinThreads) attn_join_few_kernel(const AttnArgs a, int ctas) {
  __shared__ float factor[kMaxCtas];
  __shared__ float red[2][kJoinWarps];
  __shared__ float4 so[kJoinWarps][32];
  __shared__ int found;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = min(a.group_rows, a.P * a.nq);
  const int unit = blockIdx.x / (rows * kFewSplit), i = blockIdx.x / kFewSplit - unit * rows;
  if (threadIdx.x == 0) found = -1;
  __syncthreads();
  for (int k = threadIdx.x; k < ctas; k += kJoinThreads)
    if (a.records[k].unit == unit) found = k;
  __syncthreads();
  const int c = found;
  size_t row;
  if (c < 0 || !joined_row(a, unit, i, row)) return;
  const int splits = a.records[c].splits;
  static_assert(kMaxCtas <= 2 * kJoinThreads, "two parts a thread");
  float2 x[2];
  float m = -INFINITY;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int s = threadIdx.x + e * kJoinThreads;
    x[e] = make_float2(-INFINITY, 0.f);
    if (s < splits) x[e] = a.part_ml[part_at(a, c, s, i)];
    m = fmaxf(m, x[e].x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, red[0][w]);
  float l = 0.f;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int s = threadIdx.x + e * kJoinThreads;
    const float f = x[e].x == -INFINITY ? -1.f : ex2_approx(x[e].x - m);
    if (s < splits) factor[s] = f;
    if (x[e].x != -INFINITY) l = fmaf(x[e].y, f, l);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  if (lane == 0) red[1][warp] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) l += red[1][w];
  // a warp takes four parts at a time, eight lanes each, eight such loads in flight
  constexpr int kLanes = 32 / kFewSplit, kStep = kJoinWarps * kFewSplit;
  const int dim4 = (int)(blockIdx.x % kFewSplit) * kLanes + lane % kLanes;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = warp * kFewSplit + lane / kLanes; s0 < splits; s0 += 8 * kStep) {
    float4 v[8];
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int s = s0 + e * kStep;
      f[e] = s < splits ? factor[s] : -1.f;
      v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (f[e] != -1.f) v[e] = reinterpret_cast<const float4*>(a.part_o + part_at(a, c, s, i) * kDim)[dim4];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (f[e] != -1.f) add_scaled(o, v[e], f[e]);
  }
  so[warp][lane] = o;
  __syncthreads();
  if (threadIdx.x >= kLanes) return;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w)
#pragma unroll
    for (int e = 0; e < kFewSplit; ++e) add_scaled(o, so[w][e * kLanes + lane], 1.f);
  write_row(a, row, m, l, o, dim4);
}

template <int KF, bool kBlocks, int TW, Deal kDeal>
cudaError_t launch_kf(const AttnArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map,
                      int grid, int dev, cudaStream_t stream) {
  using L = ALayout<KF>;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = smem_limit_once(attn_kernel<KF, kBlocks, TW, kDeal>, L::kSmem, dev, attr_done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_kernel<KF, kBlocks, TW, kDeal>, grid, L::kThreads, L::kSmem, stream, a, k_map, v_map);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// What it costs to deal `units` units whole to teams of tw warps on `grid` SMs: `ends`
// and, for each piece of their mean length, `piece`.  Full turns keep every warp busy,
// the last one those that it has.
struct Dealt {
  float ends, piece;
};
template <int KF, bool kBlocks>
Dealt dealt(int units, int grid, int tw) {
  using K = Cost<KF, kBlocks>;
  const int teams = grid * (kLeast / tw), full = units / teams, rest = units - full * teams;
  const float busy = (float)(rest * tw) / (float)grid;
  const float last = rest == 0 ? 0.f : busy > K::kAlone ? busy : K::kAlone;
  return {(float)(full + (rest > 0)) * (tw == 1 ? K::kEndAlone : K::kEnd),
          ((float)kLeast * (float)full + last) / (float)tw};
}

// The team size for units dealt whole: the one with which `units` of so many pieces
// would take least, and what they would.
template <int KF, bool kBlocks>
int team_for(AttnArgs& a, int grid, float pieces, float& least) {
  const int units = a.R * (int)a.by_per.d;
  int team = 0;
  for (int tw = kLeast; tw >= (kBlocks ? 2 : 1); tw /= 2) {
    // a team holds its joined list, and the parts of two warps the bits it is made with
    if (kBlocks && min(a.P, kMaxDrafts) * a.topk > team_list_words(tw)) break;
    const Dealt d = dealt<KF, kBlocks>(units, grid, tw);
    const float cost = d.ends + pieces * d.piece;
    if (team > 0 && cost >= least) continue;
    team = tw;
    least = cost;
    a.dealt_ends = d.ends;
    a.dealt_piece = d.piece;
  }
  return team;
}

// The whole cache: units of 16 pieces are assumed for the team; how long they are is
// known on the device only, which decides whether they are dealt whole at all.
template <int KF>
cudaError_t launch_paged(AttnArgs a, const CUtensorMap& k_map, const CUtensorMap& v_map, int grid,
                         int dev, cudaStream_t stream) {
  float least;
  switch (team_for<KF, false>(a, grid, 16.f, least)) {
    case 1: return launch_kf<KF, false, 1, Deal::kEither>(a, k_map, v_map, grid, dev, stream);
    case 2: return launch_kf<KF, false, 2, Deal::kEither>(a, k_map, v_map, grid, dev, stream);
    case 4: return launch_kf<KF, false, 4, Deal::kEither>(a, k_map, v_map, grid, dev, stream);
    default: return launch_kf<KF, false, 8, Deal::kEither>(a, k_map, v_map, grid, dev, stream);
  }
}

// Lists: their length bounds the units', so the host decides, for full lists (each
// further draft row's taken to add an eighth of its own), and a call that deals needs no
// join.  Only where the estimates lie apart: they are equally good for one of 368 units
// of 32 blocks (122.8 us cut, 131 dealt), and a batch of contexts shorter than their
// lists is better cut (96 units of 1 to 16 blocks 15.6, 18.7 dealt; all of 16 25.0, 22.2).
template <int KF>
cudaError_t launch_lists(AttnArgs a, const CUtensorMap& k_map, const CUtensorMap& v_map, int grid,
                         int dev, cudaStream_t stream, bool& whole) {
  using K = Cost<KF, true>;
  const float full = (float)(a.topk * (kBlock / kItem)) * (1.f + (float)(a.P - 1) / 8.f);
  const float pieces = fminf(full, (float)a.most);
  const float share = (float)(a.R * (int)a.by_per.d) / (float)grid;
  float least;
  const int team = team_for<KF, true>(a, grid, pieces, least);
  whole = least <= 0.83f * (fmaxf(share * pieces, K::kAlone) + K::kStretch * share + K::kCut);
  if (!whole) return launch_kf<KF, true, 8, Deal::kCut>(a, k_map, v_map, grid, dev, stream);
  switch (team) {
    case 2: return launch_kf<KF, true, 2, Deal::kWhole>(a, k_map, v_map, grid, dev, stream);
    case 4: return launch_kf<KF, true, 4, Deal::kWhole>(a, k_map, v_map, grid, dev, stream);
    default: return launch_kf<KF, true, 8, Deal::kWhole>(a, k_map, v_map, grid, dev, stream);
  }
}

}  // namespace

int attn_ctas() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  int n = cached_sm_count(dev);
  const int lim = grid_limit();
  if (lim > 0 && lim < n) n = lim;
  return n > attn::kMaxCtas ? attn::kMaxCtas : n;
}

cudaError_t launch_attn(int key_format, const AttnArgs& a, const CUtensorMap& k_map,
                        const CUtensorMap& v_map, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int sms = attn_ctas();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // no more CTAs than the longest contexts the page table can hold give work to
  const bool wide = a.group_rows > kTile, blocks = a.block_ids != nullptr;
  const long long units = (long long)a.R * (int)a.by_per.d;
  const long long pieces = wide ? (a.most + 1) / 2 : a.most;
  const long long line = units * (((pieces + (1ll << a.shift) - 1) >> a.shift) + a.unit_cost);
  const long long least = wide ? kLeastWide : kLeast;
  const int grid = (int)((line + least - 1) / least < sms ? (line + least - 1) / least : sms);
  bool whole = false;
  if (wide)
    e = launch_attn_wide(key_format, a, k_map, v_map, grid, dev, stream);
  else if (blocks)
    e = key_format == kBf16 ? launch_lists<kBf16>(a, k_map, v_map, grid, dev, stream, whole)
                            : launch_lists<kFp8>(a, k_map, v_map, grid, dev, stream, whole);
  else
    e = key_format == kBf16 ? launch_paged<kBf16>(a, k_map, v_map, grid, dev, stream)
                            : launch_paged<kFp8>(a, k_map, v_map, grid, dev, stream);
  if (e != cudaSuccess || whole) return e;
  const int rows = a.P * a.nq < a.group_rows ? a.P * a.nq : a.group_rows;
  e = units * 16 <= grid && a.most > 32 * 8
          ? launch_pdl(attn_join_few_kernel, (int)units * rows * kFewSplit, kJoinThreads, 0, stream, a, grid)
          : launch_pdl(attn_join_kernel, grid * ((rows + kJoinWarps - 1) / kJoinWarps), kJoinThreads, 0,
                       stream, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace idx
