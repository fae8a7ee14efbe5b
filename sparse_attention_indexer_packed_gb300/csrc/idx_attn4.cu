// Attention over an NVFP4 cache with up to 16 packed rows a unit: the mathematics, the
// split and the dealing are idx_attn.cu's.
//
// What bounds it: 144 bytes a token and head, half of what an e4m3 cache has, against the same
// products and a decode of both operands, so it is the warps' own work that bounds it, not
// HBM.  A 32-token piece costs a warp 128 conversions, 128 f16x2 products and 64 matrix
// products; on each of an SM's four schedulers the conversions (2 cycles each) come to 256
// cycles, the matrix products (8 each) to 512, all instructions together to ~600, where
// HBM's share of the piece is 215.  Measured, 16 x 131K tokens x 16 rows: 75.3 us, 0.54 of the
// bytes' rate; issue slots 50% taken, tensor cores 37%, HBM 41%.
//
// How (sm_103a):
//  * 12 warps of 168 registers, three a scheduler, nothing spilled.  Eight of 255 leave two
//    thirds of the issue slots empty (120 us), 16 of 128 spill in the loop, and a spill here
//    goes past the L1 that shared memory takes (88 us).  So the 16 queries lie in shared memory
//    in the order of the product's operand, the output alone in registers, and what a warp does
//    not need in its loop (the walk, the stretch) waits in shared memory.  Four key tiles to a
//    read of the queries instead of two 79.8, values loaded before the scores 79.1;
//  * a warp owns two stages of one piece (keys, values and their scales) and refills each as
//    soon as it has been used (three stages: 81.2).  Its copies end with the unit: a stage's 9 KB
//    are then where the warp leaves its state, and a row's 12 states are joined by one warp.  (A
//    warp that feeds the 15 others, across units: its copies, one lane after the other, took 3800
//    cycles a round: 100 us);
//  * a lane's 16 bytes of a key are 32 dims of it, two groups; its 8 bytes of a value are one
//    group, whose dims are the 16 product tiles, so one scale serves all of them.  Two
//    tokens' codes of one dim are put side by side by masks, without a permutation.  A code
//    times its scale is exact in f16, the queries are f16 as for e4m3 keys;
//  * the weights are f16 in units of 2^m, which is only raised, to 2^kHead below the row's
//    maximum, when a score passes it by 2^(kHead + kSlack), the most that f16 holds: 11 bits of
//    each, or 2^-32 of the row's largest.  So the output is seldom rescaled (raised with
//    every new maximum, nearly every piece of 16 rows did).
// Small calls: 1 x 1K tokens 9.5 us (11.8 with eight warps), 48 ragged requests x 4 heads 19.9,
// 16 x 131K with four lists of 64 blocks each 41.6 (50.5).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "idx_attn.cuh"
#include "idx_attn_rows.cuh"
#include "idx_ptx.cuh"

namespace idx {

namespace {

using namespace attn;

constexpr int kItem = 32;      // tokens of a piece
constexpr int NW = 12;         // warps
constexpr int D = 2;           // stages of a warp
constexpr float kHead = 7.f, kSlack = 8.f;   // log2 units
constexpr int kColdWords = 28;

// What a piece needs to know of a packed row, in shared memory: the scores' factor, the
// visible length (0: no such row) and the bit of its draft row.
struct Row {
  float post;
  int len;
  uint32_t bit;
};

struct L {
  static constexpr int kThreads = 32 * NW;
  static constexpr int kTileBytes = kItem * 64;      // keys or values of a piece
  static constexpr int kScaleBytes = kItem * 8;
  static constexpr int kArea = D * 2 * (kTileBytes + kScaleBytes);   // of a warp: tiles, then scales
  // floats of a row of a warp's state: a lane has 32 dims in a row, each run of 32 is four
  // floats apart from the next, which keeps row writes off one bank
  static constexpr int kStateStride = kDim + 16;
  static_assert(kTile * kStateStride * 4 <= kArea, "a state in a warp's area");
  static_assert(kArea % 512 == 0, "the 64-byte swizzle's period");
  static constexpr int kTeams = NW / 3;
  static constexpr int kQOff = NW * kArea;           // a team's queries, in operand order
  static constexpr int kPostOff = kQOff + kTeams * kTile * 256;
  static constexpr int kMlOff = kPostOff + kTeams * kTile * sizeof(Row);   // (max, sum) of a warp's rows
  static constexpr int kBarOff = kMlOff + NW * kTile * 8;
  static constexpr int kNumBars = NW * D + 1;                    // a stage's, the stall test's
  static constexpr int kColdOff = kBarOff + kNumBars * 8;        // what a warp does not need in its loop
  static constexpr int kCtlOff = kColdOff + NW * kColdWords * 4;  // flags, longest unit, one int a warp
  static constexpr int kPreOff = (kCtlOff + 8 + NW * 4 + 15) & ~15;
  static constexpr int kListOff = kPreOff + kRequestsBytes;
  static constexpr int kBytes = kListOff + kMaxList * 4;
  static constexpr int kSmem = kBytes + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  // the bits that lists are joined with lie in the team's areas, where nothing is in flight then
  static_assert(2 * kMaxBlockWords * 4 <= 2 * kArea, "block bits");
};

// The token of an NVFP4 piece's 8-token tile that is column 2t + e of the scores' tile and
// row 2t + e of the values' operand.  The order keeps the reads off one bank: the keys'
// (tokens 2t, 2t + 1 side by side) and the values' (four tokens 2t + e at once).
__device__ __forceinline__ int token4(int t, int e) { return 4 * (t >> 1) + ((t & 1) ^ (3 * e)); }

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t d;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(d) : "r"(w));
  return d;
}

// Softmax state of the two rows a lane holds (g and g + 8), and its part of the
// unnormalised output: dims 32t + j of o[j][0] (row g) and o[j][2] (row g + 8), 32t + 16 + j
// of o[j][1] and o[j][3].  m: the weights' unit, in log2 units.
struct State {
  float m0, m1, l0, l1;
  float o[16][4];
  __device__ __forceinline__ void reset() {
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  }
};

// Where a lane reads in a piece: its key (of a tile; the scores' column), that key's two
// scales, its first value's codes and scale, packed so that they cost one register.  The
// second value's (token4(t, 1) = token4(t, 0) ^ 3) follow from them.
struct Places {
  uint32_t w;
  __device__ __forceinline__ explicit Places(int lane) {
    const int t = lane & 3, g = lane >> 2;
    const int tok = token4(g >> 1, g & 1), ta = token4(t, 0);
    const uint32_t key = tok * 64 + ((t ^ (tok >> 1)) << 4), key_scale = tok * 8 + 2 * t;
    const uint32_t value = ta * 64 + (((g >> 1) ^ (ta >> 1)) << 4) + (g & 1) * 8, value_scale = ta * 8 + g;
    w = key | (key_scale << 9) | (value << 15) | (value_scale << 24);
  }
  __device__ __forceinline__ uint32_t key() const { return w & 511u; }
  __device__ __forceinline__ uint32_t key_scale() const { return (w >> 9) & 63u; }
  __device__ __forceinline__ uint32_t value() const { return (w >> 15) & 511u; }
  __device__ __forceinline__ uint32_t value_scale() const { return w >> 24; }
  static constexpr uint32_t kValue1 = (3u << 6) | (1u << 4), kScale1 = 3u << 3;
};

// One 32-token piece.  q: the queries in operand order (the lane's place in a step), step c
// takes the dims 32t + 4c + {0, 1} and + {2, 3}.  kMask: some token of the piece lies outside some row
// (past its length, or the row's draft does not list the block) or at or past glen, where
// the cache holds anything: such values are dropped by selection, not by a product with zero.
template <bool kMask>
__device__ __forceinline__ void piece(uint32_t q, const Row* rows, State& st, uint32_t stage,
                                      uint32_t scales, const Places& at, int tb, uint32_t members, int glen) {
  const int lane = threadIdx.x & 31;
  const int t = lane & 3, g = lane >> 2;
  float s[4][4];
  {
    const uint32_t krow = stage + at.key(), ks = scales + at.key_scale();
#pragma unroll
    for (int n2 = 0; n2 < 4; n2 += 2) {
      uint32_t w[2][4], sc[2], f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int nt = n2 + h;
        s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
        const uint4 u = lds128(krow + nt * 512);
        w[h][0] = u.x, w[h][1] = u.y, w[h][2] = u.z, w[h][3] = u.w;
        sc[h] = e4m3x2_to_f16x2(lds16(ks + nt * 64));
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint4 u = lds128(q + c * 512);
        const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (c % 4 == 0) f[h] = prmt(sc[h], 0u, c == 0 ? 0x1010 : 0x3232);
          uint32_t d0, d1;
          if (c & 1) e2m1x4_to_f16x2x2<1>(w[h][c / 2], d0, d1);
          else e2m1x4_to_f16x2x2<0>(w[h][c / 2], d0, d1);
          mma_f16_16816(s[n2 + h], a, hmul2(d0, f[h]), hmul2(d1, f[h]));
        }
      }
    }
  }
  const int ta = token4(t, 0), tc = token4(t, 1);   // the lane's tokens of each tile
  const float post0 = rows[g].post, post1 = rows[g + 8].post;
  const int len0 = kMask && (members & rows[g].bit) ? rows[g].len : 0;
  const int len1 = kMask && (members & rows[g + 8].bit) ? rows[g + 8].len : 0;
  float2 y0[4], y1[4];
  float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) {
    y0[nt] = make_float2(s[nt][0], s[nt][1]);
    y1[nt] = make_float2(s[nt][2], s[nt][3]);
    if (kMask) {
      const int t0 = tb + nt * 8 + ta, t1 = tb + nt * 8 + tc;
      if (t0 >= len0) y0[nt].x = -INFINITY;
      if (t1 >= len0) y0[nt].y = -INFINITY;
      if (t0 >= len1) y1[nt].x = -INFINITY;
      if (t1 >= len1) y1[nt].y = -INFINITY;
    }
    mx0 = fmaxf(mx0, fmaxf(y0[nt].x, y0[nt].y));
    mx1 = fmaxf(mx1, fmaxf(y1[nt].x, y1[nt].y));
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
  }
  // (where nothing has been seen yet m is -inf, and any score raises it)
  const float top0 = mx0 * post0, top1 = mx1 * post1;
  if (__any_sync(0xffffffffu, top0 > st.m0 + (kHead + kSlack) || top1 > st.m1 + (kHead + kSlack))) {
    const float n0 = top0 > st.m0 + (kHead + kSlack) ? top0 - kHead : st.m0;
    const float n1 = top1 > st.m1 + (kHead + kSlack) ? top1 - kHead : st.m1;
    const float c0 = n0 == -INFINITY ? 1.f : ex2_approx(st.m0 - n0), c1 = n1 == -INFINITY ? 1.f : ex2_approx(st.m1 - n1);
    st.m0 = n0, st.m1 = n1;
    st.l0 *= c0, st.l1 *= c1;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      st.o[j][0] *= c0, st.o[j][1] *= c0;
      st.o[j][2] *= c1, st.o[j][3] *= c1;
    }
  }
  const float ref0 = st.m0 == -INFINITY ? 0.f : st.m0, ref1 = st.m1 == -INFINITY ? 0.f : st.m1;
  const float2 p0 = make_float2(post0, post0), p1 = make_float2(post1, post1);
  const float2 r0 = make_float2(-ref0, -ref0), r1 = make_float2(-ref1, -ref1);
  float2 l0 = make_float2(0.f, 0.f), l1 = l0;
  uint32_t p[2][4];
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) {
    y0[nt] = ffma2_rn(y0[nt], p0, r0);
    y1[nt] = ffma2_rn(y1[nt], p1, r1);
    y0[nt].x = ex2_approx(y0[nt].x), y0[nt].y = ex2_approx(y0[nt].y);
    y1[nt].x = ex2_approx(y1[nt].x), y1[nt].y = ex2_approx(y1[nt].y);
    l0 = fadd2_rn(l0, y0[nt]);
    l1 = fadd2_rn(l1, y1[nt]);
    p[nt / 2][2 * (nt % 2)] = pack_f16(y0[nt].x, y0[nt].y);
    p[nt / 2][2 * (nt % 2) + 1] = pack_f16(y1[nt].x, y1[nt].y);
  }
  st.l0 += l0.x + l0.y;
  st.l1 += l1.x + l1.y;
  const uint32_t va = stage + L::kTileBytes + at.value(), vc = stage + L::kTileBytes + (at.value() ^ Places::kValue1);
  const uint32_t sa = scales + L::kScaleBytes + at.value_scale();
  const uint32_t sb = scales + L::kScaleBytes + (at.value_scale() ^ Places::kScale1);
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    uint2 a[2], c[2];
    uint32_t sc[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int nt = 2 * ks + h;
      a[h] = lds64(va + nt * 512);
      c[h] = lds64(vc + nt * 512);
      uint32_t x = lds8(sa + nt * 64), y = lds8(sb + nt * 64);
      if (kMask) {   // what lies past the request's tokens is zero: any scale is dropped
        if (tb + nt * 8 + ta >= glen) x = 0u;
        if (tb + nt * 8 + tc >= glen) y = 0u;
      }
      sc[h] = e4m3x2_to_f16x2(x | (y << 8));
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      // two tokens' codes of a dim side by side: the even dims, then the odd ones
      constexpr uint32_t kLow = 0x0f0f0f0fu;
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {
        uint32_t v[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = w ? a[h].y : a[h].x, y = w ? c[h].y : c[h].x;
          e2m1x8_to_f16x2x4(odd ? ((x >> 4) & kLow) | (y & ~kLow) : (x & kLow) | ((y << 4) & ~kLow), v[h]);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[h][i] = hmul2(v[h][i], sc[h]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_f16_16816(st.o[8 * w + 2 * i + odd], p[ks], v[0][i], v[1][i]);
      }
    }
  }
}

// A lane's part of a state: 16 dims of a row at a time, four floats a write.
template <class F>
__device__ __forceinline__ void each_quad(float* w0, int t, F&& f) {
  float* w1 = w0 + 8 * L::kStateStride;
#pragma unroll
  for (int j = 0; j < 16; j += 4)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      f(reinterpret_cast<float4*>(w0 + 36 * t + 16 * e + j), j, e);
      f(reinterpret_cast<float4*>(w1 + 36 * t + 16 * e + j), j, e + 2);
    }
}

// As in idx_attn.cu, in units of 0.18 us, an SM's time for a piece.
struct Cost {
  static constexpr float kAlone = 8.f, kEnd = 20.f, kStretch = 24.f, kCut = 26.f, kList = 18.f;
};

// Whether the units of the call are dealt whole to teams of TW warps: as in idx_attn.cu.
template <int TW>
__device__ __forceinline__ bool whole_units(const AttnArgs& a, const Requests& rq, int longest, int C) {
  if (a.shift > 0) return false;
  const int per = (int)a.by_per.d;
  const float units = (float)(a.R * per), each = __fdividef(1.f, (float)C);
  const float total = (float)((rq.pre[a.R] - a.R * a.unit_cost) * per), mean = __fdividef(total, units);
  const float whole = a.dealt_ends + fmaxf(mean, (float)TW) * a.dealt_piece +
                      ((float)longest - mean) * (Cost::kAlone / TW);
  const float cut = fmaxf(total * each, Cost::kAlone) + Cost::kStretch * units * each + Cost::kCut;
  return whole <= cut;
}

// Words of a team's joined list.
__host__ __device__ constexpr int team_list_words(int tw) { return kMaxList / (NW / tw); }

// Every word of a walk and of a stretch.
template <class F>
__device__ __forceinline__ void each_word(F&& f, Walk& w, Segment& s, Items& it) {
  f(w.pos), f(w.end), f(w.start), f(w.r), f(w.head), f(w.group), f(w.unit), f(w.wt), f(w.step);
  f(s.unit), f(s.r), f(s.head), f(s.group), f(s.o0), f(s.o1), f(s.cap), f(s.start);
  f(it.r), f(it.head), f(it.slot), f(it.glen), f(it.kv_head), f(it.i0), f(it.i1);
  static_assert(kColdWords >= 24, "room for them");
}

// The CTA's units, TW warps a unit: its stretch of the line (kCut, TW = NW), or whole units
// dealt in turn to the teams of all CTAs.  record: the unit the CTA started and did not end.
template <bool kBlocks, int TW, bool kCut>
__device__ __forceinline__ void run_units(const AttnArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map,
                                          uint8_t* smem, const Requests& rq, int W, int C, SplitRecord& record) {
  static_assert(TW >= 2 && NW % TW == 0 && (!kCut || TW == NW), "teams");
  const uint32_t sbase = smem_u32(smem);
  unsigned int* cta_flags = reinterpret_cast<unsigned int*>(smem + L::kCtlOff);
  // (one value a warp, and the compiler knows it)
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int team = warp / TW, member = warp % TW, c = blockIdx.x;
  uint32_t* list = reinterpret_cast<uint32_t*>(smem + L::kListOff) + team_list_words(TW) * team;
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem + team * TW * L::kArea);
  uint8_t* q_rows = smem + L::kQOff + team * (kTile * 256);
  Row* rows = reinterpret_cast<Row*>(smem + L::kPostOff) + team * kTile;
  float2* ml = reinterpret_cast<float2*>(smem + L::kMlOff);
  int* cold = reinterpret_cast<int*>(smem + L::kColdOff) + warp * kColdWords;
  auto team_sync = [&]() {
    if (TW == NW)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(TW * 32) : "memory");
  };
  // The warp's D stages are used in turn: its k-th piece lies in stage k % D.
  auto tiles_of = [&](int k) { return sbase + warp * L::kArea + (k % D) * 2 * L::kTileBytes; };
  auto scales_of = [&](int k) {
    return sbase + warp * L::kArea + D * 2 * L::kTileBytes + (k % D) * 2 * L::kScaleBytes;
  };
  auto bar_of = [&](int k) { return sbase + L::kBarOff + (warp * D + k % D) * 8; };
  const Places places(lane);
  const uint32_t q_at = smem_u32(q_rows) + lane * 16;
  bool dead = false;
  int used = 0;          // pieces this warp has waited for
  Walk walk;
  if (kCut)
    walk.begin(a, rq.pre, c < C ? W * c / C : 0, c < C ? W * (c + 1) / C : 0);
  else
    walk.begin_units(a, team * (int)gridDim.x + c, (NW / TW) * (int)gridDim.x);
  while (walk.more()) {
    Segment s = kCut ? walk.next(a, rq.pre) : walk.next_unit(a, rq.pre);
    if (!s.live) continue;
    const int row_first = s.group * kTile;
    const int nrows = min(kTile, a.P * a.nq - row_first);
    const int p0 = a.by_nq.div(row_first);
    int n_items = 0;
    if (kBlocks) {
      n_items = join_lists(a, rq, s, p0, (row_first + nrows - 1) / a.nq, list, bits,
                           threadIdx.x % (32 * TW), 32 * TW, team_sync) *
                (kBlock / kItem);
      // the areas that held the bits get copies again
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      team_sync();
    }
    Items it = make_items<kItem, kBlocks>(a, rq, s, n_items);
    // ---- the warp's pieces: items member, member + TW, ... of the stretch.  Page ids 32
    // pieces at a time, one a lane; -1: nothing to read there ------------------------
    const int n = max(0, (it.i1 - it.i0 - member + TW - 1) / TW), first = it.i0 + member, glen = it.glen;
    const int slot = it.slot, kv_head = it.kv_head;
    auto ids_of = [&](int k) {
      int tb = 0, page = -1;
      uint32_t unused;
      if (k < n && item_tokens<kItem, kBlocks>(glen, list, first + k * TW, tb, unused)) {
        page = __ldg(a.page_table + (size_t)slot * a.max_pages + tb / kPage);
        if (page < 0 || page >= a.num_pages) {
          atomicOr(cta_flags, kErrBadPage);
          page = -1;
        }
      }
      return page;
    };
    int ids = ids_of(lane);
    // Ask for the copies of piece k of the unit, the warp's piece j of all.  exist: a bit for
    // each piece in flight, the oldest lowest; pieces that do not exist arrive at once.
    uint32_t exist = 0u;
    auto issue = [&](int k, int j, int place) {
      if (k > 0 && (k & 31) == 0) ids = ids_of(k + lane);
      const int page = __shfl_sync(0xffffffffu, ids, k & 31);
      int tb;
      uint32_t unused;
      item_tokens<kItem, kBlocks>(glen, list, first + k * TW, tb, unused);
      const uint32_t bar = bar_of(j), to = tiles_of(j), sc = scales_of(j);
      exist |= page >= 0 ? 1u << place : 0u;
      const int row = (page * a.kv_heads + kv_head) * kPage + tb % kPage;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar, page >= 0 ? 2 * (L::kTileBytes + L::kScaleBytes) : 0);
        if (page >= 0) {
          tma_load_2d(to, &k_map, 0, row, bar);
          bulk_load(sc, a.k_scale + (size_t)row * 2, L::kScaleBytes, bar);
          tma_load_2d(to + L::kTileBytes, &v_map, 0, row, bar);
          bulk_load(sc + L::kScaleBytes, a.v_scale + (size_t)row * 2, L::kScaleBytes, bar);
        }
      }
    };
    auto q_index = [&](int pk, int p) {   // packed row pk of the unit head, draft row p = pk / nq
      return ((size_t)s.r * a.P + p) * a.q_heads + s.head * a.nq + (pk - p * a.nq);
    };
    // ---- the unit's queries: the warp's rows, to f16 scaled a row by the power of two that
    // brings the row's largest magnitude into [2^7, 2^8) (undone by post) ----------
    for (int k = 0; k < D && k < n && !dead; ++k) issue(k, used + k, k);
    constexpr int kMine = (kTile + TW - 1) / TW;
    uint2 qw[kMine];
    int lens[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = member + k * TW, pk = row_first + i;
      qw[k] = make_uint2(0, 0);
      // with one draft row the request's longest row is the row
      lens[k] = i < nrows && glen > 0 ? a.P == 1 ? glen : row_len(a, s.r, a.by_nq.div(pk)) : 0;
      if (i < nrows) qw[k] = __ldg(reinterpret_cast<const uint2*>(a.q + q_index(pk, a.by_nq.div(pk)) * kDim) + lane);
    }
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = member + k * TW;
      if (i >= kTile) break;
      float top = fmaxf(fmaxf(fabsf(bf16_lo(qw[k].x)), fabsf(bf16_hi(qw[k].x))),
                        fmaxf(fabsf(bf16_lo(qw[k].y)), fabsf(bf16_hi(qw[k].y))));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int x = to_2_7(top);
      auto power = [](int e) { return __uint_as_float((uint32_t)(e + 127) << 23); };   // -120 .. 120
      const float up = power(x);
      // dims 4 lane ..: step lane % 8, the operand's lane (row % 8, lane / 8), its words of row / 8
      uint32_t* to = reinterpret_cast<uint32_t*>(q_rows + (lane & 7) * 512 + ((i & 7) * 4 + lane / 8) * 16) + i / 8;
      to[0] = pack_f16(bf16_lo(qw[k].x) * up, bf16_hi(qw[k].x) * up);
      to[2] = pack_f16(bf16_lo(qw[k].y) * up, bf16_hi(qw[k].y) * up);
      if (lane == 0) {
        const int p = a.by_nq.div(row_first + i);
        const bool has = i < nrows && glen > 0;
        rows[i] = {fmaxf(a.scale_log2 * power(-x), kLeastPost), lens[k], has ? kBlocks ? 1u << (p - p0) : 1u : 0u};
      }
    }
    team_sync();
    // pieces up to here, whose blocks all of these list, need no mask
    int safe;
    uint32_t drafts;
    {
      const Row r = rows[lane & 15];
      safe = __reduce_min_sync(0xffffffffu, r.bit ? r.len : 0x7fffffff);
      drafts = __reduce_or_sync(0xffffffffu, r.bit);
    }
    // ---- the walk and the stretch wait in shared memory: the registers are the loop's ------
    if (lane == 0) {
      int* k = cold;
      each_word([&](int& x) { *k++ = x; }, walk, s, it);
    }
    __syncwarp();
    State st;
    st.reset();
    // ---- its pieces -----------------------------------------------------------
    for (int k = 0; k < n && !dead; ++k) {
      int tb;
      uint32_t members;
      item_tokens<kItem, kBlocks>(glen, list, first + k * TW, tb, members);
      const bool stall = a.stall_test && warp == 0 && used == 0;
      const bool ok = mbar_wait_bounded(stall ? sbase + L::kBarOff + NW * D * 8 : bar_of(used),
                                        stall ? 0u : (uint32_t)((used / D) & 1), a.wait_ns);
      dead = __any_sync(0xffffffffu, !ok);
      if (dead) {
        if (lane == 0) {
          atomicOr(cta_flags, kErrTimeout);
          // the copies in flight land
          for (int j = 0; j < D && k + j < n; ++j)
            (void)mbar_wait_bounded(bar_of(used + j), (uint32_t)(((used + j) / D) & 1), 200000000ull);
        }
        used += min(D, n - k);
        __syncwarp();
        break;
      }
      if (exist & 1u) {
        if (tb + kItem <= safe && (!kBlocks || (members & drafts) == drafts))
          piece<false>(q_at, rows, st, tiles_of(used), scales_of(used), places, tb, members, glen);
        else
          piece<true>(q_at, rows, st, tiles_of(used), scales_of(used), places, tb, members, glen);
      }
      // every lane's reads of the stage come before the copies that refill it
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      exist >>= 1;
      if (k + D < n) issue(k + D, used + D, D - 1);
      ++used;
    }
    {
      volatile const int* k = cold;
      each_word([&](int& x) { x = *k++; }, walk, s, it);
    }
    // ---- join the warps: a state each, then by rows ------------------------------
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
      st.l0 += __shfl_xor_sync(0xffffffffu, st.l0, o);
      st.l1 += __shfl_xor_sync(0xffffffffu, st.l1, o);
    }
    st.m0 = not_empty(st.m0, st.l0);
    st.m1 = not_empty(st.m1, st.l1);
    float* w0 = reinterpret_cast<float*>(smem + warp * L::kArea) + g * L::kStateStride;
    if (t == 0) {
      ml[warp * kTile + g] = make_float2(st.m0, st.l0);
      ml[warp * kTile + g + 8] = make_float2(st.m1, st.l1);
    }
    each_quad(w0, t, [&](float4* to, int j, int e) {
      *to = make_float4(st.o[j][e], st.o[j + 1][e], st.o[j + 2][e], st.o[j + 3][e]);
    });
    team_sync();
    const int first_row = s.group * kTile, rows_here = min(kTile, a.P * a.nq - first_row), draft0 = a.by_nq.div(first_row);
    const bool complete = !kCut || (s.o0 == 0 && s.o1 == s.cap);
    const int slot_out = 2 * c + (s.o0 == 0 ? 1 : 0);
    if (s.o0 == 0 && !complete) {
      record.unit = s.unit;
      record.splits = owner(s.start + s.cap - 1, W, C) - c + 1;
    }
    for (int i = member; i < rows_here; i += TW) {
      const int pk = first_row + i, p = a.by_nq.div(pk);
      // one state a lane: their maximum, and what each is multiplied by (-1: a warp with
      // nothing visible in the row, whose output is not read)
      float2 x = make_float2(-INFINITY, 0.f);
      if (lane < TW) x = ml[(team * TW + lane) * kTile + i];
      float m = x.x;
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      m = __shfl_sync(0xffffffffu, m, 0);
      const float f = x.x == -INFINITY ? -1.f : ex2_approx(x.x - m);
      float l = x.x == -INFINITY ? 0.f : x.y * f;
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      l = __shfl_sync(0xffffffffu, l, 0);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < TW; ++w) {
        const float fw = __shfl_sync(0xffffffffu, f, w);
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + (team * TW + w) * L::kArea) +
                                                          i * L::kStateStride + 4 * lane + 4 * (lane / 8));
        if (fw != -1.f)
          o = make_float4(fmaf(v.x, fw, o.x), fmaf(v.y, fw, o.y), fmaf(v.z, fw, o.z), fmaf(v.w, fw, o.w));
      }
      if (__any_sync(0xffffffffu, !finite4(o)))
        careful_row<kNvfp4, kItem, kBlocks>(a, it, list, a.q + q_index(pk, p) * kDim,
                                            it.glen > 0 ? row_len(a, s.r, p) : 0, p - draft0, lane, m, l, o);
      if (complete)
        write_row(a, q_index(pk, p), m, l, o, lane);
      else
        put_part(a, slot_out, i, m, l, o, lane);
    }
    // the states' places get copies again
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    team_sync();
  }
}

enum class Deal { kCut, kWhole, kEither };
template <bool kBlocks, int TW, Deal kDeal>
__global__ void __launch_bounds__(L::kThreads, 1)
    attn4_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  unsigned int* cta_flags = reinterpret_cast<unsigned int*>(smem + L::kCtlOff);
  const Requests rq = requests_at(smem + L::kPreOff);

  if (threadIdx.x < L::kNumBars) {
    mbar_init(sbase + L::kBarOff + threadIdx.x * 8, 1);
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
  const int C = min((W + kLeast - 1) / kLeast, (int)gridDim.x);
  SplitRecord record = {-1, 0};
  if constexpr (kDeal == Deal::kCut) {
    run_units<kBlocks, NW, true>(a, k_map, v_map, smem, rq, W, C, record);
  } else if constexpr (kDeal == Deal::kWhole) {
    run_units<kBlocks, TW, false>(a, k_map, v_map, smem, rq, W, C, record);
  } else {
    if (whole_units<TW>(a, rq, (int)cta_flags[1], C))
      run_units<kBlocks, TW, false>(a, k_map, v_map, smem, rq, W, C, record);
    else
      run_units<kBlocks, NW, true>(a, k_map, v_map, smem, rq, W, C, record);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    a.records[blockIdx.x] = record;
    a.err_bytes[blockIdx.x] = (uint8_t)*cta_flags;
    if (blockIdx.x == 0) *a.err_count = gridDim.x;
  }
}

template <bool kBlocks, int TW, Deal kDeal>
cudaError_t launch_one(const AttnArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map,
                       int grid, int dev, cudaStream_t stream) {
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = smem_limit_once(attn4_kernel<kBlocks, TW, kDeal>, L::kSmem, dev, attr_done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn4_kernel<kBlocks, TW, kDeal>, grid, L::kThreads, L::kSmem, stream, a, k_map, v_map);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// The team size for units dealt whole, of so many pieces: as in idx_attn.cu.
template <bool kBlocks>
int team_for(AttnArgs& a, int grid, float pieces, float& least) {
  const int units = a.R * (int)a.by_per.d;
  int team = 0;
  for (int tw : {12, 6, 3}) {   // (single warps: 256 x 8 x 100 tokens 35.3 us, 33.8 without)
    if (kBlocks && (a.P < kMaxDrafts ? a.P : kMaxDrafts) * a.topk > team_list_words(tw)) break;
    const int teams = grid * (NW / tw), full = units / teams, rest = units - full * teams;
    const float busy = (float)(rest * tw) / (float)grid;
    const float last = rest == 0 ? 0.f : busy > Cost::kAlone ? busy : Cost::kAlone;
    const float ends = (float)(full + (rest > 0)) * (Cost::kEnd + (kBlocks ? Cost::kList : 0.f));
    const float piece = ((float)NW * (float)full + last) / (float)tw;
    const float cost = ends + pieces * piece;
    if (team > 0 && cost >= least) continue;
    team = tw;
    least = cost;
    a.dealt_ends = ends;
    a.dealt_piece = piece;
  }
  return team;
}

}  // namespace

cudaError_t launch_attn4(const AttnArgs& args, const CUtensorMap& k_map, const CUtensorMap& v_map,
                         int grid, int dev, cudaStream_t stream, bool& whole) {
  AttnArgs a = args;
  float least;
  const float share = (float)(a.R * (int)a.by_per.d) / (float)grid;
  if (!a.block_ids) {
    // A table that holds short units only (the host knows its width, not the lengths: under a table
    // as wide as the longest context that may come, short units take the first figures): where dealing them whole costs about what cutting them
    // does, the call deals and needs no join (us, cut / dealt: 1 request x 2 key heads x 200 tokens
    // 7.5 / 6.0, x 600 9.8 / 8.4, x 1000 9.3 / 10.3; 16 x 8 x 200 8.6 / 6.8, x 1000 12.4 / 10.6; 64 x 8
    // x 1K 30.0 / 28.3).
    if (a.most <= 40 && a.shift == 0) {
      const int team = team_for<false>(a, grid, (float)a.most, least);
      const float piece = share * (float)a.most;
      const float cut = (piece > Cost::kAlone ? piece : Cost::kAlone) + Cost::kStretch * share + Cost::kCut;
      whole = least <= 1.1f * cut;
      if (whole) switch (team) {
          case 3: return launch_one<false, 3, Deal::kWhole>(a, k_map, v_map, grid, dev, stream);
          case 6: return launch_one<false, 6, Deal::kWhole>(a, k_map, v_map, grid, dev, stream);
          default: return launch_one<false, 12, Deal::kWhole>(a, k_map, v_map, grid, dev, stream);
        }
    }
    // else units of 16 pieces are assumed for the team; how long they are is known on the device
    // only, which decides whether they are dealt whole at all
    whole = false;
    switch (team_for<false>(a, grid, 16.f, least)) {
      case 3: return launch_one<false, 3, Deal::kEither>(a, k_map, v_map, grid, dev, stream);
      case 6: return launch_one<false, 6, Deal::kEither>(a, k_map, v_map, grid, dev, stream);
      default: return launch_one<false, 12, Deal::kEither>(a, k_map, v_map, grid, dev, stream);
    }
  }
  // the lists' length bounds the units', so the host decides, and a call that deals needs no join
  const float full = (float)(a.topk * (kBlock / kItem)) * (1.f + (float)(a.P - 1) / 8.f);
  const float pieces = full < (float)a.most ? full : (float)a.most;
  const int team = team_for<true>(a, grid, pieces, least);
  const float cut = (share * pieces > Cost::kAlone ? share * pieces : Cost::kAlone) +
                    (Cost::kStretch + Cost::kList) * share + Cost::kCut + Cost::kList;
  whole = least <= 0.83f * cut;
  if (!whole) return launch_one<true, 12, Deal::kCut>(a, k_map, v_map, grid, dev, stream);
  switch (team) {
    case 3: return launch_one<true, 3, Deal::kWhole>(a, k_map, v_map, grid, dev, stream);
    case 6: return launch_one<true, 6, Deal::kWhole>(a, k_map, v_map, grid, dev, stream);
    default: return launch_one<true, 12, Deal::kWhole>(a, k_map, v_map, grid, dev, stream);
  }
}

}  // namespace idx
