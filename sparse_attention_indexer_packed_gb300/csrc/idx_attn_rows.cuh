// Device code that both attention kernels use: lengths and items, the joined
// block list of a row group, the token-by-token row, and the output row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "idx_attn.cuh"
#include "idx_ptx.cuh"

namespace idx {
namespace attn {

// Two fp32 sums, or fused multiply-adds, in one instruction (see fmul2_rn).
__device__ __forceinline__ float2 fadd2_rn(float2 a, float2 b) {
  unsigned long long pa, pb, pd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(pa) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(pb) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(pd) : "l"(pa), "l"(pb));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(pd));
  return d;
}
__device__ __forceinline__ float2 ffma2_rn(float2 a, float2 b, float2 c) {
  unsigned long long pa, pb, pc, pd;
  asm("mov.b64 %0, {%1, %2};" : "=l"(pa) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(pb) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(pc) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(pd) : "l"(pa), "l"(pb), "l"(pc));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(pd));
  return d;
}

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxList = kMaxTopk * kMaxDrafts;  // joined block list of a group
constexpr int kMaxBlockWords = 65536 / 2 / 32;   // bits for every block of a request

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Four e4m3 codes of four floats (round to nearest even, saturating), and what
// they stand for taken off the floats.
__device__ __forceinline__ uint32_t e4m3x4_take(float (&x)[4]) {
  uint32_t d;
  asm("{\n\t.reg .b16 h0, h1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h0, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h1, %4, %3;\n\t"
      "mov.b32 %0, {h0, h1};\n\t}"
      : "=r"(d)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
  uint32_t lo, hi;
  e4m3x4_to_f16x2x2(d, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  x[0] -= a.x, x[1] -= a.y, x[2] -= b.x, x[3] -= b.y;
  return d;
}

// Four e5m2 codes of four floats (round to nearest even).
__device__ __forceinline__ uint32_t e5m2x4(const float (&x)[4]) {
  uint32_t d;
  asm("{\n\t.reg .b16 h0, h1;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 h0, %2, %1;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 h1, %4, %3;\n\t"
      "mov.b32 %0, {h0, h1};\n\t}"
      : "=r"(d)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
  return d;
}

// The exponent e that brings x * 2^e into [2^7, 2^8) (0 for zero), at most 100: every
// bf16 above 2^-93 has it, the largest -120.
__device__ __forceinline__ int to_2_7(float x) {
  int e = 0;
  if (x > 0.f) e = 7 - (((int)(__float_as_uint(x) >> 23) & 0xff) - 127);
  return min(100, e);
}

// e4m3 values.  A token enters the product with the values as weight times value
// scale, 2^(x - m) vs for a score of x (log2 units), in one f16: 11 bits, and 2^-25 of
// the output's unit.  So the unit 2^n follows the largest such product that the row
// has seen, which is then held as [2^3, 2^14]: what a token counts for sets it, neither
// its scale nor its weight alone, and the smallest products lose bits, never the
// largest.  2^n is absolute: a maximum that rises takes no part in it.
constexpr float kMostHeld = 16384.f;
// The factor from weights in units of 2^m to the output's unit.  A row that has not
// seen a score above -inf has neither.
__device__ __forceinline__ float to_unit(float m, float n) {
  return m == -INFINITY ? 0.f : ex2_approx(m - n);
}
// Whether products of up to `top`, with the factor f to the unit, may be past it.
__device__ __forceinline__ bool past_unit(float top, float f) { return !(top * f <= kMostHeld); }
// Raise n where the largest product, top 2^m, is past it: its exponent less 3.  (Where
// every product is zero n is 2^113 below the weights.)  Returns what the output
// gathered so far is to be multiplied by.
__device__ __forceinline__ float raise_unit(float top, float m, float& n) {
  if (m == -INFINITY || !past_unit(top, to_unit(m, n))) return 1.f;
  const int e = max((int)((__float_as_uint(top) >> 23) & 0xffu) - 127, -110);
  const float up = m + (float)(e - 3), factor = ex2_approx(n - up);
  n = up;
  return factor;
}

// Length of draft row p of request r, inside [0, max_pages * 64].
__device__ __forceinline__ int row_len(const AttnArgs& a, int r, int p) {
  const int L = __ldg(a.row_lens + r * a.P + p), cap = a.max_pages * kPage;
  return L < 0 ? 0 : (L > cap ? cap : L);
}

// The requests as the CTA needs them: pre[r] = sum of the unit weights of the
// requests before r (pre[R]: the total), their slots and their longest rows (0
// for a pad request).
struct Requests {
  int *pre, *slot, *len;
};
constexpr int kRequestsBytes = 3 * (kMaxGroups + 4) * 4;
__device__ __forceinline__ Requests requests_at(uint8_t* smem) {
  int* p = reinterpret_cast<int*>(smem);
  return {p, p + (kMaxGroups + 4), p + 2 * (kMaxGroups + 4)};
}

// Fill the table (every thread of the CTA, one request a thread at a time; ends
// with a barrier).  sums: one int a warp.  flags gets IDX_DEVERR_LEN_CLAMPED
// from the first CTA.  kWide (the wide kernel): where a request has 32 draft rows
// or more and the requests are two a warp at most, a warp takes a request first,
// its lanes over the rows: 4 requests of 256 rows 27.1 -> 20.2 us, 8 of 64
// 19.5 -> 18.1, 16 of 32 20.9 -> 20.5; but 128 of 64 24.6 -> 27.6 and 512 of 17
// 25.9 -> 41.0, so more requests stay one a thread.
template <int IT, bool kBlocks, bool kWide>
__device__ __forceinline__ void build_requests(const AttnArgs& a, const Requests& q, int* sums,
                                               unsigned int* flags) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nt = blockDim.x;
  int* longest = reinterpret_cast<int*>(flags + 1);   // pieces of the longest unit (not kWide)
  if (threadIdx.x == 0) *flags = 0u;
  if (!kWide && threadIdx.x == 0) *longest = 0;
  const bool many = kWide && a.P >= 32 && a.R <= 2 * (nt / 32);
  if (many) {
    for (int v = warp; v < a.R; v += nt / 32) {
      int most = 0;
      for (int p = lane; p < a.P; p += 32) most = max(most, __ldg(a.row_lens + (size_t)v * a.P + p));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
      if (lane == 0) q.len[v] = most;
    }
    __syncthreads();
  }
  int run = 0;
  for (int v0 = 0; v0 < a.R; v0 += nt) {
    const int v = v0 + threadIdx.x;
    int wt = 0, n = 0, lots = 0;
    bool clamped = false;
    if (v < a.R) {
      // every load goes out before any is used
      const int slot = __ldg(a.slot_ids + v), cap = a.max_pages * kPage;
      int most = 0;
      if (many) {
        most = q.len[v];
      } else {
#pragma unroll 4
        for (int p = 0; p < a.P; ++p) most = max(most, __ldg(a.row_lens + v * a.P + p));
      }
      const bool pad = slot < 0 || slot >= a.n_slots;
      clamped = !pad && most > cap && blockIdx.x == 0;
      n = pad ? 0 : min(most, cap);
      q.slot[v] = slot;
      q.len[v] = n;
      if (kBlocks) {
        // at most: every draft row of a group lists other blocks
        const int drafts = min(a.P, (a.group_rows + a.nq - 2) / a.nq + 1);
        wt = min((n + kBlock - 1) / kBlock, a.topk * drafts) * (kBlock / IT);
      } else {
        wt = (n + IT - 1) / IT;
      }
      lots = (wt + (1 << a.shift) - 1) >> a.shift;
      wt = lots + a.unit_cost;
    }
    int incl = wt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int before = run, total = run;
    for (int w = 0; w < nt / 32; ++w) {
      const int y = sums[w];
      if (w < warp) before += y;
      total += y;
    }
    if (v < a.R) q.pre[v] = before + incl - wt;
    if (!kWide) {
      lots = __reduce_max_sync(0xffffffffu, lots);
      if (lane == 0) atomicMax(longest, lots);
    }
    if (clamped) atomicOr(flags, kErrLenClamped);
    run = total;
    __syncthreads();   // sums is free again, and the table complete
  }
  if (threadIdx.x == 0) q.pre[a.R] = run;
  __syncthreads();
}

// The lists of draft rows p0 .. p1 (at most kMaxDrafts) of the segment's unit
// joined in ascending order: list[i] = block id | drafts that list it << 16, bit
// p - p0.  All nt threads that share the unit, tid of them this one, with their
// barrier; returns the number of blocks.  bits: 2 * kMaxBlockWords words of scratch.  A set bit a block and a running count of them
// give each entry its place, so a block listed twice takes one.
template <class Sync>
__device__ __forceinline__ int join_lists(const AttnArgs& a, const Requests& rq, const Segment& s,
                                          int p0, int p1, uint32_t* list, uint32_t* bits, int tid,
                                          int nt, const Sync& sync) {
  constexpr int kKeep = 2;   // entries a thread keeps in registers between the passes
  uint32_t* rank = bits + kMaxBlockWords;
  const int lane = tid & 31;
  const int which = a.by_list.div(s.head);
  const int longest = rq.len[s.r];
  const int words = (longest + 32 * kBlock - 1) / (32 * kBlock);
  const int entries = longest > 0 ? (p1 - p0 + 1) * a.topk : 0;
  auto entry = [&](int e, int& p) {
    const int d = a.by_topk.div(e);
    p = p0 + d;
    const int id = __ldg(a.block_ids + (((size_t)s.r * a.P + p) * a.lists + which) * a.topk + (e - d * a.topk));
    return id >= 0 && (long long)id * kBlock < row_len(a, s.r, p) ? id : -1;
  };
  int keep[kKeep], who[kKeep];
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int e = tid + k * nt;
    who[k] = 0;
    keep[k] = e < entries ? entry(e, who[k]) : -1;
  }
  for (int w = tid; w < words; w += nt) bits[w] = 0u;
  for (int w = tid; w < entries; w += nt) list[w] = 0u;
  sync();
  auto each = [&](auto&& f) {
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
      if (keep[k] >= 0) f(keep[k], who[k]);
    for (int e = tid + kKeep * nt; e < entries; e += nt) {
      int p;
      const int id = entry(e, p);
      if (id >= 0) f(id, p);
    }
  };
  each([&](int id, int) { atomicOr(&bits[id >> 5], 1u << (id & 31)); });
  sync();
  // blocks before each word: every warp for itself, and in shared memory
  int run = 0;
  for (int w0 = 0; w0 < words; w0 += 32) {
    const int w = w0 + lane;
    const int cnt = w < words ? __popc(bits[w]) : 0;
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (w < words) rank[w] = (uint32_t)(run + incl - cnt);   // every warp writes the same
    run += __shfl_sync(0xffffffffu, incl, 31);
  }
  __syncwarp();
  each([&](int id, int p) {
    const uint32_t at = rank[id >> 5] + __popc(bits[id >> 5] & ((1u << (id & 31)) - 1u));
    atomicOr(&list[at], (uint32_t)id | (1u << (16 + p - p0)));
  });
  sync();
  return run;
}

// What scores are multiplied by is never 0: a masked score's -inf would turn NaN.
// (Scores that small are 0 next to anything.)
constexpr float kLeastPost = 0x1p-126f;

// Four consecutive dims of a plane row as fp32.
template <int KF>
__device__ __forceinline__ float4 plane_f32(const uint8_t* payload, const float* scale,
                                            long long row, int lane) {
  if (KF == kBf16) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(payload + row * 256) + lane);
    return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
  }
  uint32_t lo, hi;
  e4m3x4_to_f16x2x2(__ldg(reinterpret_cast<const uint32_t*>(payload + row * 128) + lane), lo, hi);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  const float s = __ldg(scale + row);
  return make_float4(x.x * s, x.y * s, y.x * s, y.y * s);
}

// A stretch of one unit: which tokens its items are.
struct Items {
  int r, head, slot, glen, kv_head;
  int i0, i1;
};

// The items of a stretch.  n: the unit's joined items (block lists), of which the
// stretch takes the share that its positions have of the unit's.
template <int IT, bool kBlocks>
__device__ __forceinline__ Items make_items(const AttnArgs& a, const Requests& rq, const Segment& s,
                                            int n) {
  Items it;
  it.r = s.r;
  it.head = s.head;
  it.kv_head = a.by_kv.div(s.head);
  it.slot = rq.slot[s.r];
  it.glen = rq.len[s.r];
  if (kBlocks) {
    // the unit has n items, at most cap lots: every CTA takes its share of them
    const int lots = (n + (1 << a.shift) - 1) >> a.shift;
    const bool exact = lots >= s.cap;
    it.i0 = exact ? s.o0 : (int)((float)lots * (float)s.o0 / (float)s.cap);
    it.i1 = exact || s.o1 == s.cap ? min(s.o1, lots) : (int)((float)lots * (float)s.o1 / (float)s.cap);
  } else {
    n = (it.glen + IT - 1) / IT;
    it.i0 = s.o0;
    it.i1 = s.o1;
  }
  it.i0 = min(it.i0 << a.shift, n);
  it.i1 = min(it.i1 << a.shift, n);
  return it;
}

// Item i of the stretch: its first token, and for block lists the drafts that
// list its block (bit p - p0, below kMaxDrafts; a group of the whole cache may have
// more draft rows than the word has bits, and they all see it).  False: nothing there.
template <int IT, bool kBlocks>
__device__ __forceinline__ bool item_tokens(const Items& it, const uint32_t* list, int i, int& tb,
                                            uint32_t& members) {
  if (kBlocks) {
    constexpr int kPer = kBlock / IT;
    const uint32_t e = list[i / kPer];
    tb = (int)(e & 0xffffu) * kBlock + (i % kPer) * IT;
    members = e >> 16;
  } else {
    tb = i * IT;
    members = 0xffffffffu;
  }
  return tb < it.glen;
}

// Plane row of the item's first token, -1 if its page id is out of range.
__device__ __forceinline__ long long item_row(const AttnArgs& a, const Items& it, int tb) {
  const int page = __ldg(a.page_table + (size_t)it.slot * a.max_pages + tb / kPage);
  if (page < 0 || page >= a.num_pages) return -1;
  return ((long long)page * a.kv_heads + it.kv_head) * kPage + tb % kPage;
}

// The running maximum of a row's part for the join.  -inf means "no visible token"
// there, and the part is not read; a row that saw nothing but NaN scores has that
// maximum too, but its sum is NaN, and any finite value keeps it in.
__device__ __forceinline__ float not_empty(float m, float l) {
  return m == -INFINITY && l != l ? 0.f : m;
}

// One row of a stretch token by token (one warp, lane = four dims), for rows
// whose joined output is not finite: the tiled products put 0 * NaN into a row
// that does not see the NaN, this does not.
template <int KF, int IT, bool kBlocks>
__device__ __noinline__ void careful_row(const AttnArgs& a, const Items& it, const uint32_t* list,
                                         const uint16_t* q, int len, int draft_bit, int lane,
                                         float& m, float& l, float4& o) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(q) + lane);
  const float4 qv = make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
  m = -INFINITY;
  l = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = it.i0; i < it.i1; ++i) {
    int tb;
    uint32_t members;
    if (!item_tokens<IT, kBlocks>(it, list, i, tb, members)) continue;
    if (kBlocks && !((members >> draft_bit) & 1u)) continue;
    const long long row = item_row(a, it, tb);
    if (row < 0) continue;
    for (int e = 0; e < IT && tb + e < len; ++e) {
      const float4 k = plane_f32<KF>(a.k_payload, a.k_scale, row + e, lane);
      float x = qv.x * k.x + qv.y * k.y + qv.z * k.z + qv.w * k.w;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      x *= a.scale_log2;
      if (x == -INFINITY) continue;
      const float mn = fmaxf(m, x), c = ex2_approx(m - mn), p = ex2_approx(x - mn);
      const float4 v = plane_f32<KF>(a.v_payload, a.v_scale, row + e, lane);
      l = l * c + p;
      o = make_float4(o.x * c + p * v.x, o.y * c + p * v.y, o.z * c + p * v.z, o.w * c + p * v.w);
      m = mn;
    }
  }
  m = not_empty(m, l);
}

__device__ __forceinline__ bool finite4(float4 o) {
  return isfinite(o.x) && isfinite(o.y) && isfinite(o.z) && isfinite(o.w);
}

// Write a finished row: lane = four dims.
__device__ __forceinline__ void write_row(const AttnArgs& a, size_t row, float m, float l, float4 o,
                                          int lane) {
  const float inv = m == -INFINITY ? 0.f : 1.f / l;
  uint2 u;
  u.x = m == -INFINITY ? 0u : pack_bf16(o.x * inv, o.y * inv);
  u.y = m == -INFINITY ? 0u : pack_bf16(o.z * inv, o.w * inv);
  reinterpret_cast<uint2*>(a.out + row * kDim)[lane] = u;
  if (lane == 0 && a.lse) a.lse[row] = m == -INFINITY ? m : (m + log2f(l)) * kLn2;
}

}  // namespace attn
}  // namespace idx
