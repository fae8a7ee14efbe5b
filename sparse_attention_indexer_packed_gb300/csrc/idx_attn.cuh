// Shared pieces of the attention kernels: the call's arguments, the split of the
// work over CTAs, and the layout of the partial results in the workspace.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "idx_internal.cuh"

namespace idx {
namespace attn {

constexpr int kMaxCtas = 192;      // CTAs of one call (the grid is one per SM)
constexpr int kMaxDrafts = 16;     // draft rows whose block lists one row group joins

constexpr uint32_t kErrBadPage = 1u;
constexpr uint32_t kErrTimeout = 2u;
constexpr uint32_t kErrLenClamped = 4u;

// Where a unit that several CTAs share begins: written by the CTA that starts
// it, read by the join kernel.  unit < 0: this CTA starts no shared unit.
struct SplitRecord {
  int unit, splits;
};

// Division of x in [0, 2^31) by a fixed d in [1, 2^31): (x * m) >> (32 + s) with
// m = ceil(2^(32 + s) / d), s = ceil(log2 d) - 1 (Granlund and Montgomery, "Division
// by Invariant Integers using Multiplication", 1994): exact for 31-bit x.
struct Divisor {
  unsigned int d, m, s;
  static Divisor of(int d) {
    Divisor v;
    v.d = (unsigned int)d;
    v.s = 0;
    while ((2ull << v.s) < (unsigned long long)d) ++v.s;
    v.m = (unsigned int)((((1ull << 32) << v.s) + d - 1) / d);
    return v;
  }
  __device__ __forceinline__ int div(int x) const {
    return d == 1 ? x : (int)(__umulhi((unsigned int)x, m) >> s);
  }
};

}  // namespace attn

// Arguments of one attention call.  A "unit" is what shares one read of the
// keys and values: the query heads of one request that go by the same key head
// and the same block list, cut into groups of `group_rows` packed rows.  Packed
// row i of a unit is (draft row i / nq, query head unit_head * nq + i % nq).
struct AttnArgs {
  const uint16_t* q;           // bf16 [R][P][q_heads][128]
  const uint8_t* k_payload;    // plane rows (page * kv_heads + head) * 64 + token % 64
  const float* k_scale;        // one a row (fp8) or nullptr
  const uint8_t* v_payload;
  const float* v_scale;
  const int32_t* page_table;   // [n_slots][max_pages]
  const int32_t* slot_ids;     // [R]
  const int32_t* row_lens;     // [R][P]
  const int32_t* block_ids;    // [R][P][lists][topk], or nullptr: every block
  uint16_t* out;               // bf16 [R][P][q_heads][128]
  float* lse;                  // [R][P][q_heads] or nullptr
  attn::SplitRecord* records;  // [CTAs]
  float2* part_ml;             // [2 * CTAs][group_rows]: running max (log2 units) and sum
  float* part_o;               // [2 * CTAs][group_rows][128]: unnormalised output
  uint8_t* err_bytes;          // one flag byte per CTA
  uint32_t* err_count;         // CTAs that wrote a flag byte
  int64_t num_pages;
  int n_slots, max_pages;
  int R, P, q_heads, kv_heads, lists, topk;
  int heads;                   // unit heads of a request: max(kv_heads, lists)
  int nq;                      // query heads of a unit head
  int group_rows;              // packed rows of a group (16, or up to 128)
  int groups;                  // row groups of a unit head
  attn::Divisor by_per, by_groups, by_nq, by_topk;  // heads * groups, groups, nq, topk
  attn::Divisor by_kv, by_list;  // unit heads of a key head, of a list
  long long most;              // pieces a unit may have at most, as the host knows it
  int shift;                   // pieces of a position: 2^shift
  int unit_cost;               // positions that stand for a unit's end
  float dealt_ends, dealt_piece;  // estimate of units dealt whole (up to 16 rows, no lists)
  float scale_log2;            // softmax scale times log2(e)
  unsigned long long wait_ns;
  int stall_test;
};

namespace attn {

// Packed rows of a group: what one read of the keys serves.  Up to 16 rows go to
// the warp-level kernel, more to the tensor-memory one, 128 at most; a group of
// block lists joins those of kMaxDrafts draft rows at most.
inline int group_rows(int drafts, int nq, bool blocks) {
  if ((long long)drafts * nq <= 16) return 16;
  return blocks && nq * kMaxDrafts < 128 ? nq * kMaxDrafts : 128;
}

// Bytes of the workspace after the header: records, then the partials.
inline size_t records_bytes() { return (size_t)kMaxCtas * sizeof(SplitRecord); }
inline size_t part_ml_bytes(int ctas, int group_rows) {
  return (size_t)2 * ctas * group_rows * sizeof(float2);
}
inline size_t part_o_bytes(int ctas, int group_rows) {
  return (size_t)2 * ctas * group_rows * kDim * sizeof(float);
}

// ---------------------------------------------------------------------------
// The split.  Every unit of request r has weight wt(r) = cap(r) + unit_cost, cap(r)
// = its pieces (with block lists: an upper bound of them) in lots of 2^shift.  The
// units' weights lie end to end on a line of W positions, in the order (request,
// unit head, row group); CTA c of C takes [W c / C, W (c + 1) / C).  A CTA's part of
// a unit is its lots inside that range; the last unit_cost positions of a unit
// stand for the cost of ending it and hold none, except that a unit with no lot is
// ended by the CTA that holds its first position.  The host picks the shift (0 but
// for calls of many million pieces) so that W * (C + 1) stays below 2^31.
// ---------------------------------------------------------------------------
constexpr int kLeast = 8, kLeastWide = 4;   // positions a CTA takes at least
constexpr long long kMaxPositions = 0x7fffffffll / (kMaxCtas + 1);
constexpr long long kMaxUnits = 1 << 18;
constexpr int kMaxUnitCost = 32;
static_assert(kMaxUnits * (kMaxUnitCost + 1) <= kMaxPositions, "units must fit the line");

// Positions that stand for a unit's end, in pieces of its kernel.  A stretch of a
// unit costs a CTA about 2.5 us beside its pieces (queries, join, output; 5 with
// lists, which are joined too and whose copies start anew).  Too few and a CTA ends
// up with many small units; too many and the long ones wait.  Measured (us a call):
// 48 ragged requests x 4 heads 36.2 / 28.3 / 24.9 / 26.9 at 4 / 8 / 12 / 24; 24
// ragged requests with lists 25.5 / 20.6 / 17.8 / 18.1 at 4 / 8 / 24 / 48; 16 x 131K
// with lists 66.5 / 65.3 / 64.2 at 4 / 32 / 64.
inline int unit_cost(int group_rows, bool blocks) {
  return group_rows > 16 ? (blocks ? 16 : 8) : (blocks ? 32 : 12);
}

// The most half-page pieces a unit of the call may have, from what the host knows:
// the page table's width, and with block lists the entries of all draft rows.
inline long long most_pieces(int pages, long long listed) {
  return listed > 0 && listed < (pages + 1) / 2 ? 4 * listed : 2ll * pages + 2;
}

// The shift of a call of R requests with `per` units each.
inline int position_shift(int R, long long per, long long most, int unit_cost) {
  int shift = 0;
  while (R * per * (((most + (1ll << shift) - 1) >> shift) + unit_cost) > kMaxPositions && shift < 24) ++shift;
  return shift;
}

struct Segment {
  int unit;          // (r * heads + unit head) * groups + group
  int r, head, group;
  int o0, o1, cap;   // lots [o0, o1) of cap
  int start;         // the unit's first position
  bool live;         // false: nothing to do in this stretch
};

// Largest r with pre[r] <= x.
__device__ __forceinline__ int find_request(const int* pre, int R, int x) {
  int lo = 0, hi = R - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A walk over the stretches of [pos, end), unit by unit: one search at its
// start, no division after it.  Or (begin_units) over whole units, every step-th.
struct Walk {
  int pos, end, start;   // start: the current unit's first position
  int r, head, group, unit, wt;
  int step;              // 0: stretches

  __device__ __forceinline__ void begin_units(const AttnArgs& a, int first, int stride) {
    pos = first;
    end = a.R * (int)a.by_per.d;
    step = stride;
  }

  __device__ __forceinline__ void begin(const AttnArgs& a, const int* pre, int first, int last) {
    pos = first;
    end = last;
    step = 0;
    if (pos >= end) return;
    r = find_request(pre, a.R, a.by_per.div(pos));
    wt = pre[r + 1] - pre[r];
    const int per = (int)a.by_per.d, base = pre[r] * per;
    const int k = per == 1 ? 0 : (pos - base) / wt;
    start = base + k * wt;
    head = a.by_groups.div(k);
    group = k - head * a.groups;
    unit = r * per + k;
  }
  __device__ __forceinline__ bool more() const { return pos < end; }
  __device__ __forceinline__ Segment next_unit(const AttnArgs& a, const int* pre) {
    Segment s;
    s.unit = pos;
    s.r = a.by_per.div(pos);
    const int k = pos - s.r * (int)a.by_per.d;
    s.head = a.by_groups.div(k);
    s.group = k - s.head * a.groups;
    s.start = 0;
    s.cap = pre[s.r + 1] - pre[s.r] - a.unit_cost;
    s.o0 = 0;
    s.o1 = s.cap;
    s.live = true;
    pos += step;
    return s;
  }
  __device__ __forceinline__ Segment next(const AttnArgs& a, const int* pre) {
    Segment s;
    s.unit = unit;
    s.r = r;
    s.head = head;
    s.group = group;
    s.start = start;
    s.cap = wt - a.unit_cost;
    const int o = pos - start, take = min(end - pos, wt - o);
    s.o0 = min(o, s.cap);
    s.o1 = min(o + take, s.cap);
    s.live = s.o1 > s.o0 || (s.cap == 0 && o == 0);
    pos += take;
    if (o + take == wt) {
      start += wt;
      ++unit;
      if (++group == a.groups) {
        group = 0;
        if (++head == a.heads) {
          head = 0;
          if (++r < a.R) wt = pre[r + 1] - pre[r];
        }
      }
    }
    return s;
  }
};

// The CTA that holds position x.
__device__ __forceinline__ int owner(int x, int W, int C) {
  return ((x + 1) * C + W - 1) / W - 1;   // at most W (C + 1) < 2^31
}

}  // namespace attn

cudaError_t launch_attn(int key_format, const AttnArgs& args, const CUtensorMap& k_map,
                        const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_attn_wide(int key_format, const AttnArgs& args, const CUtensorMap& k_map,
                             const CUtensorMap& v_map, int grid, int dev, cudaStream_t stream);
// CTAs launch_attn uses on the current device (0: the device cannot be asked).
int attn_ctas();

}  // namespace idx
