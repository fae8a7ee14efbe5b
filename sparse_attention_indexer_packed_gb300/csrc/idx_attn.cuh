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
// The split.  Every unit of request r has weight wt(r) = items(r) + kUnitCost,
// items(r) = its pieces (with block lists: an upper bound of them).
// The units' weights lie end to end on a line of W positions, in the order
// (request, unit head, row group); CTA c of C takes [W c / C, W (c + 1) / C).
// A CTA's part of a unit is its items inside that range; the last kUnitCost
// positions of a unit stand for the cost of ending it and hold no item, except
// that a unit with no items is ended by the CTA that holds its first position.
// ---------------------------------------------------------------------------
constexpr int kUnitCost = 8;

struct Segment {
  int unit;          // (r * heads + unit head) * groups + group
  int r, head, group;
  int o0, o1, cap;   // items [o0, o1) of cap
  long long start;   // the unit's first position
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

// x / y of two positions (x >= 0, y > 0): in 32 bits where they fit, which is
// several times as fast.
__device__ __forceinline__ long long div(long long x, long long y) {
  if (((x | y) >> 32) == 0) return (unsigned int)x / (unsigned int)y;
  return x / y;
}

// A walk over the stretches of [pos, end), unit by unit: one search at its
// start, no division after it.
struct Walk {
  long long pos, end, start;   // start: the current unit's first position
  int r, head, group, unit, wt;

  __device__ __forceinline__ void begin(const int* pre, int R, int heads, int groups,
                                        long long first, long long last) {
    pos = first;
    end = last;
    if (pos >= end) return;
    const int per = heads * groups;
    r = find_request(pre, R, (int)div(pos, per));
    wt = pre[r + 1] - pre[r];
    const long long base = (long long)pre[r] * per;
    const int k = (int)div(pos - base, wt);
    start = base + (long long)k * wt;
    head = k / groups;
    group = k - head * groups;
    unit = r * per + k;
  }
  __device__ __forceinline__ bool more() const { return pos < end; }
  __device__ __forceinline__ Segment next(const int* pre, int R, int heads, int groups) {
    Segment s;
    s.unit = unit;
    s.r = r;
    s.head = head;
    s.group = group;
    s.start = start;
    s.cap = wt - kUnitCost;
    const int o = (int)(pos - start);
    const long long left = end - pos;
    const int take = left < wt - o ? (int)left : wt - o;
    s.o0 = o < s.cap ? o : s.cap;
    s.o1 = o + take < s.cap ? o + take : s.cap;
    s.live = s.o1 > s.o0 || (s.cap == 0 && o == 0);
    pos += take;
    if (o + take == wt) {
      start += wt;
      ++unit;
      if (++group == groups) {
        group = 0;
        if (++head == heads) {
          head = 0;
          if (++r < R) wt = pre[r + 1] - pre[r];
        }
      }
    }
    return s;
  }
};

// The CTA that holds position x.
__device__ __forceinline__ int owner(long long x, long long W, int C) {
  return (int)div((x + 1) * C + W - 1, W) - 1;
}

}  // namespace attn

cudaError_t launch_attn(int key_format, const AttnArgs& args, const CUtensorMap& k_map,
                        const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_attn_wide(int key_format, const AttnArgs& args, const CUtensorMap& k_map,
                             const CUtensorMap& v_map, int grid, int dev, cudaStream_t stream);
// CTAs launch_attn uses on the current device (0: the device cannot be asked).
int attn_ctas();

}  // namespace idx
