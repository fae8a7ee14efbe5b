// Attention with more than 16 packed rows a unit (draft rows x query heads of one
// key head), on the 5th-generation tensor cores.
//
// The mathematics is idx_attn.cu's; here up to 128 packed rows are the M = 128
// rows of one tcgen05 product, and a tile is one page: S = Q K^T (N = 64 tokens,
// K = 128 dims), then O += P V (N = 128 dims, K = 64 tokens), both accumulated in
// fp32 in tensor memory.  The queries and the weights P are operands in tensor
// memory, the keys and values go from TMA's tiles in shared memory straight into
// the products: no key or value passes through registers.
//
// What bounds it: the cache's bytes.  A bf16 page is 32 KB, 1400 cycles of an
// SM's share of the HBM rate; the products take ~400 of them, and of each softmax
// group's ~2800 cycles a page (two groups alternate) half is waiting for scores.
//
// How a row is laid out.  A lane of a softmax warp owns one tensor-memory lane,
// so the softmax needs no shuffle.  With 64 rows or fewer each row is given F =
// 128 / rows lanes, the query repeated in each, and each of the F lanes takes its
// own 64 / F tokens of the page: it weighs those, leaves zeros for the others, and
// so gathers an output and a (max, sum) of its own.  All 128 lanes work whatever
// the row count; the F parts meet once, at the unit's end.
//
// Roles (one CTA per SM, the split of idx_attn.cuh in pages):
//   warps 0-3, 4-7  two softmax groups; pages alternate between them, each with
//               its own S, P and O in tensor memory, so one group's arithmetic
//               runs under the other's products;
//   warp 8      TMA producer (page table, keys, values, scales; a ring of pages);
//   warp 9      issues the products, one elected lane.
// The running maximum is only raised when a score passes it by 2^8 (weights up
// to 2^8 are as exact as any): the output is rescaled then, which is rare.
//
// Precision.  bf16 cache: the weights are two bf16 (16 bits).  e4m3 cache: the
// keys meet the queries as e4m3 codes, the query split into an e4m3 term (4 of its 8
// significant bits) and an e5m2 term: what is left is a whole number up to 8 of the
// query's own last place, which 3 bits hold.  Exact for elements within 2^13 of the
// row's largest, and off by 2^-21 of the largest below (checked over every bf16
// value; with e4m3 as the second term 2^10 and 2^-17, e5m2 reaches 2^7 lower); the
// values are decoded to f16, exactly, by the group that uses them, and the weights
// times the value's scale are one f16 (11 bits; raise_unit).
//
// Measured (one GB300, calls back to back): bf16 16 x 131K with 64 rows 162 to
// 167 us, 0.87 to 0.90 of the copy peak from one GPU to another (the warp-level kernel, four groups of 16 rows:
// 548); 32 rows 157 us, 0.93.  128 rows, 8 x 64K: 72 to 74 us, 0.51: a lane's 64
// weights.  e4m3, 64 rows 160 us, 0.47; 32 rows 147: a group needs ~2700 cycles a page
// (waits 600, decoding the values 540, weights 930, two thirds of it the scales), and
// two groups alternate.  Up to 16 rows this kernel is the slower one (e4m3 16 x 131K
// 152 us against 122 at the time, 1 x 1K 12.8 against 9.3).
// Registers: 168 a thread at launch, and every instantiation spills; bytes of stores /
// loads (-Xptxas -v) for 17 to 32, 33 to 64, 65 to 128 rows: bf16 4 / 4, 92 / 48, 148 /
// 552, with lists 72 / 24, 216 / 224, 164 / 324; e4m3 156 / 224, 152 / 232, 128 / 232,
// with lists 124 / 236, 160 / 280, 160 / 276.
// Tried and slower: the values decoded by four warps of their own (161 -> 189); each
// group finishing a slice through shared memory at a unit's end (166 -> 183).
//
// Every wait is bounded, as in the score kernels.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "idx_attn.cuh"
#include "idx_attn_rows.cuh"
#include "idx_ptx.cuh"
#include "idx_tc.cuh"

namespace idx {

namespace {

using namespace attn;

constexpr int kTok = kPage;          // tokens of a tile
constexpr int kLanes = 128;          // tensor-memory lanes, product rows
constexpr float kSlack = 8.f;        // log2 units a score may pass the running maximum by
// Tensor-memory columns: the queries; S of each group, and in its place P (bf16
// caches), or P of its own, 32 columns a group (e4m3); O of each group.
constexpr int kColQ = 0, kColS = 64, kColP = 192, kColO = 256, kCols = 512;

template <int KF>
struct AWCfg;
template <>
struct AWCfg<kBf16> {
  static constexpr int kRowBytes = 256;
  static constexpr int kStages = 5;
  // bit 16: the second operand (the values) runs along N
  static constexpr uint32_t kIdQK = instr_desc(1u, kLanes, kTok);
  static constexpr uint32_t kIdPV = instr_desc(1u, kLanes, kDim) | (1u << 16);
};
template <>
struct AWCfg<kFp8> {
  static constexpr int kRowBytes = 128;
  static constexpr int kStages = 6;
  static constexpr uint32_t kIdQK = instr_desc(0u, kLanes, kTok);                // e4m3
  static constexpr uint32_t kIdQKLow = kIdQK | (1u << 7);                        // e5m2 by e4m3
  static constexpr uint32_t kIdPV = instr_desc(0u, kLanes, kDim) | (1u << 16);   // f16
};

template <int KF, int F>
struct AWLayout {
  static constexpr int NS = AWCfg<KF>::kStages;
  // Whether the softmax groups take registers from the other warps: 200 and more
  // instead of 168.  128 rows (64 scores a lane) 76 -> 67 us on 8 x 64K bf16, e4m3
  // 169 -> 162 on 16 x 131K; without it 64 rows of bf16 are 1% faster.
  static constexpr bool kSplitRegs = KF == kFp8 || F == 1;
  // two softmax groups; producer, issuer (and two idle warps: whole warpgroups)
  static constexpr int kThreads = kSplitRegs ? 384 : 320;
  static constexpr int kTile = kTok * AWCfg<KF>::kRowBytes;  // keys or values of a page
  static constexpr int kV16 = KF == kFp8 ? kTok * 256 : 0;   // decoded values, two a group
  static constexpr int kScale = KF == kFp8 ? kTok * 4 : 0;
  static constexpr int kV16Off = NS * 2 * kTile;
  static constexpr int kScaleOff = kV16Off + 4 * kV16;
  static constexpr int kBitsOff = kScaleOff + NS * 2 * kScale;     // block bits while lists are joined
  static constexpr int kMlOff = kBitsOff + 2 * kMaxBlockWords * 4;  // (max, sum, output unit) of each lane
  static constexpr int kInfoOff = kMlOff + 2 * kLanes * 16;         // valid tokens of each stage
  // full_k full_v empty_k empty_v [NS], s_full p_full pv_done s_free [2], q_full, stall, drain
  static constexpr int kBarOff = (kInfoOff + NS * 4 + 7) & ~7;
  static constexpr int kNumBars = 4 * NS + 11;
  static constexpr int kCtlOff = kBarOff + kNumBars * 8;       // flags, count, abort, tmem
  static constexpr int kPreOff = (kCtlOff + 16 + kThreads / 32 * 4 + 15) & ~15;   // and one int a warp
  static constexpr int kListOff = kPreOff + kRequestsBytes;
  static constexpr int kBytes = kListOff + kMaxList * 4;
  static constexpr int kSmem = kBytes + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kV16Off % 1024 == 0, "operand tiles on 1024 bytes");
};

// Shared-memory descriptor of an operand whose rows run along M or N: the
// 128-byte swizzle, rows of 128 bytes (64 16-bit elements of the MN extent, one
// row per K index), 8-row atoms of 1024 bytes along K; `lead` bytes to the next
// 64 elements of MN.
__device__ __forceinline__ uint64_t desc_mnmajor_sw128(uint32_t saddr, uint32_t lead) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lead >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// D (+)= A[tensor memory] * B[shared memory], the whole warp, one elected lane.
__device__ __forceinline__ void mma_ts_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts_f8(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// N consecutive 32-bit columns of the warp's 32 lanes, to and from registers.
template <int N>
__device__ __forceinline__ void tm_ld(uint32_t taddr, uint32_t* v) {
  if constexpr (N == 32) {
    uint32_t(&r)[32] = *reinterpret_cast<uint32_t(*)[32]>(v);
    tc_ld_32cols(taddr, r);
  } else {
    static_assert(N == 16, "16 or 32 columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
  }
}
template <int N>
__device__ __forceinline__ void tm_st(uint32_t taddr, const uint32_t* v) {
  if constexpr (N == 32) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
        "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
        "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15])
        : "memory");
  } else {
    static_assert(N == 8, "8, 16 or 32 columns");
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
        : "memory");
  }
}
__device__ __forceinline__ void tm_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void group_sync() {   // the two softmax groups
  asm volatile("bar.sync 1, 256;" ::: "memory");
}

// F lanes a row (128 / F rows of a group, or fewer).
template <int KF, int F, bool kBlocks>
__global__ void __launch_bounds__(AWLayout<KF, F>::kThreads, 1)
    attn_wide_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map) {
  using L = AWLayout<KF, F>;
  constexpr int NS = L::NS;
  constexpr int kPart = kTok / F;      // tokens of a lane
  constexpr int kWarpRows = 32 / F;    // rows of a softmax warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  unsigned int* ctl = reinterpret_cast<unsigned int*>(smem + L::kCtlOff);  // flags, count, abort, tmem
  volatile unsigned int* abort_flag = ctl + 2;
  const Requests rq = requests_at(smem + L::kPreOff);
  uint32_t* list = reinterpret_cast<uint32_t*>(smem + L::kListOff);
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem + L::kBitsOff);
  float4* ml = reinterpret_cast<float4*>(smem + L::kMlOff);
  volatile int* info = reinterpret_cast<volatile int*>(smem + L::kInfoOff);
  const uint32_t bars = sbase + L::kBarOff;
  auto full_k = [&](int s) { return bars + 8 * s; };
  auto full_v = [&](int s) { return bars + 8 * (NS + s); };
  auto empty_k = [&](int s) { return bars + 8 * (2 * NS + s); };
  auto empty_v = [&](int s) { return bars + 8 * (3 * NS + s); };
  auto s_full = [&](int g) { return bars + 8 * (4 * NS + g); };
  auto p_full = [&](int g) { return bars + 8 * (4 * NS + 2 + g); };
  auto pv_done = [&](int g) { return bars + 8 * (4 * NS + 4 + g); };
  auto s_free = [&](int g) { return bars + 8 * (4 * NS + 6 + g); };
  const uint32_t q_full = bars + 8 * (4 * NS + 8), stall_bar = q_full + 8, drain = q_full + 16;
  auto k_tile = [&](int s) { return sbase + s * 2 * L::kTile; };
  auto v_tile = [&](int s) { return sbase + s * 2 * L::kTile + L::kTile; };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(full_k(s), 1);
      mbar_init(full_v(s), 1);
      mbar_init(empty_k(s), 1);
      mbar_init(empty_v(s), KF == kFp8 ? 4 : 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(s_full(g), 1);
      mbar_init(p_full(g), kLanes);
      mbar_init(pv_done(g), 1);
      mbar_init(s_free(g), 4);
    }
    mbar_init(q_full, 2 * kLanes);
    mbar_init(stall_bar, 1);
    mbar_init(drain, 1);
    fence_barrier_init();
    *abort_flag = 0;
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
  }
  if (warp == 9) {
    tmem_alloc(sbase + L::kCtlOff + 12, kCols);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  build_requests<kTok, kBlocks, true>(a, rq, reinterpret_cast<int*>(ctl + 4), ctl);
  tc_fence_after();
  const uint32_t tmem = ctl[3];

  const int W = rq.pre[a.R] * (int)a.by_per.d;
  // no CTA takes less than about four pages
  const int C = min((W + kLeastWide - 1) / kLeastWide, (int)gridDim.x);
  const int c = blockIdx.x;
  const int begin = c < C ? W * c / C : 0, end = c < C ? W * (c + 1) / C : 0;
  SplitRecord record = {-1, 0};

  // A bounded wait of a whole warp; false once any role has given up.
  bool dead = false;
  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    if (dead) return false;
    bool ok = mbar_try_wait(bar, parity);
    const uint64_t t0 = ok ? 0 : global_timer_ns();
    for (uint32_t it = 0; !ok; ++it) {
      ok = mbar_try_wait(bar, parity);
      if (ok) break;
      if (it < 64u || (it & 63u) == 63u) {
        if (*abort_flag) break;
        if (global_timer_ns() - t0 > a.wait_ns) {
          atomicOr(ctl, kErrTimeout);
          *abort_flag = 1;
          break;
        }
      }
    }
    dead = !__all_sync(0xffffffffu, ok);   // a warp goes on, or stops, as one
    return !dead;
  };

  int sent_k = 0, sent_v = 0;   // pages whose copies the producer has asked for
  int tile0 = 0;            // pages of the CTA's earlier segments (producer, issuer, groups)
  int segs = 0;             // segments with pages so far
  int cnt0 = 0, cnt1 = 0;   // pages of group 0 / 1 so far
  Walk walk;
  walk.begin(a, rq.pre, begin, end);
  // The walk over the CTA's stretches, once for the softmax groups and once for the
  // others: two copies of the code, each within its warps' registers.
  auto work = [&](auto softmax) {
    while (walk.more()) {
      const Segment s = walk.next(a, rq.pre);
      if (!s.live) continue;
      const int row_first = s.group * a.group_rows;
      const int nrows = min(a.group_rows, a.P * a.nq - row_first);
      const int p0 = a.by_nq.div(row_first);
      int n_items = 0;
      if (kBlocks) {
        __syncthreads();      // every role is done with the last unit's list
        n_items = 2 * join_lists(a, rq, s, p0, (row_first + nrows - 1) / a.nq, list, bits, threadIdx.x,
                                 blockDim.x, []() { __syncthreads(); });
      }
      const Items it = make_items<kTok, kBlocks>(a, rq, s, n_items);
      // the second page of a request's last block may not exist
      int i1 = it.i1;
      if (kBlocks && i1 == n_items && n_items > 0 &&
          (int)(list[n_items / 2 - 1] & 0xffffu) * kBlock + kPage >= it.glen)
        --i1;
      const int n = max(0, i1 - it.i0);

      if constexpr (!softmax.value) {
      if (warp == 8) {
        // ---- producer ---------------------------------------------------------
        // page ids 32 items at a time, one a lane
        auto page_of = [&](int i) {
          int tb = 0, pg = -1;
          uint32_t m;
          if (i < i1 && item_tokens<kTok, kBlocks>(it, list, i, tb, m))
            pg = __ldg(a.page_table + (size_t)it.slot * a.max_pages + tb / kPage);
          if (i < i1 && (pg < 0 || pg >= a.num_pages)) {
            atomicOr(ctl, kErrBadPage);
            pg = -1;
          }
          return pg;
        };
        int next_ids = dead ? -1 : page_of(it.i0 + lane), ids = -1;
        for (int b = 0; b < n && !dead; ++b) {
          if ((b & 31) == 0) {
            ids = next_ids;
            next_ids = page_of(it.i0 + b + 32 + lane);
          }
          const int pg = __shfl_sync(0xffffffffu, ids, b & 31);
          const int tile = tile0 + b, st = tile % NS;
          const uint32_t ph = (uint32_t)((tile / NS) & 1) ^ 1u;
          int tb = 0;
          uint32_t m;
          item_tokens<kTok, kBlocks>(it, list, it.i0 + b, tb, m);
          const int row = (pg * a.kv_heads + it.kv_head) * kPage;
          if (!wait(empty_k(st), ph)) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(full_k(st), pg < 0 ? 0 : L::kTile);
            if (pg >= 0) {
              tma_load_2d(k_tile(st), &k_map, 0, row, full_k(st));
              if (KF == kBf16) tma_load_2d(k_tile(st) + L::kTile / 2, &k_map, 64, row, full_k(st));
            }
          }
          ++sent_k;
          if (!wait(empty_v(st), ph)) break;
          if (lane == 0) {
            info[st] = pg < 0 ? 0 : min(kTok, it.glen - tb);
            // both planes' scales come with the values: the group reads them, and
            // it gives the values' stage back itself
            mbar_arrive_expect_tx(full_v(st), pg < 0 ? 0 : L::kTile + 2 * L::kScale);
            if (pg >= 0) {
              tma_load_2d(v_tile(st), &v_map, 0, row, full_v(st));
              if (KF == kBf16) {
                tma_load_2d(v_tile(st) + L::kTile / 2, &v_map, 64, row, full_v(st));
              } else {
                const uint32_t sc = sbase + L::kScaleOff + st * 2 * L::kScale;
                bulk_load(sc, a.k_scale + row, L::kScale, full_v(st));
                bulk_load(sc + L::kScale, a.v_scale + row, L::kScale, full_v(st));
              }
            }
          }
          ++sent_v;
          __syncwarp();
        }
      } else if (warp == 9) {
        // ---- product issuer -----------------------------------------------------
        constexpr uint32_t kIdQK = AWCfg<KF>::kIdQK, kIdPV = AWCfg<KF>::kIdPV;
        auto qk = [&](int b) -> bool {
          const int tile = tile0 + b, st = tile % NS, g = b & 1;
          if (!wait(full_k(st), (uint32_t)((tile / NS) & 1))) return false;
          tc_fence_after();
          const uint32_t d = tmem + kColS + 64 * g;
          if (KF == kBf16) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_ts_f16(d, tmem + kColQ + ks * 8,
                         desc_kmajor_sw128(k_tile(st) + (ks >> 2) * (L::kTile / 2) + (ks & 3) * 32),
                         kIdQK, ks > 0);
          } else {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)   // the query's two terms, four steps of 32 each
              mma_ts_f8(d, tmem + kColQ + ks * 8, desc_kmajor_sw128(k_tile(st) + (ks & 3) * 32),
                        ks < 4 ? kIdQK : AWCfg<kFp8>::kIdQKLow, ks > 0);
          }
          tc_commit_warp(empty_k(st));
          tc_commit_warp(s_full(g));
          return true;
        };
        bool ok = n > 0 && !dead;
        if (ok && a.stall_test && segs == 0) ok = wait(stall_bar, 0);
        ok = ok && wait(q_full, (uint32_t)(segs & 1));
        tc_fence_after();
        ok = ok && qk(0);
        if (n > 1) ok = ok && qk(1);
        int k0 = cnt0, k1 = cnt1;
        for (int b = 0; b < n && ok; ++b) {
          const int tile = tile0 + b, st = tile % NS, g = b & 1;
          const int cnt = g ? k1++ : k0++;
          const uint32_t ph = (uint32_t)(cnt & 1);
          // e4m3: the group's next scores as soon as it has read these
          if (KF == kFp8 && b + 2 < n) ok = wait(s_free(g), ph) && qk(b + 2);
          ok = ok && wait(p_full(g), ph) && (KF == kFp8 || wait(full_v(st), (uint32_t)((tile / NS) & 1)));
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + kColO + kDim * g;
          const uint32_t p = tmem + (KF == kBf16 ? kColS + 64 * g : kColP + 32 * g);
          const uint32_t v = KF == kBf16 ? v_tile(st) : sbase + L::kV16Off + (2 * g + (cnt & 1)) * L::kV16;
#pragma unroll
          for (int ks = 0; ks < kTok / 16; ++ks) {
            const uint64_t vd = desc_mnmajor_sw128(v + ks * 2048, kTok * 128);
            mma_ts_f16(d, p + ks * 8, vd, kIdPV, b >= 2 || ks > 0);
            if (KF == kBf16) mma_ts_f16(d, p + 32 + ks * 8, vd, kIdPV, 1);
          }
          if (KF == kBf16) tc_commit_warp(empty_v(st));
          tc_commit_warp(pv_done(g));
          if (KF == kBf16 && b + 2 < n) ok = qk(b + 2);
        }
      }
      } else {
        // ---- softmax group g: pages g, g + 2, ... ------------------------------
        const int g = warp >> 2, quad = warp & 3;
        const int part = lane / kWarpRows;
        const int row = quad * kWarpRows + lane % kWarpRows;   // of the group
        const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);
        const bool live = row < nrows;
        const int pk = row_first + (live ? row : 0), p = a.by_nq.div(pk);
        const size_t q_row = ((size_t)s.r * a.P + p) * a.q_heads + s.head * a.nq + (pk - p * a.nq);
        const bool pad = it.slot < 0 || it.slot >= a.n_slots;
        const int len = live && !pad ? row_len(a, s.r, p) : 0;
        const int bit = p - p0;
        float post = a.scale_log2;
        if (n > 0) {
          // the lane's query row into tensor memory, either group half of it
          const uint4* qp = reinterpret_cast<const uint4*>(a.q + q_row * kDim);
          auto words = [&](int first, int e) {
            return live ? __ldg(qp + first + e) : make_uint4(0, 0, 0, 0);
          };
          if constexpr (KF == kBf16) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint4 u = words(8 * g, e);
              w[4 * e] = u.x, w[4 * e + 1] = u.y, w[4 * e + 2] = u.z, w[4 * e + 3] = u.w;
            }
            tm_st<32>(tl + kColQ + 32 * g, w);
          } else {
            // scaled by a power of two that brings the row's largest magnitude into
            // [2^7, 2^8), then an e4m3 and an e5m2 term: the group's half first, then the other,
            // of which it needs the magnitude only
            uint32_t w[32];
            float amax = 0.f;
            {
              float top[4] = {0.f, 0.f, 0.f, 0.f};
              uint4 other[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint4 u = words(8 * g, e);
                w[4 * e] = u.x, w[4 * e + 1] = u.y, w[4 * e + 2] = u.z, w[4 * e + 3] = u.w;
              }
#pragma unroll
              for (int e = 0; e < 8; ++e) other[e] = words(8 - 8 * g, e);
              auto largest = [&](float t, uint32_t x) { return fmaxf(t, fmaxf(fabsf(bf16_lo(x)), fabsf(bf16_hi(x)))); };
#pragma unroll
              for (int e = 0; e < 8; ++e) {
#pragma unroll
                for (int k = 0; k < 4; ++k) top[k] = largest(top[k], w[4 * e + k]);
                top[0] = largest(top[0], other[e].x), top[1] = largest(top[1], other[e].y);
                top[2] = largest(top[2], other[e].z), top[3] = largest(top[3], other[e].w);
              }
              amax = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
            }
            const int ex = to_2_7(amax);
            const float up = ldexpf(1.f, ex);
            post = fmaxf(post * ldexpf(1.f, -ex), kLeastPost);
            uint32_t lo[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x[4] = {bf16_lo(w[2 * e]) * up, bf16_hi(w[2 * e]) * up, bf16_lo(w[2 * e + 1]) * up,
                            bf16_hi(w[2 * e + 1]) * up};
              w[e] = e4m3x4_take(x);
              lo[e] = e5m2x4(x);
            }
            tm_st<16>(tl + kColQ + 16 * g, w);
            tm_st<16>(tl + kColQ + 32 + 16 * g, lo);
          }
          tm_wait_st();
          tc_fence_before();
          mbar_arrive(q_full);
        }
        float m = -INFINITY, l = 0.f;
        float unit = -INFINITY;   // e4m3: the output is held in units of 2^unit
        int cnt = g ? cnt1 : cnt0;
        const uint32_t sp = tl + kColS + 64 * g, oc = tl + kColO + kDim * g;
        const uint32_t pp = KF == kBf16 ? sp : tl + kColP + 32 * g;
        for (int b = g; b < n; b += 2, ++cnt) {
          const int tile = tile0 + b, st = tile % NS;
          int tb;
          uint32_t members;
          item_tokens<kTok, kBlocks>(it, list, it.i0 + b, tb, members);
          if (!wait(full_v(st), (uint32_t)((tile / NS) & 1))) break;
          const int valid = info[st];
          if (KF == kFp8) {
            // this page's values as f16, rows past the request's tokens as zeros, in
            // the buffer of the group's page before the last (whose product has
            // ended: that was waited for before the last page's weights)
            const int t = threadIdx.x & 127;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int k = t + 128 * e, tok = k >> 3, ch = k & 7;   // 16 codes
              uint4 u = *reinterpret_cast<const uint4*>(smem + (v_tile(st) - sbase) + tok * 128 + ((ch ^ (tok & 7)) << 4));
              if (tok >= valid) u = make_uint4(0, 0, 0, 0);
              uint4 x, y;
              e4m3x4_to_f16x2x2(u.x, x.x, x.y);
              e4m3x4_to_f16x2x2(u.y, x.z, x.w);
              e4m3x4_to_f16x2x2(u.z, y.x, y.y);
              e4m3x4_to_f16x2x2(u.w, y.z, y.w);
              // dims 16 ch .. +7 and +8 .. +15: two 16-byte chunks of a 64-dim half
              uint8_t* base = smem + L::kV16Off + (2 * g + (cnt & 1)) * L::kV16 + (ch >> 2) * (kTok * 128) + tok * 128;
              const int c0 = (ch & 3) * 2;
              *reinterpret_cast<uint4*>(base + ((c0 ^ (tok & 7)) << 4)) = x;
              *reinterpret_cast<uint4*>(base + (((c0 + 1) ^ (tok & 7)) << 4)) = y;
            }
          } else if (valid < kTok) {
            // whatever lies past the request's tokens must not meet a weight of zero
            const int t = threadIdx.x & 127;
            for (int k = valid * 16 + t; k < kTok * 16; k += 128) {
              const int tok = k >> 4, ch = k & 15;
              *reinterpret_cast<uint4*>(smem + (v_tile(st) - sbase) + (ch >> 3) * (kTok * 128) + tok * 128 + ((ch & 7) << 4)) =
                  make_uint4(0, 0, 0, 0);
            }
          }
          if (!wait(s_full(g), (uint32_t)(cnt & 1))) break;
          tc_fence_after();
          // the lane's scores
          uint32_t raw[kPart];
          if constexpr (F == 1) {
            tm_ld<32>(sp, raw);
            tm_ld<32>(sp + 32, raw + 32);
            tc_wait_ld();
          } else {
            uint32_t all[F][kPart];
#pragma unroll
            for (int f = 0; f < F; ++f) tm_ld<kPart>(sp + f * kPart, all[f]);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < kPart; ++j) {
              raw[j] = all[0][j];
#pragma unroll
              for (int f = 1; f < F; ++f) raw[j] = part == f ? all[f][j] : raw[j];
            }
          }
          if (KF == kFp8) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_free(g));
          }
          // y: the scores before the row's factor, two tokens at a time
          constexpr int kHalf = kPart / 2;
          float2 y[kHalf];
          const float* ks = reinterpret_cast<const float*>(smem + L::kScaleOff + st * 2 * L::kScale) + part * kPart;
#pragma unroll
          for (int j = 0; j < kHalf; ++j)
            y[j] = make_float2(__uint_as_float(raw[2 * j]), __uint_as_float(raw[2 * j + 1]));
          if (KF == kFp8) {
#pragma unroll
            for (int j = 0; j < kHalf; j += 2) {
              const float4 k4 = *reinterpret_cast<const float4*>(ks + 2 * j);
              y[j] = fmul2_rn(y[j], make_float2(k4.x, k4.y));
              y[j + 1] = fmul2_rn(y[j + 1], make_float2(k4.z, k4.w));
            }
          }
          const bool listed = !kBlocks || ((members >> bit) & 1u);
          const int visible = min(min(len, tb + valid) - tb, listed ? kTok : 0) - part * kPart;
          const bool masked = __any_sync(0xffffffffu, visible < kPart);
          if (masked) {
#pragma unroll
            for (int j = 0; j < kHalf; ++j) {
              if (2 * j >= visible) y[j].x = -INFINITY;
              if (2 * j + 1 >= visible) y[j].y = -INFINITY;
            }
          }
          float t0 = fmaxf(y[0].x, y[0].y), t1 = fmaxf(y[1].x, y[1].y);
#pragma unroll
          for (int j = 2; j < kHalf; j += 2) {
            t0 = fmaxf(t0, fmaxf(y[j].x, y[j].y));
            t1 = fmaxf(t1, fmaxf(y[j + 1].x, y[j + 1].y));
          }
          const float top = fmaxf(t0, t1) * post;   // post is positive: the order is kept
          float shrink = 1.f;     // what the output gathered so far is to be multiplied by
          if (top > m + (m == -INFINITY ? 0.f : kSlack)) {
            shrink = ex2_approx(m - top);
            l *= shrink;
            m = top;
          }
          const float ref = m == -INFINITY ? 0.f : m;
          const float2 pp2 = make_float2(post, post), rr2 = make_float2(-ref, -ref);
          float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
#pragma unroll
          for (int j = 0; j < kHalf; ++j) {
            y[j] = ffma2_rn(y[j], pp2, rr2);
            y[j].x = ex2_approx(y[j].x), y[j].y = ex2_approx(y[j].y);
            if (j & 1) sum1 = fadd2_rn(sum1, y[j]);
            else sum0 = fadd2_rn(sum0, y[j]);
          }
          l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
          if (KF == kFp8) {
            // times the value scales, in the output's unit, which does not move with
            // the maximum (raise_unit; weights are up to 2^8 here)
            shrink = 1.f;
            const float* vs = ks + kTok;
            float2 r[kHalf];
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < kHalf; j += 2) {
              const float4 v4 = *reinterpret_cast<const float4*>(vs + 2 * j);
              r[j] = make_float2(v4.x, v4.y);
              r[j + 1] = make_float2(v4.z, v4.w);
            }
            if (masked) {   // a masked token's scale may be anything
#pragma unroll
              for (int j = 0; j < kHalf; ++j) {
                if (2 * j >= visible) r[j].x = 0.f;
                if (2 * j + 1 >= visible) r[j].y = 0.f;
              }
            }
#pragma unroll
            for (int j = 0; j < kHalf; ++j) most = fmaxf(most, fmaxf(fabsf(r[j].x), fabsf(r[j].y)));
            if (past_unit(most, to_unit(top, unit))) {
              most = 0.f;
#pragma unroll
              for (int j = 0; j < kHalf; ++j)
                most = fmaxf(most, fmaxf(fabsf(y[j].x * r[j].x), fabsf(y[j].y * r[j].y)));
              shrink = raise_unit(most, m, unit);
            }
            const float f = to_unit(m, unit);
#pragma unroll
            for (int j = 0; j < kHalf; ++j) y[j] = fmul2_rn(fmul2_rn(y[j], make_float2(f, f)), r[j]);
          }
          // e4m3: the output is still, and P's columns free, once the last product
          // has ended (bf16: its scores came after that)
          if (KF == kFp8 && cnt > 0 && !wait(pv_done(g), (uint32_t)((cnt - 1) & 1))) break;
          if (KF == kFp8) tc_fence_after();
          if (b >= 2 && __any_sync(0xffffffffu, shrink != 1.f)) {
#pragma unroll
            for (int ch = 0; ch < kDim; ch += 32) {
              uint32_t o[32];
              tm_ld<32>(oc + ch, o);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * shrink);
              tm_st<32>(oc + ch, o);
            }
          }
          // the weights as operand rows: the lane's own tokens, zeros for the others
          uint32_t hi[kHalf], lo[kHalf];
#pragma unroll
          for (int j = 0; j < kHalf; ++j) {
            if (KF == kBf16) {
              hi[j] = pack_bf16(y[j].x, y[j].y);
              lo[j] = pack_bf16(y[j].x - bf16_lo(hi[j]), y[j].y - bf16_hi(hi[j]));
            } else {
              hi[j] = pack_f16(y[j].x, y[j].y);
            }
          }
#pragma unroll
          for (int f = 0; f < F; ++f) {
            uint32_t z[kPart / 2];
#pragma unroll
            for (int j = 0; j < kPart / 2; ++j) z[j] = F == 1 || part == f ? hi[j] : 0u;
            tm_st<kPart / 2>(pp + f * (kPart / 2), z);
            if (KF == kBf16) {
#pragma unroll
              for (int j = 0; j < kPart / 2; ++j) z[j] = F == 1 || part == f ? lo[j] : 0u;
              tm_st<kPart / 2>(pp + 32 + f * (kPart / 2), z);
            }
          }
          tm_wait_st();
          tc_fence_before();
          if (KF == kFp8 || valid < kTok) fence_async();
          mbar_arrive(p_full(g));
          if (KF == kFp8) {
            // codes and scales of the page have been read
            __syncwarp();
            if (lane == 0) mbar_arrive(empty_v(st));
          }
        }
        // ---- the unit's end: the parts and the groups meet ------------------------
        if (!dead && cnt > 0 && !wait(pv_done(g), (uint32_t)((cnt - 1) & 1))) m = -INFINITY;
        tc_fence_after();
        m = not_empty(m, l);
        ml[g * kLanes + quad * 32 + lane] = make_float4(m, l, unit, 0.f);
        group_sync();
        float M = -INFINITY, sum = 0.f;
#pragma unroll
        for (int f = 0; f < 2 * F; ++f)
          M = fmaxf(M, ml[(f / F) * kLanes + quad * 32 + lane % kWarpRows + (f % F) * kWarpRows].x);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int f = 0; f < 2 * F; ++f) {
          const float4 e = ml[(f / F) * kLanes + quad * 32 + lane % kWarpRows + (f % F) * kWarpRows];
          if (e.x != -INFINITY) sum = fmaf(e.y, ex2_approx(e.x - ref), sum);
        }
        // Either group finishes half the dims: its warps see the tensor-memory lanes
        // of both groups' outputs.  A lane without a page has gathered nothing.
        const float4 e0 = ml[quad * 32 + lane], e1 = ml[kLanes + quad * 32 + lane];
        const bool has0 = e0.x != -INFINITY, has1 = e1.x != -INFINITY;
        const float f0 = ex2_approx((KF == kFp8 ? e0.z : e0.x) - ref);
        const float f1 = ex2_approx((KF == kFp8 ? e1.z : e1.x) - ref);
        const bool complete = s.o0 == 0 && s.o1 == s.cap;
        const size_t at = (size_t)(2 * c + (s.o0 == 0 ? 1 : 0)) * a.group_rows + row;
        const float inv = M == -INFINITY ? 0.f : 1.f / sum;
        bool odd = false;
#pragma unroll 1
        for (int ch = g * (kDim / 2); ch < (g + 1) * (kDim / 2); ch += 32) {
          uint32_t o0[32], o1[32];
          tm_ld<32>(tl + kColO + ch, o0);
          tm_ld<32>(tl + kColO + kDim + ch, o1);
          tc_wait_ld();
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            v[e] = (has0 ? __uint_as_float(o0[e]) * f0 : 0.f) + (has1 ? __uint_as_float(o1[e]) * f1 : 0.f);
#pragma unroll
            for (int d = kWarpRows; d < 32; d <<= 1) v[e] += __shfl_xor_sync(0xffffffffu, v[e], d);
            odd |= !isfinite(v[e]);
          }
          if (part == 0 && live) {
            if (complete) {
              uint4* out = reinterpret_cast<uint4*>(a.out + q_row * kDim + ch);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint4 u;
                u.x = pack_bf16(v[8 * e] * inv, v[8 * e + 1] * inv);
                u.y = pack_bf16(v[8 * e + 2] * inv, v[8 * e + 3] * inv);
                u.z = pack_bf16(v[8 * e + 4] * inv, v[8 * e + 5] * inv);
                u.w = pack_bf16(v[8 * e + 6] * inv, v[8 * e + 7] * inv);
                out[e] = u;
              }
            } else {
              float4* out = reinterpret_cast<float4*>(a.part_o + at * kDim + ch);
#pragma unroll
              for (int e = 0; e < 8; ++e) out[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            }
          }
        }
        if (g == 0 && part == 0 && live) {
          if (complete) {
            if (a.lse) a.lse[q_row] = M == -INFINITY ? M : (M + log2f(sum)) * kLn2;
          } else {
            a.part_ml[at] = make_float2(M, sum);
          }
        }
        volatile unsigned int* odd_rows = ctl + 4;   // [group][quad], one bit a lane
        const uint32_t seen = __ballot_sync(0xffffffffu, odd && part == 0 && live);
        if (lane == 0) odd_rows[g * 4 + quad] = seen;
        tc_fence_before();
        group_sync();      // the outputs have been read, the next unit may write them
        // rows that met something not finite: token by token, so that only the
        // rows that see it keep it
        uint32_t todo = g == 0 ? odd_rows[quad] | odd_rows[4 + quad] : 0u;
        while (todo) {
          const int src = __ffs(todo) - 1;
          todo &= todo - 1;
          const int r2 = __shfl_sync(0xffffffffu, row, src);
          const int pk2 = row_first + r2, p2 = a.by_nq.div(pk2);
          const size_t q2 = ((size_t)s.r * a.P + p2) * a.q_heads + s.head * a.nq + (pk2 - p2 * a.nq);
          float m2, l2;
          float4 o2;
          careful_row<KF, kTok, kBlocks>(a, it, list, a.q + q2 * kDim, __shfl_sync(0xffffffffu, len, src),
                                         p2 - p0, lane, m2, l2, o2);
          if (complete) {
            write_row(a, q2, m2, l2, o2, lane);
          } else {
            const size_t at2 = (size_t)(2 * c + (s.o0 == 0 ? 1 : 0)) * a.group_rows + r2;
            if (lane == 0) a.part_ml[at2] = make_float2(m2, l2);
            reinterpret_cast<float4*>(a.part_o + at2 * kDim)[lane] = o2;
          }
        }
      }
      if (s.o0 == 0 && s.o1 != s.cap) {
        record.unit = s.unit;
        record.splits = owner(s.start + s.cap - 1, W, C) - c + 1;
      }
      tile0 += n;
      segs += n > 0;
      cnt0 += (n + 1) / 2;
      cnt1 += n / 2;
    }
  };
  // 384 threads start with 168 registers each (64,512): the last warpgroup needs
  // few, the softmax groups take what it leaves (256 x 208 + 128 x 88 = 64,512)
  if (warp >= 8) {
    if constexpr (L::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    work(std::integral_constant<bool, false>());
  } else {
    if constexpr (L::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    work(std::integral_constant<bool, true>());
  }

  // after a timeout: the copies and products in flight end before the block does
  if (warp == 8 && *abort_flag) {
    __syncwarp();
    for (int k = max(0, sent_k - NS); k < sent_k; ++k)
      (void)mbar_wait_bounded(full_k(k % NS), (uint32_t)((k / NS) & 1), 200000000ull);
    for (int k = max(0, sent_v - NS); k < sent_v; ++k)
      (void)mbar_wait_bounded(full_v(k % NS), (uint32_t)((k / NS) & 1), 200000000ull);
  }
  if (warp == 9) {
    __syncwarp();
    tc_commit_warp(drain);
    (void)mbar_wait_bounded(drain, 0, 200000000ull);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, kCols);
  if (threadIdx.x == 0) {
    a.records[c] = record;
    a.err_bytes[c] = (uint8_t)ctl[0];
    if (c == 0) *a.err_count = gridDim.x;
  }
}

template <int KF, int F, bool kBlocks>
cudaError_t launch_kfb(const AttnArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map,
                       int grid, int dev, cudaStream_t stream) {
  using L = AWLayout<KF, F>;
  static std::atomic<unsigned long long> attr_done{0};
  cudaError_t e = smem_limit_once(attn_wide_kernel<KF, F, kBlocks>, L::kSmem, dev, attr_done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_wide_kernel<KF, F, kBlocks>, grid, L::kThreads, L::kSmem, stream, a, k_map, v_map);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int KF>
cudaError_t launch_kf(const AttnArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map,
                      int grid, int dev, cudaStream_t stream) {
  const int rows = a.P * a.nq < a.group_rows ? a.P * a.nq : a.group_rows;
  const bool blocks = a.block_ids != nullptr;
#define IDX_LAUNCH(F)                                                              \
  (blocks ? launch_kfb<KF, F, true>(a, k_map, v_map, grid, dev, stream)            \
          : launch_kfb<KF, F, false>(a, k_map, v_map, grid, dev, stream))
  // (17 rows at least: launch_attn sends units of up to 16 to the other kernel)
  if (rows <= 32) return IDX_LAUNCH(4);
  if (rows <= 64) return IDX_LAUNCH(2);
  return IDX_LAUNCH(1);
#undef IDX_LAUNCH
}

}  // namespace

cudaError_t launch_attn_wide(int key_format, const AttnArgs& a, const CUtensorMap& k_map,
                             const CUtensorMap& v_map, int grid, int dev, cudaStream_t stream) {
  return key_format == kBf16 ? launch_kf<kBf16>(a, k_map, v_map, grid, dev, stream)
                             : launch_kf<kFp8>(a, k_map, v_map, grid, dev, stream);
}

}  // namespace idx
