/*
 * libidx — packed sparse-attention index scoring + block top-k for GB300 (sm_103a), and the
 * operators of the layer around it: the key-value store, attention over the paged cache or over
 * the chosen blocks (bf16, e4m3 and NVFP4 caches), the residual + RMS norm with an e4m3 result,
 * and the norm, rotation and store of a projection's queries, keys and values.
 *
 * C ABI.  Every pointer named "device" must point to device memory of the current
 * CUDA device; "host" pointers are read before the call returns.  Streams are
 * cudaStream_t values passed as void* (NULL = legacy default stream).  No call
 * below synchronises the host with the device, except the ones marked "syncs".
 *
 * Constants of the format (the pages' workloads):
 *   page = 64 tokens, block = 128 tokens, head dim D = 128, at most 16 packed rows.
 *
 * Pool planes (one index-K pool per layer; ROCm/ATOM #2745, Summary, "Pool and
 * binding": payload and scale kept as separate uint8 planes):
 *   payload: uint8 [num_pages * 64][row_bytes], physical row = page * 64 + t % 64
 *            row_bytes = 256 (bf16 keys, little-endian), 128 (e4m3 codes),
 *            64 (NVFP4: two e2m1 codes per byte, even element in the low nibble)
 *   scale:   uint8 [num_pages * 64][scale_bytes]
 *            scale_bytes = 0 (bf16: no plane), 4 (fp8: one fp32 per key),
 *            8 (NVFP4: one E4M3 scale per 16 elements, unit outer scale)
 */
#ifndef LIBIDX_IDX_H_
#define LIBIDX_IDX_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define IDX_API __attribute__((visibility("default")))
#else
#define IDX_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

#define IDX_ABI_VERSION 1
#define IDX_PAGE_SIZE 64
#define IDX_BLOCK_SIZE 128
#define IDX_DIM 128
#define IDX_MAX_PACKED_ROWS 16        /* rows of one warp-MMA tile (P*G up to this) */
#define IDX_WIDE_TILE_ROWS 128        /* rows of one tensor-core tile (P*G above 16) */
#define IDX_MAX_ROWS_PER_REQUEST 32768 /* packed_queries * gqa of one request */
#define IDX_MAX_CP_WORLD 8            /* context shards idx_topk_merge accepts */
#define IDX_MAX_TOPK 256
#define IDX_WORKSPACE_HEADER_BYTES 1024
#define IDX_MAX_REQUESTS 2048  /* per idx_score_topk call (draft rows per per-row call) */

typedef enum {
  IDX_BF16 = 0,      /* bfloat16 */
  IDX_FP8_E4M3 = 1,  /* OCP E4M3 ("fn": no infinities, max 448) with fp32 scales */
  IDX_NVFP4 = 2      /* e2m1 payload + E4M3 per-16 scales (keys and values) */
} idx_dtype;

typedef enum {
  IDX_OK = 0,
  IDX_ERR_INVALID = -1,      /* an argument is out of range or a pointer is NULL */
  IDX_ERR_UNSUPPORTED = -2,  /* a dtype combination this library does not implement */
  IDX_ERR_CUDA = -3,         /* a CUDA runtime call or kernel launch failed */
  IDX_ERR_OOM = -4           /* device allocation failed */
} idx_status;

/* Device-side error flags of a call, kept in the workspace header (read them with
 * idx_workspace_errors). */
#define IDX_DEVERR_BAD_PAGE 1u      /* a page id outside [0, num_pages): page not read */
#define IDX_DEVERR_TIMEOUT 2u       /* a pipeline wait gave up (kernel ended early) */
#define IDX_DEVERR_LEN_CLAMPED 4u   /* a row longer than max_pages * 64 was clamped */

/* One index-K pool: payload + scale planes of a paged cache. */
typedef struct idx_pool {
  int32_t dtype;              /* idx_dtype of the keys */
  int32_t page_size;          /* tokens per page: 64 */
  int32_t dim;                /* head dim: 128 */
  int32_t reserved;
  int64_t num_pages;
  void* payload;              /* device, uint8 [num_pages*64][payload_row_bytes] */
  void* scale;                /* device, uint8 [num_pages*64][scale_row_bytes]; NULL for bf16 */
  int64_t payload_row_bytes;  /* 256 | 128 | 64 */
  int64_t scale_row_bytes;    /* 0 | 4 | 8 */
} idx_pool;

/* Library / status helpers. */
IDX_API int idx_abi_version(void);
IDX_API const char* idx_status_string(int status);
/* Text of the last error raised on the calling host thread ("" if none). */
IDX_API const char* idx_last_error(void);

/*
 * idx_pool_alloc — allocate the planes of a paged index-K pool on the current device.
 * The pool layout is the one the ATOM NVFP4 index cache page describes (ROCm/ATOM
 * #2745, Summary): 72 B per NVFP4 key (64 B payload + 8 B scales), 128 B + 4 B
 * per fp8 key, 256 B per bf16 key.  Contents are uninitialised.
 *   dtype: idx_dtype; num_pages >= 1; page_size must be 64; dim must be 128.
 *   out (host): filled on success; the library owns the planes until idx_pool_free.
 * Returns IDX_ERR_INVALID for bad arguments, IDX_ERR_OOM if cudaMalloc fails.
 */
IDX_API int idx_pool_alloc(int dtype, int64_t num_pages, int page_size, int dim, idx_pool* out);

/* idx_pool_free — release planes made by idx_pool_alloc (syncs with the device
 * through cudaFree).  Zeroes *pool.  A pool whose planes the caller allocated must
 * not be passed here. */
IDX_API int idx_pool_free(idx_pool* pool);

/*
 * idx_store_nvfp4 — quantise staged bf16 keys to NVFP4 and write them into the pool
 * at their real slots (ROCm/ATOM #2745, Summary: "Store" and "Write").  Per group of
 * 16 elements: amax in fp32; scale = E4M3(amax / 6) rounded half-to-even, saturating
 * at 448; codes = e2m1(x / scale) with a correctly rounded fp32 division, rounded
 * half-to-even, saturating at 6, sign kept (a negative value rounding to 0 is 0x8);
 * a scale of 0 writes all-zero codes; element 2b goes to the low nibble of byte b.
 * Infinities saturate like any value past 6 * 448.  A NaN is left out of amax and takes the code
 * of 6; only a group of nothing but NaNs has the scale NaN (0x7f).
 *   src_bf16 (device):     bf16 [num_tokens][128], token-major staging buffer.
 *   slot_mapping (device): int64 [num_tokens], physical pool row of each key
 *                          (page * 64 + offset); a negative entry skips the key; an
 *                          entry >= num_pages*64 skips it too.
 *   pool (host):           an NVFP4 pool (caller- or library-allocated planes).
 * Asynchronous on stream.  IDX_ERR_INVALID if pool is not NVFP4 or a pointer is NULL
 * (num_tokens == 0 is a no-op).
 */
IDX_API int idx_store_nvfp4(const void* src_bf16, const int64_t* slot_mapping, int64_t num_tokens,
                    const idx_pool* pool, void* stream);

/*
 * idx_score_topk_workspace_bytes — device scratch idx_score_topk needs: a header of
 * IDX_WORKSPACE_HEADER_BYTES (device error flags) plus one fp32 block score per
 * (request, packed row, block): num_requests * packed_queries * gqa *
 * ceil(max_pages / 2) floats.  When packed_queries * gqa > IDX_MAX_PACKED_ROWS
 * (the 128-row tensor-core path) it adds, from the next 256-byte boundary, 260
 * bytes per packed row: the rows of q converted once per call to f16 (NVFP4
 * keys), and their scales.
 */
IDX_API size_t idx_score_topk_workspace_bytes(int num_requests, int packed_queries, int gqa,
                                      int max_pages);

/*
 * idx_score_topk — the packed index step of one sparse layer (sglang #45451,
 * Modifications; sglang #42614 "[AMD] MiniMax-M3 indexer CP: packed scoring for EAGLE
 * verify rows", Modifications 1).
 *
 * For request r, its P = packed_queries draft rows times G = gqa heads form its
 * packed rows; row i is (draft row i / G, head i % G).  With P*G <= 16 the rows are
 * one 16-row tile, dotted with the request's keys on the warp-level tensor-core MMA
 * with the keys read once per request up to the group's longest row.  With P*G > 16
 * (many draft rows, or a prefill chunk: P query tokens, each its own row length) the
 * rows are cut into tiles of IDX_WIDE_TILE_ROWS, each dotted on the 5th-generation
 * tensor cores (tcgen05) with the keys read once per tile up to the tile's longest
 * row.  Row i then keeps only tokens t < its own length, takes the max score of each
 * 128-token block, always keeps its first init_blocks and last local_blocks blocks
 * (from its own block count), and emits topk block ids with their scores.
 *
 *   q (device):          [R][P][G][128] bf16 (q_dtype IDX_BF16) or e4m3 codes (IDX_FP8_E4M3)
 *   q_scale (device):    fp32 [R][P*G], one scale per packed row; required for e4m3 q,
 *                        ignored (may be NULL) for bf16 q
 *   k_payload, k_scale (device): the pool planes; k_scale is ignored for bf16 keys
 *   k_dtype:             IDX_BF16 (with bf16 q), IDX_FP8_E4M3 (with e4m3 q) or
 *                        IDX_NVFP4 (with bf16 q); other pairs: IDX_ERR_UNSUPPORTED
 *   num_pages:           pages in the pool (page ids outside [0, num_pages) are not
 *                        read and set IDX_DEVERR_BAD_PAGE)
 *   page_table (device): int32 [n_slots][max_pages], page of token t of the request
 *                        in slot s = page_table[s][t / 64]
 *   slot_ids (device):   int32 [R]; a slot outside [0, n_slots) marks a pad request
 *                        (graph padding): nothing is read, all its rows are pads
 *   row_lens (device):   int32 [R][P], tokens of each draft row (its causal length);
 *                        <= 0 gives an all-pad row; > max_pages*64 is clamped
 *   init_blocks, local_blocks >= 0 with init_blocks + local_blocks <= topk
 *   topk:                1 ..IDX_MAX_TOPK
 *   out_ids (device):    int32 [R][P*G][topk]
 *   out_scores (device): fp32 [R][P*G][topk]
 *   workspace (device):  >= idx_score_topk_workspace_bytes(R, P, G, max_pages) bytes,
 *                        256-byte aligned; overwritten by every call (no clearing is
 *                        needed); its header holds the device error flags
 *                        (IDX_DEVERR_*) of the last call and the state of the
 *                        kernel's dynamic work counter, which every call leaves
 *                        ready for the next one (a fresh workspace simply runs
 *                        its first call with a static schedule).  Calls that may
 *                        overlap on the GPU (on different streams, or from
 *                        different host threads without ordering) must not share
 *                        a workspace: they race on its block scores, its error
 *                        flags and the work counter.
 * Output row i of request r: its forced blocks in ascending id order, then the chosen
 * blocks by descending score (ties to the lower id), then (-1, -inf) pads.  Scores are
 * raw q.k block maxima (fp8: code dot products times q_scale times the key's scale).
 * Asynchronous on stream; allocates nothing; capturable in a CUDA graph.
 * Host-side checks return IDX_ERR_INVALID (P*G outside [1, IDX_MAX_ROWS_PER_REQUEST],
 * topk out of range, init+local > topk, NULL pointers, R < 0 or > IDX_MAX_REQUESTS,
 * R * ceil(ceil(P*G / IDX_WIDE_TILE_ROWS) / 2) > IDX_MAX_REQUESTS when P*G > 16, n_slots or
 * max_pages < 1, workspace too
 * small or misaligned, num_pages < 1).  With R == 0 only the workspace is required
 * (its header is reset) and the per-request pointers may be NULL.
 */
IDX_API int idx_score_topk(const void* q, const float* q_scale, int q_dtype,
                   const void* k_payload, const void* k_scale, int k_dtype, int64_t num_pages,
                   const int32_t* page_table, int n_slots, int max_pages,
                   const int32_t* slot_ids, const int32_t* row_lens,
                   int num_requests, int packed_queries, int gqa,
                   int init_blocks, int local_blocks, int topk,
                   int32_t* out_ids, float* out_scores,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * idx_score_topk_lse — idx_score_topk with the log-sum-exp block score in place of the
 * block max (sglang #45451, Accuracy Tests: selected-block scores "max; lse"): a row's
 * score for block b is ln sum exp(q.k_t) over the tokens t of the block inside the row's
 * length (raw dot products, natural log).  Same arguments, outputs, selection rules and
 * workspace; out_scores holds the chosen blocks' log-sum-exp.
 */
IDX_API int idx_score_topk_lse(const void* q, const float* q_scale, int q_dtype,
                               const void* k_payload, const void* k_scale, int k_dtype,
                               int64_t num_pages, const int32_t* page_table, int n_slots,
                               int max_pages, const int32_t* slot_ids, const int32_t* row_lens,
                               int num_requests, int packed_queries, int gqa,
                               int init_blocks, int local_blocks, int topk,
                               int32_t* out_ids, float* out_scores,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * idx_score_local_blocks — the step over one context shard (indexer context
 * parallelism: sglang #42614 "[AMD] MiniMax-M3 indexer CP: packed scoring for EAGLE
 * verify rows", Motivation and Modifications 1, name the per-shard scorer
 * score_local_blocks).  The rank holding the shard calls it; idx_topk_merge then
 * combines every shard's list.
 *
 * The shard is global blocks [block_begin, block_begin + max_pages / 2) of every
 * request: page_table[s][p] is the page of the request's global tokens
 * (2 * block_begin + p) * 64 .. + 63, so max_pages must be even (whole 128-token
 * blocks; a block never straddles two shards).  row_lens, init_blocks,
 * local_blocks and topk are the row's global ones: the forced blocks and the number
 * c of candidates to choose come from the row's own global block count.  Row i of
 * request r gets the shard's forced blocks (ascending, global ids), then its best
 * min(c, candidates in the shard) candidates by score (ties to the lower id), then
 * (-1, -inf) pads.  Packed rows of one 16-row tile only (P*G <= 16).  Other
 * arguments, the workspace (sized for the shard's max_pages) and the error
 * behaviour are those of idx_score_topk; rows longer than the shard are not
 * flagged (IDX_DEVERR_LEN_CLAMPED is for whole-context calls).
 */
IDX_API int idx_score_local_blocks(const void* q, const float* q_scale, int q_dtype,
                                   const void* k_payload, const void* k_scale, int k_dtype,
                                   int64_t num_pages, const int32_t* page_table, int n_slots,
                                   int max_pages, int block_begin, const int32_t* slot_ids,
                                   const int32_t* row_lens, int num_requests,
                                   int packed_queries, int gqa, int init_blocks,
                                   int local_blocks, int topk, int32_t* out_ids,
                                   float* out_scores, void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * idx_topk_merge — the exchange step's re-selection: combine the lists of `world`
 * context shards into each row's global selection.
 *
 *   cand_ids, cand_scores (device): int32 / fp32 [world][R][P*G][topk], shard w's
 *                        idx_score_local_blocks output (any order of shards); the
 *                        shards must partition every row's blocks
 *   slot_ids, row_lens (device): as for idx_score_topk (global lengths; a slot
 *                        outside [0, n_slots) makes the request's rows pads)
 *   out_ids, out_scores (device): int32 / fp32 [R][P*G][topk]
 * Row i gets its forced blocks ascending with the score their shard reported, then
 * the best c of all the shards' other entries (score desc, ties to the lower id),
 * then (-1, -inf) pads: the same as idx_score_topk over the whole context, since
 * each shard keeps its best c candidates.  Host checks return IDX_ERR_INVALID
 * (world outside [1, IDX_MAX_CP_WORLD], R outside [0, IDX_MAX_REQUESTS], P*G out of
 * range, topk or init/local out of range, n_slots < 1, NULL pointers).
 * Asynchronous on stream; allocates nothing.
 */
IDX_API int idx_topk_merge(const int32_t* cand_ids, const float* cand_scores, int world,
                           const int32_t* slot_ids, const int32_t* row_lens, int n_slots,
                           int num_requests, int packed_queries, int gqa, int init_blocks,
                           int local_blocks, int topk, int32_t* out_ids, float* out_scores,
                           void* stream);

/*
 * idx_score_topk_perrow — the same step with every draft row scored as its own decode
 * row (the per-row kernel the packed one replaces: sglang #45451, Motivation; sglang
 * #42614, Motivation): the tile holds G live rows and each request's keys are read
 * once per draft row.  Same arguments, same outputs, same workspace size; an internal
 * ablation of the packed kernel.
 */
IDX_API int idx_score_topk_perrow(const void* q, const float* q_scale, int q_dtype,
                          const void* k_payload, const void* k_scale, int k_dtype,
                          int64_t num_pages, const int32_t* page_table, int n_slots,
                          int max_pages, const int32_t* slot_ids, const int32_t* row_lens,
                          int num_requests, int packed_queries, int gqa,
                          int init_blocks, int local_blocks, int topk,
                          int32_t* out_ids, float* out_scores,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * Key-value cache of an attention layer: two planes (keys, values) of the pool layout
 * above with kv_heads heads.  Page p of head h is head page p * kv_heads + h, so token
 * t of head h of a page lies in plane row (page * kv_heads + h) * 64 + t % 64 and each
 * head page is one contiguous tile; an idx_pool of num_pages * kv_heads pages holds one
 * plane, and with one head the layout is an index pool's.  bf16, e4m3 and NVFP4 planes.
 *
 * An NVFP4 plane's values are code * scale * outer, with one outer scale for the plane: a power
 * of two in [IDX_MIN_OUTER, IDX_MAX_OUTER] that the caller keeps and hands to every call.  With 1
 * the plane is an NVFP4 index pool's.  A group's scale has E4M3's range, 2^-9 to 448 with three
 * bits from 2^-6 on, so an outer scale is well chosen if the groups' largest magnitudes lie in
 * [2^-3, 2688] times it.
 */
#define IDX_MIN_OUTER 5.42101086242752217e-20f /* 2^-64 */
#define IDX_MAX_OUTER 1.8446744073709551616e19f /* 2^64 */


/*
 * idx_store_kv — write new keys (and values) into the cache.  bf16 planes take the bits;
 * e4m3 planes take, per row of 128, a = max(max |x|, 2^-96), scale = a / 448 and codes
 * e4m3(x * (448 * (1 / a))), each quotient and product rounded once in fp32, the code half
 * to even and saturating.  A NaN makes its row's scale and codes NaN.
 *   k_src, v_src (device): bf16 [num_tokens][kv_heads][128], k_stride / v_stride elements
 *                          between tokens (a slice of a fused projection is fine): multiples
 *                          of 8, 16-byte aligned.  v_src NULL with v_pool NULL: keys only
 *                          (an index pool's bf16 or e4m3 keys, with kv_heads = 1).
 *   slot_mapping (device): int64 [num_tokens], page * 64 + offset of each token; negative or
 *                          >= num_pages * 64 skips the token.  Slots must differ: the row
 *                          of two tokens with one slot may hold parts of both, such as the
 *                          codes of one under the scale of the other.
 *   k_pool, v_pool (host): planes of num_pages * kv_heads head pages, the same dtype.
 * Asynchronous on stream; allocates nothing; capturable.  IDX_ERR_INVALID for arguments out of range;
 * IDX_ERR_UNSUPPORTED for an NVFP4 pool (idx_store_kv_nvfp4 writes those).  num_tokens == 0 is
 * a no-op.
 */
IDX_API int idx_store_kv(const void* k_src, const void* v_src, int64_t k_stride, int64_t v_stride,
                         const int64_t* slot_mapping, int64_t num_tokens, int kv_heads,
                         const idx_pool* k_pool, const idx_pool* v_pool, void* stream);

/*
 * idx_store_kv_nvfp4 — idx_store_kv into NVFP4 planes.  Per group of 16 elements y = x / outer:
 * scale = E4M3(max |y| / 6), half to even, at most 448; codes e2m1(y / scale), half to even,
 * saturating at 6, the sign kept; a scale of 0 gives codes of 0.  An infinity is held as the
 * largest value, 6 * 448 * outer, of its sign.  With an outer scale of 1 the bytes are
 * idx_store_nvfp4's, but for groups with a NaN: here its scale is NaN (0x7f, codes 0), so that
 * the attention's rows that see it are NaN.
 *   k_pool, v_pool (host): NVFP4 planes (IDX_ERR_UNSUPPORTED for others), the scale planes 8-byte
 *                          aligned
 *   k_outer, v_outer:      the planes' outer scales (v_outer is checked without values too)
 * Everything else as for idx_store_kv.
 */
IDX_API int idx_store_kv_nvfp4(const void* k_src, const void* v_src, int64_t k_stride,
                               int64_t v_stride, const int64_t* slot_mapping, int64_t num_tokens,
                               int kv_heads, const idx_pool* k_pool, const idx_pool* v_pool,
                               float k_outer, float v_outer, void* stream);

/* The rotation of idx_norm_rope_store. */
#define IDX_MAX_ROPE_AXES 4
typedef struct idx_rope {
  const float* table;         /* device, fp32 [num_positions][rotary_dim], 16-byte aligned: the
                                 cosines of a position's rotary_dim / 2 pairs, then their sines */
  int64_t num_positions;      /* 1 .. 2^31 - 1 */
  const int32_t* positions;   /* device, int32 [axes][num_tokens]: a token's position on each axis */
  int32_t axes;               /* 1 .. IDX_MAX_ROPE_AXES: 1 for text; time, height, width for video */
  int32_t rotary_dim;         /* elements of a head that are rotated, the first ones: a multiple
                                 of 16 up to 128 */
  int32_t interleaved;        /* 0: pair i is elements (i, i + rotary_dim / 2); else (2i, 2i + 1) */
  int32_t reserved;
  uint8_t pair_axis[64];      /* the axis that pair i goes by, below axes (not read with one axis) */
} idx_rope;

/*
 * idx_norm_rope_store — from a layer's projection to where its attention takes its operands from,
 * in one pass: the root-mean-square norm of the queries and keys, head by head, their rotation by
 * position, and the store of the keys and values.  In fp32, per token and head of 128 elements:
 *   y = x / sqrt(mean(x^2) + eps) * weight     (queries, keys; a NULL weight: y = x)
 *   pair (a, b) = pair i of y's first rotary_dim elements, p = the token's position on the pair's
 *   axis: (a cos - b sin, b cos + a sin) with cos = table[p][i], sin = table[p][rotary_dim/2 + i]
 * The queries go to out_q, the keys to k_pool as idx_store_kv or idx_store_kv_nvfp4 would
 * write them if they took fp32 (one rounding; an NVFP4 code may be that of the neighbour where
 * y / scale lies within two fp32 steps of the border), the values, unchanged, to v_pool, in the
 * bytes of those calls.
 *   q, k, v (device):    bf16 [num_tokens][heads][128], q_stride, k_stride, v_stride elements
 *                        between tokens: multiples of 8, 16-byte aligned.  q NULL with out_q NULL
 *                        and q_heads 0: keys only.  v NULL with v_pool NULL: no values (index keys)
 *   q_weight, k_weight (device): bf16 [128], 16-byte aligned, or NULL: no norm of that part
 *   rope (host):         the rotation; NULL: none.  A position outside [0, num_positions) turns the
 *                        elements that go by it into NaN (and with them an e4m3 row, an NVFP4 group)
 *   slot_mapping:        as for idx_store_kv: a token that is skipped has its queries computed
 *   out_q (device):      bf16 [num_tokens][q_heads][128]; with out_q_scale (device, fp32
 *                        [num_tokens][q_heads]) e4m3 codes by idx_store_kv's rule, a query of
 *                        idx_score_topk
 *   k_pool, v_pool (host), k_outer, v_outer: bf16, e4m3 (outer scales 1) or NVFP4 planes
 * out_q must not overlap the projection.  Asynchronous on stream; allocates nothing; capturable.
 * num_tokens == 0 is a no-op.
 */
IDX_API int idx_norm_rope_store(const void* q, int64_t q_stride, int q_heads, const void* k,
                                int64_t k_stride, const void* v, int64_t v_stride, int kv_heads,
                                const void* q_weight, const void* k_weight, float eps,
                                const idx_rope* rope, const int64_t* slot_mapping,
                                int64_t num_tokens, void* out_q, float* out_q_scale,
                                const idx_pool* k_pool, const idx_pool* v_pool, float k_outer,
                                float v_outer, void* stream);

/*
 * idx_attn_workspace_bytes — device scratch of idx_attn_paged (lists 0) and idx_attn_blocks, and
 * of the same over NVFP4 caches:
 * the header, and the partial results of the units that several CTAs share.  It does not
 * depend on the number of requests or the context.  0 for arguments that do not fit together.
 */
IDX_API size_t idx_attn_workspace_bytes(int packed_queries, int q_heads, int kv_heads, int lists);

/*
 * idx_attn_paged — attention of the newest tokens (one, or P = packed_queries draft rows, a
 * request) over the whole paged cache.  Row (r, p, head) sees the tokens t < row_lens[r][p] of
 * its request: out = softmax(sm_scale * q . k_t) v_t, lse = ln sum exp(sm_scale * q . k_t).
 * The work is split evenly over the GPU along the caches' length and joined in a fixed order.
 *   q (device):          bf16 [R][P][q_heads][128]; query head j goes by key head
 *                        j / (q_heads / kv_heads)
 *   k_payload .. v_scale (device): the planes; scales are fp32 [rows], e4m3 caches only
 *   kv_dtype:            IDX_BF16 or IDX_FP8_E4M3
 *   num_pages:           pages of the cache (a page holds all heads); a page id outside
 *                        [0, num_pages) is not read, its tokens are left out and
 *                        IDX_DEVERR_BAD_PAGE is set
 *   page_table, slot_ids, row_lens: as for idx_score_topk; a pad request or a row of length
 *                        <= 0 gives out = 0, lse = -inf; lengths past max_pages * 64 are
 *                        clamped (IDX_DEVERR_LEN_CLAMPED)
 *   out (device):        bf16 [R][P][q_heads][128];  out_lse (device): fp32 [R][P][q_heads],
 *                        natural log, or NULL.  Partial results over context shards join by
 *                        it: out = sum_w out_w exp(lse_w - lse).
 *   workspace (device):  >= idx_attn_workspace_bytes(P, q_heads, kv_heads, 0), 256-byte
 *                        aligned, no clearing needed; not shared by calls that may overlap.
 *                        idx_workspace_errors reads its flags.
 * What lies in the cache past a row's length (uninitialised pages, NaN) does not reach the row.
 * Sums and softmax statistics are fp32; for the product with the values the weights are
 * held as two bf16 (bf16 cache, 2^-17 of the weight), or weight times value scale as one f16
 * (e4m3 cache): 2^-11 of it, or 2^-28 of the row's largest such product.  With an e4m3 cache a
 * query element more than 2^13 below its row's largest may be off by 2^-21 of the largest.
 * Asynchronous on stream, on the current device, where every pointer has to be; allocates
 * nothing; capturable.  R <= IDX_MAX_REQUESTS, P * q_heads <= IDX_MAX_ROWS_PER_REQUEST, num_pages *
 * kv_heads < 2^31 / 64; q_heads a multiple of kv_heads; requests times key heads (or lists)
 * times groups of 128 rows at most 2^18.
 */
IDX_API int idx_attn_paged(const void* q, const void* k_payload, const void* k_scale,
                           const void* v_payload, const void* v_scale, int kv_dtype,
                           int64_t num_pages, int kv_heads, const int32_t* page_table, int n_slots,
                           int max_pages, const int32_t* slot_ids, const int32_t* row_lens,
                           int num_requests, int packed_queries, int q_heads, float sm_scale,
                           void* out, float* out_lse, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * idx_attn_blocks — the same over the 128-token blocks that the index step chose: row
 * (r, p, head) sees the tokens t < row_lens[r][p] whose block t / 128 is in its list.
 *   block_ids (device):  int32 [R][P][lists][topk], idx_score_topk's out_ids with gqa = lists.
 *                        Query head j goes by list j / (q_heads / lists).  A list is a set: its
 *                        order does not matter, a block listed twice counts once, and ids < 0
 *                        or at or past the row's own blocks are left out.  Ids count from the
 *                        page table's first page: of merged lists a context shard subtracts its
 *                        first block, as it does from the lengths.
 *   lists:               q_heads must be a multiple of it, and lists and kv_heads one a multiple
 *                        of the other;  topk: 1 .. IDX_MAX_TOPK
 * The draft rows of a request that share a list position are packed: their lists are joined,
 * and a block that several of them chose is read once.  Everything else is as above, with the
 * workspace of idx_attn_workspace_bytes(P, q_heads, kv_heads, lists).
 */
IDX_API int idx_attn_blocks(const void* q, const void* k_payload, const void* k_scale,
                            const void* v_payload, const void* v_scale, int kv_dtype,
                            int64_t num_pages, int kv_heads, const int32_t* page_table,
                            int n_slots, int max_pages, const int32_t* slot_ids,
                            const int32_t* row_lens, const int32_t* block_ids, int lists, int topk,
                            int num_requests, int packed_queries, int q_heads, float sm_scale,
                            void* out, float* out_lse, void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * idx_attn_paged_nvfp4, idx_attn_blocks_nvfp4 — the same over NVFP4 planes: k_scale, v_scale
 * (device, 16-byte aligned) are E4M3 bytes [rows][8], k_outer, v_outer the planes' outer scales;
 * sm_scale * k_outer must be a normal fp32 number.  Codes times scales are exact in f16, where the
 * products are taken; a query element is exact within 2^21 of its row's largest; the weights
 * enter the product with the values as one f16: 2^-11 of the weight, or 2^-32 of the row's
 * largest weight.  Short requests are faster under a page table about as wide as the longest of
 * them: max_pages is all that the host knows of the lengths.
 */
IDX_API int idx_attn_paged_nvfp4(const void* q, const void* k_payload, const void* k_scale,
                                 const void* v_payload, const void* v_scale, int64_t num_pages,
                                 int kv_heads, const int32_t* page_table, int n_slots,
                                 int max_pages, const int32_t* slot_ids, const int32_t* row_lens,
                                 int num_requests, int packed_queries, int q_heads, float sm_scale,
                                 float k_outer, float v_outer, void* out, float* out_lse,
                                 void* workspace, size_t workspace_bytes, void* stream);
IDX_API int idx_attn_blocks_nvfp4(const void* q, const void* k_payload, const void* k_scale,
                                  const void* v_payload, const void* v_scale, int64_t num_pages,
                                  int kv_heads, const int32_t* page_table, int n_slots,
                                  int max_pages, const int32_t* slot_ids, const int32_t* row_lens,
                                  const int32_t* block_ids, int lists, int topk, int num_requests,
                                  int packed_queries, int q_heads, float sm_scale, float k_outer,
                                  float v_outer, void* out, float* out_lse, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * idx_add_rmsnorm_fp8 — residual addition, root-mean-square norm, e4m3 result.  Per row, in
 * fp32: h = x + residual; out_residual = bf16(h); y = h / sqrt(mean(h^2) + eps) * weight; then
 * codes and scales of y by idx_store_kv's rule, per group of IDX_NORM_GROUP elements (the last
 * one may be shorter) or per row.
 *   x (device):            bf16 [num_rows][dim], x_stride elements between rows
 *   residual (device):     the same with residual_stride, or NULL: h = x
 *   weight (device):       bf16 [dim];  group: IDX_NORM_GROUP, or 0 for the whole row
 *   out (device):          e4m3 codes [num_rows][dim]
 *   out_scale (device):    fp32 [num_rows][ceil(dim / group)], or [num_rows] with group 0
 *   out_residual (device): bf16 [num_rows][dim], or NULL; may be residual itself (when its
 *                          stride is dim)
 * With dim = 128 and group 0 the result is an e4m3 query or key of idx_score_topk with its
 * scale.  Any dim in [1, IDX_MAX_NORM_DIM] and any alignment of the elements; rows of a
 * multiple of 8 elements on 16-byte boundaries are faster.  Asynchronous on stream; allocates
 * nothing; capturable.  num_rows == 0 is a no-op.
 */
#define IDX_NORM_GROUP 128
#define IDX_MAX_NORM_DIM 32768
IDX_API int idx_add_rmsnorm_fp8(const void* x, int64_t x_stride, const void* residual,
                                int64_t residual_stride, const void* weight, int64_t num_rows,
                                int dim, int group, float eps, void* out, float* out_scale,
                                void* out_residual, void* stream);

/* idx_set_kernel_events — instrumentation for timing.  Arms, for the next
 * idx_score_topk / idx_score_topk_perrow call on the calling host thread only, up
 * to three cudaEvent_t (passed as void*, NULL to skip) that the call records on its
 * stream: before the score kernel, after the score kernel, after the top-k kernel.
 * The events are used once and then forgotten. */
IDX_API int idx_set_kernel_events(void* score_begin, void* score_end, void* topk_end);

/* idx_set_kernel_waits — ordering for pipelined callers.  Arms, for the next
 * idx_score_topk / _lse / _perrow / idx_score_local_blocks call on the calling
 * host thread only, up to two cudaEvent_t (passed as void*, NULL to skip) that
 * the call's stream waits for (cudaStreamWaitEvent): before_score before the
 * score kernel is launched, before_topk before the top-k kernel is launched.
 * The events are used once and then forgotten.  What it is for: the score
 * kernel is launched as a programmatic dependent of the kernel before it and
 * starts under it, but a wait placed right before it (a cross-stream event, a
 * captured graph's join) makes it start only after that kernel has finished.
 * A loop that copies step k + 1's inputs on another stream can hand that
 * copy's event to step k's call as before_topk: step k + 1's score kernel reads
 * its inputs only after step k's top-k has completed, which now comes after the
 * copy, and keeps its overlap with step k.  Always returns IDX_OK. */
IDX_API int idx_set_kernel_waits(void* before_score, void* before_topk);

/*
 * idx_score_topk_noalloc — idx_score_topk for callers that cannot allocate device
 * memory.  (The pages have no counterpart: it is an addition of this library.)
 *
 * Who needs it: a caller whose device memory is owned by someone else — a serving
 * engine whose memory pool must account for every byte, a plugin loaded into a host
 * framework with no allocator hook — or a caller that cannot afford the device-wide
 * synchronisation cudaMalloc / cudaFree may cause in the middle of a decode step,
 * has no way to hand idx_score_topk a workspace.  This variant keeps its block-score
 * scratch in a fixed array of IDX_NOALLOC_SCRATCH_BYTES inside the library instead;
 * every GPU that loads the library holds that array until the process exits.
 *
 * Same arguments and outputs as idx_score_topk without the workspace.  The call must
 * need at most IDX_NOALLOC_SCRATCH_BYTES of scratch, i.e.
 *   IDX_WORKSPACE_HEADER_BYTES + num_requests * packed_queries * gqa *
 *   ceil(max_pages / 2) * 4 bytes,
 * otherwise it returns IDX_ERR_INVALID before any device work.  It calls no
 * allocator.  The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current); make that first call before
 * any stream capture.  All calls share the one array and it keeps the last call's
 * contents (each call rewrites what it reads): calls that overlap on
 * the GPU — on different streams, or from different host threads — race on it and
 * must be serialised by the caller.  The device error flags of the last call on
 * the current device are read with idx_noalloc_errors.  If the device's context
 * is torn down and made anew (cudaDeviceReset), the next call looks the address
 * up again.
 */
#define IDX_NOALLOC_SCRATCH_BYTES (16 * 1024 * 1024)
IDX_API int idx_score_topk_noalloc(const void* q, const float* q_scale, int q_dtype,
                                   const void* k_payload, const void* k_scale, int k_dtype,
                                   int64_t num_pages, const int32_t* page_table, int n_slots,
                                   int max_pages, const int32_t* slot_ids,
                                   const int32_t* row_lens, int num_requests, int packed_queries,
                                   int gqa, int init_blocks, int local_blocks, int topk,
                                   int32_t* out_ids, float* out_scores, void* stream);

/* idx_noalloc_errors — the device error flags (IDX_DEVERR_*) of the last
 * idx_score_topk_noalloc call on the current device, read from the fixed scratch
 * array's header (syncs on stream; allocates nothing).  No counterpart on the
 * pages: it is the no-allocation variant's idx_workspace_errors.
 *   flags (host): receives the IDX_DEVERR_* bits. */
IDX_API int idx_noalloc_errors(void* stream, uint32_t* flags);

/* idx_set_wait_limit_ns — limit (nanoseconds, process-wide) of every pipeline wait in
 * the score and attention kernels; 0 restores the default of 2 s.  A wait that runs past it ends
 * its role: the CTA waits for its own copies in flight, frees its tensor memory,
 * sets IDX_DEVERR_TIMEOUT in the workspace header and exits, so the context stays
 * usable.  The limit is read at each call (a captured graph keeps the one of its
 * capture).  Always returns IDX_OK. */
IDX_API int idx_set_wait_limit_ns(uint64_t ns);

/* idx_set_stall_test — diagnostic (process-wide, off by default): with on != 0, in
 * every score CTA one role's first pipeline wait goes to a barrier that nothing
 * completes (the 16-row kernel: warp 0, after issuing its first copies; the
 * tensor-core kernel: the MMA issuer; the attention kernels: warp 0's first piece, and
 * the product issuer), so it runs out after the wait limit and the call ends through the timeout path described above, with IDX_DEVERR_TIMEOUT set.
 * Outputs of such a call are meaningless.  Lets a test exercise failure handling
 * on the GPU without a fault.  Always returns IDX_OK. */
IDX_API int idx_set_stall_test(int on);

/* idx_set_grid_limit — cap the number of CTAs the score kernel launches (process-
 * wide; 0 restores the default of one CTA per SM).  Results do not depend on it:
 * each block max is computed whole by one warp, so any split of the work gives the
 * same bits.  The attention kernels obey it too; there the split decides where partial
 * sums are joined, so their results agree to rounding.  Meant for tests and tuning. */
IDX_API int idx_set_grid_limit(int max_ctas);

/* idx_workspace_errors — read the device error flags of the last call that used this
 * workspace (syncs on stream).  flags (host): receives the IDX_DEVERR_* bits. */
IDX_API int idx_workspace_errors(const void* workspace, void* stream, uint32_t* flags);

#ifdef __cplusplus
}
#endif

#endif /* LIBIDX_IDX_H_ */
