/*
 * hisa.h -- C ABI of the GB300 (sm_103a) HiSA sparse-attention step.
 *
 * The step is the one described on the page "feat(deepseek-v4): implement HiSA
 * hierarchical sparse attention" (cited as [HiSA issue] with its section): score
 * pooled indexer keys, select index_topk pooled rows (flat or hierarchical), gather
 * the selected pooled KV rows and combine them with the local window and the
 * per-head sinks in one split softmax. Beside it stand the operators that a layer runs
 * around the step: hisa_rms_norm, hisa_rope, hisa_norm_rope, for a batch that shares a long
 * prefix hisa_prefix_attend and, for pooled rows kept in pages (bf16 or 4 bits),
 * hisa_cache_append, hisa_cache_read and hisa_cache_attend.
 *
 * Conventions shared by every entry point
 *  - Tensor pointers are DEVICE pointers owned by the caller; tensors are dense,
 *    row-major, with the shapes written beside each argument. The library never
 *    allocates, never frees, never synchronises the stream and keeps no state
 *    between calls (but what the runtime said of the device and of a kernel's occupancy);
 *    it is safe to call from several host threads on different streams with different
 *    workspaces.
 *  - Consecutive calls may overlap, on request: a call whose descriptor sets
 *    HISA_FLAG_CHAINED launches its kernels as programmatic dependents of the
 *    kernel before it on the stream, so it may start while that kernel finishes.
 *    hisa_select_topk then reads q, w, key_off and t0, and hisa_sparse_attend reads
 *    q, local_kv, local_len, local_pos0, kv_off, t0 and sinks before that kernel has
 *    completed; each waits for it before reading top_blk / I and before writing any
 *    output. Set the flag only when the kernel just before the call on the stream is
 *    another libhisa call and none of those early-read inputs is written by it (the
 *    usual chain: hisa_block_filter(_append) -> hisa_select_topk -> hisa_sparse_attend).
 *    With it hisa_rms_norm may read w before that kernel has completed; hisa_rope,
 *    hisa_norm_rope, hisa_prefix_attend and the hisa_cache_* calls take the flag and read
 *    nothing early.
 *    Without the flag (flags = 0) a call's kernels start after the previous work on the
 *    stream has completed, as with any ordinary launch, except kernels that read nothing
 *    before the previous grid has completed (the coarse stage's pipeline, the selects and
 *    merges that follow a call's scoring or combine kernel, and the kernels of
 *    hisa_rms_norm, hisa_rope, hisa_norm_rope, hisa_prefix_attend and the hisa_cache_*
 *    calls), which may always overlap its end.
 *  - Ragged batches: sequence b owns pooled rows [key_off[b], key_off[b+1]) of the
 *    packed key / KV arrays, so Np_b = key_off[b+1] - key_off[b] (int64, device).
 *  - Positions: t0[b] (int32, device) is the absolute token position of query
 *    row 0 of sequence b; row j sits at t = t0[b] + j ([HiSA issue] "Conventions").
 *    The visible pooled prefix is V(t) = min(Np_b, floor((t+1)/r)) ([HiSA issue]
 *    "The pooled stream and positions"). As on the page, the causal pooled mask
 *    is applied only when L > 1; single-row calls treat all Np_b rows as visible.
 *  - Head weights w are the RAW weights_proj(x) outputs (f32); the library applies
 *    H_i^-1/2 * D_i^-1/2 once per head ([HiSA issue] "The indexer query and
 *    per-head weights"). All selection scoring accumulates in f32.
 *  - Selections are sets: entries of I / top_blk are written in ascending id order,
 *    equal scores are broken by ascending id, -0.0 equals +0.0, and rows that have
 *    fewer than k candidates are padded with -1.
 *  - Host validation is synchronous: a bad argument returns HISA_EINVAL /
 *    HISA_EDTYPE / HISA_EWORKSPACE before anything is enqueued. Kernels then run
 *    asynchronously on `stream`; a failed launch returns HISA_ECUDA.
 *  - Data the host cannot see (offsets, ids, per-sequence gates) is checked on the
 *    device. A violation never faults: the kernel skips the access, writes -1 /
 *    NEG where the page defines a neutral value, and ORs a HISA_DEV_* bit into the
 *    status word held in the first 256 bytes of the workspace. Read it with
 *    hisa_device_status(); clear it with hisa_workspace_init().
 *  - Workspace: `ws` is device memory of at least hisa_workspace_bytes(op, desc)
 *    bytes, 256-byte aligned. One workspace sized for the largest op may be shared
 *    by consecutive calls on the same stream.
 */
#ifndef HISA_H
#define HISA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define HISA_API __attribute__((visibility("default")))
#else
#define HISA_API
#endif

struct CUstream_st;                  /* the type behind cudaStream_t */
typedef struct CUstream_st *hisa_stream_t;

typedef enum {
    HISA_OK = 0,
    HISA_EINVAL = -1,     /* bad descriptor field, pointer, alignment or a host-checkable gate */
    HISA_EDTYPE = -2,     /* dtype or shape combination without a kernel */
    HISA_EWORKSPACE = -3, /* workspace missing, misaligned or too small */
    HISA_ECUDA = -4,      /* a CUDA runtime call or a kernel launch failed */
    HISA_EDEVICE = -5     /* hisa_device_status(): a kernel flagged bad data */
} hisa_status;

typedef enum {
    HISA_F32 = 0,
    HISA_BF16 = 1,
    HISA_E4M3 = 2,        /* 8-bit float, 4 exponent bits, largest 448 (out of hisa_rms_norm and hisa_cache_read) */
    HISA_E2M1 = 3         /* rows in 4 bits: 4-bit floats 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, with
                             an e4m3 scale for every 16 of them (the pages of hisa_cache_* only) */
} hisa_dtype;

/* Bits of the device status word. */
#define HISA_DEV_BAD_OFFSETS 0x1u /* offsets not monotone, past keys_rows / means_rows / kv_rows, Np_b > Np_max,
                                    or a capacity too small; the sequence is skipped */
#define HISA_DEV_GATE        0x2u /* a sequence failed Np_b >= index_block*index_keep; rows are -1 */
#define HISA_DEV_BAD_ID      0x4u /* a selected id outside [-1, Np_b) reached the combine; skipped */
#define HISA_DEV_NONFINITE   0x8u /* a select saw a non-finite score */
#define HISA_DEV_BAD_BLOCK   0x10u /* a top_blk entry outside [0, nb_b); that row is written as -1 */
#define HISA_DEV_TIMEOUT     0x20u /* a kernel gave up on a bounded wait; its outputs are incomplete */

/* Bits of hisa_index_desc.flags / hisa_attn_desc.flags (all others must be 0). */
#define HISA_FLAG_CHAINED    0x1u /* may overlap the previous libhisa call on the stream (see above) */

/* Operation ids for hisa_workspace_bytes. */
#define HISA_OP_INDEX_SCORES  0
#define HISA_OP_BLOCK_MEANS   1
#define HISA_OP_BLOCK_FILTER  2
#define HISA_OP_SELECT_TOPK   3
#define HISA_OP_FLAT_TOPK     4
#define HISA_OP_SPARSE_ATTEND 5
#define HISA_OP_COMPRESS      6
#define HISA_OP_PREFIX_ATTEND 7
#define HISA_OP_CACHE         8   /* hisa_cache_append, hisa_cache_read */
#define HISA_OP_CACHE_ATTEND  9

/* Indexer problem ([HiSA issue] "Configuration", "Flat selection", "HiSA decode path"). */
typedef struct {
    int32_t B;            /* sequences (>= 1) */
    int32_t L;            /* query rows per sequence (>= 1; 1 = decode) */
    int32_t H_i;          /* indexer heads, index_n_heads */
    int32_t D_i;          /* indexer head dim, index_head_dim: 32, 64 or 128 */
    int32_t r;            /* compress ratio (>= 1) */
    int32_t index_topk;   /* k: pooled rows kept per query (1..2048) */
    int32_t index_block;  /* b: HiSA block size in pooled rows (0 disables the hierarchy) */
    int32_t index_keep;   /* keep: blocks kept by the coarse stage */
    int64_t Np_max;       /* an upper bound of Np_b over the batch (sizes grids and workspace) */
    int64_t keys_rows;    /* rows allocated in keys (>= key_off[B]); no key read goes past it */
    int64_t means_rows;   /* rows allocated in the block-mean array; no block-mean read or
                             write goes past it (0 for calls that take no means) */
    int32_t q_dtype;      /* hisa_dtype of q: HISA_F32 or HISA_BF16 */
    int32_t k_dtype;      /* hisa_dtype of the pooled indexer keys */
    int32_t flags;        /* HISA_FLAG_* bits (0 = none) */
} hisa_index_desc;

/* Attention problem ([HiSA issue] "Consuming the selection: sparse combine"). */
typedef struct {
    int32_t B, L;         /* sequences, query rows per sequence */
    int32_t H;            /* query heads sharing the single KV head: 8, 16 or 64 */
    int32_t Dh;           /* head dim: 64, 128 or 512 (with H = 8, 16, 64 respectively) */
    int32_t window;       /* sliding window: local row s is visible to t iff 0 <= t-s < window */
    int32_t W_max;        /* rows allocated per sequence in local_kv */
    int32_t r;            /* compress ratio, for V(t) */
    int32_t k;            /* width of I (ignored when I == NULL) */
    int64_t Np_max;       /* an upper bound of Np_b over the batch */
    int64_t kv_rows;      /* rows allocated in pooled_kv (>= kv_off[B]); no read goes past it */
    float scale;          /* softmax scale; <= 0 selects Dh^-1/2 */
    int32_t q_dtype;      /* hisa_dtype of q; must equal kv_dtype */
    int32_t kv_dtype;     /* hisa_dtype of local_kv and pooled_kv */
    int32_t flags;        /* HISA_FLAG_* bits (0 = none) */
    int32_t out_dtype;    /* hisa_dtype of out: HISA_F32 (0, the default) or HISA_BF16, the
                             f32 result rounded to nearest even once, after the combine */
} hisa_attn_desc;

/* The indexer's compressor ([HiSA issue] "The pooled stream and positions", "Configuration":
 * compressor.{wkv, wgate, ape, norm}, compress_rope_theta, qk_rope_head_dim). */
typedef struct {
    int32_t B;            /* sequences (>= 1) */
    int32_t D_i;          /* pooled key dim: 32, 64 or 128 */
    int32_t r;            /* compress ratio: tokens per window (1..128) */
    int32_t overlap;      /* 1: the overlap variant, projections 2*D_i wide (channels [0, D_i) pool
                             the previous window, [D_i, 2*D_i) the row's own window); 0: plain, D_i wide */
    int32_t rope_dims;    /* trailing dims rotated, even, 0..D_i (64) */
    int32_t index_block;  /* b: block size of the block-mean cache (0: no means kept) */
    int32_t n_new_max;    /* an upper bound of n_new[b] (0..1048576) */
    int32_t k_dtype;      /* hisa_dtype of the pooled key cache */
    float rope_theta;     /* RoPE base (> 1): compress_rope_theta = 160000 */
    float eps;            /* RMSNorm epsilon (> 0) */
    int64_t tok_rows;     /* rows allocated in kv and gate */
    int64_t keys_rows;    /* rows allocated in keys; no key read or write goes past it */
    int64_t means_rows;   /* rows allocated in means (0 when means is NULL) */
    int32_t flags;        /* HISA_FLAG_* bits (0 = none) */
} hisa_compress_desc;

/* The norm ahead of a layer's projections: the residual's addition, the root-mean-square
 * norm, and the output in f32, bf16 or in 8 bits with scales (hisa_rms_norm). */
typedef struct {
    int64_t rows;         /* tokens (>= 0; 0 = nothing to do) */
    int32_t cols;         /* hidden size, 1..32768 */
    int32_t x_dtype;      /* hisa_dtype of x: HISA_F32 or HISA_BF16 */
    int32_t res_dtype;    /* hisa_dtype of residual and residual_out: HISA_F32 or HISA_BF16 */
    int32_t out_dtype;    /* hisa_dtype of out: HISA_F32, HISA_BF16 or HISA_E4M3 */
    int32_t scale_group;  /* HISA_E4M3: columns that share a scale: 32, 64, 128 or 256 (a divisor of
                             cols), or 0 for one scale per row; else 0 */
    int32_t scale_pow2;   /* HISA_E4M3: 1 rounds each scale up to a power of two; else 0 */
    float eps;            /* > 0 */
    int32_t flags;        /* HISA_FLAG_* bits (0 = none) */
    int64_t ld_x, ld_res, ld_out; /* elements from one row to the next of x, of residual and
                             residual_out, of out (>= cols; ld_res is ignored without a residual) */
} hisa_norm_desc;

/* The frequencies of rotary positions ([HiSA issue] "Configuration": compress_rope_theta,
 * qk_rope_head_dim), for hisa_rope_table. Pair i of rope_dims / 2 turns by f_i radians per
 * position, f_i = theta^(-2i / rope_dims), scaled for contexts longer than the trained one: */
#define HISA_ROPE_PLAIN  0   /* f_i */
#define HISA_ROPE_LINEAR 1   /* f_i / factor: positions squeezed into the trained range */
#define HISA_ROPE_YARN   2   /* f_i / factor * g_i + f_i * (1 - g_i): the pairs that turn more than
                              * beta_fast times over orig_len positions stay, those that turn fewer
                              * than beta_slow times are squeezed, a ramp linear in i between:
                              * g_i = clamp((i - lo) / max(hi - lo, 0.001), 0, 1), with c(n) =
                              * rope_dims * ln(orig_len / (2 pi n)) / (2 ln theta), lo =
                              * max(floor(c(beta_fast)), 0), hi = min(ceil(c(beta_slow)), rope_dims - 1) */
typedef struct {
    int32_t rope_dims;    /* rotated dims, even, 2..1024 */
    int32_t kind;         /* HISA_ROPE_* */
    double theta;         /* base (> 1) */
    double factor;        /* LINEAR, YARN: > 0 (ignored otherwise) */
    double orig_len;      /* YARN: the trained length (> 0) */
    double beta_fast;     /* YARN: > 0 */
    double beta_slow;     /* YARN: > 0 */
} hisa_rope_scaling;

/* Rotary positions of one or two tensors of heads (hisa_rope), for instance queries and the
 * shared KV row of each token. All strides in elements; heads need not be dense. */
typedef struct {
    int64_t tokens;       /* >= 0 (0 = nothing to do) */
    int32_t heads;        /* heads of x (>= 1) */
    int32_t heads2;       /* heads of x2 (0 = no second tensor) */
    int32_t D;            /* head dim, 2..1024 */
    int32_t rope_dims;    /* rotated dims, even, 2..D */
    int32_t rope_first;   /* first rotated dim, 0..D - rope_dims */
    int32_t half;         /* pairs: 0 = (2i, 2i + 1), interleaved; 1 = (i, i + rope_dims / 2), halves */
    int32_t inverse;      /* 1 turns back (the angle's sign is changed) */
    int32_t src_dtype;    /* hisa_dtype of x and x2: HISA_F32 or HISA_BF16 */
    int32_t dst_dtype;    /* hisa_dtype of y and y2 */
    float mscale;         /* factor of the rotated dims (1 = none) */
    int32_t flags;        /* HISA_FLAG_* bits (0 = none) */
    int64_t x_token, x_head, y_token, y_head;       /* strides of x and y */
    int64_t x2_token, x2_head, y2_token, y2_head;   /* strides of x2 and y2 */
} hisa_rope_desc;

/* The dense combine of a batch whose sequences share their first pooled rows
 * (hisa_prefix_attend). */
typedef struct {
    int32_t B, L;         /* sequences, query rows per sequence */
    int32_t H;            /* query heads sharing the single KV head: 8, 16 or 64 */
    int32_t Dh;           /* head dim: 64, 128 or 512 (with H = 8, 16, 64 respectively) */
    int32_t window;       /* sliding window: local row s is visible to t iff 0 <= t-s < window */
    int32_t W_max;        /* rows allocated per sequence in local_kv */
    int32_t r;            /* compress ratio, for V(t) */
    int32_t flags;        /* HISA_FLAG_* bits (0 = none) */
    int64_t prefix_rows;  /* P: pooled rows that every sequence shares (>= 0) */
    int64_t Np_max;       /* an upper bound of the sequences' own pooled rows Np_b */
    int64_t kv_rows;      /* rows allocated in pooled_kv (>= kv_off[B]); no read goes past it */
    float scale;          /* softmax scale; <= 0 selects Dh^-1/2 */
    int32_t q_dtype;      /* hisa_dtype of q; must equal kv_dtype */
    int32_t kv_dtype;     /* hisa_dtype of local_kv, prefix_kv and pooled_kv */
    int32_t out_dtype;    /* hisa_dtype of out: HISA_F32 or HISA_BF16 */
} hisa_prefix_desc;

/* The norm of each head and rotary positions in one pass over one or two tensors of heads
 * (hisa_norm_rope), for instance queries and the shared KV row of each token. All strides in
 * elements; heads need not be dense. */
typedef struct {
    int64_t tokens;       /* >= 0 (0 = nothing to do) */
    int32_t heads;        /* heads of x (>= 1) */
    int32_t heads2;       /* heads of x2 (0 = no second tensor) */
    int32_t D;            /* head dim, 2..1024 */
    int32_t norm, norm2;  /* 1: the heads of x, of x2, are normed; 0: only turned */
    int32_t rope_dims;    /* rotated dims, even, 0..D (0 = none: table and pos are not read) */
    int32_t rope_first;   /* first rotated dim, 0..D - rope_dims */
    int32_t half;         /* pairs: 0 = (2i, 2i + 1), interleaved; 1 = (i, i + rope_dims / 2), halves */
    int32_t src_dtype;    /* hisa_dtype of x and x2: HISA_F32 or HISA_BF16 */
    int32_t dst_dtype;    /* hisa_dtype of y and y2 */
    float eps;            /* > 0 where something is normed */
    float mscale;         /* factor of the rotated dims (1 = none) */
    int32_t flags;        /* HISA_FLAG_* bits (0 = none) */
    int64_t x_token, x_head, y_token, y_head;       /* strides of x and y */
    int64_t x2_token, x2_head, y2_token, y2_head;   /* strides of x2 and y2 */
} hisa_norm_rope_desc;

/* Rows written to or read from a cache in pages (hisa_cache_append, hisa_cache_read). The cache is
 * `pages` pages of page_rows rows of D dims; row p of sequence b is row p % page_rows of page
 * page_table[b][p / page_rows]. Rows in HISA_BF16: cache [pages, page_rows, D]. Rows in HISA_E2M1:
 * cache [pages, page_rows, D / 2] bytes, dim 2i in the low half of byte i, dim 2i + 1 in the high one
 * (bit 3 the sign, bits 2..1 the exponent, bit 0 the mantissa), and scales
 * [pages, page_rows, D / 16] e4m3; a dim's value is 4-bit float * scale * cache_scale. */
typedef struct {
    int64_t pages;        /* pages allocated (1..2^31 - 1) */
    int32_t page_rows;    /* rows of a page, 1..65536 */
    int32_t D;            /* dims of a row: a multiple of 16, 16..1024 */
    int32_t cache_dtype;  /* HISA_BF16 or HISA_E2M1 */
    float cache_scale;    /* HISA_E2M1: a factor of all rows, 2^-60..2^60 (ignored for HISA_BF16) */
    int32_t B;            /* sequences (>= 1) */
    int32_t table_cols;   /* page numbers of each sequence in page_table (>= 1) */
    int64_t rows;         /* rows allocated in x (append) or out (read); >= 0 */
    int64_t ld;           /* elements from one row of x, or out, to the next (>= D) */
    int32_t io_dtype;     /* hisa_dtype of x: HISA_F32 or HISA_BF16; of out: those, or HISA_E4M3 */
    int32_t flags;        /* HISA_FLAG_* bits (0 = none) */
    /* hisa_cache_append only: */
    int32_t norm;         /* 1: rows are normed first; 0: not */
    float eps;            /* > 0 with norm */
    int32_t rope_dims;    /* rotated dims, even, 0..D (0 = none: table is not read) */
    int32_t rope_first;   /* first rotated dim, 0..D - rope_dims */
    int32_t half;         /* pairs, as in hisa_rope_desc */
    int32_t r;            /* row p sits at position p r (>= 1): the compress ratio, 1 for tokens */
    float mscale;         /* factor of the rotated dims (1 = none) */
} hisa_cache_desc;

/* The combine over a cache in pages (hisa_cache_attend). */
typedef struct {
    int32_t B, L;         /* sequences, query rows per sequence */
    int32_t H;            /* query heads sharing the single KV head: 8, 16 or 64 */
    int32_t Dh;           /* head dim: 64, 128 or 512 (with H = 8, 16, 64 respectively) */
    int32_t window;       /* sliding window: local row s is visible to t iff 0 <= t-s < window */
    int32_t W_max;        /* rows allocated per sequence in local_kv */
    int32_t r;            /* compress ratio, for V(t) */
    int32_t k;            /* width of I, 0..65536 (ignored when I == NULL) */
    int32_t page_rows;    /* rows of a page, 1..65536 */
    int32_t table_cols;   /* page numbers of each sequence in page_table (>= 1) */
    int64_t pages;        /* pages allocated (1..2^31 - 1) */
    int64_t Np_max;       /* an upper bound of cache_len[b]; Np_max and k each with
                             min(window, W_max) below 2^31 - 65536 */
    float scale;          /* softmax scale; <= 0 selects Dh^-1/2 */
    float cache_scale;    /* HISA_E2M1: the factor of all rows, 2^-60..2^60 (ignored for HISA_BF16) */
    int32_t q_dtype;      /* hisa_dtype of q and local_kv: HISA_F32 or HISA_BF16 */
    int32_t cache_dtype;  /* HISA_BF16 or HISA_E2M1 */
    int32_t out_dtype;    /* hisa_dtype of out: HISA_F32 or HISA_BF16 */
    int32_t flags;        /* HISA_FLAG_* bits (0 = none) */
} hisa_cache_attn_desc;

/* Bytes of device workspace `op` needs for `desc` (a hisa_index_desc* for ops 0-4,
 * a hisa_attn_desc* for op 5, a hisa_compress_desc* for op 6, a hisa_prefix_desc* for op 7, a
 * hisa_cache_desc* for op 8, a hisa_cache_attn_desc* for op 9). Always >= 256 for a valid desc; 0 for an invalid one.
 * Pure host arithmetic: needs no GPU. */
HISA_API size_t hisa_workspace_bytes(int32_t op, const void *desc);

/* Clears the device status word of `ws` (asynchronous memset on `stream`). */
HISA_API hisa_status hisa_workspace_init(void *ws, size_t ws_bytes, hisa_stream_t stream);

/* Synchronises `stream`, then copies the status word of `ws` into *flags.
 * Returns HISA_EDEVICE when any bit is set, HISA_OK otherwise. */
HISA_API hisa_status hisa_device_status(const void *ws, hisa_stream_t stream, uint32_t *flags);

/* A static, human-readable name for a status code. */
HISA_API const char *hisa_status_string(int32_t status);

/* Flat indexer scores ([HiSA issue] "Flat selection (baseline path)": s = relu(q.k),
 * score = sum_h s * scale * w; NEG = -1e30 where p >= V(t0+j) when L > 1).
 *   q      [B, L, H_i, D_i]  q_dtype      keys    [sum Np_b, D_i]  k_dtype
 *   w      [B, L, H_i]       f32 raw      key_off [B+1] int64; t0 [B] int32
 *   scores [B*L, ld_scores]  f32 out: row b*L+j holds Np_b scores; columns
 *          [Np_b, ld_scores) are not written. ld_scores >= Np_max.
 * With L > 1 this is the dense L x Np x (H_i*D_i) prefill contraction. */
HISA_API hisa_status hisa_index_scores(const hisa_index_desc *desc, const void *q, const float *w,
                              const void *keys, const int64_t *key_off, const int32_t *t0,
                              float *scores, int64_t ld_scores, void *ws, size_t ws_bytes,
                              hisa_stream_t stream);

/* Block-mean representatives ([HiSA issue] "HiSA decode path": rep = mean over the
 * index_block rows of each complete block; the tail [nb*b, Np) has no block).
 *   means     [*, D_i] f32 out; sequence b's nb_b = floor(Np_b / b) means occupy rows
 *             [means_off[b], means_off[b] + nb_b); means_off [B+1] int64 (device) must
 *             leave room for nb_b rows (else HISA_DEV_BAD_OFFSETS and nothing is written).
 *   first_block [B] int32 or NULL: blocks [first_block[b], nb_b) are (re)computed, so
 *             a decode loop appends the newly completed blocks only. NULL = from 0.
 * f32 sums: for each dimension, eight partial sums over the rows i = k (mod 8) in row
 * order, combined as ((s0 + s1) + (s2 + s3)) + ((s4 + s5) + (s6 + s7)), divided by b
 * (blocks of more than 8192 keys: one sum in row order). */
HISA_API hisa_status hisa_block_means(const hisa_index_desc *desc, const void *keys,
                             const int64_t *key_off, const int64_t *means_off,
                             const int32_t *first_block, float *means, void *ws, size_t ws_bytes,
                             hisa_stream_t stream);

/* Coarse stage ([HiSA issue] "HiSA decode path" / "HiSA batched path": cscore over
 * block means, top Kb = min(keep, nb) blocks; with L > 1 a block is eligible iff its
 * first row is visible, else cscore = NEG).
 *   means/means_off as written by hisa_block_means.
 *   top_blk  [B, L, index_keep] int32 out, ascending block ids.
 *   cscores  [B*L, ld_cscores] f32 out, optional (NULL): nb_b coarse scores per row.
 * Host gate: index_block > 0 and index_block*index_keep >= index_topk, else
 * HISA_EINVAL. Device gate: Np_b >= index_block*index_keep, else HISA_DEV_GATE and a
 * row of -1. */
HISA_API hisa_status hisa_block_filter(const hisa_index_desc *desc, const void *q, const float *w,
                              const float *means, const int64_t *means_off,
                              const int64_t *key_off, const int32_t *t0, int32_t *top_blk,
                              float *cscores, int64_t ld_cscores, void *ws, size_t ws_bytes,
                              hisa_stream_t stream);

/* hisa_block_means, then hisa_block_filter, as one call: the block means of blocks
 * [first_block[b], nb_b) are appended to `means` (same values as hisa_block_means), then
 * the coarse stage runs over all nb_b means. Arguments as in those two calls. For decode
 * (L = 1) with the DeepSeek-V4 indexer shape (H_i = 64, D_i = 128, index_block = 64, bf16
 * keys) it is one kernel, in which the new means are computed while the older means
 * stream into the coarse scoring; otherwise it makes the two calls in turn. ws must hold
 * hisa_workspace_bytes(HISA_OP_BLOCK_FILTER, desc) bytes. */
HISA_API hisa_status hisa_block_filter_append(const hisa_index_desc *desc, const void *q,
                                     const float *w, const void *keys, const int64_t *key_off,
                                     float *means, const int64_t *means_off,
                                     const int32_t *first_block, const int32_t *t0,
                                     int32_t *top_blk, float *cscores, int64_t ld_cscores,
                                     void *ws, size_t ws_bytes, hisa_stream_t stream);

/* Fine stage ([HiSA issue] "HiSA decode path" / "HiSA batched path": candidates
 * pos = top_blk[c / b]*b + c % b, exact rescoring, NEG where pos >= V(t0+j) when
 * L > 1, top k, I = pos[sel]).
 *   top_blk  [B, L, index_keep] int32 (any order; each entry in [0, nb_b)).
 *   I        [B, L, index_topk] int32 out: absolute pooled ids, ascending.
 *   fscores  [B*L, index_keep*index_block] f32 out, optional (NULL): candidate scores
 *            in ascending pos order.
 * Gates as hisa_block_filter. */
HISA_API hisa_status hisa_select_topk(const hisa_index_desc *desc, const void *q, const float *w,
                             const void *keys, const int64_t *key_off, const int32_t *t0,
                             const int32_t *top_blk, int32_t *I, float *fscores, void *ws,
                             size_t ws_bytes, hisa_stream_t stream);

/* Flat selection ([HiSA issue] "Flat selection (baseline path)": top k = min(index_topk,
 * Np_b) of the flat scores; the exact baseline and the path for 512 < Np < 1024).
 *   I [B, L, index_topk] int32 out, ascending ids, -1 beyond min(index_topk, Np_b). */
HISA_API hisa_status hisa_flat_topk(const hisa_index_desc *desc, const void *q, const float *w,
                           const void *keys, const int64_t *key_off, const int32_t *t0,
                           int32_t *I, void *ws, size_t ws_bytes, hisa_stream_t stream);

/* Allocation-free flat selection. The paper has no counterpart: this entry point exists
 * for callers that cannot allocate device memory (hosts whose runtime owns all device
 * memory through its own pool, plugins that may not allocate outside the framework's
 * allocator, loops where cudaMalloc / cudaFree would synchronise the device) and so
 * cannot pass the workspace hisa_flat_topk needs. It computes exactly what
 * hisa_flat_topk computes, with the same arguments and errors, but keeps the scores in
 * a fixed array of device memory declared inside libhisa (16 MiB + 256 bytes), which
 * every GPU that loads the library holds until the process exits. It calls no
 * cudaMalloc, cudaFree or other allocating routine.
 *   B * L * Np_max must not exceed HISA_FLAT_NOALLOC_MAX_SCORES, else HISA_EWORKSPACE
 *   before anything is enqueued.
 *   dev_status: optional (NULL) device pointer to one uint32 that receives this call's
 *   HISA_DEV_* bits (the status is cleared at the start of every call).
 * Runs on the current device. The first call on each device looks up the array's device
 * address (cudaGetSymbolAddress); make that first call before any stream capture.
 * All calls on one device share the one array: calls that may overlap on the GPU (on
 * different streams, or from several host threads without ordering) race and give
 * undefined results; order them on one stream. */
#define HISA_FLAT_NOALLOC_MAX_SCORES 4194304
HISA_API hisa_status hisa_flat_topk_noalloc(const hisa_index_desc *desc, const void *q,
                                   const float *w, const void *keys, const int64_t *key_off,
                                   const int32_t *t0, int32_t *I, uint32_t *dev_status,
                                   hisa_stream_t stream);

/* Indexer compressor ([HiSA issue] "The pooled stream and positions"): appends n_new[b]
 * pooled rows p = p_first[b] .. p_first[b] + n_new[b] - 1 to sequence b's pooled key cache,
 * each anchored at the token window [p r, p r + r - 1]: per output dim d, one softmax over
 * the gate logits gate[t] + ape[t - window start] of the window's tokens (with the overlap
 * variant also the previous window's, through their first D_i channels; row 0 has no
 * previous window) weighs their kv values; then RMSNorm with norm_w and eps, then RoPE of
 * the trailing rope_dims dims, pairs (2m, 2m+1), by the angle (p r) * rope_theta^(-2i /
 * rope_dims) for the i-th rotated pair. Afterwards every block of index_block rows that
 * the new rows complete gets its mean in `means`, with the bits hisa_block_means writes.
 *   kv, gate   [tok_rows, C] f32: wkv(x) and wgate(x) of the tokens, C = 2*D_i (overlap) or
 *              D_i. Sequence b's rows [tok_off[b], tok_off[b+1]) hold (n_new[b] + 1) * r
 *              tokens: the window before row p_first[b] (ignored when p_first[b] == 0 or
 *              without overlap), then the windows of the new rows, in token order.
 *   tok_off    [B+1] int64;  p_first, n_new [B] int32 (n_new <= n_new_max; 0 = nothing)
 *   ape        [r, C] f32;   norm_w [D_i] f32
 *   keys       [keys_rows, D_i] k_dtype in/out: pooled row p of sequence b is row
 *              key_off[b] + p; rows below p_first[b] are read for block means, and
 *              key_off[b] + p_first[b] + n_new[b] must not pass key_off[b+1].
 *   means      [means_rows, D_i] f32 out or NULL; block beta of sequence b at
 *              means_off[b] + beta (means_off [B+1] int64 must leave room for every complete
 *              block). NULL, or index_block == 0, keeps no means.
 * Offsets or counts that do not fit set HISA_DEV_BAD_OFFSETS; that sequence is skipped. */
HISA_API hisa_status hisa_compress_append(const hisa_compress_desc *desc, const float *kv,
                                 const float *gate, const int64_t *tok_off,
                                 const int32_t *p_first, const int32_t *n_new, const float *ape,
                                 const float *norm_w, void *keys, const int64_t *key_off,
                                 float *means, const int64_t *means_off, void *ws,
                                 size_t ws_bytes, hisa_stream_t stream);

/* Sparse combine ([HiSA issue] "Consuming the selection: sparse combine"): one softmax
 * over the visible local rows, the gathered pooled rows P = pooled_kv[I] and the
 * per-head sink, which joins the normaliser and carries no value; K = V.
 *   q          [B, L, H, Dh]  q_dtype (already roped)
 *   local_kv   [B, W_max, Dh] kv_dtype; local_len [B] int32 rows present (<= W_max);
 *              local_pos0 [B] int32 absolute position of local row 0
 *   pooled_kv  [sum Np_b, Dh] kv_dtype; kv_off [B+1] int64
 *   I          [B, L, k] int32 pooled ids (-1 = skip), or NULL for the dense branch over
 *              all Np_b rows. With L > 1 ids >= V(t0+j) are masked.
 *   sinks      [H] f32;  t0 [B] int32
 *   out        [B, L, H, Dh] out, f32 or bf16 as desc->out_dtype says (any device-accessible
 *              address, 16-byte aligned: device memory, or the device address of page-locked
 *              host memory, which the kernels then write directly over the host link)
 * Np_b == 0 gives local-only attention (branch 1 of the three-way branch). */
HISA_API hisa_status hisa_sparse_attend(const hisa_attn_desc *desc, const void *q, const void *local_kv,
                               const int32_t *local_len, const int32_t *local_pos0,
                               const void *pooled_kv, const int64_t *kv_off, const int32_t *I,
                               const float *sinks, const int32_t *t0, void *out, void *ws,
                               size_t ws_bytes, hisa_stream_t stream);

/* Residual addition, root-mean-square norm and output in one pass over the rows:
 *   h = x + residual (f32), rounded to res_dtype where there is a residual; residual_out = h;
 *   y = h / sqrt(mean(h^2) + eps) * w  (f32, over the row as stored);
 *   out = y rounded once, or in 8 bits: per group of scale_group columns (the row if 0) of
 *   largest magnitude a, scale = max(a, 1e-10) / 448, with scale_pow2 the next power of two at
 *   or above it, and out = y / scale rounded to nearest even (|y / scale| <= 448 but for f32
 *   rounding, which saturates). The quotient carries a few f32 roundings, so one that lies within
 *   them of the middle between two codes may take either. Squares and products are f32 too: a row
 *   whose squares overflow gives 0 (NaN where h w overflows as well). A row that holds a NaN or an infinity gives NaN where the
 *   formula does; the other rows are not affected. A row's bits depend on its values and
 *   on the layout (the strides, and where the row starts modulo 8 elements in each array), not on
 *   the other rows or their number.
 *   x            [rows, cols] x_dtype, rows ld_x apart
 *   residual     [rows, cols] res_dtype, rows ld_res apart, or NULL (h = x)
 *   w            [cols] f32
 *   residual_out [rows, cols] res_dtype, rows ld_res apart, or NULL (the sum is not kept); may be
 *                residual itself
 *   out          [rows, cols] out_dtype, rows ld_out apart; may be x itself when dtype and stride
 *                are the same
 *   scales       [rows, cols / scale_group] f32 dense ([rows] if scale_group is 0): HISA_E4M3 only,
 *                else NULL
 * Apart from those two cases no output may overlap an input. Every pointer is aligned to its
 * element; fastest where every row starts at a multiple of 8 elements and cols is one. Whole
 * 16-byte blocks that hold an element of x or residual may be read. No workspace. */
HISA_API hisa_status hisa_rms_norm(const hisa_norm_desc *desc, const void *x, const void *residual,
                          const float *w, void *residual_out, void *out, float *scales,
                          hisa_stream_t stream);

/* Fills table[rope_dims / 2] (HOST memory; pure host arithmetic) for hisa_rope: the turns per
 * position of each pair in units of 2^-64, so that position * table[i] modulo 2^64 is the
 * angle's fraction of a turn, exact at any position. The caller copies it to the device once. */
HISA_API hisa_status hisa_rope_table(const hisa_rope_scaling *scaling, uint64_t *table);

/* Rotary positions ([HiSA issue] "The pooled stream and positions", qk_rope_head_dim): for the
 * i-th pair (a, b) of dims [rope_first, rope_first + rope_dims) of every head of token n, with
 * the angle A = pos[n] * f_i (its sign changed if inverse):
 *   (a, b) -> mscale * (a cos A - b sin A, a sin A + b cos A)
 * in f32, rounded once to dst_dtype; the other dims are copied (converted).
 *   table [rope_dims / 2] uint64 (device, from hisa_rope_table);  pos [tokens] int32 (any sign)
 *   x, y  [tokens, heads, D] and x2, y2 [tokens, heads2, D] with the strides of the descriptor
 * y == x (same strides and dtype) rotates in place and touches the rotated dims alone; the
 * same for y2 == x2, and both are in place or neither is. Otherwise no output may overlap an
 * input. The heads of an output do not overlap one another (strides by which any two do, in place in their
 * rotated dims, are refused); those of an input may (a stride of 0 repeats a row).
 * Pointers are aligned to their element. No workspace. */
HISA_API hisa_status hisa_rope(const hisa_rope_desc *desc, const uint64_t *table, const int32_t *pos,
                      const void *x, void *y, const void *x2, void *y2, hisa_stream_t stream);

/* Shared-prefix combine: the dense branch of hisa_sparse_attend (I = NULL) over the pooled
 * stream made of the P shared rows followed by the sequence's own, the shared rows scored once
 * for the whole batch. For query row j of sequence b at t = t0[b] + j the softmax runs over
 * the visible local rows, all P shared rows, the own pooled rows i in [0, Np_b), Np_b =
 * kv_off[b+1] - kv_off[b], and the per-head sink, which joins the normaliser and carries no
 * value; K = V. With L > 1 own row i, at pooled position P + i, is visible iff P + i <
 * floor((t+1)/r); with L = 1 all are, as in hisa_sparse_attend. The shared rows precede every
 * sequence's own tokens and are always visible. A query row that sees nothing gives 0.
 * Logits, maxima, sums and outputs are f32. With bf16 inputs each softmax weight is rounded to
 * bf16 (by 2^-8 of it at most) for its product with the values, as in hisa_sparse_attend, also where
 * out is f32; with f32 inputs it is not.
 *   q          [B, L, H, Dh]  q_dtype (already roped)
 *   local_kv   [B, W_max, Dh] kv_dtype (NULL if W_max is 0); local_len [B] int32 rows present
 *              (<= W_max); local_pos0 [B] int32 absolute position of local row 0
 *   prefix_kv  [P, Dh] kv_dtype (NULL if P is 0)
 *   pooled_kv  [kv_rows, Dh] kv_dtype (NULL if Np_max is 0); kv_off [B+1] int64
 *   sinks      [H] f32, or NULL for none (-inf is none for that head);  t0 [B] int32
 *   out        [B, L, H, Dh] out_dtype, 16-byte aligned
 * What rows hold that a query row does not see has no effect on it. Offsets that do not fit set
 * HISA_DEV_BAD_OFFSETS; that sequence's own rows are skipped. Few query rows are split along
 * the rows they see and need the more workspace for it: a workspace that serves several batch
 * sizes takes the maximum of hisa_workspace_bytes over them. */
HISA_API hisa_status hisa_prefix_attend(const hisa_prefix_desc *desc, const void *q, const void *local_kv,
                               const int32_t *local_len, const int32_t *local_pos0,
                               const void *prefix_kv, const void *pooled_kv, const int64_t *kv_off,
                               const float *sinks, const int32_t *t0, void *out, void *ws,
                               size_t ws_bytes, hisa_stream_t stream);

/* The root-mean-square norm of each head, then rotary positions, in one pass: for head row x of
 * token n
 *   y = x / sqrt(mean(x^2) + eps) * w   (norm / norm2; else y = x),  then
 *   (a, b) -> mscale * (a cos A - b sin A, a sin A + b cos A),  A = pos[n] * f_i
 * for the i-th pair of dims [rope_first, rope_first + rope_dims) of y, all in f32 and rounded once
 * to dst_dtype. A head whose squares overflow f32 gives 0 (NaN where x w does as well); a head that holds
 * a NaN or an infinity gives NaN where the formula does, and the other heads are not affected.
 *   table [rope_dims / 2] uint64 (device, from hisa_rope_table);  pos [tokens] int32 (any sign);
 *         both NULL if rope_dims is 0
 *   x, y  [tokens, heads, D] and x2, y2 [tokens, heads2, D] with the strides of the descriptor
 *   w, w2 [D] f32, or NULL for ones (and without the norm)
 * y == x (same strides and dtype) works in place; the same for y2 == x2, and both are in place or
 * neither is. Otherwise no output may overlap an input. The heads of an output do not overlap one
 * another (strides by which any two do are refused); those of an input may. Pointers are aligned to
 * their element; fastest where every head starts at a multiple of 8 elements and rope_first and
 * rope_dims (with halves rope_dims / 2) are such. No workspace. */
HISA_API hisa_status hisa_norm_rope(const hisa_norm_rope_desc *desc, const uint64_t *table, const int32_t *pos,
                           const void *x, const float *w, void *y, const void *x2, const float *w2,
                           void *y2, hisa_stream_t stream);

/* Appends rows to a cache in pages. Packed row n of x, row_off[b] <= n < row_off[b+1], becomes row
 * p = first[b] + n - row_off[b] of sequence b: normed and turned as by hisa_norm_rope (the position is
 * p r, any 64-bit number), rounded once to bf16, or in 4 bits: for each 16 dims of largest magnitude a
 *   s = a / (6 cache_scale) rounded to e4m3 (at most 448), each dim y / (s cache_scale) rounded to
 *   nearest even (at most 6), 0 where s is 0.
 * The quotients carry an f32 rounding or two, so one that lies within them of the middle between two
 * codes may take either. Sixteen dims that hold a NaN or an infinity get the scale NaN.
 *   table      [rope_dims / 2] uint64 (NULL if rope_dims is 0)
 *   x          [rows, D] io_dtype, rows ld apart;  w [D] f32 or NULL for ones
 *   row_off    [B+1] int64, ascending;  first [B] int32 (>= 0);  page_table [B, table_cols] int32
 *   cache, scales  as hisa_cache_desc says (scales NULL for HISA_BF16), 16-byte aligned
 * Rows of x before row_off[0] or from row_off[B] on are not read. A row whose place does not fit (an
 * index past table_cols pages, a page outside [0, pages), a negative first) is left out, and so is a
 * sequence whose rows [row_off[b], row_off[b+1]) do not lie in [0, rows); both set HISA_DEV_BAD_OFFSETS.
 * Offsets that go back set it too: a row that then lies in several sequences is left out or goes to one
 * of them. No two rows of a call may have the same place. ws holds the status word (hisa_workspace_bytes(HISA_OP_CACHE, desc)). */
HISA_API hisa_status hisa_cache_append(const hisa_cache_desc *desc, const uint64_t *table, const void *x,
                              const float *w, const int64_t *row_off, const int32_t *first,
                              const int32_t *page_table, void *cache, void *scales, void *ws,
                              size_t ws_bytes, hisa_stream_t stream);

/* Reads rows out of a cache in pages: packed row n of out, row_off[b] <= n < row_off[b+1], is row
 * first[b] + n - row_off[b] of sequence b, as f32 or bf16 (the value, rounded once), or with
 * HISA_E2M1 pages as HISA_E4M3: the 4-bit floats as 8-bit ones, without their scales.
 *   out        [rows, D] io_dtype, rows ld apart, 16-byte aligned, ld a multiple of 8 (of 16 for HISA_E4M3)
 *   out_scales [rows, D / 16] f32 dense: HISA_E4M3 only, scale * cache_scale; or NULL
 * The other arguments and what a row that does not fit does are as in hisa_cache_append; such rows of
 * out, and those before row_off[0] and from row_off[B] on, stay as they were. */
HISA_API hisa_status hisa_cache_read(const hisa_cache_desc *desc, const int64_t *row_off, const int32_t *first,
                            const int32_t *page_table, const void *cache, const void *scales, void *out,
                            float *out_scales, void *ws, size_t ws_bytes, hisa_stream_t stream);

/* The combine of hisa_sparse_attend over pooled rows kept in pages: for query row j of sequence b at
 * t = t0[b] + j one softmax over the visible local rows, the pooled rows named by I (or all
 * cache_len[b] of them, I = NULL) and the per-head sink, which joins the normaliser and carries no
 * value; K = V. With L > 1 pooled row i is visible iff i < floor((t+1)/r); with L = 1 all are. A query
 * row that sees nothing gives 0. Logits, weights, maxima and sums are f32; with bf16 q of 64 heads of 512
 * dims and a bf16 out each softmax weight is rounded to bf16 (by 2^-8 of it at most), in its product with
 * the values and in the normaliser; with an f32 out it is not, and what is left is the tensor cores' f32
 * sums, which are cut off rather than rounded (1e-6 to 3e-6 of an output's norm, whatever the
 * lengths). A bf16 out's sums lose 1e-9 of themselves per row that they add up, 2e-4 over 200000.
 *   q          [B, L, H, Dh]  q_dtype (already roped)
 *   local_kv   [B, W_max, Dh] q_dtype (NULL if W_max is 0); local_len [B] int32 rows present
 *              (<= W_max); local_pos0 [B] int32 absolute position of local row 0
 *   cache, scales  as hisa_cache_desc says with D = Dh (scales NULL for HISA_BF16), 16-byte aligned
 *   page_table [B, table_cols] int32;  cache_len [B] int32: pooled rows of each sequence
 *   I          [B, L, k] int32 pooled ids (-1 = skip), or NULL for all
 *   sinks      [H] f32, or NULL for none (-inf is none for that head);  t0 [B] int32
 *   out        [B, L, H, Dh] out_dtype, 16-byte aligned
 * Two sequences may share pages. What rows hold that a query row does not see has no effect on it.
 * A cache_len that is negative, above Np_max or above table_cols pages sets HISA_DEV_BAD_OFFSETS and
 * that sequence has no pooled rows; a page outside [0, pages) sets it and its rows are skipped; an id
 * outside [-1, cache_len[b]) sets HISA_DEV_BAD_ID and is skipped. A workspace that serves
 * several batch sizes takes the maximum of hisa_workspace_bytes over them. */
HISA_API hisa_status hisa_cache_attend(const hisa_cache_attn_desc *desc, const void *q, const void *local_kv,
                              const int32_t *local_len, const int32_t *local_pos0, const void *cache,
                              const void *scales, const int32_t *page_table, const int32_t *cache_len,
                              const int32_t *I, const float *sinks, const int32_t *t0, void *out,
                              void *ws, size_t ws_bytes, hisa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* HISA_H */
