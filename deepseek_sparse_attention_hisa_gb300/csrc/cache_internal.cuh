// Internal declarations of the operators of a cache in pages: norms and rotations of heads, rows
// appended and read back, the combine. Nothing here is part of the C ABI (see include/hisa.h).
#pragma once

#include "ops_internal.cuh"

namespace hisa {

constexpr int kScaleGroup = 16;           // dims of a 4-bit row that share a scale

struct NormRopeParams {
    int64_t tokens;
    int heads, heads2, D;
    int norm, norm2;
    int dims, first, half;
    int src_bf16, dst_bf16;
    float eps, mscale;
    const uint64_t *table;
    const int32_t *pos;
    const void *x, *x2;
    const float *w, *w2;      // or nullptr
    void *y, *y2;
    int64_t x_token, x_head, y_token, y_head, x2_token, x2_head, y2_token, y2_head;
    int wide;                 // 8 elements per access fit every boundary
    // set by launch_norm_rope
    int lanes;                // threads of a team: one head at a time
    int run, runs, runs1;     // heads of a team; teams per token, of them for x
};

struct CacheParams {
    int64_t pages, rows, ld;
    int page_rows, D, B, table_cols;
    int bits4, io_dtype;
    float g;                  // cache_scale (1 for bf16 pages)
    int norm;
    float eps;
    int dims, first, half, r;
    float mscale;
    const uint64_t *table;
    const void *x;
    const float *w;           // or nullptr
    const int64_t *row_off;
    const int32_t *row_first;
    const int32_t *page_table;
    void *cache;
    uint8_t *scales;
    void *out;
    float *out_scales;
    uint32_t *status;
    int wide;                 // append: 8 elements per access fit every boundary of x and of the rotated dims
    int out32;                // read: rows of out start at multiples of 32 bytes
    int lanes, chunk;         // set by the launchers: threads of a team; consecutive rows of a warp
};

struct CacheAttnParams {
    int B, L, H, Dh, window, W_max, r, k;
    int page_rows, table_cols;
    int64_t pages, Np_max;
    float scale, g;
    const void *q, *local_kv;
    const int32_t *local_len, *local_pos0;
    const void *cache;
    const uint8_t *scales;
    const int32_t *page_table, *cache_len;
    const int32_t *I;         // [B*L, k] or nullptr
    const float *sinks;       // or nullptr
    const int32_t *t0;
    void *out;
    int q_bf16, bits4, out_bf16;
    int splits, split_rows;   // CUDA-core kernel: ranges of a query row's list, rows of each
    int cache32;              // rows in 4 bits start at multiples of 32 bytes
    int ctas, whole;          // tensor-core kernel: CTAs; whole rows in turn, not spans of all rows' tiles
    void *cuts;               // its rows that spans cut: an entry per row (by_row) or per CTA
    int by_row;
    int carries;              // a list may be long enough for sums to be carried
    float *part_o, *part_ml;  // partial sums
    float *carry;             // tensor-core kernel: sums of long lists, kCarryFloats per CTA
    uint32_t *status;
};
constexpr int kCacheCtas = kSmTarget;     // most CTAs of the tensor-core kernel
constexpr size_t kCutBytes = 32;
constexpr int kCacheTile = 48;            // its list rows per tile
constexpr int kCacheCarry = 16;           // its tiles after which an f32 output's sums move to memory
constexpr size_t kCarryFloats = 64 * 512;

// What a query row sees: local rows [lo, lo + nloc) of its window buffer, then npool entries of its
// list of pooled rows (ids of I, or rows 0, 1, ...), of which those below V are visible.
struct CacheRow {
    int64_t lo, len, V;
    int nloc, npool;
};
__device__ __forceinline__ CacheRow cache_row(const CacheAttnParams &p, int64_t row, bool report) {
    const uint32_t b = (uint32_t)row / (uint32_t)p.L;     // B L fits 32 bits
    const int64_t t = (int64_t)p.t0[b] + ((uint32_t)row - b * (uint32_t)p.L);
    CacheRow x{0, 0, 0, 0, 0};
    if (p.W_max > 0) {
        const int64_t in = p.local_len[b], nl = in < 0 ? 0 : (in > p.W_max ? p.W_max : in);
        const int64_t pos0 = p.local_pos0[b];
        int64_t lo = t - p.window + 1 - pos0, hi = t - pos0 + 1;
        lo = lo < 0 ? 0 : lo;
        hi = hi > nl ? nl : hi;
        if (hi > lo) {
            x.lo = lo;
            x.nloc = (int)(hi - lo);
        }
    }
    x.len = p.cache_len[b];
    if (x.len < 0 || x.len > p.Np_max || x.len > (int64_t)p.table_cols * p.page_rows) {
        if (report) flag(p.status, HISA_DEV_BAD_OFFSETS);
        x.len = 0;
    }
    x.V = x.len;
    if (p.L > 1) {
        const int64_t v = t + 1 < 0 ? 0 : (int64_t)((uint32_t)(t + 1) / (uint32_t)p.r);   // t + 1 fits 32 bits: L < 2^25
        x.V = v < x.len ? v : x.len;
    }
    x.npool = p.I ? p.k : (int)x.V;
    return x;
}

// The row of the pool that entry kk of a query row's list is, or -1: masked, skipped or out of place.
__device__ __forceinline__ int64_t cache_slot(const CacheAttnParams &p, int64_t row, const CacheRow &x, int kk) {
    int64_t id = kk;
    if (p.I) {
        id = p.I[row * p.k + kk];
        if (id < -1 || id >= x.len) {
            flag(p.status, HISA_DEV_BAD_ID);
            return -1;
        }
        if (id < 0 || id >= x.V) return -1;
    }
    const uint32_t at = (uint32_t)id / (uint32_t)p.page_rows;
    const int64_t page = p.page_table[(int64_t)((uint32_t)row / (uint32_t)p.L) * p.table_cols + at];
    if (page < 0 || page >= p.pages) {
        flag(p.status, HISA_DEV_BAD_OFFSETS);
        return -1;
    }
    return page * p.page_rows + ((uint32_t)id - at * (uint32_t)p.page_rows);
}

// Eight 4-bit floats (a word of a row: the first one lowest), as f32.
__device__ __forceinline__ void unpack_e2m1(uint32_t w, float (&f)[8]) {
    uint32_t h[4];
    asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4; cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b; "
        "cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d;}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}"
            : "=f"(f[2 * i]), "=f"(f[2 * i + 1]) : "r"(h[i]));
}
// A scale of type e4m3 as f32 (its NaN as NaN).
__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) {
    float f;
    asm("{.reg .b16 h, a, b; .reg .b32 w; cvt.u16.u32 h, %1; cvt.rn.f16x2.e4m3x2 w, h; mov.b32 {a, b}, w; cvt.f32.f16 %0, a;}"
        : "=f"(f) : "r"(byte & 0xffu));
    return f;
}

size_t cache_workspace_bytes(const hisa_cache_desc *d);
size_t cache_attn_workspace_bytes(const hisa_cache_attn_desc *d);

cudaError_t launch_norm_rope(const NormRopeParams &p, cudaStream_t s);
cudaError_t launch_cache_append(const CacheParams &p, cudaStream_t s);
cudaError_t launch_cache_read(const CacheParams &p, cudaStream_t s);
cudaError_t launch_cache_simt(const CacheAttnParams &p, cudaStream_t s);
// The combine on the tensor cores (64 bf16 heads of 512 dims).
bool cache_tc_supported(int H, int Dh, int q_bf16);
cudaError_t launch_cache_tc(const CacheAttnParams &p, cudaStream_t s);

}  // namespace hisa
