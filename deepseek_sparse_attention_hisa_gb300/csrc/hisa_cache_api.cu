// C ABI entry points of head norms with rotary positions and of the cache in pages: host-side
// validation, workspace layout and kernel dispatch. Declarations and the contract live in
// include/hisa.h.
#include <cmath>

#include "cache_internal.cuh"
#include "heads_apart.h"

using namespace hisa;

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = 0x7fffffffLL;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool dtype_ok(int32_t d) { return d == HISA_F32 || d == HISA_BF16; }
size_t dtype_bytes(int32_t d) { return d == HISA_F32 ? 4 : (d == HISA_BF16 ? 2 : 1); }
bool flag01(int32_t v) { return v == 0 || v == 1; }
size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
hisa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? HISA_OK : HISA_ECUDA; }
bool scale_ok(float g) { return g >= 0x1p-60f && g <= 0x1p60f; }

bool rope_ok(int D, int dims, int first, int half) {
    if (dims < 0 || (dims & 1) || dims > D || !flag01(half)) return false;
    return dims == 0 || (first >= 0 && first <= D - dims);
}
// rotated dims in whole units of 8 (with halves, either half)
bool rope_wide(int dims, int first, int half) { return dims == 0 || (first % 8 == 0 && dims % (half ? 16 : 8) == 0); }

hisa_status check_norm_rope_desc(const hisa_norm_rope_desc *d) {
    if (!d) return HISA_EINVAL;
    if (d->tokens < 0 || d->tokens > kMaxRows || d->heads < 1 || d->heads2 < 0 || d->heads > 65536 || d->heads2 > 65536)
        return HISA_EINVAL;
    if (d->D < 2 || d->D > 1024 || !flag01(d->norm) || !flag01(d->norm2) || (d->flags & ~(int32_t)HISA_FLAG_CHAINED))
        return HISA_EINVAL;
    if (!rope_ok(d->D, d->rope_dims, d->rope_first, d->half) || !std::isfinite(d->mscale)) return HISA_EINVAL;
    if ((d->norm || (d->heads2 && d->norm2)) && !(d->eps > 0.f)) return HISA_EINVAL;
    if (!dtype_ok(d->src_dtype) || !dtype_ok(d->dst_dtype)) return HISA_EDTYPE;
    const int64_t st[8] = {d->x_token, d->x_head, d->y_token, d->y_head, d->x2_token, d->x2_head, d->y2_token, d->y2_head};
    for (int i = 0; i < (d->heads2 ? 8 : 4); ++i)
        if (st[i] < 0 || st[i] > kMaxStride) return HISA_EINVAL;
    if (d->tokens * ((int64_t)d->heads + d->heads2) > ((int64_t)1 << 36)) return HISA_EINVAL;
    return HISA_OK;
}

hisa_status check_pages(int64_t pages, int32_t page_rows, int32_t table_cols, int32_t cache_dtype, float g) {
    if (pages < 1 || pages > kMaxRows || page_rows < 1 || page_rows > 65536 || table_cols < 1) return HISA_EINVAL;
    if (cache_dtype != HISA_BF16 && cache_dtype != HISA_E2M1) return HISA_EDTYPE;
    return cache_dtype == HISA_E2M1 && !scale_ok(g) ? HISA_EINVAL : HISA_OK;
}

// What append and read have in common; io_dtype is checked by each.
hisa_status check_cache_desc(const hisa_cache_desc *d) {
    if (!d) return HISA_EINVAL;
    const hisa_status st = check_pages(d->pages, d->page_rows, d->table_cols, d->cache_dtype, d->cache_scale);
    if (st != HISA_OK) return st;
    if (d->D < 16 || d->D > 1024 || d->D % 16 || d->B < 1 || d->rows < 0 || d->rows > kMaxRows) return HISA_EINVAL;
    if (d->ld < d->D || d->ld > kMaxStride || (d->flags & ~(int32_t)HISA_FLAG_CHAINED)) return HISA_EINVAL;
    return HISA_OK;
}

hisa_status check_cache_attn_desc(const hisa_cache_attn_desc *d) {
    if (!d) return HISA_EINVAL;
    const hisa_status st = check_pages(d->pages, d->page_rows, d->table_cols, d->cache_dtype, d->cache_scale);
    if (st != HISA_OK) return st;
    if (d->B < 1 || d->L < 1 || d->window < 0 || d->W_max < 0 || d->r < 1 || d->k < 0 || d->k > 65536) return HISA_EINVAL;
    if (d->Np_max < 0 || d->Np_max > kMaxRows - 65536) return HISA_EINVAL;
    // a list's entries are counted in 32 bits
    const int64_t pool = d->Np_max > d->k ? d->Np_max : d->k, local = d->W_max < d->window ? d->W_max : d->window;
    if (local + pool > kMaxRows - 65536) return HISA_EINVAL;
    if ((int64_t)d->B * d->L > kMaxRows / 64 || (d->flags & ~(int32_t)HISA_FLAG_CHAINED)) return HISA_EINVAL;
    if (!dtype_ok(d->q_dtype) || !dtype_ok(d->out_dtype)) return HISA_EDTYPE;
    if (!attend_simt_supported(d->H, d->Dh)) return HISA_EDTYPE;
    return HISA_OK;
}

// Ranges of a query row's list: at most the visible window and `pool` rows. Host arithmetic only (it
// sizes the workspace, for the wider of the two lists that a call may have: I, or all rows).
void attn_plan(const hisa_cache_attn_desc *d, int64_t pool, CacheAttnParams *p) {
    const int64_t local = d->W_max < d->window ? d->W_max : d->window, list = local + pool;
    // about as many CTAs as fit the GPU at once (one per SM for 512 dims, else eight), of a chunk of 32 rows at
    // least (64 for 512 dims, whose sums are large)
    const int64_t items = (int64_t)d->B * d->L, ctas = d->Dh == 512 ? kSmTarget : 8 * kSmTarget;
    int64_t n = ctas / items;
    const int64_t least = d->Dh == 512 ? 64 : 32, most = (list + least - 1) / least;
    n = n > most ? most : n;
    n = n < 1 ? 1 : (n > 128 ? 128 : n);
    const int64_t per = ((list + n - 1) / n + 31) / 32 * 32;
    p->split_rows = (int)(per > 0 ? per : 32);
    p->splits = (int)(list > 0 ? (list + p->split_rows - 1) / p->split_rows : 1);
}
// The tensor-core kernel's CTAs: one per SM, or as many as the device makes spans of all tiles that there can be.
// Whole rows in turn, or spans that cut rows? Cutting evens out what the CTAs do, but its sums go through memory
// and a second kernel joins them: 6 us for one row, 20 for a hundred, against 1.4 us for each tile that the busiest
// CTA is spared. Rows are taken as full with ids (k each), else as filled to 60 %. Measured, whole and cut, in us:
// 50 rows of up to 4 tiles 9.1 and 16.0, 100 of 14 25 and 37, 152 of up to 16 29 and 42, 304 of up to 16 54 and
// 65, 230 of 14 50 and 62; 16 of up to 16 26 and 21, 1 of 9 19 and 13.
void tc_plan(const hisa_cache_attn_desc *d, int64_t pool, bool ids, CacheAttnParams *p) {
    const int64_t local = d->W_max < d->window ? d->W_max : d->window;
    int64_t tiles = (local + kCacheTile - 1) / kCacheTile + (pool + kCacheTile - 1) / kCacheTile;
    tiles = tiles < 1 ? 1 : tiles;
    const int64_t rows = (int64_t)d->B * d->L, rounds = (rows + kCacheCtas - 1) / kCacheCtas;
    const double spared = (double)tiles * ((double)rounds - (ids ? 1.0 : 0.6) * (double)rows / kCacheCtas);
    p->whole = spared <= 6.0 + 0.1 * (double)(rows < 100 ? rows : 100);
    const double best = std::ceil(std::sqrt(10.0 * (double)(rows * tiles) * (double)rows));     // as on the device
    const int64_t n = p->whole ? rows : (best < (double)(rows * tiles) ? (int64_t)best : rows * tiles);
    p->ctas = (int)(n > kCacheCtas ? kCacheCtas : n);
    p->by_row = !p->whole && rows <= p->ctas;
    p->carries = d->out_dtype == HISA_F32 && tiles > kCacheCarry;
}
// The workspace behind the status: rows that spans cut, their sums (maximum and normaliser, then outputs), sums carried.
struct TcLayout {
    size_t cuts, ml, o, carry;
    explicit TcLayout(const CacheAttnParams &p)
        : cuts(round_up(p.ctas * kCutBytes)), ml(round_up(places(p) * 64 * 2 * sizeof(float))), o(places(p) * kCarryFloats * sizeof(float)),
          carry(p.carries ? p.ctas * kCarryFloats * sizeof(float) : 0) {}
    static size_t places(const CacheAttnParams &p) { return p.whole ? 0 : (size_t)2 * p.ctas; }
};
size_t tc_bytes(const hisa_cache_attn_desc *d, int64_t pool, bool ids) {
    CacheAttnParams p{};
    tc_plan(d, pool, ids, &p);
    const TcLayout w(p);
    return kStatusBytes + w.cuts + w.ml + w.o + w.carry;
}
size_t attn_sums(const hisa_cache_attn_desc *d, const CacheAttnParams &p) { return (size_t)d->B * d->L * d->H * p.splits; }
size_t attn_bytes(const hisa_cache_attn_desc *d, int64_t pool) {
    CacheAttnParams p{};
    attn_plan(d, pool, &p);
    const size_t n = attn_sums(d, p);
    return kStatusBytes + round_up(n * d->Dh * sizeof(float)) + round_up(n * 2 * sizeof(float));
}

CacheParams cache_params(const hisa_cache_desc *d, const int64_t *row_off, const int32_t *first, const int32_t *page_table,
                         const void *cache, const void *scales, void *ws) {
    CacheParams p{};
    p.pages = d->pages; p.rows = d->rows; p.ld = d->ld;
    p.page_rows = d->page_rows; p.D = d->D; p.B = d->B; p.table_cols = d->table_cols;
    p.bits4 = d->cache_dtype == HISA_E2M1; p.io_dtype = d->io_dtype;
    p.g = p.bits4 ? d->cache_scale : 1.f;
    p.row_off = row_off; p.row_first = first; p.page_table = page_table;
    p.cache = const_cast<void *>(cache);
    p.scales = static_cast<uint8_t *>(const_cast<void *>(scales));
    p.status = static_cast<uint32_t *>(ws);
    return p;
}

hisa_status check_cache_args(const hisa_cache_desc *d, const int64_t *row_off, const int32_t *first, const int32_t *page_table,
                             const void *cache, const void *scales) {
    if (!row_off || !first || !page_table || !cache || (d->cache_dtype == HISA_E2M1) != (scales != nullptr)) return HISA_EINVAL;
    if (!aligned(row_off, 8) || !aligned(first, 4) || !aligned(page_table, 4) || !aligned(cache, 16) || !aligned(scales, 16))
        return HISA_EINVAL;
    return HISA_OK;
}

}  // namespace

namespace hisa {

size_t cache_workspace_bytes(const hisa_cache_desc *d) { return check_cache_desc(d) == HISA_OK ? kStatusBytes : 0; }

size_t cache_attn_workspace_bytes(const hisa_cache_attn_desc *d) {
    if (check_cache_attn_desc(d) != HISA_OK) return 0;
    const bool tc = cache_tc_supported(d->H, d->Dh, d->q_dtype == HISA_BF16);
    const size_t all = tc ? tc_bytes(d, d->Np_max, false) : attn_bytes(d, d->Np_max);
    const size_t some = tc ? tc_bytes(d, d->k, true) : attn_bytes(d, d->k);
    return all > some ? all : some;
}

}  // namespace hisa

extern "C" {

hisa_status hisa_norm_rope(const hisa_norm_rope_desc *d, const uint64_t *table, const int32_t *pos, const void *x,
                           const float *w, void *y, const void *x2, const float *w2, void *y2, hisa_stream_t stream) {
    const hisa_status st = check_norm_rope_desc(d);
    if (st != HISA_OK) return st;
    if (d->tokens == 0) return HISA_OK;
    if (!x || !y || (d->rope_dims && (!table || !pos))) return HISA_EINVAL;
    if (d->heads2 ? (!x2 || !y2) : (x2 || y2 || w2)) return HISA_EINVAL;
    if ((w && !d->norm) || (w2 && !d->norm2)) return HISA_EINVAL;
    const size_t ss = dtype_bytes(d->src_dtype), sd = dtype_bytes(d->dst_dtype);
    if (!aligned(table, 8) || !aligned(pos, 4) || !aligned(x, ss) || !aligned(x2, ss) || !aligned(y, sd) || !aligned(y2, sd) ||
        !aligned(w, 4) || !aligned(w2, 4))
        return HISA_EINVAL;
    const bool inplace = x == y;
    if (inplace && (d->src_dtype != d->dst_dtype || d->x_token != d->y_token || d->x_head != d->y_head)) return HISA_EINVAL;
    if (d->heads2 && ((x2 == y2) != inplace ||
                      (inplace && (d->x2_token != d->y2_token || d->x2_head != d->y2_head))))
        return HISA_EINVAL;
    // heads of an output that overlap would be written by several warps, in no order
    if (!heads_apart(d->tokens, d->heads, d->y_token, d->y_head, d->D) ||
        (d->heads2 && !heads_apart(d->tokens, d->heads2, d->y2_token, d->y2_head, d->D)))
        return HISA_EINVAL;
    NormRopeParams p{};
    p.tokens = d->tokens; p.heads = d->heads; p.heads2 = d->heads2; p.D = d->D;
    p.norm = d->norm; p.norm2 = d->norm2;
    p.dims = d->rope_dims; p.first = d->rope_dims ? d->rope_first : 0; p.half = d->half;
    p.src_bf16 = d->src_dtype == HISA_BF16; p.dst_bf16 = d->dst_dtype == HISA_BF16;
    p.eps = d->eps; p.mscale = d->mscale;
    p.table = table; p.pos = pos;
    p.x = x; p.x2 = x2; p.w = w; p.w2 = w2; p.y = y; p.y2 = y2;
    p.x_token = d->x_token; p.x_head = d->x_head; p.y_token = d->y_token; p.y_head = d->y_head;
    p.x2_token = d->x2_token; p.x2_head = d->x2_head; p.y2_token = d->y2_token; p.y2_head = d->y2_head;
    // units of 8 dims: 32 or 16 bytes at every boundary
    auto wide = [](const void *a, int64_t token, int64_t head, size_t es) { return aligned(a, 8 * es) && token % 8 == 0 && head % 8 == 0; };
    p.wide = d->D % 8 == 0 && rope_wide(p.dims, p.first, p.half) && aligned(w, 16) && aligned(w2, 16) &&
             wide(x, d->x_token, d->x_head, ss) && wide(y, d->y_token, d->y_head, sd) &&
             (!d->heads2 || (wide(x2, d->x2_token, d->x2_head, ss) && wide(y2, d->y2_token, d->y2_head, sd)));
    return from_cuda(launch_norm_rope(p, reinterpret_cast<cudaStream_t>(stream)));
}

hisa_status hisa_cache_append(const hisa_cache_desc *d, const uint64_t *table, const void *x, const float *w,
                              const int64_t *row_off, const int32_t *first, const int32_t *page_table, void *cache,
                              void *scales, void *ws, size_t ws_bytes, hisa_stream_t stream) {
    hisa_status st = check_cache_desc(d);
    if (st != HISA_OK) return st;
    if (!dtype_ok(d->io_dtype)) return HISA_EDTYPE;
    if (!flag01(d->norm) || (d->norm && !(d->eps > 0.f)) || d->r < 1 || !std::isfinite(d->mscale)) return HISA_EINVAL;
    if (!rope_ok(d->D, d->rope_dims, d->rope_first, d->half)) return HISA_EINVAL;
    if (!ws || !aligned(ws, kAlign) || ws_bytes < kStatusBytes) return HISA_EWORKSPACE;
    if (d->rows == 0) return HISA_OK;
    st = check_cache_args(d, row_off, first, page_table, cache, scales);
    if (st != HISA_OK) return st;
    if (!x || (d->rope_dims && !table) || (w && !d->norm)) return HISA_EINVAL;
    if (!aligned(x, dtype_bytes(d->io_dtype)) || !aligned(table, 8) || !aligned(w, 4)) return HISA_EINVAL;
    CacheParams p = cache_params(d, row_off, first, page_table, cache, scales, ws);
    p.norm = d->norm; p.eps = d->eps;
    p.dims = d->rope_dims; p.first = d->rope_dims ? d->rope_first : 0; p.half = d->half; p.r = d->r; p.mscale = d->mscale;
    p.table = table; p.x = x; p.w = w;
    p.wide = rope_wide(p.dims, p.first, p.half) && aligned(x, 8 * dtype_bytes(d->io_dtype)) && d->ld % 8 == 0 && aligned(w, 16);
    return from_cuda(launch_cache_append(p, reinterpret_cast<cudaStream_t>(stream)));
}

hisa_status hisa_cache_read(const hisa_cache_desc *d, const int64_t *row_off, const int32_t *first, const int32_t *page_table,
                            const void *cache, const void *scales, void *out, float *out_scales, void *ws, size_t ws_bytes,
                            hisa_stream_t stream) {
    hisa_status st = check_cache_desc(d);
    if (st != HISA_OK) return st;
    const bool q8 = d->io_dtype == HISA_E4M3;
    if (!dtype_ok(d->io_dtype) && !(q8 && d->cache_dtype == HISA_E2M1)) return HISA_EDTYPE;
    if (d->ld % (q8 ? 16 : 8)) return HISA_EINVAL;
    if (!ws || !aligned(ws, kAlign) || ws_bytes < kStatusBytes) return HISA_EWORKSPACE;
    if (d->rows == 0) return HISA_OK;
    st = check_cache_args(d, row_off, first, page_table, cache, scales);
    if (st != HISA_OK) return st;
    if (!out || !aligned(out, 16) || !aligned(out_scales, 4) || (out_scales && !q8)) return HISA_EINVAL;
    CacheParams p = cache_params(d, row_off, first, page_table, cache, scales, ws);
    p.out = out; p.out_scales = out_scales;
    p.out32 = aligned(out, 32);
    return from_cuda(launch_cache_read(p, reinterpret_cast<cudaStream_t>(stream)));
}

hisa_status hisa_cache_attend(const hisa_cache_attn_desc *d, const void *q, const void *local_kv, const int32_t *local_len,
                              const int32_t *local_pos0, const void *cache, const void *scales, const int32_t *page_table,
                              const int32_t *cache_len, const int32_t *I, const float *sinks, const int32_t *t0, void *out,
                              void *ws, size_t ws_bytes, hisa_stream_t stream) {
    const hisa_status st = check_cache_attn_desc(d);
    if (st != HISA_OK) return st;
    if (!q || !out || !t0 || !cache || !page_table || !cache_len) return HISA_EINVAL;
    if (d->W_max > 0 && (!local_kv || !local_len || !local_pos0)) return HISA_EINVAL;
    if ((d->cache_dtype == HISA_E2M1) != (scales != nullptr)) return HISA_EINVAL;
    if (!aligned(q, 16) || !aligned(local_kv, 16) || !aligned(cache, 16) || !aligned(scales, 16) || !aligned(out, 16))
        return HISA_EINVAL;
    if (!aligned(local_len, 4) || !aligned(local_pos0, 4) || !aligned(page_table, 4) || !aligned(cache_len, 4) ||
        !aligned(I, 4) || !aligned(sinks, 4) || !aligned(t0, 4))
        return HISA_EINVAL;
    if (!ws || !aligned(ws, kAlign) || ws_bytes < cache_attn_workspace_bytes(d)) return HISA_EWORKSPACE;
    CacheAttnParams p{};
    p.B = d->B; p.L = d->L; p.H = d->H; p.Dh = d->Dh; p.window = d->window; p.W_max = d->W_max; p.r = d->r; p.k = d->k;
    p.page_rows = d->page_rows; p.table_cols = d->table_cols; p.pages = d->pages; p.Np_max = d->Np_max;
    p.scale = d->scale > 0.f ? d->scale : (float)(1.0 / std::sqrt((double)d->Dh));
    p.bits4 = d->cache_dtype == HISA_E2M1;
    p.g = p.bits4 ? d->cache_scale : 1.f;
    p.q = q; p.local_kv = local_kv; p.local_len = local_len; p.local_pos0 = local_pos0;
    p.cache = cache; p.scales = static_cast<const uint8_t *>(scales); p.cache32 = aligned(cache, 32);
    p.page_table = page_table; p.cache_len = cache_len; p.I = I; p.sinks = sinks; p.t0 = t0; p.out = out;
    p.q_bf16 = d->q_dtype == HISA_BF16; p.out_bf16 = d->out_dtype == HISA_BF16;
    p.status = static_cast<uint32_t *>(ws);
    char *base = static_cast<char *>(ws) + kStatusBytes;
    if (cache_tc_supported(d->H, d->Dh, p.q_bf16)) {
        tc_plan(d, I ? d->k : d->Np_max, I != nullptr, &p);
        const TcLayout w(p);
        p.cuts = base;
        p.part_ml = reinterpret_cast<float *>(base + w.cuts);
        p.part_o = reinterpret_cast<float *>(base + w.cuts + w.ml);
        p.carry = reinterpret_cast<float *>(base + w.cuts + w.ml + w.o);
        return from_cuda(launch_cache_tc(p, reinterpret_cast<cudaStream_t>(stream)));
    }
    attn_plan(d, I ? d->k : d->Np_max, &p);
    const size_t rows = attn_sums(d, p);
    p.part_o = reinterpret_cast<float *>(base);
    p.part_ml = reinterpret_cast<float *>(base + round_up(rows * d->Dh * sizeof(float)));
    return from_cuda(launch_cache_simt(p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
