// C ABI entry points of the operators around the step: host-side validation, workspace layout
// and kernel dispatch. Declarations and the contract live in include/hisa.h.
#include <cmath>

#include "ops_internal.cuh"

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

hisa_status check_norm_desc(const hisa_norm_desc *d) {
    if (!d) return HISA_EINVAL;
    if (d->rows < 0 || d->rows > kMaxRows || d->cols < 1 || d->cols > 32768) return HISA_EINVAL;
    if (!(d->eps > 0.f) || (d->flags & ~(int32_t)HISA_FLAG_CHAINED)) return HISA_EINVAL;
    if (!dtype_ok(d->x_dtype) || !dtype_ok(d->res_dtype) || (!dtype_ok(d->out_dtype) && d->out_dtype != HISA_E4M3))
        return HISA_EDTYPE;
    if (d->out_dtype == HISA_E4M3) {
        const int g = d->scale_group;
        if (g != 0 && g != 32 && g != 64 && g != 128 && g != 256) return HISA_EINVAL;
        if ((g && d->cols % g) || !flag01(d->scale_pow2)) return HISA_EINVAL;
    } else if (d->scale_group != 0 || d->scale_pow2 != 0) {
        return HISA_EINVAL;
    }
    if (d->ld_x < d->cols || d->ld_out < d->cols || d->ld_x > kMaxStride || d->ld_out > kMaxStride) return HISA_EINVAL;
    return HISA_OK;
}

hisa_status check_rope_desc(const hisa_rope_desc *d) {
    if (!d) return HISA_EINVAL;
    if (d->tokens < 0 || d->tokens > kMaxRows || d->heads < 1 || d->heads2 < 0 || d->heads > 65536 || d->heads2 > 65536)
        return HISA_EINVAL;
    if (d->D < 2 || d->D > 1024 || d->rope_dims < 2 || (d->rope_dims & 1) || d->rope_dims > d->D) return HISA_EINVAL;
    if (d->rope_first < 0 || d->rope_first > d->D - d->rope_dims) return HISA_EINVAL;
    if (!flag01(d->half) || !flag01(d->inverse) || (d->flags & ~(int32_t)HISA_FLAG_CHAINED)) return HISA_EINVAL;
    if (!std::isfinite(d->mscale)) return HISA_EINVAL;
    if (!dtype_ok(d->src_dtype) || !dtype_ok(d->dst_dtype)) return HISA_EDTYPE;
    const int64_t st[8] = {d->x_token, d->x_head, d->y_token, d->y_head, d->x2_token, d->x2_head, d->y2_token, d->y2_head};
    for (int i = 0; i < (d->heads2 ? 8 : 4); ++i)
        if (st[i] < 0 || st[i] > kMaxStride) return HISA_EINVAL;
    if (d->tokens * ((int64_t)d->heads + d->heads2) > ((int64_t)1 << 36)) return HISA_EINVAL;
    return HISA_OK;
}

hisa_status check_prefix_desc(const hisa_prefix_desc *d) {
    if (!d) return HISA_EINVAL;
    if (d->B < 1 || d->L < 1 || d->window < 0 || d->W_max < 0 || d->r < 1) return HISA_EINVAL;
    if (d->prefix_rows < 0 || d->prefix_rows > kMaxRows || d->Np_max < 0 || d->Np_max > kMaxRows) return HISA_EINVAL;
    if (d->kv_rows < 0 || d->kv_rows > kMaxRows) return HISA_EINVAL;
    if ((int64_t)d->B * d->L > kMaxRows / 64) return HISA_EINVAL;
    if (d->flags & ~(int32_t)HISA_FLAG_CHAINED) return HISA_EINVAL;
    if (!dtype_ok(d->q_dtype) || d->q_dtype != d->kv_dtype || !dtype_ok(d->out_dtype)) return HISA_EDTYPE;
    if (!attend_simt_supported(d->H, d->Dh)) return HISA_EDTYPE;
    return HISA_OK;
}

// Segments of the combine. Host arithmetic only (it sizes the workspace).
void prefix_plan(const hisa_prefix_desc *d, PrefixParams *p) {
    const int64_t queries = (int64_t)d->B * d->L;
    const int64_t local = d->W_max < d->window ? d->W_max : d->window;
    const int64_t list = local + d->Np_max;
    if (prefix_tc_supported(d->H, d->Dh, d->kv_dtype == HISA_BF16)) {
        // Pairs of CTAs walk (two query rows, segment) items, a segment an even part of the pair's
        // tiles: 32 own rows (of each query row) or 64 shared rows. The split with the shortest
        // longest walk, in tiles (about 0.7 us each): an item costs about 4 more (fill, epilogue);
        // with several segments each costs a write and a read of its sums (2 KB per query row and
        // head, both ways at about 6 TB/s), and the merge a launch. Own lists are taken as half full.
        const int64_t tiles = (d->prefix_rows + 63) / 64 + (local + 31) / 32 + (d->Np_max + 63) / 64;
        const int64_t pairs = (queries + 1) / 2;
        double best = 0.0;
        p->pre_split = 1;
        for (int64_t n = 1; n <= 64 && n <= tiles; ++n) {
            const int64_t walk = (pairs * n + kSmTarget / 2 - 1) / (kSmTarget / 2);
            double cost = (double)walk * (double)((tiles + n - 1) / n + 4);
            if (n > 1) cost += (double)n * (double)queries * 64 * 4096 / 6e12 / 0.7e-6 + 4;
            if (n == 1 || cost < best) {
                best = cost;
                p->pre_split = (int)n;
            }
        }
        return;
    }
    auto split = [](int64_t items, int64_t rows, int64_t ctas, int64_t *per) {
        // about `ctas` CTAs, at least 64 rows each
        int64_t n = ctas / (items > 0 ? items : 1);
        const int64_t most = (rows + 63) / 64;
        n = n > most ? most : n;
        n = n < 1 ? 1 : (n > 64 ? 64 : n);
        *per = ((rows + n - 1) / n + 31) / 32 * 32;
        return (int)((rows + *per - 1) / *per);
    };
    int64_t per = 0;
    // eight or more CTAs of the own lists' kernel fit an SM (one of 512 dims)
    p->tail_split = list > 0 ? split(queries, list, d->Dh == 512 ? kSmTarget : 8 * kSmTarget, &per) : 0;
    p->tail_rows = (int)(per < kMaxRows ? per : kMaxRows);
    if (d->prefix_rows == 0) return;
    if (d->kv_dtype == HISA_BF16) {
        // tiles of 128 stacked rows x ranges of whole 128-row tiles, one CTA per SM: the split with
        // the shortest longest walk, an item costing about 4 tiles more (fill, epilogue)
        const int64_t items = (queries * d->H + 127) / 128, tiles = (d->prefix_rows + 127) / 128;
        int64_t best = 0;
        for (int64_t n = 1; n <= 64 && n <= tiles; ++n) {
            const int64_t per_n = (tiles + n - 1) / n, segs = (tiles + per_n - 1) / per_n;
            const int64_t cost = (items * segs + kSmTarget - 1) / kSmTarget * (per_n + 4);
            if (n == 1 || cost < best) {
                best = cost;
                p->pre_split = (int)segs;
                p->pre_rows = per_n * 128;
            }
        }
        return;
    }
    p->pre_split = split((queries * d->H + 63) / 64, d->prefix_rows, d->Dh == 512 ? kSmTarget : kTargetCtas, &p->pre_rows);
}

// Segments whose sums go through the workspace.
size_t prefix_parts(const hisa_prefix_desc *d, const PrefixParams &p) {
    if (prefix_tc_supported(d->H, d->Dh, d->kv_dtype == HISA_BF16) && p.pre_split == 1) return 0;
    return (size_t)p.tail_split + p.pre_split;
}

}  // namespace

namespace hisa {

size_t prefix_workspace_bytes(const hisa_prefix_desc *d) {
    if (check_prefix_desc(d) != HISA_OK) return 0;
    PrefixParams p{};
    prefix_plan(d, &p);
    const size_t rows = (size_t)d->B * d->L * d->H, seg = prefix_parts(d, p);
    return kStatusBytes + round_up(seg * rows * d->Dh * sizeof(float)) + round_up(seg * rows * 2 * sizeof(float));
}

}  // namespace hisa

extern "C" {

hisa_status hisa_rms_norm(const hisa_norm_desc *d, const void *x, const void *residual, const float *w, void *residual_out,
                          void *out, float *scales, hisa_stream_t stream) {
    const hisa_status st = check_norm_desc(d);
    if (st != HISA_OK) return st;
    if (d->rows == 0) return HISA_OK;
    const bool q8 = d->out_dtype == HISA_E4M3;
    if (!x || !w || !out || (residual_out && !residual) || q8 != (scales != nullptr)) return HISA_EINVAL;
    if (residual && (d->ld_res < d->cols || d->ld_res > kMaxStride)) return HISA_EINVAL;
    const size_t sx = dtype_bytes(d->x_dtype), sr = dtype_bytes(d->res_dtype), so = dtype_bytes(d->out_dtype);
    if (!aligned(x, sx) || !aligned(residual, sr) || !aligned(residual_out, sr) || !aligned(out, so) || !aligned(w, 4) ||
        !aligned(scales, 4))
        return HISA_EINVAL;
    if (out == x && (d->out_dtype != d->x_dtype || d->ld_out != d->ld_x)) return HISA_EINVAL;
    NormParams p{};
    p.rows = d->rows; p.cols = d->cols;
    p.x_bf16 = d->x_dtype == HISA_BF16; p.res_bf16 = d->res_dtype == HISA_BF16;
    p.out_dtype = d->out_dtype; p.group = d->scale_group; p.pow2 = d->scale_pow2;
    p.groups = p.group ? d->cols / p.group : 1;
    p.unit_shift = 16;                                 // 32768 columns are 4096 units
    for (int i = 2; i <= 5; ++i)
        if (p.group == 8 << i) p.unit_shift = i;
    p.eps = d->eps;
    p.ld_x = d->ld_x; p.ld_res = residual ? d->ld_res : 0; p.ld_out = d->ld_out;
    p.x = x; p.res = residual; p.w = w; p.res_out = residual_out; p.out = out; p.scales = scales;
    // units of 8 columns: 32, 16 or 8 bytes of every tensor
    auto wide = [&](const void *a, int64_t ld, size_t es) { return aligned(a, 8 * es) && ld % 8 == 0; };
    p.wide = d->cols % 8 == 0 && aligned(w, 16) && wide(x, d->ld_x, sx) && wide(out, d->ld_out, so) &&
             (!residual || (wide(residual, d->ld_res, sr) && wide(residual_out, d->ld_res, sr)));
    auto phase = [](const void *a, size_t es) { return (int)(reinterpret_cast<uintptr_t>(a) / es % 8); };
    p.phase = phase(x, sx);
    if (p.group || phase(out, so) != p.phase || (d->ld_x - d->ld_out) % 8 ||
        (residual && (phase(residual, sr) != p.phase || (d->ld_x - d->ld_res) % 8)) ||
        (residual_out && phase(residual_out, sr) != p.phase))
        p.phase = -1;
    p.chained = (d->flags & HISA_FLAG_CHAINED) != 0;
    return from_cuda(launch_rms_norm(p, reinterpret_cast<cudaStream_t>(stream)));
}

hisa_status hisa_rope_table(const hisa_rope_scaling *s, uint64_t *table) {
    if (!s || !table) return HISA_EINVAL;
    const int d = s->rope_dims;
    if (d < 2 || d > 1024 || (d & 1) || !(s->theta > 1.0) || !std::isfinite(s->theta)) return HISA_EINVAL;
    if (s->kind != HISA_ROPE_PLAIN && s->kind != HISA_ROPE_LINEAR && s->kind != HISA_ROPE_YARN) return HISA_EINVAL;
    if (s->kind != HISA_ROPE_PLAIN && (!(s->factor > 0.0) || !std::isfinite(s->factor))) return HISA_EINVAL;
    const double two_pi = 6.283185307179586476925;
    double lo = 0.0, hi = 0.0;
    if (s->kind == HISA_ROPE_YARN) {
        if (!(s->orig_len > 0.0) || !(s->beta_fast > 0.0) || !(s->beta_slow > 0.0) || !std::isfinite(s->orig_len) ||
            !std::isfinite(s->beta_fast) || !std::isfinite(s->beta_slow))
            return HISA_EINVAL;
        auto at = [&](double turns) { return d * std::log(s->orig_len / (two_pi * turns)) / (2.0 * std::log(s->theta)); };
        lo = std::floor(at(s->beta_fast));
        hi = std::ceil(at(s->beta_slow));
        lo = lo < 0.0 ? 0.0 : lo;
        hi = hi > d - 1.0 ? d - 1.0 : hi;
    }
    for (int i = 0; i < d / 2; ++i) {
        double f = std::pow(s->theta, -2.0 * i / d);
        if (s->kind == HISA_ROPE_LINEAR) f /= s->factor;
        if (s->kind == HISA_ROPE_YARN) {
            double g = (i - lo) / (hi - lo > 0.001 ? hi - lo : 0.001);
            g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
            f = f / s->factor * g + f * (1.0 - g);
        }
        // the fraction of a turn per position; whole turns (a factor below 1 / (2 pi)) drop out,
        // since positions are whole numbers
        double turns = f / two_pi;
        turns -= std::floor(turns);
        table[i] = (uint64_t)std::ldexp(turns, 64);
    }
    return HISA_OK;
}

hisa_status hisa_rope(const hisa_rope_desc *d, const uint64_t *table, const int32_t *pos, const void *x, void *y,
                      const void *x2, void *y2, hisa_stream_t stream) {
    const hisa_status st = check_rope_desc(d);
    if (st != HISA_OK) return st;
    if (d->tokens == 0) return HISA_OK;
    if (!table || !pos || !x || !y) return HISA_EINVAL;
    if (d->heads2 ? (!x2 || !y2) : (x2 || y2)) return HISA_EINVAL;
    const size_t ss = dtype_bytes(d->src_dtype), sd = dtype_bytes(d->dst_dtype);
    if (!aligned(table, 8) || !aligned(pos, 4) || !aligned(x, ss) || !aligned(x2, ss) || !aligned(y, sd) || !aligned(y2, sd))
        return HISA_EINVAL;
    const bool inplace = x == y;
    if (inplace && (d->src_dtype != d->dst_dtype || d->x_token != d->y_token || d->x_head != d->y_head)) return HISA_EINVAL;
    if (d->heads2 && ((x2 == y2) != inplace ||
                      (inplace && (d->x2_token != d->y2_token || d->x2_head != d->y2_head))))
        return HISA_EINVAL;
    // neighbouring rows of an output that overlap (a broadcast view rotated in place, say) would be
    // written by several threads, in no order
    const int64_t written = inplace ? d->rope_dims : d->D;
    auto apart = [&](int64_t heads, int64_t token, int64_t head) {
        return (d->tokens == 1 || token >= written) && (heads <= 1 || head >= written) &&
               (d->tokens == 1 || heads <= 1 || token != head);
    };
    if (!apart(d->heads, d->y_token, d->y_head) || (d->heads2 && !apart(d->heads2, d->y2_token, d->y2_head)))
        return HISA_EINVAL;
    RopeParams p{};
    p.heads = d->heads; p.heads_all = d->heads + d->heads2;
    p.rows = d->tokens * p.heads_all;
    p.D = d->D; p.dims = d->rope_dims; p.first = d->rope_first; p.half = d->half;
    p.src_bf16 = d->src_dtype == HISA_BF16; p.dst_bf16 = d->dst_dtype == HISA_BF16;
    p.inplace = inplace;
    p.mscale = d->mscale; p.sin_sign = d->inverse ? -1.f : 1.f;
    p.table = table; p.pos = pos;
    p.x = x; p.x2 = x2; p.y = y; p.y2 = y2;
    p.x_token = d->x_token; p.x_head = d->x_head; p.y_token = d->y_token; p.y_head = d->y_head;
    p.x2_token = d->x2_token; p.x2_head = d->x2_head; p.y2_token = d->y2_token; p.y2_head = d->y2_head;
    // units of 8 dims: 32 or 16 bytes at every boundary
    auto wide = [](const void *a, int64_t token, int64_t head, size_t es) {
        return aligned(a, 8 * es) && token % 8 == 0 && head % 8 == 0;
    };
    p.wide = d->D % 8 == 0 && d->rope_first % 8 == 0 && d->rope_dims % (d->half ? 16 : 8) == 0 &&
             wide(x, d->x_token, d->x_head, ss) && wide(y, d->y_token, d->y_head, sd) &&
             (!d->heads2 || (wide(x2, d->x2_token, d->x2_head, ss) && wide(y2, d->y2_token, d->y2_head, sd)));
    return from_cuda(launch_rope(p, reinterpret_cast<cudaStream_t>(stream)));
}

hisa_status hisa_prefix_attend(const hisa_prefix_desc *d, const void *q, const void *local_kv, const int32_t *local_len,
                               const int32_t *local_pos0, const void *prefix_kv, const void *pooled_kv,
                               const int64_t *kv_off, const float *sinks, const int32_t *t0, void *out, void *ws,
                               size_t ws_bytes, hisa_stream_t stream) {
    hisa_status st = check_prefix_desc(d);
    if (st != HISA_OK) return st;
    if (!q || !out || !t0) return HISA_EINVAL;
    if (d->W_max > 0 && (!local_kv || !local_len || !local_pos0)) return HISA_EINVAL;
    if (d->prefix_rows > 0 && !prefix_kv) return HISA_EINVAL;
    if (d->Np_max > 0 && (!pooled_kv || !kv_off)) return HISA_EINVAL;
    if (!aligned(q, 16) || !aligned(local_kv, 16) || !aligned(prefix_kv, 16) || !aligned(pooled_kv, 16) || !aligned(out, 16))
        return HISA_EINVAL;
    if (!aligned(local_len, 4) || !aligned(local_pos0, 4) || !aligned(kv_off, 8) || !aligned(sinks, 4) || !aligned(t0, 4))
        return HISA_EINVAL;
    if (!ws || !aligned(ws, kAlign) || ws_bytes < prefix_workspace_bytes(d)) return HISA_EWORKSPACE;
    PrefixParams p{};
    p.B = d->B; p.L = d->L; p.H = d->H; p.Dh = d->Dh; p.window = d->window; p.W_max = d->W_max; p.r = d->r;
    p.P = d->prefix_rows; p.Np_max = d->Np_max; p.kv_rows = d->kv_rows;
    p.scale = d->scale > 0.f ? d->scale : (float)(1.0 / std::sqrt((double)d->Dh));
    p.q = q; p.local_kv = local_kv; p.prefix_kv = prefix_kv; p.pooled_kv = pooled_kv;
    p.local_len = local_len; p.local_pos0 = local_pos0; p.t0 = t0; p.kv_off = kv_off; p.sinks = sinks;
    p.out = out;
    p.bf16 = d->kv_dtype == HISA_BF16; p.out_bf16 = d->out_dtype == HISA_BF16;
    prefix_plan(d, &p);
    const size_t rows = (size_t)d->B * d->L * d->H, seg = prefix_parts(d, p);
    char *base = static_cast<char *>(ws) + kStatusBytes;
    p.part_o = reinterpret_cast<float *>(base);
    p.part_ml = reinterpret_cast<float *>(base + round_up(seg * rows * d->Dh * sizeof(float)));
    p.status = static_cast<uint32_t *>(ws);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (prefix_tc_supported(p.H, p.Dh, p.bf16)) {
        e = launch_prefix_tc(p, s);
        if (p.pre_split == 1) return from_cuda(e);
    } else {
        if (p.tail_split) e = launch_prefix_simt(p, 1, s);
        if (e == cudaSuccess && p.pre_split) e = p.bf16 ? launch_prefix_tc1(p, s) : launch_prefix_simt(p, 0, s);
    }
    if (e == cudaSuccess) e = launch_prefix_merge(p, s);
    return from_cuda(e);
}

}  // extern "C"
