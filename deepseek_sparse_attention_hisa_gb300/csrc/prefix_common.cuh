// What the kernels of the shared-prefix combine share: which rows of its own a query row sees.
#pragma once

#include "ops_internal.cuh"

namespace hisa {

// The visible part of query row q's own list: local rows [lo, lo + nloc) of its window buffer,
// then own pooled rows [0, nown).
struct Tail {
    int64_t lo, nloc, k0, nown;
};
__device__ __forceinline__ Tail tail_of(const PrefixParams &p, int row, bool report) {
    const int b = row / p.L, j = row - b * p.L;
    const int64_t t = (int64_t)p.t0[b] + j;
    Tail x{0, 0, 0, 0};
    int64_t nl = p.W_max > 0 ? p.local_len[b] : 0;
    nl = nl < 0 ? 0 : (nl > p.W_max ? p.W_max : nl);
    if (nl > 0) {
        const int64_t pos0 = p.local_pos0[b];
        int64_t lo = t - p.window + 1 - pos0, hi = t - pos0 + 1;
        lo = lo < 0 ? 0 : lo;
        hi = hi > nl ? nl : hi;
        x.lo = lo;
        x.nloc = hi > lo ? hi - lo : 0;
    }
    if (p.Np_max > 0) {
        if (seq_ok(p.kv_off, b, p.Np_max, p.kv_rows)) {
            x.k0 = p.kv_off[b];
            x.nown = p.kv_off[b + 1] - x.k0;
            if (p.L > 1) {
                const int64_t v = visible_len(t, p.r, p.P + x.nown) - p.P;
                x.nown = v < 0 ? 0 : (v < x.nown ? v : x.nown);
            }
        } else if (report) {
            flag(p.status, HISA_DEV_BAD_OFFSETS);
        }
    }
    return x;
}

}  // namespace hisa
