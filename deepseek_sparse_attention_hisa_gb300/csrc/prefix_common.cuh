// What the kernels of the shared-prefix combine share: which rows of its own a query row sees.
#pragma once

#include "ops_internal.cuh"

namespace hisa {

// A sequence's numbers, fetched together (one round trip to memory, whatever is then made of them).
struct TailIn {
    int64_t k0, k1, t0, len, pos0;
};
__device__ __forceinline__ TailIn tail_fetch(const PrefixParams &p, int row) {
    const int b = row / p.L;
    TailIn x{0, 0, 0, 0, 0};
    x.t0 = p.t0[b];
    if (p.W_max > 0) {
        x.len = p.local_len[b];
        x.pos0 = p.local_pos0[b];
    }
    if (p.Np_max > 0) {
        x.k0 = p.kv_off[b];
        x.k1 = p.kv_off[b + 1];
    }
    return x;
}

// The visible part of query row q's own list: local rows [lo, lo + nloc) of its window buffer,
// then own pooled rows [0, nown) from row k0.
struct Tail {
    int64_t lo, nloc, k0, nown;
};
__device__ __forceinline__ Tail tail_of(const PrefixParams &p, int row, const TailIn &in, bool report) {
    const int64_t t = in.t0 + row % p.L;
    Tail x{0, 0, 0, 0};
    const int64_t nl = in.len < 0 ? 0 : (in.len > p.W_max ? p.W_max : in.len);
    int64_t lo = t - p.window + 1 - in.pos0, hi = t - in.pos0 + 1;
    lo = lo < 0 ? 0 : lo;
    hi = hi > nl ? nl : hi;
    if (hi > lo) {
        x.lo = lo;
        x.nloc = hi - lo;
    }
    if (seq_ok_v(in.k0, in.k1, p.Np_max, p.kv_rows)) {
        x.k0 = in.k0;
        x.nown = in.k1 - in.k0;
        if (p.L > 1) {
            const int64_t v = visible_len(t, p.r, p.P + x.nown) - p.P;
            x.nown = v < 0 ? 0 : (v < x.nown ? v : x.nown);
        }
    } else if (report) {
        flag(p.status, HISA_DEV_BAD_OFFSETS);
    }
    return x;
}

}  // namespace hisa
