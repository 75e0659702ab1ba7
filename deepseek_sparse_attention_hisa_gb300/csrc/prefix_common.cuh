// What the kernels of the shared-prefix combine share: which rows of its own a query row sees, and
// the pieces of a softmax over logits in TMEM.
#pragma once

#include "ops_internal.cuh"
#include "tc_ptx.cuh"

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

namespace tc {

// A bounded wait by a whole warp; the common case is a barrier that has completed.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort) {
    const bool v = mbar_try_wait(bar, parity) || mbar_wait_abortable(bar, parity, abort);
    return __all_sync(0xffffffffu, v);
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
                 "%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
                   "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                   "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ float ex2(float x) {         // 2^x, relative error <= 2^-22; -inf -> +0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// True on the 64 threads of a named barrier iff v is true on all of them (a barrier itself).
__device__ __forceinline__ bool pair_all(uint32_t id, bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, 64, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"((uint32_t)v), "r"(id) : "memory");
    return r != 0u;
}

}  // namespace tc
}  // namespace hisa
