// Shared-prefix combine on the tensor cores: 64 bf16 query heads of 512 dims (one KV head, K = V).
//
// The shared rows are the same for every query row of the batch, so the query rows (64 heads
// each) stack into tiles: S = Q K^T and O += P V are dense products of 4 * 512 operations per
// (stacked row, shared row), bound by the tensor cores.
//
// A pair of CTAs (a cluster of two) takes two query rows (128 stacked rows) and one segment of
// their rows. O is 128 x 512 f32, and the pair splits its rows (cta_group::2, M = 128: CTA c holds
// rows 64 c .. + 63 in 256 of its 512 TMEM columns, at the full tensor rate, which a single CTA
// with M = 64 rows halves). Per tile of kT = 64 shared rows:
//   S [128 x 64]   = Q K^T    A = Q, each CTA its 64 rows; B = K, each CTA 32 of the 64 rows
//   O [128 x 512] += P V      A = P, each CTA its 64 rows; B = V, each CTA 256 of the 512 dims
// Both CTAs must give an operand at the same shared-memory offset, so a CTA stages the 32 rows
// it gives as K and the 256 dims it gives as V separately (32 KB each), all by TMA from L2.
// With kT = 64 the first product waits for its operands in shared memory (25 instead of 16
// cycles per 16 dims: 2 KB of Q and 1 KB of K at 128 B per cycle); larger tiles leave no room
// for two stages of each operand beside the 64 KB of Q. The ceiling is so about 78 % of the
// tensor peak.
//
// The local and own pooled rows of the two query rows come last, in tiles of the same shape:
// 32 rows of each (TMA again, but for the ragged ends of the lists). S has then 64 columns of which each CTA's
// rows use the 32 of their own query row, and the two CTAs' parts of P V are issued apart, with the
// other CTA's TMEM lanes masked off, so that nothing of one sequence's rows (a NaN, say) reaches
// the other. That does half the useful work per tile, but needs no second kernel, no second read
// of Q and no sums through memory; with one segment the epilogue writes the output itself.
//
// S products run up to kSBufs tiles ahead of the PV products, so the tensor cores do not
// wait for a tile's softmax and for the two crossings between the CTAs around it. TMEM layout of
// both accumulators: lanes 0-63 hold the CTA's 64 rows for the first half of the columns, lanes
// 64-127 the same rows for the second half, so a row's logits sit with two threads of one lane
// each, which exchange their maxima through shared memory. The running maximum is lazy: O and the
// sums are rescaled only when a tile's maximum exceeds it by more than 8 (log2 units), so p <= 256.
// P is rounded to bf16 for the second product, which takes bf16 operands (2^-8 of a weight at most,
// of random sign; a second plane of the remainders would cost half the products again); sums are
// of the unrounded weights in f32.
//
// Warps of each CTA: 0-3 softmax and epilogue (thread = TMEM lane), 4 and 6 loads, 5, 7 and 8
// (of CTA 0) MMA issue for the pair. Every wait is bounded; a timeout sets HISA_DEV_TIMEOUT and
// the CTAs leave.
//
// Measured (one GB300, whole call): 304 query rows over 16384 shared and up to 512 own rows 485 us,
// 1.38 PFLOP/s (71 % of a library product's rate); 152 query rows over 65536 shared rows 835 us, 1.57;
// 4096 query rows over 8192 3.04 ms, 1.47; 64 query rows over 8191 shared rows 82 us, where 64 of 76
// pairs work and the fill, the epilogues and the merge are about 20 us of it; 3 x 2 query rows over
// 1000: 16 us, latency.
#include "prefix_common.cuh"
#include "tc_ptx.cuh"

namespace hisa {
namespace {

using namespace tc;

constexpr int kH = 64, kDH = 512, kT = 64;
constexpr int kSoftWarps = 4, kLoadWarp = 4, kMmaWarp = 5, kLoadVWarp = 6, kMmaPvWarp = 7, kMmaWarp2 = 8,
              kThreads = 288;
constexpr int kStages = 2;                              // of K, of V and of P (two: a K stage and an S buffer then
                                                        // belong to the even or the odd tiles' S warp alone, which
                                                        // sees every phase of its barriers)
constexpr int kSBufs = 4;                               // S tiles in TMEM
constexpr uint32_t kQBytes = kH * kDH * 2;              // 64 KB: 8 chunks [64 rows x 64 dims]
constexpr uint32_t kKBytes = kT / 2 * kDH * 2;          // 32 KB: 8 chunks [32 rows x 64 dims]
constexpr uint32_t kVBytes = kT * kDH;                  // 32 KB: 4 chunks [64 rows x 64 dims]
constexpr uint32_t kPBytes = kH * kT * 2;               // 8 KB: one chunk [64 rows x 64 shared rows]
constexpr uint32_t kKChunk = kT / 2 * 128, kVChunk = kT * 128, kQChunk = kH * 128;
constexpr uint32_t kOffQ = 0, kOffK = kQBytes, kOffV = kOffK + kStages * kKBytes, kOffP = kOffV + kStages * kVBytes,
                   kOffMisc = kOffP + kStages * kPBytes;
constexpr uint32_t kColO = 0, kColS = 256, kTmemCols = 512;   // O: 256 columns, S: 32 each
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f, kLazy = 8.0f;

struct Misc {
    // pair barriers, used in CTA 0: operands have landed in both CTAs; S read and P written by both
    uint64_t kfull[kStages], vfull[kStages], qfull, sfree[kSBufs], pfull[kStages], ofree;
    // each CTA's own, signalled by the MMAs of the pair
    uint64_t kempty[kStages], vempty[kStages], qfree, sfull[kSBufs], pfree[kStages], ofull, drain;
    uint32_t tmem;
    int abort;
    float mx[2][2][kH];                                 // [tile parity][column half][row]: a tile's maxima
};
constexpr uint32_t kSmemBytes = kOffMisc + sizeof(Misc) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// The shared::cluster address of `p`'s counterpart in CTA `cta` of the cluster.
__device__ __forceinline__ uint32_t map_to(const void *p, uint32_t cta) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(cta));
    return r;
}
// One arrival on a barrier of the pair. What the waiter goes on to use is its own CTA's TMEM and
// shared memory, and the counterpart's through the pair's MMAs; each writer's fence (async proxy,
// tcgen05) stands before its arrival, so no cluster-wide release is needed (it costs about 500
// cycles, as an acquire does on the waiting side).
__device__ __forceinline__ void arrive_pair(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}
// Loads a box of the chunked map; the bytes count on `bar`, which may be the other CTA's.
__device__ __forceinline__ void load_chunks(uint32_t dst, const CUtensorMap *map, int row, int chunk, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(chunk), "r"(bar) : "memory");
}
__device__ __forceinline__ void prefetch_chunks(const CUtensorMap *map, int row) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
                 :: "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(0) : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// One arrival on `bar` in both CTAs once every MMA issued so far has completed.
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
                 :: "r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}
// The same for one CTA's lanes: `other` (0 or 1) names the CTA whose TMEM lanes stay as they are.
__device__ __forceinline__ void mma_pair_masked(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, int other) {
    const uint32_t m0 = other == 0 ? 0xffffffffu : 0u, m1 = ~m0;
    asm volatile("{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%5, %5, %5, %5, %6, %6, %6, %6}, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(m0), "r"(m1) : "memory");
}
// Tensor maps of own rows (window buffers, pooled rows): boxes of kTO rows, all or half the dims.
struct Maps {
    CUtensorMap k, v;
};

// One item: a pair of query rows and an even part [a, a + tiles) of the pair's tiles, of which the
// first `shared` hold the shared rows and the others the query rows' own lists.
constexpr int kTO = kT / 2;   // own rows of each query row per tile
struct Item {
    int row[2], seg;          // query rows of CTA 0 and 1 (the second may be past the last)
    Tail tail[2];
    int shared, a, tiles;
};
// Not inlined: one copy of the code for the five warp roles that ask for it at the kernel's start, each
// of which waited about a microsecond for instructions of its own.
__device__ __noinline__ Item item_of(const PrefixParams &p, int id, bool report) {
    Item x;
    const int pairs = (p.B * p.L + 1) / 2;
    x.seg = id / pairs;
    int own = 0;
    TailIn in[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        x.row[c] = 2 * (id - x.seg * pairs) + c;
        in[c] = tail_fetch(p, x.row[c] < p.B * p.L ? x.row[c] : x.row[0]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const bool there = x.row[c] < p.B * p.L;
        x.tail[c] = tail_of(p, there ? x.row[c] : x.row[0], in[c], report && x.seg == 0 && there);
        if (!there) x.tail[c] = Tail{0, 0, 0, 0};
        const int t = (int)((x.tail[c].nloc + kTO - 1) / kTO + (x.tail[c].nown + kTO - 1) / kTO);
        own = t > own ? t : own;
    }
    x.shared = (int)((p.P + kT - 1) / kT);
    const int total = x.shared + own, q = total / p.pre_split, r = total - q * p.pre_split;
    x.a = q * x.seg + r * x.seg / p.pre_split;         // floor(total * seg / pre_split)
    x.tiles = q * (x.seg + 1) + r * (x.seg + 1) / p.pre_split - x.a;
    return x;
}
// A query row's part of own tile i: up to kTO neighbouring rows of its window buffer, then of its
// pooled rows.
struct Part {
    int64_t row;              // first row in local_kv or pooled_kv
    int count;                // 0..kTO
    bool local;
};
__device__ __forceinline__ Part part_of(const PrefixParams &p, int row, const Tail &l, int i) {
    const int64_t nl = (l.nloc + kTO - 1) / kTO;
    const bool local = i < nl;
    const int64_t at = (local ? (int64_t)i : i - nl) * kTO, n = (local ? l.nloc : l.nown) - at;
    return Part{local ? (int64_t)(row / p.L) * p.W_max + l.lo + at : l.k0 + at, (int)(n < 0 ? 0 : (n < kTO ? n : kTO)), local};
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
k_prefix_tc(PrefixParams p, int items, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
            const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Maps lmap, const __grid_constant__ Maps omap) {
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t r0 = smem_u32(raw);
    uint8_t *smem = raw + (((r0 + 1023u) & ~1023u) - r0);
    const uint32_t sbase = smem_u32(smem);
    Misc *ms = reinterpret_cast<Misc *>(smem + kOffMisc);
    volatile int *abort = &ms->abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank();
    const int first_item = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&ms->kfull[s], 2); mbar_init(&ms->vfull[s], 2);   // one arrival of each CTA's loader
            mbar_init(&ms->pfull[s], 2 * kSoftWarps);
            mbar_init(&ms->kempty[s], 1); mbar_init(&ms->vempty[s], 1);
            mbar_init(&ms->pfree[s], 1);
        }
        for (int s = 0; s < kSBufs; ++s) {
            mbar_init(&ms->sfull[s], 1); mbar_init(&ms->sfree[s], 2 * kSoftWarps);
        }
        mbar_init(&ms->qfull, 1); mbar_init(&ms->qfree, 2);   // one commit of each S warp
        mbar_init(&ms->ofree, 2 * kSoftWarps); mbar_init(&ms->ofull, 1);
        mbar_init(&ms->drain, 3);                       // one commit of each issuing warp
        mbar_fence_init();
        ms->abort = 0;
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(&ms->tmem)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    fence_before_sync();
    __syncthreads();
    cluster_sync();                                     // both CTAs' barriers and TMEM are there
    fence_after_sync();
    const uint32_t tmem = ms->tmem;
    grid_dep_wait();
    grid_dep_trigger();
    bool ok = true;
    auto fail = [&]() {
        ok = false;
        *abort = 1;
    };

    if (warp == kLoadWarp || warp == kLoadVWarp) {
        // ---------------- loads of this CTA's share: Q and K, or V ----------------
        // (two warps: K runs ahead of V by as many tiles as S runs ahead of PV)
        const bool v = warp == kLoadVWarp;
        uint64_t *full = v ? ms->vfull : ms->kfull, *empty = v ? ms->vempty : ms->kempty;
        const uint32_t bytes = v ? kVBytes : kKBytes, dst0 = sbase + (v ? kOffV : kOffK);
        const CUtensorMap *map = v ? &vmap : &kmap;
        uint32_t g = 0;
        int n = 0, pending = -1;                        // stage whose copies are on their way
        auto settle = [&](bool newer) {                 // its copies have landed; tell the MMA warps
            if (pending < 0) return;
            if (newer) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else asm volatile("cp.async.wait_group 0;" ::: "memory");
            fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive_pair(map_to(&full[pending], 0));
            pending = -1;
        };
        const int pairs = (p.B * p.L + 1) / 2;
        for (int id = first_item; id < items && ok; id += step, ++n) {
            if (!v) {
                if (n > 0 && !wait_warp(&ms->qfree, (n - 1) & 1, abort)) { fail(); break; }
                if (lane == 0) {
                    if (rank == 0) mbar_arrive_expect_tx(&ms->qfull, 2 * kQBytes);
                    load_chunks(sbase + kOffQ, &qmap, (2 * (id % pairs) + rank) * kH, 0, map_to(&ms->qfull, 0));
                }
            }
            // the cluster's first tile, where it is the first shared one whatever the lists hold: on
            // its way before the sequences' numbers are there
            const bool early = n == 0 && id < pairs && p.P >= (int64_t)kT * p.pre_split;
            if (early && lane == 0) {
                if (rank == 0) mbar_arrive_expect_tx(&full[0], 2 * bytes);
                else arrive_pair(map_to(&full[0], 0));
                load_chunks(dst0, map, v ? 0 : rank * (kT / 2), v ? rank * 4 : 0, map_to(&full[0], 0));
            }
            const Item x = item_of(p, id, false);
            if (!v) {
                // own rows come from far: ask for them in L2 while the shared rows' tiles run
                const int row = rank ? x.row[1] : x.row[0];
                const Tail mine = rank ? x.tail[1] : x.tail[0];
                for (int i = (x.a > x.shared ? x.a : x.shared) + lane; i < x.a + x.tiles; i += 32) {
                    const Part part = part_of(p, row, mine, i - x.shared);
                    if (part.count > 0) prefetch_chunks(part.local ? &lmap.k : &omap.k, (int)part.row);
                }
            }
            if (early) g = 1;
            for (int i = x.a + (early ? 1 : 0); i < x.a + x.tiles; ++i, ++g) {
                const uint32_t s = g % kStages, par = (g / kStages - 1) & 1;
                if (g >= kStages && !__all_sync(0xffffffffu, mbar_try_wait(&empty[s], par))) {
                    settle(false);
                    if (!wait_warp(&empty[s], par, abort)) { fail(); break; }
                }
                const uint32_t dst = dst0 + s * bytes;
                if (i < x.shared) {                     // shared rows
                    if (lane == 0) {
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * bytes);
                        else arrive_pair(map_to(&full[s], 0));
                        load_chunks(dst, map, i * kT + (v ? 0 : rank * (kT / 2)), v ? rank * 4 : 0,
                                    map_to(&full[s], 0));
                    }
                    settle(false);
                    continue;
                }
                // own rows: as K this CTA's 32, all dims; as V both CTAs' 32, this CTA's 256 dims. K comes
                // whole (logits of rows past a list's end are masked), and so does V where the part is
                // whole. A ragged V part is copied with zeros for the rest of its rows, since a weight
                // of zero does not silence a NaN; an empty one is not used.
                const Part part[2] = {part_of(p, x.row[0], x.tail[0], i - x.shared), part_of(p, x.row[1], x.tail[1], i - x.shared)};
                const uint32_t block = kTO * (v ? 256 : kDH) * 2;
                uint32_t tx = 0;                        // TMA bytes of both CTAs
                bool ragged = false;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const bool tma = v ? part[c].count == kTO : part[c].count > 0;
                    tx += tma ? (v ? 2 * block : block) : 0;
                    ragged |= v && part[c].count > 0 && !tma;
                    if (tma && lane == 0 && (v || c == rank)) {
                        const Maps &m = part[c].local ? lmap : omap;
                        load_chunks(dst + (v ? c * block : 0), v ? &m.v : &m.k, (int)part[c].row, v ? rank * 4 : 0,
                                    map_to(&full[s], 0));
                    }
                }
                if (rank == 0 && lane == 0) {
                    if (ragged) asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;"
                                             :: "r"(smem_u32(&full[s])), "r"(tx) : "memory");
                    else mbar_arrive_expect_tx(&full[s], tx);
                }
                if (rank == 1 && lane == 0 && !ragged) arrive_pair(map_to(&full[s], 0));
                if (!ragged) {
                    settle(false);
                    continue;
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (part[c].count == 0 || part[c].count == kTO) continue;
                    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(part[c].local ? p.local_kv : p.pooled_kv) +
                                               part[c].row * kDH + rank * 256 + lane * 8;
                    const uint32_t to = dst + c * block + (lane >> 3) * (kTO * 128);
#pragma unroll 8
                    for (int r = 0; r < kTO; ++r) {
                        const bool in = r < part[c].count;
                        cp_async16_zfill(to + sw128_offset(r, (lane & 7) * 8), in ? static_cast<const void *>(src + r * kDH) : p.q, in);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                settle(true);
                pending = (int)s;
            }
            // an item's last tile is not held back by what the next item waits for
            settle(false);
        }
        cp_async_wait_all();
        if (!ok && rank == 0 && lane == 0) {
            // copies in flight land before the CTAs leave (bounded, whatever the abort flag says)
            for (uint32_t b = g > kStages ? g - kStages : 0; b <= g; ++b)
                mbar_wait(&full[b % kStages], (b / kStages) & 1, 1u << 20);
        }
        __syncwarp();
    } else if (warp == kMmaWarp || warp == kMmaWarp2 || warp == kMmaPvWarp) {
        // ---------------- MMA issue (CTA 0, for the pair) ----------------
        // Two warps issue S = Q K^T of the even and of the odd tiles, one O += P V: a warp's waits
        // and commits (about 900 cycles a tile) hide behind the other's products. S runs ahead of
        // PV by as many tiles as it has buffers.
        if (rank == 0 && warp != kMmaPvWarp) {
            const uint32_t mine = warp == kMmaWarp2;
            const uint32_t idesc = idesc_bf16_f32(128, kT, 0, 0);
            const uint64_t qd = smem_desc_sw128(sbase + kOffQ, 16, 1024);
            uint32_t g = 0;
            int n = 0;
            for (int id = first_item; id < items && ok; id += step, ++n) {
                const Item x = item_of(p, id, false);
                if (!wait_warp(&ms->qfull, n & 1, abort)) { fail(); break; }
                for (int i = 0; i < x.tiles; ++i, ++g) {
                    if ((g & 1) != mine) continue;
                    const uint32_t s = g % kStages, b = g % kSBufs;
                    if (!wait_warp(&ms->kfull[s], (g / kStages) & 1, abort) ||
                        (g >= kSBufs && !wait_warp(&ms->sfree[b], (g / kSBufs - 1) & 1, abort))) {
                        fail();
                        break;
                    }
                    fence_after_sync();
                    const uint64_t kd = smem_desc_sw128(sbase + kOffK + s * kKBytes, 16, 1024);
                    const uint32_t d = tmem + kColS + b * (kT / 2);
#pragma unroll
                    for (int ks = 0; ks < kDH / 16; ++ks)
                        mma_pair(d, desc_add(qd, (ks >> 2) * kQChunk + (ks & 3) * 32),
                                 desc_add(kd, (ks >> 2) * kKChunk + (ks & 3) * 32), idesc, ks > 0);
                    commit_pair(&ms->sfull[b]);
                    commit_pair(&ms->kempty[s]);
                }
                if (ok) commit_pair(&ms->qfree);
            }
        } else if (rank == 0) {
            const uint32_t idesc = idesc_bf16_f32(128, 256, 0, 1);
            uint32_t g = 0;
            int n = 0;
            for (int id = first_item; id < items && ok; id += step, ++n) {
                const Item x = item_of(p, id, false);
                bool started[2] = {false, false};       // whether the CTA's lanes of O hold sums yet
                // O starts over once the epilogues have read the item before
                if (n > 0 && !wait_warp(&ms->ofree, (n - 1) & 1, abort)) { fail(); break; }
                for (int i = 0; i < x.tiles; ++i, ++g) {
                    const uint32_t s = g % kStages;
                    if (!wait_warp(&ms->vfull[s], (g / kStages) & 1, abort) ||
                        !wait_warp(&ms->pfull[s], (g / kStages) & 1, abort)) {
                        fail();
                        break;
                    }
                    fence_after_sync();
                    const uint64_t pd = smem_desc_sw128(sbase + kOffP + s * kPBytes, 16, 1024);
                    const uint64_t vd = smem_desc_sw128(sbase + kOffV + s * kVBytes, kVChunk, 1024);
                    if (x.a + i < x.shared) {
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int ks = 0; ks < kT / 16; ++ks)
                                mma_pair(tmem + kColO + m * 128, desc_add(pd, ks * 32),
                                         desc_add(vd, m * 2 * kVChunk + ks * 2048), idesc, (ks > 0 || i > 0) ? 1u : 0u);
                        started[0] = started[1] = true;   // (these tiles come first)
                    } else {
                        // a block of 32 rows for each CTA, each onto that CTA's own lanes alone
                        const uint64_t od = smem_desc_sw128(sbase + kOffV + s * kVBytes, kTO * 128, 1024);
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int count = part_of(p, x.row[c], x.tail[c], x.a + i - x.shared).count;
                            if (count == 0) continue;
#pragma unroll
                            for (int m = 0; m < 2; ++m)
#pragma unroll
                                for (int ks = 0; ks < kTO / 16; ++ks)
                                    mma_pair_masked(tmem + kColO + m * 128, desc_add(pd, (c * 2 + ks) * 32),
                                                    desc_add(od, c * (kVBytes / 2) + m * 2 * (kTO * 128) + ks * 2048), idesc,
                                                    (ks > 0 || started[c]) ? 1u : 0u, 1 - c);
                            started[c] = true;
                        }
                    }
                    commit_pair(&ms->vempty[s]);
                    commit_pair(&ms->pfree[s]);
                }
                if (ok) commit_pair(&ms->ofull);
            }
        }
        if (rank == 0) commit_pair(&ms->drain);
        __syncwarp();
    } else {
        // ---------------- softmax and epilogue: thread = TMEM lane ----------------
        const int r = (warp & 1) * 32 + lane, half = warp >> 1;
        const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
        const float c2 = p.scale * kLog2e;
        const uint32_t pairbar = 1 + (warp & 1);        // the two warps that share 32 rows
        uint32_t g = 0;
        int n = 0;
        bool good = true;                               // no wait of this warp has run out; both warps of a
                                                        // pair leave at the same barrier
        Item x = item_of(p, first_item, tid == 0 && rank == 0), next = x;
        for (int id = first_item; id < items && ok; id += step, ++n, x = next) {
            const int row = rank ? x.row[1] : x.row[0];
            const Tail mine = rank ? x.tail[1] : x.tail[0];
            float m2 = -INFINITY, l = 0.f;
            for (int i = 0; i < x.tiles; ++i, ++g) {
                const uint32_t s = g % kStages, par = (g / kStages) & 1, sb = g % kSBufs;
                good = good && wait_warp(&ms->sfull[sb], (g / kSBufs) & 1, abort);
                fence_after_sync();
                float v[32];
                tmem_ld32(lanes + kColS + sb * (kT / 2), v);
                fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive_pair(map_to(&ms->sfree[sb], 0));
                // how many of this thread's 32 columns are rows that it sees
                const int ti = x.a + i;
                const int64_t seen = ti < x.shared ? p.P - (int64_t)ti * kT - half * kTO
                                     : half == rank ? part_of(p, row, mine, ti - x.shared).count : 0;
                const int left = seen < 32 ? (int)seen : 32;
                if (left < 32) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = k < left ? v[k] : -INFINITY;
                }
                float mx[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) mx[k] = fmaxf(v[k], v[k + 16]);
#pragma unroll
                for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
                    for (int k = 0; k < w; ++k) mx[k] = fmaxf(mx[k], mx[k + w]);
                ms->mx[g & 1][half][r] = mx[0];
                if (!pair_all(pairbar, good)) { fail(); break; }
                const float tmax = fmaxf(mx[0], ms->mx[g & 1][half ^ 1][r]) * c2;   // c2 > 0
                float alpha = 1.f;
                if (tmax > m2 + kLazy) {
                    alpha = ex2(m2 - tmax);             // first tile: 2^-inf = 0, and nothing to rescale
                    m2 = tmax;
                }
                const float ref = m2 == -INFINITY ? 0.f : m2;
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = ex2(fmaf(v[k], c2, -ref));
                uint32_t u[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
                    u[k] = *reinterpret_cast<const uint32_t *>(&b);
                }
#pragma unroll
                for (int w = 16; w >= 1; w >>= 1)
#pragma unroll
                    for (int k = 0; k < w; ++k) v[k] += v[k + w];
                l = l * alpha + v[0];
                // the P buffer's last reader, and for a rescale every product so far, has completed
                if (g >= kStages) good = good && wait_warp(&ms->pfree[s], par ^ 1, abort);
                if (__any_sync(0xffffffffu, alpha != 1.f) && i > 0) {
                    good = good && wait_warp(&ms->pfree[(g - 1) % kStages], ((g - 1) / kStages) & 1, abort);
                    fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < 256; c += 16) {
                        float o[16];
                        tmem_ld16(lanes + kColO + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] *= alpha;
                        tmem_st16(lanes + kColO + c, o);
                    }
                    tmem_st_wait();
                }
                uint8_t *pb = smem + kOffP + s * kPBytes;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<uint4 *>(pb + sw128_offset(r, half * 32 + k * 8)) =
                        make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
                fence_async_smem();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive_pair(map_to(&ms->pfull[s], 0));
            }
            if (!ok) break;
            if (id + step < items) next = item_of(p, id + step, tid == 0 && rank == 0);   // while the last products run
            good = good && wait_warp(&ms->ofull, n & 1, abort);
            fence_after_sync();
            // the row's sum joins over its two threads
            ms->mx[g & 1][half][r] = l;
            if (!pair_all(pairbar, good)) { fail(); break; }
            l += ms->mx[g & 1][half ^ 1][r];
            asm volatile("bar.sync %0, 64;" ::"r"(pairbar) : "memory");
            const bool there = row < p.B * p.L, some = !(m2 == -INFINITY && l == 0.f);   // a row was seen
            const int64_t rows = (int64_t)p.B * p.L * kH, g0 = (int64_t)row * kH + r;
            float f = 1.f;                              // with one segment: the output's scale
            if (p.pre_split == 1) {
                const float sink2 = p.sinks ? p.sinks[r] * kLog2e : -INFINITY;
                const float top = fmaxf(m2, sink2), ref = top == -INFINITY ? 0.f : top;
                const float w = exp2f(m2 - ref), den = l * w + exp2f(sink2 - ref);
                f = den == 0.f ? 0.f : w / den;         // nothing visible, no sink: 0
            }
            const int64_t at = (int64_t)x.seg * rows + g0;
            if (there && half == 0 && p.pre_split > 1)
                *reinterpret_cast<float2 *>(p.part_ml + at * 2) = make_float2(m2 * kLn2, l);
            // O goes out 128 bytes of each row at a time through shared memory (P's buffers are free):
            // the two warps of 32 rows put their 64 (row, half) pieces there and write them to memory
            // with eight neighbouring lanes per piece. They use the 4 KB of each P buffer that holds
            // their own 32 rows: the CTA's other two warps may be at the next item's P already.
            const bool to_bf16 = p.pre_split == 1 && p.out_bf16;
            uint8_t *out = p.pre_split > 1 ? reinterpret_cast<uint8_t *>(p.part_o + (int64_t)x.seg * rows * kDH)
                                           : static_cast<uint8_t *>(p.out);
            const int es = to_bf16 ? 2 : 4, dims = 128 / es;
            uint8_t *stage = smem + kOffP + (warp & 1) * (kPBytes / 2);
            auto piece_at = [&](int e) { return stage + (e >> 5) * kPBytes + (e & 31) * 128; };
            const int piece = half * 32 + lane, t64 = half * 32 + lane;
#pragma unroll 1
            for (int c = 0; c < 256; c += dims) {
                float o[32];
                tmem_ld32(lanes + kColO + c, o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = some ? o[k] * f : 0.f;
                if (to_bf16) {
                    float o2[32];
                    tmem_ld32(lanes + kColO + c + 32, o2);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o2[k] = some ? o2[k] * f : 0.f;
                    uint32_t u[32];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(o[2 * k], o[2 * k + 1]),
                                             b2 = __floats2bfloat162_rn(o2[2 * k], o2[2 * k + 1]);
                        u[k] = *reinterpret_cast<const uint32_t *>(&b);
                        u[16 + k] = *reinterpret_cast<const uint32_t *>(&b2);
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4 *>(piece_at(piece) + ((k ^ (piece & 7)) << 4)) =
                            make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<float4 *>(piece_at(piece) + ((k ^ (piece & 7)) << 4)) =
                            make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                }
                asm volatile("bar.sync %0, 64;" ::"r"(pairbar) : "memory");
                if (there) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int e = (t64 >> 3) + 8 * j, u = t64 & 7;            // piece, 16-byte unit
                        const int64_t g = (int64_t)row * kH + (warp & 1) * 32 + (e & 31);
                        *reinterpret_cast<uint4 *>(out + (g * kDH + (e >> 5) * 256 + c) * es + u * 16) =
                            *reinterpret_cast<const uint4 *>(piece_at(e) + ((u ^ (e & 7)) << 4));
                    }
                }
                asm volatile("bar.sync %0, 64;" ::"r"(pairbar) : "memory");
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive_pair(map_to(&ms->ofree, 0));
        }
    }
    if (!ok) flag(p.status, HISA_DEV_TIMEOUT);
    fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        // MMAs in flight end, and their arrivals reach both CTAs, before TMEM is freed and a CTA leaves
        // (bounded, whatever the abort flag says; begun only now, since CTA 1's issuing warps have
        // nothing to do and a wait from their start would run out in a call of a quarter second)
        mbar_wait(&ms->drain, 0, 1u << 24);
        __syncwarp();
    }
    cluster_sync();                                     // no CTA leaves while the other may signal it
    if (warp == kMmaWarp) {
        fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(kTmemCols) : "memory");
    }
}

}  // namespace

bool prefix_tc_supported(int H, int Dh, int bf16) { return H == kH && Dh == kDH && bf16; }

cudaError_t launch_prefix_tc(const PrefixParams &p, cudaStream_t s) {
    const cudaError_t attr = smem_attr_once<k_prefix_tc>((int)kSmemBytes);
    if (attr != cudaSuccess) return attr;
    const int sms = device_sm_count();
    if (sms < 2) return cudaErrorInvalidDevice;
    CUtensorMap qmap, kmap, vmap;
    const uint64_t qrows = (uint64_t)p.B * p.L * kH;
    const void *pre = p.P > 0 ? p.prefix_kv : p.q;
    const uint64_t pre_rows = p.P > 0 ? (uint64_t)p.P : qrows;
    if (!encode_bf16_chunks(&qmap, p.q, qrows, kDH, kH, 8) ||
        !encode_bf16_chunks(&kmap, pre, pre_rows, kDH, kT / 2, 8) || !encode_bf16_chunks(&vmap, pre, pre_rows, kDH, kT, 4))
        return cudaErrorInvalidValue;
    // a map has rows: an array that is not there is never loaded from
    Maps lmap, omap;
    const void *loc = p.W_max > 0 ? p.local_kv : p.q, *own = p.kv_rows > 0 && p.pooled_kv ? p.pooled_kv : p.q;
    const uint64_t loc_rows = p.W_max > 0 ? (uint64_t)p.B * p.W_max : qrows;
    const uint64_t own_rows = p.kv_rows > 0 && p.pooled_kv ? (uint64_t)p.kv_rows : qrows;
    if (!encode_bf16_chunks(&lmap.k, loc, loc_rows, kDH, kTO, 8) || !encode_bf16_chunks(&lmap.v, loc, loc_rows, kDH, kTO, 4) ||
        !encode_bf16_chunks(&omap.k, own, own_rows, kDH, kTO, 8) || !encode_bf16_chunks(&omap.v, own, own_rows, kDH, kTO, 4))
        return cudaErrorInvalidValue;
    const int items = (p.B * p.L + 1) / 2 * p.pre_split;
    const int pairs = items < sms / 2 ? items : sms / 2;
    return launch_pdl(k_prefix_tc, dim3((unsigned)(2 * pairs)), dim3(kThreads), kSmemBytes, s, 1, p, items, qmap, kmap, vmap, lmap, omap);
}

}  // namespace hisa
