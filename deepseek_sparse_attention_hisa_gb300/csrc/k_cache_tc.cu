// Combine over a cache in pages on the tensor cores: 64 bf16 query heads of 512 dims, K = V, pooled rows in 4 bits or
// bf16.
//
// A query row's list (its visible window, then the pooled rows it sees) is cut into tiles of 48 rows, all
// of one kind. Per tile:
//   S  = Q . K^T      tcgen05, M = 64 heads, N = 48 rows, K = 512           (TMEM; bf16 out: 2 buffers, f32 out: 4 sums)
//   P  = exp2(S scale log2e - m) per head, in the threads that own the head's TMEM lane
//   O^T += V^T . P^T  tcgen05, M = 128 dims x 4, N = 64 heads, K = 48       (TMEM, f32)
// The tile is staged once in bf16 (128-byte swizzle): K-major for the first product, MN-major for the
// second.
//
// Rows in 4 bits become bf16 on their way into the tile, exactly: a 4-bit float has 2 significant bits, its scale 4, the
// product 6 of bf16's 8. A code's three magnitude bits placed at the end of bf16's exponent and the start of its
// mantissa are the code times 2^-126 (its 0.5 a subnormal number), so a product with the scale times 2^118 leaves code *
// scale * 2^-8; the 2^8 and the cache's factor go into the logits and into P. Two dims take a byte permute, a shift, two
// masks and the product.
//
// Work: one CTA per SM. Lists differ in length and only the device knows them, so every CTA adds up all rows' tiles and
// takes an equal span of them (p.whole: whole rows in turn, where all lists are as long). A row that lies in one span is
// finished there; the sums of one that is cut go to memory, two places per CTA, and k_cache_join adds them up.
//
// The tensor core cuts its f32 sums off, by 1.8e-8 of a sum per product step in the mean, always towards zero: an output in
// f32 would lose 8e-6 over 3000 rows in one span and 4e-4 over 200000. Its sums therefore move to memory every 16 tiles
// and are added up there with rounding: 2.1e-6 to 2.6e-6 whatever the length. Every 8 tiles would give 1.2e-6 to 1.5e-6, but
// 64 rows over up to 16384 take 239 us instead of 220 then and 304 over 512 selected 94 instead of 83 (202 and 80 if they
// never moved). An output in bf16 takes a third of the steps and is rounded by up to 2^-8 in the end: its sums stay (2e-4
// over 200000 rows in one span).
//
// An output in f32 takes all of a weight: P goes to the second product as three bf16 planes (the rounded value, the
// rounding of what that leaves, and again), one after the other through the same buffer; two would leave 2^-18 of a
// weight out. And its logits are sums of four accumulators of 128 dims: the tensor core cuts its f32 sums off instead of
// rounding them, which adds up over the 32 steps of one. Outputs over 8 to 175 rows are 1.6e-6 to 1.9e-6 of their norm
// off with one accumulator, 0.7e-6 to 1.1e-6 with two, 0.9e-6 to 1.2e-6 with four; those over 512 rows and a window
// in one span up to 2.6e-6, most of it from the second product's sums, for which there is no room (f32 sums of the
// plain formula: 0.5e-6 to 1e-6). 64 rows over up to 16384: 220 us, and 125 us with a bf16 output; 304 over 512
// selected: 83 and 51. An output in bf16 takes the rounded value alone, and its normaliser adds up the rounded values
// too: what a large weight is off by then divides out (an output is 1.9e-3 to 2.0e-3 of its norm off, 2.3e-3 with a
// normaliser of unrounded weights; the output's own rounding is 1.7e-3).
//
// The running maximum m is lazy: O^T and l are rescaled only when a tile's maximum exceeds m by more than 32 (log2
// units). bf16 has the exponents of f32, so a weight of 2^32 is held as exactly as one of 1, and its products and sums
// stay far below 2^127; a rescaling costs as much as a tile.
//
// Bound by latency chains, not by a pipe: a tile takes 2600 cycles, of which the tensor core works 940, the row warps'
// conversion of it 1800 (and 850 of waits), the softmax 1800; with two tiles under way neither hides the other wholly.
// 64 rows over up to 16384: 125 us (runs of one program 116 to 135), 567 TFLOP/s, 36 % of the tensor pipe, 2.2
// instructions per cycle. Without the conversion and half of the products it still takes 111 us. 304 rows over 512
// selected (a row per CTA, twice): 51 us, 2.4 TB/s, of which a CTA's first tile, last tile and output take some 8 us per
// row.
//
// Warps: 0-7 softmax and epilogue, 8 S issue (and q by TMA), 9 PV issue, 10-11 places of the rows (ids, pages), up to
// four tiles ahead, 12-23 rows: a lane has a row of the tile and an eighth of its dims, the next tile's codes on their
// way while it writes this one's. Every wait is bounded; a timeout sets HISA_DEV_TIMEOUT and the CTA leaves.
#include "cache_cuts.h"
#include "cache_internal.cuh"
#include "prefix_common.cuh"

namespace hisa {
namespace {

using namespace tc;

constexpr int kH = 64, kDH = 512, kT = kCacheTile;      // heads, dims, rows of a tile
constexpr int kSoftWarps = 8, kSWarp = 8, kPvWarp = 9, kIndexWarp0 = 10, kRowWarp0 = 12, kRowWarps = kT / 4;
constexpr int kThreads = 32 * (kRowWarp0 + kRowWarps);
constexpr int kSlots = 3, kPlaces = 8;                   // staged tiles; tiles whose rows' places are known
constexpr uint32_t kChunk = kT * 128;                   // 64 dims of a tile, 128-byte swizzle
constexpr uint32_t kTile = 8 * kChunk;
constexpr uint32_t kQChunk = kH * 128, kQBytes = 8 * kQChunk, kPBytes = kH * 128;
constexpr uint32_t kOffQ = 0, kOffKV = kQBytes, kOffP = kOffKV + kSlots * kTile, kOffMisc = kOffP + kPBytes;
constexpr uint32_t kColS = 0, kSCols = 64, kColO = 4 * kSCols, kTmemCols = 512;
constexpr int kC = kT / 4;                               // tile rows of a softmax thread
constexpr float kLog2e = 1.4426950408889634f, kLazy = 32.0f;
constexpr int kBarSoft = 1;

struct Misc {
    uint64_t qfull, qfree, full[kSlots], empty[kSlots], sfull[2], sfree[2], pfull, pfree, ofull, ofree, drain;
    uint64_t ifull[kPlaces], ifree[kPlaces];
    int64_t place[kPlaces][kT];                         // row of local_kv or of the pool; -1: not seen
    uint64_t mask[kPlaces];                             // rows of a tile that are seen
    int kind[kPlaces];                                  // TileKind
    uint32_t tmem;
    int abort;
    int t0, groups;                                     // the span: first tile of its first row; CTAs that have one
    int64_t row, left, total;                           // first row, tiles; all rows' tiles
    int64_t sums[kThreads / 32];
    float alpha[kH];
    float top[4][kH], sum[4][kH];                       // of the four threads of a head
    __align__(16) float factor[kH], back[kH];            // back: of the carried sums, which refer to the maximum base
    float base[kH];
};
constexpr uint32_t kSmemBytes = kOffMisc + sizeof(Misc) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
static_assert(sizeof(Cut) == kCutBytes, "workspace layout");

__device__ __forceinline__ int local_tiles(const CacheRow &x) { return (x.nloc + kT - 1) / kT; }
__device__ __forceinline__ int tiles_of(const CacheRow &x) {
    const int n = local_tiles(x) + (x.npool + kT - 1) / kT;
    return n > 0 ? n : 1;                               // a row that sees nothing has a tile of nothing
}

// What a CTA does, in order: items, each a range of one query row's tiles.
struct Walk {
    int64_t row, left;
    int t0;
};
struct Item {
    CacheRow x;
    int nl, T, tiles;                                   // local tiles of the row; tiles here, tiles of the row
};
__device__ __forceinline__ Walk walk_start(const Misc *m) { return {m->row, m->left, m->t0}; }
__device__ __forceinline__ bool walk_item(const CacheAttnParams &p, const Walk &w, Item &it) {
    if (w.left <= 0 || w.row >= (int64_t)p.B * p.L) return false;
    it.x = cache_row(p, w.row, false);
    it.nl = local_tiles(it.x);
    it.tiles = tiles_of(it.x);
    const int64_t n = it.tiles - w.t0;
    it.T = (int)(n < w.left ? n : w.left);
    return true;
}
__device__ __forceinline__ void walk_next(const CacheAttnParams &p, Walk &w, const Item &it) {
    if (p.whole) {
        w.row += gridDim.x;
        return;
    }
    w.left -= it.T;
    w.row += 1;
    w.t0 = 0;
}

__device__ __forceinline__ void tma_q(uint32_t dst, const CUtensorMap *map, int32_t row, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(0), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void prefetch_q(const CUtensorMap *map, int32_t row) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
                 :: "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(0) : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0], %1;\n\t}" :: "r"(smem_u32(bar)), "r"(n) : "memory");
}
// Barriers of the softmax warps: true on all iff v is on one (any), on all (all).
__device__ __forceinline__ bool soft_any(bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"((uint32_t)v), "n"(kBarSoft), "n"(32 * kSoftWarps) : "memory");
    return r != 0u;
}
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync %0, %1;" :: "n"(kBarSoft), "n"(32 * kSoftWarps) : "memory"); }
__device__ __forceinline__ bool soft_all(bool v) { return !soft_any(!v); }

// Lanes 0-15 read columns [c, c + 12) of TMEM lanes base + 0 .. 15, lanes 16-31 columns [c + 12, c + 24) of
// the same ones (an M = 64 accumulator's rows live in lanes 0-15 of each quadrant).
__device__ __forceinline__ void tmem_ld12_x2(uint32_t addr, float (&v)[12]) {
    uint32_t r[12];
    asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%12], 12;\n\t"
                 "tcgen05.ld.sync.aligned.16x32bx2.x4.b32 {%8,%9,%10,%11}, [%13], 12;"
                 : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]), "=&r"(r[8]),
                   "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11])
                 : "r"(addr), "r"(addr + 8));
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 12; ++i) v[i] = __uint_as_float(r[i]);
}

// Eight codes times a scale (as bf16, times 2^118, in both halves of s), in bf16, times 2^-8.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint4 codes_to_bf16(uint32_t w, uint32_t s) {
    const uint32_t even = w << 4;
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {                       // the even dim's code at bit 12, the odd one's at bit 28
        const uint32_t u = __byte_perm(w, even, (4 + j) | (4 + j) << 4 | j << 8 | j << 12);
        r[j] = mul_bf16x2((u >> 6 & 0x01c001c0u) | (u & 0x80008000u), s);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
// Two scales of type e4m3, each as such a bf16 pair.
__device__ __forceinline__ uint2 scales_to_bf16(uint32_t two) {
    uint32_t h;
    asm("{.reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(h) : "r"(two));
    float a, b;
    asm("{.reg .b16 x, y; mov.b32 {x, y}, %2; cvt.f32.f16 %0, x; cvt.f32.f16 %1, y;}" : "=f"(a), "=f"(b) : "r"(h));
    const float up = 0x1p118f;
    uint2 r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(r.x) : "f"(a * up));
    asm("cvt.rn.bf16x2.f32 %0, %1, %1;" : "=r"(r.y) : "f"(b * up));
    return r;
}

// One elected lane of a warp (the same one every time).
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}
// The product of mma_bf16_warp, issued by the lane that holds e = 1. A descriptor is passed as its two words, of
// which only the lower (the address) changes from product to product, and the lane is elected once: with an
// election and two 64-bit sums for each, the issuing warp and not the tensor core sets the pace (39 cycles a product).
__device__ __forceinline__ void mma_elected(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                            uint32_t accumulate, uint32_t e) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
                 "setp.ne.u32 p, %6, 0;\n\tsetp.ne.u32 q, %7, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}"
                 :: "r"(d), "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(e) : "memory");
}

enum TileKind : int { kEnd = 0, kLocal = 1, kPool = 2 };
struct Codes {                                           // of 64 dims
    uint4 c[2];
    uint32_t s;
};
__device__ __forceinline__ void load32(const uint8_t *from, uint4 &a, uint4 &b) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w) : "l"(from));
}

// A list's sums so far, carried in memory: those in TMEM are put there, added to them, or take them up at the list's end. back: what a
// head's carried sums are to be multiplied by. A softmax thread has its own part, four heads of a dim per access. A call, so
// that its registers are not those of every tile.
enum CarryStep : int { kPut, kAdd, kJoin };
template <int STEP>
__device__ __noinline__ void carry_sums(float *carry, const float *back, uint32_t tmem_o) {
    const int side = threadIdx.x >> 7;
#pragma unroll 1
    for (int c = 0; c < 2 * kH; c += 16) {
        float4 *at = reinterpret_cast<float4 *>(carry + blockIdx.x * kCarryFloats) + c / 4 * (32 * kSoftWarps) + threadIdx.x;
        float4 was[4];
        if (STEP != kPut) {
#pragma unroll
            for (int q = 0; q < 4; ++q) was[q] = __ldcg(at + q * (32 * kSoftWarps));
        }
        float o[16];
        tmem_ld16(tmem_o + 2 * kH * side + c, o);
        tmem_ld_wait();
        if (STEP != kPut) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 f = *reinterpret_cast<const float4 *>(back + (c & (kH - 1)) + 4 * q);
                o[4 * q] = fmaf(was[q].x, f.x, o[4 * q]);
                o[4 * q + 1] = fmaf(was[q].y, f.y, o[4 * q + 1]);
                o[4 * q + 2] = fmaf(was[q].z, f.z, o[4 * q + 2]);
                o[4 * q + 3] = fmaf(was[q].w, f.w, o[4 * q + 3]);
            }
        }
        if (STEP != kJoin) {
#pragma unroll
            for (int q = 0; q < 4; ++q) __stcg(at + q * (32 * kSoftWarps), make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]));
        } else {
            tmem_st16(tmem_o + 2 * kH * side + c, o);
        }
    }
    if (STEP == kJoin) tmem_st_wait();
}
__device__ __forceinline__ float rescaled(float from, float to) { return from == to ? 1.f : ex2(from - to); }   // both -inf: sums of nothing

template <bool BITS4, bool OUT32>
__global__ void __launch_bounds__(kThreads, 1) k_cache_tc(const __grid_constant__ CUtensorMap qmap, CacheAttnParams p) {
    constexpr int kPlanes = OUT32 ? 3 : 1;               // of P
    constexpr int kSums = OUT32 ? 4 : 1, kBufs = OUT32 ? 1 : 2;   // accumulators of a logit; S buffers
    constexpr int kCarry = kCacheCarry;                  // tiles after which sums move (OUT32)
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = smem_u32(smem);
    Misc *misc = reinterpret_cast<Misc *>(smem + kOffMisc);
    volatile int *abort = &misc->abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Cut *cuts = reinterpret_cast<Cut *>(p.cuts);

    if (tid == 0) {
        mbar_init(&misc->qfull, 1);
        mbar_init(&misc->qfree, 1);
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&misc->full[i], 32 * kRowWarps);
            mbar_init(&misc->empty[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&misc->sfull[i], 1);
            mbar_init(&misc->sfree[i], kSoftWarps);
        }
        mbar_init(&misc->pfull, kSoftWarps);
        mbar_init(&misc->pfree, 1);
        for (int i = 0; i < kPlaces; ++i) {
            mbar_init(&misc->ifull[i], 2);
            mbar_init(&misc->ifree[i], kRowWarps + kSoftWarps);
        }
        mbar_init(&misc->ofull, 1);
        mbar_init(&misc->ofree, kSoftWarps);
        mbar_init(&misc->drain, 2);                      // one commit from each issuing warp
        mbar_fence_init();
        misc->abort = 0;
    }
    if (warp == kSWarp) {
        tmem_alloc(&misc->tmem, kTmemCols);
        tmem_relinquish();
    }
    grid_dep_wait();
    grid_dep_trigger();
    const int64_t rows = (int64_t)p.B * p.L;
    if (p.whole) {
        if (tid == 0) {
            misc->row = blockIdx.x;
            misc->left = INT64_MAX;
            misc->t0 = 0;
            misc->groups = (int)gridDim.x;
        }
        if (blockIdx.x == 0)
            for (int64_t r = tid; r < rows; r += kThreads) cache_row(p, r, true);     // lengths that do not fit are reported
    } else {
        // every row's tiles, added up; each thread has a run of rows
        const int64_t per = (rows + kThreads - 1) / kThreads, r0 = tid * per, r1 = r0 + per < rows ? r0 + per : rows;
        int64_t sum = 0;
        for (int64_t r = r0; r < r1; ++r) sum += tiles_of(cache_row(p, r, blockIdx.x == 0));
        int64_t upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) misc->sums[warp] = upto;
        __syncthreads();
        int64_t before = lane < kThreads / 32 ? misc->sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += v;
        }
        const int64_t total = __shfl_sync(0xffffffffu, before, 31);
        before = __shfl_sync(0xffffffffu, before, warp > 0 ? warp - 1 : 0);
        if (warp == 0) before = 0;
        // Spans: a tile takes its CTA about 1.4 us, and each part that a row is cut into costs the join about 0.14 us,
        // so total tiles of R rows are done soonest by sqrt(10 total R) CTAs (one row of 20001: 21.4 us with
        // 70, 28 with 152; of 1000: 14.2 with 14). At most as many as there are tiles: none is empty.
        const float best = sqrtf(10.f * (float)total * (float)rows);
        const int64_t most = total < (int64_t)gridDim.x ? total : (int64_t)gridDim.x;
        const int groups = best < (float)most ? ((int)best < 1 ? 1 : (int)best) : (int)most, c = blockIdx.x;
        const int64_t s0 = c < groups ? span_start(c, total, groups) : total, s1 = c < groups ? span_start(c + 1, total, groups) : total;
        int64_t at = before + upto - sum;
        if (tid == 0) {
            misc->left = s1 - s0;
            misc->total = total;
            misc->groups = groups;
            if (!p.by_row) cuts[blockIdx.x].row = -1;
        }
        // by_row a thread has one row at most; its entry is cleared by the CTA that has its first tile, which alone writes it,
        // before anything can be given up
        if (p.by_row && r0 < r1 && at >= s0 && at < s1) cuts[r0].row = -1;
        if (s0 >= at && s0 < at + sum) {
            for (int64_t r = r0; r < r1; ++r) {
                const int n = per == 1 ? (int)sum : tiles_of(cache_row(p, r, false));
                if (s0 < at + n) {
                    misc->row = r;
                    misc->t0 = (int)(s0 - at);
                    break;
                }
                at += n;
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = misc->tmem;
    bool ok = true;
    auto fail = [&]() {
        ok = false;
        *abort = 1;
    };
    Walk w = walk_start(misc);
    Item it;

    if (warp >= kRowWarp0) {
        // ---------------- rows: 8 rows of each tile per two warps, a row and 64 of its dims per lane ------
        const int rw = warp - kRowWarp0, r = 8 * (rw >> 1) + (lane & 7), part = 4 * (rw & 1) + (lane >> 3), sw = r & 7;
        // the place of this lane's row of tile g
        auto fetch = [&](uint32_t g, int &kind, int64_t &place) -> bool {
            const int e = g % kPlaces;
            if (!wait_warp(&misc->ifull[e], (g / kPlaces) & 1, abort)) return false;
            kind = *reinterpret_cast<volatile int *>(&misc->kind[e]);
            place = *reinterpret_cast<volatile int64_t *>(&misc->place[e][r]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&misc->ifree[e]);
            return true;
        };
        auto load = [&](int kind, int64_t place, Codes &x) {
            x.c[0] = x.c[1] = make_uint4(0u, 0u, 0u, 0u);
            x.s = 0u;
            if (!BITS4 || kind != kPool || place < 0) return;
            const uint8_t *codes = static_cast<const uint8_t *>(p.cache) + place * (kDH / 2) + part * 32;
            if (p.cache32) {
                load32(codes, x.c[0], x.c[1]);
            } else {
                x.c[0] = reinterpret_cast<const uint4 *>(codes)[0];
                x.c[1] = reinterpret_cast<const uint4 *>(codes)[1];
            }
            x.s = reinterpret_cast<const uint32_t *>(p.scales + place * (kDH / kScaleGroup))[part];
        };
        int kind = kEnd, kind2 = kEnd;
        int64_t place = -1, place2 = -1;
        uint32_t g = 0;
        // one tile: its codes x are here, those of the next one (y) are asked for
        auto step = [&](const Codes &x, Codes &y) -> bool {
            if (kind == kEnd) return false;
            if (!fetch(g + 1, kind2, place2)) { fail(); return false; }
            load(kind2, place2, y);
            const int s = g % kSlots;
            if (g >= kSlots && !wait_warp(&misc->empty[s], ((g / kSlots) - 1) & 1, abort)) { fail(); return false; }
            const uint32_t slot = sbase + kOffKV + s * kTile + r * 128;
            if (BITS4 && kind == kPool) {
                const uint2 s0 = scales_to_bf16(x.s & 0xffffu), s1 = scales_to_bf16(x.s >> 16);
                const uint32_t cw[8] = {x.c[0].x, x.c[0].y, x.c[0].z, x.c[0].w, x.c[1].x, x.c[1].y, x.c[1].z, x.c[1].w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint4 v = codes_to_bf16(cw[k], k < 2 ? s0.x : (k < 4 ? s0.y : (k < 6 ? s1.x : s1.y)));
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                 :: "r"(slot + part * kChunk + ((k ^ sw) << 4)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_n(&misc->full[s], 32);
            } else {
                const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(kind == kLocal ? p.local_kv : p.cache);
                const bool there = place >= 0;
                const __nv_bfloat16 *row = there ? src + place * kDH : static_cast<const __nv_bfloat16 *>(p.q);
#pragma unroll
                for (int k = 0; k < 8; ++k) {            // four lanes copy 64 contiguous bytes
                    const uint32_t c = 4 * (rw & 1) + (k >> 1), u = 4 * (k & 1) + (lane >> 3);
                    cp_async16_zfill(slot + c * kChunk + ((u ^ sw) << 4), there ? row + c * 64 + u * 8 : row, there);
                }
                cp_async_arrive(&misc->full[s]);
            }
            kind = kind2;
            place = place2;
            ++g;
            return true;
        };
        Codes x, y;                                      // in turn: a copy from one to the other would wait for its loads
        if (!fetch(0, kind, place)) fail();
        load(kind, place, x);
        while (step(x, y) && step(y, x)) {}
        cp_async_wait_all();
    } else if (warp == kIndexWarp0 || warp == kIndexWarp0 + 1) {
        // ---------------- places: a row of each tile per lane; ids two tiles ahead, pages one ----------------
        const int iw = warp - kIndexWarp0, r = 32 * iw + lane;
        bool have = walk_item(p, w, it);
        int ti = 0;                                      // the next tile of the item
        int akind = kEnd, aid = -1, aV = 0, alen = 0;    // its id is on its way
        const int32_t *atable = nullptr;
        int64_t aplace = -1;
        int bkind = kEnd, bpage = -1, brest = -1;        // its page is on its way
        int64_t bplace = -1;
        auto want = [&]() {
            akind = kEnd;
            aid = -1;
            aplace = -1;
            if (!have) return;
            const int t = w.t0 + ti, b = (int)((uint32_t)w.row / (uint32_t)p.L);
            if (t < it.nl) {
                const int e = t * kT + r;
                akind = kLocal;
                if (r < kT && e < it.x.nloc) aplace = (int64_t)b * p.W_max + it.x.lo + e;
            } else {
                const int kk = (t - it.nl) * kT + r;
                akind = kPool;
                aV = (int)it.x.V;
                alen = (int)it.x.len;
                atable = p.page_table + (int64_t)b * p.table_cols;
                if (r < kT && kk < it.x.npool) aid = p.I ? p.I[w.row * p.k + kk] : kk;
            }
            if (++ti == it.T) {
                walk_next(p, w, it);
                have = walk_item(p, w, it);
                ti = 0;
            }
        };
        auto page = [&]() {
            bkind = akind;
            bplace = aplace;
            brest = -1;
            if (akind != kPool) return;
            if (aid < -1 || aid >= alen) {
                if (aid != -1) flag(p.status, HISA_DEV_BAD_ID);
            } else if (aid >= 0 && aid < aV) {
                const uint32_t at = (uint32_t)aid / (uint32_t)p.page_rows;
                brest = aid - (int)(at * (uint32_t)p.page_rows);
                bpage = atable[at];
            }
        };
        want();
        page();
        want();
        for (uint32_t g = 0;; ++g) {
            int64_t place = bplace;
            const int kind = bkind;
            if (kind == kPool && brest >= 0) {
                if (bpage < 0 || bpage >= p.pages) flag(p.status, HISA_DEV_BAD_OFFSETS);
                else place = (int64_t)bpage * p.page_rows + brest;
            }
            const int e = g % kPlaces;
            if (g >= kPlaces && !wait_warp(&misc->ifree[e], ((g / kPlaces) - 1) & 1, abort)) { fail(); break; }
            if (r < kT) misc->place[e][r] = place;
            const uint32_t seen = __ballot_sync(0xffffffffu, r < kT && place >= 0);
            if (lane == 0) {
                reinterpret_cast<uint32_t *>(&misc->mask[e])[iw] = seen;
                if (iw == 0) misc->kind[e] = kind;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&misc->ifull[e]);
            if (kind == kEnd) break;
            page();
            want();
        }
    } else if (warp == kSWarp) {
        // ---------------- S = Q . K^T of every tile; q of each item ----------------
        const uint32_t id_s = idesc_bf16_f32(64, kT, 0, 0);
        const uint64_t qdesc = smem_desc_sw128(sbase + kOffQ, 16, 1024), kdesc = smem_desc_sw128(sbase + kOffKV, 16, 1024);
        const uint32_t qlo = (uint32_t)qdesc, klo = (uint32_t)kdesc, hi = (uint32_t)(qdesc >> 32), e = elect_one();
        uint32_t g = 0;
        int n = 0;
        for (; walk_item(p, w, it); walk_next(p, w, it), ++n) {
            if (n > 0 && !wait_warp(&misc->qfree, (n - 1) & 1, abort)) { fail(); break; }
            if (lane == 0) {
                mbar_arrive_expect_tx(&misc->qfull, kQBytes);
                tma_q(sbase + kOffQ, &qmap, (int32_t)(w.row * kH), &misc->qfull);
                const int64_t row = w.row + (p.whole ? gridDim.x : 1);   // the next item's
                if (row < rows && w.left > it.T) prefetch_q(&qmap, (int32_t)(row * kH));
            }
            __syncwarp();
            if (!wait_warp(&misc->qfull, n & 1, abort)) {
                fail();
                mbar_wait(&misc->qfull, n & 1, 1u << 24); // the copy lands before the CTA leaves (bounded, whatever abort says)
                __syncwarp();
                break;
            }
            for (int i = 0; i < it.T; ++i, ++g) {
                const int s = g % kSlots, sb = g % kBufs;
                if (!wait_warp(&misc->full[s], (g / kSlots) & 1, abort) ||
                    (g >= kBufs && !wait_warp(&misc->sfree[sb], ((g / kBufs) - 1) & 1, abort))) {
                    fail();
                    break;
                }
                fence_async_smem();                       // the rows were written through the generic proxy
                fence_after_sync();
                const uint32_t kd = klo + s * (kTile >> 4), d = tmem + kColS + sb * kSCols;
                constexpr int kSteps = kDH / 16 / kSums;  // of one accumulator
#pragma unroll
                for (int ks = 0; ks < kDH / 16; ++ks) {
                    const uint32_t in = (ks & 3) * 32;
                    mma_elected(d + ks / kSteps * kSCols, qlo + (((ks >> 2) * kQChunk + in) >> 4), hi, kd + (((ks >> 2) * kChunk + in) >> 4), hi, id_s,
                                ks % kSteps > 0, e);
                }
                mma_commit_warp(&misc->sfull[sb]);
            }
            if (!ok) break;
            mma_commit_warp(&misc->qfree);
        }
        mma_commit_warp(&misc->drain);
        __syncwarp();
        mbar_wait(&misc->drain, 0, 1u << 24);             // all products done before TMEM is freed
        __syncwarp();
    } else if (warp == kPvWarp) {
        // ---------------- O^T += V^T . P^T of every tile ----------------
        const uint32_t id_o = idesc_bf16_f32(128, kH, 1, 0);
        const uint64_t vdesc = smem_desc_sw128(sbase + kOffKV, kChunk, 1024), pdesc = smem_desc_sw128(sbase + kOffP, 16, 1024);
        const uint32_t vlo = (uint32_t)vdesc, vhi = (uint32_t)(vdesc >> 32), plo = (uint32_t)pdesc, phi = (uint32_t)(pdesc >> 32);
        const uint32_t e = elect_one();
        uint32_t g = 0, np = 0;                           // np: planes of P so far
        int n = 0;
        for (; walk_item(p, w, it); walk_next(p, w, it), ++n) {
            if (n > 0 && !wait_warp(&misc->ofree, (n - 1) & 1, abort)) { fail(); break; }
            fence_after_sync();
            for (int i = 0; ok && i < it.T; ++i, ++g) {
                const int s = g % kSlots;
                const uint32_t vd = vlo + s * (kTile >> 4);
                for (int pl = 0; pl < kPlanes; ++pl, ++np) {
                    if (!wait_warp(&misc->pfull, np & 1, abort)) { fail(); break; }
                    fence_async_smem();
                    fence_after_sync();
#pragma unroll 1                                         // less code for a warp that waits most of the time: 126.3 -> 125 us
                    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                        for (int ks = 0; ks < kT / 16; ++ks)
                            mma_elected(tmem + kColO + mt * kH, vd + ((2 * mt * kChunk + ks * 2048) >> 4), vhi, plo + ((ks * 32) >> 4), phi, id_o,
                                        ks > 0 || (OUT32 ? i % kCarry : i) > 0 || pl > 0, e);
                    if (pl == kPlanes - 1) mma_commit_warp(&misc->empty[s]);
                    mma_commit_warp(&misc->pfree);
                }
            }
            if (!ok) break;
            mma_commit_warp(&misc->ofull);
        }
        mma_commit_warp(&misc->drain);
        __syncwarp();
        mbar_wait(&misc->drain, 0, 1u << 24);
        __syncwarp();
    } else {
        // ---------------- softmax and epilogue ----------------
        // S has head 16 quad + l of lane l < 16 of a TMEM quadrant. Four threads share a head: lanes l and l + 16
        // of the two warps of a quadrant, 16 tile rows each.
        const int quad = warp & 3, side = warp >> 2, h = quad * 16 + (lane & 15), part = 2 * side + (lane >> 4);
        const uint32_t quadrant = tmem + ((uint32_t)(32 * quad) << 16);
        const float sink2 = p.sinks ? p.sinks[h] * kLog2e : -INFINITY;
        const float cl = p.scale * kLog2e, gp = BITS4 ? p.g * 256.f : 1.f, lg = BITS4 ? log2f(gp) : 0.f, unf = BITS4 ? 1.f / gp : 1.f;
        uint32_t g = 0, np = 0;                           // np: planes of P so far
        int n = 0;
        bool good = true, have = walk_item(p, w, it);
        for (; have; ++n) {
            // the next item, now: its loads would otherwise stand between this one's end and its first tile
            Walk w_next = w;
            Item it_next;
            walk_next(p, w_next, it);
            have = walk_item(p, w_next, it_next);
            float m2 = -INFINITY, l = 0.f;                // l: this thread's rows
            for (int i = 0; i < it.T; ++i, ++g) {
                if (OUT32 && i > 0 && i % kCarry == 0) {
                    // the sums so far move to memory, and the next product begins anew
                    if (part == 0) {
                        if (i > kCarry) misc->back[h] = rescaled(misc->base[h], m2);
                        misc->base[h] = m2;
                    }
                    if (!soft_all(good && wait_warp(&misc->pfree, (np - 1) & 1, abort))) { fail(); break; }
                    fence_after_sync();
                    if (i == kCarry) carry_sums<kPut>(p.carry, misc->back, quadrant + kColO);
                    else carry_sums<kAdd>(p.carry, misc->back, quadrant + kColO);
                }
                const int sb = g % kBufs, e = g % kPlaces;
                const bool pool = w.t0 + i >= it.nl;
                const float c2 = pool ? cl * gp : cl;
                good = good && wait_warp(&misc->ifull[e], (g / kPlaces) & 1, abort) && wait_warp(&misc->sfull[sb], (g / kBufs) & 1, abort);
                fence_after_sync();
                const uint32_t mask = (uint32_t)(*reinterpret_cast<volatile uint64_t *>(&misc->mask[e]) >> (kC * part)) & ((1u << kC) - 1u);
                float v[kC];
                tmem_ld12_x2(quadrant + kColS + sb * kSCols + 2 * kC * side, v);
#pragma unroll
                for (int j = 1; j < kSums; ++j) {
                    float more[kC];
                    tmem_ld12_x2(quadrant + kColS + j * kSCols + 2 * kC * side, more);
#pragma unroll
                    for (int k = 0; k < kC; ++k) v[k] += more[k];
                }
                fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&misc->sfree[sb]);
                    mbar_arrive(&misc->ifree[e]);
                }
                if (mask != (1u << kC) - 1u) {            // unseen rows are staged as zeros
#pragma unroll
                    for (int k = 0; k < kC; ++k)
                        if (!((mask >> k) & 1u)) v[k] = -INFINITY;
                }
                float t4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                for (int k = 4; k < kC; ++k) t4[k & 3] = fmaxf(t4[k & 3], v[k]);
                const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * c2;
                misc->top[part][h] = top;
                if (soft_any(top > m2 + kLazy || !good)) {
                    if (!soft_all(good)) { fail(); break; }
                    const float all = fmaxf(fmaxf(misc->top[0][h], misc->top[1][h]), fmaxf(misc->top[2][h], misc->top[3][h]));
                    float alpha = 1.f;
                    if (all > m2 + kLazy) {
                        if (m2 != -INFINITY) alpha = ex2(m2 - all);
                        m2 = all;
                    }
                    l *= alpha;
                    if (part == 0) misc->alpha[h] = alpha;
                    // O^T of this item so far, after the product of the tile before
                    if (!soft_all((OUT32 ? i % kCarry : i) == 0 || wait_warp(&misc->pfree, (np - 1) & 1, abort))) { fail(); break; }
                    if ((OUT32 ? i % kCarry : i) > 0) {
                        fence_after_sync();
#pragma unroll 1
                        for (int c = 2 * kH * side; c < 2 * kH * (side + 1); c += 16) {
                            float o[16];
                            tmem_ld16(quadrant + kColO + c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int q = 0; q < 16; ++q) o[q] *= misc->alpha[(c & (kH - 1)) + q];
                            tmem_st16(quadrant + kColO + c, o);
                        }
                        tmem_st_wait();
                    }
                }
                // P f = ex2(logit - m + log2 f), so that its sum is f times theirs. ex2(-inf) = +0; m2 is finite
                // once a row of this head was seen, and logits are -inf when masked
                const float ref = (m2 == -INFINITY ? 0.f : m2) - (pool ? lg : 0.f);
                const float2 cc = make_float2(c2, c2), rr = make_float2(-ref, -ref);
                float2 sums = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < kC; k += 2) {
                    const float2 z = fma2(make_float2(v[k], v[k + 1]), cc, rr), x = make_float2(ex2(z.x), ex2(z.y));
                    if (OUT32) sums = add2(sums, x);
                    v[k] = x.x;
                    v[k + 1] = x.y;
                }
#pragma unroll
                for (int pl = 0; pl < kPlanes; ++pl) {
                    uint32_t packed[kC / 2];
#pragma unroll
                    for (int k = 0; k < kC; k += 2) {
                        const __nv_bfloat162 two = __floats2bfloat162_rn(v[k], v[k + 1]);
                        packed[k / 2] = *reinterpret_cast<const uint32_t *>(&two);
                        if (!OUT32) sums = add2(sums, __bfloat1622float2(two));
                        if (pl + 1 < kPlanes) {           // what the rounding left (an infinite weight leaves NaN, as its row is)
                            v[k] -= __low2float(two);
                            v[k + 1] -= __high2float(two);
                        }
                    }
                    // P's buffer: the product before has read it. One that never ends is met at the next
                    // tile's barrier, by all
                    good = good && (np < 1 || wait_warp(&misc->pfree, (np - 1) & 1, abort));
                    uint8_t *prow = smem + kOffP + h * 128;
#pragma unroll
                    for (int u = 0; u < kC / 4; ++u) {    // 8 bytes: four rows
                        const uint32_t at = part * (2 * kC) + 8 * u;
                        *reinterpret_cast<uint2 *>(prow + (((at >> 4) ^ (h & 7)) << 4 | (at & 8))) = make_uint2(packed[2 * u], packed[2 * u + 1]);
                    }
                    fence_async_smem();
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&misc->pfull);
                    ++np;
                }
                l += (sums.x + sums.y) * (pool ? unf : 1.f);
            }
            if (!ok) break;
            // the item's statistics; then O^T -> out, or a cut row's sums
            misc->sum[part][h] = l;
            if (!soft_all(good && wait_warp(&misc->ofull, n & 1, abort))) { fail(); break; }
            if (part == 0) {
                l = (misc->sum[0][h] + misc->sum[1][h]) + (misc->sum[2][h] + misc->sum[3][h]);
                const float M = fmaxf(m2, sink2);
                const float wm = m2 == -INFINITY ? 0.f : ex2(m2 - M);
                const float den = l * wm + (sink2 == -INFINITY ? 0.f : ex2(sink2 - M));
                misc->factor[h] = den == 0.f ? 0.f : wm / den;           // nothing seen, no sink: 0
                if (OUT32 && it.T > kCarry) misc->back[h] = rescaled(misc->base[h], m2);
            }
            soft_sync();
            fence_after_sync();
            if (OUT32 && it.T > kCarry) carry_sums<kJoin>(p.carry, misc->back, quadrant + kColO);
            const bool cut = it.T < it.tiles;
            if (!cut) {
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {             // 32 heads of 128 dims
                    const int mt = 2 * side + (k >> 1), c = 32 * (k & 1), d = mt * 128 + quad * 32 + lane;
                    float o[32];
                    tmem_ld32(quadrant + kColO + mt * kH + c, o);
#pragma unroll
                    for (int q = 0; q < 32; q += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(&misc->factor[c + q]);
                        o[q] *= f.x; o[q + 1] *= f.y; o[q + 2] *= f.z; o[q + 3] *= f.w;
                    }
                    if (!OUT32) {
                        // two dims per store: even lanes take the first sixteen heads, odd ones the others
                        const bool odd = lane & 1;
                        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + (w.row * kH + c + (odd ? 16 : 0)) * kDH + (d & ~1);
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const float mine = odd ? o[q + 16] : o[q], yours = __shfl_xor_sync(0xffffffffu, odd ? o[q] : o[q + 16], 1);
                            const __nv_bfloat162 two = odd ? __floats2bfloat162_rn(yours, mine) : __floats2bfloat162_rn(mine, yours);
                            *reinterpret_cast<__nv_bfloat162 *>(out + q * kDH) = two;
                        }
                    } else {
                        float *out = static_cast<float *>(p.out) + (w.row * kH + c) * kDH + d;
#pragma unroll
                        for (int q = 0; q < 32; ++q) out[q * kDH] = o[q];
                    }
                }
            } else {
                const int place = 2 * (int)blockIdx.x + (n > 0);
                float *sums = p.part_o + (int64_t)place * kH * kDH;
                if (part == 0) reinterpret_cast<float2 *>(p.part_ml)[place * kH + h] = make_float2(m2, l);
                if (tid == 0 && w.t0 == 0) {              // the row begins here: its last tile of the span is the span's last
                    const int64_t s1 = span_start(blockIdx.x + 1, misc->total, misc->groups);
                    Cut &k = cuts[p.by_row ? w.row : (int64_t)blockIdx.x];
                    k.first = (int)blockIdx.x;
                    k.last = span_of(s1 - it.T + it.tiles - 1, misc->total, misc->groups);
                    k.place = place;
                    k.row = w.row;
                }
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    const int mt = 2 * side + (k >> 1), c = 32 * (k & 1);
                    float o[32];
                    tmem_ld32(quadrant + kColO + mt * kH + c, o);
#pragma unroll
                    for (int q = 0; q < 32; ++q) sums[(c + q) * kDH + mt * 128 + quad * 32 + lane] = o[q];
                }
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&misc->ofree);
            w = w_next;
            it = it_next;
        }
    }
    if (!ok) flag(p.status, HISA_DEV_TIMEOUT);
    fence_before_sync();
    __syncthreads();
    if (warp == kSWarp) {
        fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Joins the sums of the rows that spans cut: one row (by the CTA that has its first tile) and kJoinHeads
// heads per CTA, 128 threads of four dims to a head; where few rows have many parts, GROUPS times as many
// share one head's.
template <int GROUPS>
constexpr int kJoinHeads = GROUPS == 1 ? 4 : 1;
template <int GROUPS>
constexpr int kJoinThreads = 128 * GROUPS * kJoinHeads<GROUPS>;
template <int GROUPS>
__global__ void __launch_bounds__(kJoinThreads<GROUPS>) k_cache_join(CacheAttnParams p) {
    __shared__ float weight[kJoinHeads<GROUPS>][kCacheCtas];
    __shared__ float4 part[GROUPS == 1 ? 1 : GROUPS - 1][128];
    grid_dep_wait();
    grid_dep_trigger();
    const Cut cut = reinterpret_cast<const Cut *>(p.cuts)[blockIdx.x];
    if (!cut_fits(cut, (int64_t)p.B * p.L, p.ctas)) return;
    const int team = threadIdx.x / 128, lane = threadIdx.x & 31, grp = team % GROUPS, hs = team / GROUPS, d = (threadIdx.x % 128) * 4;
    const int h = blockIdx.y * kJoinHeads<GROUPS> + hs, first = cut.first, segs = cut.last - first + 1;
    // every span has a tile, so every CTA from the first to the last has a part of the row
    auto place = [&](int s) { return s == 0 ? cut.place : 2 * (first + s); };
    const float sink2 = p.sinks ? p.sinks[h] * kLog2e : -INFINITY;
    // maximum and normaliser by each warp for itself, a few parts per lane
    constexpr int kMine = (kCacheCtas + 31) / 32;
    float2 ml[kMine];
    float M = sink2;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int s = lane + 32 * i;
        ml[i] = make_float2(-INFINITY, 0.f);
        if (s < segs) ml[i] = reinterpret_cast<const float2 *>(p.part_ml)[place(s) * kH + h];
        M = fmaxf(M, ml[i].x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float ref = M == -INFINITY ? 0.f : M;
    float den = 0.f;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const float a = ex2(ml[i].x - ref);              // a part that saw nothing: 0 of sums that are 0
        den += ml[i].y * a;
        if (lane + 32 * i < segs) weight[hs][lane + 32 * i] = a;      // the same from every warp of the head
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    den += sink2 == -INFINITY ? 0.f : ex2(sink2 - ref);
    __syncwarp();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = grp; s < segs; s += GROUPS) {
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(p.part_o + ((int64_t)place(s) * kH + h) * kDH + d));
        const float a = weight[hs][s];
        o.x += v.x * a; o.y += v.y * a; o.z += v.z * a; o.w += v.w * a;
    }
    if constexpr (GROUPS > 1) {
        if (grp) part[grp - 1][d / 4] = o;
        __syncthreads();
        if (grp) return;
#pragma unroll
        for (int k = 0; k < GROUPS - 1; ++k) {
            const float4 v = part[k][d / 4];
            o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
        }
    }
    const float f = den == 0.f ? 0.f : 1.f / den;
    o.x *= f; o.y *= f; o.z *= f; o.w *= f;
    const int64_t at = (cut.row * kH + h) * kDH + d;
    if (p.out_bf16) {
        const __nv_bfloat162 u = __floats2bfloat162_rn(o.x, o.y), v = __floats2bfloat162_rn(o.z, o.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = o;
    }
}

template <bool BITS4, bool OUT32>
cudaError_t go(const CacheAttnParams &p, cudaStream_t s) {
    const cudaError_t attr = smem_attr_once<k_cache_tc<BITS4, OUT32>>((int)kSmemBytes);
    if (attr != cudaSuccess) return attr;
    CUtensorMap qmap;
    if (!encode_bf16_chunks(&qmap, p.q, (uint64_t)p.B * p.L * kH, kDH, kH, 8)) return cudaErrorInvalidValue;
    const cudaError_t e = launch_pdl(k_cache_tc<BITS4, OUT32>, dim3((unsigned)p.ctas), dim3(kThreads), kSmemBytes, s, 1, qmap, p);
    if (e != cudaSuccess || p.whole) return e;
    const unsigned entries = p.by_row ? (unsigned)(p.B * p.L) : (unsigned)p.ctas;
    if (p.by_row && entries <= 8)
        return launch_pdl(k_cache_join<8>, dim3(entries, kH), dim3(kJoinThreads<8>), 0, s, 1, p);
    return launch_pdl(k_cache_join<1>, dim3(entries, kH / 4), dim3(kJoinThreads<1>), 0, s, 1, p);
}

}  // namespace

bool cache_tc_supported(int H, int Dh, int q_bf16) { return H == kH && Dh == kDH && q_bf16; }

cudaError_t launch_cache_tc(const CacheAttnParams &p, cudaStream_t s) {
    if (p.out_bf16) return p.bits4 ? go<true, false>(p, s) : go<false, false>(p, s);
    return p.bits4 ? go<true, true>(p, s) : go<false, true>(p, s);
}

}  // namespace hisa
