// Combine over a cache in pages on the tensor cores: 64 bf16 query heads of 512 dims, K = V, pooled rows in
// 4 bits or bf16.
//
// A query row's list (its visible window, then the pooled rows it sees) is cut into tiles of 64 rows, all
// of one kind. Per tile:
//   S  = Q . K^T      tcgen05, M = 64 heads, N = 64 rows, K = 512           (TMEM, 2 buffers)
//   P  = exp2(S scale log2e - m) per head, in the threads that own the head's TMEM lane
//   O^T += V^T . P^T  tcgen05, M = 128 dims x 4, N = 64 heads, K = 64       (TMEM, f32)
// The tile is staged once in bf16 (128-byte swizzle): K-major for the first product, MN-major for the
// second.
//
// Rows in 4 bits become bf16 on their way into the tile, exactly: a 4-bit float has 2 significant bits,
// its scale 4, the product 6 of bf16's 8. A code's three magnitude bits placed at the end of bf16's
// exponent and the start of its mantissa are the code times 2^-126 (its 0.5 a subnormal number), so a
// product with the scale times 2^118 leaves code * scale * 2^-8; the 2^8 and the cache's factor go into
// the logits and into P. Two dims take a byte permute, two shifts, two masks and the product.
//
// Work: one CTA per SM. Lists differ in length and only the device knows them, so every CTA adds up
// all rows' tiles and takes an equal span of them (p.whole: whole rows in turn, where all lists are
// as long). A row that lies in one span is finished there; the sums of one that is cut go to memory, two
// places per CTA, and k_cache_join adds them up.
//
// The running maximum m is lazy: O^T and l are rescaled only when a tile's maximum exceeds m by more
// than 8 (log2 units), so p <= 256.
//
// Warps: 0-3 softmax, 4 S issue (and q by TMA), 5 PV issue, 6-9 epilogue, 10-17 rows. A lane of the row
// warps has one row of the tile and a quarter of its dims: the row's id is fetched three tiles ahead, its page
// two, its codes one. Every wait is bounded; a timeout sets HISA_DEV_TIMEOUT and the CTA leaves.
#include "cache_internal.cuh"
#include "prefix_common.cuh"

namespace hisa {
namespace {

using namespace tc;

constexpr int kH = 64, kDH = 512, kT = 64;              // heads, dims, rows of a tile
constexpr int kSoftWarps = 4, kSWarp = 4, kPvWarp = 5, kEpiWarp0 = 6, kRowWarp0 = 10, kRowWarps = 8;
constexpr int kThreads = 32 * (kRowWarp0 + kRowWarps);
static_assert(kEpiWarp0 % 4 == 2 && kRowWarp0 == kEpiWarp0 + 4, "each epilogue warp has a TMEM quadrant of its own");
constexpr int kSlots = 2, kBufs = 2;
constexpr uint32_t kChunk = 64 * 128;                   // 64 rows x 64 dims, 128-byte swizzle
constexpr uint32_t kTile = 8 * kChunk;
constexpr uint32_t kOffQ = 0, kOffKV = kTile, kOffP = kOffKV + kSlots * kTile, kOffMisc = kOffP + kBufs * kChunk;
constexpr uint32_t kColS = 0, kColO = 128, kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f, kLazy = 8.0f;
constexpr int kBarSoft = 1;

struct Misc {
    uint64_t qfull, qfree, full[kSlots], empty[kSlots], sfull[kBufs], sfree[kBufs], pfull[kBufs], pfree[kBufs], ofull, ofree, stat,
        drain;
    uint64_t mask[kSlots];                              // rows of a tile that are seen
    uint32_t tmem;
    int abort;
    int t0, groups;                                     // the span: first tile of its first row; CTAs that have one
    int64_t row, left, total;                           // first row, tiles; all rows' tiles
    int64_t sums[kThreads / 32];
    float alpha[2][kH];
    float stat_m[kH], stat_l[kH], factor[kH];
};
constexpr uint32_t kSmemBytes = kOffMisc + sizeof(Misc) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// A row whose tiles lie in the spans of several CTAs, by the CTA that has its first tile.
struct Cut {
    int64_t row, total;                                 // -1: none
    int last, groups;                                   // the CTA that has its last tile
    int place, pad;                                     // of the first CTA's sums
};
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
__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0], %1;\n\t}" :: "r"(smem_u32(bar)), "r"(n) : "memory");
}
// Lanes 0-15 read columns [c, c + 32) of TMEM lanes base + 0 .. 15, lanes 16-31 columns [c + 32, c + 64) of
// the same ones (an M = 64 accumulator's rows live in lanes 0-15 of each quadrant).
__device__ __forceinline__ void tmem_ld32_x2(uint32_t addr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
                 "%29,%30,%31}, [%32], 32;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
                   "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                   "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// Barriers of the four softmax warps: true on all iff v is on one (any), on all (all).
__device__ __forceinline__ bool soft_any(bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"((uint32_t)v), "n"(kBarSoft) : "memory");
    return r != 0u;
}
__device__ __forceinline__ bool soft_all(bool v) { return !soft_any(!v); }

// Eight codes times a scale (as bf16, times 2^118, in both halves of s), in bf16, times 2^-8.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint4 codes_to_bf16(uint32_t w, uint32_t s) {
    const uint32_t odd = w >> 4;
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {                       // the even dim's code at bit 0, the odd one's at bit 16
        const uint32_t u = __byte_perm(w, odd, (j | j << 4 | (4 + j) << 8 | (4 + j) << 12));
        r[j] = mul_bf16x2((u << 6 & 0x01c001c0u) | (u << 12 & 0x80008000u), s);
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

// The tiles of a CTA, as one lane of the row warps sees them: its own row of each.
enum TileKind : int { kEnd = 0, kLocal = 1, kPool = 2 };
struct Wanted {                                          // its id is on its way
    int kind, id, V, len;
    const int32_t *table;                                // the sequence's pages
    int64_t place;                                       // kLocal: the row of local_kv
};
struct Paged {                                           // its page is on its way
    int kind, page, rest;                                // row of the page; -1: none
    int64_t place;
};
struct Placed {
    int kind;
    int64_t place;                                       // row of local_kv or of the pool; -1: not seen
};
struct Codes {
    uint4 c[4];
    uint32_t s[4];
};

template <bool BITS4>
__global__ void __launch_bounds__(kThreads, 1) k_cache_tc(const __grid_constant__ CUtensorMap qmap, CacheAttnParams p) {
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
        for (int i = 0; i < 2; ++i) {
            mbar_init(&misc->full[i], 33 * kRowWarps);
            mbar_init(&misc->empty[i], 1);
            mbar_init(&misc->sfull[i], 1);
            mbar_init(&misc->sfree[i], 32 * kSoftWarps);
            mbar_init(&misc->pfull[i], 32 * kSoftWarps);
            mbar_init(&misc->pfree[i], 1);
        }
        mbar_init(&misc->ofull, 1);
        mbar_init(&misc->ofree, 128);
        mbar_init(&misc->stat, 32 * kSoftWarps);
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
        int64_t total = 0, before = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i == warp) before = total;
            total += misc->sums[i];
        }
        int64_t groups = total / p.least;
        groups = groups < 1 ? 1 : (groups > (int64_t)gridDim.x ? (int64_t)gridDim.x : groups);
        const int64_t c = blockIdx.x;
        const int64_t s0 = c < groups ? c * total / groups : total, s1 = c < groups ? (c + 1) * total / groups : total;
        int64_t at = before + upto - sum;
        if (tid == 0) {
            misc->left = s1 - s0;
            misc->total = total;
            misc->groups = (int)groups;
            cuts[blockIdx.x].row = -1;
        }
        if (s0 >= at && s0 < at + sum) {
            for (int64_t r = r0; r < r1; ++r) {
                const int n = tiles_of(cache_row(p, r, false));
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
        // ---------------- rows: this lane's row and quarter of each tile ----------------
        const int rw = warp - kRowWarp0, r = 8 * rw + (lane & 7), qd = lane >> 3;
        bool have = walk_item(p, w, it);
        int ti = 0;                                      // the next tile of the item
        // the next tile of the walk: its ids are asked for
        auto want = [&]() -> Wanted {
            Wanted a{kEnd, -1, 0, 0, nullptr, -1};
            if (!have) return a;
            const int t = w.t0 + ti;
            const int b = (int)(w.row / p.L);
            if (t < it.nl) {
                const int e = t * kT + r;
                a.kind = kLocal;
                if (e < it.x.nloc) a.place = (int64_t)b * p.W_max + it.x.lo + e;
            } else {
                const int kk = (t - it.nl) * kT + r;
                a.kind = kPool;
                a.V = (int)it.x.V;
                a.len = (int)it.x.len;
                a.table = p.page_table + (int64_t)b * p.table_cols;
                if (kk < it.x.npool) a.id = p.I ? p.I[w.row * p.k + kk] : kk;
            }
            if (++ti == it.T) {
                walk_next(p, w, it);
                have = walk_item(p, w, it);
                ti = 0;
            }
            return a;
        };
        auto page = [&](const Wanted &a) -> Paged {
            Paged b{a.kind, -1, -1, a.place};
            if (a.kind != kPool) return b;
            if (a.id < -1 || a.id >= a.len) {
                if (a.id != -1) flag(p.status, HISA_DEV_BAD_ID);
            } else if (a.id >= 0 && a.id < a.V) {
                const uint32_t at = (uint32_t)a.id / (uint32_t)p.page_rows;
                b.rest = a.id - (int)(at * (uint32_t)p.page_rows);
                b.page = a.table[at];
            }
            return b;
        };
        auto put = [&](const Paged &b) -> Placed {
            Placed c{b.kind, b.place};
            if (b.kind != kPool || b.rest < 0) return c;
            if (b.page < 0 || b.page >= p.pages) flag(p.status, HISA_DEV_BAD_OFFSETS);
            else c.place = (int64_t)b.page * p.page_rows + b.rest;
            return c;
        };
        auto load = [&](const Placed &c, Codes &x) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x.c[i] = make_uint4(0u, 0u, 0u, 0u);
                x.s[i] = 0u;
            }
            if (!BITS4 || c.kind != kPool || c.place < 0) return;
            // 16 bytes (32 dims, two scales) of every 64 of the row: four lanes read 64 contiguous ones
            const uint4 *codes = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.cache) + c.place * (kDH / 2));
            const uint16_t *sc = reinterpret_cast<const uint16_t *>(p.scales + c.place * (kDH / kScaleGroup));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x.c[i] = codes[4 * i + qd];
                x.s[i] = sc[4 * i + qd];
            }
        };
        Wanted a = want();
        Paged b = page(a);
        a = want();
        Placed cur = put(b);
        Codes x;
        load(cur, x);
        b = page(a);
        a = want();
        uint32_t g = 0;
        while (cur.kind != kEnd) {
            const Placed next = put(b);
            Codes y;
            load(next, y);
            b = page(a);
            a = want();
            const int s = g % kSlots;
            if (g >= kSlots && !wait_warp(&misc->empty[s], ((g / kSlots) - 1) & 1, abort)) { fail(); break; }
            const uint32_t seen = __ballot_sync(0xffffffffu, cur.place >= 0);
            if (lane == 0) reinterpret_cast<uint8_t *>(&misc->mask[s])[rw] = (uint8_t)seen;
            const uint32_t slot = sbase + kOffKV + s * kTile, base = slot + r * 128, sw = r & 7;
            if (BITS4 && cur.kind == kPool) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint2 sc = scales_to_bf16(x.s[i]);
                    const uint32_t cw[4] = {x.c[i].x, x.c[i].y, x.c[i].z, x.c[i].w};
                    const uint32_t chunk = base + (2 * i + (qd >> 1)) * kChunk;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 v = codes_to_bf16(cw[k], k < 2 ? sc.x : sc.y);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                     :: "r"(chunk + ((((qd & 1) * 4 + k) ^ sw) << 4)), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_n(&misc->full[s], 33);
            } else {
                const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(cur.kind == kLocal ? p.local_kv : p.cache);
                const bool v = cur.place >= 0;
                const __nv_bfloat16 *row = v ? src + cur.place * kDH : static_cast<const __nv_bfloat16 *>(p.q);
#pragma unroll 4
                for (int i = 0; i < 16; ++i) {
                    const uint32_t u = 4 * i + qd;       // 16-byte unit of the row
                    cp_async16_zfill(base + (u >> 3) * kChunk + (((u & 7) ^ sw) << 4), v ? row + u * 8 : row, v);
                }
                cp_async_arrive(&misc->full[s]);
                if (lane == 0) mbar_arrive(&misc->full[s]);   // after the mask
            }
            ++g;
            cur = next;
            x = y;
        }
        cp_async_wait_all();
    } else if (warp == kSWarp) {
        // ---------------- S = Q . K^T of every tile; q of each item ----------------
        const uint32_t id_s = idesc_bf16_f32(64, kT, 0, 0);
        const uint64_t qdesc = smem_desc_sw128(sbase + kOffQ, 16, 1024);
        uint32_t g = 0;
        int n = 0;
        for (; walk_item(p, w, it); walk_next(p, w, it), ++n) {
            if (n > 0 && !wait_warp(&misc->qfree, (n - 1) & 1, abort)) { fail(); break; }
            if (lane == 0) {
                mbar_arrive_expect_tx(&misc->qfull, kTile);
                tma_q(sbase + kOffQ, &qmap, (int32_t)(w.row * kH), &misc->qfull);
            }
            __syncwarp();
            if (!wait_warp(&misc->qfull, n & 1, abort)) { fail(); break; }
            for (int i = 0; i < it.T; ++i, ++g) {
                const int s = g % kSlots, sb = g % kBufs;
                if (!wait_warp(&misc->full[s], (g / kSlots) & 1, abort) ||
                    (g >= kBufs && !wait_warp(&misc->sfree[sb], ((g / kBufs) - 1) & 1, abort))) {
                    fail();
                    break;
                }
                fence_async_smem();                       // the rows were written through the generic proxy
                fence_after_sync();
                const uint64_t kd = smem_desc_sw128(sbase + kOffKV + s * kTile, 16, 1024);
                const uint32_t d = tmem + kColS + sb * kT;
#pragma unroll
                for (int ks = 0; ks < kDH / 16; ++ks) {
                    const uint32_t off = (ks >> 2) * kChunk + (ks & 3) * 32;
                    mma_bf16_warp(d, desc_add(qdesc, off), desc_add(kd, off), id_s, ks > 0);
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
        uint32_t g = 0;
        int n = 0;
        for (; walk_item(p, w, it); walk_next(p, w, it), ++n) {
            if (n > 0 && !wait_warp(&misc->ofree, (n - 1) & 1, abort)) { fail(); break; }
            fence_after_sync();
            for (int i = 0; i < it.T; ++i, ++g) {
                const int s = g % kSlots, pb = g % kBufs;
                if (!wait_warp(&misc->pfull[pb], (g / kBufs) & 1, abort)) { fail(); break; }
                fence_async_smem();
                fence_after_sync();
                const uint64_t vd = smem_desc_sw128(sbase + kOffKV + s * kTile, kChunk, 1024);
                const uint64_t pd = smem_desc_sw128(sbase + kOffP + pb * kChunk, 16, 1024);
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int ks = 0; ks < kT / 16; ++ks)
                        mma_bf16_warp(tmem + kColO + mt * kH, desc_add(vd, 2 * mt * kChunk + ks * 2048), desc_add(pd, ks * 32), id_o,
                                      ks > 0 || i > 0);
                mma_commit_warp(&misc->empty[s]);
                mma_commit_warp(&misc->pfree[pb]);
            }
            if (!ok) break;
            mma_commit_warp(&misc->ofull);
        }
        mma_commit_warp(&misc->drain);
        __syncwarp();
        mbar_wait(&misc->drain, 0, 1u << 24);
        __syncwarp();
    } else if (warp < kSoftWarps) {
        // ---------------- softmax: lane l owns head 16 warp + l % 16 and tile rows 32 (l / 16) .. + 31 ------
        const bool lead = lane < 16;
        const int h = warp * 16 + (lane & 15), half = lane >> 4;
        const float sink2 = p.sinks ? p.sinks[h] * kLog2e : -INFINITY;
        const float cl = p.scale * kLog2e, gp = BITS4 ? p.g * 256.f : 1.f;
        uint32_t g = 0, pv_seen[kBufs] = {};
        auto wait_pv = [&](uint32_t tile) -> bool {       // the PV product of a tile is done
            const int b = tile % kBufs;
            while (pv_seen[b] <= tile / kBufs) {
                if (!wait_warp(&misc->pfree[b], pv_seen[b] & 1, abort)) return false;
                ++pv_seen[b];
            }
            return true;
        };
        int n = 0;
        for (; walk_item(p, w, it); walk_next(p, w, it), ++n) {
            float m2 = -INFINITY, l = 0.f;
            for (int i = 0; i < it.T; ++i, ++g) {
                const int s = g % kSlots, sb = g % kBufs;
                const bool pool = w.t0 + i >= it.nl;
                const float f = pool ? gp : 1.f, c2 = cl * f;
                bool good = wait_warp(&misc->full[s], (g / kSlots) & 1, abort) && wait_warp(&misc->sfull[sb], (g / kBufs) & 1, abort);
                fence_after_sync();
                const uint32_t mask = (uint32_t)(*reinterpret_cast<volatile uint64_t *>(&misc->mask[s]) >> (32 * half));
                float v[32];
                tmem_ld32_x2(tmem + ((uint32_t)(32 * warp) << 16) + kColS + sb * kT, v);
                fence_before_sync();
                mbar_arrive(&misc->sfree[sb]);
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    v[k] = ((mask >> k) & 1u) ? v[k] * c2 : -INFINITY;
                    top = fmaxf(top, v[k]);
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                float alpha = 1.f;
                bool rescale = false;
                if (top > m2 + kLazy) {
                    if (m2 != -INFINITY) {
                        alpha = ex2(m2 - top);
                        rescale = true;
                    }
                    m2 = top;
                }
                // ex2(-inf - m) = +0; m2 is finite once a row of this head was seen, and logits are -inf when masked
                const float ref = m2 == -INFINITY ? 0.f : m2;
                float sum = 0.f;
                uint32_t packed[16];
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    const float a = ex2(v[k] - ref), b = ex2(v[k + 1] - ref);
                    sum += a + b;
                    const __nv_bfloat162 two = __floats2bfloat162_rn(a * f, b * f);
                    packed[k / 2] = *reinterpret_cast<const uint32_t *>(&two);
                }
                l = l * alpha + sum + __shfl_xor_sync(0xffffffffu, sum, 16);
                if (lead) misc->alpha[g & 1][h] = alpha;
                if (good && g >= kBufs) good = wait_pv(g - kBufs);       // P's buffer is free
                if (soft_any(rescale || !good)) {
                    if (!soft_all(good)) { fail(); break; }
                    // heads whose reference moved up: O^T after the product of the tile before (of this item)
                    if (!soft_all(i < 1 || wait_pv(g - 1))) { fail(); break; }
                    fence_after_sync();
#pragma unroll 1
                    for (int c = 0; c < 4 * kH; c += 16) {
                        float o[16];
                        const uint32_t ta = tmem + ((uint32_t)(32 * warp) << 16) + kColO + c;
                        tmem_ld16(ta, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 16; ++q) o[q] *= misc->alpha[g & 1][(c & (kH - 1)) + q];
                        tmem_st16(ta, o);
                    }
                    tmem_st_wait();
                }
                uint8_t *pbuf = smem + kOffP + sb * kChunk;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    *reinterpret_cast<uint4 *>(pbuf + sw128_offset(h, (half * 4 + u) * 8)) =
                        make_uint4(packed[4 * u], packed[4 * u + 1], packed[4 * u + 2], packed[4 * u + 3]);
                fence_async_smem();
                fence_before_sync();
                mbar_arrive(&misc->pfull[sb]);
            }
            if (!ok) break;
            // the item's statistics, once the epilogue has read the previous item's
            if (n > 0 && !soft_all(wait_warp(&misc->ofree, (n - 1) & 1, abort))) { fail(); break; }
            if (lead) {
                const float M = fmaxf(m2, sink2);
                const float wm = m2 == -INFINITY ? 0.f : exp2f(m2 - M);
                const float den = l * wm + (sink2 == -INFINITY ? 0.f : exp2f(sink2 - M));
                misc->factor[h] = den == 0.f ? 0.f : wm / den;           // nothing seen, no sink: 0
                misc->stat_m[h] = m2;
                misc->stat_l[h] = l;
            }
            mbar_arrive(&misc->stat);
        }
    } else {
        // ---------------- epilogue: O^T -> out, or a cut row's sums ----------------
        const int quad = warp & 3;                        // TMEM lanes 32 quad .. + 31 = dims
        const uint32_t to = tmem + ((uint32_t)(32 * quad) << 16) + kColO;
        int n = 0;
        for (; walk_item(p, w, it); walk_next(p, w, it), ++n) {
            // an item may be long: as many bounded waits as it has tiles
            bool done = false;
            for (int k = 0; k <= it.T && !done && !*abort; ++k)
                done = wait_warp(&misc->stat, n & 1, abort) && wait_warp(&misc->ofull, n & 1, abort);
            if (!__all_sync(0xffffffffu, done)) { fail(); break; }
            fence_after_sync();
            const bool cut = it.T < it.tiles;
            if (!cut) {
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int c = 0; c < kH; c += 16) {
                        float o[16];
                        tmem_ld16(to + mt * kH + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 16; ++q) o[q] *= misc->factor[c + q];
                        const int d = mt * 128 + quad * 32 + lane;
                        if (p.out_bf16) {
                            // two dims per store: even lanes take the first eight heads, odd ones the others
                            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + w.row * kH * kDH + (d & ~1);
                            const bool odd = lane & 1;
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                const float mine = odd ? o[q + 8] : o[q], yours = __shfl_xor_sync(0xffffffffu, odd ? o[q] : o[q + 8], 1);
                                const __nv_bfloat162 two = odd ? __floats2bfloat162_rn(yours, mine) : __floats2bfloat162_rn(mine, yours);
                                *reinterpret_cast<__nv_bfloat162 *>(out + (int64_t)(c + q + (odd ? 8 : 0)) * kDH) = two;
                            }
                        } else {
                            float *out = static_cast<float *>(p.out) + w.row * kH * kDH + d;
#pragma unroll
                            for (int q = 0; q < 16; ++q) out[(int64_t)(c + q) * kDH] = o[q];
                        }
                    }
            } else {
                const int place = 2 * (int)blockIdx.x + (n > 0);
                float *sums = p.part_o + (int64_t)place * kH * kDH;
                if (quad == 0) {
                    for (int hh = lane; hh < kH; hh += 32)
                        reinterpret_cast<float2 *>(p.part_ml)[place * kH + hh] = make_float2(misc->stat_m[hh], misc->stat_l[hh]);
                    if (lane == 0 && w.t0 == 0) {         // the row begins here: its last tile of the span is the span's last
                        const int64_t s1 = (int64_t)(blockIdx.x + 1) * misc->total / misc->groups;
                        Cut &k = cuts[blockIdx.x];
                        k.total = misc->total;
                        k.groups = misc->groups;
                        k.last = (int)(((s1 - it.T + it.tiles) * misc->groups - 1) / misc->total);
                        k.place = place;
                        k.row = w.row;
                    }
                }
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int c = 0; c < kH; c += 16) {
                        float o[16];
                        tmem_ld16(to + mt * kH + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int q = 0; q < 16; ++q) sums[(c + q) * kDH + mt * 128 + quad * 32 + lane] = o[q];
                    }
            }
            fence_before_sync();
            mbar_arrive(&misc->ofree);
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

// Joins the sums of the rows that spans cut: one row (by the CTA that has its first tile) and 4 / GROUPS
// heads per CTA, 128 threads of four dims to a head; GROUPS of them share one head's sums where few rows
// have many.
constexpr int kJoinThreads = 512;
template <int GROUPS>
__global__ void __launch_bounds__(kJoinThreads) k_cache_join(CacheAttnParams p) {
    __shared__ float weight[4 / GROUPS][kCacheCtas];
    __shared__ float4 part[GROUPS == 1 ? 1 : GROUPS - 1][128];
    grid_dep_wait();
    grid_dep_trigger();
    const Cut cut = reinterpret_cast<const Cut *>(p.cuts)[blockIdx.x];
    if (cut.row < 0) return;
    const int team = threadIdx.x / 128, grp = team % GROUPS, hs = team / GROUPS, d = (threadIdx.x % 128) * 4;
    const int h = blockIdx.y * (4 / GROUPS) + hs, first = blockIdx.x, segs = cut.last - first + 1;
    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml);
    auto place = [&](int s) { return s == 0 ? cut.place : 2 * (first + s); };
    // a span between may be empty (fewer tiles than CTAs)
    auto empty = [&](int s) {
        const int64_t c = first + s;
        return c * cut.total / cut.groups == (c + 1) * cut.total / cut.groups;
    };
    const float sink2 = p.sinks ? p.sinks[h] * kLog2e : -INFINITY;
    float M = sink2;
    for (int s = 0; s < segs; ++s)
        if (!empty(s)) M = fmaxf(M, ml[place(s) * kH + h].x);
    const float ref = M == -INFINITY ? 0.f : M;
    for (int s = threadIdx.x % 128 + 128 * grp; s < segs; s += 128 * GROUPS) {
        const float m = empty(s) ? -INFINITY : ml[place(s) * kH + h].x;
        weight[hs][s] = m == -INFINITY ? -1.f : exp2f(m - ref);          // -1: nothing there, unless NaN
    }
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = sink2 == -INFINITY ? 0.f : exp2f(sink2 - ref);
#pragma unroll 4
    for (int s = 0; s < segs; ++s) {
        if (empty(s)) continue;
        const float l = ml[place(s) * kH + h].y, a = weight[hs][s] < 0.f ? 0.f : weight[hs][s];
        den += l * a;
        if (s % GROUPS != grp) continue;
        const float4 v = __ldcs(reinterpret_cast<const float4 *>(p.part_o + ((int64_t)place(s) * kH + h) * kDH + d));
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

template <bool BITS4>
cudaError_t go(const CacheAttnParams &p, cudaStream_t s) {
    const cudaError_t attr = smem_attr_once<k_cache_tc<BITS4>>((int)kSmemBytes);
    if (attr != cudaSuccess) return attr;
    CUtensorMap qmap;
    if (!encode_bf16_chunks(&qmap, p.q, (uint64_t)p.B * p.L * kH, kDH, kH, 8)) return cudaErrorInvalidValue;
    const cudaError_t e = launch_pdl(k_cache_tc<BITS4>, dim3((unsigned)p.ctas), dim3(kThreads), kSmemBytes, s, 1, qmap, p);
    if (e != cudaSuccess || p.whole) return e;
    if ((int64_t)p.B * p.L <= 16)
        return launch_pdl(k_cache_join<4>, dim3((unsigned)p.ctas, kH), dim3(kJoinThreads), 0, s, 1, p);
    return launch_pdl(k_cache_join<1>, dim3((unsigned)p.ctas, kH / 4), dim3(kJoinThreads), 0, s, 1, p);
}

}  // namespace

bool cache_tc_supported(int H, int Dh, int q_bf16) { return H == kH && Dh == kDH && q_bf16; }

cudaError_t launch_cache_tc(const CacheAttnParams &p, cudaStream_t s) { return p.bits4 ? go<true>(p, s) : go<false>(p, s); }

}  // namespace hisa
