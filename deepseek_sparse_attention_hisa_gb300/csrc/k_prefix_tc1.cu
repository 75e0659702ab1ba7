// Shared-prefix combine on the tensor cores for bf16 heads of 64 and 128 dims: the shared rows'
// segments (the local and own rows' are k_prefix.cu's).
//
// The query rows of the batch stack into tiles of 128 (query row, head) rows, one CTA per tile and
// segment: S [128 x 128] = Q K^T and O [128 x DH] += P V, both at the full tensor rate (M = 128,
// N = 128 or DH). A tile of 128 shared rows is staged once (K = V): K-major for the first product,
// MN-major for the second. A tile has 128 x 128 exponentials for 2 * 128 * 128 * DH products; at
// 16 per cycle they take as long as both products of DH = 128 do (1024 cycles), so the exponentials
// bound it, and eight warps share them: thread = (row, half of the columns), the two threads of a
// row exchange their maxima through shared memory. Lazy rescaling, rounding of P and sums as in
// k_prefix_tc.cu.
//
// Measured: 304 query rows of 16 x 128 over 16384 shared rows 61 us, 102 us with their own lists
// (63 us before or beside them on CUDA cores), the merge included.
//
// Warps: 0-7 softmax and epilogue, 8 loads, 9 S issue, 10 PV issue. Every wait is bounded; a
// timeout sets HISA_DEV_TIMEOUT and the CTA leaves.
#include "prefix_common.cuh"

namespace hisa {
namespace {

using namespace tc;

constexpr int kR = 128, kT = 128;                       // stacked rows; shared rows per tile
constexpr int kSoftWarps = 8, kLoadWarp = 8, kSWarp = 9, kPvWarp = 10, kThreads = 352;
constexpr int kStages = 3, kBufs = 2;                   // staged tiles; S and P buffers
constexpr uint32_t kChunk = 128 * 128;                  // 128 rows x 64 elements, 128-byte swizzle
constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f, kLazy = 8.0f;

struct Misc {
    uint64_t qfull, full[kStages], empty[kStages], sfull[kBufs], sfree[kBufs], pfull[kBufs], pfree[kBufs], ofull, drain;
    uint32_t tmem;
    int abort;
    float mx[2][2][kR];                                 // [tile parity][column half][row]: a tile's maxima
};
template <int DH>
struct Lay {
    static constexpr uint32_t kTile = DH / 64 * kChunk; // Q, and a tile of shared rows
    static constexpr uint32_t kOffKV = kTile, kOffP = kOffKV + kStages * kTile, kOffMisc = kOffP + kBufs * 2 * kChunk;
    static constexpr uint32_t bytes = kOffMisc + sizeof(Misc) + 1024;
};
static_assert(Lay<128>::bytes <= 227 * 1024, "shared memory");

__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap *map, int row, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(0), "r"(smem_u32(bar)) : "memory");
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1) k_prefix_tc1(PrefixParams p, const __grid_constant__ CUtensorMap qmap,
                                                            const __grid_constant__ CUtensorMap kvmap) {
    using Y = Lay<DH>;
    extern __shared__ __align__(1024) uint8_t raw[];
    const uint32_t r0 = smem_u32(raw);
    uint8_t *smem = raw + (((r0 + 1023u) & ~1023u) - r0);
    const uint32_t sbase = smem_u32(smem);
    Misc *ms = reinterpret_cast<Misc *>(smem + Y::kOffMisc);
    volatile int *abort = &ms->abort;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t rows = (int64_t)p.B * p.L * p.H, g0 = (int64_t)blockIdx.x * kR;
    const int64_t first = (int64_t)blockIdx.y * p.pre_rows;
    const int n = (int)((first + p.pre_rows < p.P ? first + p.pre_rows : p.P) - first), tiles = (n + kT - 1) / kT;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&ms->full[s], 1); mbar_init(&ms->empty[s], 1);
        }
        for (int s = 0; s < kBufs; ++s) {
            mbar_init(&ms->sfull[s], 1); mbar_init(&ms->sfree[s], kSoftWarps);
            mbar_init(&ms->pfull[s], kSoftWarps); mbar_init(&ms->pfree[s], 1);
        }
        mbar_init(&ms->qfull, 1); mbar_init(&ms->ofull, 1); mbar_init(&ms->drain, 2);
        mbar_fence_init();
        ms->abort = 0;
    }
    if (warp == kSWarp) {
        tmem_alloc(&ms->tmem, kTmemCols);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = ms->tmem;
    if (!p.tail_split) grid_dep_wait();                 // else see the end
    grid_dep_trigger();
    bool ok = true;
    auto fail = [&]() {
        ok = false;
        *abort = 1;
    };

    if (warp == kLoadWarp) {
        if (lane == 0) {
            int i = 0;
            mbar_arrive_expect_tx(&ms->qfull, Y::kTile);
            load_rows(sbase, &qmap, (int)g0, &ms->qfull);
            for (; i < tiles; ++i) {
                const int s = i % kStages;
                if (i >= kStages && !mbar_wait_abortable(&ms->empty[s], (i / kStages - 1) & 1, abort)) { fail(); break; }
                mbar_arrive_expect_tx(&ms->full[s], Y::kTile);
                load_rows(sbase + Y::kOffKV + s * Y::kTile, &kvmap, (int)first + i * kT, &ms->full[s]);
            }
            if (!ok) {                                  // copies in flight land before the CTA leaves (bounded)
                mbar_wait(&ms->qfull, 0, 1u << 20);
                for (int b = i > kStages ? i - kStages : 0; b < i; ++b) mbar_wait(&ms->full[b % kStages], (b / kStages) & 1, 1u << 20);
            }
        }
        __syncwarp();
    } else if (warp == kSWarp || warp == kPvWarp) {
        if (warp == kSWarp) {
            const uint32_t idesc = idesc_bf16_f32(kR, kT, 0, 0);
            const uint64_t qd = smem_desc_sw128(sbase, 16, 1024);
            if (!wait_warp(&ms->qfull, 0, abort)) fail();
            for (int i = 0; i < tiles && ok; ++i) {
                const int s = i % kStages, b = i % kBufs;
                if (!wait_warp(&ms->full[s], (i / kStages) & 1, abort) ||
                    (i >= kBufs && !wait_warp(&ms->sfree[b], (i / kBufs - 1) & 1, abort))) {
                    fail();
                    break;
                }
                fence_after_sync();
                const uint64_t kd = smem_desc_sw128(sbase + Y::kOffKV + s * Y::kTile, 16, 1024);
#pragma unroll
                for (int ks = 0; ks < DH / 16; ++ks)
                    mma_bf16_warp(tmem + kColS + b * kT, desc_add(qd, (ks >> 2) * kChunk + (ks & 3) * 32),
                                  desc_add(kd, (ks >> 2) * kChunk + (ks & 3) * 32), idesc, ks > 0);
                mma_commit_warp(&ms->sfull[b]);
            }
        } else {
            const uint32_t idesc = idesc_bf16_f32(kR, DH, 0, 1);
            for (int i = 0; i < tiles; ++i) {
                const int s = i % kStages, b = i % kBufs;
                if (!wait_warp(&ms->pfull[b], (i / kBufs) & 1, abort)) { fail(); break; }
                fence_after_sync();
                const uint64_t pd = smem_desc_sw128(sbase + Y::kOffP + b * 2 * kChunk, 16, 1024);
                const uint64_t vd = smem_desc_sw128(sbase + Y::kOffKV + s * Y::kTile, kChunk, 1024);
#pragma unroll
                for (int ks = 0; ks < kT / 16; ++ks)
                    mma_bf16_warp(tmem + kColO, desc_add(pd, (ks >> 2) * kChunk + (ks & 3) * 32), desc_add(vd, ks * 2048), idesc,
                                  (ks > 0 || i > 0) ? 1u : 0u);
                mma_commit_warp(&ms->empty[s]);
                mma_commit_warp(&ms->pfree[b]);
            }
            if (ok) mma_commit_warp(&ms->ofull);
        }
        mma_commit_warp(&ms->drain);                    // MMAs in flight end before TMEM is freed (bounded)
        __syncwarp();
        mbar_wait(&ms->drain, 0, 1u << 24);
        __syncwarp();
    } else {
        const int r = (warp & 3) * 32 + lane, half = warp >> 2;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const float c2 = p.scale * kLog2e;
        const uint32_t pairbar = 1 + (warp & 3);        // the two warps that share 32 rows
        float m2 = -INFINITY, l = 0.f;
        bool good = true;                               // both warps of a pair leave at the same barrier
        for (int i = 0; i < tiles; ++i) {
            const int b = i % kBufs;
            good = good && wait_warp(&ms->sfull[b], (i / kBufs) & 1, abort);
            fence_after_sync();
            float v[64];
            {
                float a[32];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    tmem_ld32(lanes + kColS + b * kT + half * 64 + h * 32, a);
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[h * 32 + k] = a[k];
                }
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms->sfree[b]);
            const int left = n - i * kT - half * 64;
            if (left < 64) {
#pragma unroll
                for (int k = 0; k < 64; ++k) v[k] = k < left ? v[k] : -INFINITY;
            }
            float mx[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) mx[k] = fmaxf(v[k], v[k + 32]);
#pragma unroll
            for (int w = 16; w >= 1; w >>= 1)
#pragma unroll
                for (int k = 0; k < w; ++k) mx[k] = fmaxf(mx[k], mx[k + w]);
            ms->mx[i & 1][half][r] = mx[0];
            if (!pair_all(pairbar, good)) { fail(); break; }
            const float tmax = fmaxf(mx[0], ms->mx[i & 1][half ^ 1][r]) * c2;      // c2 > 0
            float alpha = 1.f;
            if (tmax > m2 + kLazy) {
                alpha = ex2(m2 - tmax);
                m2 = tmax;
            }
            const float ref = m2 == -INFINITY ? 0.f : m2;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t u[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                const float a = ex2(fmaf(v[2 * k], c2, -ref)), c = ex2(fmaf(v[2 * k + 1], c2, -ref));
                sum[k & 3] += a + c;
                const __nv_bfloat162 h = __floats2bfloat162_rn(a, c);
                u[k] = *reinterpret_cast<const uint32_t *>(&h);
            }
            l = l * alpha + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
            // the P buffer's last reader, and for a rescale every product so far, has completed
            if (i >= kBufs) good = good && wait_warp(&ms->pfree[b], (i / kBufs - 1) & 1, abort);
            if (__any_sync(0xffffffffu, alpha != 1.f) && i > 0) {
                good = good && wait_warp(&ms->pfree[(i - 1) % kBufs], ((i - 1) / kBufs) & 1, abort);
                fence_after_sync();
#pragma unroll 1
                for (int c = 0; c < DH / 2; c += 16) {
                    float o[16];
                    const uint32_t at = lanes + kColO + half * (DH / 2) + c;
                    tmem_ld16(at, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] *= alpha;
                    tmem_st16(at, o);
                }
                tmem_st_wait();
            }
            uint8_t *pb = smem + Y::kOffP + (b * 2 + half) * kChunk;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4 *>(pb + sw128_offset(r, k * 8)) = make_uint4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
            fence_async_smem();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms->pfull[b]);
        }
        if (ok) {
            good = good && wait_warp(&ms->ofull, 0, abort);
            fence_after_sync();
            ms->mx[tiles & 1][half][r] = l;             // the row's sum joins over its two threads
            if (!pair_all(pairbar, good)) fail();
        }
        if (ok) {
            l += ms->mx[tiles & 1][half ^ 1][r];
            const bool there = g0 + r < rows;
            const int64_t at = (int64_t)(p.tail_split + blockIdx.y) * rows + g0 + r;
            if (there && half == 0) *reinterpret_cast<float2 *>(p.part_ml + at * 2) = make_float2(m2 * kLn2, l);
#pragma unroll 1
            for (int c = 0; c < DH / 2; c += 32) {
                float o[32];
                tmem_ld32(lanes + kColO + half * (DH / 2) + c, o);
                if (!there) continue;
#pragma unroll
                for (int k = 0; k < 32; k += 8) store_sector(p.part_o + at * DH + half * (DH / 2) + c + k, o + k);
            }
        }
    }
    if (!ok) flag(p.status, HISA_DEV_TIMEOUT);
    fence_before_sync();
    // the own lists' kernel, beside which this one may have started, is done: the merge, which waits
    // for this grid, has both
    grid_dep_wait();
    __syncthreads();
    if (warp == kSWarp) {
        fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int DH>
cudaError_t go(const PrefixParams &p, cudaStream_t s) {
    const cudaError_t attr = smem_attr_once<k_prefix_tc1<DH>>((int)Lay<DH>::bytes);
    if (attr != cudaSuccess) return attr;
    const uint64_t rows = (uint64_t)p.B * p.L * p.H;
    CUtensorMap qmap, kvmap;
    if (!encode_bf16_chunks(&qmap, p.q, rows, DH, kR, DH / 64) || !encode_bf16_chunks(&kvmap, p.prefix_kv, (uint64_t)p.P, DH, kT, DH / 64))
        return cudaErrorInvalidValue;
    return launch_pdl(k_prefix_tc1<DH>, dim3((unsigned)((rows + kR - 1) / kR), (unsigned)p.pre_split), dim3(kThreads), Lay<DH>::bytes,
                      s, 1, p, qmap, kvmap);
}

}  // namespace

cudaError_t launch_prefix_tc1(const PrefixParams &p, cudaStream_t s) { return p.Dh == 64 ? go<64>(p, s) : go<128>(p, s); }

}  // namespace hisa
