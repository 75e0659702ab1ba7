// Rows into and out of a cache in pages.
//
// A warp takes a chunk of up to 32 consecutive packed rows: each lane finds the place of one of
// them (its sequence, its index, its page: three dependent loads, taken once per chunk), then teams of
// lanes (head_rows.cuh) take the rows in turn, the next one on its way while one is worked on.
// Reading is bound by memory: 65536 rows of 512 dims in 4 bits to f32 26 to 30 us, 5.3 to 5.8 TB/s. A call of a few rows is bound by its
// chain of loads (304 rows 4 to 5 us). Appending in 4 bits is bound by instructions: 440 of a warp per row of 512 dims (two
// units of 8 per lane: the norm, the quotients with their remainders, 32 angles), 2.9 per cycle, 65536 rows 36 us alone (2.4
// TB/s), 41 one call after another.
//
// Append, 4 bits: sixteen dims are two neighbouring lanes' units; their largest magnitude is NaN if one of
// them is. The quotient y / (s g) is a product with the reciprocal and one correction by its exact
// remainder, which gives back quotients that are exactly representable (the ties between codes are such).
#include "cache_internal.cuh"
#include "head_rows.cuh"

namespace hisa {
namespace {

// The place in the pool of packed row n and its index in its sequence; -1 if it has none.
struct Place {
    int64_t slot, index;
};
__device__ __forceinline__ Place place_of(const CacheParams &p, int64_t n) {
    if (n < p.row_off[0] || n >= p.row_off[p.B]) return {-1, 0};       // padding
    // sequences of equal length are found at once
    int lo = (int)((uint64_t)n * (uint64_t)p.B / (uint64_t)p.rows);
    int64_t begin = p.row_off[lo], end = p.row_off[lo + 1];
    if (begin > n || end <= n) {
        lo = 0;
        int hi = p.B;
        while (hi - lo > 1) {
            const int mid = lo + (hi - lo) / 2;
            if (p.row_off[mid] <= n) lo = mid;
            else hi = mid;
        }
        begin = p.row_off[lo];
        end = p.row_off[lo + 1];
    }
    // not ascending (the search may end beside the row), or past the rows: reported by check_offsets
    if (begin < 0 || begin > n || end <= n || end > p.rows) return {-1, 0};
    const int64_t first = p.row_first[lo], index = first + n - begin;
    if (first < 0 || index >= (int64_t)p.table_cols * p.page_rows) {
        flag(p.status, HISA_DEV_BAD_OFFSETS);
        return {-1, 0};
    }
    const int64_t at = index < (int64_t)1 << 32 ? (int64_t)((uint32_t)index / (uint32_t)p.page_rows) : index / p.page_rows;
    const int64_t page = p.page_table[(int64_t)lo * p.table_cols + at];
    if (page < 0 || page >= p.pages) {
        flag(p.status, HISA_DEV_BAD_OFFSETS);
        return {-1, 0};
    }
    return {page * p.page_rows + (index - at * p.page_rows), index};
}
__device__ __forceinline__ void check_offsets(const CacheParams &p) {
    if (blockIdx.x != 0) return;
    bool bad = p.row_off[0] < 0 || p.row_off[p.B] > p.rows;
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) bad = bad || p.row_off[b + 1] < p.row_off[b];
    if (bad) flag(p.status, HISA_DEV_BAD_OFFSETS);
}

constexpr uint32_t kE4m3Nan = 0x7fu;

// The largest magnitude of three, NaN if one is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Eight f32 of a 16-dim group (the other eight in the neighbouring lane) to codes and the scale's byte.
__device__ __forceinline__ uint32_t quantise(float (&y)[8], float g, float inv6g, uint32_t &scale) {
    const float a8 = max3_abs(max3_abs(y[0], y[1], y[2]), max3_abs(y[3], y[4], y[5]), max3_abs(y[6], y[7], y[7]));
    const float a = max3_abs(a8, a8, __shfl_xor_sync(0xffffffffu, a8, 1));
    // a / 6 g by the reciprocal, corrected by the exact remainder; past 448 it does not matter by how much
    float t = fminf(a * inv6g, 1e6f);
    t = fmaf(fmaf(-t, 6.f * g, a), inv6g, t);
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(t));
    scale = a < INFINITY ? (uint32_t)two & 0xffu : kE4m3Nan;
    const float step = e4m3_to_f32(scale) * g;
    float inv;                                                // to a step or two: what it scales is corrected
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(step));
    inv = step > 0.f ? inv : 0.f;                             // NaN: 0 too, and its codes say nothing
    if (a > 7.f * step) {                                     // the scale is at its largest, or 0
        const float most = 8.f * step;
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = fminf(fmaxf(y[e], -most), most);
    }
    const float2 ii = make_float2(inv, inv), ss = make_float2(-step, -step);
    float2 q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 z = make_float2(y[2 * e], y[2 * e + 1]), v = mul2(z, ii);
        q[e] = fma2(fma2(v, ss, z), ii, v);
    }
    uint32_t w;
    asm("{.reg .b8 a, b, c, d; cvt.rn.satfinite.e2m1x2.f32 a, %2, %1; cvt.rn.satfinite.e2m1x2.f32 b, %4, %3; "
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5; cvt.rn.satfinite.e2m1x2.f32 d, %8, %7; mov.b32 %0, {a, b, c, d};}"
        : "=r"(w) : "f"(q[0].x), "f"(q[0].y), "f"(q[1].x), "f"(q[1].y), "f"(q[2].x), "f"(q[2].y), "f"(q[3].x), "f"(q[3].y));
    return w;
}

// CTAs per SM that the registers leave room for: as many as there is no spilling with
template <typename S, int U, int FORM>
constexpr int kAppendCtas = FORM == kAny || U == 4 ? 2 : (U == 2 && (sizeof(S) == 4 || FORM == kHalves) ? 4 : (sizeof(S) == 4 ? 6 : 8));

template <typename S, int U, int FORM>
__global__ void __launch_bounds__(128, kAppendCtas<S, U, FORM>) k_cache_append(CacheParams p) {
    extern __shared__ __align__(16) float sm[];
    const RowShape g = row_shape(sm, p.D, p.lanes, p.first, p.dims, p.half, FORM == kAny);
    const int lane = threadIdx.x & 31, per = 32 / p.lanes, sub = lane / p.lanes;
    const int64_t n0 = ((int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32) * p.chunk;
    grid_dep_wait();
    grid_dep_trigger();
    check_offsets(p);
    if (n0 >= p.rows) return;
    const int n = (int)(p.rows - n0 < p.chunk ? p.rows - n0 : p.chunk);
    Place mine{-1, 0};
    if (lane < n) mine = place_of(p, n0 + lane);
    const S *x = static_cast<const S *>(p.x) + n0 * p.ld;
    const float inv6g = 1.f / (6.f * p.g);
    constexpr bool kHeld = FORM != kAny && U <= 2;
    float2 held[U][4];
    if (kHeld && p.w) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = i * g.T + g.tl;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                held[i][e] = u < g.units ? __ldg(reinterpret_cast<const float2 *>(p.w + 8 * u) + e) : make_float2(0.f, 0.f);
        }
    }
    RowBuf<S, U, FORM> buf = {};
    auto slot_of = [&](int r) { return __shfl_sync(0xffffffffu, mine.slot, r & 31); };
    int64_t slot = slot_of(sub);
    if (sub >= n) slot = -1;
    if (slot >= 0) buf.load(x + (int64_t)sub * p.ld, g);
    for (int r0 = 0; r0 < n; r0 += per) {
        const int r = r0 + sub;
        const int64_t index = __shfl_sync(0xffffffffu, mine.index, r & 31);
        const RowBuf<S, U, FORM> cur = buf;
        const int64_t here = slot;
        slot = slot_of(r + per);
        if (r + per >= n) slot = -1;
        if (slot >= 0) buf.load(x + (int64_t)(r + per) * p.ld, g);
        if (p.dims) {
            if (here >= 0) team_angles(g, p.table, index * p.r, p.mscale);
            __syncwarp();
        }
        float v[U][8];
        cur.template finish<kHeld>(g, p.norm, p.w, p.eps, v, held);
        if (p.bits4) {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = i * g.T + g.tl;             // lanes past the row have zeros
                uint32_t scale;
                const uint32_t w = quantise(v[i], p.g, inv6g, scale);
                if (here < 0 || u >= g.units) continue;
                reinterpret_cast<uint32_t *>(p.cache)[here * (p.D / 8) + u] = w;
                if (!(u & 1)) p.scales[here * (p.D / kScaleGroup) + u / 2] = (uint8_t)scale;
            }
        } else if (here >= 0) {
            __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(p.cache) + here * p.D;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = i * g.T + g.tl;
                if (u < g.units) store8(to + 8 * u, v[i]);
            }
        }
        __syncwarp();                                     // the angles are read before the next row's are written
    }
}

// The codes of eight dims as e4m3 bytes.
__device__ __forceinline__ uint2 codes_to_e4m3(uint32_t w) {
    uint32_t out[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t x = w >> (16 * k);
        // 0, 0.5, 1, 1.5 and 2, 3, 4, 6
        out[k] = __byte_perm(0x3c383000u, 0x4c484440u, x & 0x7777u) | (x << 4 & 0x80u) | (x << 8 & 0x8000u) |
                 (x << 12 & 0x800000u) | (x << 16 & 0x80000000u);
    }
    return make_uint2(out[0], out[1]);
}

// A lane has units of 16 dims, those that share a scale: l, l + T, ... of its team of T lanes.
template <int OUT, bool BITS4, int U>                      // OUT: hisa_dtype
__global__ void __launch_bounds__(128) k_cache_read(CacheParams p) {
    constexpr int kK = 4 / U;                              // rows in flight per team
    const int lane = threadIdx.x & 31, T = p.lanes, per = 32 / T, sub = lane / T, tl = lane & (T - 1);
    const int64_t n0 = ((int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32) * p.chunk;
    const int units = p.D / 16;
    grid_dep_wait();
    grid_dep_trigger();
    check_offsets(p);
    if (n0 >= p.rows) return;
    const int n = (int)(p.rows - n0 < p.chunk ? p.rows - n0 : p.chunk);
    int64_t mine = -1;
    if (lane < n) mine = place_of(p, n0 + lane).slot;
    for (int r0 = 0; r0 < n; r0 += per * kK) {
        int64_t slot[kK];
        uint2 w[kK][U];
        uint32_t sc[kK][U];
        Raw8<__nv_bfloat16> raw[kK][U][2];
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            const int r = r0 + k * per + sub;
            slot[k] = __shfl_sync(0xffffffffu, mine, r & 31);
            if (r >= n) slot[k] = -1;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = i * T + tl;
                if (slot[k] < 0 || u >= units) continue;
                if constexpr (BITS4) {
                    w[k][i] = reinterpret_cast<const uint2 *>(p.cache)[slot[k] * units + u];
                    sc[k][i] = p.scales[slot[k] * units + u];
                } else {
                    raw[k][i][0].v[0] = reinterpret_cast<const uint4 *>(p.cache)[(slot[k] * units + u) * 2];
                    raw[k][i][1].v[0] = reinterpret_cast<const uint4 *>(p.cache)[(slot[k] * units + u) * 2 + 1];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            if (slot[k] < 0) continue;
            const int64_t row = n0 + r0 + k * per + sub;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = i * T + tl;
                if (u >= units) continue;
                if constexpr (OUT == HISA_E4M3) {
                    const uint2 lo = codes_to_e4m3(w[k][i].x), hi = codes_to_e4m3(w[k][i].y);
                    *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(p.out) + row * p.ld + 16 * u) = make_uint4(lo.x, lo.y, hi.x, hi.y);
                    if (p.out_scales) p.out_scales[row * units + u] = e4m3_to_f32(sc[k][i]) * p.g;
                } else {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float f[8];
                        if constexpr (BITS4) {
                            unpack_e2m1(half ? w[k][i].y : w[k][i].x, f);
                            const float s = e4m3_to_f32(sc[k][i]) * p.g;
#pragma unroll
                            for (int e = 0; e < 8; e += 2) {
                                const float2 z = mul2(make_float2(f[e], f[e + 1]), make_float2(s, s));
                                f[e] = z.x;
                                f[e + 1] = z.y;
                            }
                        } else {
                            raw_to_f32(raw[k][i][half], f);
                        }
                        const int64_t at = row * p.ld + 16 * u + 8 * half;
                        if constexpr (OUT == HISA_F32) {
                            float *to = static_cast<float *>(p.out) + at;
                            if (p.out32) {
                                store_sector(to, f);
                            } else {
                                reinterpret_cast<float4 *>(to)[0] = make_float4(f[0], f[1], f[2], f[3]);
                                reinterpret_cast<float4 *>(to)[1] = make_float4(f[4], f[5], f[6], f[7]);
                            }
                        } else {
                            store8(static_cast<__nv_bfloat16 *>(p.out) + at, f);
                        }
                    }
                }
            }
        }
    }
}

// Rows of a warp's chunk: whole rounds of its teams, up to 32, while there are `warps` warps per SM.
// Reading wants as many as fit (65536 rows of 512 dims to f32 29 us with 64 per SM, 36 with 32), appending
// half of that (20000 rows of 128 f32 dims 6.9 us with 32, 8.1 with 64): a chunk's places cost a chain of loads.
int chunk_of(int64_t rows, int per, int warps, int sms) {
    int chunk = 32;
    while (chunk > per && rows / chunk < warps * (int64_t)sms) chunk /= 2;
    return chunk;
}

template <typename K>
cudaError_t launch_rows(K kernel, CacheParams p, int lanes, int warps, size_t smem, cudaStream_t s) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    p.lanes = lanes;
    p.chunk = chunk_of(p.rows, 32 / p.lanes, warps, sms);
    const int64_t all = (p.rows + p.chunk - 1) / p.chunk, grid = (all + 3) / 4;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(128), smem, s, 1, p);
}

template <typename S, int U, int FORM>
cudaError_t append_as(const CacheParams &p, cudaStream_t s) {
    return launch_rows(k_cache_append<S, U, FORM>, p, team_lanes(p.D), 32, team_smem(p.D, p.dims, 4, FORM == kAny), s);
}
template <typename S>
cudaError_t append(const CacheParams &p, cudaStream_t s) {
    const int U = team_units(p.D);
    if (!p.wide) return U == 1 ? append_as<S, 1, kAny>(p, s) : (U == 2 ? append_as<S, 2, kAny>(p, s) : append_as<S, 4, kAny>(p, s));
    if (p.half) return U == 1 ? append_as<S, 1, kHalves>(p, s) : (U == 2 ? append_as<S, 2, kHalves>(p, s) : append_as<S, 4, kHalves>(p, s));
    return U == 1 ? append_as<S, 1, kPairs>(p, s) : (U == 2 ? append_as<S, 2, kPairs>(p, s) : append_as<S, 4, kPairs>(p, s));
}
template <int OUT, bool BITS4>
cudaError_t read_as(const CacheParams &p, cudaStream_t s) {
    int T = 2;
    while (T < p.D / 16 && T < 32) T *= 2;
    return p.D <= 512 ? launch_rows(k_cache_read<OUT, BITS4, 1>, p, T, 64, 0, s) : launch_rows(k_cache_read<OUT, BITS4, 2>, p, T, 64, 0, s);
}

}  // namespace

cudaError_t launch_cache_append(const CacheParams &p, cudaStream_t s) {
    return p.io_dtype == HISA_BF16 ? append<__nv_bfloat16>(p, s) : append<float>(p, s);
}

cudaError_t launch_cache_read(const CacheParams &p, cudaStream_t s) {
    if (p.io_dtype == HISA_E4M3) return read_as<HISA_E4M3, true>(p, s);
    if (p.io_dtype == HISA_F32) return p.bits4 ? read_as<HISA_F32, true>(p, s) : read_as<HISA_F32, false>(p, s);
    return p.bits4 ? read_as<HISA_BF16, true>(p, s) : read_as<HISA_BF16, false>(p, s);
}

}  // namespace hisa
