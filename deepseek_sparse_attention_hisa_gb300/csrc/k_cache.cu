// Combine over a cache in pages on CUDA cores: every shape and type but 64 bf16 heads of 512 dims.
//
// One softmax over [visible window | pooled rows seen | sink] per query row and head, K = V. A query
// row's list is cut into ranges; a CTA takes all H heads of one query row and one range, 32 list rows
// at a time: their places are found by one warp, their values staged in f32, scores and sums kept in f32
// registers with a running maximum and sum per head. The ranges' sums join in k_prefix_merge; a list of one
// range is finished by its CTA.
//
// Bound by the FMA pipe and its shared-memory operands where the list is long, else by the latency of its few chunks
// (load, score, maximum, sum: 3 to 4 us each): 7 sequences of 3 rows of 16 x 128 in f32 over up to 1003 rows in bf16 16.6 us with the merge.
#include "cache_internal.cuh"

namespace hisa {
namespace {

constexpr int kChunk = 32;

template <int R, int DH>
struct Smem {
    static constexpr int kStride = DH + 4;               // floats per staged row: 16 bytes of pad
    static constexpr size_t bytes = (size_t)((R + kChunk) * kStride + R * (kChunk + 1)) * sizeof(float);
};

template <typename T>
__device__ __forceinline__ float4 load4(const T *p) {
    if constexpr (sizeof(T) == 4) {
        return *reinterpret_cast<const float4 *>(p);
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                           __uint_as_float(u.y & 0xffff0000u));
    }
}

template <int R>
constexpr int kPer = R == 64 ? 4 : 2;

// Thread (tr, tc) of TR x 16 owns kPer heads tr + TR i, their scores of chunk rows tc + 16 j, and
// dims 4 tc + 64 j of their sums.
template <int R, int DH, typename T, bool BITS4>
__global__ void __launch_bounds__(R / kPer<R> * 16, R == 64 ? 1 : 64 / R) k_cache_simt(CacheAttnParams p) {
    using S = Smem<R, DH>;
    constexpr int RP = kPer<R>, TR = R / RP, NT = TR * 16, DJ = DH / 64;
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *skv = sq + R * S::kStride, *sp = skv + kChunk * S::kStride;
    __shared__ int64_t places[2][kChunk];                // of a chunk's rows. -1: not seen; local rows from 1 << 62 on
    constexpr int64_t kLocal = (int64_t)1 << 62;
    const int tid = threadIdx.x, tr = tid / 16, tc = tid % 16;
    const int64_t row = blockIdx.x, rows = (int64_t)p.B * p.L * p.H;
    const int seg = blockIdx.y;
    grid_dep_wait();
    grid_dep_trigger();
    const CacheRow x = cache_row(p, row, seg == 0 && tid == 0);
    const int64_t total = (int64_t)x.nloc + x.npool, e0 = (int64_t)seg * p.split_rows;
    const int64_t e1 = e0 + p.split_rows < total ? e0 + p.split_rows : total;
    const T *q = static_cast<const T *>(p.q) + row * R * DH;
    for (int i = tid; i < R * (DH / 4); i += NT)
        *reinterpret_cast<float4 *>(sq + i / (DH / 4) * S::kStride + (i % (DH / 4)) * 4) = load4(q + i * 4);
    const T *loc = static_cast<const T *>(p.local_kv) + ((row / p.L) * p.W_max + x.lo) * DH;

    float2 acc[RP][DJ][2];
    float m[RP], l[RP];
#pragma unroll
    for (int i = 0; i < RP; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < DJ; ++j) acc[i][j][0] = acc[i][j][1] = make_float2(0.f, 0.f);
    }
    // Rows 4 dims at a time (in 4 bits two bytes); a chunk waits in registers while the one before is worked
    // on, but for 512 dims, whose sums leave no registers
    constexpr int kUnits = kChunk * (DH / 4) / NT;
    constexpr bool kAhead = kUnits <= 8;
    using Raw = typename std::conditional<sizeof(T) == 4, float4, uint2>::type;
    Raw raw[kAhead ? kUnits : 1];
    auto find = [&](int64_t c0, int64_t *place) {
        if (tid < kChunk) {
            const int64_t e = c0 + tid;
            place[tid] = e >= e1 ? -1 : (e < x.nloc ? kLocal + e : cache_slot(p, row, x, (int)(e - x.nloc)));
        }
    };
    auto fetch = [&](int i, const int64_t *place) -> Raw {   // local rows as they are, others in their first bytes
        const int64_t at = place[i / (DH / 4)];
        const int d = (i % (DH / 4)) * 4;
        Raw v{};
        if (at >= kLocal) {
            v = *reinterpret_cast<const Raw *>(loc + (at - kLocal) * DH + d);
        } else if (at >= 0) {
            if constexpr (BITS4) {
                const uint32_t w = *reinterpret_cast<const uint16_t *>(static_cast<const uint8_t *>(p.cache) + at * (DH / 2) + d / 2);
                const uint32_t s = p.scales[at * (DH / kScaleGroup) + d / kScaleGroup];
                reinterpret_cast<uint32_t &>(v) = w | s << 16;
            } else {
                reinterpret_cast<uint2 &>(v) = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.cache) + at * DH + d);
            }
        }
        return v;
    };
    auto stage = [&](int i, const Raw &r, const int64_t *place) {
        const int64_t at = place[i / (DH / 4)];
        float4 v;
        if (at >= kLocal || (!BITS4 && sizeof(T) == 2)) {
            v = load4(reinterpret_cast<const T *>(&r));
        } else if constexpr (BITS4) {
            const uint32_t w = reinterpret_cast<const uint32_t &>(r);
            const float s = e4m3_to_f32(w >> 16) * p.g;
            float f[8];
            unpack_e2m1(w & 0xffffu, f);
            v = make_float4(f[0] * s, f[1] * s, f[2] * s, f[3] * s);
        } else {
            v = load4(reinterpret_cast<const __nv_bfloat16 *>(&r));
        }
        *reinterpret_cast<float4 *>(skv + i / (DH / 4) * S::kStride + (i % (DH / 4)) * 4) = v;
    };
    find(e0, places[0]);
    find(e0 + kChunk, places[1]);
    __syncthreads();
    if constexpr (kAhead) {
#pragma unroll
        for (int k = 0; k < kUnits; ++k) raw[k] = fetch(tid + k * NT, places[0]);
    }
    int at_c = 0;
    for (int64_t c0 = e0; c0 < e1; c0 += kChunk, at_c ^= 1) {
        int64_t *place = places[at_c];
        if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < kUnits; ++k) stage(tid + k * NT, raw[k], place);
        } else {
            for (int i = tid; i < kChunk * (DH / 4); i += NT) stage(i, fetch(i, place), place);
        }
        const bool seen0 = place[tc] >= 0, seen1 = place[tc + 16] >= 0;
        __syncthreads();                                  // staged, and the places read
        if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < kUnits; ++k) raw[k] = fetch(tid + k * NT, places[at_c ^ 1]);
        }
        find(c0 + 2 * kChunk, place);
        float2 s[RP][2];                                  // even and odd dims' sums
#pragma unroll
        for (int i = 0; i < RP; ++i) s[i][0] = s[i][1] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int d = 0; d < DH; d += 4) {
            const float4 k0 = *reinterpret_cast<const float4 *>(skv + tc * S::kStride + d);
            const float4 k1 = *reinterpret_cast<const float4 *>(skv + (tc + 16) * S::kStride + d);
#pragma unroll
            for (int i = 0; i < RP; ++i) {
                const float4 a = *reinterpret_cast<const float4 *>(sq + (tr + TR * i) * S::kStride + d);
                const float2 lo = make_float2(a.x, a.y), hi = make_float2(a.z, a.w);
                s[i][0] = fma2(hi, make_float2(k0.z, k0.w), fma2(lo, make_float2(k0.x, k0.y), s[i][0]));
                s[i][1] = fma2(hi, make_float2(k1.z, k1.w), fma2(lo, make_float2(k1.x, k1.y), s[i][1]));
            }
        }
        float al[RP];
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            const float z0 = seen0 ? (s[i][0].x + s[i][0].y) * p.scale : -INFINITY;
            const float z1 = seen1 ? (s[i][1].x + s[i][1].y) * p.scale : -INFINITY;
            float mx = fmaxf(z0, z1);
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float mn = fmaxf(m[i], mx);
            const float ref = mn == -INFINITY ? 0.f : mn; // every logit so far is -inf: e^{-inf} = 0
            al[i] = expf(m[i] - ref);
            m[i] = mn;
            const float p0 = expf(z0 - ref), p1 = expf(z1 - ref);
            float sum = p0 + p1;
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l[i] = l[i] * al[i] + sum;
            sp[(tr + TR * i) * (kChunk + 1) + tc] = p0;
            sp[(tr + TR * i) * (kChunk + 1) + tc + 16] = p1;
        }
        __syncwarp();                                     // a head's 16 threads sit in one warp
#pragma unroll
        for (int i = 0; i < RP; ++i)
#pragma unroll
            for (int j = 0; j < DJ; ++j) {
                acc[i][j][0] = mul2(acc[i][j][0], make_float2(al[i], al[i]));
                acc[i][j][1] = mul2(acc[i][j][1], make_float2(al[i], al[i]));
            }
        // by fours: rows past the end are staged as zeros and weigh 0
        const int nk = e1 - c0 < kChunk ? ((int)(e1 - c0) + 3) & ~3 : kChunk;
#pragma unroll 4
        for (int k = 0; k < nk; ++k) {
            float w[RP];
#pragma unroll
            for (int i = 0; i < RP; ++i) w[i] = sp[(tr + TR * i) * (kChunk + 1) + k];
#pragma unroll
            for (int j = 0; j < DJ; ++j) {
                const float4 v = *reinterpret_cast<const float4 *>(skv + k * S::kStride + 4 * tc + 64 * j);
#pragma unroll
                for (int i = 0; i < RP; ++i) {
                    acc[i][j][0] = fma2(make_float2(w[i], w[i]), make_float2(v.x, v.y), acc[i][j][0]);
                    acc[i][j][1] = fma2(make_float2(w[i], w[i]), make_float2(v.z, v.w), acc[i][j][1]);
                }
            }
        }
        __syncthreads();                                  // the chunk has been read, places are written
    }
    if (p.splits == 1) {                                  // the whole list: the output itself
#pragma unroll
        for (int i = 0; i < RP; ++i) {
            const int h = tr + TR * i;
            const float sink = p.sinks ? p.sinks[h] : -INFINITY, M = fmaxf(m[i], sink), ref = M == -INFINITY ? 0.f : M;
            const float a = expf(m[i] - ref), den = l[i] * a + expf(sink - ref), f = den == 0.f ? 0.f : a / den;
            const int64_t at = (row * R + h) * DH + 4 * tc;
#pragma unroll
            for (int j = 0; j < DJ; ++j) {
                const float4 o = make_float4(acc[i][j][0].x * f, acc[i][j][0].y * f, acc[i][j][1].x * f, acc[i][j][1].y * f);
                if (p.out_bf16) {
                    const __nv_bfloat162 u = __floats2bfloat162_rn(o.x, o.y), v = __floats2bfloat162_rn(o.z, o.w);
                    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at + 64 * j) =
                        make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
                } else {
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at + 64 * j) = o;
                }
            }
        }
        return;
    }
    const int64_t g0 = (int64_t)seg * rows + row * R;
#pragma unroll
    for (int i = 0; i < RP; ++i) {
        const int64_t g = g0 + tr + TR * i;
        if (tc == 0) *reinterpret_cast<float2 *>(p.part_ml + g * 2) = make_float2(m[i], l[i]);
#pragma unroll
        for (int j = 0; j < DJ; ++j)
            *reinterpret_cast<float4 *>(p.part_o + g * DH + 4 * tc + 64 * j) =
                make_float4(acc[i][j][0].x, acc[i][j][0].y, acc[i][j][1].x, acc[i][j][1].y);
    }
}

template <int R, int DH, typename T, bool BITS4>
cudaError_t go(const CacheAttnParams &p, cudaStream_t s) {
    const size_t bytes = Smem<R, DH>::bytes;
    const cudaError_t e = smem_attr_once<k_cache_simt<R, DH, T, BITS4>>((int)bytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_cache_simt<R, DH, T, BITS4>, dim3((unsigned)(p.B * p.L), (unsigned)p.splits), dim3(R / kPer<R> * 16), bytes, s, 1, p);
}
template <int R, int DH>
cudaError_t types(const CacheAttnParams &p, cudaStream_t s) {
    if (p.q_bf16) return p.bits4 ? go<R, DH, __nv_bfloat16, true>(p, s) : go<R, DH, __nv_bfloat16, false>(p, s);
    return p.bits4 ? go<R, DH, float, true>(p, s) : go<R, DH, float, false>(p, s);
}

}  // namespace

cudaError_t launch_cache_simt(const CacheAttnParams &p, cudaStream_t s) {
    cudaError_t e;
    if (p.Dh == 64) e = types<8, 64>(p, s);
    else if (p.Dh == 128) e = types<16, 128>(p, s);
    else if (p.q_bf16) return cudaErrorInvalidValue;      // k_cache_tc.cu
    else e = p.bits4 ? go<64, 512, float, true>(p, s) : go<64, 512, float, false>(p, s);
    if (e != cudaSuccess || p.splits == 1) return e;
    PrefixParams m{};
    m.B = p.B; m.L = p.L; m.H = p.H; m.Dh = p.Dh;
    m.sinks = p.sinks; m.out = p.out; m.out_bf16 = p.out_bf16;
    m.tail_split = p.splits;
    m.part_o = p.part_o; m.part_ml = p.part_ml;
    return launch_prefix_merge(m, s);
}

}  // namespace hisa
