// Shared-prefix combine: the CUDA-core segments and the merge of all segments.
//
// One softmax over  [local window | P shared rows | own pooled rows | sink]  per query row and
// head, K = V. Its statistics join over disjoint sets of rows: a segment s with logits z_i and
// rows v_i keeps m_s = max z_i, l_s = sum e^{z_i - m_s}, O_s = sum e^{z_i - m_s} v_i, and
//   M = max(max_s m_s, sink),  out = sum_s e^{m_s - M} O_s / (sum_s e^{m_s - M} l_s + e^{sink - M}).
// So the shared rows, which every query row of the batch sees whole, become segments whose query
// rows are stacked across sequences (one staged chunk of shared rows serves R stacked rows),
// and the local and own rows become segments of one query row each.
//
// The kernel here serves f32, and the own lists of bf16 heads of 64 and 128 dims: R query rows x
// 32 list rows per chunk, 16 threads per two or four rows, scores and sums in f32 registers, the
// running maximum and sum per row (a rescale per chunk). Bound by the FMA pipe and its
// shared-memory operands; two products go into one instruction. Measured: the own lists (up to
// 512 rows) of 300 query rows of 16 x 128 bf16 63 us; a call of 7 x 3 query rows of 16 x 128 f32 over
// 1003 shared rows 21 us, the latency of three dependent kernels (its products would take 2.6); 76
// query rows of 64 x 512 f32 over 1000 shared rows 330 us, 34 TFLOP/s.
#include "prefix_common.cuh"

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

// One item: R stacked query rows (shared rows) or the R = H heads of one query row (its own
// list), and one segment of the list. Thread (tr, tc) of TR x 16 owns kPer rows tr + TR i,
// their scores of chunk rows tc + 16 j, and dims 4 tc + 64 j of their sums.
template <int R>
constexpr int kPer = R == 64 ? 4 : 2;
template <int R, int DH, typename T>
__global__ void __launch_bounds__(R / kPer<R> * 16, R == 64 ? 1 : 64 / R) k_prefix_simt(PrefixParams p, int tail) {
    using S = Smem<R, DH>;
    constexpr int RP = kPer<R>, TR = R / RP, NT = TR * 16, DJ = DH / 64;
    constexpr int LD = kChunk * (DH / 4) / NT;            // units of four dims per thread and chunk
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *skv = sq + R * S::kStride, *sp = skv + kChunk * S::kStride;
    const int tid = threadIdx.x, tr = tid / 16, tc = tid % 16;
    const int seg = blockIdx.y;
    const int64_t rows = (int64_t)p.B * p.L * p.H;
    const int64_t g0 = (int64_t)blockIdx.x * R;
    // The own lists' kernel comes first and lets the shared rows' start beside it, once all work
    // before it has completed; that one depends on nothing of it and waits for it at its end, so
    // that the merge, which waits for the last grid, has both.
    if (tail || !p.tail_split) grid_dep_wait();
    grid_dep_trigger();
    Tail x{0, 0, 0, 0};
    int64_t e0, e1;
    if (tail) {
        x = tail_of(p, blockIdx.x, tail_fetch(p, blockIdx.x), seg == 0 && tid == 0);
        e0 = (int64_t)seg * p.tail_rows;
        e1 = e0 + p.tail_rows;
        const int64_t n = x.nloc + x.nown;
        e1 = e1 < n ? e1 : n;
    } else {
        e0 = (int64_t)seg * p.pre_rows;
        e1 = e0 + p.pre_rows;
        e1 = e1 < p.P ? e1 : p.P;
    }
    const T *q = static_cast<const T *>(p.q);
    for (int i = tid; i < R * (DH / 4); i += NT) {
        const int r = i / (DH / 4), d = (i % (DH / 4)) * 4;
        const float4 v = g0 + r < rows ? load4(q + (g0 + r) * DH + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(sq + r * S::kStride + d) = v;
    }
    const int b = tail ? (int)blockIdx.x / p.L : 0;
    const T *loc = static_cast<const T *>(p.local_kv) + ((int64_t)b * p.W_max + x.lo) * DH;
    const T *own = static_cast<const T *>(p.pooled_kv) + x.k0 * DH;
    const T *pre = static_cast<const T *>(p.prefix_kv);

    float2 acc[RP][DJ][2];
    float m[RP], l[RP];
#pragma unroll
    for (int i = 0; i < RP; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < DJ; ++j) acc[i][j][0] = acc[i][j][1] = make_float2(0.f, 0.f);
    }
    // a chunk waits in registers while the one before is worked on, but for 512 dims: 64 more registers
    // beside 128 of sums spill (76 x 64 x 512 f32 over 1000 rows 330 us without, 373 with; 304 rows over
    // 4096 and up to 512 own 4.81 against 5.23 ms; 1 row over 8000 77 against 86 us)
    constexpr bool kAhead = LD < 16;
    using Raw = typename std::conditional<sizeof(T) == 4, float4, uint2>::type;
    Raw raw[kAhead ? LD : 1];
    auto at = [&](int64_t c0, int i) -> const T * {
        const int64_t e = c0 + i / (DH / 4);
        if (e >= e1) return nullptr;
        return (tail ? (e < x.nloc ? loc + e * DH : own + (e - x.nloc) * DH) : pre + e * DH) + (i % (DH / 4)) * 4;
    };
    auto fetch = [&](int64_t c0) {
#pragma unroll
        for (int k = 0; k < LD; ++k) {
            const T *src = at(c0, tid + k * NT);
            raw[k] = Raw{};
            if (src) raw[k] = *reinterpret_cast<const Raw *>(src);
        }
    };
    auto put = [&](int i, const float4 &v) {
        *reinterpret_cast<float4 *>(skv + i / (DH / 4) * S::kStride + (i % (DH / 4)) * 4) = v;
    };
    if constexpr (kAhead) fetch(e0);
    for (int64_t c0 = e0; c0 < e1; c0 += kChunk) {
        __syncthreads();                                  // the previous chunk has been read
        if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < LD; ++k) put(tid + k * NT, load4(reinterpret_cast<const T *>(&raw[k])));
        } else {
            for (int i = tid; i < kChunk * (DH / 4); i += NT) {
                const T *src = at(c0, i);
                put(i, src ? load4(src) : make_float4(0.f, 0.f, 0.f, 0.f));
            }
        }
        __syncthreads();
        if constexpr (kAhead) fetch(c0 + kChunk);
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
            const float z0 = c0 + tc < e1 ? (s[i][0].x + s[i][0].y) * p.scale : -INFINITY;
            const float z1 = c0 + tc + 16 < e1 ? (s[i][1].x + s[i][1].y) * p.scale : -INFINITY;
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
        __syncwarp();                                     // a row's 16 threads sit in one warp
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
        __syncwarp();                                     // sp is read before the next chunk's is written
    }
    const int64_t seg0 = (int64_t)((tail ? 0 : p.tail_split) + seg) * rows;
#pragma unroll
    for (int i = 0; i < RP; ++i) {
        const int64_t g = g0 + tr + TR * i;
        if (g >= rows) continue;
        if (tc == 0) *reinterpret_cast<float2 *>(p.part_ml + (seg0 + g) * 2) = make_float2(m[i], l[i]);
#pragma unroll
        for (int j = 0; j < DJ; ++j)
            *reinterpret_cast<float4 *>(p.part_o + (seg0 + g) * DH + 4 * tc + 64 * j) = make_float4(acc[i][j][0].x, acc[i][j][0].y, acc[i][j][1].x, acc[i][j][1].y);
    }
    if (!tail) grid_dep_wait();
}

// Joins the segments of a (query row, head) and the sink: DH / 4 threads, four dims each. Bound by
// memory: every segment's sums are read once. With few rows there are many segments to each (up to
// 128), whose loads one after another would take longer than the segments themselves (1 x 8 x 64
// f32 over 8000 shared rows: 36 us for the call, 18 so): then (ALL) a CTA's threads share one row,
// the statistics are loaded at once, and groups of DH / 4 threads take every k-th segment.
constexpr int kMergeThreads = 256, kMaxSegs = 128;

template <int DH>
__device__ __forceinline__ void put_merged(const PrefixParams &p, int64_t g, int d, float4 o, float den) {
    const float f = den == 0.f ? 0.f : 1.f / den;         // nothing visible, no sink: 0
    o.x *= f; o.y *= f; o.z *= f; o.w *= f;
    if (p.out_bf16) {
        const __nv_bfloat162 u = __floats2bfloat162_rn(o.x, o.y), v = __floats2bfloat162_rn(o.z, o.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + g * DH + d) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + g * DH + d) = o;
    }
}

template <int DH, bool ALL>
__global__ void __launch_bounds__(kMergeThreads) k_prefix_merge(PrefixParams p) {
    constexpr int kT = DH / 4, kGroups = kMergeThreads / kT;
    grid_dep_wait();
    grid_dep_trigger();
    const int64_t rows = (int64_t)p.B * p.L * p.H;
    const int grp = threadIdx.x / kT, d = (threadIdx.x % kT) * 4;
    const int nseg = p.tail_split + p.pre_split;
    auto stats = [&](int s, int64_t g) { return *reinterpret_cast<const float2 *>(p.part_ml + (s * rows + g) * 2); };
    // a segment that holds nothing has no sums to read
    auto empty = [](float2 ml) { return ml.x == -INFINITY && ml.y == 0.f; };
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (!ALL) {
        const int64_t g = (int64_t)blockIdx.x * kGroups + grp;
        if (g >= rows) return;
        const float sink = p.sinks ? p.sinks[g % p.H] : -INFINITY;
        float M = sink;
#pragma unroll 4
        for (int s = 0; s < nseg; ++s) M = fmaxf(M, stats(s, g).x);
        const float ref = M == -INFINITY ? 0.f : M;
        float den = expf(sink - ref);
#pragma unroll 4
        for (int s = 0; s < nseg; ++s) {
            const float2 ml = stats(s, g);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!empty(ml)) v = __ldcs(reinterpret_cast<const float4 *>(p.part_o + (s * rows + g) * DH + d));
            const float a = empty(ml) ? 0.f : expf(ml.x - ref);
            den += ml.y * a;
            o.x += v.x * a; o.y += v.y * a; o.z += v.z * a; o.w += v.w * a;
        }
        put_merged<DH>(p, g, d, o, den);
    } else {
        __shared__ float weight[kMaxSegs];                // e^{m - M}; -1: nothing there
        __shared__ float2 ml[kMaxSegs];
        __shared__ float4 part[kGroups][kT];
        const int64_t g = blockIdx.x;
        for (int s = threadIdx.x; s < nseg; s += kMergeThreads) ml[s] = stats(s, g);
        __syncthreads();
        const float sink = p.sinks ? p.sinks[g % p.H] : -INFINITY;
        float M = sink;
        for (int s = 0; s < nseg; ++s) M = fmaxf(M, ml[s].x);
        const float ref = M == -INFINITY ? 0.f : M;
        for (int s = threadIdx.x; s < nseg; s += kMergeThreads) weight[s] = empty(ml[s]) ? -1.f : expf(ml[s].x - ref);
        __syncthreads();
#pragma unroll 4
        for (int s = grp; s < nseg; s += kGroups) {
            const float a = weight[s];
            const bool none = a < 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!none) v = __ldcs(reinterpret_cast<const float4 *>(p.part_o + (s * rows + g) * DH + d));
            const float b = none ? 0.f : a;
            o.x += v.x * b; o.y += v.y * b; o.z += v.z * b; o.w += v.w * b;
        }
        part[grp][d / 4] = o;
        __syncthreads();
        if (grp) return;
        float den = expf(sink - ref);
        for (int s = 0; s < nseg; ++s)
            if (!(weight[s] < 0.f)) den += ml[s].y * weight[s];
#pragma unroll
        for (int k = 1; k < kGroups; ++k) {
            const float4 v = part[k][d / 4];
            o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
        }
        put_merged<DH>(p, g, d, o, den);
    }
}

template <int R, int DH, typename T>
cudaError_t go(const PrefixParams &p, int tail, cudaStream_t s) {
    const size_t bytes = Smem<R, DH>::bytes;
    const cudaError_t e = smem_attr_once<k_prefix_simt<R, DH, T>>((int)bytes);
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)p.B * p.L * p.H;
    const int64_t tiles = (rows + R - 1) / R;
    return launch_pdl(k_prefix_simt<R, DH, T>, dim3((unsigned)tiles, (unsigned)(tail ? p.tail_split : p.pre_split)),
                      dim3(R / kPer<R> * 16), bytes, s, 1, p, tail);
}

template <typename T>
cudaError_t pick(const PrefixParams &p, int tail, cudaStream_t s) {
    if (tail && p.Dh == 64) return go<8, 64, T>(p, 1, s);
    if (tail && p.Dh == 128) return go<16, 128, T>(p, 1, s);
    if constexpr (sizeof(T) == 4) {                       // in bf16: k_prefix_tc.cu and k_prefix_tc1.cu
        if (p.Dh == 64) return go<64, 64, T>(p, 0, s);
        if (p.Dh == 128) return go<64, 128, T>(p, 0, s);
        return go<64, 512, T>(p, tail, s);
    }
    return cudaErrorInvalidValue;
}

template <int DH>
cudaError_t merge(const PrefixParams &p, cudaStream_t s) {
    const int64_t rows = (int64_t)p.B * p.L * p.H;
    constexpr int kGroups = kMergeThreads / (DH / 4);
    // a CTA per row while all rows are on the GPU at once, and more segments than a thread's loads in
    // flight (at 1120 rows of 128 and 5 segments it costs 2 us)
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    if (rows <= 4 * sms && p.tail_split + p.pre_split > 4)
        return launch_pdl(k_prefix_merge<DH, true>, dim3((unsigned)rows), dim3(kMergeThreads), 0, s, 1, p);
    return launch_pdl(k_prefix_merge<DH, false>, dim3((unsigned)((rows + kGroups - 1) / kGroups)), dim3(kMergeThreads), 0, s, 1, p);
}

}  // namespace

cudaError_t launch_prefix_simt(const PrefixParams &p, int tail, cudaStream_t s) {
    return p.bf16 ? pick<__nv_bfloat16>(p, tail, s) : pick<float>(p, tail, s);
}

cudaError_t launch_prefix_merge(const PrefixParams &p, cudaStream_t s) {
    if (p.tail_split + p.pre_split > kMaxSegs) return cudaErrorInvalidValue;
    if (p.Dh == 64) return merge<64>(p, s);
    if (p.Dh == 128) return merge<128>(p, s);
    return merge<512>(p, s);
}

}  // namespace hisa
