// Rotary positions of one or two tensors of heads.
//
//   (a, b) -> mscale (a cos A - b sin A, a sin A + b cos A),  A = pos[n] * f_i
//
// The angle is taken as a fraction of a turn in 64-bit fixed point: table[i] holds f_i / (2 pi)
// in units of 2^-64, so pos * table[i] modulo 2^64 drops the whole turns exactly, at any
// position, with one 64-bit integer product and no double arithmetic (which this GPU does at a
// small fraction of its f32 rate). What is left, in [-1/2, 1/2) turns, goes to sincospi in f32.
//
// Bound by memory. The heads of all tokens are one list of rows (token, head); a thread owns one
// unit of a row (8 neighbouring dims of one or of both halves, or a copied unit) and walks the
// CTA's rows, four loads in flight, so the sine and cosine of its pairs are computed once per
// token and not once per head. In place only the rotated dims move.
#include "ops_internal.cuh"

namespace hisa {
namespace {

constexpr int kUnroll = 4;

template <int N>
__device__ __forceinline__ void load_unit(const void *base, int64_t at, int bf16, float (&f)[N]) {
    if constexpr (N == 1) {
        f[0] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(base)[at]) : static_cast<const float *>(base)[at];
    } else if (bf16) {
        const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + at);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
        const float4 a = p[0], b = p[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
}
template <int N>
__device__ __forceinline__ void store_unit(void *base, int64_t at, int bf16, const float (&f)[N]) {
    if constexpr (N == 1) {
        if (bf16) static_cast<__nv_bfloat16 *>(base)[at] = __float2bfloat16_rn(f[0]);
        else static_cast<float *>(base)[at] = f[0];
    } else if (bf16) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(base) + at) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + at);
        p[0] = make_float4(f[0], f[1], f[2], f[3]);
        p[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// N dims per unit (8, or 1 where a boundary is not a multiple of 8). A rotated unit is two
// blocks of N dims, `lo` and `hi`: for the half layout the pairs (lo + e, hi + e); interleaved,
// for N = 8 one block holding 4 pairs (hi unused), for N = 1 the pair (lo, hi).
template <int N, bool HALF>
__global__ void __launch_bounds__(N == 8 ? 256 : 1024) k_rope(RopeParams p) {
    constexpr bool kTwo = HALF || N == 1;                 // a rotated unit is two blocks
    constexpr int kPairs = kTwo ? N : N / 2;
    const int n_rot = p.dims / (kTwo ? 2 * N : N);
    const int n = n_rot + (p.inplace ? 0 : (p.D - p.dims) / N);
    const int per = blockDim.x / n;                       // rows the CTA takes at once
    const int unit = threadIdx.x % n, sub = threadIdx.x / n;
    const int64_t r0 = (int64_t)blockIdx.x * p.rows_per_cta;
    int64_t r1 = r0 + p.rows_per_cta;
    r1 = r1 < p.rows ? r1 : p.rows;
    const bool rot = unit < n_rot;
    int lo, hi = 0;
    uint64_t freq[kPairs];
    if (rot) {
        if (HALF) { lo = p.first + unit * N; hi = lo + p.dims / 2; }
        else if (N == 1) { lo = p.first + 2 * unit; hi = lo + 1; }
        else lo = p.first + unit * N;
#pragma unroll
        for (int e = 0; e < kPairs; ++e) freq[e] = __ldg(p.table + unit * kPairs + e);
    } else {
        lo = (unit - n_rot) * N;                          // copied units: the dims before, then after, the rotated
        if (lo >= p.first) lo += p.dims;
    }
    grid_dep_wait();
    float cs[kPairs], sn[kPairs];
    int64_t have = -1;                                    // the token of cs and sn
    for (int64_t base = r0 + sub; base < r1; base += (int64_t)per * kUnroll) {
        float a[kUnroll][N], b[kTwo ? kUnroll : 1][N];
        int64_t tok[kUnroll];
        int head[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int64_t row = base + (int64_t)k * per;
            tok[k] = row / p.heads_all;
            head[k] = (int)(row - tok[k] * p.heads_all);
            if (row >= r1) continue;
            const bool two = head[k] >= p.heads;
            const void *src = two ? p.x2 : p.x;
            const int64_t at = two ? tok[k] * p.x2_token + (head[k] - p.heads) * p.x2_head
                                   : tok[k] * p.x_token + head[k] * p.x_head;
            load_unit<N>(src, at + lo, p.src_bf16, a[k]);
            if constexpr (kTwo)
                if (rot) load_unit<N>(src, at + hi, p.src_bf16, b[k]);
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            if (base + (int64_t)k * per >= r1) break;
            if (rot) {
                if (tok[k] != have) {
                    have = tok[k];
                    const int64_t pos = p.pos[have];
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) {
                        const int64_t turns = (int64_t)((uint64_t)pos * freq[e]);      // modulo one turn
                        float s, c;
                        sincospif(2.f * (__ll2float_rn(turns) * 0x1p-64f), &s, &c);
                        cs[e] = c * p.mscale;
                        sn[e] = s * p.mscale * p.sin_sign;
                    }
                }
                if constexpr (kTwo) {
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float u = a[k][e], v = b[k][e];
                        a[k][e] = u * cs[e] - v * sn[e];
                        b[k][e] = u * sn[e] + v * cs[e];
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) {
                        const float u = a[k][2 * e], v = a[k][2 * e + 1];
                        a[k][2 * e] = u * cs[e] - v * sn[e];
                        a[k][2 * e + 1] = u * sn[e] + v * cs[e];
                    }
                }
            }
            const bool two = head[k] >= p.heads;
            void *dst = two ? p.y2 : p.y;
            const int64_t at = two ? tok[k] * p.y2_token + (head[k] - p.heads) * p.y2_head
                                   : tok[k] * p.y_token + head[k] * p.y_head;
            store_unit<N>(dst, at + lo, p.dst_bf16, a[k]);
            if constexpr (kTwo)
                if (rot) store_unit<N>(dst, at + hi, p.dst_bf16, b[k]);
        }
    }
}

template <int N>
cudaError_t launch_n(RopeParams p, cudaStream_t s) {
    const bool two = p.half || N == 1;
    const int n = p.dims / (two ? 2 * N : N) + (p.inplace ? 0 : (p.D - p.dims) / N);
    const int most = N == 8 ? 256 : 1024;                 // n <= 128 units of 8, n <= 1023 of 1
    int per = most / n;
    if (N == 1 && per > 1) per = (256 + n - 1) / n < per ? (256 + n - 1) / n : per;
    if (per > p.rows) per = (int)p.rows;
    const int threads = per * n;
    // rows per CTA: four loads per thread, more once every SM has several CTAs, so that a token's
    // sines serve more of its heads
    const int64_t few = (int64_t)per * kUnroll;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    int64_t mul = p.rows / (few * sms * 8);
    mul = mul < 1 ? 1 : (mul > 4 ? 4 : mul);
    p.rows_per_cta = (int)(few * mul);
    const int64_t grid = (p.rows + p.rows_per_cta - 1) / p.rows_per_cta;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto kernel = p.half ? k_rope<N, true> : k_rope<N, false>;
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(threads), 0, s, p.chained, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, cudaStream_t s) {
    if (p.rows == 0) return cudaSuccess;
    return p.wide ? launch_n<8>(p, s) : launch_n<1>(p, s);
}

}  // namespace hisa
