// Residual addition, root-mean-square norm and output (f32, bf16, or e4m3 with scales) in one
// pass: every input element is read once and every output element written once.
//
//   h = round(x + residual);  y = h * w / sqrt(mean(h^2) + eps);  out = round(y)  or
//   scale_g = max(max_g |y|, 1e-10) / 448 (up to a power of two),  out = e4m3(y / scale_g)
//
// Bound by memory: about 6 operations per element against 4 to 16 bytes. A team of threads
// holds a whole row in registers (a warp for rows of at most 1024 columns, else a CTA), so the
// sum of squares, the scales and the output need no second read. Teams walk the rows with a
// grid stride, and a team fetches its next row before it reduces the current one, so the
// barrier of the reduction does not leave the memory system idle. Sums are f32: each thread's
// own columns in order, then a fixed tree over lanes and warps, so a row's result does not
// depend on the other rows or on the launch.
#include <cuda_fp8.h>

#include "ops_internal.cuh"

namespace hisa {
namespace {

struct None {};                       // no residual

template <typename T> struct Raw8 { uint4 v[sizeof(T) / 2]; };   // 8 elements as loaded
template <> struct Raw8<None> {};

template <typename T>
__device__ __forceinline__ void load_raw(Raw8<T> &r, const void *base, int64_t at) {
    if constexpr (!std::is_same<T, None>::value) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const T *>(base) + at);
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.v[i] = __ldcs(p + i);
    }
}
__device__ __forceinline__ void unpack(const Raw8<__nv_bfloat16> &r, float (&f)[8]) {
    const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const Raw8<float> &r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(r.v[i].x);
        f[4 * i + 1] = __uint_as_float(r.v[i].y);
        f[4 * i + 2] = __uint_as_float(r.v[i].z);
        f[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
}
__device__ __forceinline__ uint4 pack_bf16(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(void *base, int64_t at, bool bf16, const float (&f)[8]) {
    if (bf16) {
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(base) + at) = pack_bf16(f);
    } else {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + at);
        p[0] = make_float4(f[0], f[1], f[2], f[3]);
        p[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Largest magnitude as bits: NaN orders above infinity, so a group that holds one gets a NaN scale.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int lanes) {
    for (int o = lanes >> 1; o >= 1; o >>= 1) {
        const uint32_t u = __shfl_xor_sync(0xffffffffu, v, o);
        v = u > v ? u : v;
    }
    return v;
}

// Scale of a group whose largest magnitude has these bits. The floor keeps the quotient normal.
__device__ __forceinline__ float scale_of(uint32_t bits, int pow2) {
    float a = __uint_as_float(bits);
    a = a < 1e-10f ? 1e-10f : a;
    float s = a / 448.f;
    if (pow2 && s < INFINITY) {
        const uint32_t u = __float_as_uint(s);
        s = __uint_as_float((u & 0x7f800000u) + ((u & 0x007fffffu) ? 0x00800000u : 0u));
    }
    return s;
}

// Sum (or maximum) over the block's warps: one partial per warp, one barrier. Callers alternate
// between two arrays, so the next call's writes meet no late reader.
__device__ __forceinline__ float block_sum(float v, float *red, int warps) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += red[w];
    return s;
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *red, int warps) {
    v = lanes_max(v, 32);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t s = 0;
    for (int w = 0; w < warps; ++w) s = red[w] > s ? red[w] : s;
    return s;
}

// Rows moved in units of 8 columns. WARP: a warp per row, else the CTA per row.
template <typename XT, typename RT, int VPT, bool WARP>
__global__ void __launch_bounds__(VPT <= 2 || WARP ? 512 : 1024, VPT <= 2 && !WARP ? 2 : 1) k_norm_wide(NormParams p) {
    constexpr bool kRes = !std::is_same<RT, None>::value;
    constexpr bool kPrefetch = VPT <= 2 || WARP;
    __shared__ float red[2][32];
    __shared__ uint32_t redm[2][32];
    const int T = WARP ? 32 : blockDim.x;
    const int t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int warps = blockDim.x >> 5;
    const int nvec = p.cols >> 3;
    const int64_t step = WARP ? (int64_t)gridDim.x * warps : gridDim.x;
    const float inv = 1.f / (float)p.cols;
    int64_t row = WARP ? (int64_t)blockIdx.x * warps + (threadIdx.x >> 5) : blockIdx.x;

    float w[VPT][8];                                  // this thread's columns, the same for every row
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = i * T + t;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[i][e] = 0.f;
        if (v < nvec) {
            const float4 *wp = reinterpret_cast<const float4 *>(p.w + (int64_t)v * 8);
            const float4 a = __ldg(wp), b = __ldg(wp + 1);
            w[i][0] = a.x; w[i][1] = a.y; w[i][2] = a.z; w[i][3] = a.w;
            w[i][4] = b.x; w[i][5] = b.y; w[i][6] = b.z; w[i][7] = b.w;
        }
    }
    grid_dep_wait();
    Raw8<XT> x[VPT];
    Raw8<RT> r[VPT];
    auto fetch = [&](int64_t at) {
        if (at >= p.rows) return;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * T + t;
            if (v < nvec) {
                load_raw(x[i], p.x, at * p.ld_x + (int64_t)v * 8);
                load_raw(r[i], p.res, at * p.ld_res + (int64_t)v * 8);
            }
        }
    };
    fetch(row);
    for (int par = 0; row < p.rows; row += step, par ^= 1) {
        float h[VPT][8];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * T + t;
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = 0.f;
            if (v >= nvec) continue;
            unpack(x[i], h[i]);
            if constexpr (kRes) {
                float q[8];
                unpack(r[i], q);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] += q[e];
                if constexpr (std::is_same<RT, __nv_bfloat16>::value) {
                    Raw8<__nv_bfloat16> back;
                    back.v[0] = pack_bf16(h[i]);
                    unpack(back, h[i]);                // the norm is over the sum as stored
                }
                if (p.res_out) store8(p.res_out, row * p.ld_res + (int64_t)v * 8, std::is_same<RT, __nv_bfloat16>::value, h[i]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss += h[i][e] * h[i][e];
        }
        if (kPrefetch) fetch(row + step);
        ss = WARP ? warp_sum(ss) : block_sum(ss, red[par], warps);
        const float f = 1.f / sqrtf(ss * inv + p.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = h[i][e] * f * w[i][e];
        if (p.out_dtype != HISA_E4M3) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int v = i * T + t;
                if (v < nvec) store8(p.out, row * p.ld_out + (int64_t)v * 8, p.out_dtype == HISA_BF16, h[i]);
            }
        } else {
            uint32_t top[VPT];
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                top[i] = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t u = mag(h[i][e]);
                    top[i] = u > top[i] ? u : top[i];
                }
            }
            if (p.group == 0) {
#pragma unroll
                for (int i = 1; i < VPT; ++i) top[0] = top[i] > top[0] ? top[i] : top[0];
                const uint32_t all = WARP ? lanes_max(top[0], 32) : block_max(top[0], redm[par], warps);
#pragma unroll
                for (int i = 0; i < VPT; ++i) top[i] = all;
            } else {
#pragma unroll
                for (int i = 0; i < VPT; ++i) top[i] = lanes_max(top[i], p.group >> 3);
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int v = i * T + t;
                if (v >= nvec) continue;
                const float s = scale_of(top[i], p.pow2);
                const float q = 1.f / s;               // one division per unit; y * q is within an f32 step or two of y / s
                const int lane0 = p.group ? (v & ((p.group >> 3) - 1)) : v;
                if (lane0 == 0) p.scales[p.group ? row * (p.cols / p.group) + v / (p.group >> 3) : row] = s;
                uint32_t c[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(h[i][4 * k] * q, h[i][4 * k + 1] * q),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(h[i][4 * k + 2] * q, h[i][4 * k + 3] * q),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    c[k] = lo | (hi << 16);
                }
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.out) + row * p.ld_out + (int64_t)v * 8) =
                    make_uint2(c[0], c[1]);
            }
        }
        if (!kPrefetch) fetch(row + step);
    }
}

template <typename T>
__device__ __forceinline__ float load1(const void *base, int64_t at) {
    if constexpr (std::is_same<T, None>::value) return 0.f;
    else return to_f32(__ldcs(static_cast<const T *>(base) + at));
}

// Rows whose starts are not 16-byte aligned or whose length is not a multiple of 8: one CTA per
// row, single elements, neighbouring threads on neighbouring columns. A warp's 32 columns lie
// in one scale group (groups are multiples of 32), whose maximum is joined in shared memory.
template <typename XT, typename RT, int EPT>
__global__ void __launch_bounds__(1024, 1) k_norm_narrow(NormParams p) {
    constexpr bool kRes = !std::is_same<RT, None>::value;
    __shared__ float red[2][32];
    __shared__ uint32_t redm[2][32];
    __shared__ uint32_t gmax[1024];
    const int T = blockDim.x, t = threadIdx.x, warps = T >> 5;
    const float inv = 1.f / (float)p.cols;
    grid_dep_wait();
    int par = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, par ^= 1) {
        float h[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const int c = i * T + t;
            h[i] = c < p.cols ? load1<XT>(p.x, row * p.ld_x + c) : 0.f;
        }
        if constexpr (kRes) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const int c = i * T + t;
                if (c < p.cols) h[i] += load1<RT>(p.res, row * p.ld_res + c);
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const int c = i * T + t;
            if constexpr (kRes) {
                const int64_t at = row * p.ld_res + c;
                if constexpr (std::is_same<RT, __nv_bfloat16>::value) {
                    const __nv_bfloat16 b = __float2bfloat16_rn(h[i]);
                    h[i] = __bfloat162float(b);
                    if (p.res_out && c < p.cols) static_cast<__nv_bfloat16 *>(p.res_out)[at] = b;
                } else {
                    if (p.res_out && c < p.cols) static_cast<float *>(p.res_out)[at] = h[i];
                }
            }
            ss += h[i] * h[i];
        }
        ss = block_sum(ss, red[par], warps);
        const float f = 1.f / sqrtf(ss * inv + p.eps);
        uint32_t all = 0;
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const int c = i * T + t;
            h[i] = c < p.cols ? h[i] * f * __ldg(p.w + c) : 0.f;
        }
        if (p.out_dtype != HISA_E4M3) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const int c = i * T + t;
                if (c >= p.cols) continue;
                if (p.out_dtype == HISA_BF16)
                    static_cast<__nv_bfloat16 *>(p.out)[row * p.ld_out + c] = __float2bfloat16_rn(h[i]);
                else
                    static_cast<float *>(p.out)[row * p.ld_out + c] = h[i];
            }
            continue;
        }
        if (p.group == 0) {
#pragma unroll
            for (int i = 0; i < EPT; ++i) all = mag(h[i]) > all ? mag(h[i]) : all;
            all = block_max(all, redm[par], warps);
        } else {
#pragma unroll
            for (int i = 0; i < EPT; ++i) {
                const uint32_t m = lanes_max(mag(h[i]), 32);
                const int c = i * T + t;
                if ((t & 31) == 0 && c < p.cols) gmax[c >> 5] = m;
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
            const int c = i * T + t;
            if (c >= p.cols) continue;
            uint32_t top = all;
            if (p.group) {
                const int g0 = c / p.group * (p.group >> 5);
                for (int k = 0; k < (p.group >> 5); ++k) top = gmax[g0 + k] > top ? gmax[g0 + k] : top;
            }
            const float s = scale_of(top, p.pow2);
            if (p.group ? c % p.group == 0 : c == 0) p.scales[p.group ? row * (p.cols / p.group) + c / p.group : row] = s;
            static_cast<uint8_t *>(p.out)[row * p.ld_out + c] = __nv_cvt_float_to_fp8(h[i] * (1.f / s), __NV_SATFINITE, __NV_E4M3);
        }
        if (p.group) __syncthreads();                  // gmax is read before the next row's is written
    }
}

template <auto Kernel>
cudaError_t go(const NormParams &p, int threads, int64_t rows_per_cta, cudaStream_t s) {
    // as many CTAs as the SMs hold at once; they walk the rows
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    int per = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, Kernel, threads, 0);
    if (e != cudaSuccess) return e;
    const int64_t want = (p.rows + rows_per_cta - 1) / rows_per_cta, most = (int64_t)sms * (per > 0 ? per : 1);
    return launch_pdl(Kernel, dim3((unsigned)(want < most ? want : most)), dim3(threads), 0, s, p.chained, p);
}

template <typename XT, typename RT>
cudaError_t pick(const NormParams &p, cudaStream_t s) {
    if (p.wide) {
        const int nvec = p.cols / 8;
        // up to 1024 columns a warp holds the row (no barrier); above, a CTA of up to 512 threads
        // with one or two units each, or of up to 1024 with four
        if (nvec <= 32) return go<k_norm_wide<XT, RT, 1, true>>(p, 256, 8, s);
        if (nvec <= 64) return go<k_norm_wide<XT, RT, 2, true>>(p, 256, 8, s);
        if (nvec <= 128) return go<k_norm_wide<XT, RT, 4, true>>(p, 256, 8, s);
        if (nvec <= 512) return go<k_norm_wide<XT, RT, 1, false>>(p, (nvec + 31) / 32 * 32, 1, s);
        if (nvec <= 1024) return go<k_norm_wide<XT, RT, 2, false>>(p, ((nvec + 1) / 2 + 31) / 32 * 32, 1, s);
        return go<k_norm_wide<XT, RT, 4, false>>(p, ((nvec + 3) / 4 + 31) / 32 * 32, 1, s);
    }
    if (p.cols <= 8192) return go<k_norm_narrow<XT, RT, 8>>(p, ((p.cols + 7) / 8 + 31) / 32 * 32, 1, s);
    return go<k_norm_narrow<XT, RT, 32>>(p, ((p.cols + 31) / 32 + 31) / 32 * 32, 1, s);
}

}  // namespace

cudaError_t launch_rms_norm(const NormParams &p, cudaStream_t s) {
    if (p.rows == 0) return cudaSuccess;
    if (!p.res) return p.x_bf16 ? pick<__nv_bfloat16, None>(p, s) : pick<float, None>(p, s);
    if (p.res_bf16) return p.x_bf16 ? pick<__nv_bfloat16, __nv_bfloat16>(p, s) : pick<float, __nv_bfloat16>(p, s);
    return p.x_bf16 ? pick<__nv_bfloat16, float>(p, s) : pick<float, float>(p, s);
}

}  // namespace hisa
