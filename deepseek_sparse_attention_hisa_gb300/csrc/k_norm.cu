// Residual addition, root-mean-square norm and output (f32, bf16, or e4m3 with scales) in one
// pass: every input element is read once and every output element written once.
//
//   h = round(x + residual);  y = h * w * rsqrt(mean(h^2) + eps);  out = round(y)  or
//   scale_g = max(max_g |y|, 1e-10) / 448 (up to a power of two),  out = e4m3(y / scale_g)
//
// Bound by memory: about 6 operations per element against 4 to 16 bytes. A team of threads
// holds a whole row in registers (a warp for rows of at most 1024 columns, else a CTA), so the
// sum of squares, the scales and the output need no second read. Teams walk the rows with a
// grid stride, and the next rows are on their way while a team reduces the current one, so the
// barrier of the reduction does not leave the memory system idle. Sums are f32: each thread's
// own columns in order, then a fixed tree over lanes and warps, so a row's result does not
// depend on the other rows or on how many there are. Which columns a thread owns follows the
// alignment of the row's start where that differs from row to row (cut units, below): the same
// row at another remainder modulo 8 elements, or taken by another kernel for its strides, is
// summed in another order.
//
// Measured: 16384 x 7168 bf16 with a bf16 residual to e4m3 by 128: 121 us, 6.8 TB/s, what a plain
// copy reaches; without a residual 82 us, bound by its instructions (about 20 per element); 304 x
// 7168: 4 to 5 us, one call, launch and one round trip to memory; 1001 x 5003 f32: 9.2 us, of which 5.9 are
// its bytes (two to three rows per CTA, one after another, do not hide the latency); 16384 x 5003
// bf16 60 us, 5.5 TB/s.
#include <cuda_fp8.h>

#include <atomic>

#include "ops_internal.cuh"
#include "tc_ptx.cuh"

namespace hisa {
namespace {

constexpr int kMaxCols = 32768;        // what the entry point accepts
constexpr int kMaxSmem = 220 * 1024;   // dynamic shared memory of a CTA (beside up to 5 KB declared)

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
// Unit v of a row that starts at `row`, in global memory or (SM) staged in shared memory.
template <bool SM>
__device__ __forceinline__ void store8(uint8_t *row, int v, bool bf16, const float (&f)[8]) {
    if (bf16) {
        reinterpret_cast<uint4 *>(row)[v] = pack_bf16(f);
    } else if (SM) {
        reinterpret_cast<float4 *>(row)[2 * v] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(row)[2 * v + 1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        store_sector(reinterpret_cast<float *>(row) + 8 * v, f);
    }
}

// Elements [lo, hi) of unit v.
template <typename T>
__device__ __forceinline__ void store_part(uint8_t *row, int v, int lo, int hi, const float (&f)[8]) {
    T *at = reinterpret_cast<T *>(row) + 8 * v;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if (e < lo || e >= hi) continue;
        if constexpr (sizeof(T) == 4) at[e] = f[e];
        else if constexpr (sizeof(T) == 2) at[e] = __float2bfloat16_rn(f[e]);
        else at[e] = __nv_cvt_float_to_fp8(f[e], __NV_SATFINITE, __NV_E4M3);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// The larger magnitude; NaN if either is one, so a group that holds a NaN gets a NaN scale.
__device__ __forceinline__ float max_mag(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}
__device__ __forceinline__ float max_mag(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint4 add_bf16(uint4 a, uint4 b) {
    auto add = [](uint32_t x, uint32_t y) {
        uint32_t r;
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
        return r;
    };
    return make_uint4(add(a.x, b.x), add(a.y, b.y), add(a.z, b.z), add(a.w, b.w));
}
// Over aligned groups of `lanes` lanes (a power of two).
__device__ __forceinline__ float lanes_max(float v, int lanes) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        if (lanes > o) v = max_mag(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Scale of a group of largest magnitude a. The floor keeps the quotient normal.
__device__ __forceinline__ float scale_of(float a, int pow2) {
    a = a < 1e-10f ? 1e-10f : a;
    // a / 448, correctly rounded: Markstein's step on the product with the rounded reciprocal
    // (an infinity or NaN stays one)
    const float s0 = a * (1.f / 448.f);
    float s = a < INFINITY ? fmaf(fmaf(-448.f, s0, a), 1.f / 448.f, s0) : a;
    if (pow2 && s < INFINITY) {
        const uint32_t u = __float_as_uint(s);
        s = __uint_as_float((u & 0x7f800000u) + ((u & 0x007fffffu) ? 0x00800000u : 0u));
    }
    return s;
}

// Joins one value per warp over the CTA: a partial each, one barrier, and the 32 slots (unused
// ones hold 0) read as vectors. Callers alternate between two arrays, so the next call's writes
// meet no late reader.
__device__ __forceinline__ float sum_of(const float *red) {
    float2 a = make_float2(0.f, 0.f), b = a;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h == 1 && blockDim.x <= 512) break;
#pragma unroll
        for (int w = 4 * h; w < 4 * h + 4; ++w) {
            const float4 u = reinterpret_cast<const float4 *>(red)[w];
            a = add2(a, make_float2(u.x, u.y));
            b = add2(b, make_float2(u.z, u.w));
        }
    }
    a = add2(a, b);
    return a.x + a.y;
}
__device__ __forceinline__ float max_of(const float *red) {
    float s = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h == 1 && blockDim.x <= 512) break;
#pragma unroll
        for (int w = 4 * h; w < 4 * h + 4; ++w) {
            const float4 u = reinterpret_cast<const float4 *>(red)[w];
            s = max_mag(max_mag(s, u.x, u.y), u.z, u.w);
        }
    }
    return s;
}
__device__ __forceinline__ float block_sum(float v, float *red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return sum_of(red);
}
__device__ __forceinline__ void block_sum_max(float &v, float &top, float *red, float *redm) {
    v = warp_sum(v);
    top = lanes_max(top, 32);
    if ((threadIdx.x & 31) == 0) {
        red[threadIdx.x >> 5] = v;
        redm[threadIdx.x >> 5] = top;
    }
    __syncthreads();
    v = sum_of(red);
    top = max_of(redm);
}
__device__ __forceinline__ float block_max(float v, float *red) {
    v = lanes_max(v, 32);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return max_of(red);
}

// What both kernels of 8-column units do with a row. With t = h w, f = 1 / sqrt(mean(h^2) + eps) > 0
// and y = t f, a group's largest |y| is f times its largest |t| (rounding is monotone), so the
// scales need no pass after the reduction.
// SM: through shared memory; RAG: the row's first and last unit may be cut.
template <typename RT, int VPT, bool SM, bool RAG>
struct Row {
    float h[VPT][8];                                  // the row, then t
    float top[VPT];                                   // largest |t| of the unit's group
    float2 ss2 = {0.f, 0.f};

    __device__ __forceinline__ float ss() const { return ss2.x + ss2.y; }

    // Unit i: h = x (+ residual, rounded as stored, and put to rrow), its squares, t = h w. Its columns
    // [lo, n) are there.
    template <typename XT>
    __device__ __forceinline__ void take(int i, int v, int lo, int n, uint8_t *rrow, const Raw8<XT> &x, const Raw8<RT> &r,
                                         const float (&w)[8]) {
        const bool cut = RAG && (lo > 0 || n < 8);
        if (n <= 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = 0.f;
            return;
        }
        if constexpr (std::is_same<XT, __nv_bfloat16>::value && std::is_same<RT, __nv_bfloat16>::value) {
            // the sum in bf16 is the f32 sum rounded: one that f32 cannot hold is no tie of bf16
            Raw8<__nv_bfloat16> sum;
            sum.v[0] = add_bf16(x.v[0], r.v[0]);
            unpack(sum, h[i]);
            if (rrow && cut) store_part<RT>(rrow, v, lo, n, h[i]);
            else if (rrow) reinterpret_cast<uint4 *>(rrow)[v] = sum.v[0];
        } else {
            unpack(x, h[i]);
            if constexpr (!std::is_same<RT, None>::value) {
                float q[8];
                unpack(r, q);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] += q[e];
                if constexpr (std::is_same<RT, __nv_bfloat16>::value) {
                    Raw8<__nv_bfloat16> back;
                    back.v[0] = pack_bf16(h[i]);
                    unpack(back, h[i]);                // the norm is over the sum as stored
                }
                if (rrow && cut) store_part<RT>(rrow, v, lo, n, h[i]);
                else if (rrow) store8<SM>(rrow, v, std::is_same<RT, __nv_bfloat16>::value, h[i]);
            }
        }
        if (cut || (SM && n < 8)) {                    // the blocks that hold the row's ends hold more
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = e >= lo && e < n ? h[i][e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            float2 u = make_float2(h[i][e], h[i][e + 1]);
            ss2 = fma2(u, u, ss2);
            u = mul2(u, make_float2(w[e], w[e + 1]));
            h[i][e] = u.x;
            h[i][e + 1] = u.y;
        }
    }
    // Largest |t| per unit, joined over a group's lanes (or, for one scale per row, this thread's units).
    __device__ __forceinline__ void tops(const NormParams &p) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const float a = max_mag(h[i][0], h[i][1], h[i][2]), b = max_mag(h[i][3], h[i][4], h[i][5]);
            top[i] = max_mag(max_mag(a, h[i][6], h[i][7]), b);
        }
        if (p.group) {
            const int lanes = p.group >> 3;
#pragma unroll
            for (int i = 0; i < VPT; ++i) top[i] = lanes_max(top[i], lanes);
        } else {
#pragma unroll
            for (int i = 1; i < VPT; ++i) top[0] = max_mag(top[0], top[i]);
        }
    }
    __device__ __forceinline__ void same_top(float v) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) top[i] = v;
    }
    __device__ __forceinline__ void times(int i, float f) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 u = mul2(make_float2(h[i][e], h[i][e + 1]), make_float2(f, f));
            h[i][e] = u.x;
            h[i][e + 1] = u.y;
        }
    }
    __device__ __forceinline__ void put(const NormParams &p, int i, int v, int lo, int n, float *scales, uint8_t *orow, float f) {
        const bool cut = RAG && (lo > 0 || n < 8);
        if (p.out_dtype != HISA_E4M3) {
            times(i, f);
            if (cut) {
                if (p.out_dtype == HISA_BF16) store_part<__nv_bfloat16>(orow, v, lo, n, h[i]);
                else store_part<float>(orow, v, lo, n, h[i]);
                return;
            }
            store8<SM>(orow, v, p.out_dtype == HISA_BF16, h[i]);
            return;
        }
        const float s = scale_of(top[i] * f, p.pow2);
        const float q = __fdividef(f, s);              // t q is within a few f32 steps of y / s
        const int g = v >> p.unit_shift;               // the unit's group (0 for one scale per row)
        if (v == g << p.unit_shift) scales[g] = s;
        times(i, q);
        if (cut) {
            store_part<uint8_t>(orow, v, lo, n, h[i]);
            return;
        }
        uint32_t c[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(h[i][4 * k], h[i][4 * k + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(h[i][4 * k + 2], h[i][4 * k + 3]), __NV_SATFINITE, __NV_E4M3);
            c[k] = lo | (hi << 16);
        }
        reinterpret_cast<uint2 *>(orow)[v] = make_uint2(c[0], c[1]);
    }
};

__device__ __forceinline__ int out_bytes(const NormParams &p) {
    return p.out_dtype == HISA_F32 ? 4 : (p.out_dtype == HISA_BF16 ? 2 : 1);
}
// Where unit 0 of a row lies, s elements before the row.
__device__ __forceinline__ uint8_t *out_row(const NormParams &p, int64_t row, int s = 0) {
    return static_cast<uint8_t *>(p.out) + (row * p.ld_out - s) * out_bytes(p);
}
template <typename RT>
__device__ __forceinline__ uint8_t *res_row(const NormParams &p, int64_t row, int s = 0) {
    if constexpr (std::is_same<RT, None>::value) return nullptr;
    else return p.res_out ? reinterpret_cast<uint8_t *>(static_cast<RT *>(p.res_out) + row * p.ld_res - s) : nullptr;
}

__device__ __forceinline__ void load_w(const float *base, int v, int nvec, float (&w)[8]) {
    const float4 *wp = reinterpret_cast<const float4 *>(base + (int64_t)(v < nvec ? v : 0) * 8);
    const float4 a = __ldg(wp), b = __ldg(wp + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// Rows that do not start at a multiple of 8 elements, but at the same remainder s in every array
// (contiguous arrays of any width): the units are the aligned ones, unit v columns 8 v - s .. + 7,
// the first and the last cut. A team's rows lie a multiple of 8 rows apart, so s is the team's
// constant and the weights are shifted once. (The shift of every row through shared memory, which
// k_norm_ragged makes, takes 12.4 instead of 9.2 us for 1001 x 5003 f32.)
__device__ __forceinline__ int shift_of(const NormParams &p, int64_t row) { return (int)((p.phase + row * p.ld_x) & 7); }
__device__ __forceinline__ void load_w_cut(const NormParams &p, int v, int s, float (&w)[8]) {
    float a[16];                                       // columns 8 v - 8 .. 8 v + 7
    const bool whole = (reinterpret_cast<uintptr_t>(p.w) & 15) == 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int c = 8 * v - 8 + 4 * j;
        if (whole && c >= 0 && c + 4 <= p.cols) {
            const float4 u = __ldg(reinterpret_cast<const float4 *>(p.w + c));
            a[4 * j] = u.x; a[4 * j + 1] = u.y; a[4 * j + 2] = u.z; a[4 * j + 3] = u.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[4 * j + e] = c + e >= 0 && c + e < p.cols ? __ldg(p.w + c + e) : 0.f;
        }
    }
    const int d = 8 - s;                               // 1 .. 8
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = d & 8 ? a[i + 8] : a[i];
#pragma unroll
    for (int i = 0; i < 11; ++i) a[i] = d & 4 ? a[i + 4] : a[i];
#pragma unroll
    for (int i = 0; i < 9; ++i) a[i] = d & 2 ? a[i + 2] : a[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = d & 1 ? a[i + 1] : a[i];
}
// The pieces of a cut unit that hold one of its columns [lo, n).
template <typename T>
__device__ __forceinline__ void load_raw_cut(Raw8<T> &r, const uint8_t *row, int v, int lo, int n) {
    if constexpr (!std::is_same<T, None>::value) {
        constexpr int kP = sizeof(T) / 2, kE = 8 / kP; // pieces per unit, elements per piece
        const uint4 *p = reinterpret_cast<const uint4 *>(row) + v * kP;
#pragma unroll
        for (int i = 0; i < kP; ++i)
            if (kE * i < n && kE * i + kE > lo) r.v[i] = __ldcs(p + i);
    }
}

// Rows of at most 1024 columns: a warp per row, the next row's loads in flight in registers.
template <typename XT, typename RT, int VPT, bool RAG>
__global__ void __launch_bounds__(256, VPT == 1 ? 4 : (VPT == 2 ? 3 : 2)) k_norm_warp(NormParams p) {
    const int t = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 5);       // a multiple of 8
    int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int s = RAG ? shift_of(p, row) : 0, nvec = (p.cols + s + 7) >> 3;
    auto lo = [&](int v) { return RAG && v == 0 ? s : 0; };
    auto hi = [&](int v) { const int n = p.cols + s - 8 * v; return v >= nvec ? 0 : RAG && n < 8 ? n : 8; };
    const float inv = 1.f / (float)p.cols;
    float w[VPT][8];
    if (!p.chained) grid_dep_wait();
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (RAG) load_w_cut(p, i * 32 + t, s, w[i]);
        else load_w(p.w, i * 32 + t, nvec, w[i]);
    }
    if (p.chained) grid_dep_wait();
    grid_dep_trigger();
    Raw8<XT> x[VPT];
    Raw8<RT> r[VPT];
    auto fetch = [&](int64_t at) {
        if (at >= p.rows) return;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * 32 + t;
            if constexpr (RAG) {
                load_raw_cut<XT>(x[i], reinterpret_cast<const uint8_t *>(static_cast<const XT *>(p.x) + at * p.ld_x - s), v, lo(v), hi(v));
                if constexpr (!std::is_same<RT, None>::value)
                    load_raw_cut<RT>(r[i], reinterpret_cast<const uint8_t *>(static_cast<const RT *>(p.res) + at * p.ld_res - s), v, lo(v), hi(v));
            } else if (v < nvec) {
                load_raw(x[i], p.x, at * p.ld_x + (int64_t)v * 8);
                load_raw(r[i], p.res, at * p.ld_res + (int64_t)v * 8);
            }
        }
    };
    fetch(row);
    for (; row < p.rows; row += step) {
        Row<RT, VPT, false, RAG> m;
        uint8_t *rrow = res_row<RT>(p, row, s), *orow = out_row(p, row, s);
#pragma unroll
        for (int i = 0; i < VPT; ++i) m.take(i, i * 32 + t, lo(i * 32 + t), hi(i * 32 + t), rrow, x[i], r[i], w[i]);
        fetch(row + step);
        if (p.out_dtype == HISA_E4M3) {
            m.tops(p);
            if (!p.group) m.same_top(lanes_max(m.top[0], 32));
        }
        const float f = rsqrtf(warp_sum(m.ss()) * inv + p.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (i * 32 + t < nvec) m.put(p, i, i * 32 + t, lo(i * 32 + t), hi(i * 32 + t), p.scales + row * p.groups, orow, f);
    }
}

// Longer rows: a CTA per row. Rows to come are copied to shared memory asynchronously, STAGES - 1
// of them in flight; a warp copies exactly the units that it reads itself, so it waits for its
// own copies and needs no barrier for them.
template <typename XT, typename RT, int VPT, int STAGES, bool RAG>
__global__ void __launch_bounds__(1024, 1) k_norm_cta(NormParams p) {
    constexpr int kX = sizeof(XT) / 2, kR = std::is_same<RT, None>::value ? 0 : sizeof(RT) / 2;   // 16-byte pieces per unit
    extern __shared__ __align__(16) uint4 ring[];     // [stage]: the row of x, the row of residual
    __shared__ __align__(16) float red[2][32], redm[2][32];
    const int T = blockDim.x, t = threadIdx.x;
    const int s = RAG ? shift_of(p, blockIdx.x) : 0, nvec = (p.cols + s + 7) >> 3;
    const int held = RAG ? (p.cols + 14) >> 3 : nvec; // units of a stage
    auto lo = [&](int v) { return RAG && v == 0 ? s : 0; };
    auto hi = [&](int v) { const int n = p.cols + s - 8 * v; return v >= nvec ? 0 : RAG && n < 8 ? n : 8; };
    const float inv = 1.f / (float)p.cols;
    if (t < 32) red[0][t] = red[1][t] = redm[0][t] = redm[1][t] = 0.f;
    __syncthreads();
    constexpr bool kHoldW = VPT <= 2;                 // this thread's weights stay in registers
    float w[kHoldW ? VPT : 1][8];
    auto weights = [&](int v, float (&to)[8]) {
        if constexpr (RAG) load_w_cut(p, v, s, to);
        else load_w(p.w, v, nvec, to);
    };
    if (kHoldW && p.chained) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) weights(i * T + t, w[kHoldW ? i : 0]);
    }
    grid_dep_wait();
    grid_dep_trigger();
    // Everything that a row needs of its number moves on by a constant where registers allow: rows
    // are short enough for the multiplications to count.
    constexpr bool kStep = VPT <= 2;
    const int q0x = (t & ~31) * kX + (t & 31), q0r = (t & ~31) * kR + (t & 31);      // this thread's first pieces
    const uint8_t *nx = reinterpret_cast<const uint8_t *>(static_cast<const XT *>(p.x) + blockIdx.x * p.ld_x - s) + 16 * q0x;
    const int64_t step_x = gridDim.x * p.ld_x * (int64_t)sizeof(XT);
    const uint8_t *nr = nullptr;
    int64_t step_r = 0;
    if constexpr (kR > 0) {
        nr = reinterpret_cast<const uint8_t *>(static_cast<const RT *>(p.res) + blockIdx.x * p.ld_res - s) + 16 * q0r;
        step_r = gridDim.x * p.ld_res * (int64_t)sizeof(RT);
    }
    const uint32_t stage_b = (uint32_t)(kX + kR) * held * 16, ring0 = tc::smem_u32(ring);
    int64_t next = blockIdx.x;                        // the row to copy next
    // the pieces that hold an element of the row
    auto piece = [&](int q, int per) { return (!RAG || (q + 1) * 8 > s * per) && q * 8 < (RAG ? p.cols + s : nvec * 8) * per; };
    auto copy = [&](int stage) {
        if (next < p.rows) {
            if constexpr (!kStep) {
                nx = reinterpret_cast<const uint8_t *>(static_cast<const XT *>(p.x) + next * p.ld_x - s) + 16 * q0x;
                if constexpr (kR > 0) nr = reinterpret_cast<const uint8_t *>(static_cast<const RT *>(p.res) + next * p.ld_res - s) + 16 * q0r;
            }
            const uint32_t dst = ring0 + stage * stage_b;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
#pragma unroll
                for (int k = 0; k < kX; ++k) {        // the warp's units i T + t & ~31 .. + 31
                    const int q = i * T * kX + 32 * k;
                    if (piece(q0x + q, kX)) tc::cp_async16(dst + 16 * (q0x + q), nx + 16 * q);
                }
#pragma unroll
                for (int k = 0; k < kR; ++k) {
                    const int q = i * T * kR + 32 * k;
                    if (piece(q0r + q, kR)) tc::cp_async16(dst + 16 * (kX * held + q0r + q), nr + 16 * q);
                }
            }
            if constexpr (kStep) {
                nx += step_x;
                nr += step_r;
            }
        }
        next += gridDim.x;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) copy(k);
    if (kHoldW && !p.chained) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) weights(i * T + t, w[kHoldW ? i : 0]);
    }
    uint8_t *orow = out_row(p, blockIdx.x, s), *rrow = res_row<RT>(p, blockIdx.x, s);
    const int64_t step_o = gridDim.x * p.ld_out * out_bytes(p);
    float *srow = p.scales + (int64_t)blockIdx.x * p.groups;
    int stage = 0, par = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, par ^= 1) {
        if (STAGES == 1) copy(0);
        asm volatile("cp.async.wait_group %0;" :: "n"(STAGES > 1 ? STAGES - 2 : 0) : "memory");
        __syncwarp();
        const uint4 *src = ring + stage * (kX + kR) * held;
        if constexpr (!kStep) {
            orow = out_row(p, row, s);
            rrow = res_row<RT>(p, row, s);
            srow = p.scales + row * p.groups;
        }
        Row<RT, VPT, false, RAG> m;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * T + t;
            Raw8<XT> x;
            Raw8<RT> r;
            if (v < nvec) {
#pragma unroll
                for (int k = 0; k < kX; ++k) x.v[k] = src[v * kX + k];
                if constexpr (kR > 0) {
#pragma unroll
                    for (int k = 0; k < kR; ++k) r.v[k] = src[kX * held + v * kR + k];
                }
            }
            if constexpr (!kHoldW) weights(v, w[0]);
            m.take(i, v, lo(v), hi(v), rrow, x, r, w[kHoldW ? i : 0]);
        }
        __syncwarp();
        if (STAGES > 1) {
            // into the stage read by the row before
            copy(stage == 0 ? STAGES - 1 : stage - 1);
            stage = stage + 1 == STAGES ? 0 : stage + 1;
        }
        if (p.out_dtype == HISA_E4M3) m.tops(p);
        float sum = m.ss();
        if (p.out_dtype == HISA_E4M3 && !p.group) {
            float top = m.top[0];
            block_sum_max(sum, top, red[par], redm[par]);
            m.same_top(top);
        } else {
            sum = block_sum(sum, red[par]);
        }
        const float f = rsqrtf(sum * inv + p.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (i * T + t < nvec) m.put(p, i, i * T + t, lo(i * T + t), hi(i * T + t), srow, orow, f);
        if constexpr (kStep) {
            orow += step_o;
            if (rrow) rrow += step_r;
            srow += (int64_t)gridDim.x * p.groups;
        }
    }
}

template <typename T>
__device__ __forceinline__ float load1(const void *base, int64_t at) {
    if constexpr (std::is_same<T, None>::value) return 0.f;
    else return to_f32(__ldcs(static_cast<const T *>(base) + at));
}
template <typename T>
constexpr size_t kElem = std::is_same<T, None>::value ? 0 : sizeof(T);
// Bytes of a staged row: the blocks that cover it, and those that shifted reads and the last unit
// may touch past them.
__host__ __device__ constexpr size_t stage_bytes(int cols, size_t es) {
    return es ? ((size_t)cols * es + 15 + 15) / 16 * 16 + 64 : 0;
}

// The 16-byte blocks that hold row `row` of an array, whole: up to 15 bytes before and after the
// row come along (they share a block with an element of it).
template <typename T>
__device__ __forceinline__ void copy_row(uint8_t *dst, const void *base, int64_t at, int cols) {
    if constexpr (!std::is_same<T, None>::value) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(static_cast<const T *>(base) + at), lo = a & ~(uintptr_t)15;
        const int pieces = (int)((a - lo + (size_t)cols * sizeof(T) + 15) / 16);
        for (int i = threadIdx.x; i < pieces; i += blockDim.x)
            tc::cp_async16(tc::smem_u32(dst + 16 * i), reinterpret_cast<const void *>(lo + 16 * i));
    }
}
template <typename T>
__device__ __forceinline__ int row_offset(const void *base, int64_t at) {
    if constexpr (std::is_same<T, None>::value) return 0;
    else return (int)(reinterpret_cast<uintptr_t>(static_cast<const T *>(base) + at) & 15);
}
// 16 bytes from any byte offset of a 16-byte aligned shared-memory buffer: two aligned reads and
// a shift that is the same for a whole row.
__device__ __forceinline__ uint4 read_shifted(const uint8_t *buf, int off) {
    const uint4 a = *reinterpret_cast<const uint4 *>(buf + (off & ~15)), b = *reinterpret_cast<const uint4 *>(buf + (off & ~15) + 16);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = (off & 8) ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = (off & 4) ? w[i + 1] : w[i];
    const int s = (off & 3) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s), __funnelshift_r(w[2], w[3], s),
                      __funnelshift_r(w[3], w[4], s));
}
// Writes n bytes (of `es`-byte elements) staged at a buffer's start: whole 16-byte blocks of the
// destination at once, the row's ragged ends by elements.
__device__ __forceinline__ void write_row(uint8_t *dst, const uint8_t *staged, int n, int es) {
    const int a = (int)(reinterpret_cast<uintptr_t>(dst) & 15);
    uint8_t *lo = dst - a;
    for (int i = threadIdx.x; 16 * i < a + n; i += blockDim.x) {
        if (16 * i >= a && 16 * i + 16 <= a + n) {
            *reinterpret_cast<uint4 *>(lo + 16 * i) = read_shifted(staged, 16 * i - a);
            continue;
        }
        const int b0 = 16 * i > a ? 16 * i : a, b1 = 16 * i + 16 < a + n ? 16 * i + 16 : a + n;
        for (int b = b0; b < b1; b += es) {
            if (es == 4) *reinterpret_cast<uint32_t *>(lo + b) = *reinterpret_cast<const uint32_t *>(staged + b - a);
            else if (es == 2) *reinterpret_cast<uint16_t *>(lo + b) = *reinterpret_cast<const uint16_t *>(staged + b - a);
            else lo[b] = staged[b - a];
        }
    }
}

// Rows that start at different remainders in different arrays, or with groups that the aligned units
// would straddle: the same units of 8 columns, a CTA per row. Rows come in and go out through shared memory in the aligned
// 16-byte blocks that cover them, and the shift between blocks and units is made in registers. One
// row is staged and the next one asked for as soon as it has been read; two (which cost CTAs per SM)
// were no faster: 16384 x 5003 bf16 with residual 136 against 135 us, 4096 x 6001 f32 with f32 residual
// 109 against 83, 8192 x 12001 bf16 116 against 120.
template <typename XT, typename RT, int VPT>
__global__ void __launch_bounds__(1024, 1) k_norm_ragged(NormParams p) {
    extern __shared__ __align__(16) uint4 ring[];     // x, residual, out, residual_out
    __shared__ __align__(16) float red[2][32], redm[2][32];
    const int T = blockDim.x, t = threadIdx.x, nvec = (p.cols + 7) >> 3;
    const float inv = 1.f / (float)p.cols;
    const int es = out_bytes(p);
    const size_t xb = stage_bytes(p.cols, kElem<XT>), rb = stage_bytes(p.cols, kElem<RT>);
    uint8_t *in = reinterpret_cast<uint8_t *>(ring), *obuf = in + xb + rb;
    uint8_t *rbuf = obuf + stage_bytes(p.cols, es);
    if (t < 32) red[0][t] = red[1][t] = redm[0][t] = redm[1][t] = 0.f;
    constexpr bool kHoldW = VPT <= 2;
    float w[kHoldW ? VPT : 1][8];
    const bool whole_w = (reinterpret_cast<uintptr_t>(p.w) & 15) == 0;
    auto load_some = [&](int v, float (&to)[8]) {
        if (whole_w && v * 8 + 8 <= p.cols) {          // single elements, 32 bytes apart, cost four times the wavefronts
            load_w(p.w, v, nvec, to);
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) to[e] = v * 8 + e < p.cols ? __ldg(p.w + v * 8 + e) : 0.f;
    };
    if (!p.chained) grid_dep_wait();
    if constexpr (kHoldW) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) load_some(i * T + t, w[i]);
    }
    __syncthreads();
    if (p.chained) grid_dep_wait();
    grid_dep_trigger();
    auto copy = [&](int64_t row) {
        if (row < p.rows) {
            copy_row<XT>(in, p.x, row * p.ld_x, p.cols);
            copy_row<RT>(in + xb, p.res, row * p.ld_res, p.cols);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    copy(blockIdx.x);
    int par = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, par ^= 1) {
        const int ax = row_offset<XT>(p.x, row * p.ld_x), ar = row_offset<RT>(p.res, row * p.ld_res);
        uint8_t *rrow = res_row<RT>(p, row), *orow = out_row(p, row);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();                               // every thread's blocks of this row have landed, and
                                                       // the row before has been written out
        Row<RT, VPT, true, false> m;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * T + t;
            Raw8<XT> x;
            Raw8<RT> r;
            if (v < nvec) {
#pragma unroll
                for (int k = 0; k < (int)kElem<XT> / 2; ++k) x.v[k] = read_shifted(in, ax + 8 * (int)kElem<XT> * v + 16 * k);
                if constexpr (kElem<RT> > 0) {
#pragma unroll
                    for (int k = 0; k < (int)kElem<RT> / 2; ++k)
                        r.v[k] = read_shifted(in + xb, ar + 8 * (int)kElem<RT> * v + 16 * k);
                }
            }
            if constexpr (!kHoldW) load_some(v, w[0]);
            m.take(i, v, 0, p.cols - 8 * v, rrow ? rbuf : nullptr, x, r, w[kHoldW ? i : 0]);
        }
        if (p.out_dtype == HISA_E4M3) m.tops(p);
        float sum = m.ss();
        if (p.out_dtype == HISA_E4M3 && !p.group) {
            float top = m.top[0];
            block_sum_max(sum, top, red[par], redm[par]);
            m.same_top(top);
        } else {
            sum = block_sum(sum, red[par]);
        }
        const float f = rsqrtf(sum * inv + p.eps);
        copy(row + gridDim.x);                         // every thread has read this row (the sum's barrier)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (i * T + t < nvec) m.put(p, i, i * T + t, 0, 8, p.scales + row * p.groups, obuf, f);
        __syncthreads();                               // the staged outputs are whole
        write_row(orow, obuf, p.cols * es, es);
        if (rrow) write_row(rrow, rbuf, p.cols * (int)kElem<RT>, (int)kElem<RT>);
    }
}

// Rows too long to be staged: one CTA per row, single elements, neighbouring threads on
// neighbouring columns, the row read again (from L2) instead of held.
template <typename XT, typename RT>
__global__ void __launch_bounds__(1024, 1) k_norm_long(NormParams p) {
    constexpr bool kRes = !std::is_same<RT, None>::value;
    __shared__ __align__(16) float red[2][32], redm[2][32];
    const int T = blockDim.x, t = threadIdx.x;
    const float inv = 1.f / (float)p.cols;
    if (t < 32) red[0][t] = red[1][t] = redm[0][t] = redm[1][t] = 0.f;
    __syncthreads();
    grid_dep_wait();
    grid_dep_trigger();
    int par = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, par ^= 1) {
        auto value = [&](int c) {
            float h = load1<XT>(p.x, row * p.ld_x + c);
            if constexpr (kRes) h += load1<RT>(p.res, row * p.ld_res + c);
            if constexpr (std::is_same<RT, __nv_bfloat16>::value) h = __bfloat162float(__float2bfloat16_rn(h));
            return h;
        };
        float ss = 0.f, top = 0.f;
        for (int c = t; c < p.cols; c += T) {
            const float h = value(c);
            ss += h * h;
            top = max_mag(top, h * __ldg(p.w + c));
        }
        const float f = rsqrtf(block_sum(ss, red[par]) * inv + p.eps);
        if (p.out_dtype == HISA_E4M3 && !p.group) top = block_max(top, redm[par]);
        for (int c0 = 0; c0 < p.cols; c0 += T) {
            const int c = c0 + t;
            const bool in = c < p.cols;
            const float h = in ? value(c) : 0.f;
            const float y = in ? h * __ldg(p.w + c) : 0.f;
            if constexpr (kRes) {
                if (in && p.res_out) {
                    if constexpr (sizeof(RT) == 2) static_cast<RT *>(p.res_out)[row * p.ld_res + c] = __float2bfloat16_rn(h);
                    else static_cast<RT *>(p.res_out)[row * p.ld_res + c] = h;
                }
            }
            const int64_t at = row * p.ld_out + c;
            if (p.out_dtype == HISA_F32) {
                if (in) static_cast<float *>(p.out)[at] = y * f;
            } else if (p.out_dtype == HISA_BF16) {
                if (in) static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(y * f);
            } else {
                // a group of up to 256 columns spans 1, 2, 4 or 8 warps of this step (T is a multiple of 256)
                float m = top;
                if (p.group) {
                    m = lanes_max(y, 32);
                    if ((t & 31) == 0) redm[par][t >> 5] = m;
                    __syncthreads();
                    const int w0 = (t >> 5) & ~((p.group >> 5) - 1);
                    for (int k = 0; k < (p.group >> 5); ++k) m = max_mag(m, redm[par][w0 + k]);
                    __syncthreads();
                }
                if (in) {
                    const float s = scale_of(m * f, p.pow2);
                    const int g = c >> (p.unit_shift + 3);
                    if (c == g << (p.unit_shift + 3)) p.scales[row * p.groups + g] = s;
                    static_cast<uint8_t *>(p.out)[at] = __nv_cvt_float_to_fp8(y * __fdividef(f, s), __NV_SATFINITE, __NV_E4M3);
                }
            }
        }
    }
}

// A team's rows are `apart` rows apart, or a multiple of that.
template <auto Kernel>
cudaError_t go(const NormParams &p, int threads, int64_t rows_per_cta, size_t smem, cudaStream_t s, int64_t apart = 1) {
    if (smem) {
        const cudaError_t e = smem_attr_once<Kernel>(kMaxSmem);
        if (e != cudaSuccess) return e;
    }
    // as many CTAs as the SMs hold at once; they walk the rows
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int64_t want = (p.rows + rows_per_cta - 1) / rows_per_cta;
    int64_t most = sms;
    if (want > sms) {
        // asked of the runtime (0.35 us of host time) once for a device and shape, the last of which
        // is kept: device, threads, smem and the answer in one word, so threads may race
        static std::atomic<uint64_t> last{0};
        int per = 0, dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t key = ((uint64_t)(dev + 1) << 48) | ((uint64_t)threads << 32) | ((uint64_t)smem << 8);
        const uint64_t was = last.load(std::memory_order_relaxed);
        if ((was & ~(uint64_t)255) == key) {
            per = (int)(was & 255);
        } else {
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, Kernel, threads, smem);
            if (e != cudaSuccess) return e;
            last.store(key | (uint64_t)per, std::memory_order_relaxed);
        }
        most = (int64_t)sms * (per > 0 ? per : 1);
        most = most > apart ? most / apart * apart : apart;
    } else if (want > 1) {
        most = want;
    }
    return launch_pdl(Kernel, dim3((unsigned)(want < most ? want : most)), dim3(threads), smem, s, 1, p);
}

// Units of 8 columns, aligned in memory.
template <typename XT, typename RT, bool RAG>
cudaError_t pick_units(const NormParams &p, int nvec, cudaStream_t s) {
    auto up = [](int n) { return (n + 31) / 32 * 32; };
    const size_t row = (size_t)nvec * 8 * (kElem<XT> + kElem<RT>);
    // up to 1024 columns a warp holds the row, with no barrier (16384 x 256 bf16 3.7 against 5.9 us by a
    // CTA per row, 512 6.0 against 6.7; at 1024 1001 rows 3.4 against 3.6, 16384 rows 12.7 against 12.5, to
    // 8 bits with a residual 22.0 against 20.0); above, a CTA of up to 512 threads with a unit each, or of
    // up to 1024 with two; with four only where two do not hold the row, or its bytes leave no room for
    // three of it (16384 x 7168 bf16 with residual to e4m3 by four 169 against 122 us, 8192 x 16384 bf16 95
    // against 81). Three stages are two rows in flight per
    // CTA. Where two CTAs of two units per thread share an SM, one row each in flight is enough and
    // keeps what DRAM serves at once closer together (16384 x 7168 bf16 with residual to e4m3: 122
    // against 142 us; 5003 f32 with f32 residual, where three stages leave room for one CTA, 199
    // against 238). Alone on its SM a CTA needs both (8192 x 16384 bf16: 81 against 89 us).
    if (nvec <= 32) return go<k_norm_warp<XT, RT, 1, RAG>>(p, 256, 8, 0, s);
    if (nvec <= 64) return go<k_norm_warp<XT, RT, 2, RAG>>(p, 256, 8, 0, s);
    if (nvec <= 128) return go<k_norm_warp<XT, RT, 4, RAG>>(p, 256, 8, 0, s);
    if (nvec <= 512) return go<k_norm_cta<XT, RT, 1, 3, RAG>>(p, up(nvec), 1, 3 * row, s, RAG ? 8 : 1);
    if (nvec <= 1024 && 4 * row <= kMaxSmem) return go<k_norm_cta<XT, RT, 2, 2, RAG>>(p, up((nvec + 1) / 2), 1, 2 * row, s, RAG ? 8 : 1);
    if (nvec <= 2048 && 3 * row <= kMaxSmem) return go<k_norm_cta<XT, RT, 2, 3, RAG>>(p, up((nvec + 1) / 2), 1, 3 * row, s, RAG ? 8 : 1);
    // (what no row of these types reaches is not built)
    constexpr size_t kUnit = 8 * (kElem<XT> + kElem<RT>);
    if constexpr (3 * 2049 * kUnit <= kMaxSmem) {
        if (3 * row <= kMaxSmem) return go<k_norm_cta<XT, RT, 4, 3, RAG>>(p, up((nvec + 3) / 4), 1, 3 * row, s, RAG ? 8 : 1);
    }
    if constexpr (3 * 4096 * kUnit > kMaxSmem)
        return go<k_norm_cta<XT, RT, 4, 1, RAG>>(p, up((nvec + 3) / 4), 1, row, s, RAG ? 8 : 1);
    return cudaErrorInvalidValue;
}

template <typename XT, typename RT>
cudaError_t pick(const NormParams &p, cudaStream_t s) {
    const int nvec = (p.cols + 7) / 8, cut = (p.cols + 14) / 8;
    const size_t unit = 8 * (kElem<XT> + kElem<RT>);
    auto up = [](int n) { return (n + 31) / 32 * 32; };
    if (p.wide && nvec * unit <= kMaxSmem) return pick_units<XT, RT, false>(p, nvec, s);
    if (p.phase >= 0 && cut <= 4096 && cut * unit <= kMaxSmem) return pick_units<XT, RT, true>(p, cut, s);
    const size_t in = stage_bytes(p.cols, kElem<XT>) + stage_bytes(p.cols, kElem<RT>);
    const size_t out = stage_bytes(p.cols, p.out_dtype == HISA_F32 ? 4 : (p.out_dtype == HISA_BF16 ? 2 : 1)) +
                       (p.res_out ? stage_bytes(p.cols, kElem<RT>) : 0);
    if (in + out <= kMaxSmem) {
        if (nvec <= 512) return go<k_norm_ragged<XT, RT, 1>>(p, up(nvec), 1, in + out, s);
        if (nvec <= 2048) return go<k_norm_ragged<XT, RT, 2>>(p, up((nvec + 1) / 2), 1, in + out, s);
        return go<k_norm_ragged<XT, RT, 4>>(p, up((nvec + 3) / 4), 1, in + out, s);
    }
    // (f32 output and the kept sum at most; the bf16 rows without a residual all fit.) Staged rows are
    // taken wherever they fit: 4096 x 20011 bf16 100 us so, 312 read twice; 4096 x 13001 f32 with f32
    // residual 189 against 372. 4096 x 32768 f32 with f32 residual, which do not: 904 us.
    if constexpr (kMaxCols * (kElem<XT> + 2 * kElem<RT> + 4) > kMaxSmem) return go<k_norm_long<XT, RT>>(p, 1024, 1, 0, s);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rms_norm(const NormParams &p, cudaStream_t s) {
    if (p.rows == 0) return cudaSuccess;
    if (!p.res) return p.x_bf16 ? pick<__nv_bfloat16, None>(p, s) : pick<float, None>(p, s);
    if (p.res_bf16) return p.x_bf16 ? pick<__nv_bfloat16, __nv_bfloat16>(p, s) : pick<float, __nv_bfloat16>(p, s);
    return p.x_bf16 ? pick<__nv_bfloat16, float>(p, s) : pick<float, float>(p, s);
}

}  // namespace hisa
