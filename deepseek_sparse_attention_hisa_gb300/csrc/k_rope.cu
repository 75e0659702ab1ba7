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
// CTA's rows, 64 bytes in flight (128 for f32 halves). While they are, the CTA computes the sines
// and cosines of the batch's few tokens into shared memory, once per token and pair and not once
// per head, on all its threads (each thread computing its own pairs held the half layout at a
// sixth of this rate). In place only the rotated dims move.
//
// Measured: 4096 tokens of 64 + 1 heads of 512, f32 to bf16: 124 us, 6.6 TB/s, 97 % of a plain
// copy's rate; 2047 tokens of 64 x 128 bf16, 64 dims rotated in the half layout: 15.5 us (9.9 are
// its bytes; the batches of a CTA, one after another, each expose a round trip to memory, the angles'
// latency and a barrier); the last 64 dims of 304 tokens of 64 + 1 heads in place: 4.7 to 5.2 us per
// call, which its launch bounds. Single elements, where a boundary is no multiple of 8: 4096 x 65 x 512
// bf16 with dims 447 to 510 rotated 470 us (89 with 448 to 511), 304 tokens in place 6.8 us.
#include "ops_internal.cuh"

namespace hisa {
namespace {

// A unit as loaded: 8 dims in 16-byte pieces, or one.
template <typename T, int N> struct Unit { uint4 v[sizeof(T) / 2]; };
template <typename T> struct Unit<T, 1> { T v; };

template <typename T, int N>
__device__ __forceinline__ void load_unit(const void *base, int64_t at, Unit<T, N> &u) {
    const T *p = static_cast<const T *>(base) + at;
    if constexpr (N == 1) {
        u.v = *p;
    } else {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) u.v[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
}
template <typename T, int N>
__device__ __forceinline__ void to_floats(const Unit<T, N> &u, float (&f)[N]) {
    if constexpr (N == 1) {
        f[0] = to_f32(u.v);
    } else if constexpr (sizeof(T) == 2) {
        const uint32_t w[4] = {u.v[0].x, u.v[0].y, u.v[0].z, u.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[4 * i] = __uint_as_float(u.v[i].x); f[4 * i + 1] = __uint_as_float(u.v[i].y);
            f[4 * i + 2] = __uint_as_float(u.v[i].z); f[4 * i + 3] = __uint_as_float(u.v[i].w);
        }
    }
}
template <typename T, int N>
__device__ __forceinline__ void store_unit(void *base, int64_t at, const float (&f)[N]) {
    T *p = static_cast<T *>(base) + at;
    if constexpr (N == 1) {
        if constexpr (sizeof(T) == 2) *p = __float2bfloat16_rn(f[0]);
        else *p = f[0];
    } else if constexpr (sizeof(T) == 2) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        store_sector(p, f);
    }
}

// N dims per unit (8, or 1 where a boundary is not a multiple of 8). A rotated unit is two
// blocks of N dims, `lo` and `hi`: for the half layout the pairs (lo + e, hi + e); interleaved,
// for N = 8 one block holding 4 pairs (hi unused), for N = 1 the pair (lo, hi).
// Rows per thread in flight: four of 16 bytes, two of more. More in flight spreads what DRAM serves
// at once (4096 x 65 x 512 f32 to bf16: 125 us with two, 132 with four) and costs the half layout
// its registers (2047 x 64 x 128 bf16, all dims: 13.1 us with two, 13.9 with four); fewer leave DRAM
// idle (interleaved bf16, 4096 x 65 x 512: 90 us with four, 94 with three, 104 with two).
template <typename S, int N, bool HALF>
constexpr int kUnroll = N == 8 && (HALF || sizeof(S) == 4) ? 2 : 4;

template <typename S, typename D, int N, bool HALF>
__global__ void __launch_bounds__(N == 8 ? 256 : 1024, N == 8 ? 4 : 1) k_rope(RopeParams p) {
    constexpr int kU = kUnroll<S, N, HALF>;
    constexpr bool kTwo = HALF || N == 1;                 // a rotated unit is two blocks
    constexpr int kPairs = kTwo ? N : N / 2;
    const int n_rot = p.dims / (kTwo ? 2 * N : N);
    const int n = n_rot + (p.inplace ? 0 : (p.D - p.dims) / N);
    const int sub = threadIdx.x / n, unit = threadIdx.x - sub * n, per = p.per;
    const int64_t r0 = blockIdx.x * p.rows_per_cta;
    const int mine = (int)(p.rows - r0 < p.rows_per_cta ? p.rows - r0 : p.rows_per_cta);
    const bool rot = unit < n_rot;
    const int pairs = p.dims / 2;
    int lo, hi = 0;
    if (rot) {
        if (HALF) { lo = p.first + unit * N; hi = lo + p.dims / 2; }
        else if (N == 1) { lo = p.first + 2 * unit; hi = lo + 1; }
        else lo = p.first + unit * N;
    } else {
        lo = (unit - n_rot) * N;                          // copied units: the dims before, then after, the rotated
        if (lo >= p.first) lo += p.dims;
    }
    // [token of the batch][pair]: mscale (cos, sin). For a unit of 8 dims two pairs' cosines, then
    // their sines, and the units' first two pairs come first, then their next two: neighbouring
    // lanes read neighbouring 16 bytes (unit by unit they would meet in a quarter of the banks).
    extern __shared__ __align__(16) float turn[];
    grid_dep_wait();
    grid_dep_trigger();
    // the first row's token and head (grid * heads_all fits 32 bits), and this thread's from there on
    const uint32_t past = blockIdx.x * (uint32_t)p.cta_head;
    int64_t tok0 = (int64_t)blockIdx.x * p.cta_tok + past / (uint32_t)p.heads_all;
    int head0 = (int)(past % (uint32_t)p.heads_all);
    const int sub_tok = sub / p.heads_all, sub_head = sub - sub_tok * p.heads_all;
    for (int done = 0; done < mine; done += p.batch) {
        const int here = mine - done < p.batch ? mine - done : p.batch;
        const int left = here - sub;                      // rows k per < left are there
        const S *x0 = static_cast<const S *>(p.x) + tok0 * p.x_token, *x20 = static_cast<const S *>(p.x2) + tok0 * p.x2_token;
        Unit<S, N> a[kU], b[kTwo ? kU : 1];
        int tok[kU], head[kU];                            // token (from tok0 on) and head of row k
        head[0] = head0 + sub_head;
        tok[0] = sub_tok;
        if (head[0] >= p.heads_all) {
            head[0] -= p.heads_all;
            ++tok[0];
        }
#pragma unroll
        for (int k = 0; k < kU; ++k) {
            if (k > 0) {
                tok[k] = tok[k - 1] + p.step_tok;
                head[k] = head[k - 1] + p.step_head;
                if (head[k] >= p.heads_all) {
                    head[k] -= p.heads_all;
                    ++tok[k];
                }
            }
            if (k * per < left) {
                const S *src = head[k] < p.heads ? x0 + tok[k] * p.x_token + head[k] * p.x_head
                                                 : x20 + tok[k] * p.x2_token + (head[k] - p.heads) * p.x2_head;
                load_unit<S, N>(src, lo, a[k]);
                if constexpr (kTwo)
                    if (rot) load_unit<S, N>(src, hi, b[k]);
            }
        }
        const uint32_t angles = ((uint32_t)(head0 + here - 1) / (uint32_t)p.heads_all + 1) * pairs;
        for (uint32_t i = threadIdx.x; i < angles; i += blockDim.x) {
            const uint32_t tk = i / (uint32_t)pairs, pair = i - tk * pairs;
            const int64_t pos = p.pos[tok0 + tk];
            const int64_t turns = (int64_t)((uint64_t)pos * __ldg(p.table + pair));           // modulo one turn
            float s, c;
            sincospif(2.f * (__ll2float_rn(turns) * 0x1p-64f), &s, &c);
            c *= p.mscale;
            s *= p.mscale * p.sin_sign;
            if constexpr (N == 1) {
                turn[2 * i] = c;
                turn[2 * i + 1] = s;
            } else {
                const uint32_t of = pair / kPairs, at = pair % kPairs;
                float *to = turn + 2 * tk * pairs + ((at >> 1) * n_rot + of) * 4 + (at & 1);
                to[0] = c;
                to[2] = s;
            }
        }
        __syncthreads();
        D *y0 = static_cast<D *>(p.y) + tok0 * p.y_token, *y20 = static_cast<D *>(p.y2) + tok0 * p.y2_token;
#pragma unroll
        for (int k = 0; k < kU; ++k) {
            if (k * per >= left) break;
            D *dst = head[k] < p.heads ? y0 + tok[k] * p.y_token + head[k] * p.y_head
                                       : y20 + tok[k] * p.y2_token + (head[k] - p.heads) * p.y2_head;
            float u[N];
            to_floats<S, N>(a[k], u);
            if (rot) {
                const float *cs = turn + 2 * tok[k] * pairs;
                if constexpr (N == 1) {
                    float v[1];
                    to_floats<S, N>(b[k], v);
                    const float x = u[0], y = v[0], c = cs[2 * unit], s = cs[2 * unit + 1];
                    u[0] = x * c - y * s;
                    v[0] = x * s + y * c;
                    store_unit<D, N>(dst, hi, v);
                } else {
                    float v[kTwo ? N : 1];
                    if constexpr (kTwo) to_floats<S, N>(b[k], v);
#pragma unroll
                    for (int e = 0; e < kPairs; e += 2) {     // two pairs at once
                        const float4 t4 = reinterpret_cast<const float4 *>(cs)[(e / 2) * n_rot + unit];
                        const float2 c = make_float2(t4.x, t4.y), s = make_float2(t4.z, t4.w), ns = make_float2(-t4.z, -t4.w);
                        float &x0r = u[kTwo ? e : 2 * e], &x1r = u[kTwo ? e + 1 : 2 * e + 2];
                        float &y0r = kTwo ? v[kTwo ? e : 0] : u[kTwo ? e : 2 * e + 1];
                        float &y1r = kTwo ? v[kTwo ? e + 1 : 0] : u[kTwo ? e : 2 * e + 3];
                        const float2 x = make_float2(x0r, x1r), y = make_float2(y0r, y1r);
                        const float2 xt = fma2(y, ns, mul2(x, c)), yt = fma2(x, s, mul2(y, c));
                        x0r = xt.x; x1r = xt.y;
                        y0r = yt.x; y1r = yt.y;
                    }
                    if constexpr (kTwo) store_unit<D, N>(dst, hi, v);
                }
            }
            store_unit<D, N>(dst, lo, u);
        }
        if (done + p.batch < mine) __syncthreads();       // the angles are read before the next batch's are written
        tok0 += p.batch_tok;
        head0 += p.batch_head;
        if (head0 >= p.heads_all) {
            head0 -= p.heads_all;
            ++tok0;
        }
    }
}

template <typename S, typename D, int N, bool HALF>
cudaError_t launch_as(RopeParams p, cudaStream_t s) {
    constexpr bool kTwo = HALF || N == 1;
    constexpr int kU = kUnroll<S, N, HALF>;
    const int n = p.dims / (kTwo ? 2 * N : N) + (p.inplace ? 0 : (p.D - p.dims) / N);
    const int most = N == 8 ? 256 : 1024;                 // n <= 128 units of 8, n <= 1023 of 1
    int per = most / n;
    if (N == 1 && per > 1) per = (256 + n - 1) / n < per ? (256 + n - 1) / n : per;
    if (per > p.rows) per = (int)p.rows;
    // the angles of a batch of rows, of as many tokens as it can touch (at most 16 KB for one row
    // at a time, so the loop ends)
    auto shared = [&](int per_) {
        const int64_t tokens = ((int64_t)per_ * kU + p.heads_all - 2) / p.heads_all + 1;
        return (size_t)tokens * (p.dims / 2) * sizeof(float2);
    };
    while (shared(per) > 40 * 1024) per = (per + 1) / 2;
    const int threads = per * n;
    // rows per CTA: whole batches, so that one round of CTAs (four per SM) takes all
    const int64_t few = (int64_t)per * kU;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int64_t batches = (p.rows + few - 1) / few, mul = (batches + 4 * sms - 1) / (4 * sms);
    p.rows_per_cta = few * mul;
    p.per = per;
    p.batch = (int)few;
    p.cta_tok = (int)(p.rows_per_cta / p.heads_all); p.cta_head = (int)(p.rows_per_cta % p.heads_all);
    p.batch_tok = (int)(few / p.heads_all); p.batch_head = (int)(few % p.heads_all);
    p.step_tok = per / p.heads_all; p.step_head = per % p.heads_all;
    const int64_t grid = (p.rows + p.rows_per_cta - 1) / p.rows_per_cta;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(k_rope<S, D, N, HALF>, dim3((unsigned)grid), dim3(threads), shared(per), s, 1, p);
}

template <typename S, typename D>
cudaError_t launch_types(const RopeParams &p, cudaStream_t s) {
    if (p.wide) return p.half ? launch_as<S, D, 8, true>(p, s) : launch_as<S, D, 8, false>(p, s);
    return p.half ? launch_as<S, D, 1, true>(p, s) : launch_as<S, D, 1, false>(p, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, cudaStream_t s) {
    if (p.rows == 0) return cudaSuccess;
    if (p.src_bf16)
        return p.dst_bf16 ? launch_types<__nv_bfloat16, __nv_bfloat16>(p, s) : launch_types<__nv_bfloat16, float>(p, s);
    return p.dst_bf16 ? launch_types<float, __nv_bfloat16>(p, s) : launch_types<float, float>(p, s);
}

}  // namespace hisa
