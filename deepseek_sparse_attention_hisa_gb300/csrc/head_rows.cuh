// One row (a head of a token, a cached row) in the registers of a team of lanes: loaded, normed and
// turned in f32. A team is 2, 4, 8, 16 or 32 neighbouring lanes of a warp; lane l of it owns the units
// l, l + T, ... of 8 neighbouring dims (T lanes, at most U units each), so that a warp's accesses
// are whole lines.
//
//   y = x / sqrt(mean(x^2) + eps) * w;  (a, b) -> mscale (a cos A - b sin A, a sin A + b cos A)
//
// The angle is a fraction of a turn in 64-bit fixed point (pos * table[i] modulo 2^64, as in
// k_rope.cu). A team computes the sines and cosines of a position together, one pair per lane at a
// time, into its own part of shared memory; the lanes of rotated units read them from there (a lane
// that computed those of its own units would take four to eight in turn while the other lanes wait).
// In the half layout a rotated unit's partners are a shuffle away where a lane has one unit; where it has
// more, it loads the unit of its partners as well: a second read of a line that the warp reads anyway.
//
// Where units do not fit (rows or rotated dims that start anywhere, D no multiple of 8) elements are
// loaded and stored one by one and partners are exchanged through shared memory (ANY).
#pragma once

#include "ops_internal.cuh"

namespace hisa {

enum RowForm : int { kPairs = 0, kHalves = 1, kAny = 2 };

template <typename S> struct Raw8 { uint4 v[sizeof(S) / 2]; };   // 8 elements

__device__ __forceinline__ void raw_to_f32(const Raw8<__nv_bfloat16> &r, float (&f)[8]) {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void raw_to_f32(const Raw8<float> &r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(r.v[i].x); f[4 * i + 1] = __uint_as_float(r.v[i].y);
        f[4 * i + 2] = __uint_as_float(r.v[i].z); f[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
}
__device__ __forceinline__ Raw8<__nv_bfloat16> raw_load(const __nv_bfloat16 *p) {
    Raw8<__nv_bfloat16> r;
    r.v[0] = *reinterpret_cast<const uint4 *>(p);
    return r;
}
__device__ __forceinline__ Raw8<float> raw_load(const float *p) {        // a whole sector per lane and access
    Raw8<float> r;
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r.v[0].x), "=r"(r.v[0].y), "=r"(r.v[0].z), "=r"(r.v[0].w), "=r"(r.v[1].x), "=r"(r.v[1].y), "=r"(r.v[1].z), "=r"(r.v[1].w)
                 : "l"(p));
    return r;
}
// n of 8 elements, one by one; the others 0
__device__ __forceinline__ Raw8<float> raw_load_any(const float *p, int n) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = i < n ? p[i] : 0.f;
    Raw8<float> r;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        r.v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                            __float_as_uint(f[4 * i + 3]));
    return r;
}
__device__ __forceinline__ Raw8<__nv_bfloat16> raw_load_any(const __nv_bfloat16 *p, int n) {
    const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (2 * i < n ? (uint32_t)q[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)q[2 * i + 1] << 16 : 0u);
    Raw8<__nv_bfloat16> r;
    r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    return r;
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) { store_sector(p, v); }
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store_any(float *p, const float (&v)[8], int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = v[i];
}
__device__ __forceinline__ void store_any(__nv_bfloat16 *p, const float (&v)[8], int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = __float2bfloat16_rn(v[i]);
}

// What all rows of a launch have in common, and this lane's place in its team.
struct RowShape {
    int D, T, tl;             // dims; lanes of the team, this one's
    int units;                // of 8 dims, the last one cut if D is no multiple of 8 (ANY)
    int first, dims;          // the rotated dims
    int half;
    float inv;                // 1 / D
    float2 *turn;             // the team's [dims / 2] (cos, sin), times mscale
    float *row;               // ANY: the team's [8 units] f32
};

// Writes the team's angles; the caller synchronises the warp before they are read.
__device__ __forceinline__ void team_angles(const RowShape &g, const uint64_t *table, int64_t pos, float mscale) {
    for (int i = g.tl; i < g.dims / 2; i += g.T) {
        const int64_t turns = (int64_t)((uint64_t)pos * __ldg(table + i));        // modulo one turn
        float s, c;
        sincospif(2.f * (__ll2float_rn(turns) * 0x1p-64f), &s, &c);
        g.turn[i] = make_float2(c * mscale, s * mscale);
    }
}

template <typename S, int U, int FORM>
struct RowBuf {
    static constexpr bool kSecond = FORM == kHalves && U > 1;
    Raw8<S> a[U], b[kSecond ? U : 1];                    // units, their partners

    __device__ __forceinline__ void load(const S *x, const RowShape &g) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = i * g.T + g.tl;
            if (u >= g.units) continue;
            if constexpr (FORM == kAny) {
                a[i] = raw_load_any(x + 8 * u, g.D - 8 * u);
            } else {
                a[i] = raw_load(x + 8 * u);
                if constexpr (kSecond) {
                    const int n = g.dims / 8, ru = u - g.first / 8;
                    if (ru >= 0 && ru < n) b[i] = raw_load(x + 8 * (ru < n / 2 ? u + n / 2 : u - n / 2));
                }
            }
        }
    }

    // The row's f32 values, normed (norm) and turned, in y[i] for unit i T + tl. All lanes of the warp
    // take part. HELD: w's values of this lane's units are in held, and w only says that there are any.
    template <bool HELD = false>
    __device__ __forceinline__ void finish(const RowShape &g, bool norm, const float *w, float eps, float (&y)[U][8],
                                           const float2 (*held)[4] = nullptr) const {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i * g.T + g.tl < g.units) {
                raw_to_f32(a[i], y[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[i][e] = 0.f;
            }
        }
        // teams of one warp may differ in whether they norm: all take part in the sum
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float2 q = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 8; e += 2) q = fma2(make_float2(y[i][e], y[i][e + 1]), make_float2(y[i][e], y[i][e + 1]), q);
            sum += q.x + q.y;
        }
        for (int o = g.T >> 1; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float f = rsqrtf(sum * g.inv + eps);            // within 2 steps of f32
        auto scaled = [&](float (&v)[8], int u, int own) {
            if (!norm) return;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 s = mul2(make_float2(v[e], v[e + 1]), make_float2(f, f));
                v[e] = s.x;
                v[e + 1] = s.y;
            }
            if (!w) return;
            if constexpr (FORM == kAny) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (8 * u + e < g.D) v[e] *= __ldg(w + 8 * u + e);
            } else if (HELD && own >= 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 s = mul2(make_float2(v[2 * e], v[2 * e + 1]), held[own < 0 ? 0 : own][e]);
                    v[2 * e] = s.x;
                    v[2 * e + 1] = s.y;
                }
            } else {
                const float4 w0 = __ldg(reinterpret_cast<const float4 *>(w + 8 * u)), w1 = __ldg(reinterpret_cast<const float4 *>(w + 8 * u) + 1);
                const float2 ww[4] = {make_float2(w0.x, w0.y), make_float2(w0.z, w0.w), make_float2(w1.x, w1.y), make_float2(w1.z, w1.w)};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 s = mul2(make_float2(v[2 * e], v[2 * e + 1]), ww[e]);
                    v[2 * e] = s.x;
                    v[2 * e + 1] = s.y;
                }
            }
        };
        if constexpr (FORM == kHalves && U == 1) {
            // one unit per lane: the partner's is in the lane half the rotated units away
            const int n = g.dims / 8, ru = g.tl - g.first / 8;
            const bool low = ru < n / 2;
            if (g.tl < g.units) scaled(y[0], g.tl, 0);
            if (n) {
                float q[8];
                const int from = (threadIdx.x & 31) + (low ? n / 2 : -(n / 2));
#pragma unroll
                for (int e = 0; e < 8; ++e) q[e] = __shfl_sync(0xffffffffu, y[0][e], from & 31);
                if (ru >= 0 && ru < n) {
                    const float4 *cs = reinterpret_cast<const float4 *>(g.turn + 8 * (low ? ru : ru - n / 2));
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 t = cs[k];
                        y[0][2 * k] = y[0][2 * k] * t.x + q[2 * k] * (low ? -t.y : t.y);
                        y[0][2 * k + 1] = y[0][2 * k + 1] * t.z + q[2 * k + 1] * (low ? -t.w : t.w);
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = i * g.T + g.tl;
                if (u >= g.units) continue;
                scaled(y[i], u, i);
                if constexpr (FORM == kAny) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) g.row[8 * u + e] = y[i][e];
                } else {
                    const int n = g.dims / 8, ru = u - g.first / 8;
                    if (ru < 0 || ru >= n) continue;
                    if constexpr (FORM == kPairs) {
                        const float4 *cs = reinterpret_cast<const float4 *>(g.turn + 4 * ru);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float4 t = cs[k];
                            const float a0 = y[i][4 * k], b0 = y[i][4 * k + 1], a1 = y[i][4 * k + 2], b1 = y[i][4 * k + 3];
                            y[i][4 * k] = a0 * t.x - b0 * t.y;
                            y[i][4 * k + 1] = a0 * t.y + b0 * t.x;
                            y[i][4 * k + 2] = a1 * t.z - b1 * t.w;
                            y[i][4 * k + 3] = a1 * t.w + b1 * t.z;
                        }
                    } else {
                        const bool low = ru < n / 2;
                        float q[8];
                        raw_to_f32(b[i], q);
                        scaled(q, low ? u + n / 2 : u - n / 2, -1);
                        const float4 *cs = reinterpret_cast<const float4 *>(g.turn + 8 * (low ? ru : ru - n / 2));
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float4 t = cs[k];
                            y[i][2 * k] = y[i][2 * k] * t.x + q[2 * k] * (low ? -t.y : t.y);
                            y[i][2 * k + 1] = y[i][2 * k + 1] * t.z + q[2 * k + 1] * (low ? -t.w : t.w);
                        }
                    }
                }
            }
        }
        if constexpr (FORM == kAny) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = i * g.T + g.tl;
                if (u >= g.units) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int d = 8 * u + e, rd = d - g.first;
                    if (rd < 0 || rd >= g.dims) continue;
                    const int h = g.dims / 2;
                    const bool low = g.half ? rd < h : !(rd & 1);
                    const int step = g.half ? h : 1;
                    const float2 t = g.turn[g.half ? (low ? rd : rd - h) : rd >> 1];
                    const float q = g.row[low ? d + step : d - step];
                    y[i][e] = y[i][e] * t.x + q * (low ? -t.y : t.y);
                }
            }
            __syncwarp();                                     // the row is read before the next one is written
        }
    }
};

// Lanes of a team for rows of D dims, and the units of each lane (1, 2 or 4).
inline int team_lanes(int D) {
    const int units = (D + 7) / 8;
    int T = 2;
    while (T < units && T < 32) T *= 2;
    return T;
}
inline int team_units(int D) { return D <= 256 ? 1 : (D <= 512 ? 2 : 4); }
// Dynamic shared memory of a CTA of `warps` warps.
inline size_t team_smem(int D, int dims, int warps, bool any) {
    const int teams = warps * (32 / team_lanes(D));
    return (size_t)teams * ((size_t)(dims / 2) * sizeof(float2) + (any ? (size_t)((D + 7) / 8) * 8 * sizeof(float) : 0)) + 16;
}

// This lane's RowShape: the CTA's shared memory holds all teams' angles, then (ANY) their rows.
__device__ __forceinline__ RowShape row_shape(float *sm, int D, int T, int first, int dims, int half, bool any) {
    RowShape g;
    g.D = D; g.T = T; g.units = (D + 7) / 8; g.inv = 1.f / (float)D;
    g.first = first; g.dims = dims; g.half = half;
    const int lane = threadIdx.x & 31;
    g.tl = lane & (T - 1);
    const int team = (int)threadIdx.x / T, teams = (int)blockDim.x / T;
    g.turn = reinterpret_cast<float2 *>(sm) + (size_t)team * (dims / 2);
    g.row = any ? sm + (size_t)teams * dims + (size_t)team * g.units * 8 : nullptr;
    return g;
}

}  // namespace hisa
