// The norm of each head and rotary positions in one pass over queries and keys.
//
// Bound by memory: each head is read once and written once. A team of lanes (head_rows.cuh) takes a run of up to 8 heads
// of one token, so that a token's sines and cosines are computed once per run. In flight are 32 warps per SM, each with
// one head of more than 256 dims or, for each of its teams, four of fewer (two in f32): 4096 x 65 x 512 f32 to bf16 133
// us with one head per team, 150 with two (more than memory serves at once, and registers); 2047 x 64 x 128 bf16 with
// halves 25.1, 21.3 and 19.9 us with one, two and four. Runs of 16 heads: 147 us and the same.
//
// Measured: the first of these 6.1 TB/s, 90 % of a plain copy's rate; the second 18.2 us now, 3.7 TB/s: a chain of load, sum over
// lanes, angles and store per head, with too few bytes in flight; a token of 64 + 1 heads of 512 4.7 us per call.
#include "cache_internal.cuh"
#include "head_rows.cuh"

namespace hisa {
namespace {

template <int FORM>
constexpr int kWarps = FORM == kAny ? 4 : 8;

template <typename S, typename Y, int U, int FORM>
__global__ void __launch_bounds__(32 * kWarps<FORM>, FORM == kAny ? 1 : (U == 4 ? 2 : 4)) k_norm_rope(NormRopeParams p) {
    constexpr int kK = U > 1 ? 1 : (sizeof(S) == 2 ? 4 : 2);   // heads in flight per team
    extern __shared__ __align__(16) float sm[];
    const RowShape g = row_shape(sm, p.D, p.lanes, p.first, p.dims, p.half, FORM == kAny);
    const int64_t item = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / p.lanes;
    grid_dep_wait();
    grid_dep_trigger();
    const int64_t tok = item / p.runs;
    const int run = (int)(item - tok * p.runs);
    const bool there = tok < p.tokens;                    // a warp's last teams may have nothing to do
    const bool two = run >= p.runs1;
    const int h0 = (two ? run - p.runs1 : run) * p.run, heads = two ? p.heads2 : p.heads;
    const S *x = static_cast<const S *>(two ? p.x2 : p.x) + (there ? tok * (two ? p.x2_token : p.x_token) : 0);
    Y *y = static_cast<Y *>(two ? p.y2 : p.y) + (there ? tok * (two ? p.y2_token : p.y_token) : 0);
    const int64_t xh = two ? p.x2_head : p.x_head, yh = two ? p.y2_head : p.y_head;
    const float *w = two ? p.w2 : p.w;
    const bool norm = two ? p.norm2 : p.norm;
    const int n = there ? (heads - h0 < p.run ? heads - h0 : p.run) : 0;
    for (int k0 = 0; k0 < p.run; k0 += kK) {              // the same trips for all teams of a warp
        RowBuf<S, U, FORM> buf[kK] = {};
#pragma unroll
        for (int k = 0; k < kK; ++k)
            if (k0 + k < n) buf[k].load(x + (h0 + k0 + k) * xh, g);
        if (k0 == 0 && p.dims && there) team_angles(g, p.table, p.pos[tok], p.mscale);
        __syncwarp();                                     // the angles; and in place a head is loaded before it is written
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            float v[U][8];
            buf[k].finish(g, norm, w, p.eps, v);
            if (k0 + k >= n) continue;
            Y *to = y + (h0 + k0 + k) * yh;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = i * g.T + g.tl;
                if (u >= g.units) continue;
                if constexpr (FORM == kAny) store_any(to + 8 * u, v[i], p.D - 8 * u);
                else store8(to + 8 * u, v[i]);
            }
        }
    }
}

template <typename S, typename Y, int U, int FORM>
cudaError_t go(NormRopeParams p, cudaStream_t s) {
    p.lanes = team_lanes(p.D);
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // heads of a run: as many as leave a warp for every scheduler slot of the GPU
    p.run = 8;
    auto teams = [&](int run) { return p.tokens * ((p.heads + run - 1) / run + (p.heads2 + run - 1) / run); };
    while (p.run > 1 && teams(p.run) * p.lanes / 32 < 32 * (int64_t)sms) p.run /= 2;
    p.runs1 = (p.heads + p.run - 1) / p.run;
    p.runs = p.runs1 + (p.heads2 + p.run - 1) / p.run;
    const int threads = 32 * kWarps<FORM>;
    const int64_t grid = (p.tokens * p.runs * p.lanes + threads - 1) / threads;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    const size_t smem = team_smem(p.D, p.dims, kWarps<FORM>, FORM == kAny);
    return launch_pdl(k_norm_rope<S, Y, U, FORM>, dim3((unsigned)grid), dim3(threads), smem, s, 1, p);
}

template <typename S, typename Y>
cudaError_t forms(const NormRopeParams &p, cudaStream_t s) {
    const int U = team_units(p.D);
    if (!p.wide) return U == 1 ? go<S, Y, 1, kAny>(p, s) : (U == 2 ? go<S, Y, 2, kAny>(p, s) : go<S, Y, 4, kAny>(p, s));
    if (p.half) return U == 1 ? go<S, Y, 1, kHalves>(p, s) : (U == 2 ? go<S, Y, 2, kHalves>(p, s) : go<S, Y, 4, kHalves>(p, s));
    return U == 1 ? go<S, Y, 1, kPairs>(p, s) : (U == 2 ? go<S, Y, 2, kPairs>(p, s) : go<S, Y, 4, kPairs>(p, s));
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams &p, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (p.src_bf16) return p.dst_bf16 ? forms<B, B>(p, s) : forms<B, float>(p, s);
    return p.dst_bf16 ? forms<float, B>(p, s) : forms<float, float>(p, s);
}

}  // namespace hisa
