// Internal declarations of the operators around the step (norm, rotary positions,
// shared-prefix combine). Nothing here is part of the C ABI (see include/hisa.h).
#pragma once

#include "hisa_internal.cuh"

namespace hisa {

// The kernels here are launched as programmatic dependents, always: each waits for the grid before
// it (grid_dep_wait) before it touches memory that grid may write, and lets the next one be
// scheduled (grid_dep_trigger) right after, so that launches overlap and no grid runs beside the
// one two back.

// Two f32 operations by one instruction (each rounded as alone): many rows are bound by the
// number of instructions before they are by memory.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{.reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x;}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{.reg .b64 x, y; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; add.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x;}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{.reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7}; fma.rn.f32x2 x, x, y, z; "
        "mov.b64 {%0, %1}, x;}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// Eight f32 to a 32-byte aligned address in one access: a whole sector per thread, where two
// 16-byte stores each leave half of one.
__device__ __forceinline__ void store_sector(float *dst, const float *v) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "l"(dst), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

struct NormParams {
    int64_t rows;
    int cols;
    int x_bf16, res_bf16;
    int out_dtype;            // hisa_dtype
    int group;                // columns per scale (0: the row)
    int groups;               // scales per row
    int unit_shift;           // log2 of the 8-column units per scale (the row: past every unit)
    int pow2;
    float eps;
    int64_t ld_x, ld_res, ld_out;
    const void *x;            // [rows, cols]
    const void *res;          // [rows, cols] or nullptr
    const float *w;           // [cols]
    void *res_out;            // [rows, cols] or nullptr
    void *out;                // [rows, cols]
    float *scales;            // [rows, cols / group] (8-bit output)
    int wide;                 // every row start is aligned to 8 elements, cols % 8 == 0
    int phase;                // row 0's start modulo 8 elements if every row's is the same in all arrays, and
                              // scales are per row; else -1
    int chained;              // w may be read before the previous grid has completed
};

struct RopeParams {
    int64_t rows;             // tokens * (heads + heads2)
    int heads, heads_all;     // of x; of x and x2
    int D, dims, first, half;
    int src_bf16, dst_bf16;
    int inplace;
    float mscale, sin_sign;
    const uint64_t *table;
    const int32_t *pos;
    const void *x, *x2;
    void *y, *y2;
    int64_t x_token, x_head, y_token, y_head, x2_token, x2_head, y2_token, y2_head;
    // set by launch_rope: rows of a CTA, of a batch, and that a CTA takes at once, and the tokens and
    // heads that each of them is (the kernel then divides nothing of 64 bits)
    int64_t rows_per_cta;
    int batch, per;
    int cta_tok, cta_head, batch_tok, batch_head, step_tok, step_head;
    int wide;                 // 8 elements per access fit every boundary
};

// One shared-prefix combine. Partials of a segment (a range of the shared rows, or of a query
// row's own list) are unnormalised sums with their running maximum and sum of exponentials.
struct PrefixParams {
    int B, L, H, Dh, window, W_max, r;
    int64_t P, Np_max, kv_rows;
    float scale;
    const void *q, *local_kv, *prefix_kv, *pooled_kv;
    const int32_t *local_len, *local_pos0, *t0;
    const int64_t *kv_off;
    const float *sinks;       // or nullptr
    void *out;
    int bf16, out_bf16;
    int tail_split;           // segments [0, tail_split): a query row's local and own rows
    int tail_rows;            // list rows of one of them
    int pre_split;            // segments [tail_split, tail_split + pre_split): shared rows (on the
                              // tensor cores all rows, and no tail segments)
    int64_t pre_rows;         // shared rows of one of them (not for 512 bf16 dims)
    float *part_o;            // [segments, B * L * H, Dh]
    float *part_ml;           // [segments, B * L * H, 2]: maximum (of the logits), sum
    uint32_t *status;
};

// Encodes a 3-D tensor map over bf16 [rows, cols]: chunks of 64 columns as the slowest
// dimension, so one box of box_chunks x box_rows x 64 lands as box_chunks swizzled (128-byte)
// K-major operand chunks. False if the driver has no encoder or rejects the map.
bool encode_bf16_chunks(CUtensorMap *map, const void *base, uint64_t rows, uint64_t cols, uint32_t box_rows,
                        uint32_t box_chunks);

size_t prefix_workspace_bytes(const hisa_prefix_desc *d);

cudaError_t launch_rms_norm(const NormParams &p, cudaStream_t s);
cudaError_t launch_rope(const RopeParams &p, cudaStream_t s);
cudaError_t launch_prefix_simt(const PrefixParams &p, int tail, cudaStream_t s);
// The whole combine on the tensor cores for 64 bf16 heads of 512 dims: pre_split segments of each
// query row's rows (own and shared), or with one segment the output itself.
bool prefix_tc_supported(int H, int Dh, int bf16);
cudaError_t launch_prefix_tc(const PrefixParams &p, cudaStream_t s);
// The shared rows' segments on the tensor cores for bf16 heads of 64 and 128 dims.
cudaError_t launch_prefix_tc1(const PrefixParams &p, cudaStream_t s);
cudaError_t launch_prefix_merge(const PrefixParams &p, cudaStream_t s);

}  // namespace hisa
