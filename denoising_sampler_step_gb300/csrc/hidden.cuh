// What the operators on the hidden stream share (token_embed.cu, rms_norm.cu): rows of fp32, bf16 or
// E4M3 entries taken eight columns at a time, and the arguments their launchers take.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dgsamp.h"
#include "dg_common.cuh"

namespace dg {

// A matrix of rows; `ld` in elements.
struct Rows {
    void *p;
    int64_t ld;
    int dtype;  // dg_dtype
};

inline int entry_size(int dtype) { return dtype == DG_F32 ? 4 : dtype == DG_BF16 ? 2 : 1; }

// Whether every row starts where eight entries can be moved by the widest accesses (E4M3: 8 bytes, else 16).
inline bool wide_rows(const Rows &m) {
    const uintptr_t a = m.dtype == DG_E4M3 ? 7 : 15;
    return !m.p || ((reinterpret_cast<uintptr_t>(m.p) & a) == 0 && (((uintptr_t)m.ld * entry_size(m.dtype)) & a) == 0);
}

namespace hidden {

struct E4m3 {
    uint8_t code;
};

// Eight entries as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
    float4 a, b;
};
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
};
template <>
struct Raw8<E4m3> {
    uint2 a;
};

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Eight entries at q, those from n on anything (kWide) or zeros.  Without kWide they lie `step` apart, so that
// neighbouring threads read neighbouring entries.  kWide: q starts where rows may (wide_rows), and whole 16-byte groups (E4M3: 8) that hold an entry are read, without a branch: a choice between
// kinds of loads at run time, or a branch on n, kept rows from being in flight side by side.
template <bool kWide>
__device__ __forceinline__ void load8(Raw8<float> &r, const float *q, int n, int step = 1) {
    if constexpr (kWide) {
        r.a = *reinterpret_cast<const float4 *>(q);
        r.b = n > 4 ? *reinterpret_cast<const float4 *>(q + 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j * step < n ? q[j * step] : 0.0f;
        r.a = make_float4(v[0], v[1], v[2], v[3]);
        r.b = make_float4(v[4], v[5], v[6], v[7]);
    }
}
template <bool kWide>
__device__ __forceinline__ void load8(Raw8<__nv_bfloat16> &r, const __nv_bfloat16 *q, int n, int step = 1) {
    if constexpr (kWide) {
        r.a = *reinterpret_cast<const uint4 *>(q);
    } else {
        uint32_t w[4];
        const uint16_t *u = reinterpret_cast<const uint16_t *>(q);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = (2 * j * step < n ? (uint32_t)u[2 * j * step] : 0u) |
                   ((2 * j + 1) * step < n ? (uint32_t)u[(2 * j + 1) * step] << 16 : 0u);
        r.a = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
template <bool kWide>
__device__ __forceinline__ void load8(Raw8<E4m3> &r, const E4m3 *q, int n, int step = 1) {
    if constexpr (kWide) {
        r.a = *reinterpret_cast<const uint2 *>(q);
    } else {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j * step < n) w[j >> 2] |= (uint32_t)q[j * step].code << (8 * (j & 3));
        r.a = make_uint2(w[0], w[1]);
    }
}

__device__ __forceinline__ void unpack8(float (&v)[8], const Raw8<float> &r) {
    v[0] = r.a.x, v[1] = r.a.y, v[2] = r.a.z, v[3] = r.a.w;
    v[4] = r.b.x, v[5] = r.b.y, v[6] = r.b.z, v[7] = r.b.w;
}
__device__ __forceinline__ void unpack8(float (&v)[8], const Raw8<__nv_bfloat16> &r) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[2 * j] = bf16_low(w[j]), v[2 * j + 1] = bf16_high(w[j]);
}
// (every E4M3 value is a half)
__device__ __forceinline__ void unpack8(float (&v)[8], const Raw8<E4m3> &r) {
    const uint32_t w[2] = {r.a.x, r.a.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w[j >> 1] >> (16 * (j & 1)))));
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
            : "=f"(v[2 * j]), "=f"(v[2 * j + 1])
            : "r"(h2));
    }
}

// Zeros in place of the values from n on.
__device__ __forceinline__ void mask8(float (&v)[8], int n, int step = 1) {
    if (n <= 7 * step)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = j * step < n ? v[j] : 0.0f;
}

// The first n of eight values, each rounded once.
template <bool kWide>
__device__ __forceinline__ void store8(float *q, const float (&v)[8], int n, int step = 1) {
    if (kWide && n >= 8) {
        *reinterpret_cast<float4 *>(q) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(q + 4) = make_float4(v[4], v[5], v[6], v[7]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j * step < n) q[j * step] = v[j];
}
template <bool kWide>
__device__ __forceinline__ void store8(__nv_bfloat16 *q, const float (&v)[8], int n, int step = 1) {
    const uint4 w = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    if (kWide && n >= 8) {
        *reinterpret_cast<uint4 *>(q) = w;
        return;
    }
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j * step < n) reinterpret_cast<uint16_t *>(q)[j * step] = (uint16_t)(u[j >> 1] >> (16 * (j & 1)));
}
template <bool kWide>
__device__ __forceinline__ void store8(E4m3 *q, const float (&v)[8], int n, int step = 1) {
    const uint2 w = make_uint2(pack_e4m3x2(v[0], v[1]) | pack_e4m3x2(v[2], v[3]) << 16,
                               pack_e4m3x2(v[4], v[5]) | pack_e4m3x2(v[6], v[7]) << 16);
    if (kWide && n >= 8) {
        *reinterpret_cast<uint2 *>(q) = w;
        return;
    }
    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j * step < n) q[j * step].code = (uint8_t)(u[j >> 2] >> (8 * (j & 3)));
}

// Eight entries of a type known at run time only, fp32 or not (bf16).
struct Any8 {
    uint4 a, b;
};
__device__ __forceinline__ void load8(Any8 &r, const void *p, bool f32, int64_t at, int n, int step) {
    if (f32) {
        Raw8<float> t;
        load8<false>(t, static_cast<const float *>(p) + at, n, step);
        r.a = *reinterpret_cast<const uint4 *>(&t.a);
        r.b = *reinterpret_cast<const uint4 *>(&t.b);
    } else {
        Raw8<__nv_bfloat16> t;
        load8<false>(t, static_cast<const __nv_bfloat16 *>(p) + at, n, step);
        r.a = t.a;
    }
}
__device__ __forceinline__ void unpack8(float (&v)[8], const Any8 &r, bool f32) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    if (f32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[2 * j] = bf16_low(w[j]), v[2 * j + 1] = bf16_high(w[j]);
    }
}
template <bool kWide>
__device__ __forceinline__ void store8(void *p, bool f32, int64_t at, const float (&v)[8], int n, int step = 1) {
    if (f32)
        store8<kWide>(static_cast<float *>(p) + at, v, n, step);
    else
        store8<kWide>(static_cast<__nv_bfloat16 *>(p) + at, v, n, step);
}

}  // namespace hidden

// ---------------------------------------------------------------- launchers

struct EmbedRows {
    Rows table;          // row j is vocabulary entry vocab_start + j; forward: read, backward: the gradient
    const float *scale;  // E4M3: one per row
    int64_t V, vocab_start, vocab_end;
    int64_t R, d;
    const int32_t *token;
    float gamma;
    Rows rows;        // [R, d]: forward the output, backward the gradient of it
    bool accumulate;  // backward: add to the gradient that is there
};
cudaError_t launch_token_embed(const EmbedRows &a, cudaStream_t stream);
size_t token_embed_backward_bytes(int64_t R, int64_t d);
cudaError_t launch_token_embed_backward(const EmbedRows &a, void *workspace, cudaStream_t stream);

constexpr int64_t kMaxNormWidth = 32768;
struct NormRows {
    Rows x, residual, hidden, out;  // residual, hidden: p may be NULL
    float *scale, *rstd;            // scale: with an E4M3 out; rstd: may be NULL
    const void *weight;             // may be NULL
    int weight_dtype;
    float weight_offset, eps;
    int64_t R, d;
};
cudaError_t launch_rms_norm(const NormRows &a, cudaStream_t stream);

struct NormBackRows {
    Rows grad, hidden, grad_hidden, grad_x;  // grad_hidden: p may be NULL
    const float *rstd;
    const void *weight;  // may be NULL
    int weight_dtype;
    float weight_offset;
    void *grad_weight;  // [d] of weight_dtype, may be NULL
    int64_t R, d;
};
size_t rms_norm_backward_bytes(int64_t R, int64_t d);
cudaError_t launch_rms_norm_backward(const NormBackRows &a, void *workspace, cudaStream_t stream);

cudaError_t launch_head_e4m3(const uint8_t *X, int64_t ldx, const float *x_scale, int64_t R, int64_t d,
                             const uint8_t *Q, int64_t ldq, const float *scale, int64_t V, void *logits, int dtype,
                             int64_t ldl, cudaStream_t stream, const char **msg);

}  // namespace dg
