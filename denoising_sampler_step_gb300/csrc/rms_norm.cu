// Root-mean-square norm of the hidden stream with the residual's addition, and its gradient.
//
//   h = x + residual,  rstd = 1 / sqrt(mean h^2 + eps),  y = h rstd (offset + weight)
//   dh = grad_hidden + rstd (g - xh mean(g xh)),  g = dy (offset + weight),  xh = h rstd
//   dweight = sum over the rows of dy xh
//
// Both are bound by HBM: a CTA keeps a row in registers from its load to its last store, so that every
// matrix is moved once.  Forward, the norm is taken of the fp32 sum h, not of the h that is stored (which
// is rounded once).  An 8-bit output takes the row's largest |y| before the first code is written:
// scale = amax / 448 and codes = e4m3(y / scale), as the table's rows are quantised.  Backward, a thread
// keeps its columns' part of dweight in fp32 registers over all rows of its CTA; a second kernel adds the
// CTAs' parts in a fixed order.
#include <algorithm>

#include "dg_internal.h"
#include "hidden.cuh"

namespace dg {

namespace {

using namespace hidden;

// Threads of a row's CTA, by the eights of columns that each takes (row_shape).
constexpr int max_threads(int n) { return n == 1 ? 256 : n == 2 ? 512 : 1024; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Sum over the CTA, the same in every thread; `parts` is free again after the next barrier but one.
__device__ __forceinline__ float cta_sum(float v, float *parts) {
    v = warp_sum(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < warps; ++w) v += parts[w];
    return v;
}

// The largest magnitude's bits over the CTA: as whole numbers NaN is above infinity.
__device__ __forceinline__ uint32_t cta_max(uint32_t v, uint32_t *parts) {
    v = __reduce_max_sync(0xffffffffu, v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = v;
    __syncthreads();
    for (int w = 0; w < warps; ++w) v = max(v, parts[w]);
    return v;
}

struct NormParams {
    NormRows a;
};

template <typename TX, typename TR, typename TO, int N, bool kWide>
__global__ void __launch_bounds__(max_threads(N)) rms_norm_kernel(const NormParams p) {
    constexpr bool kCodes = sizeof(TO) == 1;
    __shared__ float sums[32];
    __shared__ uint32_t maxima[32];
    const NormRows &a = p.a;
    const int64_t r = blockIdx.x;
    const int d = (int)a.d;
    const TX *x = static_cast<const TX *>(a.x.p) + r * a.x.ld;
    const TR *res = static_cast<const TR *>(a.residual.p) + (a.residual.p ? r * a.residual.ld : 0);
    float v[N][8];
    {
        Raw8<TX> rx[N];
        Raw8<TR> rr[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = 8 * (threadIdx.x + i * blockDim.x);
            if (c < d) load8<kWide>(rx[i], x + c, d - c);
        }
        if (a.residual.p)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = 8 * (threadIdx.x + i * blockDim.x);
                if (c < d) load8<kWide>(rr[i], res + c, d - c);
            }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = 8 * (threadIdx.x + i * blockDim.x);
            if (c < d) {
                unpack8(v[i], rx[i]);
                if (a.residual.p) {
                    float t[8];
                    unpack8(t, rr[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] += t[j];
                }
                mask8(v[i], d - c);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
            }
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float q = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) q = fmaf(v[i][j], v[i][j], q);
        s += q;
    }
    if (a.hidden.p)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = 8 * (threadIdx.x + i * blockDim.x);
            if (c < d) store8_any<kWide>(a.hidden.p, a.hidden.dtype, r * a.hidden.ld + c, v[i], d - c);
        }
    const float mean = cta_sum(s, sums) / (float)d;
    const float rstd = 1.0f / sqrtf(mean + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = 8 * (threadIdx.x + i * blockDim.x);
        if (c < d) {
            float w[8];
            if (a.weight) {
                load8_any<kWide>(w, a.weight, a.weight_dtype, c, d - c);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * (a.weight_offset + w[j]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] *= rstd;
            }
            if constexpr (kCodes) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < d) top = max(top, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
            }
        }
    }
    TO *out = static_cast<TO *>(a.out.p) + r * a.out.ld;
    float scale = 0.0f;
    if constexpr (kCodes) {
        scale = __fdiv_rn(__uint_as_float(cta_max(top, maxima)), 448.0f);
        if (threadIdx.x == 0) a.scale[r] = scale;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = 8 * (threadIdx.x + i * blockDim.x);
        if (c < d) {
            if constexpr (kCodes) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = scale != 0.0f ? __fdiv_rn(v[i][j], scale) : 0.0f;
            }
            store8<kWide>(out + c, v[i], d - c);
        }
    }
}

struct NormBackParams {
    NormBackRows a;
    float *parts;  // [gridDim.x, part_ld]
    int64_t part_ld;
};

template <typename TG, typename TH, typename TD, int N, bool kWide>
__global__ void __launch_bounds__(max_threads(N)) rms_norm_backward_kernel(const NormBackParams p) {
    __shared__ float sums[2][32];
    const NormBackRows &a = p.a;
    const int d = (int)a.d;
    float dw[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x, turn ^= 1) {
        Raw8<TG> rg[N];
        Raw8<TH> rh[N];
        Raw8<TD> rd[N];
        const TG *gp = static_cast<const TG *>(a.grad.p) + r * a.grad.ld;
        const TH *hp = static_cast<const TH *>(a.hidden.p) + r * a.hidden.ld;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = 8 * (threadIdx.x + i * blockDim.x);
            if (c < d) {
                load8<kWide>(rg[i], gp + c, d - c);
                load8<kWide>(rh[i], hp + c, d - c);
            }
        }
        if (a.grad_hidden.p) {
            const TD *dp = static_cast<const TD *>(a.grad_hidden.p) + r * a.grad_hidden.ld;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = 8 * (threadIdx.x + i * blockDim.x);
                if (c < d) load8<kWide>(rd[i], dp + c, d - c);
            }
        }
        const float rstd = a.rstd[r];
        float g[N][8], xh[N][8];
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = 8 * (threadIdx.x + i * blockDim.x);
            if (c < d) {
                float w[8], q = 0.0f;
                unpack8(g[i], rg[i]);
                unpack8(xh[i], rh[i]);
                mask8(g[i], d - c);
                mask8(xh[i], d - c);
                if (a.weight) load8_any<kWide>(w, a.weight, a.weight_dtype, c, d - c);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    xh[i][j] *= rstd;
                    dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
                    if (a.weight) g[i][j] *= a.weight_offset + w[j];
                    q = fmaf(g[i][j], xh[i][j], q);
                }
                s += q;
            }
        }
        const float mean = cta_sum(s, sums[turn]) / (float)d;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = 8 * (threadIdx.x + i * blockDim.x);
            if (c < d) {
                float t[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) t[j] = 0.0f;
                if (a.grad_hidden.p) unpack8(t, rd[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[i][j] = fmaf(rstd, fmaf(-mean, xh[i][j], g[i][j]), t[j]);
                store8<kWide>(static_cast<TH *>(a.grad_x.p) + r * a.grad_x.ld + c, g[i], d - c);
            }
        }
    }
    if (a.grad_weight)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = 8 * (threadIdx.x + i * blockDim.x);
            if (c < d) store8<true>(p.parts + blockIdx.x * p.part_ld + c, dw[i], 8);
        }
}

// dweight from the CTAs' parts: a warp row of 32 columns, the CTA's warps a share of the parts each.
__global__ void __launch_bounds__(1024) norm_weight_kernel(const float *__restrict__ parts, int64_t part_ld, int n,
                                                           int64_t d, void *__restrict__ out, int dtype) {
    __shared__ float acc[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    const int per = (n + 31) / 32;
    float s = 0.0f;
    if (c < d)
        for (int i = warp * per; i < min(n, (warp + 1) * per); ++i) s += parts[i * part_ld + c];
    acc[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < d) {
        s = 0.0f;
        for (int w = 0; w < 32; ++w) s += acc[w][lane];
        if (dtype == DG_F32)
            static_cast<float *>(out)[c] = s;
        else
            static_cast<__nv_bfloat16 *>(out)[c] = __float2bfloat16_rn(s);
    }
}

bool wide_vector(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Threads of a row's CTA and eights of columns per thread; wide: all rows start where the widest accesses may.
struct Shape {
    int threads, n;
    bool wide;
};
Shape row_shape(int64_t d, bool wide) {
    const int64_t eights = (d + 7) / 8;
    const int n = !wide ? 4 : eights <= 256 ? 1 : eights <= 1024 ? 2 : 4;
    return {(int)(((eights + n - 1) / n + 31) / 32 * 32), n, wide};
}

template <typename TX, typename TR, typename TO>
void norm_width(const NormParams &p, const Shape &s, cudaStream_t stream) {
    const unsigned grid = (unsigned)p.a.R;
    if (!s.wide)
        rms_norm_kernel<TX, TR, TO, 4, false><<<grid, s.threads, 0, stream>>>(p);
    else if (s.n == 1)
        rms_norm_kernel<TX, TR, TO, 1, true><<<grid, s.threads, 0, stream>>>(p);
    else if (s.n == 2)
        rms_norm_kernel<TX, TR, TO, 2, true><<<grid, s.threads, 0, stream>>>(p);
    else
        rms_norm_kernel<TX, TR, TO, 4, true><<<grid, s.threads, 0, stream>>>(p);
}
template <typename TX, typename TR>
void norm_out(const NormParams &p, const Shape &s, cudaStream_t stream) {
    if (p.a.out.dtype == DG_F32)
        norm_width<TX, TR, float>(p, s, stream);
    else if (p.a.out.dtype == DG_BF16)
        norm_width<TX, TR, __nv_bfloat16>(p, s, stream);
    else
        norm_width<TX, TR, E4m3>(p, s, stream);
}
template <typename TX>
void norm_residual(const NormParams &p, const Shape &s, cudaStream_t stream) {
    if (p.a.residual.p && p.a.residual.dtype == DG_F32)
        norm_out<TX, float>(p, s, stream);
    else
        norm_out<TX, __nv_bfloat16>(p, s, stream);
}

template <typename TG, typename TH, typename TD>
void back_width(const NormBackParams &p, const Shape &s, unsigned grid, cudaStream_t stream) {
    if (!s.wide)
        rms_norm_backward_kernel<TG, TH, TD, 4, false><<<grid, s.threads, 0, stream>>>(p);
    else if (s.n == 1)
        rms_norm_backward_kernel<TG, TH, TD, 1, true><<<grid, s.threads, 0, stream>>>(p);
    else if (s.n == 2)
        rms_norm_backward_kernel<TG, TH, TD, 2, true><<<grid, s.threads, 0, stream>>>(p);
    else
        rms_norm_backward_kernel<TG, TH, TD, 4, true><<<grid, s.threads, 0, stream>>>(p);
}
template <typename TG, typename TH>
void back_residual(const NormBackParams &p, const Shape &s, unsigned grid, cudaStream_t stream) {
    if (p.a.grad_hidden.p && p.a.grad_hidden.dtype == DG_F32)
        back_width<TG, TH, float>(p, s, grid, stream);
    else
        back_width<TG, TH, __nv_bfloat16>(p, s, grid, stream);
}

int64_t part_stride(int64_t d) { return (d + 7) / 8 * 8; }

// CTAs of the backward pass: as many rows in work as the SMs' threads allow.
int64_t back_grid(int64_t R, const Shape &s) {
    return std::min<int64_t>(R, (int64_t)std::max(1, device_sm_count()) * std::max(1, std::min(16, 1024 / s.threads)));
}

}  // namespace

cudaError_t launch_rms_norm(const NormRows &a, cudaStream_t stream) {
    const NormParams p{a};
    const Shape s = row_shape(a.d, wide_rows(a.x) && wide_rows(a.residual) && wide_rows(a.hidden) && wide_rows(a.out) &&
                                       wide_vector(a.weight));
    if (a.x.dtype == DG_F32)
        norm_residual<float>(p, s, stream);
    else
        norm_residual<__nv_bfloat16>(p, s, stream);
    return cudaGetLastError();
}

size_t rms_norm_backward_bytes(int64_t R, int64_t d) {
    const int64_t most = std::max(back_grid(R, row_shape(d, true)), back_grid(R, row_shape(d, false)));
    return (size_t)most * (size_t)part_stride(d) * sizeof(float);
}

cudaError_t launch_rms_norm_backward(const NormBackRows &a, void *workspace, cudaStream_t stream) {
    const NormBackParams p{a, static_cast<float *>(workspace), part_stride(a.d)};
    const Shape s = row_shape(a.d, wide_rows(a.grad) && wide_rows(a.hidden) && wide_rows(a.grad_hidden) &&
                                       wide_rows(a.grad_x) && wide_vector(a.weight));
    const unsigned grid = (unsigned)back_grid(a.R, s);
    const bool g32 = a.grad.dtype == DG_F32, h32 = a.hidden.dtype == DG_F32;
    if (a.R > 0) {
        if (g32 && h32)
            back_residual<float, float>(p, s, grid, stream);
        else if (g32)
            back_residual<float, __nv_bfloat16>(p, s, grid, stream);
        else if (h32)
            back_residual<__nv_bfloat16, float>(p, s, grid, stream);
        else
            back_residual<__nv_bfloat16, __nv_bfloat16>(p, s, grid, stream);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (a.grad_weight)
        norm_weight_kernel<<<(unsigned)((a.d + 31) / 32), 1024, 0, stream>>>(p.parts, p.part_ld, a.R > 0 ? (int)grid : 0,
                                                                            a.d, a.grad_weight, a.weight_dtype);
    return cudaGetLastError();
}

}  // namespace dg
