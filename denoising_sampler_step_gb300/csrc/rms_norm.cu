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

// Threads of a row's CTA at most, by the eights of columns that each takes: forward and backward.
constexpr int max_threads(int n) { return n == 1 ? 256 : n == 2 ? 512 : 1024; }
constexpr int max_back_threads(int n) { return n == 4 ? 1024 : 512; }

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

// A row as it lies in memory, this thread's columns of it.
template <typename TG, typename TH, typename TD, int N>
struct BackRow {
    Raw8<TG> g[N];
    Raw8<TH> h[N];
    Raw8<TD> up[N];
    float rstd;
};

// Loads in flight side by side: a thread past the row's end reads its last eight columns again, in place of a branch.
template <bool kUp, bool kWide, typename TG, typename TH, typename TD, int N>
__device__ __forceinline__ void load_row(BackRow<TG, TH, TD, N> &row, const NormBackRows &a, int64_t r, const int (&col)[N]) {
    const TG *g = static_cast<const TG *>(a.grad.p) + r * a.grad.ld;
    const TH *h = static_cast<const TH *>(a.hidden.p) + r * a.hidden.ld;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        load8<kWide>(row.g[i], g + col[i], (int)a.d - col[i]);
        load8<kWide>(row.h[i], h + col[i], (int)a.d - col[i]);
    }
    if constexpr (kUp) {
        const TD *up = static_cast<const TD *>(a.grad_hidden.p) + r * a.grad_hidden.ld;
#pragma unroll
        for (int i = 0; i < N; ++i) load8<kWide>(row.up[i], up + col[i], (int)a.d - col[i]);
    }
    row.rstd = a.rstd[r];
}

// kUp: with grad_hidden.  The next row is loaded while this one is reduced and stored.
template <typename TG, typename TH, typename TD, int N, bool kUp, bool kWide>
__global__ void __launch_bounds__(max_back_threads(N)) rms_norm_backward_kernel(const NormBackParams p) {
    __shared__ float sums[2][32];
    const NormBackRows &a = p.a;
    const int d = (int)a.d, last = (d - 1) / 8 * 8;
    int col[N];
    float w[N][8], dw[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int c = 8 * (threadIdx.x + i * blockDim.x);
        col[i] = min(c, last);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f, w[i][j] = 1.0f;
        if (a.weight) {
            load8_any<kWide>(w[i], a.weight, a.weight_dtype, col[i], d - col[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[i][j] += a.weight_offset;
        }
        mask8(w[i], d - c);  // (all zeros past the row's end)
    }
    const float inv_d = 1.0f / (float)d;
    BackRow<TG, TH, TD, N> row;
    if (blockIdx.x < a.R) load_row<kUp, kWide>(row, a, blockIdx.x, col);
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x, turn ^= 1) {
        float g[N][8], xh[N][8], up[kUp ? N : 1][8];
        const float rstd = row.rstd;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float q = 0.0f;
            unpack8(g[i], row.g[i]);
            unpack8(xh[i], row.h[i]);
            if constexpr (kUp) unpack8(up[i], row.up[i]);
            mask8(g[i], d - 8 * (int)(threadIdx.x + i * blockDim.x));  // (nothing past the row's end counts)
            mask8(xh[i], d - 8 * (int)(threadIdx.x + i * blockDim.x));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[i][j] *= rstd;
                dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
                g[i][j] *= w[i][j];
                q = fmaf(g[i][j], xh[i][j], q);
            }
            s += q;
        }
        if (r + gridDim.x < a.R) load_row<kUp, kWide>(row, a, r + gridDim.x, col);
        const float mean = cta_sum(s, sums[turn]) * inv_d;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = 8 * (threadIdx.x + i * blockDim.x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g[i][j] = rstd * fmaf(-mean, xh[i][j], g[i][j]);
                if constexpr (kUp) g[i][j] += up[i][j];
            }
            if (c < d) store8<kWide>(static_cast<TH *>(a.grad_x.p) + r * a.grad_x.ld + c, g[i], d - c);
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

// Eights of columns per thread, the fewest with which a row fits a CTA; off the boundaries (not wide) one kernel is
// enough for all rows but the widest.
template <typename Max>
int eights_per_thread(int64_t d, bool wide, int narrow, Max most) {
    const int64_t eights = (d + 7) / 8;
    for (const int n : {1, 2})
        if (eights <= n * most(n) && (wide || n == narrow)) return n;
    return 4;
}
int row_threads(int64_t d, int n) { return (int)((((d + 7) / 8 + n - 1) / n + 31) / 32 * 32); }

template <typename TX, typename TR, typename TO>
void norm_width(const NormParams &p, bool wide, cudaStream_t stream) {
    const unsigned grid = (unsigned)p.a.R;
    const int n = eights_per_thread(p.a.d, wide, 2, max_threads), threads = row_threads(p.a.d, n);
    (wide ? n == 1   ? rms_norm_kernel<TX, TR, TO, 1, true>
            : n == 2 ? rms_norm_kernel<TX, TR, TO, 2, true>
                     : rms_norm_kernel<TX, TR, TO, 4, true>
     : n == 2 ? rms_norm_kernel<TX, TR, TO, 2, false>
              : rms_norm_kernel<TX, TR, TO, 4, false>)<<<grid, threads, 0, stream>>>(p);
}
template <typename TX, typename TR>
void norm_out(const NormParams &p, bool wide, cudaStream_t stream) {
    if (p.a.out.dtype == DG_F32)
        norm_width<TX, TR, float>(p, wide, stream);
    else if (p.a.out.dtype == DG_BF16)
        norm_width<TX, TR, __nv_bfloat16>(p, wide, stream);
    else
        norm_width<TX, TR, E4m3>(p, wide, stream);
}
template <typename TX>
void norm_residual(const NormParams &p, bool wide, cudaStream_t stream) {
    if (p.a.residual.p && p.a.residual.dtype == DG_F32)
        norm_out<TX, float>(p, wide, stream);
    else
        norm_out<TX, __nv_bfloat16>(p, wide, stream);
}

int64_t part_stride(int64_t d) { return (d + 7) / 8 * 8; }

// CTAs of the backward pass at most: as many as the SMs could hold.
int64_t back_grid_most(int64_t R, int64_t d) {
    return std::min<int64_t>(R, (int64_t)std::max(1, device_sm_count()) * std::min(32, 2048 / row_threads(d, 4)));
}

// One wave of CTAs, each of which keeps its columns' sums over all its rows; *grid: how many.
template <typename TG, typename TH, typename TD, int N, bool kUp, bool kWide>
cudaError_t launch_back(const NormBackParams &p, unsigned *grid, cudaStream_t stream) {
    const auto kernel = rms_norm_backward_kernel<TG, TH, TD, N, kUp, kWide>;
    const int threads = row_threads(p.a.d, N);
    int per_sm = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0);
    if (e != cudaSuccess) return e;
    *grid = (unsigned)std::min(back_grid_most(p.a.R, p.a.d), (int64_t)std::max(1, device_sm_count()) * std::max(1, per_sm));
    kernel<<<*grid, threads, 0, stream>>>(p);
    return cudaGetLastError();
}
template <typename TG, typename TH, typename TD, bool kUp>
cudaError_t back_width(const NormBackParams &p, bool wide, unsigned *grid, cudaStream_t stream) {
    const int n = eights_per_thread(p.a.d, wide, 1, max_back_threads);
    if (wide)
        return n == 1   ? launch_back<TG, TH, TD, 1, kUp, true>(p, grid, stream)
               : n == 2 ? launch_back<TG, TH, TD, 2, kUp, true>(p, grid, stream)
                        : launch_back<TG, TH, TD, 4, kUp, true>(p, grid, stream);
    return n == 1 ? launch_back<TG, TH, TD, 1, kUp, false>(p, grid, stream)
                  : launch_back<TG, TH, TD, 4, kUp, false>(p, grid, stream);
}
template <typename TG, typename TH>
cudaError_t back_residual(const NormBackParams &p, bool wide, unsigned *grid, cudaStream_t stream) {
    if (!p.a.grad_hidden.p) return back_width<TG, TH, float, false>(p, wide, grid, stream);
    return p.a.grad_hidden.dtype == DG_F32 ? back_width<TG, TH, float, true>(p, wide, grid, stream)
                                           : back_width<TG, TH, __nv_bfloat16, true>(p, wide, grid, stream);
}

}  // namespace

cudaError_t launch_rms_norm(const NormRows &a, cudaStream_t stream) {
    const NormParams p{a};
    const bool wide = wide_rows(a.x) && wide_rows(a.residual) && wide_rows(a.hidden) && wide_rows(a.out) &&
                      wide_vector(a.weight);
    if (a.x.dtype == DG_F32)
        norm_residual<float>(p, wide, stream);
    else
        norm_residual<__nv_bfloat16>(p, wide, stream);
    return cudaGetLastError();
}

size_t rms_norm_backward_bytes(int64_t R, int64_t d) {
    return (size_t)back_grid_most(R, d) * (size_t)part_stride(d) * sizeof(float);
}

cudaError_t launch_rms_norm_backward(const NormBackRows &a, void *workspace, cudaStream_t stream) {
    const NormBackParams p{a, static_cast<float *>(workspace), part_stride(a.d)};
    const bool wide = wide_rows(a.grad) && wide_rows(a.hidden) && wide_rows(a.grad_hidden) && wide_rows(a.grad_x) &&
                      wide_vector(a.weight);
    unsigned grid = 0;
    if (a.R > 0) {
        const bool g32 = a.grad.dtype == DG_F32, h32 = a.hidden.dtype == DG_F32;
        const cudaError_t e = g32 ? h32 ? back_residual<float, float>(p, wide, &grid, stream)
                                        : back_residual<float, __nv_bfloat16>(p, wide, &grid, stream)
                              : h32 ? back_residual<__nv_bfloat16, float>(p, wide, &grid, stream)
                                    : back_residual<__nv_bfloat16, __nv_bfloat16>(p, wide, &grid, stream);
        if (e != cudaSuccess) return e;
    }
    if (a.grad_weight)
        norm_weight_kernel<<<(unsigned)((a.d + 31) / 32), 1024, 0, stream>>>(p.parts, p.part_ld, (int)grid, a.d,
                                                                            a.grad_weight, a.weight_dtype);
    return cudaGetLastError();
}

}  // namespace dg
