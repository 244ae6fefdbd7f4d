// Root-mean-square norm of the hidden stream with the residual's addition, and its gradient.
//
//   h = x + residual,  rstd = 1 / sqrt(mean h^2 + eps),  y = h rstd (offset + weight)
//   dh = grad_hidden + rstd (g - xh mean(g xh)),  g = dy (offset + weight),  xh = h rstd
//   dweight = sum over the rows of dy xh
//
// Both are bound by HBM.  A CTA takes every gridDim.x-th row and keeps it in registers from its arrival to its last
// store, so that every matrix is moved once; the rows to come arrive meanwhile in a ring of shared memory by bulk
// copies that a warp of their own sends for (with the next row in registers an SM held too few rows to keep the memory
// busy; sent for by a warp that also computes, the copies held every row up).  What is left per row and thread is some
// 150 instructions: types are known at compile time, and arithmetic is in pairs.  Forward, the norm is taken of the
// fp32 sum h, not of the h that is stored (which is rounded once).  An 8-bit output takes the row's largest |y| before
// the first code is written: scale = amax / 448 and codes = e4m3(y / scale), as the table's rows are quantised.
// Backward, a thread keeps its columns' part of dweight in fp32 registers over all rows of its CTA; a second kernel adds
// the CTAs' parts in a fixed order.  Rows that start off 16-byte boundaries, and rows that do not fit, are read where
// they lie.
//
// 8,192 rows of 2,816: bf16 with an fp32 residual to codes, hidden kept, 44 us (5.8 TB/s of 254 MB; between other work
// 39 us); the gradient in bf16 with the residual's 34 us (5.4 TB/s), some 4 of them the second kernel's.  What keeps them from a
// copy's rate is latency: an SM holds 6 to 8 rows, and a row's two sums over its threads stop its loads' consumer.  One row of
// 2,816: 2.6 us.  Rows read where they lie: 20,001 x 1,001 bf16 62 us, its gradient 82 us.
// Above 8,192 columns a thread's eight eights do not fit its registers: 2,000 x 10,001 bf16 29 us (0.41 of a copy's rate; 0.6 kB
// spilled a thread), the gradient 106 us (0.17; 2.2 kB); 2,000 x 8,192 17 us (0.58) and 29 us (0.50).
#include <algorithm>
#include <atomic>

#include "dg_internal.h"
#include "hidden.cuh"
#include "vocab_row.cuh"

namespace dg {

namespace {

using namespace hidden;
using vocab::add2;
using vocab::f32x2;
using vocab::fma2;
using vocab::mul2;
using vocab::pair;
using vocab::unpair;

constexpr int kMaxStages = 16;
constexpr int kRingHeader = 16 * kMaxStages;  // the ring's barriers, and room past its end: a thread reads eight
constexpr int kRingTail = 32;                 // columns where fewer are left
constexpr int kSmemPerSm = 224 * 1024, kSmemLimit = 232448 - 1024;  // of an SM's CTAs, and of one

// Threads that work on a row at most, by the eights of columns that each takes.
__host__ __device__ constexpr int max_threads(int n) { return n == 1 || n == 8 ? 512 : 256; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// A barrier of the row's threads.
__device__ __forceinline__ void row_sync(int threads) { asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory"); }

// Sum over the row's threads, the same in all; `parts` is free again after the next barrier but one.
__device__ __forceinline__ float row_sum(float v, float *parts, int threads) {
    v = warp_sum(v);
    if (threads == 32) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) parts[threadIdx.x >> 5] = v;
    row_sync(threads);
    return warp_sum(lane < threads >> 5 ? parts[lane] : 0.0f);
}

// The largest magnitude's bits: as whole numbers NaN is above infinity.
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *parts, int threads) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (threads == 32) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) parts[threadIdx.x >> 5] = v;
    row_sync(threads);
    return __reduce_max_sync(0xffffffffu, lane < threads >> 5 ? parts[lane] : 0u);
}

// 1 / sqrt(x) within some 2^-23: the hardware's, and a Newton step where x is positive and finite.  (The exact root
// and quotient were a tenth of the forward kernel's instructions.)
__device__ __forceinline__ float inv_sqrt(float x) {
    const float r = rsqrtf(x);
    return x > 0.0f && x < INFINITY ? fmaf(0.5f * r, fmaf(-x * r, r, 1.0f), r) : r;
}

// Rows of up to three matrices on their way through shared memory.
struct Source {
    Rows m[3];
    int bytes[3];  // of a row, in whole 16-byte groups; 0: no such matrix
    int stages, stage_bytes;
};

// The CTA's k-th row, blockIdx.x + k gridDim.x, is in slot k % stages: `full` once it has arrived, `empty` once every
// warp of the row's threads has read it.
struct Ring {
    uint8_t *slots;
    uint64_t *full, *empty;
    volatile int *gave_up;
    int stages, stage_bytes;
    int slot = 0;
    uint32_t phase = 0;

    __device__ __forceinline__ Ring(const Source &src, uint4 *smem, volatile int *flag, int threads)
        : slots(reinterpret_cast<uint8_t *>(smem) + kRingHeader), full(reinterpret_cast<uint64_t *>(smem)),
          empty(full + kMaxStages), gave_up(flag), stages(src.stages), stage_bytes(src.stage_bytes) {
        if (threadIdx.x == 0) {
            *gave_up = 0;
            for (int s = 0; s < stages; ++s) {
                mbar_init(smem_u32(&full[s]), 1);
                mbar_init(smem_u32(&empty[s]), threads >> 5);
            }
            fence_mbar_init();
        }
        __syncthreads();
    }
    __device__ __forceinline__ void next() {
        if (++slot == stages) {
            slot = 0;
            phase ^= 1;
        }
    }
    // One thread sends for all of the CTA's rows.
    __device__ __forceinline__ void send(const Source &src, int64_t R) {
        bool again = false;  // the slot has been used before
        for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
            if (again && !mbar_wait(smem_u32(&empty[slot]), phase ^ 1, gave_up)) return;
            const uint32_t bar = smem_u32(&full[slot]);
            uint32_t at = smem_u32(slots) + (uint32_t)slot * stage_bytes;
            mbar_arrive_expect_tx(bar, (uint32_t)stage_bytes);
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                if (src.bytes[q] == 0) continue;
                const char *row = static_cast<const char *>(src.m[q].p) + r * src.m[q].ld * (src.m[q].dtype == DG_F32 ? 4 : 2);
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(at),
                             "l"(row), "r"(src.bytes[q]), "r"(bar)
                             : "memory");
                at += src.bytes[q];
            }
            next();
            if (slot == 0) again = true;
        }
    }
    // The row's slot, once it has arrived.  (A wait that gave up has recorded it, and the row is computed of what is there.)
    __device__ __forceinline__ const uint8_t *wait() {
        mbar_wait(smem_u32(&full[slot]), phase, gave_up);
        return slots + slot * stage_bytes;
    }
    // This warp has read the slot for the last time.
    __device__ __forceinline__ void release() {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&empty[slot]));
    }
    // Copies in flight after a wait gave up land before the CTA leaves.
    __device__ __forceinline__ void leave() {
        __syncthreads();
        if (*gave_up) {
            const unsigned long long t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
        }
    }
};

// This thread's columns: from 8 (threadIdx.x + i threads) on.  Past the row's end it reads the row's last ones, counts
// zeros and writes nothing.
template <int N>
struct Columns {
    int at[N], read[N], n[N];
    __device__ __forceinline__ Columns(int width, int threads) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            at[i] = 8 * (threadIdx.x + i * threads);
            read[i] = min(at[i], (width - 1) / 8 * 8);
            n[i] = width - at[i];
        }
    }
};

// The same where rows are read element by element: eight columns `step` apart, neighbouring threads' side by side.
template <int N>
struct Strided {
    int at[N], n[N], step;
    __device__ __forceinline__ Strided(int width, int threads) : step(threads) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            at[i] = threadIdx.x + i * 8 * threads;
            n[i] = width - at[i];
        }
    }
};

// Eight columns as pairs, those from n on as zeros.
__device__ __forceinline__ void mask4(f32x2 (&v)[4], int n) {
    if (n < 8)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a, b;
            unpair(v[j], a, b);
            v[j] = pair(2 * j < n ? a : 0.0f, 2 * j + 1 < n ? b : 0.0f);
        }
}
template <bool kF32>
__device__ __forceinline__ void read4(f32x2 (&v)[4], const uint8_t *row, int at, int n) {
    if constexpr (kF32) {
        const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(row + 4 * at);
        const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(row + 4 * at + 16);
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    } else {
        const uint4 a = *reinterpret_cast<const uint4 *>(row + 2 * at);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = pair(bf16_low(w[j]), bf16_high(w[j]));
    }
    mask4(v, n);
}
__device__ __forceinline__ void singles(float (&v)[8], const f32x2 (&p)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) unpair(p[j], v[2 * j], v[2 * j + 1]);
}

// offset + weight in these columns (ones without a weight), zeros past the row's end.
__device__ __forceinline__ void load_weight(float (&w)[8], const void *weight, int dtype, float offset, int at, int n, int step) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.0f;
    if (weight) {
        Any8 raw;
        load8(raw, weight, dtype == DG_F32, at, n, step);
        unpack8(w, raw, dtype == DG_F32);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] += offset;
    }
    mask8(w, n, step);
}
template <int N>
__device__ __forceinline__ void load_weight(f32x2 (&w)[N][4], const void *weight, int dtype, float offset,
                                            const Columns<N> &col) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float v[8];
        load_weight(v, weight, dtype, offset, col.at[i], col.n[i], 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[i][j] = pair(v[2 * j], v[2 * j + 1]);
    }
}

// A matrix of a row: none, bf16, or fp32.
enum { kNone = 0, kBf16 = 1, kF32 = 2 };
int kind_of(const Rows &m) { return !m.p ? kNone : m.dtype == DG_F32 ? kF32 : kBf16; }

// ---------------------------------------------------------------- forward

struct NormParams {
    NormRows a;
    Source src;  // x, residual
};

// y / scale in place of -y, rounded once: quotients of bf16 operands are often ties between two codes, and a rounding more
// takes the other one.  The product with the scale's reciprocal is put right by its remainder, which a fused product leaves
// exact (Markstein's correction; 8,192 x 2,816 43.9 us, with divisions 51.7); from -y the sum keeps the sign of a zero.
// Scales so small that a remainder would not be a normal number, and those that are no number, divide.
__device__ __forceinline__ void to_codes(f32x2 (&v)[4], float scale) {
    if (scale >= 0x1p-80f && scale < INFINITY) {
        const float inv = 1.0f / scale;
        const f32x2 rr = pair(-inv, -inv), ss = pair(scale, scale);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x2 q = mul2(v[j], rr);
            v[j] = fma2(fma2(q, ss, v[j]), rr, q);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float a, b;
            unpair(v[j], a, b);
            v[j] = scale != 0.0f ? pair(__fdiv_rn(a, -scale), __fdiv_rn(b, -scale)) : 0;
        }
    }
}
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// kX, kRes: what x and the residual are; hidden has the residual's type (none: no hidden).
template <int N, int kX, int kRes, bool kCodes>
__global__ void __launch_bounds__(max_threads(N) + 32) rms_norm_kernel(const NormParams p) {
    extern __shared__ uint4 smem[];
    __shared__ float sums[2][32];
    __shared__ uint32_t maxima[2][32];
    __shared__ int gave_up;
    const NormRows &a = p.a;
    const int d = (int)a.d, threads = blockDim.x - 32;
    Ring ring(p.src, smem, &gave_up, threads);
    if ((int)threadIdx.x >= threads) {
        if ((int)threadIdx.x == threads) ring.send(p.src, a.R);
        ring.leave();
        return;
    }
    const Columns<N> col(d, threads);
    const float inv_d = 1.0f / (float)d;
    const bool out32 = a.out.dtype == DG_F32;
    f32x2 w[N][4];
    load_weight(w, a.weight, a.weight_dtype, a.weight_offset, col);
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x, turn ^= 1) {
        f32x2 v[N][4], sq = 0;
        const uint8_t *row = ring.wait();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            read4<kX == kF32>(v[i], row, col.read[i], col.n[i]);
            if constexpr (kRes != kNone) {
                f32x2 t[4];
                read4<kRes == kF32>(t, row + p.src.bytes[0], col.read[i], col.n[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = add2(v[i][j], t[j]);
            }
            f32x2 q = mul2(v[i][0], v[i][0]);
#pragma unroll
            for (int j = 1; j < 4; ++j) q = fma2(v[i][j], v[i][j], q);
            sq = add2(sq, q);
        }
        ring.release();
        ring.next();
        float s0, s1;
        unpair(sq, s0, s1);
        const float rstd = inv_sqrt(fmaf(row_sum(s0 + s1, sums[turn], threads), inv_d, a.eps));
        if constexpr (kRes != kNone)
            if (a.hidden.p)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    float h[8];
                    singles(h, v[i]);
                    if (col.n[i] > 0) store8<true>(a.hidden.p, kRes == kF32, r * a.hidden.ld + col.at[i], h, col.n[i]);
                }
        if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
        uint32_t top = 0;
        const f32x2 rr = kCodes ? pair(-rstd, -rstd) : pair(rstd, rstd);  // (to_codes takes -y)
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i][j] = mul2(mul2(v[i][j], rr), w[i][j]);
                if constexpr (kCodes) {
                    // (past the row's end 0, or NaN where the whole row has one)
                    float y0, y1;
                    unpair(v[i][j], y0, y1);
                    top = max(top, max(magnitude(y0), magnitude(y1)));
                }
            }
        float scale = 0.0f;
        if constexpr (kCodes) {
            scale = __fdiv_rn(__uint_as_float(row_max(top, maxima[turn], threads)), 448.0f);
            if (threadIdx.x == 0) a.scale[r] = scale;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float y[8];
            if constexpr (kCodes) to_codes(v[i], scale);
            singles(y, v[i]);
            if (col.n[i] > 0) {
                if constexpr (kCodes)
                    store8<true>(static_cast<E4m3 *>(a.out.p) + r * a.out.ld + col.at[i], y, col.n[i]);
                else
                    store8<true>(a.out.p, out32, r * a.out.ld + col.at[i], y, col.n[i]);
            }
        }
    }
    ring.leave();
}

// Rows read where they lie, element by element; any types.
template <int N>
__global__ void __launch_bounds__(max_threads(N)) rms_norm_plain_kernel(const NormParams p) {
    __shared__ float sums[2][32];
    __shared__ uint32_t maxima[2][32];
    const NormRows &a = p.a;
    const int d = (int)a.d, threads = blockDim.x;
    const Strided<N> col(d, threads);
    const bool codes = a.out.dtype == DG_E4M3;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x, turn ^= 1) {
        float v[N][8], s = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            Any8 raw;
            load8(raw, a.x.p, a.x.dtype == DG_F32, r * a.x.ld + col.at[i], col.n[i], col.step);
            unpack8(v[i], raw, a.x.dtype == DG_F32);
            if (a.residual.p) {
                float t[8];
                load8(raw, a.residual.p, a.residual.dtype == DG_F32, r * a.residual.ld + col.at[i], col.n[i], col.step);
                unpack8(t, raw, a.residual.dtype == DG_F32);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += t[j];
            }
            mask8(v[i], col.n[i], col.step);
            float q = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) q = fmaf(v[i][j], v[i][j], q);
            s += q;
        }
        const float rstd = inv_sqrt(fmaf(row_sum(s, sums[turn], threads), 1.0f / (float)d, a.eps));
        if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (a.hidden.p && col.n[i] > 0)
                store8<false>(a.hidden.p, a.hidden.dtype == DG_F32, r * a.hidden.ld + col.at[i], v[i], col.n[i], col.step);
            float w[8];
            load_weight(w, a.weight, a.weight_dtype, a.weight_offset, col.at[i], col.n[i], col.step);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = v[i][j] * rstd * w[j];
                top = max(top, magnitude(v[i][j]));
            }
        }
        float scale = 0.0f;
        if (codes) {
            scale = __fdiv_rn(__uint_as_float(row_max(top, maxima[turn], threads)), 448.0f);
            if (threadIdx.x == 0) a.scale[r] = scale;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (col.n[i] <= 0) continue;
            if (codes) {
                f32x2 q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = pair(-v[i][2 * j], -v[i][2 * j + 1]);
                to_codes(q, scale);
                singles(v[i], q);
                store8<false>(static_cast<E4m3 *>(a.out.p) + r * a.out.ld + col.at[i], v[i], col.n[i], col.step);
            } else {
                store8<false>(a.out.p, a.out.dtype == DG_F32, r * a.out.ld + col.at[i], v[i], col.n[i], col.step);
            }
        }
    }
}

// ---------------------------------------------------------------- backward

struct NormBackParams {
    NormBackRows a;
    Source src;    // grad, hidden, grad_hidden
    float *parts;  // [gridDim.x, part_ld]
    int64_t part_ld;
};

template <int N, bool kG32, bool kH32, int kUp>
__global__ void __launch_bounds__(max_threads(N) + 32) rms_norm_backward_kernel(const NormBackParams p) {
    extern __shared__ uint4 smem[];
    __shared__ float sums[2][32];
    __shared__ int gave_up;
    const NormBackRows &a = p.a;
    const int d = (int)a.d, threads = blockDim.x - 32;
    grid_launch_dependents();  // (the sum of the parts waits for this kernel's end on the SMs)
    Ring ring(p.src, smem, &gave_up, threads);
    if ((int)threadIdx.x >= threads) {
        if ((int)threadIdx.x == threads) ring.send(p.src, a.R);
        ring.leave();
        return;
    }
    const Columns<N> col(d, threads);
    const float inv_d = 1.0f / (float)d;
    f32x2 w[N][4], dw[N][4];
    load_weight(w, a.weight, a.weight_dtype, a.weight_offset, col);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[i][j] = 0;
    float next_rstd = blockIdx.x < a.R ? a.rstd[blockIdx.x] : 0.0f;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x, turn ^= 1) {
        f32x2 g[N][4], xh[N][4], sq = 0;
        const float rstd = next_rstd;
        const f32x2 rr = pair(rstd, rstd);
        if (r + gridDim.x < a.R) next_rstd = a.rstd[r + gridDim.x];
        const uint8_t *row = ring.wait();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            read4<kG32>(g[i], row, col.read[i], col.n[i]);
            read4<kH32>(xh[i], row + p.src.bytes[0], col.read[i], col.n[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                xh[i][j] = mul2(xh[i][j], rr);
                dw[i][j] = fma2(g[i][j], xh[i][j], dw[i][j]);
                g[i][j] = mul2(g[i][j], w[i][j]);
                sq = fma2(g[i][j], xh[i][j], sq);
            }
        }
        float s0, s1;
        unpair(sq, s0, s1);
        const float mean = row_sum(s0 + s1, sums[turn], threads) * inv_d;
        const f32x2 mm = pair(-mean, -mean);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            f32x2 up[4];
            if constexpr (kUp != kNone) read4<kUp == kF32>(up, row + p.src.bytes[0] + p.src.bytes[1], col.read[i], col.n[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                g[i][j] = mul2(rr, fma2(mm, xh[i][j], g[i][j]));
                if constexpr (kUp != kNone) g[i][j] = add2(g[i][j], up[j]);
            }
            float y[8];
            singles(y, g[i]);
            if (col.n[i] > 0) store8<true>(a.grad_x.p, kH32, r * a.grad_x.ld + col.at[i], y, col.n[i]);
        }
        ring.release();
        ring.next();
    }
    if (a.grad_weight)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (col.n[i] > 0) {
                float y[8];
                singles(y, dw[i]);
                store8<true>(p.parts + blockIdx.x * p.part_ld + col.at[i], y, 8);
            }
    ring.leave();
}

// Rows read where they lie, element by element; any types.
template <int N>
__global__ void __launch_bounds__(max_threads(N)) rms_norm_backward_plain_kernel(const NormBackParams p) {
    __shared__ float sums[2][32];
    const NormBackRows &a = p.a;
    const int d = (int)a.d, threads = blockDim.x;
    const Strided<N> col(d, threads);
    float dw[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.R; r += gridDim.x, turn ^= 1) {
        const float rstd = a.rstd[r];
        float g[N][8], xh[N][8], s = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float w[8], q = 0.0f;
            Any8 raw;
            load_weight(w, a.weight, a.weight_dtype, a.weight_offset, col.at[i], col.n[i], col.step);
            load8(raw, a.grad.p, a.grad.dtype == DG_F32, r * a.grad.ld + col.at[i], col.n[i], col.step);
            unpack8(g[i], raw, a.grad.dtype == DG_F32);
            load8(raw, a.hidden.p, a.hidden.dtype == DG_F32, r * a.hidden.ld + col.at[i], col.n[i], col.step);
            unpack8(xh[i], raw, a.hidden.dtype == DG_F32);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                xh[i][j] *= rstd;
                dw[i][j] = fmaf(g[i][j], xh[i][j], dw[i][j]);
                g[i][j] *= w[j];
                q = fmaf(g[i][j], xh[i][j], q);
            }
            s += q;
        }
        const float mean = row_sum(s, sums[turn], threads) * (1.0f / (float)d);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (col.n[i] <= 0) continue;
            float up[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) up[j] = 0.0f;
            if (a.grad_hidden.p) {
                Any8 raw;
                load8(raw, a.grad_hidden.p, a.grad_hidden.dtype == DG_F32, r * a.grad_hidden.ld + col.at[i], col.n[i], col.step);
                unpack8(up, raw, a.grad_hidden.dtype == DG_F32);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) g[i][j] = rstd * fmaf(-mean, xh[i][j], g[i][j]) + up[j];
            store8<false>(a.grad_x.p, a.grad_x.dtype == DG_F32, r * a.grad_x.ld + col.at[i], g[i], col.n[i], col.step);
        }
    }
    if (a.grad_weight)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (col.n[i] > 0) store8<false>(p.parts + blockIdx.x * p.part_ld + col.at[i], dw[i], col.n[i], col.step);
}

// dweight from the CTAs' parts, 16 columns a CTA: 128 parts at once, four lanes each, so that a thread's loads are in
// flight together.  It is resident while the parts are written: they are read past L1, and not as constant data.
constexpr int kWeightThreads = 512, kWeightCols = 16;
__global__ void __launch_bounds__(kWeightThreads) norm_weight_kernel(const float *parts, int64_t part_ld, int n, int64_t d,
                                                                     void *out, int dtype) {
    __shared__ float4 acc[kWeightThreads / 32][kWeightCols / 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = (int64_t)blockIdx.x * kWeightCols + lane % 4 * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    grid_dependency_wait();
    if (c < part_ld)
#pragma unroll 8
        for (int i = threadIdx.x / 4; i < n; i += kWeightThreads / 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(parts + i * part_ld + c));
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
        s.x += __shfl_xor_sync(0xffffffffu, s.x, off);
        s.y += __shfl_xor_sync(0xffffffffu, s.y, off);
        s.z += __shfl_xor_sync(0xffffffffu, s.z, off);
        s.w += __shfl_xor_sync(0xffffffffu, s.w, off);
    }
    if (lane < 4) acc[warp][lane] = s;
    __syncthreads();
    const int64_t col = (int64_t)blockIdx.x * kWeightCols + threadIdx.x;
    if (threadIdx.x < kWeightCols && col < d) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kWeightThreads / 32; ++i) sum += reinterpret_cast<const float *>(acc[i])[threadIdx.x];
        if (dtype == DG_F32)
            static_cast<float *>(out)[col] = sum;
        else
            static_cast<__nv_bfloat16 *>(out)[col] = __float2bfloat16_rn(sum);
    }
}

// ---------------------------------------------------------------- plan

int row_threads(int64_t d, int n) { return (int)((((d + 7) / 8 + n - 1) / n + 31) / 32 * 32); }

// Eights of columns per thread.  Many rows: two where that leaves four warps, whose instructions per row are then fewer
// (8,192 x 2,816, gradient: 34 us against 42).  Few rows to an SM: one, for a row's time (one row of 2,816: 2.5 us
// against 3.0).
constexpr int kFewRowsPerSm = 32;
int eights_per_thread(int64_t d, int64_t R) {
    const int64_t eights = (d + 7) / 8;
    const bool few = R <= kFewRowsPerSm * (int64_t)std::max(1, device_sm_count());
    return eights <= (few ? max_threads(1) : 128) ? 1 : eights <= 2 * max_threads(2) ? 2 : eights <= 4 * max_threads(4) ? 4 : 8;
}

// A launch: CTAs of a row each, as many as the SMs hold, the shared memory left to each as its ring.
struct Plan {
    bool ring;
    int n, threads, smem;  // threads: of a row
    unsigned grid;
};
constexpr int kRingFixed = kRingHeader + kRingTail, kMaxCtas = 16;  // bytes; CTAs of an SM

// `wide`: the matrices that are written may be reached by the widest accesses.
Plan make_plan(Source *src, int64_t R, int64_t d, bool wide) {
    Plan plan{};
    src->stage_bytes = 0;
    bool ring = wide;
    for (int q = 0; q < 3; ++q) {
        src->bytes[q] = src->m[q].p ? (int)((d * entry_size(src->m[q].dtype) + 15) / 16 * 16) : 0;
        src->stage_bytes += src->bytes[q];
        ring = ring && wide_rows(src->m[q]);
    }
    plan.ring = ring && src->stage_bytes <= kSmemLimit - kRingFixed;
    plan.n = plan.ring ? eights_per_thread(d, R) : (d + 7) / 8 <= max_threads(1) ? 1 : 8;
    plan.threads = row_threads(d, plan.n);
    const int64_t sms = std::max(1, device_sm_count());
    plan.grid = (unsigned)std::min<int64_t>(R, sms * std::min(kMaxCtas, 2048 / plan.threads));
    return plan;
}

// The rest of a ring's plan, for a kernel of so many registers a thread.
void plan_ring(Plan *plan, Source *src, int64_t R, int regs, bool even) {
    const int64_t sms = std::max(1, device_sm_count()), rows_per_sm = (R + sms - 1) / sms;
    const int held = 65536 / ((regs + 7) / 8 * 8 * (plan->threads + 32));
    int ctas = (int)std::max<int64_t>(1, std::min<int64_t>(rows_per_sm, std::min(held, kMaxCtas)));
    while (ctas > 1 && kSmemPerSm / ctas - 1024 - kRingFixed < 2 * src->stage_bytes) --ctas;  // two rows at least for each
    const int room = std::min(kSmemLimit, kSmemPerSm / ctas - 1024) - kRingFixed;
    const int64_t rows_per_cta = (rows_per_sm + ctas - 1) / ctas;
    src->stages = (int)std::max<int64_t>(1, std::min<int64_t>(std::min(kMaxStages, room / src->stage_bytes), rows_per_cta));
    plan->smem = kRingFixed + src->stages * src->stage_bytes;
    plan->grid = (unsigned)std::min<int64_t>(R, sms * ctas);
    if (!even) return;
    // no more CTAs than the rounds of rows need: each leaves a part to be added up (gradient, 1,000 x 1,024: 6.2 us
    // for 6.9; forward, where they leave nothing, 2,000 x 2,816: 15.4 for 14.5)
    const int64_t rounds = (R + plan->grid - 1) / plan->grid;
    plan->grid = (unsigned)((R + rounds - 1) / rounds);
}

// What is asked of the device once per kernel.
struct Asked {
    std::atomic<int> regs[64];  // 0: not yet
};
template <typename Params>
cudaError_t launch_ring(void (*kernel)(Params), Asked &asked, Params p, Plan plan, bool even, unsigned *grid, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    int regs = e == cudaSuccess && dev < 64 ? asked.regs[dev].load(std::memory_order_acquire) : 0;
    if (e == cudaSuccess && regs == 0) {
        cudaFuncAttributes attr;
        e = cudaFuncGetAttributes(&attr, kernel);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e == cudaSuccess) regs = attr.numRegs;
        if (e == cudaSuccess && dev < 64) asked.regs[dev].store(regs, std::memory_order_release);
    }
    if (e != cudaSuccess) return e;
    plan_ring(&plan, &p.src, p.a.R, regs, even);
    *grid = plan.grid;
    kernel<<<plan.grid, plan.threads + 32, plan.smem, stream>>>(p);
    return cudaGetLastError();
}

template <int N, int kX, int kRes, bool kCodes>
cudaError_t forward(const NormParams &p, const Plan &plan, cudaStream_t stream) {
    static Asked asked;
    unsigned grid;
    return launch_ring(rms_norm_kernel<N, kX, kRes, kCodes>, asked, p, plan, false, &grid, stream);
}
template <int N, int kX, int kRes>
cudaError_t forward_out(const NormParams &p, const Plan &plan, cudaStream_t stream) {
    return p.a.out.dtype == DG_E4M3 ? forward<N, kX, kRes, true>(p, plan, stream) : forward<N, kX, kRes, false>(p, plan, stream);
}
template <int N, int kX>
cudaError_t forward_residual(const NormParams &p, const Plan &plan, cudaStream_t stream) {
    const int kind = kind_of(p.a.residual);
    return kind == kNone   ? forward_out<N, kX, kNone>(p, plan, stream)
           : kind == kBf16 ? forward_out<N, kX, kBf16>(p, plan, stream)
                           : forward_out<N, kX, kF32>(p, plan, stream);
}
template <int N>
cudaError_t forward_types(const NormParams &p, const Plan &plan, cudaStream_t stream) {
    return p.a.x.dtype == DG_F32 ? forward_residual<N, kF32>(p, plan, stream) : forward_residual<N, kBf16>(p, plan, stream);
}

template <int N, bool kG32, bool kH32, int kUp>
cudaError_t backward(const NormBackParams &p, const Plan &plan, unsigned *grid, cudaStream_t stream) {
    static Asked asked;
    return launch_ring(rms_norm_backward_kernel<N, kG32, kH32, kUp>, asked, p, plan, true, grid, stream);
}
template <int N, bool kG32, bool kH32>
cudaError_t backward_up(const NormBackParams &p, const Plan &plan, unsigned *grid, cudaStream_t stream) {
    const int kind = kind_of(p.a.grad_hidden);
    return kind == kNone   ? backward<N, kG32, kH32, kNone>(p, plan, grid, stream)
           : kind == kBf16 ? backward<N, kG32, kH32, kBf16>(p, plan, grid, stream)
                           : backward<N, kG32, kH32, kF32>(p, plan, grid, stream);
}
template <int N>
cudaError_t backward_types(const NormBackParams &p, const Plan &plan, unsigned *grid, cudaStream_t stream) {
    const bool h32 = p.a.hidden.dtype == DG_F32;
    if (p.a.grad.dtype == DG_F32)
        return h32 ? backward_up<N, true, true>(p, plan, grid, stream) : backward_up<N, true, false>(p, plan, grid, stream);
    return h32 ? backward_up<N, false, true>(p, plan, grid, stream) : backward_up<N, false, false>(p, plan, grid, stream);
}

int64_t part_stride(int64_t d) { return (d + 7) / 8 * 8; }

}  // namespace

cudaError_t launch_rms_norm(const NormRows &a, cudaStream_t stream) {
    NormParams p{a, {}};
    p.src.m[0] = a.x;
    p.src.m[1] = a.residual;
    // hidden of another type than the residual, or without one, has no kernel of its own: rows are read where they lie (8,192 x
    // 2,816 bf16 with an fp32 hidden 148 us, of the residual's type 33 us)
    const bool plain = a.hidden.p && (!a.residual.p || a.hidden.dtype != a.residual.dtype);
    const Plan plan = make_plan(&p.src, a.R, a.d, !plain && wide_rows(a.hidden) && wide_rows(a.out));
    if (plan.ring)
        return plan.n == 1   ? forward_types<1>(p, plan, stream)
               : plan.n == 2 ? forward_types<2>(p, plan, stream)
               : plan.n == 4 ? forward_types<4>(p, plan, stream)
                             : forward_types<8>(p, plan, stream);
    (plan.n == 1 ? rms_norm_plain_kernel<1> : rms_norm_plain_kernel<8>)<<<plan.grid, plan.threads, 0, stream>>>(p);
    return cudaGetLastError();
}

size_t rms_norm_backward_bytes(int64_t R, int64_t d) {
    const int64_t most = std::min<int64_t>(R, kMaxCtas * (int64_t)std::max(1, device_sm_count()));
    return (size_t)most * (size_t)part_stride(d) * sizeof(float);
}

cudaError_t launch_rms_norm_backward(const NormBackRows &a, void *workspace, cudaStream_t stream) {
    NormBackParams p{a, {}, static_cast<float *>(workspace), part_stride(a.d)};
    unsigned grid = 0;
    if (a.R > 0) {
        p.src.m[0] = a.grad;
        p.src.m[1] = a.hidden;
        p.src.m[2] = a.grad_hidden;
        const Plan plan = make_plan(&p.src, a.R, a.d, wide_rows(a.grad_x));
        grid = plan.grid;
        cudaError_t e;
        if (plan.ring) {
            e = plan.n == 1   ? backward_types<1>(p, plan, &grid, stream)
                : plan.n == 2 ? backward_types<2>(p, plan, &grid, stream)
                : plan.n == 4 ? backward_types<4>(p, plan, &grid, stream)
                              : backward_types<8>(p, plan, &grid, stream);
        } else {
            (plan.n == 1 ? rms_norm_backward_plain_kernel<1>
                         : rms_norm_backward_plain_kernel<8>)<<<plan.grid, plan.threads, 0, stream>>>(p);
            e = cudaGetLastError();
        }
        if (e != cudaSuccess) return e;
    }
    if (!a.grad_weight) return cudaSuccess;
    // (starts while the rows' kernel ends)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.d + kWeightCols - 1) / kWeightCols), 1, 1);
    cfg.blockDim = dim3(kWeightThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = a.R > 0 ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_weight_kernel, (const float *)p.parts, p.part_ld, (int)grid, a.d, a.grad_weight,
                              a.weight_dtype);
}

}  // namespace dg
