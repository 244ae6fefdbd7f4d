// Device helpers of the kernels that read rows of logits in fp32 or bf16 (row_loss.cu,
// row_topk.cu).
#pragma once

#include <cuda_bf16.h>
#include <float.h>

#include "dg_common.cuh"
#include "row_loss.cuh"

namespace dg {
namespace vocab {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
    return __bfloat162float(v);
}
// One rounding (to nearest even) where the storage type is bf16.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// Bits of the device error word beside the timeout's.
constexpr unsigned int kErrorIndexRange = 2u;

// Running maximum and sum of exponentials of a softmax: s = sum of exp((x - m) / T).
struct MaxSum {
    float m, s;
};

// The maximum as a subtrahend: finite also while nothing but -inf has been seen, so that
// -inf entries give exp(-inf) = 0 instead of NaN.
__device__ __forceinline__ float finite_max(float m) { return fmaxf(m, -FLT_MAX); }

// exp((x - m) / T) with c = log2(e) / T.  The difference is taken first: x c - m c would lose
// the entries next to the maximum to rounding, and overflow where both are the type's lowest.
__device__ __forceinline__ float exp_below(float x, float m, float c) { return ex2_approx((x - m) * c); }

// With log2(e) / T as two floats (row_loss.cuh); what follows takes either.
__device__ __forceinline__ float exp_below(float x, float m, const Scale &c) {
    const float d = x - m;
    return ex2_approx(fmaf(d, c.hi, d * c.lo));
}

template <typename C>
__device__ __forceinline__ void merge(MaxSum &a, const MaxSum &b, const C &c) {
    const float m = fmaxf(a.m, b.m);
    const float f = finite_max(m);
    a.s = a.s * exp_below(a.m, f, c) + b.s * exp_below(b.m, f, c);
    a.m = m;
}

// Two floats in one register pair, for the instructions that work on both (sm_100 family).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(f32x2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// exp_below of both: the same roundings, with minus_m = (-m, -m), and cc = (c, c) or hi and lo pairs.
__device__ __forceinline__ f32x2 exp_below2(f32x2 x, f32x2 minus_m, f32x2 hi, f32x2 lo) {
    const f32x2 d = add2(x, minus_m);
    float a, b;
    unpair(fma2(d, hi, mul2(d, lo)), a, b);
    return pair(ex2_approx(a), ex2_approx(b));
}
__device__ __forceinline__ f32x2 exp_below2(f32x2 x, f32x2 minus_m, f32x2 cc) {
    float lo, hi;
    unpair(mul2(add2(x, minus_m), cc), lo, hi);
    return pair(ex2_approx(lo), ex2_approx(hi));
}

__device__ __forceinline__ f32x2 exp_below2(f32x2 x, f32x2 minus_m, float c) {
    return exp_below2(x, minus_m, pair(c, c));
}
__device__ __forceinline__ f32x2 exp_below2(f32x2 x, f32x2 minus_m, const Scale &c) {
    return exp_below2(x, minus_m, pair(c.hi, c.hi), pair(c.lo, c.lo));
}

// The largest of N values, and their sum, as trees: chains of N dependent operations would leave a
// warp waiting for most of its time.
template <int N>
__device__ __forceinline__ float tree_max(const float *x) {
    if constexpr (N == 1) return x[0];
    if constexpr (N == 2) return fmaxf(x[0], x[1]);
    if constexpr (N >= 3) {
        constexpr int A = N / 3, B = (N - A) / 2;
        return max3f(tree_max<A>(x), tree_max<B>(x + A), tree_max<N - A - B>(x + A + B));
    }
}
template <int N>
__device__ __forceinline__ float tree_sum(const float *x) {
    if constexpr (N == 1) return x[0];
    if constexpr (N >= 2) return tree_sum<N / 2>(x) + tree_sum<N - N / 2>(x + N / 2);
}

// Folds N values into the state.
template <int N, typename C>
__device__ __forceinline__ void fold(MaxSum &st, const float (&x)[N], const C &c) {
    const float bm = tree_max<N>(x);
    if (bm > st.m) {
        st.s *= exp_below(st.m, bm, c);
        st.m = bm;
    }
    const float f = finite_max(st.m);
    float e[N];
#pragma unroll
    for (int j = 0; j < N; ++j) e[j] = exp_below(x[j], f, c);
    st.s += tree_sum<N>(e);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// The 32 lanes' states as one, the same in every lane: the maximum first, so that each sum is
// rescaled once.
template <typename C>
__device__ __forceinline__ MaxSum warp_merge(MaxSum st, const C &c) {
    const float m = warp_max(st.m);
    return MaxSum{m, warp_sum(st.s * exp_below(st.m, finite_max(m), c))};
}

// A 16-byte vector of the row: its entries as pairs of floats, their maximum over several vectors,
// and the way back.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kLow = 0xff800000u;  // -inf
    __device__ static __forceinline__ void pairs(const uint4 &v, f32x2 *p) {
        p[0] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
        p[1] = pair(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    __device__ static __forceinline__ uint4 pack(const f32x2 *p) {
        float a, b, c, d;
        unpair(p[0], a, b);
        unpair(p[1], c, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
    }
    template <int K>
    __device__ static __forceinline__ float largest(const uint4 (&v)[K]) {
        float f[4 * K];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            f[4 * i] = __uint_as_float(v[i].x);
            f[4 * i + 1] = __uint_as_float(v[i].y);
            f[4 * i + 2] = __uint_as_float(v[i].z);
            f[4 * i + 3] = __uint_as_float(v[i].w);
        }
        return tree_max<4 * K>(f);
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static constexpr uint32_t kLow = 0xff80ff80u;
    __device__ static __forceinline__ f32x2 widen(uint32_t w) {
        return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    __device__ static __forceinline__ void pairs(const uint4 &v, f32x2 *p) {
        p[0] = widen(v.x);
        p[1] = widen(v.y);
        p[2] = widen(v.z);
        p[3] = widen(v.w);
    }
    __device__ static __forceinline__ uint32_t narrow(f32x2 v) {
        float lo, hi;
        unpair(v, lo, hi);
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    __device__ static __forceinline__ uint4 pack(const f32x2 *p) {
        return make_uint4(narrow(p[0]), narrow(p[1]), narrow(p[2]), narrow(p[3]));
    }
    __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    // in bf16, two at a time: a maximum rounds nothing
    template <int K>
    __device__ static __forceinline__ float largest(const uint4 (&v)[K]) {
        uint32_t m[K];
#pragma unroll
        for (int i = 0; i < K; ++i) m[i] = max2(max2(v[i].x, v[i].y), max2(v[i].z, v[i].w));
#pragma unroll
        for (int d = 1; d < K; d *= 2)
#pragma unroll
            for (int i = 0; i + d < K; i += 2 * d) m[i] = max2(m[i], m[i + d]);
        return fmaxf(__uint_as_float(m[0] << 16), __uint_as_float(m[0] & 0xffff0000u));
    }
};

// Folds K vectors into the state.
template <typename T, int K, typename C>
__device__ __forceinline__ void fold_vecs(MaxSum &st, const uint4 (&v)[K], const C &c) {
    const float bm = Vec<T>::largest(v);
    if (bm > st.m) {
        st.s *= exp_below(st.m, bm, c);
        st.m = bm;
    }
    const float f = -finite_max(st.m);
    const f32x2 minus_m = pair(f, f);
    constexpr int P = Vec<T>::N / 2;
    f32x2 sum[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < K; ++i) {
        f32x2 p[P];
        Vec<T>::pairs(v[i], p);
#pragma unroll
        for (int j = 0; j < P; ++j) sum[j & 1] = add2(sum[j & 1], exp_below2(p[j], minus_m, c));
    }
    float a, b;
    unpair(add2(sum[0], sum[1]), a, b);
    st.s += a + b;
}

// ------------------------------------------------------------------ rings

// Global -> shared bulk copy of `bytes` (a multiple of 16, both addresses 16-byte aligned),
// completing on the barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar,
                                          uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], "
        "%4;" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(policy)
        : "memory");
}

// mbar_wait in few instructions (kernels whose warps run different code wait in many places, and are
// slowed by what does not fit the instruction cache): gives up after kWaitLimitNs, or at once where
// another wait of the CTA has given up.
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            record_timeout();
            return false;
        }
    }
    return true;
}
// Whether the phase is over, without a wait.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// e^x by the hardware's power of two: relative error (|x| + 4) 2^-23 or so.
__device__ __forceinline__ float exp_fast(float x) { return ex2_approx(x * kLog2e); }

}  // namespace vocab
}  // namespace dg
