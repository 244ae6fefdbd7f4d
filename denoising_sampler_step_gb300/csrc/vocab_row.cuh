// Device helpers of the kernels that read rows of logits in fp32 or bf16 (row_loss.cu,
// row_topk.cu).
#pragma once

#include <cuda_bf16.h>
#include <float.h>

#include "dg_common.cuh"

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

__device__ __forceinline__ void merge(MaxSum &a, const MaxSum &b, float c) {
    const float m = fmaxf(a.m, b.m);
    const float f = finite_max(m);
    a.s = a.s * exp_below(a.m, f, c) + b.s * exp_below(b.m, f, c);
    a.m = m;
}

template <int N>
__device__ __forceinline__ void fold(MaxSum &st, const float (&x)[N], float c) {
    float bm = x[0];
#pragma unroll
    for (int j = 1; j < N; ++j) bm = fmaxf(bm, x[j]);
    if (bm > st.m) {
        st.s *= exp_below(st.m, bm, c);
        st.m = bm;
    }
    const float f = finite_max(st.m);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) sum += exp_below(x[j], f, c);
    st.s += sum;
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
__device__ __forceinline__ MaxSum warp_merge(MaxSum st, float c) {
    const float m = warp_max(st.m);
    return MaxSum{m, warp_sum(st.s * exp_below(st.m, finite_max(m), c))};
}

// ------------------------------------------------------------------ rings and clusters

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

// mbar_wait that returns at once where another wait of the CTA has already given up.
__device__ __forceinline__ bool ring_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    return mbar_wait(bar, parity, abort_flag);
}
__device__ __forceinline__ bool ring_wait_cluster(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if (*abort_flag) return false;
    return mbar_wait_cluster(bar, parity, abort_flag);
}

// Stores to, and an arrival on, shared memory of a CTA of the cluster (shared::cluster addresses);
// the arrival releases the thread's earlier stores to a wait with cluster-scope acquire.
__device__ __forceinline__ void st_cluster_v4(uint32_t dst, float a, float b, float c, float d) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "f"(a), "f"(b), "f"(c), "f"(d)
                 : "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t dst, float a) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(a) : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

}  // namespace vocab
}  // namespace dg
