// The K largest logits of every row, in order, ties to the lowest index, and the tempered
// log-sum-exp.  Contract in include/dgsamp.h.
//
// One CTA per row: a radix selection over the entries' order-preserving integer keys (four
// passes of 8 bits over the row) finds the K-th largest value, a last pass collects what lies
// above it and the first entries equal to it, and a bitonic network orders the K.
#include "dg_internal.h"
#include "row_loss.cuh"
#include "vocab_row.cuh"

namespace dg {

namespace {

using namespace vocab;

constexpr int kThreads = 512;

// Larger floats have larger keys; -0 and +0 the same one.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) row_topk_kernel(RowTopKArgs a) {
    __shared__ uint32_t hist[256];
    __shared__ uint64_t best[kMaxTopK];
    __shared__ MaxSum warp_state[kThreads / 32];
    __shared__ uint32_t s_prefix, s_need, s_above, s_equal[kThreads];
    __shared__ uint32_t s_tied;
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.logits) + row * a.ldl;
    const int tid = threadIdx.x, K = a.K;
    const int64_t V = a.V;
    const float c = kLog2e / a.T;

    if (a.lse) {
        MaxSum st{-INFINITY, 0.0f};
        for (int64_t v = tid; v < V; v += kThreads) {
            const float one[1] = {to_f32(x[v])};
            fold(st, one, c);
        }
        st = warp_merge(st, c);
        if ((tid & 31) == 0) warp_state[tid >> 5] = st;
        __syncthreads();
        if (tid == 0) {
            for (int i = 1; i < kThreads / 32; ++i) merge(st, warp_state[i], c);
            a.lse[row] = st.m == -INFINITY ? __int_as_float(0x7fc00000) : st.m / a.T + logf(st.s);
        }
    }

    uint32_t prefix = 0, need = (uint32_t)K;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int64_t v = tid; v < V; v += kThreads) {
            const uint32_t k = order_key(to_f32(x[v]));
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1u);
        }
        __syncthreads();
        if (tid == 0) {
            int b = 255;
            uint32_t n = need;
            while (b > 0 && hist[b] < n) n -= hist[b--];
            s_prefix = prefix | ((uint32_t)b << shift);
            s_need = n;
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
    }
    // `need` entries equal to the key `prefix` are taken, in index order, and all above it
    if (tid == 0) s_above = s_tied = 0;
    __syncthreads();
    for (int64_t v0 = 0; v0 < V; v0 += kThreads) {
        const int64_t v = v0 + tid;
        const uint32_t k = v < V ? order_key(to_f32(x[v])) : 0u;
        const bool eq = v < V && k == prefix;
        if (v < V && k > prefix) {
            const uint32_t at = atomicAdd(&s_above, 1u);
            if (at < (uint32_t)K) best[at] = ((uint64_t)k << 32) | (0xffffffffu - (uint32_t)v);
        }
        s_equal[tid] = eq;
        const int any = __syncthreads_or(eq);
        if (any) {
            if (eq) {
                uint32_t rank = s_tied;
                for (int i = 0; i < tid; ++i) rank += s_equal[i];
                if (rank < need)
                    best[(uint32_t)K - need + rank] = ((uint64_t)k << 32) | (0xffffffffu - (uint32_t)v);
            }
            __syncthreads();
            if (tid == 0)
                for (int i = 0; i < kThreads; ++i) s_tied += s_equal[i];
        }
        __syncthreads();
    }
    int n2 = 1;
    while (n2 < K) n2 *= 2;
    for (int i = K + tid; i < n2; i += kThreads) best[i] = 0;
    __syncthreads();
    for (int size = 2; size <= n2; size *= 2)
        for (int stride = size / 2; stride > 0; stride /= 2) {
            for (int i = tid; i < n2 / 2; i += kThreads) {
                const int lo = 2 * i - (i & (stride - 1)), hi = lo + stride;
                const bool down = (lo & size) == 0;
                const uint64_t p = best[lo], q = best[hi];
                if ((p < q) == down) {
                    best[lo] = q;
                    best[hi] = p;
                }
            }
            __syncthreads();
        }
    for (int k = tid; k < K; k += kThreads) {
        const uint32_t v = 0xffffffffu - (uint32_t)best[k];
        a.values[row * a.ldk + k] = to_f32(x[v]);
        a.indices[row * a.ldk + k] = (int32_t)v;
    }
}

}  // namespace

size_t row_topk_workspace_bytes(int64_t, int64_t, int, int) { return 16; }

cudaError_t launch_row_topk(const RowTopKArgs &a, void *, cudaStream_t stream) {
    if (a.dtype == DG_BF16)
        row_topk_kernel<__nv_bfloat16><<<(unsigned)a.R, kThreads, 0, stream>>>(a);
    else
        row_topk_kernel<float><<<(unsigned)a.R, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace dg
