// Losses on rows of full-vocabulary logits, with their gradients: token log-probabilities, the
// clipped policy loss with a KL term, the preference loss's rows, and distillation from a
// teacher's top logits.  Formulas and contracts are in include/dgsamp.h.
//
// With z = x / T, m = max x, s = sum exp((x - m) / T):  lse = m / T + ln s,
// p_v = exp((x_v - m) / T) / s.  One CTA per row; the row passes through shared memory in
// chunks, once for the statistics and once more for the gradient.
#include "row_loss.cuh"

#include "dg_internal.h"
#include "vocab_row.cuh"

namespace dg {

namespace {

using namespace vocab;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 4096;
// Below this ln p_0 the bucket's probability is no normal fp32 number and its term is left out.
constexpr float kTailFloor = -87.0f;

struct Shared {
    float chunk[kChunk];
    float xk[kMaxTopK];  // the student's logits at the teacher's entries
    MaxSum warp_state[kWarps];
    float warp_red[3][kWarps];
    float token_x;
};

__device__ __forceinline__ float block_sum(float v, float *slots) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = 0.0f;
    for (int i = 0; i < kWarps; ++i) r += slots[i];
    return r;
}

__device__ __forceinline__ MaxSum block_merge(MaxSum st, MaxSum *slots, float c) {
    st = warp_merge(st, c);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = st;
    __syncthreads();
    MaxSum r = slots[0];
    for (int i = 1; i < kWarps; ++i) merge(r, slots[i], c);
    return r;
}

// The teacher's distribution over its K entries: q_k = exp((t_k - off) / T) * scale.
struct Teacher {
    float off, log_scale;  // ln q_k = (t_k - off) / T + log_scale
    float mass, rest;      // sum of q over the entries, and the tail's q_0
};

template <typename T, int HEAD, int PASS>
__global__ void __launch_bounds__(kThreads) row_loss_kernel(RowLossArgs a) {
    __shared__ Shared sh;
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.logits) + row * a.ldl;
    T *g = static_cast<T *>(a.grad) + row * a.ldg;
    const int tid = threadIdx.x;
    const float c = kLog2e / a.T;
    const float w = a.weight ? a.weight[row] : 1.0f;
    const int64_t V = a.V;

    int tok = 0;
    float coef = 0.0f;
    bool live = w != 0.0f;
    if (HEAD == kHeadToken) {
        tok = a.token[row];
        if (tok >= V) {
            if (tid == 0) atomicOr(&g_device_error, kErrorIndexRange);
            tok = -1;
        }
        live = live && tok >= 0;
        if (PASS == kPassBackward && live) {
            coef = a.dlogp[row] * w / a.T;
            live = coef != 0.0f;
        }
    }
    if (!live) {
        if (PASS & kPassForward) {
            if (tid == 0) {
                if (a.loss) a.loss[row] = 0.0f;
                if (a.lse) a.lse[row] = 0.0f;
                if (a.logp) a.logp[row] = 0.0f;
                if (a.kl) a.kl[row] = 0.0f;
                if (a.clipped) a.clipped[row] = 0;
                if (a.dlogp) a.dlogp[row] = 0.0f;
                if (a.tail_logp) a.tail_logp[row] = 0.0f;
            }
        }
        if (PASS & kPassBackward)
            for (int64_t v = tid; v < V; v += kThreads) g[v] = from_f32<T>(0.0f);
        return;
    }

    // ---- the teacher's entries
    const int32_t *idx = HEAD == kHeadDistill ? a.indices + row * a.ldk : nullptr;
    const float *t = HEAD == kHeadDistill ? a.teacher + row * a.ldk : nullptr;
    Teacher te{};
    if (HEAD == kHeadDistill) {
        if (a.teacher_lse) {
            te.off = 0.0f;
            te.log_scale = -a.teacher_lse[row];
        } else {
            MaxSum ts{-INFINITY, 0.0f};
            for (int k = tid; k < a.K; k += kThreads)
                if (idx[k] >= 0 && idx[k] < V) {
                    const float one[1] = {t[k]};
                    fold(ts, one, c);
                }
            ts = block_merge(ts, sh.warp_state, c);
            te.off = finite_max(ts.m);
            te.log_scale = ts.s > 0.0f ? -logf(ts.s) : -INFINITY;  // no mass: every q is 0
        }
        float qs = 0.0f;
        for (int k = tid; k < a.K; k += kThreads) {
            if (idx[k] >= V) atomicOr(&g_device_error, kErrorIndexRange);
            if (idx[k] >= 0 && idx[k] < V) qs += expf((t[k] - te.off) / a.T + te.log_scale);
        }
        te.mass = block_sum(qs, sh.warp_red[0]);
        te.rest = a.teacher_lse ? fmaxf(0.0f, 1.0f - te.mass) : 0.0f;
    }

    // ---- statistics
    float m = 0.0f, inv_s = 0.0f, lse, logp0 = 0.0f;
    if (PASS & kPassForward) {
        MaxSum st{-INFINITY, 0.0f};
        for (int64_t v0 = 0; v0 < V; v0 += kChunk) {
            const int n = (int)min((int64_t)kChunk, V - v0);
            for (int i = tid; i < n; i += kThreads) sh.chunk[i] = to_f32(x[v0 + i]);
            __syncthreads();
            if (HEAD == kHeadToken) {
                if (tid == 0 && tok >= v0 && tok < v0 + n) sh.token_x = sh.chunk[tok - v0];
            } else {
                // the teacher's entries leave the chunk: what is folded is the tail
                for (int k = tid; k < a.K; k += kThreads)
                    if (idx[k] >= v0 && idx[k] < v0 + n) {
                        sh.xk[k] = sh.chunk[idx[k] - v0];
                        sh.chunk[idx[k] - v0] = -INFINITY;
                    }
                __syncthreads();
            }
            for (int i = tid; i < n; i += kThreads) {
                const float one[1] = {sh.chunk[i]};
                fold(st, one, c);
            }
            __syncthreads();
        }
        st = block_merge(st, sh.warp_state, c);
        const MaxSum tail = st;
        if (HEAD == kHeadDistill) {
            MaxSum top{-INFINITY, 0.0f};
            for (int k = tid; k < a.K; k += kThreads)
                if (idx[k] >= 0 && idx[k] < V) {
                    const float one[1] = {sh.xk[k]};
                    fold(top, one, c);
                }
            top = block_merge(top, sh.warp_state, c);
            merge(st, top, c);
        }
        m = st.m;
        inv_s = 1.0f / st.s;
        const float lns = logf(st.s);
        lse = m == -INFINITY ? __int_as_float(0x7fc00000) : m / a.T + lns;
        if (tid == 0 && a.lse) a.lse[row] = lse;

        if (HEAD == kHeadToken) {
            __syncthreads();
            const float logp = (sh.token_x - m) / a.T - lns;
            float dlogp = 0.0f;
            if (a.policy) {
                const float A = a.advantage[row];
                const float ratio = expf(logp - a.old_logp[row]);
                const float raw = ratio * A;
                const float cut = fminf(fmaxf(ratio, 1.0f - a.clip_low), 1.0f + a.clip_high) * A;
                const bool clipped = raw > cut;
                float loss = -(clipped ? cut : raw), kl = 0.0f;
                dlogp = clipped ? 0.0f : -raw;
                if (a.ref_logp) {
                    const float d = a.ref_logp[row] - logp;
                    const float e = expm1f(d);
                    kl = e - d;
                    loss = fmaf(a.kl_coef, kl, loss);
                    dlogp = fmaf(-a.kl_coef, e, dlogp);
                }
                if (tid == 0) {
                    if (a.loss) a.loss[row] = loss;
                    if (a.kl) a.kl[row] = kl;
                    if (a.clipped) a.clipped[row] = clipped;
                }
            }
            if (tid == 0) {
                if (a.logp) a.logp[row] = logp;
                if (a.dlogp) a.dlogp[row] = dlogp;
            }
            coef = dlogp * w / a.T;
        } else {
            float l = 0.0f;
            for (int k = tid; k < a.K; k += kThreads)
                if (idx[k] >= 0 && idx[k] < V) {
                    const float lq = (t[k] - te.off) / a.T + te.log_scale;
                    const float q = expf(lq);
                    if (q > 0.0f) l += q * (lq - ((sh.xk[k] - m) / a.T - lns));
                }
            l = block_sum(l, sh.warp_red[0]);
            if (a.teacher_lse) {
                // near 1 from the ratio of the sums: the logarithms' difference would round it off
                const float part = tail.s * exp_below(tail.m, finite_max(m), c);
                logp0 = part > 1e-3f * st.s ? logf(part / st.s)
                        : tail.s > 0.0f     ? (tail.m - m) / a.T + logf(tail.s) - lns
                                            : -INFINITY;
                if (te.rest > 0.0f && logp0 > kTailFloor) l += te.rest * (logf(te.rest) - logp0);
                if (tid == 0 && a.tail_logp) a.tail_logp[row] = logp0;
            }
            if (tid == 0 && a.loss) a.loss[row] = a.T * a.T * l;
        }
    } else {
        lse = a.lse[row];
        if (HEAD == kHeadDistill) {
            if (a.teacher_lse) logp0 = a.tail_logp[row];
            for (int k = tid; k < a.K; k += kThreads)
                if (idx[k] >= 0 && idx[k] < V) sh.xk[k] = to_f32(x[idx[k]]);
            __syncthreads();
        }
    }
    if (!(PASS & kPassBackward)) return;

    // ---- gradient
    const float f = finite_max(m);
    float mass = 0.0f, tail_factor = 0.0f;
    if (HEAD == kHeadDistill) {
        coef = w * a.T;
        mass = te.mass;
        tail_factor = te.mass;
        if (a.teacher_lse && logp0 > kTailFloor) {
            mass += te.rest;
            tail_factor = mass - te.rest * expf(-logp0);
        }
    }
    auto prob = [&](float v) {
        return (PASS & kPassForward) ? exp_below(v, f, c) * inv_s : ex2_approx((v / a.T - lse) * kLog2e);
    };
    for (int64_t v = tid; v < V; v += kThreads) {
        const float p = prob(to_f32(x[v]));
        float d;
        if (HEAD == kHeadToken)
            d = coef * ((v == tok ? 1.0f : 0.0f) - p);
        else
            d = coef * (p * tail_factor);
        g[v] = from_f32<T>(d);
    }
    if (HEAD == kHeadDistill) {
        __syncthreads();
        for (int k = tid; k < a.K; k += kThreads)
            if (idx[k] >= 0 && idx[k] < V) {
                const float q = expf((t[k] - te.off) / a.T + te.log_scale);
                g[idx[k]] = from_f32<T>(coef * (mass * prob(sh.xk[k]) - q));
            }
    }
}

template <typename T, int HEAD>
void launch_pass(const RowLossArgs &a, RowLossPass pass, cudaStream_t stream) {
    const unsigned blocks = (unsigned)a.R;
    switch (pass) {
        case kPassForward: row_loss_kernel<T, HEAD, kPassForward><<<blocks, kThreads, 0, stream>>>(a); break;
        case kPassBackward: row_loss_kernel<T, HEAD, kPassBackward><<<blocks, kThreads, 0, stream>>>(a); break;
        default: row_loss_kernel<T, HEAD, kPassStep><<<blocks, kThreads, 0, stream>>>(a); break;
    }
}

// One CTA per pair: each sequence's sum of weighted log ratios (fp64, so that a long sequence's
// sum does not lose what the pair's difference is made of), the pair's loss, and the derivative of
// every row's log-probability.
__global__ void __launch_bounds__(kThreads) pair_loss_kernel(PairLossArgs a) {
    __shared__ double slots[kWarps];
    __shared__ double seq_sum[2];
    const int pair = blockIdx.x, tid = threadIdx.x;
    int64_t begin[2], end[2];
    for (int j = 0; j < 2; ++j) {
        begin[j] = min(max((int64_t)a.seq_start[2 * pair + j], (int64_t)0), a.R);
        end[j] = min(max((int64_t)a.seq_start[2 * pair + j + 1], begin[j]), a.R);
        double v = 0.0;
        for (int64_t r = begin[j] + tid; r < end[j]; r += kThreads) {
            const float w = a.weight ? a.weight[r] : 1.0f;
            if (w != 0.0f && a.token[r] >= 0)
                v += (double)w * ((double)a.logp[r] - (a.ref_logp ? (double)a.ref_logp[r] : 0.0));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if ((tid & 31) == 0) slots[tid >> 5] = v;
        __syncthreads();
        if (tid == 0) {
            double s = 0.0;
            for (int i = 0; i < kWarps; ++i) s += slots[i];
            seq_sum[j] = s;
        }
        __syncthreads();
    }
    const float z = (float)(a.beta * (seq_sum[0] - seq_sum[1]));
    // -ln sigmoid(z) = max(-z, 0) + ln(1 + exp(-|z|)); sigmoid from the same exponential
    const float e = expf(-fabsf(z)), soft = log1pf(e);
    const float up = fmaxf(-z, 0.0f) + soft, down = fmaxf(z, 0.0f) + soft;
    const float sig = (z >= 0.0f ? 1.0f : e) / (1.0f + e), sig_neg = (z >= 0.0f ? e : 1.0f) / (1.0f + e);
    const float dz = a.label_smoothing * sig - (1.0f - a.label_smoothing) * sig_neg;
    const float pw = a.pair_weight ? a.pair_weight[pair] : 1.0f;
    if (tid == 0) {
        a.loss[pair] = (1.0f - a.label_smoothing) * up + a.label_smoothing * down;
        if (a.log_ratio) {
            a.log_ratio[2 * pair] = (float)seq_sum[0];
            a.log_ratio[2 * pair + 1] = (float)seq_sum[1];
        }
    }
    for (int j = 0; j < 2; ++j) {
        const float d = pw == 0.0f ? 0.0f : (j == 0 ? a.beta : -a.beta) * dz * pw;
        for (int64_t r = begin[j] + tid; r < end[j]; r += kThreads) {
            const float w = a.weight ? a.weight[r] : 1.0f;
            a.dlogp[r] = (w != 0.0f && a.token[r] >= 0) ? d * w : 0.0f;
        }
    }
}

}  // namespace

cudaError_t launch_row_loss(const RowLossArgs &a, RowLossHead head, RowLossPass pass, cudaStream_t stream) {
    if (a.dtype == DG_BF16) {
        if (head == kHeadToken)
            launch_pass<__nv_bfloat16, kHeadToken>(a, pass, stream);
        else
            launch_pass<__nv_bfloat16, kHeadDistill>(a, pass, stream);
    } else {
        if (head == kHeadToken)
            launch_pass<float, kHeadToken>(a, pass, stream);
        else
            launch_pass<float, kHeadDistill>(a, pass, stream);
    }
    return cudaGetLastError();
}

cudaError_t launch_pair_loss(const PairLossArgs &a, cudaStream_t stream) {
    pair_loss_kernel<<<(unsigned)a.P, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace dg
