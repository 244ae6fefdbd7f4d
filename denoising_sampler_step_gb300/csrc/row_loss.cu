// Losses on rows of full-vocabulary logits, with their gradients: token log-probabilities, the
// clipped policy loss with a KL term, the preference loss's rows, and distillation from a
// teacher's top logits.  Formulas and contracts are in include/dgsamp.h.
//
// With z = x / T, m = max x, s = sum exp((x - m) / T):  lse = m / T + ln s,
// p_v = exp((x_v - m) / T) / s.
//
// HBM-bound: a loss reads each logit once, a gradient reads it once and writes it once, at some
// ten flops per entry.  The statistics must be complete before the first gradient entry can be
// written, so a row that is not kept on the chip is read twice.  Here a cluster of C CTAs takes a
// row, each CTA one slice of it, and a slice stays in shared memory between the two passes:
//   - a loader thread streams the slice into a ring of shared-memory stages with bulk copies
//     (cp.async.bulk, an mbarrier per stage);
//   - the folding threads take each stage's running maximum and sum as it arrives, and leave it
//     where it is;
//   - the slices' (m, s) go to every CTA of the cluster through distributed shared memory;
//   - the folding threads turn the stages into gradients, write those from registers, and hand the
//     stages back; the loader has meanwhile filled the ring's other stages with the next row.
// The clusters are persistent: cluster i takes rows i, i + n, ...  Rows too long for the ring
// pass through it twice (the second time mostly from L2).
#include <atomic>

#include "dg_internal.h"
#include "row_loss.cuh"
#include "vocab_row.cuh"

namespace dg {

namespace {

using namespace vocab;

constexpr int kMaxStages = 16;
constexpr int kMaxCluster = 8;
// Below this ln p_0 the bucket's probability is no normal fp32 number and its term is left out.
constexpr float kTailFloor = -87.0f;

struct Plan {
    int cluster;   // CTAs per row
    int stages;    // of the ring
    bool resident;  // a slice fits the ring: it is read once
};

// A slice's part of the row's statistics, posted to every CTA of the cluster.
struct __align__(16) Post {
    MaxSum rest;  // every entry (tokens), or those outside the teacher's (distillation)
    MaxSum top;   // the teacher's entries; for tokens top.m is the token's logit (-inf elsewhere)
};

template <int NT>
struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t posted[2], summed[2];
    Post post[2][kMaxCluster];
    float part_loss[2][kMaxCluster];
    Post warp_post[2][NT / 32];       // by row parity: a fast warp may be one row ahead
    MaxSum warp_teacher[2][NT / 32];
    float warp_loss[NT / 32];
    float tail[8];  // the row's last V % (16 / sizeof(T)) entries
    int abort_flag;
};

// One 16-byte vector of the row as floats, and back.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void unpack(const uint4 &v, float *x) {
        x[0] = __uint_as_float(v.x);
        x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z);
        x[3] = __uint_as_float(v.w);
    }
    __device__ static __forceinline__ uint4 pack(const float *x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
    static constexpr uint32_t kLow = 0xff800000u;  // -inf
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void unpack(const uint4 &v, float *x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static __forceinline__ uint32_t pack2(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    __device__ static __forceinline__ uint4 pack(const float *x) {
        return make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
    }
    static constexpr uint32_t kLow = 0xff80ff80u;
};

__device__ __forceinline__ void cluster_arrive_wait() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// The live rows of the call, decided alike by the loader and the folding threads.
template <int HEAD, int PASS>
struct RowScalars {
    float w;     // weight; backward over tokens: the coefficient weight * dlogp
    int tok;
    bool live;
    float lse, logp0;     // backward
    float A, old, ref;    // the policy loss

    __device__ __forceinline__ void load(const RowLossArgs &a, int64_t row) {
        w = a.weight ? a.weight[row] : 1.0f;
        tok = 0;
        if (HEAD == kHeadToken) {
            tok = a.token[row];
            if (PASS == kPassBackward && w != 0.0f) w *= a.dlogp[row];
        }
        if (PASS == kPassBackward) {
            lse = a.lse[row];
            logp0 = HEAD == kHeadDistill && a.teacher_lse ? a.tail_logp[row] : 0.0f;
        } else if (HEAD == kHeadToken && a.policy) {
            A = a.advantage[row];
            old = a.old_logp[row];
            ref = a.ref_logp ? a.ref_logp[row] : 0.0f;
        }
    }
    __device__ __forceinline__ void decide(int64_t V) {
        live = w != 0.0f;
        if (HEAD == kHeadToken) live = live && tok >= 0 && tok < V;
    }
};

template <typename T, int HEAD, int PASS, int NT, int VPT>
__global__ void __launch_bounds__(NT + 32, NT == 512 ? 1 : 512 / NT)
    row_loss_kernel(const RowLossArgs a, const Plan plan) {
    constexpr bool kForward = (PASS & kPassForward) != 0, kBackward = (PASS & kPassBackward) != 0;
    constexpr int N = Vec<T>::N;
    constexpr int kStageVecs = NT * VPT;             // 16-byte vectors of a stage
    constexpr int kStageElems = kStageVecs * N;
    constexpr int kWarps = NT / 32;
    constexpr int KPT = HEAD == kHeadDistill ? kMaxTopK / NT : 1;  // teacher's entries per thread
    extern __shared__ __align__(128) uint4 ring[];
    __shared__ Shared<NT> sh;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = plan.cluster, NS = plan.stages;
    const int rank = C > 1 ? (int)cluster_ctarank() : 0;
    const int64_t first = blockIdx.x / C, step = gridDim.x / C;
    const int64_t V = a.V, nv = V / N;
    // whole 128-byte lines per slice; the last CTA also has the entries after the last vector
    const int64_t per = ((nv + C - 1) / C + 7) / 8 * 8;
    const int64_t v_begin = min(nv, rank * per);
    const int len = (int)(min(nv, v_begin + per) - v_begin);
    const int chunks = (len + kStageVecs - 1) / kStageVecs;
    const int ntail = rank == C - 1 ? (int)(V - nv * N) : 0;
    const int loads = chunks * (kForward && kBackward && !plan.resident ? 2 : 1);

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.posted[i]), C);
            mbar_init(smem_u32(&sh.summed[i]), C);
        }
        sh.abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (C > 1) cluster_arrive_wait();  // the peers' barriers are ready

    if (warp == kWarps) {
        // ------------------------------------------------------------ loader
        if (lane == 0) {
            const uint64_t policy = l2_policy_evict_first();
            const uint64_t keep = l2_policy_evict_normal();
            int slot = 0;
            uint32_t use = 0;  // times the ring has been around
            bool ok = true;
            RowScalars<HEAD, PASS> next;
            if (first < a.R) next.load(a, first);
            for (int64_t row = first; row < a.R && ok; row += step) {
                RowScalars<HEAD, PASS> now = next;
                if (row + step < a.R) next.load(a, row + step);
                now.decide(V);
                if (!now.live) continue;
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.logits) + row * a.ldl) +
                                   v_begin;
                for (int i = 0; i < loads && ok; ++i) {
                    const int c = i < chunks ? i : i - chunks;
                    if (use > 0) ok = ring_wait(smem_u32(&sh.empty[slot]), (use - 1) & 1, &sh.abort_flag);
                    if (!ok) break;
                    const uint32_t bytes = (uint32_t)min(kStageVecs, len - c * kStageVecs) * 16u;
                    const uint32_t bar = smem_u32(&sh.full[slot]);
                    mbar_arrive_expect_tx(bar, bytes);
                    bulk_load(smem_u32(ring + slot * kStageVecs), src + (int64_t)c * kStageVecs, bytes, bar,
                              i + chunks < loads ? keep : policy);
                    if (++slot == NS) {
                        slot = 0;
                        ++use;
                    }
                }
            }
            // a CTA that gave up leaves only after its copies in flight have landed
            if (!ok)
                for (int i = 0; i < NS; ++i) {
                    const uint32_t issued = use + (i < slot ? 1 : 0);
                    if (issued > 0) drain_wait(smem_u32(&sh.full[i]), (issued - 1) & 1);
                }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ folding threads
        // A wait that gives up (a second without the bytes it waits for) raises the abort flag and
        // the device error word; the threads then run through their rows without waiting.
        const float c = kLog2e / a.T;
        int slot = 0;
        uint32_t phase = 0;
        uint32_t nlive = 0;
        auto full_wait = [&](int s, uint32_t ph) { ring_wait(smem_u32(&sh.full[s]), ph, &sh.abort_flag); };
        auto release = [&](int s) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.empty[s]));
        };
        auto sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory"); };

        RowScalars<HEAD, PASS> next;
        if (first < a.R) next.load(a, first);
        for (int64_t row = first; row < a.R; row += step) {
            RowScalars<HEAD, PASS> now = next;
            if (row + step < a.R) next.load(a, row + step);
            now.decide(V);
            T *g = static_cast<T *>(a.grad) + row * a.ldg;
            uint4 *gv = reinterpret_cast<uint4 *>(g) + v_begin;
            const T *x = static_cast<const T *>(a.logits) + row * a.ldl;
            if (!now.live) {
                if (rank == 0 && tid == 0) {
                    if (HEAD == kHeadToken && now.w != 0.0f && now.tok >= V)
                        atomicOr(&g_device_error, kErrorIndexRange);
                    if (kForward) {
                        if (a.loss) a.loss[row] = 0.0f;
                        if (a.lse) a.lse[row] = 0.0f;
                        if (a.logp) a.logp[row] = 0.0f;
                        if (a.kl) a.kl[row] = 0.0f;
                        if (a.clipped) a.clipped[row] = 0;
                        if (a.dlogp) a.dlogp[row] = 0.0f;
                        if (a.tail_logp) a.tail_logp[row] = 0.0f;
                    }
                }
                if (kBackward) {
                    for (int i = tid; i < len; i += NT) gv[i] = make_uint4(0, 0, 0, 0);
                    if (tid < ntail) g[nv * N + tid] = from_f32<T>(0.0f);
                }
                continue;
            }
            const int par = nlive & 1;
            const uint32_t post_phase = (nlive >> 1) & 1;
            ++nlive;

            // the teacher's entries this thread holds: k = tid + j NT
            float tk[KPT], xk[KPT];
            int at[KPT];           // place in the slice (elements), -1: another CTA's, -2: none
            MaxSum teacher{-INFINITY, 0.0f};
            float tlse = 0.0f;
            if (HEAD == kHeadDistill) {
                const int32_t *idx = a.indices + row * a.ldk;
                const float *t = a.teacher + row * a.ldk;
                tlse = a.teacher_lse ? a.teacher_lse[row] : 0.0f;
#pragma unroll
                for (int j = 0; j < KPT; ++j) {
                    const int k = tid + j * NT;
                    at[j] = -2;
                    xk[j] = -INFINITY;
                    tk[j] = -INFINITY;
                    if (k < a.K) {
                        const int v = idx[k];
                        if (v >= V) atomicOr(&g_device_error, kErrorIndexRange);
                        if (v >= 0 && v < V) {
                            const int64_t off = v - v_begin * N;
                            at[j] = off >= 0 && off < (int64_t)len * N + ntail ? (int)off : -1;
                            tk[j] = t[k];
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < KPT; ++j)
                    if (at[j] != -2) {
                        const float one[1] = {tk[j]};
                        fold(teacher, one, c);
                    }
            }
            auto log_q = [&](int j, float off, float log_scale) { return (tk[j] - off) / a.T + log_scale; };

            float m = 0.0f, inv_s = 0.0f, lns = 0.0f, logp0 = 0.0f, coef = 0.0f;
            float off = 0.0f, log_scale = 0.0f, mass = 0.0f, q_rest = 0.0f;
            const int slot0 = slot;
            const uint32_t phase0 = phase;

            // ---------------------------------------------------------------- statistics
            if (kForward) {
                MaxSum st{-INFINITY, 0.0f}, top{-INFINITY, 0.0f};
                if (ntail > 0) {
                    if (HEAD == kHeadToken) {
                        if (tid < ntail) {
                            const float one[1] = {to_f32(x[nv * N + tid])};
                            fold(st, one, c);
                        }
                    } else {
                        if (tid < ntail) sh.tail[tid] = to_f32(x[nv * N + tid]);
                        sync();
#pragma unroll
                        for (int j = 0; j < KPT; ++j)
                            if (at[j] >= len * N) {
                                xk[j] = sh.tail[at[j] - len * N];
                                sh.tail[at[j] - len * N] = -INFINITY;
                            }
                        sync();
                        if (tid < ntail) {
                            const float one[1] = {sh.tail[tid]};
                            fold(st, one, c);
                        }
                    }
                }
                const int64_t tok_at = HEAD == kHeadToken ? now.tok - v_begin * N : -1;
                float x_tok = -INFINITY;
                if (HEAD == kHeadToken && tid == 0 && tok_at >= (int64_t)len * N && tok_at < (int64_t)len * N + ntail)
                    x_tok = to_f32(x[now.tok]);
                for (int ch = 0; ch < chunks; ++ch) {
                    full_wait(slot, phase);
                    uint4 *stage = ring + slot * kStageVecs;
                    const int n = min(kStageVecs, len - ch * kStageVecs);
                    T *elems = reinterpret_cast<T *>(stage);
                    const int e0 = ch * kStageElems;
                    if (HEAD == kHeadToken) {
                        if (tid == 0 && tok_at >= e0 && tok_at < e0 + (int64_t)n * N) x_tok = to_f32(elems[tok_at - e0]);
                    } else {
                        // the teacher's entries leave the stage: what is folded is the bucket
#pragma unroll
                        for (int j = 0; j < KPT; ++j)
                            if (at[j] >= e0 && at[j] < e0 + n * N) {
                                xk[j] = to_f32(elems[at[j] - e0]);
                                elems[at[j] - e0] = from_f32<T>(-INFINITY);
                                fence_proxy_async_smem();  // before the copy that refills the stage
                            }
                        sync();
                    }
                    float f[VPT * N];
#pragma unroll
                    for (int i = 0; i < VPT; ++i) {
                        const int at_v = tid + i * NT;
                        const uint4 v = at_v < n ? stage[at_v]
                                                 : make_uint4(Vec<T>::kLow, Vec<T>::kLow, Vec<T>::kLow, Vec<T>::kLow);
                        Vec<T>::unpack(v, f + i * N);
                    }
                    if (!(kBackward && plan.resident)) release(slot);
                    fold(st, f, c);
                    if (++slot == NS) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (HEAD == kHeadDistill) {
#pragma unroll
                    for (int j = 0; j < KPT; ++j)
                        if (at[j] >= 0) {
                            const float one[1] = {xk[j]};
                            fold(top, one, c);
                        }
                }
                // warp, CTA, cluster: in a fixed order, so that results repeat bit for bit
                st = warp_merge(st, c);
                if (HEAD == kHeadDistill) {
                    top = warp_merge(top, c);
                    teacher = warp_merge(teacher, c);
                } else {
                    top.m = __shfl_sync(0xffffffffu, x_tok, 0);
                }
                if (lane == 0) {
                    sh.warp_post[par][warp] = Post{st, top};
                    if (HEAD == kHeadDistill) sh.warp_teacher[par][warp] = teacher;
                }
                sync();
                const Post none{{-INFINITY, 0.0f}, {-INFINITY, 0.0f}};
                const Post mine = lane < kWarps ? sh.warp_post[par][lane] : none;
                st = warp_merge(mine.rest, c);
                if (HEAD == kHeadDistill) {
                    top = warp_merge(mine.top, c);
                    teacher = warp_merge(lane < kWarps ? sh.warp_teacher[par][lane] : none.rest, c);
                } else {
                    top.m = sh.warp_post[par][0].top.m;  // thread 0 has read it
                }
                if (C > 1) {
                    if (tid < C) {
                        const uint32_t dst = map_to_cta(smem_u32(&sh.post[par][rank]), tid);
                        st_cluster_v4(dst, st.m, st.s, top.m, top.s);
                        mbar_arrive_cluster(map_to_cta(smem_u32(&sh.posted[par]), tid));
                    }
                    ring_wait_cluster(smem_u32(&sh.posted[par]), post_phase, &sh.abort_flag);
                    const Post theirs = lane < C ? sh.post[par][lane] : none;
                    st = warp_merge(theirs.rest, c);
                    if (HEAD == kHeadDistill)
                        top = warp_merge(theirs.top, c);
                    else
                        top.m = warp_max(theirs.top.m);
                }
                const MaxSum rest = st;
                if (HEAD == kHeadDistill) merge(st, top, c);
                m = st.m;
                inv_s = 1.0f / st.s;
                lns = logf(st.s);
                const bool writes = rank == 0 && tid == 0;
                if (writes && a.lse) a.lse[row] = m == -INFINITY ? __int_as_float(0x7fc00000) : m / a.T + lns;
                if (HEAD == kHeadToken) {
                    const float logp = (top.m - m) / a.T - lns;
                    float dlogp = 0.0f;
                    if (a.policy) {
                        const float ratio = expf(logp - now.old);
                        const float raw = ratio * now.A;
                        const float cut = fminf(fmaxf(ratio, 1.0f - a.clip_low), 1.0f + a.clip_high) * now.A;
                        const bool clipped = raw > cut;
                        float loss = -(clipped ? cut : raw), kl = 0.0f;
                        dlogp = clipped ? 0.0f : -raw;
                        if (a.ref_logp) {
                            // e^d - 1 in one function: d is small, and the difference is what counts
                            const float d = now.ref - logp;
                            const float e = expm1f(d);
                            kl = e - d;
                            loss = fmaf(a.kl_coef, kl, loss);
                            dlogp = fmaf(-a.kl_coef, e, dlogp);
                        }
                        if (writes) {
                            if (a.loss) a.loss[row] = loss;
                            if (a.kl) a.kl[row] = kl;
                            if (a.clipped) a.clipped[row] = clipped;
                        }
                    }
                    if (writes) {
                        if (a.logp) a.logp[row] = logp;
                        if (a.dlogp) a.dlogp[row] = dlogp;
                    }
                    coef = dlogp * now.w / a.T;
                } else if (a.teacher_lse) {
                    // near 1 from the ratio of the sums: the logarithms' difference would round it off
                    const float part = rest.s * exp_below(rest.m, finite_max(m), c);
                    logp0 = part > 1e-3f * st.s ? logf(part / st.s)
                            : rest.s > 0.0f     ? (rest.m - m) / a.T + logf(rest.s) - lns
                                                : -INFINITY;
                    if (writes && a.tail_logp) a.tail_logp[row] = logp0;
                }
            } else {
                // p = exp((x - T lse) / T): T lse as m, what its rounding lost as a factor
                m = now.lse * a.T;
                inv_s = expf(-fmaf(now.lse, a.T, -m) / a.T);
                if (HEAD == kHeadToken) {
                    coef = now.w / a.T;
                } else {
                    logp0 = now.logp0;
#pragma unroll
                    for (int j = 0; j < KPT; ++j)
                        if (at[j] >= 0) xk[j] = to_f32(x[v_begin * N + at[j]]);
                    teacher = warp_merge(teacher, c);
                    if (lane == 0) sh.warp_teacher[par][warp] = teacher;
                    sync();  // also: the entries are read before the gradient may replace them
                    teacher = warp_merge(lane < kWarps ? sh.warp_teacher[par][lane] : MaxSum{-INFINITY, 0.0f}, c);
                }
            }

            // ---------------------------------------------------------------- the teacher's terms
            if (HEAD == kHeadDistill) {
                // ln q_k = (t_k - off) / T + log_scale; no mass at all: every q is 0
                if (a.teacher_lse) {
                    log_scale = -tlse;
                    mass = teacher.s > 0.0f ? expf(teacher.m / a.T - tlse) * teacher.s : 0.0f;
                    q_rest = fmaxf(0.0f, 1.0f - mass);
                } else {
                    off = finite_max(teacher.m);
                    log_scale = teacher.s > 0.0f ? -logf(teacher.s) : -INFINITY;
                    mass = teacher.s > 0.0f ? 1.0f : 0.0f;
                }
                if (kForward && a.loss) {
                    float l = 0.0f;
#pragma unroll
                    for (int j = 0; j < KPT; ++j)
                        if (at[j] >= 0) {
                            const float lq = log_q(j, off, log_scale), q = expf(lq);
                            if (q > 0.0f) l += q * (lq - ((xk[j] - m) / a.T - lns));
                        }
                    l = warp_sum(l);
                    if (lane == 0) sh.warp_loss[warp] = l;
                    sync();
                    if (warp == 0) {
                        l = warp_sum(lane < kWarps ? sh.warp_loss[lane] : 0.0f);
                        if (C > 1) {
                            if (lane == 0) {
                                st_cluster_f32(map_to_cta(smem_u32(&sh.part_loss[par][rank]), 0), l);
                                mbar_arrive_cluster(map_to_cta(smem_u32(&sh.summed[par]), 0));
                            }
                            if (rank == 0) {
                                // (the barrier counts C arrivals, all of them on the leader's)
                                ring_wait_cluster(smem_u32(&sh.summed[par]), post_phase, &sh.abort_flag);
                                l = warp_sum(lane < C ? sh.part_loss[par][lane] : 0.0f);
                            }
                        }
                        if (rank == 0 && lane == 0) {
                            if (a.teacher_lse && q_rest > 0.0f && logp0 > kTailFloor)
                                l += q_rest * (logf(q_rest) - logp0);
                            a.loss[row] = a.T * a.T * l;
                        }
                    }
                }
            }
            if (!kBackward) continue;

            // ---------------------------------------------------------------- gradient
            const float f_max = finite_max(m);
            float tail_factor = mass;
            if (HEAD == kHeadDistill) {
                coef = now.w * a.T;
                if (a.teacher_lse && logp0 > kTailFloor) {
                    mass += q_rest;
                    tail_factor = mass - q_rest * expf(-logp0);
                }
            }
            const float scale = (HEAD == kHeadToken ? -coef : coef * tail_factor) * inv_s;
            // the token's vector in the slice, and its place in it
            const int64_t tok_off = HEAD == kHeadToken ? now.tok - v_begin * N : -1;
            const int tok_vec = tok_off >= 0 && tok_off < (int64_t)len * N ? (int)(tok_off / N) : -1;
            const int tok_elem = (int)(now.tok % N);
            if (kForward && plan.resident) {
                slot = slot0;
                phase = phase0;
            }
            for (int ch = 0; ch < chunks; ++ch) {
                if (!(kForward && plan.resident)) full_wait(slot, phase);
                const uint4 *stage = ring + slot * kStageVecs;
                const int v0 = ch * kStageVecs;
                const int n = min(kStageVecs, len - v0);
                uint4 in[VPT];
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (tid + i * NT < n) in[i] = stage[tid + i * NT];
                release(slot);
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int at_v = tid + i * NT;
                    if (at_v < n) {
                        float f[N];
                        Vec<T>::unpack(in[i], f);
#pragma unroll
                        for (int e = 0; e < N; ++e) f[e] = scale * exp_below(f[e], f_max, c);
                        if (HEAD == kHeadToken && tok_vec == v0 + at_v) {
#pragma unroll
                            for (int e = 0; e < N; ++e)
                                if (e == tok_elem) f[e] += coef;
                        }
                        gv[v0 + at_v] = Vec<T>::pack(f);
                    }
                }
                if (++slot == NS) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            if (tid < ntail) {
                const int64_t v = nv * N + tid;
                float d = scale * exp_below(to_f32(x[v]), f_max, c);
                if (HEAD == kHeadToken && v == now.tok) d += coef;
                g[v] = from_f32<T>(d);
            }
            if (HEAD == kHeadDistill) {
                sync();  // the entries below replace what the loop wrote there
#pragma unroll
                for (int j = 0; j < KPT; ++j)
                    if (at[j] >= 0) {
                        const float p = exp_below(xk[j], f_max, c) * inv_s;
                        const float q = expf(log_q(j, off, log_scale));
                        g[v_begin * N + at[j]] = from_f32<T>(coef * (mass * p - q));
                    }
            }
        }
    }
    if (C > 1) cluster_arrive_wait();  // no CTA leaves while a peer may still post to it
}

constexpr int kPairThreads = 256;

// One CTA per pair: each sequence's sum of weighted log ratios (fp64, so that a long sequence's
// sum does not lose what the pair's difference is made of), the pair's loss, and the derivative of
// every row's log-probability.
__global__ void __launch_bounds__(kPairThreads) pair_loss_kernel(PairLossArgs a) {
    __shared__ double slots[(kPairThreads / 32)];
    __shared__ double seq_sum[2];
    const int pair = blockIdx.x, tid = threadIdx.x;
    int64_t begin[2], end[2];
    for (int j = 0; j < 2; ++j) {
        begin[j] = min(max((int64_t)a.seq_start[2 * pair + j], (int64_t)0), a.R);
        end[j] = min(max((int64_t)a.seq_start[2 * pair + j + 1], begin[j]), a.R);
        double v = 0.0;
        for (int64_t r = begin[j] + tid; r < end[j]; r += kPairThreads) {
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
            for (int i = 0; i < (kPairThreads / 32); ++i) s += slots[i];
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
        for (int64_t r = begin[j] + tid; r < end[j]; r += kPairThreads) {
            const float w = a.weight ? a.weight[r] : 1.0f;
            a.dlogp[r] = (w != 0.0f && a.token[r] >= 0) ? d * w : 0.0f;
        }
    }
}

// ------------------------------------------------------------------ launch

// Launch shapes: folding threads, vectors per thread and stage, CTAs per SM, stages of the ring.
struct Shape {
    int threads, vecs, per_sm, stages;
    int stage_bytes() const { return threads * vecs * 16; }
};
constexpr int kShapes = 3;
constexpr Shape kShape[kShapes] = {{128, 4, 4, 6}, {256, 4, 2, 6}, {512, 2, 1, 13}};

template <typename T, int HEAD, int PASS>
const void *kernel_of(int shape) {
    switch (shape) {
        case 0: return (const void *)row_loss_kernel<T, HEAD, PASS, 128, 4>;
        case 1: return (const void *)row_loss_kernel<T, HEAD, PASS, 256, 4>;
        default: return (const void *)row_loss_kernel<T, HEAD, PASS, 512, 2>;
    }
}

template <typename T>
const void *kernel_of(int head, int pass, int shape) {
    if (head == kHeadToken) {
        if (pass == kPassForward) return kernel_of<T, kHeadToken, kPassForward>(shape);
        if (pass == kPassBackward) return kernel_of<T, kHeadToken, kPassBackward>(shape);
        return kernel_of<T, kHeadToken, kPassStep>(shape);
    }
    if (pass == kPassForward) return kernel_of<T, kHeadDistill, kPassForward>(shape);
    if (pass == kPassBackward) return kernel_of<T, kHeadDistill, kPassBackward>(shape);
    return kernel_of<T, kHeadDistill, kPassStep>(shape);
}

const void *kernel_of(int dtype, int head, int pass, int shape) {
    return dtype == DG_BF16 ? kernel_of<__nv_bfloat16>(head, pass, shape) : kernel_of<float>(head, pass, shape);
}

cudaLaunchConfig_t launch_config(const Shape &sh, int clusters, int C, cudaStream_t stream,
                                 cudaLaunchAttribute *attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * C), 1, 1);
    cfg.blockDim = dim3((unsigned)(sh.threads + 32), 1, 1);
    cfg.dynamicSmemBytes = (size_t)sh.stages * sh.stage_bytes();
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Clusters of C CTAs the device holds at once, asked of the runtime once per device and kernel
// (the kernel's shared-memory limit is raised on the way; it belongs to the device's context).
constexpr int kMaxDevices = 16;
cudaError_t resident_clusters(int dtype, int head, int pass, int shape, int log_c, int *out) {
    static std::atomic<int> cache[kMaxDevices][2][2][3][kShapes][4];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int> *slot = dev < kMaxDevices ? &cache[dev][dtype][head][pass - 1][shape][log_c] : nullptr;
    if (slot && (*out = slot->load(std::memory_order_acquire)) > 0) return cudaSuccess;
    const void *fn = kernel_of(dtype, head, pass, shape);
    const Shape &sh = kShape[shape];
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, sh.stages * sh.stage_bytes());
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = launch_config(sh, 1, 1 << log_c, nullptr, attr);
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, fn, &cfg);
    if (e != cudaSuccess) return e;
    *out = n < 1 ? 1 : n;
    if (slot) slot->store(*out, std::memory_order_release);
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_row_loss(const RowLossArgs &a, RowLossHead head, RowLossPass pass, cudaStream_t stream) {
    const int64_t row_bytes = a.V * (a.dtype == DG_BF16 ? 2 : 4);
    int best_shape = 0, best_log_c = 0, best_clusters = 0;
    double best = 0.0;
    bool best_resident = false;
    for (int s = 0; s < kShapes; ++s)
        for (int lc = 0; lc < 4; ++lc) {
            const int C = 1 << lc;
            const Shape &sh = kShape[s];
            const double slice = (double)row_bytes / C;
            if (lc > 0 && slice < 8192) break;
            int n = 0;
            const cudaError_t e = resident_clusters(a.dtype, head, pass, s, lc, &n);
            if (e != cudaSuccess) return e;
            const bool resident = pass == kPassStep && slice <= (double)(sh.stages - 1) * sh.stage_bytes();
            const double passes = pass == kPassForward ? 1.0 : pass == kPassBackward ? 2.0 : resident ? 2.0 : 3.0;
            const double rounds = (double)((a.R + n - 1) / n);
            const double cost = rounds * (slice * passes * sh.per_sm + (lc > 0 ? 80e3 : 40e3));
            if (best_clusters == 0 || cost < best) {
                best = cost;
                best_shape = s;
                best_log_c = lc;
                best_clusters = (int)(a.R < n ? a.R : n);
                best_resident = resident;
            }
        }
    const Plan plan{1 << best_log_c, kShape[best_shape].stages, best_resident};
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = launch_config(kShape[best_shape], best_clusters, plan.cluster, stream, attr);
    void *args[2] = {const_cast<RowLossArgs *>(&a), const_cast<Plan *>(&plan)};
    return cudaLaunchKernelExC(&cfg, kernel_of(a.dtype, head, pass, best_shape), args);
}

cudaError_t launch_pair_loss(const PairLossArgs &a, cudaStream_t stream) {
    pair_loss_kernel<<<(unsigned)a.P, kPairThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace dg
