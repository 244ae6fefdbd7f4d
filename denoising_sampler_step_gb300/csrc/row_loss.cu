// Losses on rows of full-vocabulary logits, with their gradients: token log-probabilities, the
// clipped policy loss with a KL term, the preference loss's rows, and distillation from a
// teacher's top logits.  Formulas and contracts are in include/dgsamp.h.
//
// With z = x / T, m = max x, s = sum exp((x - m) / T):  lse = m / T + ln s,
// p_v = exp((x_v - m) / T) / s.
//
// HBM-bound: a loss reads each logit once, a gradient reads it once and writes it once, at some
// ten flops per entry.  The statistics of a row must be complete before the first entry of its
// gradient can be written, so a row that is not kept on the chip is read twice.  Here the rows are
// cut into tiles, tile t goes to CTA t mod (one CTA per SM), and a tile stays in the CTA's ring of
// shared-memory stages from its load until its gradient is written.  The whole chip works on a few
// rows at a time; while a row's statistics are exchanged through global memory, every CTA folds the
// tiles that follow and the loads run further ahead, so that neither the exchange nor a barrier
// leaves the memory idle.  Rows of up to kMaxTile bytes are one tile and need no exchange.
//
// Measured, 1,024 rows of 262,144 entries, against a plain copy's 6,780 GB/s: policy loss fp32 forward
// 101%, step 88%, backward 97%; bf16 82%, 83%, 88%; distillation, K = 64 with the bucket, fp32 94%, 87%, 95%,
// bf16 74%, 81%, 91%; a step with K = 512 77%, with K = 1,024 64% (each tile's share of the teacher's entries is
// found by looking at all of them).  What is left in a step: reads and writes that alternate, and in bf16
// the folding warps, which have twice the entries per byte.
//
// In a CTA, each warp or group of warps walks the CTA's tiles at its own pace, held together by an
// mbarrier per stage and step:
//   - the loader brings the tiles of live rows into the ring (cp.async.bulk) and describes them there;
//   - the zero warp writes the gradients and results of the rows left out;
//   - the clearing warps (distillation) list the teacher's entries of a tile and take them out of it, so
//     that what is folded is the bucket of the others: no difference of two sums;
//   - the folding warps take the tile's maximum and sum of exponentials;
//   - the posting warp writes the tile's sum to the workspace;
//   - the owner warps gather the sums of every gridDim-th row, compute its loss and what its gradient
//     needs, and publish that;
//   - the watching warp polls for the published rows, one lane per stage;
//   - the gradient warps turn tiles into gradients, written from registers;
//   - the settling warps write a gradient's few special entries (the token's, the teacher's) over
//     what the gradient warps left there, and hand the stage back.
// The roles' loops share one instruction cache, so they are kept short: tiles are worked out once, by the
// loader, and loops of unknown length are not unrolled.  (A distillation step of 1,024 x 262,144 fp32
// entries, K = 64: 357 us; with each role working its tiles out, 76 KB of code instead of 57, 418; with
// its loops unrolled, 88 KB, 557.)
// CTAs wait for one another's sums, so the launch is cooperative; every wait is bounded, and a role
// whose wait gives up leaves.
#include <atomic>

#include "dg_internal.h"
#include "row_loss.cuh"
#include "vocab_row.cuh"

namespace dg {

namespace {

using namespace vocab;

// Entries down to here are masked (both types' lowest finite values and -inf): a bucket of such entries alone
// has no distribution of its own, and its term is left out.  (Times T below 1: ln p_0 stays a finite fp32 number.)
constexpr float kMasked = -3.38e38f;
// q_0 is a difference from 1 of what teacher_lse and the teacher's logits give, each rounded to fp32, and known
// to about (|teacher_lse| + 4) 2^-22.  Times an ln p_0 below -87 (a vocabulary masked by, say, -1e4 in teacher
// and student alike) such a rest would be a loss of its own, so there it counts as 0.
constexpr float kTailFloor = 0x1p60f * 1.64581143e-38f;  // (2^60 e^-87: see bucket_terms)

struct Plan {
    int stages;      // of the ring
    int tile_vecs;   // 16-byte vectors of a tile and a stage
    int tiles;       // per row
    int row_step, j_step;  // from one of a CTA's tiles to the next
    unsigned long long *sums;  // [R, tiles] posted sums (a MaxSum as 64 bits; 0: not yet)
    struct RowClose *rows;     // [R] published rows
};

// What the gradient of a row needs: g_v = scale exp((x_v - base) / T), and at the special entries
// coef (mass p_v - q_v) with p_v = inv_s exp((x_v - m) / T) and, over a teacher's entries,
// ln q = (t - off) / T + log_scale (a token: q = 1, mass 1, and the sign in coef).
// base is m, but the bucket's own maximum where there is a bucket: p_0 may be far below 1, and a scale over
// exp((x_v - m) / T) would have to hold q_0 / p_0, past fp32's range, times what has vanished in it.
// It is published as four 64-bit words, none of which is ever 0 (there yet: all four are not): a
// maximum, base or offset of 0 is -0, and 1 / s is no 0.
struct __align__(16) RowClose {
    float m, scale, inv_s, coef, mass, off, log_scale, base;
};
__device__ __forceinline__ float never_zero(float v) { return v == 0.0f ? -0.0f : v; }

template <int HEAD, int PASS, bool SPLIT>
struct Roles {
    static constexpr bool kForward = (PASS & kPassForward) != 0, kBackward = (PASS & kPassBackward) != 0;
    // (16 folding warps where no others do arithmetic: policy loss forward, bf16, 97 us; 8 warps 109)
    static constexpr int kClear = HEAD == kHeadDistill ? 3 : 0, kPost = kForward && SPLIT ? 1 : 0,
                         kOwn = kForward ? (SPLIT ? 2 : 4) : 0, kWatch = kForward && kBackward && SPLIT ? 1 : 0,
                         kSettle = kBackward ? 2 : 0, kFold = !kForward ? 0 : kBackward ? 8 : 16, kGrad = kBackward ? 8 : 0;
    // first warps (the loader is 0, the zero warp 1)
    static constexpr int clear = 2, post = clear + kClear, own = post + kPost, watch = own + kOwn,
                         settle = watch + kWatch, fold = settle + kSettle, grad = fold + kFold, end = grad + kGrad;
    static constexpr int kThreads = 32 * end;
};

// A tile in its stage.
struct __align__(16) Tile {
    int64_t row;  // -1: there are no more
    int first;    // its first entry in the row
    int len;      // entries in whole vectors, in the stage
    int end;      // and with the row's last V % (16 / sizeof(T)) entries, which no copy brings
    int tok;      // the row's token
    float w;      // weight; backward over tokens: the coefficient weight * dlogp
};

struct Shared {
    uint64_t full[kMaxStages], issued[kMaxStages], cleared[kMaxStages], folded[kMaxStages], ready[kMaxStages],
        done[kMaxStages], empty[kMaxStages];
    Tile tile[kMaxStages];
    RowClose close[kMaxStages];
    MaxSum warp_sum[kMaxStages][16];
    int entries[kMaxStages];          // of the teacher's in the tile
    uint32_t tail_taken[kMaxStages];  // which of the row's last entries are among them
    int abort_flag;
};

// What decides whether a row is live.
template <int HEAD, int PASS>
struct RowKey {
    float w;
    int tok;
    __device__ __forceinline__ void load(const RowLossArgs &a, int64_t row) {
        w = a.weight ? a.weight[row] : 1.0f;
        tok = 0;
        if (HEAD == kHeadToken) {
            tok = a.token[row];
            if (PASS == kPassBackward && w != 0.0f) w *= a.dlogp[row];
        }
    }
    __device__ __forceinline__ bool live(int64_t V) const {
        return w != 0.0f && (HEAD != kHeadToken || (tok >= 0 && tok < V));
    }
};

// The teacher's part of a row's numbers: what is known without the student's statistics, and its mass
// outside the entries.
__device__ __forceinline__ float teacher_terms(const RowLossArgs &a, const MaxSum &teacher, float teacher_lse,
                                               float w, RowClose *cl) {
    cl->coef = w * a.T;
    if (a.teacher_lse) {
        cl->off = -0.0f;
        cl->log_scale = -teacher_lse;
        cl->mass = teacher.s > 0.0f ? exp_fast(teacher.m / a.T - teacher_lse) * teacher.s : 0.0f;
        return fmaxf(0.0f, 1.0f - cl->mass);
    }
    // (no mass at all: every q is 0)
    cl->off = never_zero(finite_max(teacher.m));
    cl->log_scale = teacher.s > 0.0f ? -logf(teacher.s) : -INFINITY;
    cl->mass = teacher.s > 0.0f ? 1.0f : 0.0f;
    return 0.0f;
}
// And with the student's p_0 = part / s of the bucket: the scale and base of the gradient outside the teacher's
// entries.  tail_m and tail_s are the bucket's own maximum and sum, so p_v = p_0 exp((x_v - tail_m) / T) / tail_s
// there, and the gradient is coef p_v (M - q_0 / p_0), M = sum of q_k and q_0, without that quotient (and exactly
// 0 where p_0 = q_0 = 1).  Returns what of q_rest counts as q_0.  (One division, and not the exact one, on the way
// to a published row: with two exact ones a step of 2,048 x 262,144 fp32 rows, K = 128, took 645 us, not 632.)
// c = log2(e) / T.  p_0 against its floor in 2^60ths: part itself has vanished some ln(V) above it.
__device__ __forceinline__ float bucket_terms(const RowLossArgs &a, float c, float teacher_lse, float part, float s,
                                              float tail_m, float tail_s, float q_rest, RowClose *cl) {
    cl->base = cl->m;
    cl->scale = cl->coef * cl->mass * cl->inv_s;
    if (!a.teacher_lse || !(tail_m > kMasked * fminf(a.T, 1.0f))) return 0.0f;
    const bool far = ex2_approx(fmaf(tail_m - cl->m, c, 60.0f)) * tail_s < kTailFloor * s;
    if (far && q_rest <= (fabsf(teacher_lse) + 4.0f) * 0x1p-22f) q_rest = 0.0f;
    cl->mass += q_rest;
    cl->base = never_zero(tail_m);
    cl->scale = cl->coef * __fdividef(fmaf(cl->mass, part, -q_rest * s), s * tail_s);
    return q_rest;
}

// What rounding lost of sum = a + b.
__device__ __forceinline__ float lost_by_sum(float a, float b, float sum) {
    const float bb = sum - a;
    return (a - (sum - bb)) + (b - bb);
}

// Two words of a row's numbers, in the order in which they lie in memory.
__device__ __forceinline__ unsigned long long two_words(float lo, float hi) {
    return (unsigned long long)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ void publish(RowClose *out, const RowClose &cl) {
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(out), "l"(two_words(cl.m, cl.scale)),
                 "l"(two_words(cl.inv_s, cl.coef))
                 : "memory");
    asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(reinterpret_cast<char *>(out) + 16),
                 "l"(two_words(cl.mass, cl.off)), "l"(two_words(cl.log_scale, cl.base))
                 : "memory");
}
// Whether the row is there; then *cl holds it.
__device__ __forceinline__ bool look_up(const RowClose *in, RowClose *cl) {
    unsigned long long w[4];
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(w[0]), "=l"(w[1]) : "l"(in) : "memory");
    asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];"
                 : "=l"(w[2]), "=l"(w[3])
                 : "l"(reinterpret_cast<const char *>(in) + 16)
                 : "memory");
    auto lo = [](unsigned long long v) { return __uint_as_float((uint32_t)v); };
    auto hi = [](unsigned long long v) { return __uint_as_float((uint32_t)(v >> 32)); };
    *cl = RowClose{lo(w[0]), hi(w[0]), lo(w[1]), hi(w[1]), lo(w[2]), hi(w[2]), lo(w[3]), hi(w[3])};
    return w[0] && w[1] && w[2] && w[3];
}

// From a saved log-sum-exp, p = exp((x - T lse) / T): T lse as m, what its rounding lost as a factor.
__device__ __forceinline__ RowClose close_saved(const RowLossArgs &a, float lse) {
    RowClose cl{};
    cl.m = never_zero(finite_max(lse * a.T));
    cl.inv_s = expf(-fmaf(lse, a.T, -lse * a.T) / a.T);
    cl.base = cl.m;
    return cl;
}
__device__ __forceinline__ RowClose close_token(const RowLossArgs &a, float w, float lse) {
    RowClose cl = close_saved(a, lse);
    cl.coef = -w / a.T;
    cl.mass = 1.0f;
    cl.scale = cl.coef * cl.inv_s;
    return cl;
}

// A posted sum, polled for at most kWaitLimitNs (0: gave up).
__device__ __forceinline__ unsigned long long poll_sum(const unsigned long long *p, volatile int *abort_flag) {
    unsigned long long v;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t i = 0;; ++i) {
        asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
        if (v) return v;
        if ((i & 15u) == 15u) {
            if (*abort_flag) return 0;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                *abort_flag = 1;
                record_timeout();
                return 0;
            }
        }
    }
}

// (x - m) / T - ln s to the nearest float, and in *low what that leaves: a pair's sums, differences from a
// reference's log-probabilities, are small beside them.  What each operation rounds off is exact in fp32.
// The hardware's power of two is 5e-8 too small on average, and so is s but for its largest term, 1,
// which is exact: little in a row, but the same in every row of a sequence, so the share is put back.  (With
// log2(e) / T as one float it is not: its rounding is the other way.  The mean error of ln p over 4,000
// rows is 3e-8 at T = 1, below 5e-8 at others; without this and the two floats up to 5e-7.)
// once = false: the operations' own roundings stay (the policy loss, whose step's code has to be short: without
// them 2,048 x 262,144 bf16 rows took 324 us instead of 317).
template <bool TWO>
__device__ __forceinline__ float log_prob(float x, float m, float T, float lns, float inv_s, bool once, float *low) {
    const float d = x - m, q = d / T, r = q - lns;
    *low = 0.0f;
    if (!(fabsf(r) < INFINITY)) return r;
    if (!once) return TWO ? r + (((q - r) - lns) - 5e-8f * (1.0f - inv_s)) : r;
    const float e = lost_by_sum(q, -lns, r) + (fmaf(-q, T, d) + lost_by_sum(x, -m, d)) / T -
                    (TWO ? 5e-8f * (1.0f - inv_s) : 0.0f);
    const float p = r + e;
    *low = e - (p - r);
    return p;
}

template <bool TWO>
__device__ __forceinline__ auto log2e_over_T(const RowLossArgs &a, float c) {
    if constexpr (TWO)
        return a.scale;
    else
        return c;
}

template <typename T, int HEAD, int PASS, bool SPLIT, bool TWO>
__global__ void __launch_bounds__(Roles<HEAD, PASS, SPLIT>::kThreads, 1)
    row_loss_kernel(const RowLossArgs a, const Plan plan) {
    using W = Roles<HEAD, PASS, SPLIT>;
    constexpr bool kForward = W::kForward, kBackward = W::kBackward;
    constexpr bool kDistill = HEAD == kHeadDistill;
    constexpr int N = Vec<T>::N;
    using Key = RowKey<HEAD, PASS>;
    extern __shared__ __align__(128) uint4 ring[];
    __shared__ Shared sh;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int NS = plan.stages;
    const int V = (int)a.V;
    const bool in_place = a.grad == a.logits;
    const float c = kLog2e / a.T, inv_T = 1.0f / a.T;
    const auto sums_c = log2e_over_T<TWO>(a, c);  // of the sums
    const MaxSum none{-INFINITY, 0.0f};
    // per stage the teacher's entries: place in the tile, the teacher's and the student's logit
    const int kp = a.K;
    int *const lists = reinterpret_cast<int *>(ring + (size_t)NS * plan.tile_vecs);

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.issued[i]), 1);
            mbar_init(smem_u32(&sh.cleared[i]), kDistill ? W::kClear : 1);
            mbar_init(smem_u32(&sh.folded[i]), kForward ? W::kFold : 1);
            mbar_init(smem_u32(&sh.ready[i]), SPLIT || !kForward ? 1 : W::kOwn);
            mbar_init(smem_u32(&sh.done[i]), kBackward ? W::kGrad : 1);
            // forward: the folding warps and who reads their sums; else the settling warps
            mbar_init(smem_u32(&sh.empty[i]), kBackward ? W::kSettle : W::kFold + (SPLIT ? W::kPost : W::kOwn));
        }
        sh.abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();

    if (kForward) grid_launch_dependents();

    // A wait that gives up (a second without what it waits for) raises the abort flag and the device
    // error word; every role then leaves at its next wait.
    auto wait = [&](uint64_t &bar, uint32_t parity) { return ring_wait(smem_u32(&bar), parity & 1, &sh.abort_flag); };
    auto arrive = [&](uint64_t &bar) {  // the warp's, once all its lanes are here
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar));
    };
    // Runs f(stage, its use) over the CTA's tiles in their stages, each once `bar` says that it is there.
    // A barrier's parity tells a phase only from the ones next to it.  Where warps take tiles in turn,
    // the others pass by a tile only in its order, and with an arrival of their own on what it needs to
    // leave its stage: so no warp is ever more than a phase from a barrier that it waits on.
    auto each_tile = [&](uint64_t *bar, auto f) {
        uint32_t lap = 0;
#pragma unroll 1
        for (int slot = 0;;) {
            if (!wait(bar[slot], lap) || sh.tile[slot].row < 0) break;
            f(slot, lap);
            if (++slot == NS) {
                slot = 0;
                ++lap;
            }
        }
    };
    auto stage = [&](int slot) { return ring + (size_t)slot * plan.tile_vecs; };
    auto tile_x = [&](const Tile &t) { return static_cast<const T *>(a.logits) + t.row * a.ldl + t.first; };
    auto tile_g = [&](const Tile &t) { return static_cast<T *>(a.grad) + t.row * a.ldg + t.first; };
    auto log_q = [&](float t, float off, float log_scale) { return (t - off) * inv_T + log_scale; };

    if (warp < 2) {
        // ------------------------------------------------------------ loader, zero warp
        const uint64_t policy = l2_policy_evict_first();
        const int nv = V / N;
        int slot = 0;
        uint32_t lap = 0;
        bool ok = true;
        int64_t row = blockIdx.x / (unsigned)plan.tiles;
        int j = (int)(blockIdx.x % (unsigned)plan.tiles);
        Key next;
        float next_close = 0.0f;
        auto fetch = [&](int64_t r) {
            next.load(a, r);
            if (!kForward && warp == 0 && !kDistill) next_close = next.live(V) ? a.lse[r] : 0.0f;
            if (!kForward && warp == 0 && kDistill && lane < 8)
                next_close = reinterpret_cast<const float *>(plan.rows + r)[lane];
        };
        auto take_stage = [&]() {
            // (also its last copy has landed: an aborted CTA's roles leave stages as they are)
            if (lap > 0) ok = wait(sh.empty[slot], lap - 1) && wait(sh.full[slot], lap - 1);
            ok = ok && !*(volatile int *)&sh.abort_flag;
        };
        auto next_stage = [&]() {
            if (++slot == NS) {
                slot = 0;
                ++lap;
            }
        };
        if (!kForward) grid_dependency_wait();  // on what the kernel before it computes
        if (row < a.R) fetch(row);
#pragma unroll 1
        while (row < a.R && ok) {
            const Key key = next;
            const float my_close = next_close;
            Tile t;
            t.row = row;
            t.first = j * plan.tile_vecs * N;
            const int vecs = min(plan.tile_vecs, nv - j * plan.tile_vecs);
            t.len = vecs * N;
            t.end = j == plan.tiles - 1 ? V - t.first : t.len;
            t.tok = key.tok;
            t.w = key.w;
            const bool starts_row = j == 0;
            row += plan.row_step;
            j += plan.j_step;
            if (j >= plan.tiles) {
                j -= plan.tiles;
                ++row;
            }
            if (row < a.R) fetch(row);
            const bool live = key.live(V);
            if (warp == 0 && live) {
                take_stage();
                if (ok) {
                    if (!kForward && kDistill && lane < 8) reinterpret_cast<float *>(&sh.close[slot])[lane] = my_close;
                    if (!kForward && !kDistill && lane == 0) sh.close[slot] = close_token(a, key.w, my_close);
                    if (lane == 0) sh.tile[slot] = t;
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&sh.issued[slot]));
                        mbar_arrive_expect_tx(smem_u32(&sh.full[slot]), (uint32_t)vecs * 16u);
                        if (vecs) bulk_load(smem_u32(stage(slot)), tile_x(t), (uint32_t)vecs * 16u, smem_u32(&sh.full[slot]), policy);
                    }
                    next_stage();
                }
            }
            if (warp == 1 && !live) {
                if (kBackward) {
                    T *g = tile_g(t);
                    uint4 *gv = reinterpret_cast<uint4 *>(g);
#pragma unroll 4
                    for (int v = lane; v < vecs; v += 32) gv[v] = make_uint4(0, 0, 0, 0);
                    if (lane < t.end - t.len) g[t.len + lane] = from_f32<T>(0.0f);
                }
                if (HEAD == kHeadToken && starts_row && lane == 0 && key.w != 0.0f && key.tok >= V)
                    atomicOr(&g_device_error, kErrorIndexRange);
                if (kForward && starts_row && lane == 0) {
                    if (a.lse) a.lse[t.row] = 0.0f;
                    if (a.loss) a.loss[t.row] = 0.0f;
                    if (a.logp) a.logp[t.row] = 0.0f;
                    if (a.kl) a.kl[t.row] = 0.0f;
                    if (a.clipped) a.clipped[t.row] = 0;
                    if (a.dlogp) a.dlogp[t.row] = 0.0f;
                    if (a.tail_logp) a.tail_logp[t.row] = 0.0f;
                }
            }
        }
        if (warp == 0) {
            if (ok) take_stage();
            __syncwarp();
            if (lane == 0) {
                if (ok) {
                    sh.tile[slot].row = -1;
                    mbar_arrive(smem_u32(&sh.issued[slot]));
                    mbar_arrive(smem_u32(&sh.full[slot]));
                } else {
                    // a CTA that gave up leaves only after its copies in flight have landed
                    for (int i = 0; i < NS; ++i) {
                        const uint32_t loads = lap + (i < slot ? 1 : 0);
                        if (loads > 0) drain_wait(smem_u32(&sh.full[i]), (loads - 1) & 1);
                    }
                }
            }
        }
    } else if (warp < W::post) {
        // ------------------------------------------------------------ clearing warps, a tile each in turn
        uint32_t turn = 0;
        each_tile(sh.issued, [&](int slot, uint32_t lap) {
            const bool own = turn == (uint32_t)(warp - W::clear);
            if (++turn == (W::kClear > 0 ? W::kClear : 1)) turn = 0;
            if (own) {
                const Tile t = sh.tile[slot];
                const int32_t *idx = a.indices + t.row * a.ldk;
                const float *tl = a.teacher + t.row * a.ldk;
                int *const at = lists + (size_t)slot * 3 * kp;
                float *const lt = reinterpret_cast<float *>(at + kp), *const lx = lt + kp;
                int count = 0;
                uint32_t tail = 0;
                bool beyond = false;
                constexpr int kAhead = 16;  // loads at once (K = 1,024: 533 us a step; with 4, 657)
#pragma unroll 1
                for (int k0 = lane; k0 - lane < kp; k0 += 32 * kAhead) {
                    int v[kAhead];
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) v[i] = k0 + 32 * i < kp ? idx[k0 + 32 * i] : -1;
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        if (k0 - lane + 32 * i >= kp) break;
                        const int off = v[i] - t.first;
                        const bool here = v[i] >= t.first && off < t.end;
                        beyond |= v[i] >= V;
                        const uint32_t votes = __ballot_sync(0xffffffffu, here);
                        if (here) {
                            const int n = count + __popc(votes & ((1u << lane) - 1));
                            at[n] = off;
                            if (kBackward) lt[n] = __int_as_float(k0 + 32 * i);
                            if (off >= t.len) tail |= 1u << (off - t.len);
                        }
                        count += __popc(votes);
                    }
                }
                __syncwarp();
                if (kBackward) {
#pragma unroll 1
                    for (int k = lane; k < count; k += 32) lt[k] = tl[__float_as_int(lt[k])];
                }
                if (beyond) atomicOr(&g_device_error, kErrorIndexRange);
                tail = __reduce_or_sync(0xffffffffu, tail);
                if (lane == 0) {
                    sh.entries[slot] = count;
                    sh.tail_taken[slot] = tail;
                }
                __syncwarp();
                // the entries leave the tile
                if (!wait(sh.full[slot], lap)) return;
                T *elems = reinterpret_cast<T *>(stage(slot));
#pragma unroll 1
                for (int k = lane; k < count; k += 32) {
                    const int e = at[k];
                    lx[k] = to_f32(e < t.len ? elems[e] : tile_x(t)[e]);
                    if (kForward && e < t.len) elems[e] = from_f32<T>(-INFINITY);
                }
                if (kForward && count > 0) fence_proxy_async_smem();  // before the copy that refills the stage
            }
            arrive(sh.cleared[slot]);
        });
    } else if (kForward && warp < W::own) {
        // ------------------------------------------------------------ posting warp
        each_tile(sh.full, [&](int slot, uint32_t lap) {
            if (!wait(sh.folded[slot], lap)) return;
            const MaxSum st = warp_merge(lane < W::kFold ? sh.warp_sum[slot][lane] : none, sums_c);
            if (lane == 0) {
                // (never all zero bits: a maximum of 0 has a sum of at least 1)
                unsigned long long *out = plan.sums + sh.tile[slot].row * plan.tiles +
                                          (unsigned)sh.tile[slot].first / (unsigned)(plan.tile_vecs * N);
                asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(out), "l"(two_words(st.s, st.m)) : "memory");
            }
            if (!kBackward) arrive(sh.empty[slot]);
        });
    } else if (kForward && warp < W::watch) {
        // ------------------------------------------------------------ owner warps, a row each in turn
        const int me = warp - W::own;
        auto close_row = [&](int64_t row, float w, int tok, int slot, uint32_t lap) {
            const T *x = static_cast<const T *>(a.logits) + row * a.ldl;
            float A = 0.0f, old = 0.0f, ref = 0.0f, x_tok = 0.0f, teacher_lse = 0.0f, spread = 0.0f, q_rest = 0.0f;
            RowClose cl{};
            MaxSum top = none, teacher = none;
            const int32_t *idx = a.indices + row * a.ldk;
            const float *tl = a.teacher + row * a.ldk;
            if (HEAD == kHeadToken) {
                x_tok = to_f32(x[tok]);
                if (a.policy) {
                    A = a.advantage[row];
                    old = a.old_logp[row];
                    ref = a.ref_logp ? a.ref_logp[row] : 0.0f;
                }
            } else {
                if (a.teacher_lse) teacher_lse = a.teacher_lse[row];
                constexpr int kAhead = 4;
#pragma unroll 1
                for (int k0 = lane; k0 - lane < kp; k0 += 32 * kAhead) {
                    float xv[kAhead], tv[kAhead];
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        const int v = k0 + 32 * i < kp ? idx[k0 + 32 * i] : -1;
                        const bool valid = v >= 0 && v < V;
                        xv[i] = valid ? to_f32(x[v]) : -INFINITY;
                        tv[i] = valid ? tl[k0 + 32 * i] : -INFINITY;
                    }
                    fold(top, xv, sums_c);
                    fold(teacher, tv, sums_c);
                }
                top = warp_merge(top, sums_c);
                teacher = warp_merge(teacher, sums_c);
                // for the loss (here, because the gradient may replace the logits once the row is
                // published): sum of e_k [(t_k - t_max) - (x_k - x_max)] / T
#pragma unroll 1
                for (int k0 = lane; k0 - lane < kp && a.loss; k0 += 32 * kAhead) {
                    float xv[kAhead], tv[kAhead];
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        const int v = k0 + 32 * i < kp ? idx[k0 + 32 * i] : -1;
                        const bool valid = v >= 0 && v < V;
                        xv[i] = valid ? to_f32(x[v]) : 0.0f;
                        tv[i] = valid ? tl[k0 + 32 * i] : -INFINITY;
                    }
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        const float dt = tv[i] - finite_max(teacher.m), e = ex2_approx(dt * c);
                        if (e > 0.0f) spread += e * (dt - (xv[i] - finite_max(top.m)));
                    }
                }
                spread = warp_sum(spread) / a.T;
                q_rest = teacher_terms(a, teacher, teacher_lse, w, &cl);
            }
            __syncwarp();
            // the row's sum: of the entries outside the teacher's, or of all
            MaxSum rest = none;
            if (SPLIT) {
#pragma unroll 1
                for (int i = lane; i < plan.tiles; i += 32) {
                    const unsigned long long v = poll_sum(plan.sums + row * plan.tiles + i, &sh.abort_flag);
                    merge(rest, MaxSum{__uint_as_float((uint32_t)(v >> 32)), __uint_as_float((uint32_t)v)}, sums_c);
                }
                __syncwarp();
            } else {
                wait(sh.full[slot], lap);
                wait(sh.folded[slot], lap);
                if (lane < W::kFold) rest = sh.warp_sum[slot][lane];
            }
            rest = warp_merge(rest, sums_c);

            MaxSum st = rest;
            if (kDistill) merge(st, top, sums_c);
            const float m = st.m;
            cl.m = never_zero(finite_max(m));
            cl.inv_s = 1.0f / st.s;
            const float lns = logf(st.s);
            float logp = 0.0f, logp0 = 0.0f, part = 0.0f, loss = 0.0f, kl = 0.0f, dlogp = 0.0f;
            bool clipped = false;
            // (little before the row is published: the other CTAs wait)
            if (HEAD == kHeadToken) {
                // (divided by T: a product with 1 / T would be off by the same share in every row)
                float low;
                logp = log_prob<TWO>(x_tok, m, a.T, lns, cl.inv_s, !kBackward && !a.policy, &low);
                if (!kBackward && a.keep_low) dlogp = low;
                if (a.policy) {
                    const float ratio = exp_fast(logp - old);
                    const float raw = A != 0.0f ? ratio * A : 0.0f;  // (also where the ratio is infinite)
                    const float cut = fminf(fmaxf(ratio, 1.0f - a.clip_low), 1.0f + a.clip_high) * A;
                    clipped = raw > cut;
                    loss = -(clipped ? cut : raw);
                    dlogp = clipped ? 0.0f : -raw;
                    if (a.ref_logp) {
                        // e^d - 1 in one function: d is small, and the difference is what counts
                        const float d = ref - logp;
                        const float e = expm1f(d);
                        kl = e - d;
                        if (a.kl_coef != 0.0f) {
                            loss = fmaf(a.kl_coef, kl, loss);
                            dlogp = fmaf(-a.kl_coef, e, dlogp);
                        }
                    }
                }
                cl.coef = -dlogp * w * inv_T;
                cl.mass = 1.0f;
                cl.scale = cl.coef * cl.inv_s;
                cl.base = cl.m;
            } else {
                part = rest.s * exp_below(rest.m, cl.m, sums_c);
                q_rest = bucket_terms(a, c, teacher_lse, part, st.s, rest.m, rest.s, q_rest, &cl);
            }
            if (kBackward) {
                if (SPLIT) {
                    // a gradient that replaces the logits waits until they have been read here
                    if (in_place) __threadfence();
                    if (lane == 0) publish(plan.rows + row, cl);
                } else if (lane == 0) {
                    sh.close[slot] = cl;
                }
                __syncwarp();
            }
            if (!SPLIT) arrive(kBackward ? sh.ready[slot] : sh.empty[slot]);
            if (kDistill && a.teacher_lse) {
                // near 1 from the ratio of the sums: the logarithms' difference would round it off
                logp0 = part > 1e-3f * st.s ? logf(part / st.s)
                        : rest.s > 0.0f     ? (rest.m - m) / a.T + logf(rest.s) - lns
                                            : -INFINITY;
            }
            if (kDistill && teacher.s > 0.0f) {
                // q_k = e_k share with e_k = exp((t_k - t_max) / T)
                const float log_share = a.teacher_lse ? teacher.m / a.T - teacher_lse : cl.log_scale;
                loss = exp_fast(log_share) *
                       fmaf(teacher.s, log_share + (m - finite_max(top.m)) / a.T + lns, spread);
            }
            if (kDistill) {
                if (q_rest > 0.0f) loss += q_rest * (logf(q_rest) - logp0);
                loss *= a.T * a.T;
            }
            if (lane == 0) {
                if (a.lse) a.lse[row] = m == -INFINITY ? __int_as_float(0x7fc00000) : m / a.T + lns;
                if (a.loss) a.loss[row] = loss;
                if (a.logp) a.logp[row] = logp;
                if (a.kl) a.kl[row] = kl;
                if (a.clipped) a.clipped[row] = clipped;
                if (a.dlogp) a.dlogp[row] = dlogp;
                if (a.tail_logp) a.tail_logp[row] = logp0;
            }
        };
        if (SPLIT) {
#pragma unroll 1
            for (int64_t row = blockIdx.x + (int64_t)me * gridDim.x; row < a.R; row += (int64_t)W::kOwn * gridDim.x) {
                Key key;
                key.load(a, row);
                if (key.live(V)) close_row(row, key.w, key.tok, 0, 0);
                if (*(volatile int *)&sh.abort_flag) break;
            }
        } else {
            uint32_t turn = 0;
            each_tile(sh.issued, [&](int slot, uint32_t lap) {
                if (turn++ % (W::kOwn > 0 ? W::kOwn : 1) == (uint32_t)me)
                    close_row(sh.tile[slot].row, sh.tile[slot].w, sh.tile[slot].tok, slot, lap);
                else
                    arrive(kBackward ? sh.ready[slot] : sh.empty[slot]);
            });
        }
    } else if (kBackward && warp < W::settle) {
        // ------------------------------------------------------------ watching warp: lane l, stage l
        const RowClose *pending = nullptr;  // the row this lane waits for
        uint32_t lap = 0;
        bool marked = false;                         // this lane's stage holds the mark of the end
        unsigned long long last = globaltimer_ns();  // when something last came
#pragma unroll 1
        while (!__any_sync(0xffffffffu, *(volatile int *)&sh.abort_flag)) {
            bool came = false;
            if (lane < NS && !pending && !marked && mbar_test_wait(smem_u32(&sh.issued[lane]), lap & 1)) {
                came = true;
                ++lap;
                if (sh.tile[lane].row < 0)
                    marked = true;
                else
                    pending = plan.rows + sh.tile[lane].row;
            }
            RowClose cl;
            if (pending && look_up(pending, &cl)) {
                if (in_place) __threadfence();
                sh.close[lane] = cl;
                mbar_arrive(smem_u32(&sh.ready[lane]));
                came = true;
                pending = nullptr;
            }
            // (all that was issued before the mark has been seen once a look after it finds nothing new)
            const bool busy = __any_sync(0xffffffffu, came || pending);
            if (!busy && __any_sync(0xffffffffu, marked)) break;
            const unsigned long long now = globaltimer_ns();
            if (__any_sync(0xffffffffu, came)) {
                last = now;
            } else if (now - last > kWaitLimitNs) {
                *(volatile int *)&sh.abort_flag = 1;
                record_timeout();
            }
        }
    } else if (kBackward && warp < W::fold) {
        // ------------------------------------------------------------ settling warps, a tile each in turn
        uint32_t turn = 0;
        each_tile(sh.full, [&](int slot, uint32_t lap) {
            if (turn++ % 2 == (uint32_t)(warp - W::settle)) {
                const Tile t = sh.tile[slot];
                T *g = tile_g(t);
                if (kDistill && !wait(sh.cleared[slot], lap)) return;
                const int at_tok = t.tok - t.first;
                const bool here = HEAD == kHeadToken && at_tok >= 0 && at_tok < t.end;
                const int count = kDistill ? sh.entries[slot] : here;
                if (count > 0 || t.end > t.len) {
                    if (kForward && !wait(sh.ready[slot], lap)) return;
                    const RowClose cl = sh.close[slot];
                    auto p_of = [&](float x) { return exp_below(x, cl.m, c); };
                    const int *at = lists + (size_t)slot * 3 * kp;
                    const float *lt = reinterpret_cast<const float *>(at + kp), *lx = lt + kp;
                    const T *x = tile_x(t);
                    float x_tok = 0.0f;
                    if (here)
                        x_tok = to_f32(at_tok < t.len ? reinterpret_cast<const T *>(stage(slot))[at_tok] : x[at_tok]);
                    // the row's last entries, no vector of the tile: those that are no special ones
                    const uint32_t taken = kDistill ? sh.tail_taken[slot]
                                                    : here && at_tok >= t.len ? 1u << (at_tok - t.len) : 0u;
                    if (lane < t.end - t.len && !(taken >> lane & 1))
                        g[t.len + lane] = from_f32<T>(cl.scale * exp_below(to_f32(x[t.len + lane]), cl.base, c));
                    if (!wait(sh.done[slot], lap)) return;
                    if (kDistill) {
#pragma unroll 1
                        for (int k = lane; k < count; k += 32) {
                            const float q = exp_fast(log_q(lt[k], cl.off, cl.log_scale));
                            g[at[k]] = from_f32<T>(cl.coef * (cl.mass * (p_of(lx[k]) * cl.inv_s) - q));
                        }
                    } else if (here && lane == 0) {
                        g[at_tok] = from_f32<T>(cl.coef * (p_of(x_tok) * cl.inv_s - 1.0f));
                    }
                } else if (!wait(sh.done[slot], lap)) {
                    return;
                }
            }
            arrive(sh.empty[slot]);
        });
    } else if (kForward && warp < W::grad) {
        // ------------------------------------------------------------ folding warps
        constexpr int kThreads = W::kFold * 32, kVecs = 4;  // vectors per thread at once
        const int my_warp = warp - W::fold, tid = my_warp * 32 + lane;
        each_tile(sh.full, [&](int slot, uint32_t lap) {
            if (kDistill && !wait(sh.cleared[slot], lap)) return;
            const uint4 *vecs = stage(slot);
            const int len = sh.tile[slot].len, nvecs = len / N;
            MaxSum st = none;
#pragma unroll 1
            for (int v0 = tid; v0 - tid < nvecs; v0 += kThreads * kVecs) {
                uint4 in[kVecs];
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    in[i] = v0 + i * kThreads < nvecs
                                ? vecs[v0 + i * kThreads]
                                : make_uint4(Vec<T>::kLow, Vec<T>::kLow, Vec<T>::kLow, Vec<T>::kLow);
                fold_vecs<T>(st, in, sums_c);
            }
            if (tid < sh.tile[slot].end - len) {
                const Tile t = sh.tile[slot];
                const bool taken = kDistill && (sh.tail_taken[slot] >> tid & 1);
                const float one[1] = {taken ? -INFINITY : to_f32(tile_x(t)[len + tid])};
                fold(st, one, sums_c);
            }
            __syncwarp();
            // in a fixed order, so that results repeat bit for bit
            st = warp_merge(st, sums_c);
            if (lane == 0) {
                sh.warp_sum[slot][my_warp] = st;
                mbar_arrive(smem_u32(&sh.folded[slot]));
                if (!kBackward) mbar_arrive(smem_u32(&sh.empty[slot]));
            }
        });
    } else if (kBackward) {
        // ------------------------------------------------------------ gradient warps
        constexpr int kThreads = W::kGrad * 32, kVecs = 4;
        const int tid = threadIdx.x - W::grad * 32;
        const f32x2 cc = pair(c, c);
        each_tile(sh.full, [&](int slot, uint32_t lap) {
            if (kForward && !wait(sh.ready[slot], lap)) return;
            const uint4 *vecs = stage(slot);
            const float base = sh.close[slot].base, scale = sh.close[slot].scale;
            const f32x2 minus_base = pair(-base, -base), scales = pair(scale, scale);
            uint4 *gv = reinterpret_cast<uint4 *>(tile_g(sh.tile[slot]));
            const int nvecs = sh.tile[slot].len / N;
#pragma unroll 1
            for (int v0 = tid; v0 < nvecs; v0 += kThreads * kVecs) {
                uint4 in[kVecs];
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    if (v0 + i * kThreads < nvecs) in[i] = vecs[v0 + i * kThreads];
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    if (v0 + i * kThreads < nvecs) {
                        f32x2 p[N / 2];
                        Vec<T>::pairs(in[i], p);
#pragma unroll
                        for (int e = 0; e < N / 2; ++e) p[e] = mul2(exp_below2(p[e], minus_base, cc), scales);
                        gv[v0 + i * kThreads] = Vec<T>::pack(p);
                    }
            }
            arrive(sh.done[slot]);
        });
    }
}

// Distillation, backward alone: what the gradient of each row needs, from the saved log-sum-exp.  A warp
// per row.
constexpr int kCloseWarps = 8;
__global__ void __launch_bounds__(32 * kCloseWarps) row_close_kernel(const RowLossArgs a, RowClose *rows) {
    const int64_t row = (int64_t)blockIdx.x * kCloseWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    grid_launch_dependents();
    if (row >= a.R) return;
    const float w = a.weight ? a.weight[row] : 1.0f, c = kLog2e / a.T;
    if (w == 0.0f) return;
    RowClose cl = close_saved(a, a.lse[row]);
    MaxSum teacher{-INFINITY, 0.0f};
#pragma unroll 1
    for (int k = lane; k < a.K; k += 32) {
        const int v = a.indices[row * a.ldk + k];
        const float one[1] = {v >= 0 && v < a.V ? a.teacher[row * a.ldk + k] : -INFINITY};
        fold(teacher, one, c);
    }
    teacher = warp_merge(teacher, c);
    const float teacher_lse = a.teacher_lse ? a.teacher_lse[row] : 0.0f;
    const float q_rest = teacher_terms(a, teacher, teacher_lse, w, &cl);
    // the bucket's log-sum-exp stands for its maximum, with a sum of 1 but for what the roundings lost
    const float lse = a.lse[row], logp0 = a.teacher_lse ? a.tail_logp[row] : 0.0f;
    const float tail = lse + logp0, tail_m = tail * a.T;
    const float lost = fmaf(tail, a.T, -tail_m) / a.T + lost_by_sum(lse, logp0, tail);
    bucket_terms(a, c, teacher_lse, expf(logp0), 1.0f, tail_m, expf(lost), q_rest, &cl);
    if (lane == 0) rows[row] = cl;
}

constexpr int kPairThreads = 256, kPairWarps = kPairThreads / 32;

// One CTA per pair: each sequence's sum of weighted log ratios (fp64, so that a long sequence's
// sum does not lose what the pair's difference is made of; dlogp holds the log-probabilities' low parts
// until then), the pair's loss, and the derivative of every row's log-probability.
__global__ void __launch_bounds__(kPairThreads) pair_loss_kernel(PairLossArgs a) {
    __shared__ double slots[kPairWarps];
    __shared__ double seq_sum[2];
    const int pair = blockIdx.x, tid = threadIdx.x;
    grid_launch_dependents();
    grid_dependency_wait();
    int64_t begin[2], end[2];
#pragma unroll 1
    for (int j = 0; j < 2; ++j) {
        begin[j] = min(max((int64_t)a.seq_start[2 * pair + j], (int64_t)0), a.R);
        end[j] = min(max((int64_t)a.seq_start[2 * pair + j + 1], begin[j]), a.R);
        double v = 0.0;
#pragma unroll 1
        for (int64_t r = begin[j] + tid; r < end[j]; r += kPairThreads) {
            const float w = a.weight ? a.weight[r] : 1.0f;
            if (w != 0.0f && a.token[r] >= 0 && a.token[r] < a.V)
                v += (double)w * ((double)a.logp[r] + (double)a.dlogp[r] - (a.ref_logp ? (double)a.ref_logp[r] : 0.0));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if ((tid & 31) == 0) slots[tid >> 5] = v;
        __syncthreads();
        if (tid == 0) {
            double s = 0.0;
#pragma unroll 1
            for (int i = 0; i < kPairWarps; ++i) s += slots[i];
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
    // the rows before the first sequence and behind the last
#pragma unroll 1
    for (int64_t r = tid; pair == 0 && r < begin[0]; r += kPairThreads) a.dlogp[r] = 0.0f;
#pragma unroll 1
    for (int64_t r = end[1] + tid; pair == a.P - 1 && r < a.R; r += kPairThreads) a.dlogp[r] = 0.0f;
#pragma unroll 1
    for (int j = 0; j < 2; ++j) {
        const float d = pw == 0.0f ? 0.0f : (j == 0 ? a.beta : -a.beta) * dz * pw;
#pragma unroll 1
        for (int64_t r = begin[j] + tid; r < end[j]; r += kPairThreads) {
            const float w = a.weight ? a.weight[r] : 1.0f;
            a.dlogp[r] = (w != 0.0f && a.token[r] >= 0 && a.token[r] < a.V) ? d * w : 0.0f;
        }
    }
}

// ------------------------------------------------------------------ launch

static_assert(sizeof(Shared) <= kSharedBytes, "");

struct Kernel {
    const void *fn;
    int threads;
};
template <typename T, int HEAD, int PASS, bool SPLIT, bool TWO>
Kernel one_kernel() {
    return Kernel{(const void *)row_loss_kernel<T, HEAD, PASS, SPLIT, TWO>, Roles<HEAD, PASS, SPLIT>::kThreads};
}
template <typename T, int HEAD, bool TWO>
Kernel kernel_of(int pass, bool split) {
    if (pass == kPassForward)
        return split ? one_kernel<T, HEAD, kPassForward, true, TWO>() : one_kernel<T, HEAD, kPassForward, false, TWO>();
    return split ? one_kernel<T, HEAD, kPassStep, true, TWO>() : one_kernel<T, HEAD, kPassStep, false, TWO>();
}
template <typename T>
Kernel kernel_of(int head, int pass, bool split, bool two) {
    // a gradient alone exchanges and sums nothing
    if (pass == kPassBackward)
        return head == kHeadToken ? one_kernel<T, kHeadToken, kPassBackward, false, false>()
                                  : one_kernel<T, kHeadDistill, kPassBackward, false, false>();
    if (head == kHeadDistill) return kernel_of<T, kHeadDistill, false>(pass, split);
    return two ? kernel_of<T, kHeadToken, true>(pass, split) : kernel_of<T, kHeadToken, false>(pass, split);
}

constexpr int kMaxDevices = 64;

// The kernel's shared-memory limit, raised once per device (it belongs to the device's context).
cudaError_t allow_shared(const void *fn, int index) {
    static std::atomic<int> set[48][kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < kMaxDevices && set[index][dev].load(std::memory_order_acquire))) return e;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e == cudaSuccess && dev < kMaxDevices) set[index][dev].store(1, std::memory_order_release);
    return e;
}

// chained: the kernel before it on the stream is one of this file's, which lets this one start early.
cudaError_t launch_pass(RowLossArgs a, bool chained, RowLossHead head, RowLossPass pass, void *workspace,
                        cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    const int K = head == kHeadDistill ? a.K : 0;
    const Tiling tl = tile_row(a.V, element_size(a.dtype), K);
    const int64_t total = a.R * tl.tiles;
    const int grid = (int)(total < sms ? total : sms);
    const int stages = ring_stages(tl, K);
    Plan plan{stages, tl.tile_vecs, tl.tiles, grid / tl.tiles, grid % tl.tiles, nullptr, nullptr};
    plan.rows = static_cast<RowClose *>(workspace);
    plan.sums = reinterpret_cast<unsigned long long *>(plan.rows + a.R);
    cudaError_t e;
    const bool bf16 = a.dtype == DG_BF16;
    if (pass == kPassBackward && head == kHeadDistill) {
        const unsigned blocks = (unsigned)((a.R + kCloseWarps - 1) / kCloseWarps);
        row_close_kernel<<<blocks, 32 * kCloseWarps, 0, stream>>>(a, plan.rows);
        e = cudaGetLastError();
    } else if (pass != kPassBackward && tl.tiles > 1) {
        e = cudaMemsetAsync(workspace, 0, (size_t)a.R * (sizeof(RowClose) + 8 * (size_t)tl.tiles), stream);
    } else {
        e = cudaSuccess;
    }
    if (e != cudaSuccess) return e;
    const bool split = tl.tiles > 1;
    const bool two = head == kHeadToken && pass != kPassBackward && two_floats(a.T, &a.scale);
    const Kernel k = bf16 ? kernel_of<__nv_bfloat16>(head, pass, split, two) : kernel_of<float>(head, pass, split, two);
    e = allow_shared(k.fn, (bf16 ? 24 : 0) + (head == kHeadDistill ? 12 : 0) + ((int)pass - 1) * 4 + (split ? 2 : 0) + two);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)k.threads);
    cfg.dynamicSmemBytes = (size_t)stages * stage_bytes(tl, K);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    if (pass != kPassBackward && split) {
        // CTAs that exchange sums must all be running
        attr[cfg.numAttrs].id = cudaLaunchAttributeCooperative;
        attr[cfg.numAttrs++].val.cooperative = 1;
    } else if (pass == kPassBackward && (chained || head == kHeadDistill)) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    void *args[2] = {&a, &plan};
    return cudaLaunchKernelExC(&cfg, k.fn, args);
}

// The workspace: the rows' numbers, their sums (the shortest tiles are those of the longest lists, with
// either number of stages), then three floats per row for a step in two passes.
size_t exchange_bytes(int64_t R, int64_t V, int dtype) {
    const int size = element_size(dtype);
    const int few = tile_row(V, size, kFewEntries).tiles, many = tile_row(V, size, kMaxTopK).tiles;
    const int tiles = few > many ? few : many;
    return (size_t)R * (sizeof(RowClose) + 8 * (size_t)tiles);
}

}  // namespace

size_t row_loss_workspace_bytes(int64_t R, int64_t V, int dtype) {
    return exchange_bytes(R, V, dtype) + (size_t)R * 3 * sizeof(float);
}

cudaError_t launch_row_loss(const RowLossArgs &a, RowLossHead head, RowLossPass pass, void *workspace,
                            cudaStream_t stream, bool chained) {
    const int sms = device_sm_count(), K = head == kHeadDistill ? a.K : 0, size = element_size(a.dtype);
    if (sms <= 0) return cudaErrorNoDevice;
    if (!workspace && takes_workspace(a.V, size, head, pass)) return cudaErrorInvalidValue;
    if (pass != kPassStep || !reads_twice(tile_row(a.V, size, K), K, a.R, sms))
        return launch_pass(a, chained, head, pass, workspace, stream);
    RowLossArgs f = a;
    float *saved = reinterpret_cast<float *>(static_cast<char *>(workspace) + exchange_bytes(a.R, a.V, a.dtype));
    if (!f.lse) f.lse = saved;
    if (!f.dlogp) f.dlogp = saved + a.R;
    if (a.teacher_lse && !f.tail_logp) f.tail_logp = saved + 2 * a.R;
    f.grad = nullptr;
    const cudaError_t e = launch_pass(f, false, head, kPassForward, workspace, stream);
    if (e != cudaSuccess) return e;
    f.grad = a.grad;
    return launch_pass(f, true, head, kPassBackward, workspace, stream);
}

cudaError_t launch_pair_loss(const PairLossArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.P);
    cfg.blockDim = dim3(kPairThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pair_loss_kernel, a);
}

}  // namespace dg
