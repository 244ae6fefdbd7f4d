// The K largest logits of every row, in order, ties to the lowest index, and the tempered
// log-sum-exp.  Contract in include/dgsamp.h.
//
// HBM-bound: every logit is read once.  An entry is a 64-bit key (its value in an
// order-preserving integer form above its complemented index), so that all keys differ and "the K
// largest" means one set whatever the order in which they are met.  A CTA streams a contiguous
// piece of the rows through a ring of shared-memory stages and keeps a buffer of candidates:
//   - the entries above the threshold, the K-th largest key met so far, are pushed (entries equal
//     to its value come later in the row, so they lose to those already held);
//   - when the next step might not fit, a radix selection cuts the buffer to its K largest, whose
//     smallest is the new threshold.  After the first few thousand entries of a row hardly any
//     entry passes: a step costs a maximum and a comparison per entry.
// The rows are cut into steps of 2,048 entries and the steps dealt out evenly, so that every CTA
// reads as much as every other; a row that several CTAs share leaves each one's K candidates in the
// workspace, and a second kernel takes the K largest of those.
#include <atomic>

#include "dg_internal.h"
#include "row_loss.cuh"
#include "vocab_row.cuh"

namespace dg {

namespace {

using namespace vocab;

constexpr int kThreads = 256;                 // selecting threads
constexpr int kWarps = kThreads / 32;
constexpr int kStep = 2048;                   // entries between two looks at the buffer
constexpr int kPerThread = kStep / kThreads;
constexpr int kBuffer = 4096;                 // candidates
constexpr int kStageBytes = 8192;
constexpr int kStages = 5;
constexpr int kPerSm = 3;
constexpr int kMinSteps = 4;                  // a CTA's least share, where a row is split

struct Shared {
    uint64_t buf[kBuffer];
    uint32_t hist[256];
    uint64_t full[kStages], empty[kStages];
    MaxSum warp_state[kWarps];
    uint32_t warp_lo[kWarps], warp_hi[kWarps];
    uint32_t count, digit, need, done;
    int abort_flag;
};

// Larger floats have larger keys; -0 and +0 the same one; every number's key is above 0.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t entry(float x, uint32_t index) {
    return ((uint64_t)order_key(x) << 32) | (0xffffffffu - index);
}

__device__ __forceinline__ void sync() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }
__device__ __forceinline__ bool sync_or(bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)p), "n"(kThreads)
        : "memory");
    return r != 0;
}

// Cuts the buffer's first n <= kBuffer entries (0 where there is none) to its K largest, in any
// order at the front (0 after them where there are fewer); returns the smallest one's value, its
// index left out.  All selecting threads; n >= K.
__device__ __forceinline__ uint64_t select_top(Shared &sh, int n, int K) {
    constexpr int R = kBuffer / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t r[R];
    uint32_t lo = 0xffffffffu, hi = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        r[i] = tid + i * kThreads < n ? sh.buf[tid + i * kThreads] : 0;
        if (tid + i * kThreads < n) {
            lo = min(lo, (uint32_t)(r[i] >> 32));
            hi = max(hi, (uint32_t)(r[i] >> 32));
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        sh.warp_lo[warp] = lo;
        sh.warp_hi[warp] = hi;
    }
    if (tid == 0) sh.count = 0;
    sync();
    lo = __reduce_min_sync(0xffffffffu, sh.warp_lo[lane & (kWarps - 1)]);
    hi = __reduce_max_sync(0xffffffffu, sh.warp_hi[lane & (kWarps - 1)]);
    // the digits start at the first bit in which the values differ: most keys share the top ones
    int top = 64 - (lo == hi ? 32 : __clz(lo ^ hi));  // bits below this one are undecided
    uint64_t prefix = top == 64 ? 0 : ((uint64_t)hi << 32) >> top;  // of the K-th largest, so far
    uint32_t need = (uint32_t)K;
    while (true) {
        const int shift = max(0, top - 8);
        const int bits = top - shift;
        for (int i = tid; i < 256; i += kThreads) sh.hist[i] = 0;
        sync();
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (tid + i * kThreads < n && (top == 64 || (r[i] >> top) == prefix))
                atomicAdd(&sh.hist[(uint32_t)(r[i] >> shift) & ((1u << bits) - 1)], 1u);
        sync();
        if (warp == 0) {
            // lane l holds the digits 255 - 8 l down to 248 - 8 l; counts from the largest digit on
            uint32_t h[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[i] = sh.hist[255 - 8 * lane - i];
                sum += h[i];
            }
            uint32_t upto = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += o;
            }
            uint32_t before = upto - sum;
            if (before < need && need <= upto) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (before < need && need <= before + h[i]) {
                        sh.digit = 255 - 8 * lane - i;
                        sh.need = need - before;
                        sh.done = h[i] == need - before;
                    }
                    before += h[i];
                }
            }
        }
        sync();
        prefix = (prefix << bits) | sh.digit;
        need = sh.need;
        top = shift;
        // every entry of the last digit is wanted, or the keys are decided to the last bit
        if (sh.done || top == 0) break;
    }
    const uint64_t least = top == 64 ? 0 : prefix << top;
    uint64_t smallest = ~0ull;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool take = tid + i * kThreads < n && r[i] >= least && r[i] != 0;
        if (take) smallest = min(smallest, r[i]);
        const uint32_t votes = __ballot_sync(0xffffffffu, take);
        if (votes) {
            uint32_t base = 0;
            if (lane == 0) base = atomicAdd(&sh.count, (uint32_t)__popc(votes));
            base = __shfl_sync(0xffffffffu, base, 0);
            if (take) sh.buf[base + __popc(votes & ((1u << lane) - 1))] = r[i];
        }
    }
    const uint32_t h32 = __reduce_min_sync(0xffffffffu, (uint32_t)(smallest >> 32));
    if (lane == 0) sh.warp_lo[warp] = h32;
    sync();
    for (int i = (int)sh.count + tid; i < K; i += kThreads) sh.buf[i] = 0;
    sync();
    return (uint64_t)__reduce_min_sync(0xffffffffu, sh.warp_lo[lane & (kWarps - 1)]) << 32;
}

// Orders the buffer's first K entries from the largest down.
__device__ __forceinline__ void sort_top(Shared &sh, int K) {
    const int tid = threadIdx.x;
    int n2 = 1;
    while (n2 < K) n2 *= 2;
    for (int i = K + tid; i < n2; i += kThreads) sh.buf[i] = 0;
    sync();
    for (int size = 2; size <= n2; size *= 2)
        for (int stride = size / 2; stride > 0; stride /= 2) {
            for (int i = tid; i < n2 / 2; i += kThreads) {
                const int a = 2 * i - (i & (stride - 1)), b = a + stride;
                const uint64_t p = sh.buf[a], q = sh.buf[b];
                if ((p < q) == ((a & size) == 0)) {
                    sh.buf[a] = q;
                    sh.buf[b] = p;
                }
            }
            sync();
        }
}

struct Layout {
    int64_t steps_per_row;  // ceil(V / kStep)
    int64_t steps;          // of all rows
    int ctas;
    int pieces;             // most CTAs that share a row
};

// The steps of CTA b: [b * steps / ctas, (b + 1) * steps / ctas).
__host__ __device__ __forceinline__ int64_t share_begin(const Layout &l, int64_t b) {
    return b * l.steps / l.ctas;
}
// The CTA that holds step s.
__device__ __forceinline__ int64_t share_of(const Layout &l, int64_t s) {
    int64_t b = s * l.ctas / l.steps;
    while (share_begin(l, b + 1) <= s) ++b;
    return b;
}

// The workspace: per row and piece the maximum and sum, then its K candidates.
__device__ __forceinline__ uint64_t *piece_entries(void *ws, const Layout &l, int64_t R, int K, int64_t row,
                                                   int64_t piece) {
    return static_cast<uint64_t *>(ws) + R * l.pieces + (row * l.pieces + piece) * K;
}
__device__ __forceinline__ MaxSum *piece_state(void *ws, const Layout &l, int64_t row, int64_t piece) {
    return static_cast<MaxSum *>(ws) + row * l.pieces + piece;
}

__device__ __forceinline__ float row_lse(const MaxSum &st, float T) {
    return st.m == -INFINITY ? __int_as_float(0x7fc00000) : st.m / T + logf(st.s);
}

__device__ __forceinline__ void write_row(const RowTopKArgs &a, int64_t row, const uint64_t *best) {
    for (int k = threadIdx.x; k < a.K; k += kThreads) {
        const uint64_t e = best[k];
        const uint32_t v = 0xffffffffu - (uint32_t)e;
        a.values[row * a.ldk + k] = key_value((uint32_t)(e >> 32));
        a.indices[row * a.ldk + k] = (int32_t)v;
    }
}

template <typename T, bool LSE>
__global__ void __launch_bounds__(kThreads + 32, kPerSm)
    topk_pieces_kernel(const RowTopKArgs a, const Layout lay, void *ws) {
    constexpr int kSize = sizeof(T), N = 16 / kSize;
    constexpr int kStepBytes = kStep * kSize;
    constexpr int kStepsPerStage = kStageBytes / kStepBytes;  // 1 (fp32) or 2 (bf16)
    constexpr int kVecs = kPerThread / N;                     // 16-byte vectors per thread and step
    extern __shared__ __align__(128) unsigned char ring[];
    Shared &sh = *reinterpret_cast<Shared *>(ring + kStages * kStageBytes);

    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t V = a.V, nv = V / N * N;  // entries that bulk copies bring
    const int64_t begin = share_begin(lay, blockIdx.x), end = share_begin(lay, (int64_t)blockIdx.x + 1);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), kWarps);
        }
        sh.abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    grid_launch_dependents();

    if (tid >= kThreads) {
        // ------------------------------------------------------------ loader
        if (lane == 0) {
            const uint64_t policy = l2_policy_evict_first();
            int slot = 0;
            uint32_t use = 0;
            bool ok = true;
            for (int64_t s = begin; s < end && ok;) {
                const int64_t row = s / lay.steps_per_row, s0 = s % lay.steps_per_row;
                const int64_t n = min(end - s, lay.steps_per_row - s0);
                const T *x = static_cast<const T *>(a.logits) + row * a.ldl;
                for (int64_t i = 0; i < n && ok; i += kStepsPerStage) {
                    const int64_t v0 = (s0 + i) * kStep;
                    const int64_t v1 = min(nv, (s0 + min(i + kStepsPerStage, n)) * kStep);
                    if (use > 0) ok = ring_wait(smem_u32(&sh.empty[slot]), (use - 1) & 1, &sh.abort_flag);
                    if (!ok) break;
                    const uint32_t bytes = v1 > v0 ? (uint32_t)(v1 - v0) * kSize : 0u, bar = smem_u32(&sh.full[slot]);
                    mbar_arrive_expect_tx(bar, bytes);
                    if (bytes) bulk_load(smem_u32(ring + slot * kStageBytes), x + v0, bytes, bar, policy);
                    if (++slot == kStages) {
                        slot = 0;
                        ++use;
                    }
                }
                s += n;
            }
            // a CTA that gave up leaves only after its copies in flight have landed
            if (!ok)
                for (int i = 0; i < kStages; ++i) {
                    const uint32_t issued = use + (i < slot ? 1 : 0);
                    if (issued > 0) drain_wait(smem_u32(&sh.full[i]), (issued - 1) & 1);
                }
        }
        return;
    }

    // ---------------------------------------------------------------- selecting threads
    const float c = kLog2e / a.T;
    int slot = 0;
    uint32_t phase = 0;
    for (int64_t s = begin; s < end;) {
        const int64_t row = s / lay.steps_per_row, s0 = s % lay.steps_per_row;
        const int64_t n = min(end - s, lay.steps_per_row - s0);
        const T *x = static_cast<const T *>(a.logits) + row * a.ldl;
        MaxSum st{-INFINITY, 0.0f};
        float threshold = 0.0f;
        bool open = true;  // fewer than K entries seen: everything is a candidate
        int held = 0;      // entries placed while open
        if (tid == 0) sh.count = 0;
        sync();
        for (int64_t i = 0; i < n; ++i) {
            const int part = (int)(i % kStepsPerStage);
            if (part == 0) ring_wait(smem_u32(&sh.full[slot]), phase, &sh.abort_flag);
            const int64_t v0 = (s0 + i) * kStep;
            const uint4 *stage = reinterpret_cast<const uint4 *>(ring + slot * kStageBytes + part * kStepBytes);
            float f[kPerThread];
            const bool whole = v0 + kStep <= nv;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int e0 = (tid + j * kThreads) * N;
                const uint4 v = stage[tid + j * kThreads];
                if constexpr (N == 4) {
                    f[4 * j] = __uint_as_float(v.x);
                    f[4 * j + 1] = __uint_as_float(v.y);
                    f[4 * j + 2] = __uint_as_float(v.z);
                    f[4 * j + 3] = __uint_as_float(v.w);
                } else {
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        f[2 * q] = __uint_as_float(u[q] << 16);
                        f[2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
                    }
                }
                if (!whole) {
                    // the row's end: what the copy did not bring, from memory or not there
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (v0 + e0 + e >= nv) f[j * N + e] = v0 + e0 + e < V ? to_f32(x[v0 + e0 + e]) : -INFINITY;
                }
            }
            if (part == kStepsPerStage - 1 || i + 1 == n) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.empty[slot]));
                if (++slot == kStages) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            if (LSE) fold(st, f, c);
            bool crowded = false;
            if (open) {
                // every entry has its place; those past the row's end are 0, below all others
#pragma unroll
                for (int j = 0; j < kPerThread; ++j) {
                    const int e = (tid + j / N * kThreads) * N + j % N;
                    sh.buf[held + e] = v0 + e < V ? entry(f[j], (uint32_t)(v0 + e)) : 0;
                }
                held += kStep;
                if (held >= a.K) crowded = true;
            } else {
                float bm = f[0];
#pragma unroll
                for (int j = 1; j < kPerThread; ++j) bm = fmaxf(bm, f[j]);
                if (bm > threshold) {
#pragma unroll
                    for (int j = 0; j < kPerThread; ++j)
                        if (f[j] > threshold) {
                            const int e = (tid + j / N * kThreads) * N + j % N;
                            const uint32_t p = atomicAdd(&sh.count, 1u);
                            sh.buf[p] = entry(f[j], (uint32_t)(v0 + e));
                            crowded = crowded || p >= (uint32_t)(kBuffer - kStep);
                        }
                }
            }
            // the buffer is cut when the next step might not fit, and at the end of the piece
            if (sync_or(crowded) || i + 1 == n) {
                const int got = open ? held : (int)sh.count;
                if (got > a.K || open) {
                    if (got >= a.K) {
                        sync();  // every thread has read the count
                        const uint64_t least = select_top(sh, got, a.K);
                        threshold = key_value((uint32_t)(least >> 32));
                        open = false;
                        held = a.K;
                    }
                }
            }
        }
        // ------------------------------------------------------------ the piece's result
        const int got = open ? held : a.K;  // open: a short piece, padded with 0 to a step
        const int64_t cta0 = share_of(lay, row * lay.steps_per_row);
        if (LSE) {
            st = warp_merge(st, c);
            if (lane == 0) sh.warp_state[tid >> 5] = st;
            sync();
            st = warp_merge(lane < kWarps ? sh.warp_state[lane] : MaxSum{-INFINITY, 0.0f}, c);
        }
        if (n == lay.steps_per_row) {
            sync();
            sort_top(sh, a.K);
            write_row(a, row, sh.buf);
            if (LSE && tid == 0) a.lse[row] = row_lse(st, a.T);
        } else {
            sync();
            uint64_t *out = piece_entries(ws, lay, a.R, a.K, row, blockIdx.x - cta0);
            for (int k = tid; k < a.K; k += kThreads) out[k] = k < got ? sh.buf[k] : 0;
            if (LSE && tid == 0) *piece_state(ws, lay, row, blockIdx.x - cta0) = st;
        }
        sync();  // the buffer is free for the next row
        s += n;
    }
}

// Takes the K largest of a split row's candidates.
template <bool LSE>
__global__ void __launch_bounds__(kThreads) topk_merge_kernel(const RowTopKArgs a, const Layout lay, void *ws) {
    __shared__ Shared sh;
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t row = blockIdx.x;
    const int64_t first = share_of(lay, row * lay.steps_per_row);
    const int64_t last = share_of(lay, (row + 1) * lay.steps_per_row - 1);
    if (first == last) return;  // the pieces kernel has written the row
    const int64_t total = (last - first + 1) * a.K;
    const uint64_t *in = piece_entries(ws, lay, a.R, a.K, row, 0);
    uint64_t least = 0;
    int held = 0;
    if (tid == 0) sh.count = 0;
    sync();
    for (int64_t e0 = 0; e0 < total;) {
        // as many as the buffer takes; what lies below the K-th largest so far is passed over
        const int room = kBuffer - held;
        const int n = (int)min((int64_t)room, total - e0);
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t e = in[e0 + i];
            if (e >= least && e != 0) sh.buf[held + atomicAdd(&sh.count, 1u)] = e;
        }
        sync();
        const int got = held + (int)sh.count;
        sync();
        e0 += n;
        if (got > a.K) {
            least = select_top(sh, got, a.K);
            held = a.K;
        } else {
            held = got;
        }
        sync();
        if (tid == 0) sh.count = 0;
        sync();
    }
    sort_top(sh, a.K);
    write_row(a, row, sh.buf);
    if (LSE && tid < 32) {
        const float c = kLog2e / a.T;
        MaxSum st{-INFINITY, 0.0f};
        for (int64_t p = lane; p <= last - first; p += 32) merge(st, *piece_state(ws, lay, row, p), c);
        st = warp_merge(st, c);
        if (lane == 0) a.lse[row] = row_lse(st, a.T);
    }
}

constexpr size_t kDynamic = kStages * kStageBytes + sizeof(Shared);

// The deal of the rows' steps over the device's CTAs.
bool layout(int64_t R, int64_t V, int K, Layout *l) {
    const int sms = device_sm_count();
    if (sms <= 0) return false;
    l->steps_per_row = (V + kStep - 1) / kStep;
    l->steps = R * l->steps_per_row;
    // a piece of a row costs a selection and K candidates to merge: no fewer than kMinSteps steps,
    // nor than 8 K entries
    const int64_t least = max((int64_t)kMinSteps, ((int64_t)8 * K + kStep - 1) / kStep);
    const int64_t want = (l->steps + least - 1) / least;
    l->ctas = (int)max((int64_t)1, min((int64_t)sms * kPerSm, want));
    const int64_t share = l->steps / l->ctas;  // every CTA has at least this
    l->pieces = (int)min((l->steps_per_row + share - 1) / share + 1, l->steps_per_row);
    return true;
}

template <typename T, bool LSE>
cudaError_t launch(const RowTopKArgs &a, const Layout &lay, void *ws, cudaStream_t stream) {
    const void *fn = (const void *)topk_pieces_kernel<T, LSE>;
    constexpr int kMaxDevices = 64;
    static std::atomic<int> attr_set[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !attr_set[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDynamic);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) attr_set[dev].store(1, std::memory_order_release);
    }
    topk_pieces_kernel<T, LSE><<<(unsigned)lay.ctas, kThreads + 32, kDynamic, stream>>>(a, lay, ws);
    e = cudaGetLastError();
    // no row is shared where every CTA's share is whole rows
    if (e != cudaSuccess || (lay.steps % lay.ctas == 0 && (lay.steps / lay.ctas) % lay.steps_per_row == 0)) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.R);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, topk_merge_kernel<LSE>, a, lay, ws);
}

}  // namespace

size_t row_topk_workspace_bytes(int64_t R, int64_t V, int K, int) {
    Layout l;
    if (!layout(R, V, K, &l)) return 0;
    return (size_t)R * l.pieces * (sizeof(MaxSum) + (size_t)K * sizeof(uint64_t));
}

cudaError_t launch_row_topk(const RowTopKArgs &a, void *workspace, cudaStream_t stream) {
    Layout l;
    if (!layout(a.R, a.V, a.K, &l)) return cudaErrorNoDevice;
    if (a.dtype == DG_BF16)
        return a.lse ? launch<__nv_bfloat16, true>(a, l, workspace, stream)
                     : launch<__nv_bfloat16, false>(a, l, workspace, stream);
    return a.lse ? launch<float, true>(a, l, workspace, stream) : launch<float, false>(a, l, workspace, stream);
}

}  // namespace dg
