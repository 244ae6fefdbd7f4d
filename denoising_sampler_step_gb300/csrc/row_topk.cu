// The K largest logits of every row, in order, ties to the lowest index, and the tempered
// log-sum-exp.  Contract in include/dgsamp.h.
//
// HBM-bound: every logit is read once.  An entry is a 64-bit key (its value in an
// order-preserving integer form above its complemented index), so that all keys differ and "the K
// largest" means one set whatever the order in which they are met.  A CTA streams a contiguous
// piece of the rows through a ring of shared-memory stages and keeps a buffer of candidates: the
// entries above a threshold that the K-th largest of the piece cannot be below.
//   - The first step's threshold is a value that K of its 256 threads' maxima reach (of its 1,024 vectors'
//     where K is large): at least K entries reach it, and not many more do.  Without it the first steps
//     passed whole into the buffer, and every row began with two cuts of 4,096 entries.
//   - When the buffer fills up it is cut to its K largest and a few more, whose smallest is the new
//     threshold (entries equal to it come later in the row, so they lose to those already held).
//   - A cut finds the K-th largest by histograms of 256 bins over the range of the keys, of the bin
//     that holds it, and so on; it stops as soon as what lies in and above that bin is few enough.
// So a step costs a maximum per vector, and a second look at the vectors of lanes whose maximum is
// above the threshold.
// The rows are cut into steps of 16 KB and the steps dealt out evenly, so that every CTA reads as
// much as every other; a row that several CTAs share leaves each one's K candidates in the
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
constexpr int kVecs = 4;                      // 16-byte vectors per thread and step
constexpr int kStageBytes = kVecs * kThreads * 16;  // a step
constexpr int kStages = 2;
constexpr int kBuffer = 4096;               // candidates
constexpr int kPerSm = 2;
constexpr int kMinSteps = 1;                  // a CTA's least share, where a row is split
constexpr int kRanked = 256;                  // most candidates ordered by counting

// Candidates beyond K that a cut may leave (each less costs it another look at them).
__host__ __device__ constexpr int cut_slack(int K) { return K / 8 + 16; }

struct Shared {
    uint64_t buf[kBuffer];
    uint32_t hist[256];
    uint64_t full[kStages], empty[kStages];
    MaxSum warp_state[kWarps];
    uint32_t warp_lo[kWarps], warp_hi[kWarps];
    uint32_t count, least, digit, before, inside;
    int overflow, abort_flag;
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

// The number of selecting threads with p.
__device__ __forceinline__ int sync_count(bool p) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.popc.aligned.u32 %0, 1, %2, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)p), "n"(kThreads)
        : "memory");
    return r;
}

// A lower edge of the K largest of the buffer's first n entries: at least K of them reach it, and at
// most K + slack.
// All selecting threads; n >= K.
__device__ __noinline__ uint64_t edge_of(Shared &sh, int n, int K, int slack) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (n <= K + slack) return 0;
    // The bins start at a value that at least K entries reach: the threads' least one, or where there
    // are K threads with entries, the least of their largest.
    uint32_t least = 0xffffffffu, hi32 = 0;
#pragma unroll 2
    for (int i = tid; i < n; i += kThreads) {
        const uint32_t v = (uint32_t)(sh.buf[i] >> 32);
        least = min(least, v);
        hi32 = max(hi32, v);
    }
    uint32_t lo32 = K <= kThreads && tid < n ? hi32 : least;
    lo32 = __reduce_min_sync(0xffffffffu, lo32);
    hi32 = __reduce_max_sync(0xffffffffu, hi32);
    if (lane == 0) {
        sh.warp_lo[warp] = lo32;
        sh.warp_hi[warp] = hi32;
    }
    for (int i = tid; i < 256; i += kThreads) sh.hist[i] = 0;
    sync();
    lo32 = __reduce_min_sync(0xffffffffu, sh.warp_lo[lane & (kWarps - 1)]);
    hi32 = __reduce_max_sync(0xffffffffu, sh.warp_hi[lane & (kWarps - 1)]);
    uint64_t lo = (uint64_t)lo32 << 32;
    int shift = max(0, 56 - __clzll((int64_t)(((uint64_t)(hi32 - lo32) << 32) | 0xffffffffu)));
    int bits = 8;  // the bins: entries with (key - lo) >> shift below 2^bits
    uint32_t need = (uint32_t)K;
#pragma unroll 1
    while (true) {
#pragma unroll 2
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t e = sh.buf[i], d = (e - lo) >> shift;
            if (e >= lo && (d >> bits) == 0) atomicAdd(&sh.hist[(uint32_t)d], 1u);
        }
        sync();
        if (warp == 0) {
            // lane l holds the bins 255 - 8 l down to 248 - 8 l; counts from the largest one on
            const uint4 *bins = reinterpret_cast<const uint4 *>(sh.hist) + 62 - 2 * lane;
            const uint4 b1 = bins[0], b0 = bins[1];
            const uint32_t h[8] = {b0.w, b0.z, b0.y, b0.x, b1.w, b1.z, b1.y, b1.x};
            const uint32_t sum = b0.x + b0.y + b0.z + b0.w + b1.x + b1.y + b1.z + b1.w;
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
                        sh.before = before;
                        sh.inside = h[i];
                    }
                    before += h[i];
                }
            }
        }
        sync();
        lo += (uint64_t)sh.digit << shift;
        need -= sh.before;
        if (shift == 0 || sh.inside - need <= (uint32_t)slack) return lo;
        bits = min(8, shift);
        shift -= bits;
        for (int i = tid; i < 256; i += kThreads) sh.hist[i] = 0;
        sync();
    }
}

// Keeps those of the buffer's first n entries that reach `least` and lie before the row's entry
// `end`; sets the count and the smallest one's value.  All selecting threads.
__device__ __noinline__ void keep(Shared &sh, int n, uint64_t least, uint32_t end) {
    const int tid = threadIdx.x, lane = tid & 31;
    constexpr int kAtOnce = 2;
    if (tid == 0) {
        sh.count = 0;
        sh.least = 0xffffffffu;
    }
    uint32_t smallest = 0xffffffffu;
#pragma unroll 1
    for (int b = 0; b < n; b += kAtOnce * kThreads) {
        uint64_t r[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int at = b + tid + i * kThreads;
            r[i] = at < n ? sh.buf[at] : 0;
        }
        sync();  // what follows writes over places read so far
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if (r[i] != 0 && r[i] >= least && 0xffffffffu - (uint32_t)r[i] < end) {
                sh.buf[atomicAdd(&sh.count, 1u)] = r[i];
                smallest = min(smallest, (uint32_t)(r[i] >> 32));
            }
        }
    }
    smallest = __reduce_min_sync(0xffffffffu, smallest);
    if (lane == 0) atomicMin(&sh.least, smallest);
    sync();
}

// The K largest of the buffer's first n entries, from the largest down, to the row's outputs.
__device__ __noinline__ void write_top(Shared &sh, const RowTopKArgs &a, int64_t row, int n) {
    const int tid = threadIdx.x, K = a.K;
    int n2 = K <= kRanked / 2 - kRanked / 16 ? kRanked / 2 : kRanked;  // to be put in order
    while (n2 < K) n2 *= 2;
    if (n > n2) {
        keep(sh, n, edge_of(sh, n, K, n2 - K), 0xffffffffu);
        n = (int)sh.count;
    }
    auto write = [&](int k, uint64_t e) {
        a.values[row * a.ldk + k] = key_value((uint32_t)(e >> 32));
        a.indices[row * a.ldk + k] = (int32_t)(0xffffffffu - (uint32_t)e);
    };
    for (int i = n + tid; i < n2; i += kThreads) sh.buf[i] = 0;
    sync();
    if (n2 <= kRanked) {
        // an entry's place is the number of larger ones, counted by neighbouring threads
        constexpr int kParts = kThreads > kRanked ? kThreads / kRanked : 1;
        const ulonglong2 *all = reinterpret_cast<const ulonglong2 *>(sh.buf);
#pragma unroll 1
        for (int k = tid / kParts; k < (n + 31) / 32 * 32; k += kThreads / kParts) {
            const uint64_t e = sh.buf[k];
            int place = 0;
#pragma unroll 4
            for (int i = tid % kParts; i < (n + 1) / 2; i += kParts) {
                const ulonglong2 o = all[i];
                place += (o.x > e) + (o.y > e);
            }
#pragma unroll
            for (int off = 1; off < kParts; off *= 2) place += __shfl_xor_sync(0xffffffffu, place, off);
            if (tid % kParts == 0 && k < n && place < K) write(place, e);
        }
        return;
    }
    for (int size = 2; size <= n2; size *= 2)
        for (int stride = size / 2; stride > 0; stride /= 2) {
            for (int i = tid; i < n2 / 2; i += kThreads) {
                const int p = 2 * i - (i & (stride - 1)), q = p + stride;
                const uint64_t u = sh.buf[p], v = sh.buf[q];
                if ((u < v) == ((p & size) == 0)) {
                    sh.buf[p] = v;
                    sh.buf[q] = u;
                }
            }
            sync();
        }
    for (int k = tid; k < K; k += kThreads) write(k, sh.buf[k]);
}

// Steps are counted in 32 bits: 2^31 of them are 32 TiB of logits.
struct Layout {
    int steps_per_row;  // ceil(V / entries of a step)
    int steps;          // of all rows
    int ctas;
    int pieces;             // most CTAs that share a row
};

// The steps of CTA b: [b * steps / ctas, (b + 1) * steps / ctas).
__host__ __device__ __forceinline__ int share_begin(const Layout &l, int b) {
    return (int)((int64_t)b * l.steps / l.ctas);
}
// The CTA that holds step s.
__device__ __forceinline__ int share_of(const Layout &l, int s) {
    int b = (int)((int64_t)s * l.ctas / l.steps);
    while (share_begin(l, b + 1) <= s) ++b;
    return b;
}

// The workspace: per row and piece the maximum and sum, then its K candidates.
__device__ __forceinline__ uint64_t *piece_entries(void *ws, const Layout &l, int64_t R, int K, int64_t row,
                                                   int64_t piece) {
    return static_cast<uint64_t *>(ws) + R * l.pieces + (row * l.pieces + piece) * (K + cut_slack(K));
}
__device__ __forceinline__ MaxSum *piece_state(void *ws, const Layout &l, int64_t row, int64_t piece) {
    return static_cast<MaxSum *>(ws) + row * l.pieces + piece;
}

__device__ __forceinline__ float row_lse(const MaxSum &st, float T) {
    return st.m == -INFINITY ? __int_as_float(0x7fc00000) : st.m / T + logf(st.s);
}

template <typename T, bool LSE>
__global__ void __launch_bounds__(kThreads + 32, kPerSm)
    topk_pieces_kernel(const RowTopKArgs a, const Layout lay, void *ws) {
    constexpr int N = Vec<T>::N;
    constexpr int kStep = kStageBytes / sizeof(T);
    // after a cut, and as long as a vector of every thread still fits
    constexpr int kFits = kBuffer - kThreads * N;
    static_assert(kFits >= kMaxTopK + cut_slack(kMaxTopK) && kBuffer >= kVecs * kThreads, "");
    extern __shared__ __align__(128) unsigned char ring[];
    Shared &sh = *reinterpret_cast<Shared *>(ring + kStages * kStageBytes);

    const int tid = threadIdx.x, lane = tid & 31;
    const int V = (int)a.V, nv = V / N;  // entries, and vectors that bulk copies bring
    const int begin = share_begin(lay, blockIdx.x), end = share_begin(lay, blockIdx.x + 1);
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

    int slot = 0;
    uint32_t use = 0;
    auto next_stage = [&]() {
        if (++slot == kStages) {
            slot = 0;
            ++use;
        }
    };
    // vectors of the row's step i
    auto vecs_of = [&](int i) { return max(0, min(kVecs * kThreads, nv - i * (kVecs * kThreads))); };
    if (tid >= kThreads) {
        // ------------------------------------------------------------ loader
        if (lane != 0) return;
        const uint64_t policy = l2_policy_evict_first();
        bool ok = true;
        int row = begin / lay.steps_per_row, i = begin % lay.steps_per_row;
#pragma unroll 1
        for (int s = begin; s < end; ++s) {
            if (use > 0) ok = ring_wait(smem_u32(&sh.empty[slot]), (use - 1) & 1, &sh.abort_flag);
            if (!ok) break;
            const uint32_t bytes = (uint32_t)vecs_of(i) * 16u, bar = smem_u32(&sh.full[slot]);
            mbar_arrive_expect_tx(bar, bytes);
            if (bytes)
                bulk_load(smem_u32(ring + slot * kStageBytes), static_cast<const T *>(a.logits) + row * a.ldl + (int64_t)i * kStep,
                          bytes, bar, policy);
            next_stage();
            if (++i == lay.steps_per_row) {
                i = 0;
                ++row;
            }
        }
        // a CTA that gave up leaves only after its copies in flight have landed
        if (!ok)
            for (int k = 0; k < kStages; ++k) {
                const uint32_t issued = use + (k < slot ? 1 : 0);
                if (issued > 0) drain_wait(smem_u32(&sh.full[k]), (issued - 1) & 1);
            }
        return;
    }

    // ---------------------------------------------------------------- selecting threads
    const float c = kLog2e / a.T;
    const uint4 low = make_uint4(Vec<T>::kLow, Vec<T>::kLow, Vec<T>::kLow, Vec<T>::kLow);
    const int slack = cut_slack(a.K), limit = min(kFits, max(1024, 4 * a.K));
#pragma unroll 1
    for (int s = begin; s < end;) {
        const int row = s / lay.steps_per_row, s0 = s - row * lay.steps_per_row;
        const int n = min(end - s, lay.steps_per_row - s0);
        const bool whole = n == lay.steps_per_row;
        const T *x = static_cast<const T *>(a.logits) + row * a.ldl;
        MaxSum st{-INFINITY, 0.0f};
        float threshold = 0.0f;
        if (tid == 0) {
            sh.count = 0;
            sh.overflow = 0;
        }
        sync();
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            // (where the ring gave up: stale bytes, but all in bounds, and the error word is set)
            ring_wait(smem_u32(&sh.full[slot]), use & 1, &sh.abort_flag);
            const int v0 = (s0 + i) * kStep, here = vecs_of(s0 + i);
            const uint4 *stage = reinterpret_cast<const uint4 *>(ring + slot * kStageBytes);
            const bool last = i + 1 == n, ends_row = s0 + i + 1 == lay.steps_per_row;
            uint4 in[kVecs];
#pragma unroll
            for (int j = 0; j < kVecs; ++j) in[j] = tid + j * kThreads < here ? stage[tid + j * kThreads] : low;
            // the row's last V % N entries, which no copy brings
            const bool tail = ends_row && tid < V - nv * N;
            const float one[1] = {tail ? to_f32(x[nv * N + tid]) : -INFINITY};
            const float bm = Vec<T>::largest(in);
            if (i == 0) {
                // A value that K of the threads' maxima reach, or of their vectors' where K is too many:
                // bit by bit, until not many more than K reach it.
                constexpr int kMost = kThreads * 7 / 8;
                uint32_t key[kVecs], edge = 0;
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    const uint4 v[1] = {in[j]};
                    key[j] = order_key(Vec<T>::largest(v));
                }
                if (a.K <= kMost) key[0] = order_key(bm);
#pragma unroll 1
                for (uint32_t bit = 1u << 31; bit; bit >>= 1) {
                    int reach = sync_count(key[0] >= (edge | bit));
                    if (a.K > kMost) {
#pragma unroll
                        for (int j = 1; j < kVecs; ++j) reach += sync_count(key[j] >= (edge | bit));
                    }
                    if (reach >= a.K) edge |= bit;
                    if (reach >= a.K && reach <= a.K + a.K / 8) break;
                }
                // Candidates are above the threshold: it is the next number below the edge (below 0 is not
                // -0), and below -inf, as where there is no edge, a NaN: every entry is a candidate.
                threshold = edge > 0 ? key_value(edge - (edge == order_key(0.0f) ? 2 : 1)) : __int_as_float(0x7fc00000);
            }
            if (LSE) {
                fold_vecs<T>(st, in, c);
                if (ends_row) fold(st, one, c);
            }
            // all vectors at once; where that is more than the buffer takes, once more one at a time
            int width = kVecs;
#pragma unroll 1
            for (int j0 = 0; j0 < kVecs;) {
                const bool ends = last && j0 + width == kVecs;
                bool crowded = false;
                if (__any_sync(0xffffffffu, !(bm <= threshold))) {
                    // a bit per entry of the lane's that is a candidate
                    uint32_t mask = 0;
#pragma unroll
                    for (int j = 0; j < kVecs; ++j) {
                        const uint4 v[1] = {in[j]};
                        if (__any_sync(0xffffffffu, !(Vec<T>::largest(v) <= threshold)) && j >= j0 && j < j0 + width &&
                            tid + j * kThreads < here) {
                            f32x2 p[N / 2];
                            Vec<T>::pairs(in[j], p);
#pragma unroll
                            for (int e = 0; e < N / 2; ++e) {
                                float f, g;
                                unpair(p[e], f, g);
                                mask |= (f <= threshold ? 0u : 1u << (j * N + 2 * e)) |
                                        (g <= threshold ? 0u : 2u << (j * N + 2 * e));
                            }
                        }
                    }
                    // their places: one addition per warp
                    const int mine = __popc(mask);
                    int upto = mine;
#pragma unroll
                    for (int off = 1; off < 32; off <<= 1) {
                        const int o = __shfl_up_sync(0xffffffffu, upto, off);
                        if (lane >= off) upto += o;
                    }
                    int at = 0;
                    if (lane == 31 && upto > 0) at = (int)atomicAdd(&sh.count, (uint32_t)upto);
                    at = __shfl_sync(0xffffffffu, at, 31) + upto - mine;
#pragma unroll 1
                    for (; mask; mask &= mask - 1, ++at) {
                        const int bit = __ffs(mask) - 1, e = (tid + bit / N * kThreads) * N + bit % N;
                        if (at < kBuffer)
                            sh.buf[at] = entry(to_f32(reinterpret_cast<const T *>(stage)[e]), (uint32_t)(v0 + e));
                        else
                            sh.overflow = 1;
                        crowded = at >= limit;
                    }
                }
                if (tail && j0 + width == kVecs && !(one[0] <= threshold)) {
                    const int at = (int)atomicAdd(&sh.count, 1u);
                    if (at < kBuffer)
                        sh.buf[at] = entry(one[0], (uint32_t)(nv * N + tid));
                    else
                        sh.overflow = 1;
                    crowded |= at >= limit;
                }
                if (sync_or(crowded) || (ends && !whole)) {
                    if (width == kVecs && sh.overflow) {
                        keep(sh, kBuffer, 0, (uint32_t)v0);
                        if (tid == 0) sh.overflow = 0;
                        width = 1;
                        continue;
                    }
                    const int got = (int)sh.count;
                    sync();  // every thread has read the count
                    if (got > limit || (ends && !whole && got > a.K + slack)) {
                        keep(sh, got, edge_of(sh, got, a.K, slack), 0xffffffffu);
                        threshold = key_value(sh.least);
                    }
                }
                j0 += width;
            }
            if (lane == 0) mbar_arrive(smem_u32(&sh.empty[slot]));
            next_stage();
        }
        // ------------------------------------------------------------ the piece's result
        if (LSE) {
            st = warp_merge(st, c);
            if (lane == 0) sh.warp_state[tid >> 5] = st;
            sync();
            st = warp_merge(lane < kWarps ? sh.warp_state[lane] : MaxSum{-INFINITY, 0.0f}, c);
        }
        const int got = (int)sh.count;
        if (whole) {
            write_top(sh, a, row, got);
            if (LSE && tid == 0) a.lse[row] = row_lse(st, a.T);
        } else {
            const int piece = (int)blockIdx.x - share_of(lay, row * lay.steps_per_row);
            uint64_t *out = piece_entries(ws, lay, a.R, a.K, row, piece);
            for (int k = tid; k < a.K + slack; k += kThreads) out[k] = k < got ? sh.buf[k] : 0;
            if (LSE && tid == 0) *piece_state(ws, lay, row, piece) = st;
        }
        sync();  // the buffer is free for the next row
        s += n;
    }
}

// Takes the K largest of a split row's candidates.
template <bool LSE>
__global__ void __launch_bounds__(kThreads) topk_merge_kernel(const RowTopKArgs a, const Layout lay, void *ws) {
    extern __shared__ __align__(128) unsigned char ring[];
    Shared &sh = *reinterpret_cast<Shared *>(ring);
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    const int row = blockIdx.x;
    const int first = share_of(lay, row * lay.steps_per_row);
    const int last = share_of(lay, (row + 1) * lay.steps_per_row - 1);
    if (first == last) return;  // the pieces kernel has written the row
    const int total = (last - first + 1) * (a.K + cut_slack(a.K));
    const uint64_t *in = piece_entries(ws, lay, a.R, a.K, row, 0);
    uint64_t least = 0;
    if (tid == 0) sh.count = 0;
    sync();
    // as many at once as the buffer takes; what lies below the K-th largest so far is passed over
    for (int e0 = 0; e0 < total;) {
        const int n = min(kBuffer - (int)sh.count, total - e0);
        sync();
        for (int i = tid; i < n; i += kThreads) {
            const uint64_t e = in[e0 + i];
            if (e >= least && e != 0) sh.buf[atomicAdd(&sh.count, 1u)] = e;
        }
        sync();
        e0 += n;
        const int got = (int)sh.count;
        sync();
        if (e0 < total && got > a.K) {
            least = edge_of(sh, got, a.K, 0);
            keep(sh, got, least, 0xffffffffu);
        }
    }
    write_top(sh, a, row, (int)sh.count);
    if (LSE && tid < 32) {
        const float c = kLog2e / a.T;
        MaxSum st{-INFINITY, 0.0f};
        for (int p = lane; p <= last - first; p += 32) merge(st, *piece_state(ws, lay, row, p), c);
        st = warp_merge(st, c);
        if (lane == 0) a.lse[row] = row_lse(st, a.T);
    }
}

constexpr size_t kDynamic = kStages * kStageBytes + sizeof(Shared);

// The deal of the rows' steps over the device's CTAs.
bool layout(int64_t R, int64_t V, int K, int dtype, Layout *l) {
    const int sms = device_sm_count();
    if (sms <= 0) return false;
    const int64_t step = kStageBytes / (dtype == DG_BF16 ? 2 : 4);
    const int64_t per_row = (V + step - 1) / step, steps = R * per_row;
    if (steps > INT32_MAX) return false;
    l->steps_per_row = (int)per_row;
    l->steps = (int)steps;
    // a piece of a row costs a selection and K candidates to merge: no fewer than kMinSteps steps,
    // nor than 8 K entries
    const int64_t least = max((int64_t)kMinSteps, (8 * (int64_t)K + step - 1) / step);
    const int64_t want = (l->steps + least - 1) / least;
    l->ctas = (int)max((int64_t)1, min((int64_t)sms * kPerSm, want));
    const int share = l->steps / l->ctas;  // every CTA has at least this
    l->pieces = min((l->steps_per_row + share - 1) / share + 1, l->steps_per_row);
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
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(topk_merge_kernel<LSE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
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
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, topk_merge_kernel<LSE>, a, lay, ws);
}

}  // namespace

size_t row_topk_workspace_bytes(int64_t R, int64_t V, int K, int dtype) {
    Layout l;
    if (!layout(R, V, K, dtype, &l)) return 0;
    return (size_t)R * l.pieces * (sizeof(MaxSum) + (size_t)(K + cut_slack(K)) * sizeof(uint64_t));
}

cudaError_t launch_row_topk(const RowTopKArgs &a, void *workspace, cudaStream_t stream) {
    Layout l;
    if (!layout(a.R, a.V, a.K, a.dtype, &l)) return cudaErrorNoDevice;
    if (a.dtype == DG_BF16)
        return a.lse ? launch<__nv_bfloat16, true>(a, l, workspace, stream)
                     : launch<__nv_bfloat16, false>(a, l, workspace, stream);
    return a.lse ? launch<float, true>(a, l, workspace, stream) : launch<float, false>(a, l, workspace, stream);
}

}  // namespace dg
