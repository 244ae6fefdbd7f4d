// The K largest logits of every row, in order, ties to the lowest index, and the tempered
// log-sum-exp.  Contract in include/dgsamp.h.
//
// HBM-bound: every logit is read once.  An entry is a 64-bit key (its value in an
// order-preserving integer form above its complemented index), so that all keys differ and "the K
// largest" means one set whatever the order in which they are met.  The rows are cut into units of 8 KB
// and the units dealt out evenly, so that every CTA reads as much as every other, a row or
// a contiguous piece of one after the other; a row that several CTAs share leaves each one's candidates
// in the workspace, and a second kernel takes the K largest of those.
//
// In a CTA, groups of warps take a piece's tiles from a ring of shared-memory stages:
//   - the loader fills the ring;
//   - the filtering warps push the entries above a threshold, which the piece's K-th largest cannot be
//     below, into the piece's buffer of candidates.  Each warp walks the tiles at its own pace;
//   - the folding warps take the maxima and sums of the log-sum-exp;
//   - the finishing warps, a piece each in turn, order a finished piece's candidates while the others are at
//     the next pieces.
// The threshold: each filtering warp takes the maxima of 512 groups of what it has seen of the piece and
// finds a value that K / 4 of them reach; the least of the four warps' values is reached by K entries,
// and by not many more.  It is found anew, without a barrier, whenever the data seen has doubled, so that
// the candidates of a piece of n entries are some K (1 + ln(n / K)).  Should a buffer fill up all the
// same (a row in ascending order), the filtering warps meet and cut it to its K largest and a few more,
// whose smallest is the new threshold; entries equal to it come later in the row, or are looked at once
// more.  A cut finds the K-th largest by histograms of 256 bins over the range of the
// keys, of the bin that holds it, and so on; it stops as soon as what lies in and above that bin is few
// enough.
#include <atomic>

#include "dg_internal.h"
#include "row_loss.cuh"
#include "vocab_row.cuh"

namespace dg {

namespace {

using namespace vocab;

// Two CTAs per SM, of four filtering and four folding warps: a tile costs a filtering warp some 300
// instructions whether it holds candidates or not, and a piece has waits that another CTA fills.  1,024 x
// 262,144 fp32, K = 64, with the log-sum-exp: 198 us; one CTA of twice the warps 262, and with twice the
// tiles 209; tiles of 16 KB 261; a second finishing warp, which takes registers from the others, 204.
constexpr int kPerSm = 2;
constexpr int kFilter = 4, kFolds = 4, kFinish = 1;  // warps
constexpr int kBuffers = 2;                   // of candidates
constexpr int kThreads = 32 * kFilter;        // filtering threads
constexpr int kUnitBytes = 8192;              // what the rows are dealt out in
constexpr int kTileUnits = 4;
constexpr int kTileBytes = kTileUnits * kUnitBytes;
constexpr int kVecs = 4;                      // 16-byte vectors that a folding thread takes at once
constexpr int kTileVecs = kTileBytes / 16 / kThreads;  // and those a filtering thread has in a tile
constexpr int kStages = 2;
constexpr int kBuffer = 2560;                 // candidates
// A CTA's least share, where a row is split.  One row of 262,144 fp32 entries, K = 32: 12.6 us; with 2
// units, so twice the CTAs and candidates to merge, 14.5, with 8 14.1.
constexpr int kMinUnits = 4;
constexpr int kMergeThreads = 256, kMergeBuffer = 4096;
constexpr int kRanked = 256;                  // most candidates ordered by counting
// Most that the finishing warp puts in order beside the next row; more would keep the others waiting for
// it.  By the finishing and by the filtering warps: 1,000 x 50,001 fp32, K = 300, 126 and 138 us; 2,048 x
// 8,000 fp32, K = 400, 161 and 116; 256 x 262,144 bf16, K = 1,024, 133 and 98.
constexpr int kFew = 384;

// Candidates beyond K that a cut may leave (each less costs it another look at them).
__host__ __device__ constexpr int cut_slack(int K) { return K / 8 + 16; }
// Above this many the buffer is cut.
__host__ __device__ constexpr int cut_limit(int K) { return K + cut_slack(K) + 256 > 1024 ? K + cut_slack(K) + 256 : 1024; }
static_assert(cut_limit(kMaxTopK) + 32 * 8 <= kBuffer, "");

// What a selection by a group of warps shares.
struct Select {
    uint32_t hist[256];
    uint32_t warp_lo[16], warp_hi[16];
    uint32_t digit, before, inside;
    unsigned long long least;  // the smallest key kept
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

template <int THREADS>
__device__ __forceinline__ void sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}
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

// The bin (from the largest down) in which the running count of a histogram of 256 reaches `need`: lane l
// looks at the bins 255 - 8 l down to 248 - 8 l.  True in one lane.
__device__ __forceinline__ bool find_bin(const uint32_t *hist, uint32_t need, uint32_t *digit, uint32_t *before_it,
                                         uint32_t *inside) {
    const int lane = threadIdx.x & 31;
    const uint4 *bins = reinterpret_cast<const uint4 *>(hist) + 62 - 2 * lane;
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
    const bool here = before < need && need <= upto;
    if (here) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (before < need && need <= before + h[i]) {
                *digit = 255 - 8 * lane - i;
                *before_it = before;
                *inside = h[i];
            }
            before += h[i];
        }
    }
    return here;
}

// The bins of a first look: keys (key - lo) >> shift below 256.
__device__ __forceinline__ int first_shift(uint32_t lo32, uint32_t hi32) {
    return 56 - __clzll((int64_t)(((uint64_t)(hi32 - lo32) << 32) | 0xffffffffu));
}

// A lower edge of the K largest of n entries: at least K of them reach it, and at most K + slack.
// THREADS threads; n >= K.
template <int THREADS>
__device__ __noinline__ uint64_t edge_of(Select &se, const uint64_t *buf, int n, int K, int slack) {
    const int tid = threadIdx.x % THREADS, lane = tid & 31, warp = tid >> 5;
    if (n <= K + slack) return 0;
    // The bins start at a value that at least K entries reach: the threads' least one, or where there
    // are K threads with entries, the least of their largest.
    uint32_t least = 0xffffffffu, hi32 = 0;
#pragma unroll 2
    for (int i = tid; i < n; i += THREADS) {
        const uint32_t v = (uint32_t)(buf[i] >> 32);
        least = min(least, v);
        hi32 = max(hi32, v);
    }
    uint32_t lo32 = K <= THREADS && tid < n ? hi32 : least;
    lo32 = __reduce_min_sync(0xffffffffu, lo32);
    hi32 = __reduce_max_sync(0xffffffffu, hi32);
    if (lane == 0) {
        se.warp_lo[warp] = lo32;
        se.warp_hi[warp] = hi32;
    }
    for (int i = tid; i < 256; i += THREADS) se.hist[i] = 0;
    sync<THREADS>();
    lo32 = __reduce_min_sync(0xffffffffu, se.warp_lo[lane & (THREADS / 32 - 1)]);
    hi32 = __reduce_max_sync(0xffffffffu, se.warp_hi[lane & (THREADS / 32 - 1)]);
    uint64_t lo = (uint64_t)lo32 << 32;
    int shift = first_shift(lo32, hi32), bits = 8;
    uint32_t need = (uint32_t)K;
#pragma unroll 1
    while (true) {
#pragma unroll 2
        for (int i = tid; i < n; i += THREADS) {
            const uint64_t e = buf[i], d = (e - lo) >> shift;
            if (e >= lo && (d >> bits) == 0) atomicAdd(&se.hist[(uint32_t)d], 1u);
        }
        sync<THREADS>();
        if (warp == 0) find_bin(se.hist, need, &se.digit, &se.before, &se.inside);
        sync<THREADS>();
        lo += (uint64_t)se.digit << shift;
        need -= se.before;
        if (shift == 0 || se.inside - need <= (uint32_t)slack) return lo;
        bits = min(8, shift);
        shift -= bits;
        for (int i = tid; i < 256; i += THREADS) se.hist[i] = 0;
        sync<THREADS>();
    }
}

// Keeps those of n entries that reach `least` (an entry of 0 is none); sets the count and the smallest
// key kept.  THREADS threads.
template <int THREADS>
__device__ __noinline__ void keep(Select &se, uint64_t *buf, uint32_t *count, int n, uint64_t least) {
    const int tid = threadIdx.x % THREADS;
    constexpr int kAtOnce = 2;
    if (tid == 0) {
        *count = 0;
        se.least = ~0ull;
    }
    uint64_t smallest = ~0ull;
#pragma unroll 1
    for (int b = 0; b < n; b += kAtOnce * THREADS) {
        uint64_t r[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int at = b + tid + i * THREADS;
            r[i] = at < n ? buf[at] : 0;
        }
        sync<THREADS>();  // what follows writes over places read so far
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if (r[i] != 0 && r[i] >= least) {
                buf[atomicAdd(count, 1u)] = r[i];
                smallest = min(smallest, r[i]);
            }
        }
    }
    if (smallest != ~0ull) atomicMin(&se.least, (unsigned long long)smallest);
    sync<THREADS>();
}

__device__ __forceinline__ void write_entry(const RowTopKArgs &a, int64_t row, int k, uint64_t e) {
    a.values[row * a.ldk + k] = key_value((uint32_t)(e >> 32));
    a.indices[row * a.ldk + k] = (int32_t)(0xffffffffu - (uint32_t)e);
}

// Puts n2 (a power of two) entries in order, from the largest down.
template <typename Sync>
__device__ __forceinline__ void sort_entries(uint64_t *buf, int n2, int tid, int threads, Sync sync_all) {
#pragma unroll 1
    for (int size = 2; size <= n2; size *= 2)
#pragma unroll 1
        for (int stride = size / 2; stride > 0; stride /= 2) {
#pragma unroll 2
            for (int i = tid; i < n2 / 2; i += threads) {
                const int p = 2 * i - (i & (stride - 1)), q = p + stride;
                const uint64_t u = buf[p], v = buf[q];
                if ((u < v) == ((p & size) == 0)) {
                    buf[p] = v;
                    buf[q] = u;
                }
            }
            sync_all();
        }
}

// The same for up to 256 entries in a warp's registers: entry 8 lane + r is r[r].
__device__ __forceinline__ void sort_warp(uint64_t (&r)[8], int n2) {
    const int lane = threadIdx.x & 31;
    auto order = [](uint64_t &u, uint64_t &v, bool down) {
        const uint64_t hi = u > v ? u : v, lo = u > v ? v : u;
        u = down ? hi : lo;
        v = down ? lo : hi;
    };
#pragma unroll 1
    for (int size = 2; size <= n2; size *= 2) {
#pragma unroll 1
        for (int far = size / 16; far > 0; far /= 2) {
            const bool larger = ((lane & far) == 0) == ((8 * lane & size) == 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint64_t o = __shfl_xor_sync(0xffffffffu, r[i], far);
                r[i] = (o > r[i]) == larger ? o : r[i];
            }
        }
        if (size >= 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) order(r[i], r[i + 4], (8 * lane & size) == 0 || size < 8);
        }
        if (size >= 4) {
#pragma unroll
            for (int i = 0; i < 8; i += (i & 1) ? 3 : 1) order(r[i], r[i + 2], ((8 * lane + i) & size) == 0);
        }
#pragma unroll
        for (int i = 0; i < 8; i += 2) order(r[i], r[i + 1], ((8 * lane + i) & size) == 0);
    }
}

// edge_of and keep by one warp; at least K entries are known to reach the value `reached`.
__device__ __forceinline__ int cut_warp(uint32_t *hist, uint64_t *buf, int n, int K, int slack, uint32_t reached) {
    const int lane = threadIdx.x & 31;
    uint32_t lo32 = 0xffffffffu, hi32 = 0;
#pragma unroll 4
    for (int i = lane; i < n; i += 32) {
        const uint32_t v = (uint32_t)(buf[i] >> 32);
        lo32 = min(lo32, v);
        hi32 = max(hi32, v);
    }
    lo32 = max(reached, __reduce_min_sync(0xffffffffu, lo32));
    hi32 = __reduce_max_sync(0xffffffffu, hi32);
    uint64_t lo = (uint64_t)lo32 << 32;
    int shift = first_shift(lo32, hi32), bits = 8;
    uint32_t need = (uint32_t)K;
#pragma unroll 1
    while (true) {
        uint4 *bins = reinterpret_cast<uint4 *>(hist);
        bins[lane] = bins[lane + 32] = make_uint4(0, 0, 0, 0);
        __syncwarp();
#pragma unroll 4
        for (int i = lane; i < n; i += 32) {
            const uint64_t e = buf[i], d = (e - lo) >> shift;
            if (e >= lo && (d >> bits) == 0) atomicAdd(&hist[(uint32_t)d], 1u);
        }
        __syncwarp();
        uint32_t digit, before, inside;
        const int from = __ffs(__ballot_sync(0xffffffffu, find_bin(hist, need, &digit, &before, &inside))) - 1;
        lo += (uint64_t)__shfl_sync(0xffffffffu, digit, from) << shift;
        need -= __shfl_sync(0xffffffffu, before, from);
        if (shift == 0 || __shfl_sync(0xffffffffu, inside, from) - need <= (uint32_t)slack) break;
        bits = min(8, shift);
        shift -= bits;
    }
    int held = 0;
#pragma unroll 1
    for (int b = 0; b < n; b += 32) {
        const uint64_t e = b + lane < n ? buf[b + lane] : 0;
        const bool take = e != 0 && e >= lo;
        const uint32_t votes = __ballot_sync(0xffffffffu, take);
        if (take) buf[held + __popc(votes & ((1u << lane) - 1))] = e;
        held += __popc(votes);
    }
    __syncwarp();
    return held;
}

// Places for n entries, so many that a cut to them needs few looks: a power of two.
__device__ __forceinline__ int places(int K) {
    int n2 = 32;
    while (n2 < K + (K <= 224 ? K / 8 : 0)) n2 *= 2;
    return n2;
}

// Units are counted in 32 bits: 2^31 of them are 16 TiB of logits.
struct Layout {
    int units_per_row;  // ceil(V / entries of a unit)
    int units;          // of all rows
    int ctas;
    bool whole;         // every CTA's share is whole rows
    int pieces;             // most CTAs that share a row
};

// The units of CTA b: [b * units / ctas, (b + 1) * units / ctas), or so many rows.
__host__ __device__ __forceinline__ int share_begin(const Layout &l, int b) {
    if (l.whole) return (int)((int64_t)b * (l.units / l.units_per_row) / l.ctas) * l.units_per_row;
    return (int)((int64_t)b * l.units / l.ctas);
}
// The CTA that holds unit s.
__device__ __forceinline__ int share_of(const Layout &l, int s) {
    int b = (int)((int64_t)s * l.ctas / l.units);
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

// The K > kFew largest of the n entries of a whole row, from the largest down, to the row's outputs.
// THREADS threads.
template <int THREADS>
__device__ __noinline__ void write_many(Select &se, uint64_t *buf, uint32_t *count, int n, const RowTopKArgs &a,
                                        int row) {
    const int tid = threadIdx.x % THREADS, n2 = places(a.K);
    if (n > n2) {
        keep<THREADS>(se, buf, count, n, edge_of<THREADS>(se, buf, n, a.K, n2 - a.K));
        n = (int)*(volatile uint32_t *)count;
    }
    for (int i = n + tid; i < n2; i += THREADS) buf[i] = 0;
    sync<THREADS>();
    sort_entries(buf, n2, tid, THREADS, []() { sync<THREADS>(); });
    for (int k = tid; k < a.K; k += THREADS) write_entry(a, row, k, buf[k]);
}

struct Shared {
    uint64_t buf[kBuffers][kBuffer];
    uint32_t hist[kFinish][256];  // the finishing warps'
    Select sel;                   // the filtering warps'
    uint64_t full[kStages], empty[kStages];
    uint64_t given[kBuffers], taken[kBuffers];
    MaxSum state[kBuffers][kFolds];  // the folding warps'
    uint32_t edge[kFilter];      // values that so many of each filtering warp has seen reach
    uint16_t list[kFilter][32 * kTileVecs + 32];
    uint32_t reached[kBuffers];  // a value that K entries of the buffer reach
    uint32_t count[kBuffers];
    int got, abort_flag;
};

template <bool LSE>
struct Roles {
    static constexpr int kFold = LSE ? kFolds : 0, fold = kFilter, finish = fold + kFold,
                         loader = finish + kFinish, kAll = 32 * (loader + 1);
};

// MANY: K > kFew, and the filtering warps put a whole row's candidates in order.
template <typename T, bool LSE, bool MANY>
__global__ void __launch_bounds__(Roles<LSE>::kAll, kPerSm)
    topk_pieces_kernel(const RowTopKArgs a, const Layout lay, void *ws) {
    using W = Roles<LSE>;
    constexpr int N = Vec<T>::N;
    constexpr int kUnit = kUnitBytes / sizeof(T), kUnitVecs = kUnitBytes / 16;
    extern __shared__ __align__(128) unsigned char ring[];
    Shared &sh = *reinterpret_cast<Shared *>(ring + kStages * kTileBytes);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int V = (int)a.V, nv = V / N;  // entries, and vectors that bulk copies bring
    const int begin = share_begin(lay, blockIdx.x), end = share_begin(lay, blockIdx.x + 1);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), kFilter + W::kFold);
        }
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(smem_u32(&sh.given[i]), kFilter + W::kFold);
            mbar_init(smem_u32(&sh.taken[i]), 1);
            sh.count[i] = 0;
        }
        sh.abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    grid_launch_dependents();

    // A wait that gives up sets the abort flag and the error word; every role goes on to its end all the
    // same, over what the stages happen to hold, and waits no more.
    auto wait = [&](uint64_t &bar, uint32_t parity) { ring_wait(smem_u32(&bar), parity & 1, &sh.abort_flag); };
    auto arrive = [&](uint64_t &bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar));
    };
    const float c = kLog2e / a.T;
    const int limit = cut_limit(a.K), slack = cut_slack(a.K);
    const MaxSum none{-INFINITY, 0.0f};
    const uint4 low = make_uint4(Vec<T>::kLow, Vec<T>::kLow, Vec<T>::kLow, Vec<T>::kLow);
    // the stage, and the piece with its buffer
    int slot = 0, b = 0;
    uint32_t use = 0, turn = 0;
    auto next_stage = [&]() {
        if (++slot == kStages) {
            slot = 0;
            ++use;
        }
    };
    auto next_piece = [&]() {
        if (++b == kBuffers) {
            b = 0;
            ++turn;
        }
    };
    int row = begin / lay.units_per_row, u0 = begin - row * lay.units_per_row;

    if (warp == W::loader) {
        // ------------------------------------------------------------ loader
        if (lane != 0) return;
        const uint64_t policy = l2_policy_evict_first();
        bool ok = true;
#pragma unroll 1
        for (int s = begin; s < end && ok; ++row, u0 = 0) {
            const int n = min(end - s, lay.units_per_row - u0);
            s += n;
            const T *x = static_cast<const T *>(a.logits) + row * a.ldl + (int64_t)u0 * kUnit;
            int left = min(n * kUnitVecs, nv - u0 * kUnitVecs);  // vectors
#pragma unroll 1
            for (int u = 0; u < n; u += kTileUnits) {
                if (use > 0) ok = ring_wait(smem_u32(&sh.empty[slot]), (use - 1) & 1, &sh.abort_flag);
                if (!ok) break;
                const uint32_t bytes = (uint32_t)max(0, min(left, kTileUnits * kUnitVecs)) * 16u;
                const uint32_t bar = smem_u32(&sh.full[slot]);
                mbar_arrive_expect_tx(bar, bytes);
                if (bytes) bulk_load(smem_u32(ring + slot * kTileBytes), x, bytes, bar, policy);
                x += kTileUnits * kUnit;
                left -= kTileUnits * kUnitVecs;
                next_stage();
            }
        }
        // a CTA that gave up leaves only after its copies in flight have landed
        if (!ok)
            for (int k = 0; k < kStages; ++k) {
                const uint32_t issued = use + (k < slot ? 1 : 0);
                if (issued > 0) drain_wait(smem_u32(&sh.full[k]), (issued - 1) & 1);
            }
    } else if (warp < W::fold) {
        // ------------------------------------------------------------ filtering warps
        const int tid = threadIdx.x;
        // The first threshold and its successors: of m warps each finds a value that want of the maxima of
        // its groups of vectors reach.
        const int m = min(kFilter, a.K), want = (a.K + m - 1) / m;
        uint32_t *count = nullptr;
        // An entry is a candidate above `threshold`, or above `tied` (of which one equal to the threshold is
        // above) in a tile that is not behind the last entry kept by a cut.
        float threshold = 0.0f, tied = 0.0f;
        int last_kept = 0;
        auto crowded = [&]() { return *(volatile uint32_t *)count > (uint32_t)limit; };
        // The number below the key's (below 0 is not -0), and below -inf a NaN, which no entry is not above.
        auto under = [](uint32_t key) { return key_value(key - (key == order_key(0.0f) ? 2 : 1)); };
        // All filtering warps; whether any has more to look at.  Cuts the buffer where it is crowded.
        auto meet = [&](bool more) {
            more = sync_or(more);
            if (tid == 0) sh.got = (int)*(volatile uint32_t *)count;
            sync<kThreads>();
            const int got = min(sh.got, kBuffer);
            if (got > limit) {
                keep<kThreads>(sh.sel, sh.buf[b], count, got, edge_of<kThreads>(sh.sel, sh.buf[b], got, a.K, slack));
                const uint32_t key = (uint32_t)(sh.sel.least >> 32);
                threshold = key_value(key);
                tied = under(key);
                last_kept = (int)(0xffffffffu - (uint32_t)sh.sel.least);
            }
            return more;
        };
#pragma unroll 1
        for (int s = begin; s < end; ++row, u0 = 0, next_piece()) {
            const int n = min(end - s, lay.units_per_row - u0);
            s += n;
            count = &sh.count[b];
            if (turn > 0) wait(sh.taken[b], turn - 1);
            float group[kTileVecs];  // the largest so far of the tiles' vectors at a place
            uint32_t edge = 0;
#pragma unroll
            for (int j = 0; j < kTileVecs; ++j) group[j] = -INFINITY;
#pragma unroll 1
            for (int u = 0; u < n; u += kTileUnits, next_stage()) {
                // (a warp at a meeting may be the one that keeps the stage from being filled)
                unsigned long long t0 = 0;
#pragma unroll 1
                while (!__all_sync(0xffffffffu, mbar_try_wait(smem_u32(&sh.full[slot]), use & 1))) {
                    if (u > 0 && __any_sync(0xffffffffu, crowded())) meet(true);
                    const unsigned long long now = globaltimer_ns();
                    if (t0 == 0) t0 = now;
                    if (now - t0 > kWaitLimitNs) {
                        *(volatile int *)&sh.abort_flag = 1;
                        record_timeout();
                    }
                    if (__any_sync(0xffffffffu, *(volatile int *)&sh.abort_flag)) break;
                }
                const uint4 *stage = reinterpret_cast<const uint4 *>(ring + slot * kTileBytes);
                const int first = (u0 + u) * kUnit;
                const int vecs = max(0, min(min(kTileUnits, n - u) * kUnitVecs, nv - (u0 + u) * kUnitVecs));
                float largest[kTileVecs];  // -inf where there is no vector
#pragma unroll
                for (int j = 0; j < kTileVecs; ++j) {
                    const uint4 v[1] = {stage[tid + j * kThreads]};  // (what lies behind the vectors is left out)
                    largest[j] = tid + j * kThreads < vecs ? Vec<T>::largest(v) : -INFINITY;
                    group[j] = fmaxf(group[j], largest[j]);
                }
                const int tiles = u / kTileUnits + 1;
                if ((tiles & (tiles - 1)) == 0 || u + kTileUnits >= n) {
                    // Each time the data has doubled, and at its end: between the last edge, which enough groups reach, and
                    // the largest of all, by halves until not many more reach it.
                    float most = group[0], least = group[0];
#pragma unroll
                    for (int j = 1; j < kTileVecs; ++j) {
                        most = fmaxf(most, group[j]);
                        least = fminf(least, group[j]);
                    }
                    // (as many as there are lanes reach the least of the lanes' largest)
                    uint32_t lo = max(edge, __reduce_min_sync(0xffffffffu, order_key(want <= 32 ? most : least)));
                    uint32_t hi = __reduce_max_sync(0xffffffffu, order_key(most)) + 1;
#pragma unroll 1
                    while (hi - lo > 1) {
                        const uint32_t mid = lo + (hi - lo) / 2;
                        const float bar = key_value(mid);
                        int reach = 0;
#pragma unroll
                        for (int j = 0; j < kTileVecs; ++j) reach += group[j] >= bar;
                        reach = __reduce_add_sync(0xffffffffu, reach);
                        if (reach >= want) {
                            lo = mid;
                            if (reach <= want + want / 4 + 1) break;
                        } else {
                            hi = mid;
                        }
                    }
                    edge = lo;
                    if (lane == 0) *(volatile uint32_t *)&sh.edge[warp] = edge;
                    if (u == 0) {
                        sync<kThreads>();
                        threshold = tied = __int_as_float(0x7fc00000);  // NaN: every entry is a candidate
                        last_kept = -1;
                    }
                    // the m-th largest of the warps' edges; from the second time on some may be old ones, which
                    // are lower
                    uint32_t of_warps = *(volatile uint32_t *)&sh.edge[lane & (kFilter - 1)];
                    uint32_t at_least = __reduce_min_sync(0xffffffffu, of_warps);
                    if (m < kFilter) {
#pragma unroll 1
                        for (int i = 0; i < m; ++i) {
                            at_least = __reduce_max_sync(0xffffffffu, of_warps);
                            const int from = __ffs(__ballot_sync(0xffffffffu, of_warps == at_least)) - 1;
                            if ((lane & (kFilter - 1)) == from) of_warps = 0;
                        }
                    }
                    if (tid == 0) sh.reached[b] = at_least;
                    threshold = fmaxf(threshold, under(at_least));  // (a NaN is not the larger)
                    tied = fmaxf(tied, under(at_least));
                }
                const float above = first > last_kept ? threshold : tied;
                // the warp's vectors with a candidate, and the row's last V % N entries, which no copy brings
                uint16_t *list = sh.list[warp];
                int looks = 0;
                auto add = [&](bool hit, int id) {
                    const uint32_t votes = __ballot_sync(0xffffffffu, hit);
                    if (hit) list[looks + __popc(votes & ((1u << lane) - 1))] = (uint16_t)id;
                    looks += __popc(votes);
                };
#pragma unroll
                for (int j = 0; j < kTileVecs; ++j)
                    add(!(largest[j] <= above) && tid + j * kThreads < vecs, 32 * j + lane);
                if (u + kTileUnits >= n && u0 + n == lay.units_per_row) add(tid < V - nv * N, 32 * kTileVecs + lane);
                __syncwarp();
                uint64_t *to = sh.buf[b];
#pragma unroll 1
                for (int i = lane; i - lane < looks; i += 32) {
                    bool left = i < looks;
                    const int id = left ? list[i] : 0;
                    // (again after a meeting, where the buffer was full)
#pragma unroll 1
                    while (__any_sync(0xffffffffu, left)) {
                        const float bar = first > last_kept ? threshold : tied;
                        bool full = false;
                        if (left) {
                            const T *x;
                            uint32_t mask = 0;
                            int index;
                            if (id < 32 * kTileVecs) {
                                const int v = 32 * warp + id % 32 + id / 32 * kThreads;
                                x = reinterpret_cast<const T *>(stage + v);
                                index = first + v * N;
                                f32x2 p[N / 2];
                                Vec<T>::pairs(stage[v], p);
#pragma unroll
                                for (int e = 0; e < N / 2; ++e) {
                                    float f, g;
                                    unpair(p[e], f, g);
                                    mask |= (f <= bar ? 0u : 1u << (2 * e)) | (g <= bar ? 0u : 2u << (2 * e));
                                }
                            } else {
                                index = nv * N + id % 32;
                                x = static_cast<const T *>(a.logits) + row * a.ldl + index;
                                mask = to_f32(*x) <= bar ? 0 : 1;
                            }
                            const int mine = __popc(mask);
                            int at = (int)atomicAdd(count, (uint32_t)mine);
                            left = full = at + mine > kBuffer;
#pragma unroll 1
                            for (; mask; mask &= mask - 1, ++at) {
                                const int e = __ffs(mask) - 1;
                                if (at < kBuffer) to[at] = full ? 0 : entry(to_f32(x[e]), (uint32_t)(index + e));
                            }
                        }
                        __syncwarp();
                        if (__any_sync(0xffffffffu, full)) meet(true);
                    }
                }
                arrive(sh.empty[slot]);
                if (__any_sync(0xffffffffu, crowded())) meet(true);
            }
            while (meet(false)) {}
            if (MANY && n == lay.units_per_row) {
                const int got = min((int)*(volatile uint32_t *)count, kBuffer);
                sync<kThreads>();  // every thread has read the count
                write_many<kThreads>(sh.sel, sh.buf[b], count, got, a, row);
            }
            arrive(sh.given[b]);
        }
    } else if (LSE && warp < W::finish) {
        // ------------------------------------------------------------ folding warps
        const int tid = threadIdx.x - 32 * W::fold;
#pragma unroll 1
        for (int s = begin; s < end; ++row, u0 = 0, next_piece()) {
            const int n = min(end - s, lay.units_per_row - u0);
            s += n;
            MaxSum st = none;
#pragma unroll 1
            for (int u = 0; u < n; u += kTileUnits, next_stage()) {
                wait(sh.full[slot], use);
                const uint4 *stage = reinterpret_cast<const uint4 *>(ring + slot * kTileBytes);
                const int vecs = max(0, min(min(kTileUnits, n - u) * kUnitVecs, nv - (u0 + u) * kUnitVecs));
#pragma unroll 1
                for (int v0 = tid; v0 - tid < vecs; v0 += 32 * W::kFold * kVecs) {
                    uint4 in[kVecs];
#pragma unroll
                    for (int j = 0; j < kVecs; ++j)
                        in[j] = v0 + j * 32 * W::kFold < vecs ? stage[v0 + j * 32 * W::kFold] : low;
                    fold_vecs<T>(st, in, c);
                }
                arrive(sh.empty[slot]);
                if (u + kTileUnits >= n && u0 + n == lay.units_per_row && tid < V - nv * N) {
                    const float one[1] = {to_f32(static_cast<const T *>(a.logits)[row * a.ldl + nv * N + tid])};
                    fold(st, one, c);
                }
                __syncwarp();
            }
            st = warp_merge(st, c);
            if (turn > 0) wait(sh.taken[b], turn - 1);
            if (lane == 0) sh.state[b][warp - W::fold] = st;
            arrive(sh.given[b]);
        }
    } else {
        // ------------------------------------------------------------ finishing warps, a piece each in turn
        const int me = warp - W::finish;
#pragma unroll 1
        for (int s = begin; s < end; ++row, u0 = 0, next_piece()) {
            const int units = min(end - s, lay.units_per_row - u0);
            s += units;
            if ((kBuffers * turn + b) % kFinish != me) continue;
            wait(sh.given[b], turn);
            uint64_t *buf = sh.buf[b];
            int n = min((int)sh.count[b], kBuffer);
            const bool whole = units == lay.units_per_row;
            const int n2 = places(a.K), most = !whole ? a.K + slack : MANY ? kBuffer : n2;
            if (n > most) n = cut_warp(sh.hist[me], buf, n, a.K, most - a.K, sh.reached[b]);
            if (!whole) {
                const int piece = (int)blockIdx.x - share_of(lay, row * lay.units_per_row);
                uint64_t *out = piece_entries(ws, lay, a.R, a.K, row, piece);
                for (int k = lane; k < most; k += 32) out[k] = k < n ? buf[k] : 0;
                if (LSE) {
                    const MaxSum st = warp_merge(lane < kFolds ? sh.state[b][lane] : none, c);
                    if (lane == 0) *piece_state(ws, lay, row, piece) = st;
                }
            } else {
                if (!MANY && n2 <= kRanked) {
                    uint64_t r[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) r[i] = 8 * lane + i < n ? buf[8 * lane + i] : 0;
                    sort_warp(r, n2);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (8 * lane + i < a.K) write_entry(a, row, 8 * lane + i, r[i]);
                } else if (!MANY) {
                    for (int i = n + lane; i < n2; i += 32) buf[i] = 0;
                    __syncwarp();
                    sort_entries(buf, n2, lane, 32, []() { __syncwarp(); });
                    for (int k = lane; k < a.K; k += 32) write_entry(a, row, k, buf[k]);
                }
                if (LSE) {
                    const MaxSum st = warp_merge(lane < kFolds ? sh.state[b][lane] : none, c);
                    if (lane == 0) a.lse[row] = row_lse(st, a.T);
                }
            }
            __syncwarp();
            if (lane == 0) sh.count[b] = 0;
            arrive(sh.taken[b]);
        }
    }
}

struct MergeShared {
    uint64_t buf[kMergeBuffer];
    Select sel;
    uint32_t count;
};

// Takes the K largest of a split row's candidates.
template <bool LSE>
__global__ void __launch_bounds__(kMergeThreads) topk_merge_kernel(const RowTopKArgs a, const Layout lay, void *ws) {
    __shared__ __align__(16) MergeShared sh;
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, K = a.K;
    // block b stands for the boundary between the shares b and b + 1; the first one in a row merges it
    const int at = share_begin(lay, blockIdx.x + 1), row = at / lay.units_per_row, start = row * lay.units_per_row;
    if (at == start || share_begin(lay, blockIdx.x) > start) return;
    const int first = blockIdx.x;
    const int last = share_of(lay, start + lay.units_per_row - 1);
    const int total = (last - first + 1) * (K + cut_slack(K));
    const uint64_t *in = piece_entries(ws, lay, a.R, K, row, 0);
    uint64_t least = 0;
    if (tid == 0) sh.count = 0;
    sync<kMergeThreads>();
    // as many at once as the buffer takes; what lies below the K-th largest so far is passed over
#pragma unroll 1
    for (int e0 = 0; e0 < total;) {
        const int n = min(kMergeBuffer - (int)sh.count, total - e0);
        sync<kMergeThreads>();
#pragma unroll 4
        for (int i = tid; i < n; i += kMergeThreads) {
            const uint64_t e = in[e0 + i];
            if (e >= least && e != 0) sh.buf[atomicAdd(&sh.count, 1u)] = e;
        }
        sync<kMergeThreads>();
        e0 += n;
        const int got = (int)sh.count;
        sync<kMergeThreads>();
        const int most = e0 < total ? K + cut_slack(K) : max(K, min(kRanked, 2 * K + 32));
        if (got > most) {
            least = edge_of<kMergeThreads>(sh.sel, sh.buf, got, K, most - K);
            keep<kMergeThreads>(sh.sel, sh.buf, &sh.count, got, least);
        }
    }
    const int n = (int)sh.count;
    if (n <= kRanked) {
        // an entry's place is the number of larger ones
#pragma unroll 1
        for (int k = tid; k < n; k += kMergeThreads) {
            const uint64_t e = sh.buf[k];
            int place = 0;
#pragma unroll 4
            for (int i = 0; i < n; ++i) place += sh.buf[i] > e;
            if (place < K) write_entry(a, row, place, e);
        }
    } else {
        int n2 = 2 * kRanked;
        while (n2 < n) n2 *= 2;
        for (int i = n + tid; i < n2; i += kMergeThreads) sh.buf[i] = 0;
        sync<kMergeThreads>();
        sort_entries(sh.buf, n2, tid, kMergeThreads, []() { sync<kMergeThreads>(); });
        for (int k = tid; k < K; k += kMergeThreads) write_entry(a, row, k, sh.buf[k]);
    }
    if (LSE && tid < 32) {
        const float c = kLog2e / a.T;
        MaxSum st{-INFINITY, 0.0f};
        for (int p = lane; p <= last - first; p += 32) merge(st, *piece_state(ws, lay, row, p), c);
        st = warp_merge(st, c);
        if (lane == 0) a.lse[row] = row_lse(st, a.T);
    }
}

constexpr size_t kDynamic = kStages * kTileBytes + sizeof(Shared);

// The deal of the rows' units over the device's CTAs.
bool layout(int64_t R, int64_t V, int K, int dtype, Layout *l) {
    const int sms = device_sm_count();
    if (sms <= 0) return false;
    const int64_t unit = kUnitBytes / element_size(dtype);
    const int64_t per_row = (V + unit - 1) / unit, units = R * per_row;
    if (!row_topk_fits(R, V, dtype)) return false;
    l->units_per_row = (int)per_row;
    l->units = (int)units;
    // a piece of a row costs a selection and K candidates to merge: no fewer than kMinUnits units,
    // nor than 8 K entries (but a row is never too little for a CTA)
    const int64_t least = max((int64_t)kMinUnits, (8 * (int64_t)K + unit - 1) / unit);
    const int64_t want = max((units + least - 1) / least, R);
    l->ctas = (int)max((int64_t)1, min((int64_t)sms * kPerSm, want));
    // Whole rows, or shares as even as can be: what the longest share of whole rows has beyond an even one
    // (and 64 KB more a row, what a row costs whatever its length), against the second kernel and the pieces
    // that even shares add: as much as reading 120 KB.  1,000 x 50,001 bf16, K = 200: 57.0 us whole, 60.5 in
    // even shares; 400 x 50,001 fp32, K = 64: 39.6 and 36.7.
    const int64_t most = (R + l->ctas - 1) / l->ctas, row_bytes = per_row * kUnitBytes;
    l->whole = (most * l->ctas - R) * (row_bytes + 64 * 1024) <= (int64_t)l->ctas * 120 * 1024;
    const int share = l->units / l->ctas;  // every CTA has at least this
    l->pieces = min((l->units_per_row + share - 1) / share + 1, l->units_per_row);
    return true;
}

template <typename T, bool LSE, bool MANY>
cudaError_t launch(const RowTopKArgs &a, const Layout &lay, void *ws, cudaStream_t stream) {
    const void *fn = (const void *)topk_pieces_kernel<T, LSE, MANY>;
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
    topk_pieces_kernel<T, LSE, MANY><<<(unsigned)lay.ctas, Roles<LSE>::kAll, kDynamic, stream>>>(a, lay, ws);
    e = cudaGetLastError();
    // no row is shared where every CTA's share is whole rows
    if (e != cudaSuccess || lay.whole || lay.ctas == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(lay.ctas - 1));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, topk_merge_kernel<LSE>, a, lay, ws);
}

template <typename T, bool LSE>
cudaError_t launch(const RowTopKArgs &a, const Layout &lay, void *ws, cudaStream_t stream) {
    return a.K > kFew ? launch<T, LSE, true>(a, lay, ws, stream) : launch<T, LSE, false>(a, lay, ws, stream);
}

}  // namespace

bool row_topk_fits(int64_t R, int64_t V, int dtype) {
    const int64_t unit = kUnitBytes / element_size(dtype);
    return R * ((V + unit - 1) / unit) <= INT32_MAX;
}

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
