// The embedding table's rows at a canvas' tokens, and the table's gradient from that of the rows.
//
//   out[r] = gamma s_t W[t - vocab_start],  t = token[r] in [vocab_start, vocab_end), else 0
//   gW[v] (+)= gamma sum over {r : token[r] = v} of g[r]
//
// Forward: a gather, bound by HBM (a table row and an output row per position) and by latency where there
// are few positions: 16 positions of 256 columns 1.65 us, 8,192 bf16 rows of 2,816 from E4M3 codes 13.5 us (69 MB, 5.1 TB/s).
//
// Backward: the positions are put in order of their tokens, equal ones by position, so that every table row is
// written once, from its positions in order: no atomics on values, results repeat bit for bit.  The order is found in
// runs, by counting or by a radix sort in shared memory (sort_tokens says when), that are merged by search; a
// radix sort by a cluster took 20 us and more, its passes waiting on barriers and scattered stores.  The sorted
// positions are cut into units of up to 32; a warp takes a unit and 256 columns.  A token that ends within the next unit
// is finished by the warp it began in.  One that covers a whole unit and its neighbours (a mask or padding token)
// leaves one fp32 part per unit, and a last kernel adds its parts in order.  Up to kFewRows positions one kernel does
// all of it, every CTA for a few columns of all positions, the parts in shared memory.  The kernels of a call start
// while the one before them ends; the order is found while the gradient is cleared.
//
// Clearing is bound by HBM: 262,144 x 2,816 bf16 and 8,192 positions 228 us, 6.7 TB/s.  Without it the sums are bound by the
// latency of their loads, and the call by the four kernels that wait for one another: 20,001 positions of 1,001 41 us, of
// them some 21 the sums.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "dg_internal.h"
#include "hidden.cuh"

namespace dg {

namespace {

using namespace hidden;

constexpr unsigned int kIndexRange = 2u;  // the device error word's bit for a token past the vocabulary

// ---------------------------------------------------------------- forward

constexpr int kGatherThreads = 256;

struct GatherParams {
    EmbedRows a;
    int lanes;  // threads of a row
};

template <typename TT, typename TO, bool kWide>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const GatherParams p) {
    const EmbedRows &a = p.a;
    const int per_cta = kGatherThreads / p.lanes;
    const int lane = threadIdx.x % p.lanes;
    const int d = (int)a.d, last = (d - 1) / 8 * 8;
    constexpr int kAhead = kWide ? 32 / (2 * sizeof(TT)) < 12 ? 32 / (2 * sizeof(TT)) : 12 : 2;  // loads in flight
    for (int64_t r = (int64_t)blockIdx.x * per_cta + threadIdx.x / p.lanes; r < a.R; r += (int64_t)gridDim.x * per_cta) {
        const int64_t t = a.token[r];
        const bool on = t >= a.vocab_start && t < a.vocab_end;
        if (t >= a.V && lane == 0) atomicOr(&g_device_error, kIndexRange);
        const TT *src = static_cast<const TT *>(a.table.p) + (on ? (t - a.vocab_start) * a.table.ld : 0);
        const float f = on && a.scale ? a.scale[t - a.vocab_start] : 1.0f;
        TO *dst = static_cast<TO *>(a.rows.p) + r * a.rows.ld;
        const int step = kWide ? 1 : p.lanes;  // between a thread's eight columns
        for (int c0 = kWide ? 8 * lane : lane; c0 < d; c0 += kAhead * 8 * p.lanes) {
            Raw8<TT> raw[kAhead];
            if (on)
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {  // (past the row's end its last columns again)
                    const int c = kWide ? min(c0 + i * 8 * p.lanes, last) : c0 + i * 8 * p.lanes;
                    load8<kWide>(raw[i], src + c, d - c, step);
                }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int c = c0 + i * 8 * p.lanes;
                if (c >= d) break;
                float v[8];
                if (on) {
                    unpack8(v, raw[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = v[j] * f * a.gamma;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
                }
                store8<kWide>(dst + c, v, d - c, step);
            }
        }
    }
}

template <typename TT, typename TO>
void gather_wide(const GatherParams &p, unsigned grid, cudaStream_t stream) {
    if (wide_rows(p.a.table) && wide_rows(p.a.rows))
        gather_kernel<TT, TO, true><<<grid, kGatherThreads, 0, stream>>>(p);
    else
        gather_kernel<TT, TO, false><<<grid, kGatherThreads, 0, stream>>>(p);
}
template <typename TT>
void gather_out(const GatherParams &p, unsigned grid, cudaStream_t stream) {
    if (p.a.rows.dtype == DG_F32)
        gather_wide<TT, float>(p, grid, stream);
    else
        gather_wide<TT, __nv_bfloat16>(p, grid, stream);
}

// ---------------------------------------------------------------- the order of the tokens

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 8, kMaxBins = 1 << kDigitBits;
// Up to kSortMost positions are ordered in runs, which are then merged; more by a cluster of kSortCtas (the largest size that
// every device takes).  Frequencies of text, bf16 of 512 columns added to fp32: 65,536 positions 61.6 us and by the cluster 81.4,
// 131,072 107 and 133, 262,144 234 and 237, 524,288 574 and 436; so the limit errs low by a factor of four.
constexpr int kSortMost = 65536;
constexpr int kSortCtas = 8;

// Where everything lies in the workspace.
struct SortSpace {
    int32_t *key[2], *pos[2];  // sorted: [0]; [1]: the runs, or between passes
    int2 *list;                // (unit, key) of the tokens that leave parts
    int32_t *count;
    float *parts;              // [unit][0: begun before it, 1: begun in it][part_ld]
    int64_t part_ld;
};

struct SortParams {
    const int32_t *token;
    int64_t V, vocab_start, vocab_end;
    int32_t R, none;  // none: the key of a position without a table row, above all others
    int run;          // positions that are ordered together
    int passes, bits;
    SortSpace s;
};

__device__ __forceinline__ int32_t key_of(const SortParams &p, int64_t t) {
    if (t >= p.V) atomicOr(&g_device_error, kIndexRange);
    return t >= p.vocab_start && t < p.vocab_end ? (int32_t)(t - p.vocab_start) : p.none;
}

__device__ __forceinline__ int32_t token_key(const SortParams &p, int64_t i) { return key_of(p, p.token[i]); }

// The keys of n positions from `first` on, with the largest number up to the next multiple of four.
__device__ __forceinline__ void gather_keys(const SortParams &p, int first, int n, int32_t *keys) {
    constexpr int kAhead = 8;  // loads in flight
    const int padded = (n + 3) / 4 * 4;
    for (int i0 = threadIdx.x; i0 < padded; i0 += kAhead * blockDim.x) {
        int32_t t[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * blockDim.x;
            t[j] = i < n ? p.token[first + i] : 0;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * blockDim.x;
            if (i < padded) keys[i] = i < n ? key_of(p, t[j]) : INT32_MAX;
        }
    }
}

// Inclusive sum over the lanes.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += o;
    }
    return v;
}

__device__ __forceinline__ uint32_t cluster_load(const void *local, uint32_t cta) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_cta(smem_u32(local), cta)) : "memory");
    return v;
}
// The order of positions by counting: a position's place is the number of positions before it, those with a smaller
// key and those before it with the same one.  q of T threads per position i compare it with every T-th four of the
// keys (`keys`, up to the next multiple of four past R filled with the largest number); all T get the sum.
template <int T>
__device__ __forceinline__ int count_before(const int32_t *keys, int R, int i, int q) {
    const int32_t k = keys[i];
    const int4 *fours = reinterpret_cast<const int4 *>(keys);
    const int own = i / 4, all = (R + 3) / 4;
    int n = 0, g = q;
    // equal keys count where they come earlier (k < 2^31 - 1)
#pragma unroll 4
    for (; g < own; g += T) {
        const int4 o = fours[g];
        n += (o.x <= k) + (o.y <= k) + (o.z <= k) + (o.w <= k);
    }
    if (g == own) {
        const int4 o = fours[g];
        n += (o.x < k || (o.x == k && i % 4 > 0)) + (o.y < k || (o.y == k && i % 4 > 1)) +
             (o.z < k || (o.z == k && i % 4 > 2)) + (o.w < k);
        g += T;
    }
#pragma unroll 4
    for (; g < all; g += T) {
        const int4 o = fours[g];
        n += (o.x < k) + (o.y < k) + (o.z < k) + (o.w < k);
    }
#pragma unroll
    for (int off = 1; off < T; off <<= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
    return n;
}

// By one CTA, up to kFewRows positions.  A gradient that is added to, fp32 (V = 32,000, d = 512; with the limit at 256 and at 512):
// 256 positions 8.4 us and 9.3, 512 11.0 and 13.7 (1,024 threads leave 64 registers each: the kernels that add spill 90 to 180
// bytes a thread, and 24 of the 32 warps only help to find the order).  A cleared one finds the order under the clearing, and one kernel in place of
// three follows it, so that up to 512 one kernel is as fast or faster: 300 positions 22.1 us for 26.2, 512 25.6 for 26.8; 300 of
// 1,001 34.1 for 39.3; of 2,816 over 262,144 bf16 rows 208 for 213; and 512 of 256 over 4,096 12.4 for 11.1 in a graph, but called
// in 14.5 for 14.7.
template <bool kAdd>
constexpr int kFewRows = kAdd ? 256 : 512;
template <int kRows>
__device__ __forceinline__ void order_few(const SortParams &p, int32_t *unsorted, int32_t *key_s, int32_t *pos_s) {
    constexpr int T = kSortThreads / kRows;
    gather_keys(p, 0, p.R, unsorted);
    __syncthreads();
    const int i = threadIdx.x / T;
    const int n = count_before<T>(unsorted, p.R, min(i, p.R - 1), threadIdx.x % T);
    if (i < p.R && threadIdx.x % T == 0) {
        key_s[n] = unsorted[i];
        pos_s[n] = i;
    }
    __syncthreads();
}

// By the whole chip, runs of p.run positions: place c of [1] takes run c, or [0] the only one.  A warp takes four
// positions at once against the keys that its lanes share out: shared memory would hold it up with one.
constexpr int kOneRun = 2048, kNearRun = 1024, kCountThreads = 512, kCountItems = kCountThreads / 32 * 4;
__global__ void __launch_bounds__(kCountThreads) count_tokens_kernel(const SortParams p) {
    __shared__ __align__(16) int32_t keys[kOneRun];
    grid_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.s.count = 0;
    const int ctas = p.run / kCountItems, first = (int)blockIdx.x / ctas * p.run, n = min(p.run, p.R - first);
    gather_keys(p, first, n, keys);
    __syncthreads();
    const int4 *fours = reinterpret_cast<const int4 *>(keys);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int all = (n + 3) / 4, own = (int)blockIdx.x % ctas * (kCountItems / 4) + warp;
    if (own < all) {
        const int4 mine = fours[own];
        const int32_t k[4] = {mine.x, mine.y, mine.z, mine.w};
        int before[4] = {0, 0, 0, 0};
#pragma unroll 4
        for (int g = lane; g < all; g += 32) {
            const int4 o = fours[g];
            const int earlier = g < own;  // equal keys count where they come earlier
            if (g == own) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int32_t t = k[q] - 1 + earlier;
                before[q] += (o.x <= t) + (o.y <= t) + (o.z <= t) + (o.w <= t);
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            int at = __reduce_add_sync(0xffffffffu, before[q]);
#pragma unroll
            for (int j = 0; j < 4; ++j) at += k[j] < k[q] || (k[j] == k[q] && j < q);
            const int i = 4 * own + q;
            if (lane == q && i < n) {
                const int to = p.R > p.run;
                p.s.key[to][first + at] = k[q];
                p.s.pos[to][first + at] = first + i;
            }
        }
    }
    // what clears the gradient has completed before this kernel has, and so before the sums begin
    grid_dependency_wait();
}

// Merges counted runs, all keys in shared memory: an item's place is its own place in its run, and in the other runs that
// of the first larger key (runs before it) or of the first one not smaller (after it).  Four threads per item share the
// other runs.
constexpr int kNearRows = 24576, kNearThreads = 512, kNearShare = 4;
__global__ void __launch_bounds__(kNearThreads) merge_near_kernel(const SortParams p) {
    extern __shared__ int4 near_fours[];
    const int32_t *keys = reinterpret_cast<const int32_t *>(near_fours);
    grid_dependency_wait();
    grid_launch_dependents();
    const int item = (int)blockIdx.x * (kNearThreads / kNearShare) + threadIdx.x / kNearShare, q = threadIdx.x % kNearShare;
    const int i = min(item, p.R - 1), own = i / kNearRun, runs = (p.R + kNearRun - 1) / kNearRun;
    const int32_t place = p.s.pos[1][i];
    const int4 *fours = reinterpret_cast<const int4 *>(p.s.key[1]);  // (whole 16 bytes each: lay_out)
    const int all = (p.R + 3) / 4;
    constexpr int kAhead = 8;
    for (int g0 = threadIdx.x; g0 < all; g0 += kAhead * kNearThreads) {
        int4 v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) v[j] = fours[min(g0 + j * kNearThreads, all - 1)];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (g0 + j * kNearThreads < all) near_fours[g0 + j * kNearThreads] = v[j];
    }
    __syncthreads();
    const int32_t k = keys[i];
    int at = q == 0 ? i - own * kNearRun : 0;
    for (int c = q; c < runs; c += kNearShare) {
        if (c == own) continue;
        const int32_t *run = keys + c * kNearRun;
        const int n = min(kNearRun, p.R - c * kNearRun), t = k + (c < own);
        int found = 0;
#pragma unroll
        for (int step = kNearRun; step > 0; step >>= 1)
            if (found + step <= n && run[found + step - 1] < t) found += step;
        at += found;
    }
#pragma unroll
    for (int off = 1; off < kNearShare; off <<= 1) at += __shfl_xor_sync(0xffffffffu, at, off);
    if (item < p.R && q == 0) {
        p.s.key[0][at] = k;
        p.s.pos[0][at] = place;
    }
}

// The lanes whose digit is this lane's; `in`: the lanes that have one.
__device__ __forceinline__ uint32_t same_digit(uint32_t digit, uint32_t in) {
    uint32_t same = in;
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b) {
        const uint32_t set = __ballot_sync(0xffffffffu, (digit >> b) & 1);
        same &= (digit >> b) & 1 ? set : ~set;
    }
    return same;
}

// Exclusive sums over the digits of this CTA's counts by digit and warp, in place, and each digit's total: 1024 / bins
// threads sum a digit's 16 pairs of counts.
constexpr int kHistPitch = kSortWarps + 2;  // (17 words: a column's rows lie in different banks)
__device__ __forceinline__ void scan_warps(uint32_t *hist, uint32_t *total, int bits) {
    const int per = min(16, kSortThreads >> bits), pairs = 16 / per;
    const int b = threadIdx.x / per, q = threadIdx.x % per;
    uint32_t *h = hist + b * (kHistPitch / 2) + q * pairs;
    uint32_t sum = 0;
    if (b < 1 << bits)
        for (int i = 0; i < pairs; ++i) sum += (h[i] & 0xFFFFu) + (h[i] >> 16);
    uint32_t upto = sum;
    for (int off = 1; off < per; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, upto, off);
        if (q >= off) upto += o;
    }
    if (b < 1 << bits) {
        uint32_t run = upto - sum;
        for (int i = 0; i < pairs; ++i) {
            const uint32_t c = h[i], mid = run + (c & 0xFFFFu);
            h[i] = run | mid << 16;
            run = mid + (c >> 16);
        }
        if (q == per - 1) total[b] = run;
    }
}

// A run of kRun positions by a stable radix sort in one CTA, least digit first, an item's key and position in
// registers and, between passes, in shared memory; a warp takes N * 32 items in a row.  Run c goes to place c of [1].
// Digits of at most 8 bits: with 10, two passes in place of three, clearing and summing the counts
// took longer than the pass that it saved.
constexpr int kRun = 4096;
__global__ void __launch_bounds__(kSortThreads) sort_run_kernel(const SortParams p) {
    constexpr int N = kRun / kSortThreads;
    __shared__ int32_t key_s[kRun], pos_s[kRun];
    __shared__ uint32_t total[kMaxBins], start[kMaxBins], warp_total[kSortWarps];
    __shared__ uint16_t hist[kMaxBins][kHistPitch];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int bins = 1 << p.bits;
    const int local0 = warp * (N * 32) + lane;  // item j of this thread: local0 + 32 j
    const int64_t first = (int64_t)blockIdx.x * kRun;
    const uint32_t lane_bit = 1u << lane;
    grid_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.s.count = 0;
    int32_t key[N], pos[N];
    uint32_t in[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int64_t i = first + local0 + 32 * j;
        pos[j] = (int32_t)i;
        key[j] = i < p.R ? token_key(p, i) : 0;
        in[j] = __ballot_sync(0xffffffffu, i < p.R);
    }
    uint32_t *h32 = reinterpret_cast<uint32_t *>(&hist[0][0]);
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * p.bits;
        for (int b = threadIdx.x; b < bins * (kHistPitch / 2); b += kSortThreads) h32[b] = 0;
        uint32_t same[N], below[N];
#pragma unroll
        for (int j = 0; j < N; ++j) same[j] = same_digit((uint32_t)(key[j] >> shift) & (bins - 1), in[j]);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint32_t dig = (uint32_t)(key[j] >> shift) & (bins - 1);
            const uint32_t less = __popc(same[j] & (lane_bit - 1));
            below[j] = hist[dig][warp] + less;
            __syncwarp();
            if ((in[j] & lane_bit) && less == 0) hist[dig][warp] += (uint16_t)__popc(same[j]);
            __syncwarp();
        }
        __syncthreads();
        scan_warps(h32, total, p.bits);
        __syncthreads();
        const uint32_t all = (int)threadIdx.x < bins ? total[threadIdx.x] : 0, sum = warp_scan(all, lane);
        if (lane == 31) warp_total[warp] = sum;
        __syncthreads();
        if (threadIdx.x < kMaxBins) {  // (whole warps)
            const uint32_t w = __reduce_add_sync(0xffffffffu, lane < warp ? warp_total[lane] : 0);
            start[threadIdx.x] = sum - all + w;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (in[j] & lane_bit) {
                const uint32_t dig = (uint32_t)(key[j] >> shift) & (bins - 1);
                const uint32_t at = start[dig] + hist[dig][warp] + below[j];
                key_s[at] = key[j];
                pos_s[at] = pos[j];
            }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (in[j] & lane_bit) {
                key[j] = key_s[local0 + 32 * j];
                pos[j] = pos_s[local0 + 32 * j];
            }
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (in[j] & lane_bit) {
            p.s.key[1][first + local0 + 32 * j] = key[j];
            p.s.pos[1][first + local0 + 32 * j] = pos[j];
        }
    // what clears the gradient has completed before this kernel has, and so before the sums begin
    grid_dependency_wait();
}

// Merges runs of kRun likewise, from global memory.
__global__ void __launch_bounds__(256) merge_runs_kernel(const SortParams p) {
    constexpr int kAtOnce = 4;  // searches
    grid_dependency_wait();
    grid_launch_dependents();
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= p.R) return;
    constexpr int run = kRun;
    const int own = i / run, runs = (p.R + run - 1) / run;
    const int32_t k = p.s.key[1][i];
    int at = i - own * run;
    for (int c0 = 0; c0 < runs; c0 += kAtOnce) {
        int lo[kAtOnce], hi[kAtOnce], below[kAtOnce];
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
            const int c = c0 + q;
            lo[q] = min(c * run, p.R);
            hi[q] = c < runs && c != own ? min((c + 1) * run, p.R) : lo[q];
            at -= lo[q];
            below[q] = c < own ? k + 1 : k;  // (k < 2^31 - 1)
        }
        for (int step = run; step > 0; step >>= 1)
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q)
                if (lo[q] < hi[q]) {
                    const int mid = (lo[q] + hi[q]) >> 1;
                    if (p.s.key[1][mid] < below[q])
                        lo[q] = mid + 1;
                    else
                        hi[q] = mid;
                }
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) at += lo[q];
    }
    p.s.key[0][at] = k;
    p.s.pos[0][at] = p.s.pos[1][i];
}

// The sort of more positions: a stable radix sort, least digit first, by one cluster through global memory (L2).
__global__ void __launch_bounds__(kSortThreads) sort_far_kernel(const SortParams p) {
    __shared__ uint32_t hist[kMaxBins][kSortWarps + 1];
    __shared__ uint32_t total[kMaxBins], start[kMaxBins], warp_total[kMaxBins / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ctas = (int)gridDim.x, rank = (int)blockIdx.x;  // one cluster
    const int bins = 1 << p.bits;
    const int per = ((p.R + ctas * kSortWarps - 1) / (ctas * kSortWarps) + 31) / 32 * 32;
    const int64_t i0 = (int64_t)(rank * kSortWarps + warp) * per;
    const int n = i0 >= p.R ? 0 : (int)min((int64_t)per, p.R - i0);
    grid_launch_dependents();
    if (rank == 0 && threadIdx.x == 0) *p.s.count = 0;

    for (int pass = 0; pass < p.passes; ++pass) {
        // an odd number of passes begins from the tokens into [0], an even one into [1]
        const int to = (p.passes - 1 - pass) & 1;
        const int shift = pass * p.bits;
        auto key_at = [&](int64_t i) { return pass > 0 ? __ldcg(p.s.key[to ^ 1] + i) : token_key(p, i); };
        for (int b = threadIdx.x; b < bins * (kSortWarps + 1); b += kSortThreads) (&hist[0][0])[b] = 0;
        __syncthreads();
        for (int i = lane; i < (n + 31) / 32 * 32; i += 32) {
            const uint32_t dig = i < n ? (uint32_t)(key_at(i0 + i) >> shift) & (bins - 1) : 0xFFFFFFFFu;
            const uint32_t same = __match_any_sync(0xffffffffu, dig);
            if (i < n && (same & ((1u << lane) - 1)) == 0) hist[dig][warp] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        for (int b = warp; b < bins; b += kSortWarps) {
            const uint32_t own = hist[b][lane], sum = warp_scan(own, lane);
            hist[b][lane] = sum - own;
            if (lane == 31) total[b] = sum;
        }
        __syncthreads();
        cluster_sync_all();
        uint32_t all = 0, before = 0;
        if ((int)threadIdx.x < bins)
            for (int c = 0; c < ctas; ++c) {
                const uint32_t t = cluster_load(&total[threadIdx.x], (uint32_t)c);
                all += t;
                if (c < rank) before += t;
            }
        const uint32_t sum = warp_scan(all, lane);
        if (warp < kMaxBins / 32 && lane == 31) warp_total[warp] = sum;
        __syncthreads();
        if ((int)threadIdx.x < bins) {
            uint32_t base = before + sum - all;
            for (int w = 0; w < warp; ++w) base += warp_total[w];
            start[threadIdx.x] = base;
        }
        __syncthreads();
        for (int i = lane; i < (n + 31) / 32 * 32; i += 32) {
            const bool in = i < n;
            const int32_t k = in ? key_at(i0 + i) : 0;
            const uint32_t dig = in ? (uint32_t)(k >> shift) & (bins - 1) : 0xFFFFFFFFu;
            const uint32_t same = __match_any_sync(0xffffffffu, dig);
            const uint32_t less = __popc(same & ((1u << lane) - 1));
            uint32_t at = 0;
            if (in) at = start[dig] + hist[dig][warp] + less;
            __syncwarp();
            if (in) {
                if (less == 0) hist[dig][warp] += __popc(same);
                p.s.key[to][at] = k;
                p.s.pos[to][at] = pass > 0 ? __ldcg(p.s.pos[to ^ 1] + i0 + i) : (int32_t)(i0 + i);
            }
            __syncwarp();
        }
        __threadfence();  // the next pass, and the next kernel, read what other CTAs wrote here
        cluster_sync_all();
        __syncthreads();
    }
    grid_dependency_wait();
}

// ---------------------------------------------------------------- the sums

constexpr int kSumWarps = 4, kSumAhead = 4;

struct SumParams {
    EmbedRows a;
    SortSpace s;
    int32_t none;
    int unit, units, slabs;  // sorted positions of a unit; slabs of 256 columns
    int unit_warps, cta_units, slab_ctas;  // warps of a unit in a CTA, units of a CTA, CTAs that share a unit's slabs
};

// What a unit [u0, u1) of sorted positions sums: [lo, hi), of which the first token's part, begun before it, goes to
// slot 0, and the last one's, going on after it, to slot 1.
struct UnitRange {
    int lo, hi;
    bool part0, part1;
};

// `key(i)` for i in [u0 - U - 1, u1 + U] gives the sorted key, or -1 where there is no position.  A token that covers a
// whole unit and both its neighbouring positions leaves parts: as its positions are consecutive, a unit sees that from
// itself, the unit before and the unit after.  A shorter one is summed by the unit it begins in.  All lanes take
// part and get the same answer.
template <typename Key>
__device__ __forceinline__ UnitRange unit_range(const Key &key, int u0, int u1, int U, int32_t none, int lane) {
    UnitRange r{u0, u1, false, false};
    auto until = [&](int i, int end, auto same) {  // the first position from i on that is not `same`, or end
        while (true) {
            const uint32_t other = __ballot_sync(0xffffffffu, i + lane >= end || !same(key(i + lane)));
            if (other) return i + __ffs(other) - 1;
            i += 32;
        }
    };
    const int32_t first = key(u0), last = key(u1 - 1);
    const bool carry = first != none && key(u0 - 1) == first;
    if (carry) {
        r.part0 = key(u0 - U - 1) == first || (u1 == u0 + U && key(u1) == first);
        if (!r.part0) r.lo = until(u0, u1, [&](int32_t k) { return k == first; });
    }
    if (last != none && key(u1) == last && !(carry && last == first)) {
        r.part1 = key(u1 + U) == last;
        if (!r.part1) r.hi = until(u1, u1 + U, [&](int32_t k) { return k == last; });
    }
    if (last == none) r.hi = until(u0, u1, [&](int32_t k) { return k != none; });
    return r;
}

// gW[key][c ..] (+)= gamma sum; old: what is there, with accumulate; step: between the eight columns without kWide
template <typename TT, bool kAdd, bool kWide>
__device__ __forceinline__ void write_row(const EmbedRows &a, int32_t key, int c, int step, const float (&sum)[8],
                                          const Raw8<TT> &old) {
    float v[8];
    if constexpr (kAdd) {
        unpack8(v, old);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += sum[j] * a.gamma;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = sum[j] * a.gamma;
    }
    store8<kWide>(static_cast<TT *>(a.table.p) + (int64_t)key * a.table.ld + c, v, (int)a.d - c, step);
}

// Sums the positions [r.lo, r.hi) of a unit in eight columns from c on: each token's to its row, parts to part(slot).
// The rows of kAhead positions are in flight at once, and with them the rows that their sums may be added to (those of
// one token's positions come from L1 but once), without a branch between the loads.
template <int kAhead, typename TG, typename TT, bool kAdd, bool kWide, typename Key, typename Pos, typename Part>
__device__ __forceinline__ void sum_unit(const EmbedRows &a, const Key &key, const Pos &pos, const Part &part, const UnitRange &r,
                                         int u0, int c, int step) {
    const int n = (int)a.d - c;
    const TG *g = static_cast<const TG *>(a.rows.p) + c;
    const TT *table = static_cast<const TT *>(a.table.p) + c;
    const int32_t first = key(u0);
    float acc[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) acc[t] = 0.0f;
    for (int i = r.lo; i < r.hi; i += kAhead) {
        Raw8<TG> raw[kAhead];
        Raw8<TT> old[kAhead];
        int32_t k[kAhead + 1];
#pragma unroll
        for (int j = 0; j <= kAhead; ++j) k[j] = i + j < r.hi ? key(i + j) : -1;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            load8<kWide>(raw[j], g + (int64_t)pos(min(i + j, r.hi - 1)) * a.rows.ld, n, step);
            if constexpr (kAdd) load8<kWide>(old[j], table + (int64_t)max(k[j], 0) * a.table.ld, n, step);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            float v[8];
            unpack8(v, raw[j]);
#pragma unroll
            for (int t = 0; t < 8; ++t) acc[t] += v[t];
            if (k[j] != k[j + 1]) {  // (at the end -1 follows the last key, and itself)
                if (r.part0 && k[j] == first)
                    part(0, acc);
                else if (r.part1 && i + j + 1 == r.hi)
                    part(1, acc);
                else
                    write_row<TT, kAdd, kWide>(a, k[j], c, step, acc, old[j]);
#pragma unroll
                for (int t = 0; t < 8; ++t) acc[t] = 0.0f;
            }
        }
    }
}

template <typename TG, typename TT, bool kAdd, bool kWide>
__global__ void __launch_bounds__(32 * kSumWarps) sum_rows_kernel(const SumParams p) {
    extern __shared__ int32_t near[];  // this CTA's keys, with a unit and one before and after, and positions
    const EmbedRows &a = p.a;
    const int U = p.unit, span = p.cta_units * U, n = span + 2 * U + 2;
    const int group = (int)blockIdx.x / p.slab_ctas, base = group * span, k0 = base - U - 1, R = (int)a.R;
    grid_dependency_wait();
    grid_launch_dependents();
    for (int i = threadIdx.x; i < n; i += blockDim.x) near[i] = k0 + i >= 0 && k0 + i < R ? p.s.key[0][k0 + i] : -1;
    for (int i = threadIdx.x; i < span + U; i += blockDim.x) near[n + i] = base + i < R ? p.s.pos[0][base + i] : 0;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m = group * p.cta_units + warp / p.unit_warps;
    if (m >= p.units) return;
    const int slab0 = (int)blockIdx.x % p.slab_ctas * p.unit_warps + warp % p.unit_warps;
    const int u0 = m * U, u1 = min(R, u0 + U);
    auto key = [&](int i) { return near[i - k0]; };
    auto pos = [&](int i) { return near[n + (i - base)]; };
    const UnitRange r = unit_range(key, u0, u1, U, p.none, lane);
    if (r.lo >= r.hi) return;
    if (r.part1 && slab0 == 0 && lane == 0) p.s.list[atomicAdd(p.s.count, 1)] = make_int2(m, key(u1 - 1));
    const int c = slab0 * 256 + (kWide ? 8 : 1) * lane, step = kWide ? 1 : 32;
    if (c < a.d)
        sum_unit<kSumAhead, TG, TT, kAdd, kWide>(a, key, pos, [&](int slot, const float (&acc)[8]) {
            store8<kWide>(p.s.parts + ((int64_t)m * 2 + slot) * p.s.part_ld + c, acc, kWide ? 8 : (int)a.d - c, step);
        }, r, u0, c, step);
}

constexpr int kJoinWarps = 8;

// Tokens that left parts: unit m's second part, then the first parts of the units after it that begin
// with the same token.  A CTA takes a token and 128 columns, its warps a share of the parts each.
template <typename TT, bool kAdd, bool kWide>
__global__ void __launch_bounds__(32 * kJoinWarps) join_parts_kernel(const SumParams p) {
    __shared__ float acc[kJoinWarps][128];
    const EmbedRows &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slabs = (int)((a.d + 127) / 128);
    grid_dependency_wait();
    const int64_t items = (int64_t)*p.s.count * slabs;
    for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int2 e = p.s.list[item / slabs];
        const int c = (int)(item % slabs) * 128 + 4 * lane;
        int n = 0;  // units after the first one
        while (true) {
            const int64_t m = (int64_t)e.x + 1 + n + threadIdx.x;
            const int more = __syncthreads_count(m < p.units && p.s.key[0][m * p.unit] == e.y);
            n += more;
            if (more < (int)blockDim.x) break;
        }
        const int per = (n + 1 + kJoinWarps - 1) / kJoinWarps;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < a.d) {
            const int last = min(n + 1, (warp + 1) * per);
#pragma unroll 4
            for (int i = warp * per; i < last; ++i) {
                const int64_t slot = ((int64_t)e.x + i) * 2 + (i == 0);
                const float4 v = *reinterpret_cast<const float4 *>(p.s.parts + slot * p.s.part_ld + c);
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
        }
        *reinterpret_cast<float4 *>(&acc[warp][4 * lane]) = s;
        __syncthreads();
        if (threadIdx.x < 16) {
            const int c8 = (int)(item % slabs) * 128 + 8 * threadIdx.x;
            if (c8 < a.d) {
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[j] = 0.0f;
                    for (int w = 0; w < kJoinWarps; ++w) v[j] += acc[w][8 * threadIdx.x + j];
                }
                Raw8<TT> old;
                if constexpr (kAdd)
                    load8<kWide>(old, static_cast<const TT *>(a.table.p) + (int64_t)e.y * a.table.ld + c8, (int)a.d - c8);
                write_row<TT, kAdd, kWide>(a, e.y, c8, 1, v, old);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- few positions

constexpr int kFewUnit = 4, kFewLanes = 4;  // positions of a unit; threads of a unit, eight columns each
constexpr int kFewCols = 8 * kFewLanes;

// All of it in one kernel: a CTA orders the positions for itself, and sums kFewCols columns of all of them, four threads
// per unit; parts stay in shared memory.
template <typename TG, typename TT, bool kAdd, bool kWide>
__global__ void __launch_bounds__(kSortThreads) few_rows_kernel(const SumParams p, const SortParams sp) {
    constexpr int kRows = kFewRows<kAdd>;
    __shared__ __align__(16) float parts[kRows / kFewUnit][2][kFewCols];
    __shared__ __align__(16) int32_t unsorted[kRows];
    __shared__ int32_t key_s[kRows], pos_s[kRows];
    const EmbedRows &a = p.a;
    order_few<kRows>(sp, unsorted, key_s, pos_s);
    grid_dependency_wait();  // (what clears the gradient)
    const int R = (int)a.R, U = kFewUnit;
    auto key = [&](int i) { return i >= 0 && i < R ? key_s[i] : -1; };
    auto pos = [&](int i) { return pos_s[i]; };
    const int quad = threadIdx.x / kFewLanes, sub = threadIdx.x % kFewLanes;
    const int at = (kWide ? 8 : 1) * sub, step = kWide ? 1 : kFewLanes;  // of the CTA's columns, this thread's eight
    const int c = (int)blockIdx.x * kFewCols + at;
    const int units = (R + U - 1) / U;
    // (a warp holds eight units: their ranges one after another, each by all lanes)
    UnitRange r{0, 0, false, false};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int q = 0; q < 32 / kFewLanes; ++q) {
        const int m = warp * (32 / kFewLanes) + q;
        if (m >= units) break;
        const UnitRange t = unit_range(key, m * U, min(R, m * U + U), U, p.none, lane);
        if (q == lane / kFewLanes) r = t;
    }
    const bool on = quad < units && c < a.d;
    if (on && r.lo < r.hi)
        sum_unit<4, TG, TT, kAdd, kWide>(a, key, pos, [&](int slot, const float (&acc)[8]) {
            store8<kWide>(&parts[quad][slot][at], acc, kFewCols - at, step);
        }, r, quad * U, c, step);
    __syncthreads();
    // tokens that left parts: their unit's second, then the first ones of those after it, by all of the warp
    uint32_t longs = __ballot_sync(0xffffffffu, quad < units && r.part1 && sub == 0);
    while (longs) {
        const int owner = (warp * 32 + __ffs(longs) - 1) / kFewLanes;
        longs &= longs - 1;
        const int32_t k = key_s[owner * U + U - 1];
        float acc[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) acc[t] = lane < kFewLanes ? parts[owner][1][at + t * step] : 0.0f;
        for (int m = owner + 1 + lane / kFewLanes; m < units && key_s[m * U] == k; m += 32 / kFewLanes) {
            Raw8<float> raw;
            float v[8];
            load8<kWide>(raw, &parts[m][0][at], kFewCols - at, step);
            unpack8(v, raw);
#pragma unroll
            for (int t = 0; t < 8; ++t) acc[t] += v[t];
        }
#pragma unroll
        for (int off = kFewLanes; off < 32; off <<= 1)
#pragma unroll
            for (int t = 0; t < 8; ++t) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], off);
        if (lane < kFewLanes && c < a.d) {
            Raw8<TT> old;
            if constexpr (kAdd)
                load8<kWide>(old, static_cast<const TT *>(a.table.p) + (int64_t)k * a.table.ld + c, (int)a.d - c, step);
            write_row<TT, kAdd, kWide>(a, k, c, step, acc, old);
        }
    }
}

template <typename TT, bool kWide>
__global__ void __launch_bounds__(256) clear_rows_kernel(const EmbedRows a, int64_t rows) {
    const int d = (int)a.d, lane = threadIdx.x & 31;
    const float zero[8] = {};
    grid_launch_dependents();  // the order of the tokens is found meanwhile
    for (int64_t v = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); v < rows; v += (int64_t)gridDim.x * 8)
        for (int c = (kWide ? 8 : 1) * lane; c < d; c += 256)
            store8<kWide>(static_cast<TT *>(a.table.p) + v * a.table.ld + c, zero, d - c, kWide ? 1 : 32);
}

// ---------------------------------------------------------------- plan

// Sorted positions of a unit: long ones, which leave fewer parts, where that still leaves every SM some warps
// (8,192 x 2,816: 37.7 us with 32, 38.5 with 16; 8,192 x 512 with 8 26.9 for 23.2).
constexpr int kUnit = 16, kLongUnit = 32;
constexpr int64_t kLongFrom = 32 * 2048;  // positions times slabs of 256 columns
int unit_of(int64_t R, int64_t d) { return (d + 255) / 256 * R >= kLongFrom ? kLongUnit : kUnit; }

size_t align16(size_t b) { return (b + 15) & ~size_t(15); }

SortSpace lay_out(uint8_t *base, int64_t R, int64_t d, int unit, size_t *bytes) {
    SortSpace s;
    const int64_t units = (R + unit - 1) / unit;
    size_t at = 0;
    auto take = [&](size_t n) {
        uint8_t *q = base + at;
        at += align16(n);
        return q;
    };
    s.count = reinterpret_cast<int32_t *>(take(16));
    for (int i = 0; i < 2; ++i) {
        s.key[i] = reinterpret_cast<int32_t *>(take((size_t)R * 4));
        s.pos[i] = reinterpret_cast<int32_t *>(take((size_t)R * 4));
    }
    s.list = reinterpret_cast<int2 *>(take((size_t)units * 8));
    s.part_ld = (d + 7) / 8 * 8;
    s.parts = reinterpret_cast<float *>(take((size_t)units * 2 * (size_t)s.part_ld * 4));
    *bytes = at;
    return s;
}

// Launches that start while the kernel before them ends.
template <typename... Args>
cudaError_t launch_chained(void (*kernel)(Args...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, bool chained,
                           unsigned cluster, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = chained ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t ensure_merge_attributes() {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < kMaxDevices && done[dev].load(std::memory_order_acquire))) return e;
    e = cudaFuncSetAttribute(merge_near_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNearRows * (int)sizeof(int32_t));
    if (e == cudaSuccess && dev < kMaxDevices) done[dev].store(1, std::memory_order_release);
    return e;
}

// chained: after the kernel that clears the gradient, which starts after all that was launched before it
cudaError_t sort_tokens(SortParams sp, bool chained, cudaStream_t stream) {
    if (sp.R > kSortMost) return launch_chained(sort_far_kernel, kSortCtas, kSortThreads, 0, stream, chained, kSortCtas, sp);
    // Runs counted side by side and merged in shared memory take half the time of radix runs merged from global memory:
    // d = 512, 5,000 positions 15.4 us and 23.6, 16,000 25.9 and 29.3, 24,576 34.9 and 37.3; 32,768 45.7 and 42.8,
    // 57,344 86.5 and 58.7, as every CTA of the merge loads all keys.  Up to kOneRun they are one run: 2,048 positions 12.8 us and, merged of two,
    // 13.6; 3,000 14.9 and 14.3.
    if (sp.R <= kNearRows) {
        const bool one = sp.R <= kOneRun;
        sp.run = one ? kOneRun : kNearRun;
        cudaError_t e = launch_chained(count_tokens_kernel, (unsigned)((sp.R + kCountItems - 1) / kCountItems), kCountThreads, 0,
                                       stream, chained, 1u, sp);
        if (e == cudaSuccess && !one) e = ensure_merge_attributes();
        if (e != cudaSuccess || one) return e;
        const int items = kNearThreads / kNearShare;
        return launch_chained(merge_near_kernel, (unsigned)((sp.R + items - 1) / items), kNearThreads,
                              (size_t)(sp.R + 3) / 4 * sizeof(int4), stream, true, 1u, sp);
    }
    const cudaError_t e = launch_chained(sort_run_kernel, (unsigned)((sp.R + kRun - 1) / kRun), kSortThreads, 0, stream, chained, 1u, sp);
    if (e != cudaSuccess) return e;
    return launch_chained(merge_runs_kernel, (unsigned)((sp.R + 255) / 256), 256u, 0, stream, true, 1u, sp);
}

template <typename TG, typename TT, bool kAdd, bool kWide>
cudaError_t sums(const SumParams &p, const SortParams &sp, cudaStream_t stream) {
    if (p.a.R <= kFewRows<kAdd>)
        return launch_chained(few_rows_kernel<TG, TT, kAdd, kWide>, (unsigned)((p.a.d + kFewCols - 1) / kFewCols), kSortThreads, 0,
                              stream, !kAdd, 1u, p, sp);
    cudaError_t e = sort_tokens(sp, !kAdd, stream);
    if (e != cudaSuccess) return e;
    const unsigned ctas = (unsigned)((p.units + p.cta_units - 1) / p.cta_units * p.slab_ctas);
    const size_t smem = (size_t)(2 * p.cta_units * p.unit + 3 * p.unit + 2) * sizeof(int32_t);
    e = launch_chained(sum_rows_kernel<TG, TT, kAdd, kWide>, ctas, 32u * p.unit_warps * p.cta_units, smem, stream, true, 1u, p);
    if (e != cudaSuccess) return e;
    return launch_chained(join_parts_kernel<TT, kAdd, kWide>, (unsigned)std::max(1, device_sm_count() * 4), 32u * kJoinWarps, 0,
                          stream, true, 1u, p);
}

}  // namespace

cudaError_t launch_token_embed(const EmbedRows &a, cudaStream_t stream) {
    GatherParams p{a, 32};
    const int64_t sms = std::max(1, device_sm_count()), eights = (a.d + 7) / 8;
    // a warp per row where the rows alone give the SMs eight warps each, more threads per row where they do not (bf16 of
    // 2,816, a warp and the rule: 64 positions 2.95 us and 2.0, 512 3.0 and 2.4; with 1,024 threads an SM for 256 512
    // positions took 3.3, 2,000 5.4 for 4.35)
    while (p.lanes < kGatherThreads && a.R * p.lanes < sms * 256 && p.lanes < eights) p.lanes *= 2;
    const int64_t per = kGatherThreads / p.lanes;
    const unsigned grid = (unsigned)std::min<int64_t>((a.R + per - 1) / per, sms * 64);
    if (a.table.dtype == DG_F32)
        gather_out<float>(p, grid, stream);
    else if (a.table.dtype == DG_BF16)
        gather_out<__nv_bfloat16>(p, grid, stream);
    else
        gather_out<E4m3>(p, grid, stream);
    return cudaGetLastError();
}

// What any call of up to R positions and d columns needs, so that a workspace for the largest call serves smaller ones:
// calls just too small for long units leave twice the parts of those just above.
size_t token_embed_backward_bytes(int64_t R, int64_t d) {
    size_t most, bytes;
    lay_out(nullptr, R, d, unit_of(R, d), &most);
    if (unit_of(R, d) == kUnit) return most;  // (so are all smaller calls')
    // the largest calls of short units, slab by slab; of kUnit positions and fewer there is one unit of either length
    for (int64_t slabs = 1; slabs <= (d + 255) / 256 && (kLongFrom - 1) / slabs > kUnit; ++slabs) {
        lay_out(nullptr, std::min(R, (kLongFrom - 1) / slabs), std::min(d, slabs * 256), kUnit, &bytes);
        most = std::max(most, bytes);
    }
    return most;
}

cudaError_t launch_token_embed_backward(const EmbedRows &a, void *workspace, cudaStream_t stream) {
    const int64_t rows = a.vocab_end - a.vocab_start;
    if (!a.accumulate) {
        const unsigned grid = (unsigned)std::min<int64_t>((rows + 7) / 8, (int64_t)std::max(1, device_sm_count()) * 32);
        const bool f32 = a.table.dtype == DG_F32, wide = wide_rows(a.table);
        (f32 ? wide ? clear_rows_kernel<float, true> : clear_rows_kernel<float, false>
         : wide ? clear_rows_kernel<__nv_bfloat16, true>
                : clear_rows_kernel<__nv_bfloat16, false>)<<<grid, 256, 0, stream>>>(a, rows);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (a.R == 0) return cudaSuccess;
    size_t bytes;
    SortParams sp{};
    sp.s = lay_out(static_cast<uint8_t *>(workspace), a.R, a.d, unit_of(a.R, a.d), &bytes);
    sp.token = a.token;
    sp.V = a.V;
    sp.vocab_start = a.vocab_start;
    sp.vocab_end = a.vocab_end;
    sp.R = (int32_t)a.R;
    sp.none = (int32_t)rows;
    int bits = 1;
    while ((rows >> bits) != 0) ++bits;
    sp.passes = (bits + kDigitBits - 1) / kDigitBits;
    sp.bits = (bits + sp.passes - 1) / sp.passes;
    SumParams p{};
    p.a = a;
    p.s = sp.s;
    p.none = sp.none;
    p.unit = unit_of(a.R, a.d);
    p.units = (int)((a.R + p.unit - 1) / p.unit);
    p.slabs = (int)((a.d + 255) / 256);
    p.unit_warps = std::min(p.slabs, kSumWarps);
    p.cta_units = kSumWarps / p.unit_warps;
    p.slab_ctas = (p.slabs + p.unit_warps - 1) / p.unit_warps;
    auto typed = [&](auto add, auto wide) {
        constexpr bool kAdd = decltype(add)::value, kWide = decltype(wide)::value;
        if (a.rows.dtype == DG_F32)
            return a.table.dtype == DG_F32 ? sums<float, float, kAdd, kWide>(p, sp, stream)
                                           : sums<float, __nv_bfloat16, kAdd, kWide>(p, sp, stream);
        return a.table.dtype == DG_F32 ? sums<__nv_bfloat16, float, kAdd, kWide>(p, sp, stream)
                                       : sums<__nv_bfloat16, __nv_bfloat16, kAdd, kWide>(p, sp, stream);
    };
    const std::true_type yes;
    const std::false_type no;
    return wide_rows(a.rows) && wide_rows(a.table) ? (a.accumulate ? typed(yes, yes) : typed(no, yes))
                                                   : (a.accumulate ? typed(yes, no) : typed(no, no));
}

}  // namespace dg
