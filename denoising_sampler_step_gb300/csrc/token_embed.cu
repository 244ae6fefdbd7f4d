// The embedding table's rows at a canvas' tokens, and the table's gradient from that of the rows.
//
//   out[r] = gamma s_t W[t - vocab_start],  t = token[r] in [vocab_start, vocab_end), else 0
//   gW[v] (+)= gamma sum over {r : token[r] = v} of g[r]
//
// Forward: a gather, bound by HBM (a table row and an output row per position) and by latency where there
// are few positions.
//
// Backward: the positions are put in order of their tokens by a stable radix sort in one cluster (its
// keys stay in L2), so that every table row is written by one warp from its positions in order: no
// atomics on values, results repeat bit for bit.  The sorted positions are cut into units; a warp takes
// a unit and 256 columns.  A token that ends within the next unit is finished by the warp it began in.
// One that covers a whole unit and its neighbours (a mask or padding token) leaves one fp32 part per
// unit, and a last kernel adds its parts in order.
#include <algorithm>

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
    bool wide_table, wide_out;
};

template <typename TT, typename TO>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const GatherParams p) {
    const EmbedRows &a = p.a;
    const int per_cta = kGatherThreads / p.lanes;
    const int lane = threadIdx.x % p.lanes;
    const int d = (int)a.d;
    for (int64_t r = (int64_t)blockIdx.x * per_cta + threadIdx.x / p.lanes; r < a.R; r += (int64_t)gridDim.x * per_cta) {
        const int64_t t = a.token[r];
        const bool on = t >= a.vocab_start && t < a.vocab_end;
        if (t >= a.V && lane == 0) atomicOr(&g_device_error, kIndexRange);
        const TT *src = static_cast<const TT *>(a.table.p) + (on ? (t - a.vocab_start) * a.table.ld : 0);
        const float f = on && a.scale ? a.scale[t - a.vocab_start] : 1.0f;
        TO *dst = static_cast<TO *>(a.rows.p) + r * a.rows.ld;
        for (int c0 = 8 * lane; c0 < d; c0 += 4 * 8 * p.lanes) {
            Raw8<TT> raw[4];
            if (on)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = c0 + i * 8 * p.lanes;
                    if (c < d) load8(raw[i], src + c, d - c, p.wide_table);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
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
                store8(dst + c, v, d - c, p.wide_out);
            }
        }
    }
}

template <typename TT>
void gather_out(const GatherParams &p, unsigned grid, cudaStream_t stream) {
    if (p.a.rows.dtype == DG_F32)
        gather_kernel<TT, float><<<grid, kGatherThreads, 0, stream>>>(p);
    else
        gather_kernel<TT, __nv_bfloat16><<<grid, kGatherThreads, 0, stream>>>(p);
}

// ---------------------------------------------------------------- the order of the tokens

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 256;

// Where everything lies in the workspace.
struct SortSpace {
    int32_t *key[2], *pos[2];  // sorted: [0]
    int2 *list;                // (unit, key) of the tokens that leave parts
    int32_t *count;
    float *parts;              // [unit][0: begun before it, 1: begun in it][part_ld]
    int64_t part_ld;
};

struct SortParams {
    const int32_t *token;
    int64_t V, vocab_start, vocab_end;
    int32_t R, none;  // none: the key of a position without a table row, above all others
    int passes, bits;
    SortSpace s;
};

__global__ void __launch_bounds__(kSortThreads) sort_tokens_kernel(const SortParams p) {
    __shared__ uint32_t hist[kMaxBins][kSortWarps + 1];
    __shared__ uint32_t total[kMaxBins], start[kMaxBins], warp_total[kMaxBins / 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int ctas = (int)gridDim.x, rank = (int)blockIdx.x;  // one cluster
    const int bins = 1 << p.bits;
    const int per = ((p.R + ctas * kSortWarps - 1) / (ctas * kSortWarps) + 31) / 32 * 32;
    const int64_t i0 = (int64_t)(rank * kSortWarps + warp) * per;
    const int n = i0 >= p.R ? 0 : (int)min((int64_t)per, p.R - i0);
    if (rank == 0 && threadIdx.x == 0) *p.s.count = 0;

    for (int pass = 0; pass < p.passes; ++pass) {
        // an odd number of passes begins from the tokens into [0], an even one into [1]
        const int to = (p.passes - 1 - pass) & 1;
        const int shift = pass * p.bits;
        auto key_at = [&](int64_t i) -> int32_t {
            if (pass > 0) return __ldcg(p.s.key[to ^ 1] + i);
            const int64_t t = p.token[i];
            if (t >= p.V) atomicOr(&g_device_error, kIndexRange);
            return t >= p.vocab_start && t < p.vocab_end ? (int32_t)(t - p.vocab_start) : p.none;
        };
        for (int b = threadIdx.x; b < bins * (kSortWarps + 1); b += kSortThreads) (&hist[0][0])[b] = 0;
        __syncthreads();
        for (int i = lane; i < (n + 31) / 32 * 32; i += 32) {
            const uint32_t dig = i < n ? (uint32_t)(key_at(i0 + i) >> shift) & (bins - 1) : 0xFFFFFFFFu;
            const uint32_t same = __match_any_sync(0xffffffffu, dig);
            if (i < n && (same & ((1u << lane) - 1)) == 0) hist[dig][warp] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        // over the warps of this CTA, then over the CTAs, then over the digits
        for (int b = warp; b < bins; b += kSortWarps) {
            const uint32_t own = hist[b][lane];
            uint32_t sum = own;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(0xffffffffu, sum, off);
                if (lane >= off) sum += o;
            }
            hist[b][lane] = sum - own;
            if (lane == 31) total[b] = sum;
        }
        __syncthreads();
        if (ctas > 1) cluster_sync_all();
        uint32_t all = 0, before = 0;
        if ((int)threadIdx.x < bins) {
            const uint32_t mine = smem_u32(&total[threadIdx.x]);
            for (int c = 0; c < ctas; ++c) {
                uint32_t t;
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(t) : "r"(map_to_cta(mine, (uint32_t)c)) : "memory");
                all += t;
                if (c < rank) before += t;
            }
        }
        uint32_t sum = all;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += o;
        }
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
            const uint32_t below = __popc(same & ((1u << lane) - 1));
            uint32_t at = 0;
            if (in) at = start[dig] + hist[dig][warp] + below;
            __syncwarp();
            if (in) {
                if (below == 0) hist[dig][warp] += __popc(same);
                p.s.key[to][at] = k;
                p.s.pos[to][at] = pass > 0 ? __ldcg(p.s.pos[to ^ 1] + i0 + i) : (int32_t)(i0 + i);
            }
            __syncwarp();
        }
        __threadfence();  // the next pass, and the next kernel, read what other CTAs wrote here
        if (ctas > 1) cluster_sync_all();
        __syncthreads();
    }
}

// ---------------------------------------------------------------- the sums

struct SumParams {
    EmbedRows a;
    SortSpace s;
    int32_t none;
    int unit, units, slabs;  // sorted positions of a unit; slabs of 256 columns
    bool wide_grad, wide_table;
};

__device__ __forceinline__ void load_entry8(float (&v)[8], const float *q, int n, bool wide) {
    Raw8<float> r;
    load8(r, q, n, wide);
    unpack8(v, r);
}
__device__ __forceinline__ void load_entry8(float (&v)[8], const __nv_bfloat16 *q, int n, bool wide) {
    Raw8<__nv_bfloat16> r;
    load8(r, q, n, wide);
    unpack8(v, r);
}

// gW[key][c ..] (+)= gamma sum
template <typename TT>
__device__ __forceinline__ void write_row(const EmbedRows &a, int32_t key, int c, const float (&sum)[8], bool wide) {
    TT *dst = static_cast<TT *>(a.table.p) + (int64_t)key * a.table.ld + c;
    const int n = (int)a.d - c;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    if (a.accumulate) load_entry8(v, dst, n, wide);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = a.accumulate ? v[j] + sum[j] * a.gamma : sum[j] * a.gamma;
    store8(dst, v, n, wide);
}

constexpr int kSumWarps = 4;

template <typename TG, typename TT>
__global__ void __launch_bounds__(32 * kSumWarps) sum_rows_kernel(const SumParams p) {
    const EmbedRows &a = p.a;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kSumWarps + (threadIdx.x >> 5);
    const int m = (int)(w / p.slabs), slab = (int)(w % p.slabs);
    if (m >= p.units) return;
    const int R = (int)a.R, U = p.unit;
    const int32_t *key = p.s.key[0], *pos = p.s.pos[0];
    const int64_t u0 = (int64_t)m * U, u1 = min((int64_t)R, u0 + U);
    const int32_t first = key[u0], last = key[u1 - 1];
    if (first == p.none) return;

    // a token begun before this unit: the warp it began in finishes it, unless it covers a whole unit
    // and both its neighbours (this one or the one before, if any); then each unit leaves its part
    int64_t lo = u0, hi = u1;
    bool part0 = false, part1 = false;
    if (u0 > 0 && key[u0 - 1] == first) {
        part0 = (u0 > U && key[u0 - U - 1] == first) || (u1 == u0 + U && u1 < R && key[u1] == first);
        if (!part0) {
            while (true) {  // the next token's first position, or the unit's end
                const int64_t i = lo + lane;
                const uint32_t other = __ballot_sync(0xffffffffu, i >= u1 || key[i] != first);
                if (other) {
                    lo += __ffs(other) - 1;
                    break;
                }
                lo += 32;
            }
            if (lo >= u1 || key[lo] == p.none) return;
        }
    }
    // a token that goes on past this unit, and began in it
    if (u1 < R && last != p.none && key[u1] == last && !(last == first && lo == u0 && u0 > 0 && key[u0 - 1] == first)) {
        part1 = u1 + U < R && key[u1 + U] == last;
        if (!part1) {
            while (true) {
                const int64_t i = hi + lane;
                const uint32_t other = __ballot_sync(0xffffffffu, i >= R || key[i] != last);
                if (other) {
                    hi += __ffs(other) - 1;
                    break;
                }
                hi += 32;
            }
        } else if (slab == 0 && lane == 0) {
            p.s.list[atomicAdd(p.s.count, 1)] = make_int2(m, last);
        }
    }

    const int c = slab * 256 + 8 * lane;
    const int d = (int)a.d;
    const TG *g = static_cast<const TG *>(a.rows.p);
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    int32_t cur = key[lo];
    auto flush = [&](bool at_end) {
        if (c < d) {
            if ((part0 && cur == first) || (part1 && at_end)) {
                float *dst = p.s.parts + ((int64_t)m * 2 + (part0 && cur == first ? 0 : 1)) * p.s.part_ld + c;
                store8(dst, acc, 8, true);
            } else {
                write_row<TT>(a, cur, c, acc, p.wide_table);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    };
    constexpr int kAhead = 8;
    bool done = false;
    for (int64_t i = lo; i < hi && !done; i += kAhead) {
        Raw8<TG> raw[kAhead];
        int32_t k[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            k[j] = i + j < hi ? key[i + j] : p.none;
            if (k[j] != p.none && c < d) load8(raw[j], g + (int64_t)pos[i + j] * a.rows.ld + c, d - c, p.wide_grad);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (done) continue;
            if (k[j] == p.none) {
                done = true;
                continue;
            }
            if (k[j] != cur) {
                flush(false);
                cur = k[j];
            }
            if (c < d) {
                float v[8];
                unpack8(v, raw[j]);
#pragma unroll
                for (int t = 0; t < 8; ++t) acc[t] += v[t];
            }
        }
    }
    flush(true);
}

constexpr int kJoinWarps = 8;

// Tokens that left parts: unit m's second part, then the first parts of the units after it that begin
// with the same token.  A CTA takes a token and 128 columns, its warps a share of the parts each.
template <typename TT>
__global__ void __launch_bounds__(32 * kJoinWarps) join_parts_kernel(const SumParams p) {
    __shared__ float acc[kJoinWarps][128];
    const EmbedRows &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slabs = (int)((a.d + 127) / 128);
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
        if (c < a.d)
            for (int i = warp * per; i < min(n + 1, (warp + 1) * per); ++i) {
                const int64_t slot = ((int64_t)e.x + i) * 2 + (i == 0);
                const float4 v = *reinterpret_cast<const float4 *>(p.s.parts + slot * p.s.part_ld + c);
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
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
                write_row<TT>(a, e.y, c8, v, p.wide_table);
            }
        }
        __syncthreads();
    }
}

template <typename TT>
__global__ void __launch_bounds__(256) clear_rows_kernel(const EmbedRows a, int64_t rows, bool wide) {
    const int d = (int)a.d, eights = (d + 7) / 8;
    const float zero[8] = {};
    for (int64_t v = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); v < rows; v += (int64_t)gridDim.x * 8)
        for (int c = threadIdx.x & 31; c < eights; c += 32)
            store8(static_cast<TT *>(a.table.p) + v * a.table.ld + 8 * c, zero, d - 8 * c, wide);
}

// ---------------------------------------------------------------- plan

int unit_of(int64_t R) { return R >= 32768 ? 64 : R >= 8192 ? 32 : 8; }

size_t align16(size_t b) { return (b + 15) & ~size_t(15); }

SortSpace lay_out(uint8_t *base, int64_t R, int64_t d, size_t *bytes) {
    SortSpace s;
    const int64_t units = (R + unit_of(R) - 1) / unit_of(R);
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

template <typename TG, typename TT>
cudaError_t sums(const SumParams &p, cudaStream_t stream) {
    const int64_t warps = (int64_t)p.units * p.slabs;
    sum_rows_kernel<TG, TT><<<(unsigned)((warps + kSumWarps - 1) / kSumWarps), 32 * kSumWarps, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.a.R <= p.unit) return e;
    join_parts_kernel<TT><<<(unsigned)std::max(1, device_sm_count() * 4), 32 * kJoinWarps, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_embed(const EmbedRows &a, cudaStream_t stream) {
    GatherParams p{a, 32, wide_rows(a.table), wide_rows(a.rows)};
    const int64_t sms = std::max(1, device_sm_count()), eights = (a.d + 7) / 8;
    // a warp per row where the rows alone fill the chip, more threads per row where they do not
    while (p.lanes < kGatherThreads && a.R * p.lanes < sms * 2048 && p.lanes < eights) p.lanes *= 2;
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

size_t token_embed_backward_bytes(int64_t R, int64_t rows, int64_t d) {
    (void)rows;
    size_t bytes;
    lay_out(nullptr, R, d, &bytes);
    return bytes;
}

cudaError_t launch_token_embed_backward(const EmbedRows &a, void *workspace, cudaStream_t stream) {
    const int64_t rows = a.vocab_end - a.vocab_start;
    const bool wide_table = wide_rows(a.table);
    if (!a.accumulate && rows > 0) {
        const unsigned grid = (unsigned)std::min<int64_t>((rows + 7) / 8, (int64_t)std::max(1, device_sm_count()) * 32);
        if (a.table.dtype == DG_F32)
            clear_rows_kernel<float><<<grid, 256, 0, stream>>>(a, rows, wide_table);
        else
            clear_rows_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, rows, wide_table);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (a.R == 0) return cudaSuccess;
    size_t bytes;
    SortParams sp{};
    sp.s = lay_out(static_cast<uint8_t *>(workspace), a.R, a.d, &bytes);
    sp.token = a.token;
    sp.V = a.V;
    sp.vocab_start = a.vocab_start;
    sp.vocab_end = a.vocab_end;
    sp.R = (int32_t)a.R;
    sp.none = (int32_t)rows;
    int bits = 1;
    while ((rows >> bits) != 0) ++bits;
    sp.passes = (bits + 7) / 8;
    sp.bits = (bits + sp.passes - 1) / sp.passes;
    cudaLaunchConfig_t cfg = {};
    const unsigned ctas = a.R <= 2048 ? 1 : 8;
    cfg.gridDim = dim3(ctas, 1, 1);
    cfg.blockDim = dim3(kSortThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, sort_tokens_kernel, sp);
    if (e != cudaSuccess) return e;
    SumParams p{};
    p.a = a;
    p.s = sp.s;
    p.none = sp.none;
    p.unit = unit_of(a.R);
    p.units = (int)((a.R + p.unit - 1) / p.unit);
    p.slabs = (int)((a.d + 255) / 256);
    p.wide_grad = wide_rows(a.rows);
    p.wide_table = wide_table;
    if (a.rows.dtype == DG_F32)
        return a.table.dtype == DG_F32 ? sums<float, float>(p, stream) : sums<float, __nv_bfloat16>(p, stream);
    return a.table.dtype == DG_F32 ? sums<__nv_bfloat16, float>(p, stream) : sums<__nv_bfloat16, __nv_bfloat16>(p, stream);
}

}  // namespace dg
