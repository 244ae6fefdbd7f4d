// Logits of the tied 8-bit head: logits[r, v] = sx[r] sw[v] sum_k X[r, k] Q[v, k], both operands E4M3
// codes, one scale per position and one per vocabulary row (applied to the fp32 sum).
//
// The vocabulary is the M side of the product and the positions its N side: a tcgen05 CTA pair
// (cta_group::2) multiplies 256 vocabulary rows (128 in each CTA) by up to 256 positions (half of them
// in each CTA's shared memory), K = 32 per instruction, 256 codes per ring slot.  So a single position costs
// an N of 32, a table row is read once per 256 positions, and the accumulator's lanes are consecutive
// vocabulary entries.  The pairs are persistent: two accumulators in TMEM (2 x 256 columns) let the stores
// of one tile run under the next tile's product.  Where one tile takes all positions, their codes stay in
// shared memory; the table's rows per tile are then as many as make the rounds of tiles even.
//
// Bound by HBM up to some 300 positions (table + logits), by the E4M3 MMA rate above.  V = 262,144,
// d = 2,816: 1 position 111 us (6.7 TB/s), 256 with fp32 logits 163 us (6.2 TB/s), with bf16 ones 151 us; 2,048 with
// bf16 ones 870 us (3.48 PFLOP/s) for a call by itself, 1,030 us in a row of calls, where the chip's power limit
// lowers the clock.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "dg_common.cuh"
#include "dg_internal.h"
#include "hidden.cuh"

namespace dg {

namespace {

constexpr int kTileV = 256;                 // vocabulary rows of a pair's product
constexpr int kRowsCta = kTileV / 2;        // of them in each CTA; a tile takes the first rows_cta of these
constexpr int kMinRows = 32;
constexpr int kMaxTileR = 256;              // positions of a tile
constexpr int kBlockK = 128;                // codes of a block and row: one 128-byte swizzle atom
constexpr int kSlotBlocks = 2;              // blocks of a ring slot, one load for the two of either operand
constexpr int kMaxStages = 12;
constexpr int kEpilogueWarps = 8;           // two per TMEM lane quarter
constexpr int kWarpLoad = kEpilogueWarps, kWarpMma = kEpilogueWarps + 1;
constexpr int kThreads = (kEpilogueWarps + 2) * 32;
constexpr int kTmemCols = 512;
constexpr int kSmemLimit = 232448;          // shared memory of a CTA
constexpr int kResidentBytes = 96 * 1024;   // a CTA's half of the positions, at most, to stay in it
constexpr int kBarrierBytes = 512;
constexpr int kStageBytes = 8192;           // of logits on their way out: two buffers for each half of the epilogue
constexpr int kFewPositions = 64;           // up to these the logits are stored from registers

struct HeadParams {
    const float *x_scale, *w_scale;
    void *logits;
    int64_t ldl, tiles;
    int rows_cta;
    int R, V, tile_r, r_tiles, k_blocks, k_steps;  // blocks and steps of 32 that cover d
    int full_blocks;  // of them those that lie wholly below d
    int stages, stage_bytes, resident_bytes;
    uint32_t idesc;
    int stream_table;   // each table byte is read once: leave L2 first
    int stream_logits;  // the logits do not stay in L2 either way (128 positions, fp32: 136.1 us for 140.9)
    int staged;         // logits go through shared memory
};

// Instruction descriptor of kind::f8f6f4 with E4M3 A and B, fp32 accumulator, both K-major.
constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// True in one lane of a converged warp.  The compiler then knows that a single thread issues what follows: with
// `lane == 0` in its place an instruction took 120 cycles to issue, a ring slot's four as long as their products.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

// One arrival, with release at cluster scope, on a barrier of any CTA of the cluster.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The 32 columns (positions) of a chunk that this lane holds for its vocabulary entry v; the first `live` lanes
// have one; sx: lane c holds the scale of position row0 + c.
__device__ __forceinline__ void store_chunk(const HeadParams &p, float *logits, const uint32_t (&acc)[32], int row0, int v,
                                            int lane, int live, float sw, float sx, uint64_t policy) {
    float *dst = logits + (int64_t)row0 * p.ldl + v;
    const int n = lane < live ? min(32, p.R - row0) : 0;
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        const float s = __shfl_sync(0xffffffffu, sx, c);
        if (c < n)
            asm volatile("st.global.L2::cache_hint.f32 [%0], %1, %2;" ::"l"(dst + c * p.ldl),
                         "f"(__uint_as_float(acc[c]) * sw * s), "l"(policy)
                         : "memory");
    }
}

// bf16: neighbouring lanes swap a value so that each writes two vocabulary entries of one position
// (half the stores; rows start on 16-byte boundaries, so the pair is 4-byte aligned).
__device__ __forceinline__ void store_chunk(const HeadParams &p, __nv_bfloat16 *logits, const uint32_t (&acc)[32],
                                            int row0, int v, int lane, int live, float sw, float sx,
                                            uint64_t policy) {
    const int odd = lane & 1, v0 = v - odd;
    const int n = min(32, p.R - row0);
    __nv_bfloat16 *dst = logits + (int64_t)(row0 + odd) * p.ldl + v0;
#pragma unroll
    for (int c = 0; c < 32; c += 2) {
        const float s0 = __shfl_sync(0xffffffffu, sx, c), s1 = __shfl_sync(0xffffffffu, sx, c + 1);
        const float a = __uint_as_float(acc[c]) * sw * s0, b = __uint_as_float(acc[c + 1]) * sw * s1;
        const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
        if (c + odd < n) {
            __nv_bfloat16 *q = dst + c * p.ldl;
            const float lo = odd ? got : a, hi = odd ? b : got;
            if (lane - odd + 1 < live)
                asm volatile("st.global.L2::cache_hint.b32 [%0], %1, %2;" ::"l"(q), "r"(hidden::pack_bf16(lo, hi)), "l"(policy)
                             : "memory");
            else if (lane - odd < live)
                *q = __float2bfloat16_rn(lo);
        }
    }
}

// 32 lanes x 16 consecutive fp32 columns, as tmem_ld_32x32b_x32.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

// Logits through shared memory: a half of the epilogue (four warps, a lane quarter each) gathers kTokens positions of
// all the tile's table rows, [position][table row], which one thread sends out as one tile; rows and columns past the
// matrix are cut off there.  So a position's logits leave as one piece of 256 or 512 bytes, where a warp's own stores
// were pieces of 64 or 128 that took twice the time of the bytes (256 positions, fp32: 185 us;
// 128: 139.6 us and as tiles 136.1).  Up to kFewPositions the logits are a small part of the bytes, and the ring has the
// room instead (64 positions 126.5 us, as tiles 128.2).
template <typename T>
constexpr int kTokens = kStageBytes / (kRowsCta * (int)sizeof(T));

// Whether all threads of the half say yes: they go on, or stop, together.
__device__ __forceinline__ bool half_vote(int half, bool yes) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, %2, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)yes), "r"(half + 1)
        : "memory");
    return all != 0;
}
__device__ __forceinline__ void half_sync(int half) { asm volatile("bar.sync %0, 128;" ::"r"(half + 1) : "memory"); }

__device__ __forceinline__ void put_logits(uint32_t at, int pitch, const uint32_t (&acc)[16], int entry, float sw, float sx, int c0,
                                           float) {
#pragma unroll
    for (int c = 0; c < 16; ++c) {
        const float y = __uint_as_float(acc[c]) * sw * __shfl_sync(0xffffffffu, sx, c0 + c);
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + (uint32_t)(c * pitch + 4 * entry)), "f"(y) : "memory");
    }
}
// bf16: neighbouring lanes swap a value so that each puts two table rows' logits of one position.
__device__ __forceinline__ void put_logits(uint32_t at, int pitch, const uint32_t (&acc)[16], int entry, float sw, float sx, int c0,
                                           __nv_bfloat16) {
    const int odd = entry & 1;
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
        const float a = __uint_as_float(acc[c]) * sw * __shfl_sync(0xffffffffu, sx, c0 + c);
        const float b = __uint_as_float(acc[c + 1]) * sw * __shfl_sync(0xffffffffu, sx, c0 + c + 1);
        const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
        const uint32_t y = hidden::pack_bf16(odd ? got : a, odd ? b : got);
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + (uint32_t)((c + odd) * pitch + 2 * (entry - odd))), "r"(y) : "memory");
    }
}

template <typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    head_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_x2, const __grid_constant__ CUtensorMap tm_w2,
                const __grid_constant__ CUtensorMap tm_out, const HeadParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem_raw);  // the even CTA's: both CTAs' tiles have landed
    uint64_t *empty = full + kMaxStages;                      // the slot's products are done
    uint64_t *acc_full = empty + kMaxStages;                  // a tile's products are done
    uint64_t *acc_empty = acc_full + 2;                       // the even CTA's: the accumulator has been read
    uint64_t *drained = acc_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const uint32_t staging = (smem_u32(smem_raw) + kBarrierBytes + 1023u) & ~1023u;
    const uint32_t resident = staging + (p.staged ? 4 * kStageBytes : 0);
    const uint32_t ring = resident + p.resident_bytes;
    // a CTA's half of the positions and its table rows, per block
    const uint32_t x_bytes = (uint32_t)(p.tile_r / 2) * kBlockK, w_bytes = (uint32_t)p.rows_cta * kBlockK;
    const int slots = (p.k_blocks + kSlotBlocks - 1) / kSlotBlocks;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&acc_full[b]), 1);
            mbar_init(smem_u32(&acc_empty[b]), 2 * kEpilogueWarps);
        }
        mbar_init(smem_u32(drained), 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&tm_x);
        prefetch_tmap(&tm_w);
    }
    __syncwarp();
    if (warp == 0) tmem_alloc_pair<kTmemCols>(smem_u32(tmem_slot));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync_all();  // the peer's barriers exist before any copy or commit reaches them
    const uint32_t tmem_base = *tmem_slot;
    bool ok = true;  // false once this thread gave up on a wait

    if (warp == kWarpLoad) {
        if (elect_one()) {
            const uint32_t lead_full = map_to_cta(smem_u32(&full[0]), 0);
            const uint64_t w_policy = p.stream_table ? l2_policy_evict_first() : l2_policy_evict_normal();
            const uint64_t x_policy = l2_policy_evict_normal();
            const bool keep = p.resident_bytes > 0;
            // blocks 2k and 2k + 1 of an operand's rows: one load where both lie wholly below d, else each by
            // itself, what lies past d as zeros
            auto load = [&](const void *tm2, const void *tm, uint32_t at, uint32_t block_bytes, uint32_t bar, int k, int row,
                            uint64_t policy) {
                if (2 * k + 1 < p.full_blocks) {
                    tma_load_3d_pair_hint(at, tm2, bar, 0, row, 2 * k, policy);
                } else {
                    tma_load_2d_pair_hint(at, tm, bar, 2 * k * kBlockK, row, policy);
                    if (2 * k + 1 < p.k_blocks)
                        tma_load_2d_pair_hint(at + block_bytes, tm, bar, (2 * k + 1) * kBlockK, row, policy);
                }
            };
            int s = 0;
            uint32_t use = 0;
            for (int64_t t = pair; t < p.tiles && ok; t += pairs) {
                const int v0 = (int)(t / p.r_tiles) * 2 * p.rows_cta + (int)rank * p.rows_cta;
                const int r0 = (int)(t % p.r_tiles) * p.tile_r + (int)rank * (p.tile_r / 2);
                for (int k = 0; k < slots; ++k) {
                    if (use > 0 && !mbar_wait(smem_u32(&empty[s]), (use - 1) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const bool with_x = !keep || t == pair;  // resident positions come with the first tile's slots
                    if (rank == 0)
                        mbar_arrive_expect_tx(smem_u32(&full[s]), 2 * (w_bytes + (with_x ? x_bytes : 0)) *
                                                                      (uint32_t)min(2, p.k_blocks - 2 * k));
                    const uint32_t at = ring + (uint32_t)s * p.stage_bytes, bar = lead_full + 8u * (uint32_t)s;
                    load(&tm_w2, &tm_w, at, w_bytes, bar, k, v0, w_policy);
                    if (with_x)
                        load(&tm_x2, &tm_x, keep ? resident + 2 * k * x_bytes : at + 2 * w_bytes, x_bytes, bar, k, r0,
                             x_policy);
                    if (++s == p.stages) {
                        s = 0;
                        ++use;
                    }
                }
            }
        }
    } else if (warp == kWarpMma) {
        if (rank == 0 && elect_one()) {
            const bool keep = p.resident_bytes > 0;
            int s = 0, n = 0;
            uint32_t ph = 0;
            for (int64_t t = pair; t < p.tiles && ok; t += pairs, ++n) {
                const int b = n & 1;
                if (n >= 2 && !mbar_wait(smem_u32(&acc_empty[b]), (uint32_t)((n >> 1) - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)b * 256u;
                for (int k = 0; k < slots; ++k) {
                    if (!mbar_wait(smem_u32(&full[s]), ph, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = ring + (uint32_t)s * p.stage_bytes;
                    const uint64_t a = smem_desc(at, 16, 1024, 2);
                    const uint64_t x = smem_desc(keep ? resident + 2 * k * x_bytes : at + 2 * w_bytes, 16, 1024, 2);
                    // 32 codes a step: 32 bytes further along both operands' rows
                    if (2 * k + 1 < p.full_blocks) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            umma_e4m3_pair(d_tmem, a + (j / 4) * (w_bytes >> 4) + 2 * (j % 4),
                                           x + (j / 4) * (x_bytes >> 4) + 2 * (j % 4), p.idesc, (k | j) != 0);
                    } else {
                        const int steps = p.k_steps - 8 * k;  // of the slot, the last one's cover d
                        for (int j = 0; j < min(8, steps); ++j)
                            umma_e4m3_pair(d_tmem, a + (j / 4) * (w_bytes >> 4) + 2 * (j % 4),
                                           x + (j / 4) * (x_bytes >> 4) + 2 * (j % 4), p.idesc, (k | j) != 0);
                    }
                    umma_commit_pair(smem_u32(&empty[s]), 3);
                    if (++s == p.stages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                if (ok) umma_commit_pair(smem_u32(&acc_full[b]), 3);
            }
            if (!ok) {  // products in flight finish before the pair's shared memory is given up
                umma_commit_pair(smem_u32(drained), 1);
                drain_wait(smem_u32(drained), 0);
            }
        }
    } else {
        const int quarter = warp & 3, half = warp >> 2;  // TMEM lanes, and every other chunk of columns
        const uint32_t lead_empty = map_to_cta(smem_u32(&acc_empty[0]), 0);
        T *logits = static_cast<T *>(p.logits);
        const uint64_t policy = p.stream_logits ? l2_policy_evict_first() : l2_policy_evict_normal();
        // a tile's scales are loaded while the tile before it is stored: a load takes thousands of cycles
        // beside the ring's traffic
        float sx[4], sx_next[4], sw, sw_next = 0.0f;
        auto load_scales = [&](int64_t t) {
            const int v = (int)(t / p.r_tiles) * 2 * p.rows_cta + (int)rank * p.rows_cta + quarter * 32 + lane;
            const int r = (int)(t % p.r_tiles) * p.tile_r + half * 32 + lane;
            sw_next = t < p.tiles && quarter * 32 + lane < p.rows_cta && v < p.V ? __ldg(p.w_scale + v) : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) sx_next[i] = t < p.tiles && r + 64 * i < p.R ? __ldg(p.x_scale + r + 64 * i) : 0.0f;
        };
        load_scales(pair);
        const bool sender = quarter == 0 && lane == 0;
        int n = 0, buffer = 0;
        for (int64_t t = pair; t < p.tiles; t += pairs, ++n) {
            const int b = n & 1;
            const int v = (int)(t / p.r_tiles) * 2 * p.rows_cta + (int)rank * p.rows_cta + quarter * 32 + lane;
            const int r0 = (int)(t % p.r_tiles) * p.tile_r;
            const int live = min(p.rows_cta, p.V - (v - quarter * 32 - lane)) - quarter * 32;  // entries of this quarter
            sw = sw_next;
#pragma unroll
            for (int i = 0; i < 4; ++i) sx[i] = sx_next[i];
            load_scales(t + pairs);
            ok = mbar_wait(smem_u32(&acc_full[b]), (uint32_t)(n >> 1) & 1, abort_flag);
            if (!half_vote(half, ok)) break;
            tc_fence_after();
            const uint32_t at = tmem_base + (uint32_t)b * 256u + ((uint32_t)(quarter * 32) << 16);
            const int pitch = p.rows_cta * (int)sizeof(T), entry = quarter * 32 + lane, v0 = v - entry;
            // (a tile that ends inside a 16-byte group is stored from registers: sent out, it wrote the whole group)
            if (p.staged && (v0 + p.rows_cta <= p.V || (p.V * (int64_t)sizeof(T)) % 16 == 0)) {
                if (v0 < p.V) {
#pragma unroll 1
                    for (int c = half * 32; c < p.tile_r && r0 + c < p.R; c += 64) {
                        const float sc = c < 64 ? sx[0] : c < 128 ? sx[1] : c < 192 ? sx[2] : sx[3];
#pragma unroll 1
                        for (int k = 0; k < 32; k += kTokens<T>, buffer ^= 1) {
                            const uint32_t to = staging + (uint32_t)(2 * half + buffer) * kStageBytes;
                            // the tile sent from this buffer before has left it
                            if (sender) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                            half_sync(half);
#pragma unroll
                            for (int q = 0; q < kTokens<T>; q += 16) {
                                uint32_t acc[16];
                                tmem_ld_32x32b_x16(at + c + k + q, acc);
                                tmem_ld_wait();
                                const int c0 = k + q;
                                const float s16 = c0 ? __shfl_down_sync(0xffffffffu, sc, 16) : sc;
                                if (quarter * 32 < p.rows_cta)  // (whole quarters: rows_cta is a multiple of 32)
                                    put_logits(to + (uint32_t)(q * pitch), pitch, acc, entry, sw, s16, 0, T());
                            }
                            fence_proxy_async_smem();
                            half_sync(half);
                            if (sender && r0 + c + k < p.R) {
                                asm volatile(
                                    "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group.L2::cache_hint"
                                    " [%0, {%2, %3}], [%1], %4;" ::"l"(&tm_out),
                                    "r"(to), "r"(v0), "r"(r0 + c + k), "l"(policy)
                                    : "memory");
                            }
                            if (sender) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        }
                    }
                }
            } else
#pragma unroll 1
            for (int c = half * 32; live > 0 && c < p.tile_r && r0 + c < p.R; c += 64) {
                uint32_t acc[32];
                tmem_ld_32x32b_x32(at + c, acc);
                tmem_ld_wait();
                store_chunk(p, logits, acc, r0 + c, v, lane, live, sw, c < 64 ? sx[0] : c < 128 ? sx[1] : c < 192 ? sx[2] : sx[3],
                            policy);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(lead_empty + 8u * (uint32_t)b);
        }
        if (sender) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    __syncthreads();
    if (*abort_flag) {
        // loads in flight land within microseconds; the even CTA's barriers count the odd CTA's too
        const unsigned long long t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
    }
    tc_fence_before();
    cluster_sync_all();  // neither CTA leaves while the other may still read from it or signal it
    if (warp == 0) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair<kTmemCols>(tmem_base);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

cudaError_t ensure_head_attributes() {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(head_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(head_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e == cudaSuccess && dev < kMaxDevices) done[dev].store(1, std::memory_order_release);
    return e;
}

// Rows of codes [rows, d] as boxes of one block by `box` rows (what lies past either end is 0), and, in a view of
// the blocks that lie wholly below d, of two blocks.
bool encode_codes(PFN_cuTensorMapEncodeTiled_v12000 encode, CUtensorMap *tm, CUtensorMap *tm2, const uint8_t *codes,
                  int64_t rows, int64_t d, int64_t ld, int box) {
    const int64_t blocks = d / kBlockK;
    const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows}, dims2[3] = {kBlockK, (cuuint64_t)rows, (cuuint64_t)blocks};
    const cuuint64_t strides[2] = {(cuuint64_t)ld, kBlockK};
    const cuuint32_t boxes[3] = {kBlockK, (cuuint32_t)box, kSlotBlocks};
    const cuuint32_t estr[3] = {1, 1, 1};
    auto make = [&](CUtensorMap *m, int rank, const cuuint64_t *dim) {
        return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<uint8_t *>(codes), dim, strides, boxes, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (!make(tm, 2, dims)) return false;
    *tm2 = *tm;  // (not used with fewer blocks)
    return blocks < kSlotBlocks || make(tm2, 3, dims2);
}

}  // namespace

cudaError_t launch_head_e4m3(const uint8_t *X, int64_t ldx, const float *x_scale, int64_t R, int64_t d,
                             const uint8_t *Q, int64_t ldq, const float *scale, int64_t V, void *logits, int dtype,
                             int64_t ldl, cudaStream_t stream, const char **msg) {
    *msg = "head";
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) {
        *msg = "cuTensorMapEncodeTiled is not available from the driver";
        return cudaErrorNotSupported;
    }
    HeadParams p{};
    p.R = (int)R;
    p.V = (int)V;
    p.r_tiles = (int)((R + kMaxTileR - 1) / kMaxTileR);
    p.tile_r = (int)(((R + p.r_tiles - 1) / p.r_tiles + 31) / 32 * 32);
    // as many rounds of tiles as the largest ones take, and no more table rows in a tile than make those rounds
    // even (whole 32s: a warp stores whole lines of fp32 logits)
    const int64_t pairs = std::max(1, device_sm_count() / 2);
    const int64_t rounds = ((V + kTileV - 1) / kTileV * p.r_tiles + pairs - 1) / pairs;
    const int64_t v_tiles = std::max<int64_t>(1, rounds * pairs / p.r_tiles);
    p.rows_cta = (int)std::min<int64_t>(kRowsCta, std::max<int64_t>(kMinRows, ((V + 2 * v_tiles - 1) / (2 * v_tiles) + 31) / 32 * 32));
    p.tiles = (V + 2 * p.rows_cta - 1) / (2 * p.rows_cta) * p.r_tiles;
    p.k_blocks = (int)((d + kBlockK - 1) / kBlockK);
    p.k_steps = (int)((d + 31) / 32);
    p.full_blocks = (int)(d / kBlockK);
    // the positions' codes are the same for every tile where one tile holds them all (64 positions 126.5 us, sent for with
    // every tile 128.7).  A product reads kRowsCta
    // table rows from where a tile's begin, whatever lies there past the tile's own: the last slot's need room
    const int slots = (p.k_blocks + kSlotBlocks - 1) / kSlotBlocks;
    const int x_slot = kSlotBlocks * (p.tile_r / 2) * kBlockK, slack = (kRowsCta - p.rows_cta) * kBlockK;
    p.resident_bytes = p.r_tiles == 1 && slots <= kResidentBytes / x_slot ? slots * x_slot : 0;
    p.stage_bytes = kSlotBlocks * p.rows_cta * kBlockK + (p.resident_bytes ? 0 : x_slot);
    p.staged = R > kFewPositions;
    const int fixed = kBarrierBytes + 1024 + (p.staged ? 4 * kStageBytes : 0) + p.resident_bytes + slack;
    p.stages = std::min(kMaxStages, (kSmemLimit - fixed) / p.stage_bytes);
    p.idesc = idesc_e4m3_f32(kTileV, p.tile_r);
    p.stream_table = p.r_tiles == 1;
    p.stream_logits = R * V * entry_size(dtype) > (64LL << 20);
    p.x_scale = x_scale;
    p.w_scale = scale;
    p.logits = logits;
    p.ldl = ldl;
    CUtensorMap tm_x, tm_w, tm_x2, tm_w2;
    if (!encode_codes(encode, &tm_x, &tm_x2, X, R, d, ldx, p.tile_r / 2) ||
        !encode_codes(encode, &tm_w, &tm_w2, Q, V, d, ldq, p.rows_cta)) {
        *msg = "a tensor map of the head's codes could not be encoded";
        return cudaErrorInvalidValue;
    }
    CUtensorMap tm_out = tm_x;  // (not used without staging)
    if (p.staged) {
        const cuuint64_t dims[2] = {(cuuint64_t)V, (cuuint64_t)R}, strides[1] = {(cuuint64_t)ldl * entry_size(dtype)};
        const cuuint32_t boxes[2] = {(cuuint32_t)p.rows_cta,
                                     (cuuint32_t)(dtype == DG_BF16 ? kTokens<__nv_bfloat16> : kTokens<float>)};
        const cuuint32_t estr[2] = {1, 1};
        if (encode(&tm_out, dtype == DG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, logits,
                   dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                   CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
            *msg = "a tensor map of the head's logits could not be encoded";
            return cudaErrorInvalidValue;
        }
    }
    const cudaError_t e = ensure_head_attributes();
    if (e != cudaSuccess) return e;
    const unsigned grid = 2 * (unsigned)std::min(p.tiles, pairs);
    // (a CTA takes all of an SM's TMEM: no other one beside it)
    const int smem = std::max(fixed + p.stages * p.stage_bytes, kSmemLimit / 2 + 1024);
    if (dtype == DG_BF16)
        head_kernel<__nv_bfloat16><<<grid, kThreads, smem, stream>>>(tm_x, tm_w, tm_x2, tm_w2, tm_out, p);
    else
        head_kernel<float><<<grid, kThreads, smem, stream>>>(tm_x, tm_w, tm_x2, tm_w2, tm_out, p);
    return cudaGetLastError();
}

}  // namespace dg
