// How the loss kernels cut rows into tiles, and what follows from it: the passes a call makes over its rows
// and whether it takes a workspace.  Host arithmetic without CUDA, which row_loss.cu launches by and the
// entry points check their workspace by.
#pragma once

#include <stdint.h>

namespace dg {

// What a row's loss is taken from.
enum RowLossHead {
    kHeadToken = 0,   // the log-probability of one token per row
    kHeadDistill = 1  // a teacher's top logits
};
// Which passes a call makes over a row.
enum RowLossPass {
    kPassForward = 1,   // statistics and losses
    kPassBackward = 2,  // the gradient from the statistics a forward call saved
    kPassStep = 3       // both in one call
};

constexpr int kMaxTopK = 1024;

constexpr int kMaxStages = 16;
// Shared memory of the ring of stages: a CTA's 227 KB but for what is not the ring's (row_loss.cu's Shared).
constexpr int kSharedBytes = 4112;
constexpr int kRingBytes = 227 * 1024 - kSharedBytes;
constexpr int kListBytes = 12;  // per entry of a teacher's table and stage
// Bytes of a row that is one tile: with 32 KB, so two tiles and an exchange, a policy step of 2,048 x 12,000
// fp32 entries takes 43.7 us instead of 35.1.
constexpr int kMaxTile = 64 * 1024;
// Stages that the tiles of longer rows leave room for.  1,024 x 262,144, policy step fp32 and distillation
// step (K = 64) bf16, us: 5 stages 360 and 194, 7 stages 353 and 197, 9 (tiles of 24 KB) 356 and 217, 14 356
// and 239.  A long list of a teacher's entries is looked through once per tile: K = 512, fp32, 5 stages 412,
// 7 stages 423; K = 1,024 493 and 534.
constexpr int kFewEntries = 256;
constexpr int good_stages(int K) { return K > kFewEntries ? 5 : 7; }
// Bytes that a list of K entries (K = 0: tokens) leaves a tile beside it.
constexpr int tile_bytes(int K) { return kRingBytes / good_stages(K) - K * kListBytes; }
static_assert(tile_bytes(kFewEntries) >= 24 * 1024 && tile_bytes(kMaxTopK) >= 24 * 1024, "tiles of fewer bytes are slower");

// Tiles of a row: the whole row up to kMaxTile bytes, else equal parts, in whole 128-byte lines, of
// which good_stages(K) fit the ring beside their lists.
struct Tiling {
    int tile_vecs, tiles;
};
inline Tiling tile_row(int64_t V, int element_size, int K) {
    const int64_t nv = V * element_size / 16;
    if (nv * 16 <= kMaxTile) return Tiling{(int)((nv + 7) / 8 * 8 > 0 ? (nv + 7) / 8 * 8 : 8), 1};
    const int64_t limit = tile_bytes(K) / 128 * 8;  // vectors
    const int64_t n = (nv + limit - 1) / limit;
    const int64_t per = ((nv + n - 1) / n + 7) / 8 * 8;
    return Tiling{(int)per, (int)((nv + per - 1) / per)};
}

// A stage holds a tile and the tile's list of a teacher's K entries.
inline int stage_bytes(const Tiling &t, int K) { return t.tile_vecs * 16 + K * kListBytes; }
inline int ring_stages(const Tiling &t, int K) {
    const int n = kRingBytes / stage_bytes(t, K);
    return n < kMaxStages ? n : kMaxStages;
}

// Whether a step over R rows reads them twice, a forward pass and a backward pass with the workspace between
// them.  A row in one read stays in the rings until it is complete: a CTA must have room for its share of one
// row and the next.  A row of one tile waits for no other CTA, so that its own stage is enough.
inline bool reads_twice(const Tiling &t, int K, int64_t R, int sms) {
    if (t.tiles == 1) return false;
    const int64_t grid = R * t.tiles < sms ? R * t.tiles : sms;
    return (t.tiles + grid - 1) / grid + 2 > ring_stages(t, K);
}

// Whether a call uses the workspace: sums that CTAs exchange, what a forward pass leaves for a backward pass,
// or the rows' numbers that row_close_kernel works out.
inline bool takes_workspace(int64_t V, int element_size, RowLossHead head, RowLossPass pass) {
    return tile_row(V, element_size, 0).tiles > 1 || (head == kHeadDistill && pass == kPassBackward);
}

}  // namespace dg
