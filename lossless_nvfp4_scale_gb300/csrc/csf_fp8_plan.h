// Which kernel of csf_fp8.cuh a call of csf_fp8_matmul takes, and what it is
// launched with: arithmetic on the call's sizes, for the host alone.  Internal
// to the library.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace csfk {
namespace f8 {

constexpr int kMaxStages = 8;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kMaxExperts = 8192;
constexpr int kMaxSplit = 8;
constexpr int kSplitSlots = 64;          // slots of a tile that a cluster shares
constexpr uint32_t kTileBytes = 128 * 128;
constexpr int kSumWarps = 8;
constexpr uint32_t kTurnBytes = kSumWarps * 32 * 128;      // a piece of 32 rows of 128 bytes each
// Steps whose factors are held: those of the ring's stages, and of partial
// sums that are formed (4 steps at most) or taken out.
constexpr int kFactorSteps = 16;
static_assert(kFactorSteps >= kMaxStages + 5, "factors are written when their stage is free");

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages], acc_full[4], acc_empty[4];
    uint32_t tmem, abort, warp_sum[16];
    float amax[2][2][128];       // by tile, half and row
};

// Tiles of 128 or 256 columns, or those with the depth shared.
enum Shape { kOne = 0, kTwo = 1, kOneShared = 2, kTwoShared = 3 };

struct Call {
    int sms;             // of the device
    int64_t slots;
    int32_t experts;
    int32_t F, blocks;   // output columns, blocks of 128 of the depth
    bool gated;
};

struct Plan {
    int shape, split;            // split: blocks of a cluster that share a tile's depth
    int32_t nt;                  // most slots per tile
    int32_t tile_step, row_tiles;   // columns of the weights' outputs from a tile to the next, tiles of them
    int32_t stages;              // fewer than 2: there is no room
    uint32_t stage_bytes;
    int64_t smem;                // dynamic shared memory
    int64_t most_tiles;          // at most
};

inline void lay(Plan &p, const Call &c, int shape) {
    const bool wide = shape == kTwo || shape == kTwoShared;
    const int64_t busy = std::min<int64_t>(c.experts, c.slots);
    p.shape = shape;
    p.tile_step = wide && !c.gated ? 256 : 128;
    p.row_tiles = (c.F + p.tile_step - 1) / p.tile_step;
    p.nt = shape >= kOneShared ? kSplitSlots : 128;
    p.stage_bytes = kTileBytes * (wide ? 3 : 2);
    const int64_t region = shape >= kOneShared ? (int64_t)kSplitSlots * 512 * (shape == kTwoShared ? 2 : 1) : kTurnBytes;
    const int64_t fixed = 1024 + region + 8 * ((int64_t)c.experts + 1) + 16;
    const int64_t held = ((int64_t)sizeof(Shared) + kFactorSteps * 512 * (wide ? 2 : 1) + 1023) / 1024 * 1024;
    p.stages = (int32_t)std::min<int64_t>(kMaxStages, (kSmemLimit - held - fixed) / p.stage_bytes);
    p.smem = std::max<int64_t>(fixed + p.stages * (int64_t)p.stage_bytes, 120 * 1024);      // never two blocks on an SM: each holds the whole tensor memory
    p.most_tiles = (int64_t)p.row_tiles * (busy + c.slots / p.nt);
}

inline Plan plan_of(const Call &c) {
    const int64_t busy = std::min<int64_t>(c.experts, c.slots);      // experts with slots, at most
    // A tile's width by the rounds of tiles that it takes, a round of 128 columns
    // 0.65 of one of 256 as measured with 5120 columns and depth.  Experts' last
    // slot tiles are half full on average.  512 / 2048 / 8191 slots of a dense 5120
    // x 5120: 128 columns 31 / 71 / 236 us, 256 24.3 / 64.2 / 193.
    auto tiles_of = [&](int step) {
        const int64_t rows = c.experts == 1 ? (c.slots + 127) / 128 : std::max(busy, busy / 2 + c.slots / 128);
        return rows * ((c.F + step - 1) / step);
    };
    const int units = std::max(c.sms, 1);
    auto rounds = [&](int64_t t) { return (double)((t + units - 1) / units); };
    const int whole = !c.gated && 0.65 * rounds(tiles_of(128)) <= rounds(tiles_of(256)) ? kOne : kTwo;
    Plan p;
    p.split = 1;
    lay(p, c, whole);
    // Few tiles, whatever they would be: clusters share their depth.  Clusters of
    // half the SMs' blocks are placed at once, larger ones than pairs of more in
    // turns: one slot of 2048 x 5120 takes 14.5 us in 16 clusters of 8 and 9.3 in
    // 16 of 4, of 5120 x 5120 15.4 in 40 blocks and 12.3 in 40 pairs.
    const int64_t slot_tiles = c.experts == 1 ? (c.slots + kSplitSlots - 1) / kSplitSlots : busy + c.slots / kSplitSlots;
    const int64_t few = (int64_t)((c.F + 127) / 128) * slot_tiles;
    while (p.split < kMaxSplit && few * p.split * 2 <= (p.split == 1 ? c.sms : c.sms / 2) && c.blocks >= 4 * p.split) p.split *= 2;
    // Gated, the sums handed round are twice as many: two blocks share where few
    // rows or much depth pay for them.  1 / 32 / 64 slots of 8192 x 2048 take 12.6 /
    // 13.9 / 16.4 us in twos and 13.9 / 14.3 / 14.9 whole, 256 of 4096 x 5120 23.9
    // and 24.6; in fours and eights all gain (64 of 1024 x 2048 10.9 and 12.7, 1 of
    // 4096 x 5120 14.9 and 23.3).
    const int64_t tiles_with_slots = c.experts == 1 ? slot_tiles : busy;
    if (c.gated && p.split == 2 && c.slots > 32 * tiles_with_slots && c.blocks < 32) p.split = 1;
    if (p.split > 1) {
        lay(p, c, c.gated ? kTwoShared : kOneShared);      // (fewer columns, so that more blocks have some)
        if (p.stages < 2) {      // many experts' prefixes leave too little for the sums handed round
            p.split = 1;
            lay(p, c, whole);
        }
    }
    return p;
}

}  // namespace f8
}  // namespace csfk
