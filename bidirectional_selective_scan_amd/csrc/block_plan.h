// Host side of the recurrent block's operators (gated recurrence, block norm): execution plans and
// every argument check an entry point makes before its first HIP call. Plain C++, as plan.h.
#ifndef VIMSCAN_BLOCK_PLAN_H
#define VIMSCAN_BLOCK_PLAN_H

#include <cstddef>
#include <cstdint>

#include "vimscan.h"

namespace vimscan_host {

constexpr int kGatedStride = VIMSCAN_GATED_STRIDE;
// Rows of a tile (128 at most) lie within the 2^31 bytes that one buffer resource's offsets span.
constexpr int64_t kMaxRowStride = int64_t(1) << 22;
// Workgroups of 256 threads: a grid holds fewer than 2^32 threads. (So few tiles also keep every position of
// the last tile below 2^31.)
constexpr int64_t kMaxGatedWgs = (int64_t(1) << 24) - 1;
// Single tokens: rows x parts of 64 channels.
constexpr int64_t kMaxStepParts = int64_t(1) << 24;
constexpr int64_t kNormMaxWidth = 32768;

// Tiling of the gated recurrence: a workgroup of 256 threads takes kGatedBlock channels of a tile of
// tokens, each thread tile * kGatedBlock / 256 elements.
constexpr int kGatedBlock = 64;
constexpr int kGatedFwdTile = 128;
constexpr int kGatedFwdTileSmall = 64;
constexpr int kGatedBwdTile = 64;
// Tiles per group of the hand-over: a tile folds the aggregates of the tiles before it in its group
// onto the state that the group before left.
constexpr int kGatedGroup = 16;
static_assert(kGatedBwdTile == kGatedStride, "the backward pass starts each tile from a saved state");

// Plan of a gated recurrence over whole sequences.
struct GatedPlan {
    int64_t tokens, nseq, Lp;      // Lp: tokens per sequence, 0 when packed
    int64_t tile, tiles, groups;   // tokens per workgroup, workgroups along the tokens, hand-over groups
    int64_t ncb, wgs;
    bool packed;
    bool chain;                    // tiles hand states on to each other
    // workspace: tile maps and group states of the hand-over, partial sums of dlam
    size_t off_inc, off_part, ws;
};

int make_gated_plan(const vimscan_launch* l, int64_t seg_len, bool packed, int64_t nseq, bool backward, GatedPlan* p);
// The checks of a call after its plan. grad is NULL for the forward pass; y, h_last and states are
// those of the forward pass.
int check_gated_call(const vimscan_gated* g, const void* y, const float* h_last, const float* states,
                     const vimscan_gated_grad* grad, const vimscan_launch* l, const GatedPlan& p);
int check_gated_step(const vimscan_gated* g, const float* state, int64_t nslots, const int32_t* slots_in,
                     const int32_t* slots_out, const void* y, const vimscan_launch* l);

// Plan of a block norm: how a row is spread over lanes.
struct NormPlan {
    int64_t rows, D;
    int64_t wgs, rows_per_wg;
    size_t ws;
};

int make_norm_plan(const vimscan_launch* l, bool backward, NormPlan* p);
int check_norm_call(const vimscan_norm* n, const void* sum, const void* out, const vimscan_norm_grad* grad,
                    const vimscan_launch* l, const NormPlan& p);

}  // namespace vimscan_host

#endif  // VIMSCAN_BLOCK_PLAN_H
