// Host side of the recurrent block's operators (gated recurrence, block norm, layer norm): execution plans and
// every argument check an entry point makes before its first HIP call. Plain C++, as plan.h.
#ifndef VIMSCAN_BLOCK_PLAN_H
#define VIMSCAN_BLOCK_PLAN_H

#include <cstddef>
#include <cstdint>

#include "vimscan.h"

namespace vimscan_host {

constexpr int kGatedStride = VIMSCAN_GATED_STRIDE;
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

// How a block norm's row is spread: over lanes of one wave (waves = 1) or over waves of 64, each lane nv vectors of
// vec channels. A workgroup of 256 threads works on several narrow rows at once; wide rows take one of up to 1024.
struct NormSpread {
    int nv, lanes, waves, vec;
    constexpr int64_t width() const { return int64_t(nv) * lanes * waves * vec; }   // channels at most
    constexpr int threads() const { return waves > 4 ? 64 * waves : 256; }
    constexpr int rows() const { return threads() / (lanes * waves); }
};
// The spreads from narrow to wide; a row takes the first that holds it. Forward fewer waves with more of a row
// each; backward, where a channel takes three times the registers, more waves past 1024 channels (all stages, fp32
// residuals: 13056 x 1536 bf16 91 us with 8 waves, 93 with the forward's 4; 4099 x 8192 all bf16 176 us with 16
// waves, which keep the weights' gradients in LDS, 251 with the forward's 8, which spill).
constexpr NormSpread kNormForward[] = {{1, 16, 1, 4}, {1, 32, 1, 4}, {1, 64, 1, 4}, {2, 64, 1, 4},
                                       {3, 64, 1, 4}, {4, 64, 1, 4}, {2, 64, 4, 4}, {4, 64, 4, 4},
                                       {4, 64, 8, 4}, {4, 64, 16, 4}, {8, 64, 16, 4}};
constexpr NormSpread kNormBackward[] = {{1, 16, 1, 4}, {1, 32, 1, 4}, {1, 64, 1, 4}, {2, 64, 1, 4},
                                        {3, 64, 1, 4}, {4, 64, 1, 4}, {1, 64, 8, 4}, {1, 64, 16, 4},
                                        {2, 64, 16, 4}, {4, 64, 16, 4}, {8, 64, 16, 4}};
// fp32 rows whose width is no multiple of 4: single channels, either direction.
constexpr NormSpread kNormSingles[] = {{4, 16, 1, 1}, {4, 32, 1, 1}, {4, 64, 1, 1}, {8, 64, 1, 1}, {4, 64, 4, 1},
                                       {4, 64, 8, 1}, {8, 64, 8, 1}, {8, 64, 16, 1}, {16, 64, 16, 1}, {32, 64, 16, 1}};

// Plan of a block norm. A workgroup takes spread.rows() rows at a time.
struct NormPlan {
    int64_t rows, D;
    int64_t wgs, rows_per_wg;      // workgroups launched, and the rows that the first of them takes
    size_t ws;                     // rows of partial weight gradients for each (three; of a layer norm two)
};

int make_norm_plan(const vimscan_launch* l, bool backward, NormPlan* p);
// Of a layer norm: the same spreads, two rows of partial weight gradients.
int make_layernorm_plan(const vimscan_launch* l, bool backward, NormPlan* p);
int check_layernorm_call(const vimscan_layernorm* n, const void* sum, const void* out, const vimscan_layernorm_grad* grad,
                         const vimscan_launch* l, const NormPlan& p);
int check_norm_call(const vimscan_norm* n, const void* sum, const void* out, const vimscan_norm_grad* grad,
                    const vimscan_launch* l, const NormPlan& p);

}  // namespace vimscan_host

#endif  // VIMSCAN_BLOCK_PLAN_H
