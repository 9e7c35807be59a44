// Host side of the recurrent block's operators (gated recurrence, block norm): execution plans and
// every argument check an entry point makes before its first HIP call. Plain C++, as plan.h.
#ifndef VIMSCAN_BLOCK_PLAN_H
#define VIMSCAN_BLOCK_PLAN_H

#include <cstddef>
#include <cstdint>

#include "vimscan.h"

namespace vimscan_host {

constexpr int kGatedStride = VIMSCAN_GATED_STRIDE;
constexpr int64_t kMaxRowStride = int64_t(1) << 24;
constexpr int64_t kMaxGatedWgs = int64_t(1) << 24;  // x 256 threads: a grid's limit of 2^32 threads
constexpr int64_t kNormMaxWidth = 32768;

// Plan of a gated recurrence over whole sequences.
struct GatedPlan {
    int64_t tokens, nseq, Lp;  // Lp: tokens per sequence, 0 when packed
    int64_t ncb, wgs;
    bool packed;
    size_t off_dlam, ws;
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
