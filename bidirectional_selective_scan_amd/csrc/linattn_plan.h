// Host side of linear attention: execution plans and every argument check an entry point makes before
// its first HIP call. Plain C++, as plan.h.
#ifndef VIMSCAN_LINATTN_PLAN_H
#define VIMSCAN_LINATTN_PLAN_H

#include <cstddef>
#include <cstdint>

#include "vimscan.h"

namespace vimscan_host {

constexpr int64_t kLinMaxDim = 128;    // of dk and dv
constexpr int kLinChunk = 32;          // tokens that a wave works on at once
// Tokens that a sum of the decays' gradient reaches over. Between windows the state and its gradient are written, read and multiplied
// (8 dk dv bytes each way): backward of 128 x 197 x 12 heads of 64 x 64 bf16, us, windows of 64: 199, 128: 160, 256: 152, sequences whole: 146;
// 1 x 16385 x 24: 364, 308, 276, 250. Shorter ones keep a token's rounding (and NaN) nearer to it.
constexpr int kLinWindow = 128;
constexpr int64_t kLinLongest = 8192;   // tokens of packed sequences that a plan may leave whole on their mean alone
constexpr int64_t kMaxHeadStride = int64_t(1) << 38;
// Workgroups of 64 threads (a wave) and of 256: a grid holds fewer than 2^32 threads.
constexpr int64_t kMaxLinWaves = (int64_t(1) << 26) - 1, kMaxLinWgs = (int64_t(1) << 24) - 1;

// Tiles of 16 that a wave's state has over a contracted dimension (at least as wide as it) and over an
// output dimension, of which a wave takes a block of 2 or 4. Two in fp32 and over more than 64 contracted channels, where four
// leave room for one wave a SIMD (64 packed x up to 1025 x 24 heads of 128 x 64 bf16: 228 us, 337 with four; 1 x 2048 x 8 of
// 64 x 64 fp32, forward and backward: 117 us, 151 with four); in bf16 four are faster else (128 x 197 x 12 of 64 x 64,
// forward and backward: 207 us, 263 with two).
constexpr int lin_contract_tiles(int64_t d) { return d <= 32 ? 2 : d <= 64 ? 4 : 8; }
constexpr int lin_output_tiles(int bytes, int64_t k, int64_t v) { return v <= 32 || k > 64 || bytes == 4 ? 2 : 4; }
constexpr int64_t lin_blocks(int bytes, int64_t k, int64_t v) {
    return (v + 16 * lin_output_tiles(bytes, k, v) - 1) / (16 * lin_output_tiles(bytes, k, v));
}

// Waves a SIMD that the registers of a pass are cut for (512 a SIMD lane; measured: cut for more, they spill).
constexpr int lin_waves_per_simd(int bytes, int nk, int nv) {
    return bytes == 4 ? (nk * nv <= 4 ? 3 : nk * nv <= 8 ? 2 : 1) : nk * nv <= 4 ? 4 : nk * nv <= 8 ? 3 : nk * nv <= 16 ? 2 : 1;
}

struct LinPlan {
    int64_t tokens, nseq, Lp;          // Lp: tokens per sequence, 0 when packed
    int64_t H, G, dk, dv;
    bool packed, split;
    int64_t seg, segs, slots;          // split: tokens per segment, segments per uniform sequence; segments in all
    int64_t waves;                     // of the pass that writes y (or dv)
    // workspace: the segments' states and decays; backward also their gradients, the terms of the decays'
    // gradient, and gradients of shared q and k by head
    size_t off_s, off_e, off_tot, off_rq, off_rk, off_cd, off_hs, off_pq, off_pk, ws;
    // at its end, for the decays' gradient alone: the borders of windows inside segments, and the state, its gradient and their product
    // at each
    int64_t borders, seg_borders;      // in all; of a segment of a uniform sequence
    size_t off_ms, off_me, off_bd, ws_plain;   // ws_plain: what a backward pass without the decays' gradient needs
};

// Numbers that waves hold of a head's state, all blocks of output channels, whole tiles.
constexpr int64_t lin_state_floats(int bytes, int64_t k, int64_t v) {
    return int64_t(256) * lin_contract_tiles(k) * lin_output_tiles(bytes, k, v) * lin_blocks(bytes, k, v);
}

// Whether passes (contracted, output) = (k, v) and (v, k) can be one launch: the same instance, equally many waves.
constexpr bool lin_alike(int bytes, int64_t k, int64_t v) {
    return lin_contract_tiles(k) == lin_contract_tiles(v) && lin_output_tiles(bytes, k, v) == lin_output_tiles(bytes, v, k) &&
           lin_blocks(bytes, k, v) == lin_blocks(bytes, v, k);
}

// Packed sequence q takes the slots from offsets[q] / seg + q on: up to the next sequence's first these are
// floor(offsets[q + 1] / seg) - floor(offsets[q] / seg) + 1 >= ceil(length / seg), one for each of its segments.
int make_linattn_plan(const vimscan_launch* l, int64_t seg_len, int64_t heads, int64_t groups, bool packed, int64_t nseq,
                      bool backward, LinPlan* p);
int check_linattn_call(const vimscan_linattn* a, const void* y, const float* h_last, const vimscan_linattn_grad* grad,
                       const vimscan_launch* l, const LinPlan& p);
int check_linattn_step(const vimscan_linattn* a, const float* state, int64_t nslots, const int32_t* slots_in,
                       const int32_t* slots_out, const void* y, const vimscan_launch* l);

}  // namespace vimscan_host

#endif  // VIMSCAN_LINATTN_PLAN_H
