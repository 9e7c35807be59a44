// Device code of linear attention with a decay for each head (include/vimscan.h, vimscan_linattn_*): the pass
// over whole sequences that the forward and the backward kernels share.
//
// The pass. With a reader r (rows of K numbers), a key k (K) and a value v (V numbers) for every token, and
// decays a_t = exp(g_t):
//     S_t = a_t S_{t-1} + k_t^T v_t,   o_t = r_t S_t
// The forward pass is (q, k, v); the gradient of q is (dy, v, k), those of k and v are (v, dy, q) and (k, q, dy)
// from the sequence's end, their decays moved by one token. In chunks of 32 tokens, G_t the sum of g over the chunk up to t:
//     o_t = e^{G_t} r_t S_in + sum_{s <= t} e^{G_t - G_s} (r_t . k_s) v_s,   S_out = e^{G_end} S_in + sum_s e^{G_end - G_s} k_s^T v_s
// so all but the decays is matrix products.
//
// What bounds it: memory, up to heads of 64 x 64 (bf16: 512 bytes and 55 matrix instructions of 16 cycles a token and head). So a
// wave does all of a head (or 64 output channels of it) alone: it reads every number once, the state never leaves
// its registers, and nothing waits for another wave. The operands are laid out so that what one product leaves
// in the accumulators is the next one's operand as it stands (lane = 16 grp + col):
//   * the scores are formed transposed, rows = key tokens, columns = reader tokens: a lane holds the tokens 4 grp + 0..3
//     of a column, which is how the next product (values times scores) takes its right operand;
//   * o is formed transposed too, rows = channels: a lane ends with 4 NV consecutive channels of one token;
//   * the state has rows = key channels, columns = value channels; row m of its tile i is channel NK m + i, column m
//     of its tile j is channel NV m + j, so a lane reads NK (or NV) consecutive channels of its tokens, and as the left
//     operand of r S it is in place as well.
// bf16: the numbers of the inputs are exact operands. Those in fp32 (state, scores, decayed keys) are split
// into two bf16 parts, both multiplied: 16 of their 24 bits, 2^-17 relative, far below the outputs' rounding; one part alone
// would leave 2^-9 in the state, which is fp32 in memory. fp32: fp32 matrix instructions.
// Sums of g are in fp64, and their differences taken from a pair of fp32, so that a token of strong decay does not cost its
// neighbours digits.
#ifndef VIMSCAN_LINATTN_DEVICE_H
#define VIMSCAN_LINATTN_DEVICE_H

#include <hip/hip_runtime.h>

#include <cstdint>

#include "block_device.h"
#include "linattn_plan.h"

namespace vimscan_dev {

constexpr int kChunk = vimscan_host::kLinChunk;
constexpr int kWaves = vimscan_host::kLinWaves;
// An offset outside every buffer resource: the hardware gives 0 for such a load and drops such a store.
constexpr uint32_t kOutside = 0x80000000u;
constexpr int kRsrcFlags = 0x00020000;

using V4f = float __attribute__((ext_vector_type(4)));
using V8bf = __bf16 __attribute__((ext_vector_type(8)));
using U4 = uint32_t __attribute__((ext_vector_type(4)));
using U2v = uint32_t __attribute__((ext_vector_type(2)));
using S2 = uint16_t __attribute__((ext_vector_type(2)));

// Which of the kernels a pass is.
enum LinKind {
    kLocal,    // the state that a segment adds, from nothing
    kForward,  // the operator itself
    kGradient  // a gradient, and its part of the decays'
};

// [tokens][heads / div][D] with strides in elements.
struct LinRows {
    const void* p;
    int64_t ld, hs;
    int32_t div;
};

struct LinArgs {
    LinRows r, k, v;
    int32_t H, K, V;           // heads, contracted and output dimension
    int32_t blocks;            // of output channels
    const float* g;
    int64_t ld_g;              // 0: one for each head
    const int32_t* offsets;
    int64_t tokens, Lp, seg;
    int32_t nseq, segs, split, rev;
    int64_t slots, waves;
    int32_t back;              // walk from the segment's end (on top of rev), decays moved by one
    float key_scale, out_scale;
    // state before the segment: of its sequence or, by_slot, of itself; NULL: 0. Element (i, j) is at i row + j col
    const float* s0;
    int64_t s0_row, s0_col;
    int32_t s0_by_slot;
    float* s_end;              // kLocal: of the segment; else of the sequence, written by its last segment; dense K x V
    float* tot;                // kLocal: the segment's decay
    void* o;                   // [tokens][H][V], dense
    int32_t o_f32;             // in fp32 whatever the io type
    // kGradient, where the decays' gradient is wanted: dots[block][token][head] = w . o without a token's pair with itself
    LinRows w;
    float* dots;
    const float* e;            // gradient of the state behind the segment (as s0); cdot[slot][head][block] = <S, e>
    int64_t e_row, e_col;
    int32_t e_by_slot;
    float* cdot;
};

// A segment of a sequence, in tokens: walking positions w0 .. w0 + n of the sequence, at rows first .. first + n.
struct LinSegment {
    int64_t seq, first;
    int64_t n;
    bool valid, head, last;    // the sequence's first or last segment
};

__device__ __forceinline__ int64_t uniform(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(static_cast<uint64_t>(v) >> 32));
    return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

// The bounds of a packed sequence; offsets that break their rules still give rows inside the arrays.
__device__ __forceinline__ void lin_bounds(const LinArgs& a, int64_t seq, int64_t* lo, int64_t* hi) {
    int64_t x = a.offsets[seq], y = a.offsets[seq + 1];
    x = x < 0 ? 0 : x > a.tokens ? a.tokens : x;
    y = y < x ? x : y > a.tokens ? a.tokens : y;
    *lo = x;
    *hi = y;
}
__device__ __forceinline__ int64_t lin_base(const LinArgs& a, int64_t seq) {
    int64_t x = a.offsets[seq];
    x = x < 0 ? 0 : x > a.tokens ? a.tokens : x;
    return x / a.seg + seq;
}

__device__ __forceinline__ LinSegment lin_segment(const LinArgs& a, int64_t slot) {
    LinSegment s;
    int64_t lo, hi, j = 0;
    if (!a.offsets) {
        s.seq = slot / a.segs;
        j = slot - s.seq * a.segs;
        lo = s.seq * a.Lp;
        hi = lo + a.Lp;
    } else {
        if (a.split) {
            // the sequence whose slots start at or before this one: 64 candidates at a time
            int64_t from = 0, to = a.nseq;
            while (to - from > 1) {
                const int64_t step = (to - from + 63) / 64, at = from + static_cast<int64_t>(threadIdx.x & 63) * step;
                const bool before = at < to && lin_base(a, at) <= slot;
                const int cnt = __popcll(__ballot(before));
                from += (cnt > 0 ? cnt - 1 : 0) * step;
                to = to < from + step ? to : from + step;
            }
            s.seq = from;
            j = slot - lin_base(a, from);
        } else {
            s.seq = slot;
        }
        lin_bounds(a, s.seq, &lo, &hi);
    }
    const int64_t len = hi - lo, w0 = a.split ? j * a.seg : 0;
    const int64_t w1 = a.split && w0 + a.seg < len ? w0 + a.seg : len;
    s.valid = j == 0 || (j > 0 && w0 < len);
    s.head = j == 0;
    s.last = w1 == len;
    s.n = uniform(w1 - w0);
    s.first = uniform(a.rev ? hi - w1 : lo + w0);
    s.seq = uniform(s.seq);
    return s;
}

// The state before (or the gradient behind) a segment.
__device__ __forceinline__ const float* lin_state(const float* p, int32_t by_slot, int64_t slot, int64_t seq, const LinArgs& a,
                                                  int64_t h) {
    return p ? p + ((by_slot ? slot : seq) * a.H + h) * (static_cast<int64_t>(a.K) * a.V) : nullptr;
}

// ---------------------------------------------------------------------------------------------
// Rows in registers

// 4 N consecutive channels of one token, from channel 4 N grp on.
template <typename IO, int N> struct RowPart;
template <int N> struct RowPart<Bf16, N> {
    uint32_t w[2 * N];
    __device__ __forceinline__ float get(int k) const { return (k & 1) ? bf16_hi(w[k / 2]) : bf16_lo(w[k / 2]); }
};
template <int N> struct RowPart<float, N> {
    float w[4 * N];
    __device__ __forceinline__ float get(int k) const { return w[k]; }
};
// N consecutive channels, from channel N col on, of the tokens 4 grp + 0..3 and 16 + 4 grp + 0..3 of a chunk.
template <typename IO, int N> struct ColPart;
template <int N> struct ColPart<Bf16, N> {
    uint32_t w[8][N / 2];
    __device__ __forceinline__ float get(int t, int k) const { return (k & 1) ? bf16_hi(w[t][k / 2]) : bf16_lo(w[t][k / 2]); }
};
template <int N> struct ColPart<float, N> {
    float w[8][N];
    __device__ __forceinline__ float get(int t, int k) const { return w[t][k]; }
};

// n dwords at an offset.
template <int kDwords>
__device__ __forceinline__ void load_dwords(__amdgpu_buffer_rsrc_t rsrc, uint32_t vo, uint32_t* o) {
    if constexpr (kDwords == 1) {
        o[0] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, vo, 0, 0);
    } else if constexpr (kDwords == 2) {
        const U2v w = __builtin_bit_cast(U2v, __builtin_amdgcn_raw_buffer_load_b64(rsrc, vo, 0, 0));
        o[0] = w[0];
        o[1] = w[1];
    } else {
        static_assert(kDwords % 4 == 0, "whole vectors");
#pragma unroll
        for (int k = 0; k < kDwords / 4; ++k) {
            const U4 w = __builtin_bit_cast(U4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, vo + 16 * k, 0, 0));
#pragma unroll
            for (int j = 0; j < 4; ++j) o[4 * k + j] = w[j];
        }
    }
}

// N channels from channel c of a row at an offset, those past D read as 0. kVec: all or none of them are below D.
template <typename IO, int N, bool kVec, typename W>
__device__ __forceinline__ void load_channels(__amdgpu_buffer_rsrc_t rsrc, uint32_t row, int c, int D, W* out) {
    constexpr int e = sizeof(IoElem<IO>);
    uint32_t* o = reinterpret_cast<uint32_t*>(out);
    if constexpr (kVec) {
        load_dwords<N * e / 4>(rsrc, c < D ? row + static_cast<uint32_t>(c * e) : kOutside, o);
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t at = c + k < D ? row + static_cast<uint32_t>((c + k) * e) : kOutside;
            if constexpr (e == 4) {
                o[k] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, at, 0, 0);
            } else {
                const uint32_t w = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(rsrc, at, 0, 0));
                if (k & 1) o[k / 2] |= w << 16;
                else o[k / 2] = w;
            }
        }
    }
}

// One array's rows of a head: where they are, and a chunk of them as a buffer resource.
template <typename IO, bool kVec>
struct HeadRows {
    uint64_t base;
    uint32_t ld;        // bytes from token to token
    int D;
    __amdgpu_buffer_rsrc_t rsrc;
    __device__ __forceinline__ void init(const LinRows& x, int64_t h, int d) {
        constexpr int e = sizeof(IoElem<IO>);
        base = reinterpret_cast<uint64_t>(x.p) + static_cast<uint64_t>(h / x.div * x.hs * e);
        ld = static_cast<uint32_t>(x.ld * e);
        D = x.p ? d : 0;    // (an array that is absent reads as 0)
    }
    // the rows of tokens first .. first + n, n <= kChunk
    __device__ __forceinline__ void chunk(int64_t first, int n) {
        constexpr int e = sizeof(IoElem<IO>);
        const int64_t at = uniform(static_cast<int64_t>(base + static_cast<uint64_t>(first) * ld));
        rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(at), 0, D > 0 ? (n - 1) * ld + D * e : 0, kRsrcFlags);
    }
    // the lane's part of row t of a chunk (t = its token in memory order; outside 0 .. n - 1: zeros)
    template <int N>
    __device__ __forceinline__ void part(int t, int grp, RowPart<IO, N>& o) const {
        constexpr int e = sizeof(IoElem<IO>);
        const uint32_t row = static_cast<uint32_t>(t) * ld;
        // (pieces of N channels; of two rather eight at once)
        constexpr int P = N == 2 ? 8 : N;
#pragma unroll
        for (int k = 0; k < 4 * N; k += P) load_channels<IO, P, kVec>(rsrc, row, 4 * N * grp + k, D, &o.w[k * e / 4]);
    }
    template <int N>
    __device__ __forceinline__ void columns(int (&t)[8], int c, ColPart<IO, N>& o) const {
#pragma unroll
        for (int k = 0; k < 8; ++k) load_channels<IO, N, kVec>(rsrc, static_cast<uint32_t>(t[k]) * ld, c, D, o.w[k]);
    }
};

// ---------------------------------------------------------------------------------------------
// Products. Two or three numbers that stand for one: in bf16 a value and its remainder.

struct Split8 {
    U4 hi, lo;
};
// The pair (a, b) at dword i of a split operand.
__device__ __forceinline__ void split_pair(Split8& s, int i, float a, float b) {
    const uint32_t h = bf16_pair(a, b);
    s.hi[i] = h;
    s.lo[i] = bf16_pair(a - bf16_lo(h), b - bf16_hi(h));
}
__device__ __forceinline__ V4f mfma(U4 a, U4 b, V4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V8bf, a), __builtin_bit_cast(V8bf, b), c, 0, 0, 0);
}
__device__ __forceinline__ V4f mfma(float a, float b, V4f c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// The operand of step s (32 channels) of a token's part.
template <int N>
__device__ __forceinline__ U4 row_operand(const RowPart<Bf16, N>& p, int s) {
    constexpr int m = N / 2;
    return U4{p.w[s], p.w[m + s], p.w[2 * m + s], p.w[3 * m + s]};
}
// Channel k of the eight tokens, as an operand over the tokens.
template <int N>
__device__ __forceinline__ U4 col_operand(const ColPart<Bf16, N>& p, int k) {
    const uint32_t sel = (k & 1) ? 0x07060302u : 0x05040100u;
    U4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __builtin_amdgcn_perm(p.w[2 * i + 1][k / 2], p.w[2 * i][k / 2], sel);
    return o;
}

// o += (state)^T (rows), for one tile of value channels and 16 tokens.
template <typename IO, int NK>
__device__ __forceinline__ V4f scores(const RowPart<IO, NK>& k, const RowPart<IO, NK>& r) {
    V4f c = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (sizeof(IoElem<IO>) == 2) {
#pragma unroll
        for (int s = 0; s < NK / 2; ++s) c = mfma(row_operand<NK>(k, s), row_operand<NK>(r, s), c);
    } else {
#pragma unroll
        for (int s = 0; s < 4 * NK; ++s) c = mfma(k.w[s], r.w[s], c);
    }
    return c;
}

// exp2 of the difference of two sums held as pairs.
__device__ __forceinline__ float decay_between(float2 to, float2 from) { return fast_exp2((to.x - from.x) + (to.y - from.y)); }

// Sum over the lanes up to this one of its half of the wave, in fp64.
template <int kCtrl, int kRows>
__device__ __forceinline__ double add_shifted(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), kCtrl, kRows, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), kCtrl, kRows, 0xf, true);
    return v + __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ double half_wave_sums(double v) {
    v = add_shifted<0x111, 0xf>(v);  // from the lane 1, 2, 4, 8 below in its row of 16
    v = add_shifted<0x112, 0xf>(v);
    v = add_shifted<0x114, 0xf>(v);
    v = add_shifted<0x118, 0xf>(v);
    return add_shifted<0x142, 0xa>(v);  // the last lane of rows 0 and 2 to rows 1 and 3
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(b), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), lane);
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ float2 as_pair(double v) {
    const float hi = static_cast<float>(v);
    return make_float2(hi, static_cast<float>(v - hi));
}
// A log decay in units of log 2. Below -200 (a factor of 0 in fp32) it is held there, so that sums of minus infinity have
// differences; NaN stays.
__device__ __forceinline__ double log2_decay(float g) { return static_cast<double>(g < -200.0f ? -200.0f : g) * 1.4426950408889634; }

__device__ __forceinline__ float over_groups(float v) {   // sum over the four lanes of a column
    float p, q;
    swap16(v, &p, &q);
    swap32(p + q, &p, &q);
    return p + q;
}

// Orders a wave's LDS accesses: its lanes read what others of them wrote.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Workgroup id -> logical id: the hardware deals workgroups to the 8 XCDs round-robin; this gives each XCD one
// contiguous range, so that heads that share rows (and a segment's blocks) meet in one L2.
__device__ __forceinline__ int64_t xcd_order(int64_t i, int64_t n) {
    const int64_t q = n >> 3, r = n & 7, x = i & 7, k = i >> 3;
    return (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + k;
}

// ---------------------------------------------------------------------------------------------
// The pass: one wave per segment, head and block of 16 NV output channels. NK tiles of 16 hold the K contracted
// channels.

template <typename IO, int NK, int NV, bool kVec, int kKind>
__global__ __launch_bounds__(64 * kWaves) void k_lin_pass(LinArgs a) {
    constexpr bool kBf16 = sizeof(IoElem<IO>) == 2;
    constexpr int e = sizeof(IoElem<IO>);
    __shared__ float2 sums[kWaves][kChunk];
    const int lane = static_cast<int>(threadIdx.x) & 63, wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int grp = lane >> 4, col = lane & 15;
    const int64_t task = xcd_order(blockIdx.x, gridDim.x) * kWaves + wave;
    if (task >= a.waves) return;
    const int block = static_cast<int>(task % a.blocks);
    const int64_t rest = task / a.blocks, h = rest % a.H, slot = rest / a.H;
    const LinSegment sg = lin_segment(a, slot);
    if (!sg.valid) return;
    const bool desc = (a.rev != 0) != (a.back != 0);
    const int c0 = block * 16 * NV, vc = c0 + NV * col, vr = c0 + 4 * NV * grp;   // the lane's value channels

    // state: S[i][j][r] = channel NK (4 grp + r) + i, channel vc + j
    V4f S[NK][NV];
    const int64_t ks = static_cast<int64_t>(a.K) * a.V;
    {
        const float* s0 = kKind == kLocal ? nullptr : lin_state(a.s0, a.s0_by_slot, slot, sg.seq, a, h);
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int x = NK * (4 * grp + r) + i, y = vc + j;
                    S[i][j][r] = s0 && x < a.K && y < a.V ? s0[x * a.s0_row + y * a.s0_col] : 0.0f;
                }
    }

    HeadRows<IO, kVec> R, K, V, W;
    R.init(a.r, h, a.K);
    K.init(a.k, h, a.K);
    V.init(a.v, h, a.V);
    if constexpr (kKind == kGradient) W.init(a.w, h, a.V);
    const bool dots = kKind == kGradient && a.dots;

    const int64_t n = sg.n;
    RowPart<IO, NK> rr[2], kr[2];
    ColPart<IO, NK> kc;
    ColPart<IO, NV> vcol;
    float gv = 0.0f;
    int64_t mem = 0;     // the chunk's lowest token
    int cnt = 0;
    auto place = [&](int64_t at, int64_t* first, int* c) {
        *c = static_cast<int>(n - at < kChunk ? n - at : kChunk);
        *first = desc ? sg.first + n - at - *c : sg.first + at;
    };
    // (walking position i of a chunk of c tokens is its row i or c - 1 - i)
    auto load = [&](int64_t at) {
        int64_t first;
        int c;
        place(at, &first, &c);
        auto row = [&](int i) { return desc ? c - 1 - i : i; };
        K.chunk(first, c);
        V.chunk(first, c);
        int t[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) t[k] = row((k & 4) * 4 + 4 * grp + (k & 3));
        if constexpr (kKind != kLocal) {
            R.chunk(first, c);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                K.part(row(16 * j + col), grp, kr[j]);
                R.part(row(16 * j + col), grp, rr[j]);
            }
        }
        K.columns(t, NK * col, kc);
        V.columns(t, vc, vcol);
        // the decay of the chunk's walking position lane % 32; moved by one token where the walk goes back
        const int i = lane & 31;
        const int64_t w = at + i - (a.back ? 1 : 0);
        gv = 0.0f;
        if (i < c && w >= 0) {
            const int64_t tok = desc ? sg.first + n - 1 - w : sg.first + w;
            gv = a.ld_g ? a.g[tok * a.ld_g + h] : a.g[h];
        }
    };

    double all = 0.0;    // sum of the decays so far
    if (n > 0) load(0);
    for (int64_t at = 0; at < n; at += kChunk) {
        place(at, &mem, &cnt);
        // sums of the log decays over the chunk
        const double run = half_wave_sums(log2_decay(gv));
        const double total = lane_value(run, 31);
        const float2 end = as_pair(total);
        if (kKind == kLocal) all += total;
        wave_sync();
        if (lane < kChunk) sums[wave][lane] = as_pair(run);
        wave_sync();
        float2 gs[8];    // of the lane's eight tokens
#pragma unroll
        for (int k = 0; k < 8; ++k) gs[k] = sums[wave][(k & 4) * 4 + 4 * grp + (k & 3)];

        V4f O[2][NV];
        [[maybe_unused]] float P[2][2][4];   // [key tile][reader tile], rows of keys
        if constexpr (kKind != kLocal) {
            // r S_in, then its decay
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int v = 0; v < NV; ++v) O[j][v] = V4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if constexpr (kBf16) {
#pragma unroll
                    for (int s = 0; s < NK / 2; ++s) {
                        Split8 st;
#pragma unroll
                        for (int i = 0; i < 4; ++i) split_pair(st, i, S[2 * s][v][i], S[2 * s + 1][v][i]);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const U4 x = row_operand<NK>(rr[j], s);
                            O[j][v] = mfma(st.hi, x, O[j][v]);
                            O[j][v] = mfma(st.lo, x, O[j][v]);
                        }
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int i = 0; i < NK; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j) O[j][v] = mfma(S[i][v][r], rr[j].w[NK * r + i], O[j][v]);
                }
            }
            float2 gt[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                gt[j] = sums[wave][16 * j + col];
                const float into = fast_exp2(gt[j].x + gt[j].y);
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int r = 0; r < 4; ++r) O[j][v][r] *= into;
            }
            // scores, decayed; a pair of a token and an earlier one is left out by selection (it may be NaN)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = i; j < 2; ++j) {
                    const V4f x = scores<IO, NK>(kr[i], rr[j]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float d = decay_between(gt[j], gs[4 * i + r]) * (x[r] * a.key_scale);
                        P[i][j][r] = i < j || 4 * grp + r <= col ? d : 0.0f;
                    }
                }
#pragma unroll
            for (int r = 0; r < 4; ++r) P[1][0][r] = 0.0f;
        }
        // keys decayed to the chunk's end, as operands over the tokens
        float out[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) out[k] = decay_between(end, gs[k]) * a.key_scale;
        [[maybe_unused]] U4 vop[NV];
        [[maybe_unused]] Split8 kop[NK];
        [[maybe_unused]] ColPart<IO, NK> kd;
        [[maybe_unused]] ColPart<IO, NV> vd;
        bool finite = true;
        if constexpr (kBf16) {
#pragma unroll
            for (int j = 0; j < NV; ++j) vop[j] = col_operand<NV>(vcol, j);
#pragma unroll
            for (int i = 0; i < NK; ++i)
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    split_pair(kop[i], m, kc.get(2 * m, i) * out[2 * m], kc.get(2 * m + 1, i) * out[2 * m + 1]);
            if constexpr (kKind == kForward) {
                S2 most = {0, 0};
#pragma unroll
                for (int k = 0; k < 8; ++k)
#pragma unroll
                    for (int j = 0; j < NV / 2; ++j)
                        most = __builtin_elementwise_max(most, __builtin_bit_cast(S2, vcol.w[k][j] & 0x7fff7fffu));
                finite = most[0] < 0x7f80 && most[1] < 0x7f80;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
#pragma unroll
                for (int i = 0; i < NK; ++i) kd.w[k][i] = kc.w[k][i] * out[k];
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    vd.w[k][j] = vcol.w[k][j];
                    if constexpr (kKind == kForward) finite = finite && __builtin_fabsf(vcol.w[k][j]) < __builtin_inff();
                }
            }
        }
        // the next chunk's numbers are on their way during the products that follow
        if (at + kChunk < n) load(at + kChunk);

        if constexpr (kKind != kLocal) {
            // o += P v
            auto add = [&](const float (&p)[2][2][4], int j) {
                if constexpr (kBf16) {
                    Split8 x;
#pragma unroll
                    for (int m = 0; m < 4; ++m) split_pair(x, m, p[m / 2][j][2 * (m & 1)], p[m / 2][j][2 * (m & 1) + 1]);
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        O[j][v] = mfma(vop[v], x.hi, O[j][v]);
                        O[j][v] = mfma(vop[v], x.lo, O[j][v]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i <= j; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int v = 0; v < NV; ++v) O[j][v] = mfma(vd.w[4 * i + r][v], p[i][j][r], O[j][v]);
                }
            };
            if constexpr (kKind == kForward) {
                if (__all(finite)) {
                    add(P, 0);
                    add(P, 1);
                } else {
                    // a NaN or infinity among the values must not reach the tokens before it, as 0 times it would:
                    // the product without them, then they alone, token by token
                    if constexpr (kBf16) {
                        U4 keep[NV];
#pragma unroll
                        for (int v = 0; v < NV; ++v) {
                            keep[v] = vop[v];
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                const uint32_t w = vop[v][m];
                                vop[v][m] = ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0xffffu) |
                                            ((w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0xffff0000u);
                            }
                        }
                        add(P, 0);
                        add(P, 1);
#pragma unroll
                        for (int v = 0; v < NV; ++v) vop[v] = keep[v];
                    } else {
                        ColPart<IO, NV> keep = vd;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
#pragma unroll
                            for (int v = 0; v < NV; ++v)
                                if (!(__builtin_fabsf(vd.w[k][v]) < __builtin_inff())) vd.w[k][v] = 0.0f;
                        add(P, 0);
                        add(P, 1);
                        vd = keep;
                    }
                    HeadRows<IO, kVec> X = V;
                    X.chunk(mem, cnt);
                    for (int s = 0; s < cnt; ++s) {
                        RowPart<IO, NV> x;
                        const uint32_t row = static_cast<uint32_t>(desc ? cnt - 1 - s : s) * X.ld;
#pragma unroll
                        for (int k = 0; k < 4 * NV; k += NV)
                            load_channels<IO, NV, kVec>(X.rsrc, row, vr + k, X.D, &x.w[k * e / 4]);
                        const int from = ((s & 15) >> 2) * 16 + col;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float p = 0.0f;
#pragma unroll
                            for (int i = 0; i < 2; ++i)
#pragma unroll
                                for (int r = 0; r < 4; ++r) {
                                    const float there = __shfl(P[i][j][r], from);
                                    if (i == (s >> 4) && r == (s & 3)) p = there;
                                }
#pragma unroll
                            for (int v = 0; v < NV; ++v)
#pragma unroll
                                for (int r = 0; r < 4; ++r) {
                                    const float xv = x.get(NV * r + v);
                                    if (s <= 16 * j + col && !(__builtin_fabsf(xv) < __builtin_inff()))
                                        O[j][v][r] = fmaf(p, xv, O[j][v][r]);
                                }
                        }
                    }
                }
            } else {
                if (dots) {
                    // without the pairs of a token with itself; then those
                    float own[2][2][4];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const bool same = i == j && 4 * grp + r == col;
                                own[i][j][r] = same ? P[i][j][r] : 0.0f;
                                P[i][j][r] = same ? 0.0f : P[i][j][r];
                            }
                    W.chunk(mem, cnt);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int i = 16 * j + col, row = desc ? cnt - 1 - i : i;
                        RowPart<IO, NV> w;
#pragma unroll
                        for (int k = 0; k < 4 * NV; k += NV)
                            load_channels<IO, NV, kVec>(W.rsrc, static_cast<uint32_t>(row) * W.ld, vr + k, W.D, &w.w[k * e / 4]);
                        add(P, j);
                        float dot = 0.0f;
#pragma unroll
                        for (int v = 0; v < NV; ++v)
#pragma unroll
                            for (int r = 0; r < 4; ++r) dot = fmaf(O[j][v][r], w.get(NV * r + v), dot);
                        dot = over_groups(dot) * a.out_scale;
                        if (grp == 0 && i < cnt)
                            a.dots[(static_cast<int64_t>(block) * a.tokens + mem + row) * a.H + h] = dot;
                        add(own, j);
                    }
                } else {
                    add(P, 0);
                    add(P, 1);
                }
            }
            // o is written: row t is 4 NV consecutive channels of the lane
            const int oe = a.o_f32 ? 4 : e;
            const int64_t stride = static_cast<int64_t>(a.H) * a.V * oe;
            const int64_t dst = uniform(reinterpret_cast<int64_t>(a.o) + mem * stride + h * a.V * oe);
            const __amdgpu_buffer_rsrc_t orsrc = __builtin_amdgcn_make_buffer_rsrc(
                reinterpret_cast<void*>(dst), 0, static_cast<uint32_t>((cnt - 1) * stride + a.V * oe), kRsrcFlags);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int i = 16 * j + col;
                const uint32_t row = static_cast<uint32_t>(desc ? cnt - 1 - i : i) * static_cast<uint32_t>(stride);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int c = vr + NV * r;
                    float x[NV];
#pragma unroll
                    for (int v = 0; v < NV; ++v) x[v] = O[j][v][r] * a.out_scale;
                    if (!kBf16 || a.o_f32) {
#pragma unroll
                        for (int v = 0; v < NV; ++v)
                            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[v]), orsrc,
                                                                  c + v < a.V ? row + (c + v) * 4 : kOutside, 0, 0);
                    } else if constexpr (kVec && NV == 4) {
                        const U2v w = {bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])};
                        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(U2v, w), orsrc, c < a.V ? row + c * 2 : kOutside, 0, 0);
                    } else if constexpr (kVec && NV == 2) {
                        __builtin_amdgcn_raw_buffer_store_b32(bf16_pair(x[0], x[1]), orsrc, c < a.V ? row + c * 2 : kOutside, 0, 0);
                    } else {
#pragma unroll
                        for (int v = 0; v < NV; ++v)
                            __builtin_amdgcn_raw_buffer_store_b16(bf16_bits(x[v]), orsrc, c + v < a.V ? row + (c + v) * 2 : kOutside, 0, 0);
                    }
                }
            }
        }
        // S = e^{G_end} S + keys^T values
        const float keep = fast_exp2(end.x + end.y);
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int j = 0; j < NV; ++j) {
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i][j][r] *= keep;
                if constexpr (kBf16) {
                    S[i][j] = mfma(kop[i].hi, vop[j], S[i][j]);
                    S[i][j] = mfma(kop[i].lo, vop[j], S[i][j]);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) S[i][j] = mfma(kd.w[k][i], vd.w[k][j], S[i][j]);
                }
            }
    }

    // what is left: the decay of the last token, where decays were moved; the segment's or sequence's state
    float rest_decay = 1.0f;
    if (a.back && n > 0) {
        const int64_t tok = desc ? sg.first : sg.first + n - 1;
        const double g = log2_decay(a.ld_g ? a.g[tok * a.ld_g + h] : a.g[h]);
        const float2 p = as_pair(g);
        rest_decay = fast_exp2(p.x + p.y);
    }
    if constexpr (kKind == kGradient) {
        if (a.cdot) {
            const float* ep = lin_state(a.e, a.e_by_slot, slot, sg.seq, a, h);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NK; ++i)
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int x = NK * (4 * grp + r) + i, y = vc + j;
                        if (ep && x < a.K && y < a.V) sum = fmaf(S[i][j][r], ep[x * a.e_row + y * a.e_col], sum);
                    }
            sum = over_groups(sum);
            for (int m = 1; m < 16; m *= 2) sum += __shfl_xor(sum, m);
            if (lane == 0) a.cdot[(slot * a.H + h) * a.blocks + block] = sum;
        }
    }
    if (kKind == kLocal && a.tot && block == 0 && lane == 0) {
        const float2 p = as_pair(all);
        a.tot[slot * a.H + h] = fast_exp2(p.x + p.y);
    }
    const bool write = a.s_end && (kKind == kLocal || (a.back ? sg.head : sg.last));
    if (write) {
        float* dst = a.s_end + ((kKind == kLocal ? slot : sg.seq) * a.H + h) * ks;
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int x = NK * (4 * grp + r) + i;
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (x < a.K && vc + j < a.V) dst[static_cast<int64_t>(x) * a.V + vc + j] = S[i][j][r] * rest_decay;
            }
    }
}

// Queues a pass on a grid of its waves.
template <typename IO, int kKind>
void launch_lin_pass(const LinArgs& a, bool vec, hipStream_t s);

}  // namespace vimscan_dev

#endif  // VIMSCAN_LINATTN_DEVICE_H
