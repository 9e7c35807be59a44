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
// What bounds it: by its floor memory (bf16, heads of 64 x 64: 512 bytes and 16 K operations a token and head); as built the chain of a
// chunk's steps (tile in, scores, products, tile out), which a SIMD's one to three waves cover in part: 1 x 65537 x 24 heads of
// 64 x 64 bf16 204 us for 803 MB, 3.9 TB/s, VALU busy 41%, matrix cores 18%; the gradients of q and k of 128 x 197 x 12 111 us, VALU
// 45%. A wave does all of a head (or 32 or 64 output channels of it) alone: it reads every number once, the state never leaves
// its registers, and nothing waits for another wave. The operands are laid out so that what one product leaves
// in the accumulators is the next one's operand as it stands (lane = 16 grp + col):
//   * the scores are formed transposed, rows = key tokens, columns = reader tokens: a lane holds the tokens 4 grp + 0..3
//     of a column, which is how the next product (values times scores) takes its right operand;
//   * o is formed transposed too, rows = channels: a lane ends with 4 NV consecutive channels of one token;
//   * the state has rows = key channels, columns = value channels. Column m of its tile j is channel NV m + j, row 4 grp + r
//     of its tile i is channel 4 NK grp + 8 (i / 2) + 2 r + i % 2: a lane's rows are the 4 NK consecutive channels that it
//     reads of a key or reader, in an order in which pairs of tiles are in place as the left operand of r S, and
//     as columns they are read in pairs.
// bf16: the numbers of the inputs are exact operands. Those in fp32 (state, scores, decayed values) are two or three bf16
// parts, each multiplied: three of what makes states and the terms of the decays' gradient, two of what is read for an output (y and the
// gradients of q, k and v, those by head that the sums of shared heads take in fp32 among them). fp32: fp32 matrix instructions.
// Sums of g are in fp64, and their differences taken from a pair of fp32, so that a token of strong decay does not cost its
// neighbours digits.
#ifndef VIMSCAN_LINATTN_DEVICE_H
#define VIMSCAN_LINATTN_DEVICE_H

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "block_device.h"
#include "linattn_plan.h"

namespace vimscan_dev {

constexpr int kChunk = vimscan_host::kLinChunk;
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
    kGradient,     // a gradient
    kGradientDots  // a gradient, with its part of the decays'
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
    int32_t once;              // inputs that are not kept in the caches
    int32_t back;              // walk from the segment's end (on top of rev), decays moved by one
    float key_scale, out_scale;
    // state before a sequence (in the pass' walk; NULL: 0) and before its other segments, by slot. Element (i, j) is at i row + j col
    const float* s0;
    const float* s0_seg;
    int64_t s0_row, s0_col;
    float* s_end;              // kLocal: of the segment; else of the sequence, written by its last segment; dense K x V
    float* tot;                // kLocal: the segment's decay
    // (kLocal leaves out the segment that its walk ends with: nothing comes after it)
    void* o;                   // [tokens][H][V], dense
    int32_t o_f32;             // in fp32 whatever the io type
    // kGradientDots: dots[block][token][head] = w . o without a token's pair with itself
    LinRows w;
    float* dots;
    const float* e;            // gradient of the state behind a sequence, e_seg its other segments (as s0); cdot[slot][head][block] = <S, e>
    const float* e_seg;
    int64_t e_row, e_col;
    float* cdot;
    // kGradientDots: the state at the borders of windows (of dq: S_{t-1}, of dk: exp(g_t) D_t, t the first token behind the border in
    // the walk of S), [border][H][block], as the wave has it in its registers
    float* marks;
    int32_t seg_borders;       // of a segment of a uniform sequence
};

// Passes of one launch: equally many waves each, of the same instance.
struct LinPasses {
    int32_t count;
    LinArgs a[3];
};

// A segment of a sequence, in tokens: walking positions w0 .. w0 + n of the sequence, at rows first .. first + n.
struct LinSegment {
    int64_t seq, first;
    int64_t n;
    int64_t border;            // its first border of windows: those of a segment are consecutive, no two segments share one
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
    s.border = uniform(a.offsets ? (lo + w0) / vimscan_host::kLinWindow : slot * a.seg_borders);
    s.seq = uniform(s.seq);
    return s;
}

// Whether a lane's part of a state, NK x NV tiles of which K rows and V columns are the head's, holds any of those.
__device__ __forceinline__ bool lin_lane_holds(int lane, int NK, int NV, int K, int V) {
    return 4 * NK * (lane >> 4) < K && NV * (lane & 15) < V;
}

// The state before (or the gradient behind) a segment: the sequence's at its edge, else the segment's own.
__device__ __forceinline__ const float* lin_state(const float* of_seq, const float* of_slot, bool edge, int64_t slot, int64_t seq,
                                                  const LinArgs& a, int64_t h) {
    const float* p = edge ? of_seq : of_slot;
    return p ? p + ((edge ? seq : slot) * a.H + h) * (static_cast<int64_t>(a.K) * a.V) : nullptr;
}

// ---------------------------------------------------------------------------------------------
// Rows. A chunk's rows of an array go from memory to registers in pieces of 16 bytes, consecutive lanes taking consecutive
// pieces (a lane's own operands are 16 to 64 bytes of a row of its own: loaded as such, the address unit takes 64 rows
// an instruction and bounds the pass), and from there to a tile in LDS, from which the operands are read.

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
// N channels of the tokens 4 grp + 0..3 and 16 + 4 grp + 0..3 of a chunk.
template <typename IO, int N> struct ColPart;
template <int N> struct ColPart<Bf16, N> { uint32_t w[8][N / 2]; };
template <int N> struct ColPart<float, N> { float w[8][N]; };

// A tile of kChunk rows of 16 N channels. Rows are 16 bytes longer than their channels, which spreads the lanes' rows over the banks.
template <typename IO, int N>
struct Tile {
    static constexpr int e = sizeof(IoElem<IO>), kRow = 16 * N * e + 16, kBytes = kChunk * kRow;
    static constexpr int kPieces = N * e, kLoads = kChunk * kPieces / 64;   // pieces of a row, loads of a lane
    static constexpr int kChannels = 16 / e;                                // of a piece
    // the lane's piece of its first row and of each that follows (its rows are 64 / kPieces apart)
    __device__ __forceinline__ static int piece(int lane) { return lane % kPieces; }
    __device__ __forceinline__ static int row(int lane, int k) { return lane / kPieces + k * (64 / kPieces); }

    __device__ __forceinline__ static void put(char* tile, int lane, const U4 (&x)[kLoads]) {
        char* p = tile + row(lane, 0) * kRow + piece(lane) * 16;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) *reinterpret_cast<U4*>(p + k * (64 / kPieces) * kRow) = x[k];
    }
    __device__ __forceinline__ static void part(const char* tile, int row, int grp, RowPart<IO, N>& o) {
        const U4* p = reinterpret_cast<const U4*>(tile + row * kRow + 4 * N * e * grp);
#pragma unroll
        for (int k = 0; k < N * e / 4; ++k) {
            const U4 w = p[k];
            __builtin_memcpy(&o.w[16 / e * k / (e == 2 ? 2 : 1)], &w, 16);
        }
    }
    // of the values: channels N col on. row0: the row of the lane's first token, step: from one to the next
    __device__ __forceinline__ static void columns(const char* tile, int row0, int step, int col, ColPart<IO, N>& o) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const char* p = tile + (row0 + ((k & 4) * 4 + (k & 3)) * step) * kRow + N * e * col;
            if constexpr (N * e == 4) __builtin_memcpy(o.w[k], __builtin_assume_aligned(p, 4), 4);
            else if constexpr (N * e == 8) __builtin_memcpy(o.w[k], __builtin_assume_aligned(p, 8), 8);
            else __builtin_memcpy(o.w[k], __builtin_assume_aligned(p, 16), N * e);
        }
    }
    // of the keys: channel i is that of row col of the state's tile i
    __device__ __forceinline__ static void state_columns(const char* tile, int row0, int step, int col, ColPart<IO, N>& o) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const char* p = tile + (row0 + ((k & 4) * 4 + (k & 3)) * step) * kRow + (4 * N * (col / 4) + 2 * (col % 4)) * e;
#pragma unroll
            for (int i = 0; i < N; i += 2) __builtin_memcpy(&o.w[k][i * e / 4], __builtin_assume_aligned(p + 4 * i * e, 2 * e), 2 * e);
        }
    }
};

// A value that the compiler takes as new: what depends on it is formed anew in every chunk, in an instruction or two, and does not
// take a register over the loop.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

// The offset in a row of a piece that starts at channel c, for rows of D channels: whole or outside.
template <typename T>
__device__ __forceinline__ uint32_t piece_at(int c, int D) { return c < D ? static_cast<uint32_t>(c * sizeof(IoElem<T>)) : kOutside; }
// Cache policy of the passes' loads. kOnce: the lines are not kept. Calls whose inputs do not fit the memory-side cache take it:
// lines that are kept throw out others, written ones among them, for nothing (64 x 1025 x 24 heads of 64 x 64 bf16 202 us, kept 218; 1 x 65537 x 24
// 300, 325); those that fit are read again by the passes that follow (128 x 197 x 12 of 64 x 64, backward 160 us kept, 187 not). Where other waves
// ask for the same lines they are kept at any size (32 x 1025 x 16 of 128 x 128, four blocks a head, 211 us kept, 276 not; 64 x 1025 x 24 of
// 32 x 32, two heads a line, 216, 230; 64 x 1025 x 12 of 64 x 64 fp32 269, 285; 64 x 1025 x 24 in 4 groups, backward 1128, 1160).
// Gradients in bf16 are written so always, y never (64 packed x up to 1025 x 24 in one group of 128 x 64: 217 us so, 227 kept;
// 1 x 65537 x 24 of 64 x 64: 306, 301; 32 x 1025 x 16 of 128 x 128: 288, 279; 128 x 197 x 12 alike).
constexpr int kKeep = 0, kOnce = 2;
template <int kPolicy>
__device__ __forceinline__ U4 load_b128(__amdgpu_buffer_rsrc_t rsrc, uint32_t at) {
    return __builtin_bit_cast(U4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, 0, kPolicy));
}
// A lane's piece of a row: kChannels channels from c on, those past D as 0. kVec: all or none are, and the offset is the piece's
// own; else it is the row's.
template <typename IO, bool kVec, int kPolicy = kKeep>
__device__ __forceinline__ U4 load_piece(__amdgpu_buffer_rsrc_t rsrc, uint32_t row, int c, int D) {
    constexpr int e = sizeof(IoElem<IO>), n = 16 / e;
    if constexpr (kVec) {
        return load_b128<kPolicy>(rsrc, row);
    } else {
        U4 o = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < n; ++k) {
            const uint32_t at = c + k < D ? row + static_cast<uint32_t>((c + k) * e) : kOutside;
            if constexpr (e == 4) o[k] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, at, 0, 0);
            else o[k / 2] |= static_cast<uint32_t>(static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(rsrc, at, 0, 0))) << 16 * (k & 1);
        }
        return o;
    }
}

// One array's rows of a head: where they are, and a chunk of them as a buffer resource. A lane's offsets in a chunk are
// the same for every chunk; the resource moves.
template <typename IO>
struct HeadRows {
    uint64_t base;
    uint32_t ld;        // bytes from token to token
    int D;
    __device__ __forceinline__ void init(const LinRows& x, int64_t h, int d) {
        constexpr int e = sizeof(IoElem<IO>);
        base = reinterpret_cast<uint64_t>(x.p) + static_cast<uint64_t>(h / x.div * x.hs * e);
        ld = static_cast<uint32_t>(x.ld * e);
        D = x.p ? d : 0;    // (an array that is absent reads as 0)
    }
    // the rows of tokens first .. first + n, n <= kChunk (none: everything reads as 0)
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk(int64_t first, int n) const {
        constexpr int e = sizeof(IoElem<IO>);
        const int64_t at = uniform(static_cast<int64_t>(base + static_cast<uint64_t>(first) * ld));
        return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(at), 0, D > 0 && n > 0 ? (n - 1) * ld + D * e : 0,
                                                 kRsrcFlags);
    }
    // where a lane's first row of a chunk is; kVec: its piece of it, from channel c0 on
    template <int N, bool kVec>
    __device__ __forceinline__ uint32_t at(int c0, int lane) const {
        using T = Tile<IO, N>;
        return T::row(lane, 0) * ld + (kVec ? piece_at<IO>(c0 + T::piece(lane) * T::kChannels, D) : 0u);
    }
    // a lane's pieces of a chunk
    template <int N, bool kVec, int kPolicy>
    __device__ __forceinline__ void load(int64_t first, int n, uint32_t at, int c0, int lane, U4 (&o)[Tile<IO, N>::kLoads]) const {
        using T = Tile<IO, N>;
        const auto rsrc = chunk(first, n);
        const uint32_t row = opaque(at);
#pragma unroll
        for (int k = 0; k < T::kLoads; ++k)
            o[k] = load_piece<IO, kVec, kPolicy>(rsrc, row + static_cast<uint32_t>(k * (64 / T::kPieces)) * ld, c0 + T::piece(lane) * T::kChannels, D);
    }
};

// ---------------------------------------------------------------------------------------------
// Products. In bf16 a number in fp32 is the sum of one to three bf16 parts, each the rounding of what the ones before it
// leave: at most 2^-8, 2^-17 or 2^-26 of it are lost.

// Four pairs of numbers as an operand: the next part of each, which is taken from them.
__device__ __forceinline__ U4 next_part(float (&x)[8]) {
    U4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = bf16_pair(x[2 * i], x[2 * i + 1]);
        x[2 * i] -= bf16_lo(w[i]);
        x[2 * i + 1] -= bf16_hi(w[i]);
    }
    return w;
}
__device__ __forceinline__ V4f mfma(U4 a, U4 b, V4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V8bf, a), __builtin_bit_cast(V8bf, b), c, 0, 0, 0);
}
__device__ __forceinline__ V4f mfma(float a, float b, V4f c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// The operand of step s (32 channels) of a token's part.
template <int N>
__device__ __forceinline__ U4 row_operand(const RowPart<Bf16, N>& p, int s) {
    return U4{p.w[4 * s], p.w[4 * s + 1], p.w[4 * s + 2], p.w[4 * s + 3]};
}
// The channel, among a lane's 4 NK, of row r of its four and tile i of the state.
__device__ __forceinline__ constexpr int state_channel(int i, int r) { return 8 * (i / 2) + 2 * r + i % 2; }
// Channel k of the eight tokens, as an operand over the tokens.
template <int N>
__device__ __forceinline__ U4 col_operand(const ColPart<Bf16, N>& p, int k) {
    const uint32_t sel = (k & 1) ? 0x07060302u : 0x05040100u;
    U4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __builtin_amdgcn_perm(p.w[2 * i + 1][k / 2], p.w[2 * i][k / 2], sel);
    return o;
}

// The scores of 16 keys (rows) and 16 readers (columns).
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
// A wave's state and arrays [K][V] of fp32, element (x, y) at x row + y col: four consecutive numbers at a time where they are
// (one at a time a wave's start and end cost microseconds), else one.
template <int NK, int NV, typename F4, typename F1>
__device__ __forceinline__ void state_elements(const void* p, int K, int V, int64_t row, int64_t col, int grp, int vc, F4&& four, F1&& one) {
    const bool at16 = reinterpret_cast<uintptr_t>(p) % 16 == 0;
    if (NV == 4 && col == 1 && at16 && V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int x = 4 * NK * grp + state_channel(i, r);
                if (x < K && vc < V) four(x * row + vc, [&](int k, auto&& f) { f(i, k, r); });
            }
    } else if (row == 1 && at16 && K % 8 == 0) {
#pragma unroll
        for (int i = 0; i < NK; i += 2)
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int r = 0; r < 4; r += 2) {   // channels 8 (i / 2) + 2 r + 0..3: tiles i, i + 1 of rows r, r + 1
                    const int x = 4 * NK * grp + state_channel(i, r);
                    if (x < K && vc + j < V) four(x + (vc + j) * col, [&](int k, auto&& f) { f(i + k % 2, j, r + k / 2); });
                }
    } else {
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int x = 4 * NK * grp + state_channel(i, r), y = vc + j;
                    if (x < K && y < V) one(x * row + y * col, i, j, r);
                }
    }
}

// The pass: one wave (a workgroup) per segment, head and block of 16 NV output channels. NK tiles of 16 hold the K
// contracted channels. A chunk's rows are loaded while the chunk before is worked on.

// Waves a SIMD that the registers are cut for.
template <typename IO, int NK, int NV> constexpr int kLinWavesPerSimd = vimscan_host::lin_waves_per_simd(sizeof(IoElem<IO>), NK, NV);

template <typename IO, int NK, int NV, int kKind>
struct LinTiles {
    // The output's tile (fp32) is in place of the readers', and of what lies behind them.
    static constexpr int kO = kKind == kLocal ? 0 : Tile<float, NV>::kBytes, kR = kKind == kLocal ? 0 : Tile<IO, NK>::kBytes;
    static constexpr int kFirst = kO > kR ? kO : kR, kK = kFirst, kV = kK + Tile<IO, NK>::kBytes, kBytes = kV + Tile<IO, NV>::kBytes;
};

template <typename IO, int NK, int NV, bool kVec, int kKind>
__global__ __launch_bounds__(64, (kLinWavesPerSimd<IO, NK, NV>)) void k_lin_pass(LinPasses passes) {
    constexpr bool kBf16 = sizeof(IoElem<IO>) == 2;
    constexpr int e = sizeof(IoElem<IO>);
    // bf16: how many parts. The scores and the state, where they are read, take two (2^-17 of a term) where an output that is rounded to
    // bf16 comes of them: with one their rounding is as large as the output's own (its error 1.4 times the least) for 3% (8 x 1025 x 12
    // heads of 64 x 64 47 us, 46 with one) to 12% (128 x 197 x 12 47 us, 41; 64 packed x up to 1025 x 24 of 128 x 64 228, 205). The
    // terms of the decays' gradient, in fp32, nearly cancel: three. The decayed values make the state, which is fp32 in memory: three.
    constexpr int kReadParts = kKind == kGradientDots ? 3 : 2, kValueParts = 3;
    using L = LinTiles<IO, NK, NV, kKind>;
    using TK = Tile<IO, NK>;
    using TV = Tile<IO, NV>;
    using TO = Tile<float, NV>;
    __shared__ __align__(16) char lds[L::kBytes];
    __shared__ float2 sums[kChunk];
    __shared__ float same[kKind == kGradientDots ? kChunk : 1];   // the scores of tokens with themselves
    char* const tr = lds;
    char* const tk = lds + L::kK;
    char* const tv = lds + L::kV;
    const int lane = static_cast<int>(threadIdx.x), grp = lane >> 4, col = lane & 15;
    // (the passes of a head side by side: they read the same rows)
    int64_t task = xcd_order(blockIdx.x, gridDim.x);
    const int which = static_cast<int>(task % passes.count);
    const LinArgs& a = passes.a[which];
    task /= passes.count;
    const int block = static_cast<int>(task % a.blocks);
    const int64_t rest = task / a.blocks, h = rest % a.H, slot = rest / a.H;
    const LinSegment sg = lin_segment(a, slot);
    if (!sg.valid || (kKind == kLocal && (a.back ? sg.head : sg.last))) return;
    const bool desc = (a.rev != 0) != (a.back != 0);
    const int c0 = block * 16 * NV, vc = c0 + NV * col;   // the block's and the lane's value channels

    // state, over e^scaled: S[i][j][r] = key channel 4 NK grp + state_channel(i, r), value channel vc + j
    V4f S[NK][NV];
    const int64_t ks = static_cast<int64_t>(a.K) * a.V;
    {
        const float* s0 = kKind == kLocal ? nullptr : lin_state(a.s0, a.s0_seg, a.back ? sg.last : sg.head, slot, sg.seq, a, h);
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int j = 0; j < NV; ++j) S[i][j] = V4f{0.0f, 0.0f, 0.0f, 0.0f};
        if (s0)
            state_elements<NK, NV>(s0, a.K, a.V, a.s0_row, a.s0_col, grp, vc,
                [&](int64_t at, auto&& place) {
                    const V4f w = *reinterpret_cast<const V4f*>(s0 + at);
#pragma unroll
                    for (int k = 0; k < 4; ++k) place(k, [&](int i, int j, int r) { S[i][j][r] = w[k]; });
                },
                [&](int64_t at, int i, int j, int r) { S[i][j][r] = s0[at]; });
    }

    HeadRows<IO> R, K, V, W;
    R.init(a.r, h, a.K);
    K.init(a.k, h, a.K);
    V.init(a.v, h, a.V);
    if constexpr (kKind == kGradientDots) W.init(a.w, h, a.V);

    // Chunk m holds 32 walking positions i, at its row i or, walking down, 31 - i. The tokens that a last chunk lacks
    // are behind its rows; walking down the first chunk lacks them, before the first token. Either way they are at rows from
    // cnt on, outside the resource: no keys, no values, no decay.
    const int64_t n = sg.n;
    const int chunks = static_cast<int>((n + kChunk - 1) / kChunk), lack = static_cast<int>(static_cast<int64_t>(chunks) * kChunk - n);
    auto place = [&](int m, int64_t* first, int* c) {
        *first = desc ? sg.first + n + lack - static_cast<int64_t>(m + 1) * kChunk : sg.first + static_cast<int64_t>(m) * kChunk;
        *c = m >= chunks ? 0 : m == (desc ? 0 : chunks - 1) ? kChunk - lack : kChunk;
    };
    const int flip = desc ? kChunk - 1 : 0;               // (row of position i: i ^ flip)
    const int my_row = (lane & (kChunk - 1)) ^ flip, row0 = col ^ flip, grow0 = (4 * grp) ^ flip, step = desc ? -1 : 1;
    const uint32_t g_ld = static_cast<uint32_t>(a.ld_g) * 4;
    const uint32_t r_at = R.template at<NK, kVec>(0, lane), k_at = K.template at<NK, kVec>(0, lane);
    const uint32_t v_at = V.template at<NV, kVec>(c0, lane);
    // the output's rows: 2 NV lanes to a row, eight channels each
    constexpr int kLanes = 2 * NV, kRows = 64 / kLanes;
    const int orow = lane / kLanes, oc = c0 + lane % kLanes * 8, oe = a.o_f32 ? 4 : e;
    const uint32_t o_ld = static_cast<uint32_t>(a.H) * a.V * oe;
    const uint32_t o_at = orow * o_ld + (kVec ? (oc < a.V ? static_cast<uint32_t>(oc * oe) : kOutside) : 0u);
    [[maybe_unused]] const uint32_t w_at = orow * W.ld + (kVec ? piece_at<IO>(oc, W.D) : 0u);

    U4 sr[kKind == kLocal ? 1 : TK::kLoads], sk[TK::kLoads], sv[TV::kLoads];
    float gv = 0.0f;
    // (past the last chunk: zeros, and no branch, behind which what is loaded would be waited for)
    auto load = [&](int m) {
        int64_t first;
        int c;
        place(m, &first, &c);
        auto rows = [&](auto policy) {
            constexpr int kPolicy = decltype(policy)::value;
            if constexpr (kKind != kLocal) R.template load<NK, kVec, kPolicy>(first, c, r_at, 0, lane, sr);
            K.template load<NK, kVec, kPolicy>(first, c, k_at, 0, lane, sk);
            V.template load<NV, kVec, kPolicy>(first, c, v_at, c0, lane, sv);
        };
        if (kVec && a.once) rows(std::integral_constant<int, kOnce>{});
        else rows(std::integral_constant<int, kKeep>{});
        // the decay of the lane's position (of its half of the wave); moved by one token where the walk goes back, the segment's
        // own tokens only
        const int move = a.back ? (desc ? 1 : -1) : 0, rel = static_cast<int>(first - sg.first) + my_row + move;
        const bool in = my_row < c && rel >= 0 && rel < static_cast<int>(n);
        const int64_t at = uniform(reinterpret_cast<int64_t>(a.g) + ((first + move) * a.ld_g + h) * 4);
        const auto gb = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(at), 0, (kChunk - 1) * g_ld + 4, kRsrcFlags);
        gv = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(gb, in ? my_row * g_ld : kOutside, 0, 0));
    };

    double all = 0.0;      // sum of the log decays so far (in units of log 2, as all here)
    double scaled = 0.0;   // that since the state was scaled
    if (chunks > 0) load(0);
    for (int m = 0; m < chunks; ++m) {
        int64_t mem;     // the chunk's lowest token, and how many it has
        int cnt;
        place(m, &mem, &cnt);
        // sums of the log decays over the chunk: before its rows are waited for or, with 128 contracted channels, during the
        // products with the state (32 x 1025 x 16 heads of 128 x 128: 278 us, 289 before; but 128 x 197 x 12 of 64 x 64 50, 46 before, 1 x 65537 x 24
        // 367, 301)
        constexpr bool kSumLate = NK == 8 && kKind != kLocal;
        const float g = gv;
        double total = 0.0;
        auto sum_up = [&] {
            const double run = half_wave_sums(log2_decay(g));
            total = lane_value(run, 31);
            if (kKind == kLocal) all += total;
            if (lane < kChunk) sums[lane] = as_pair(run + scaled);
        };
        wave_sync();
        if constexpr (!kSumLate) sum_up();
        if constexpr (kKind != kLocal) TK::put(tr, lane, sr);
        TK::put(tk, lane, sk);
        TV::put(tv, lane, sv);
        wave_sync();
        load(m + 1);
        __builtin_amdgcn_sched_barrier(0);   // (else the compiler moves loads down behind the products)
        if constexpr (kSumLate) sum_up();

        V4f O[2][NV];
        [[maybe_unused]] float P[2][2][4];   // [key tile][reader tile], rows of keys
        if constexpr (kKind != kLocal) {
            RowPart<IO, NK> rr[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) TK::part(tr, row0 + 16 * j * step, grp, rr[j]);
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
                        float x[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = S[2 * s + i % 2][v][i / 2];
                        auto part = [&] {
                            const U4 w = next_part(x);
#pragma unroll
                            for (int j = 0; j < 2; ++j) O[j][v] = mfma(w, row_operand<NK>(rr[j], s), O[j][v]);
                        };
#pragma unroll
                        for (int p = 0; p < kReadParts; ++p) part();
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int i = 0; i < NK; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j) O[j][v] = mfma(S[i][v][r], rr[j].w[state_channel(i, r)], O[j][v]);
                }
            }
            if constexpr (kSumLate) wave_sync();
            float2 gt[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                gt[j] = sums[16 * j + col];
                const float into = fast_exp2(gt[j].x + gt[j].y) * a.out_scale;
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int r = 0; r < 4; ++r) O[j][v][r] *= into;
            }
            // scores, decayed; a pair of a token and an earlier one is left out by selection (it may be NaN)
            const float scale = a.key_scale * a.out_scale;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                RowPart<IO, NK> kr;
                TK::part(tk, row0 + 16 * i * step, grp, kr);
                float2 gs[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) gs[r] = sums[16 * i + 4 * grp + r];
#pragma unroll
                for (int j = i; j < 2; ++j) {
                    const V4f x = scores<IO, NK>(kr, rr[j]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float d = decay_between(gt[j], gs[r]) * (x[r] * scale);
                        P[i][j][r] = i < j || 4 * grp + r <= col ? d : 0.0f;
                        if constexpr (kKind == kGradientDots) {
                            // (a token's own score apart: it is added where the output is written)
                            if (i == j && 4 * grp + r == col) same[16 * i + col] = d;
                            P[i][j][r] = i < j || 4 * grp + r < col ? d : 0.0f;
                        }
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) P[1][0][r] = 0.0f;
        }
        // The numbers of the chunk's columns, in bf16 as operands over the tokens.
        U4 vop[NV], kop[NK];
        ColPart<IO, NV> vcol;
        TV::columns(tv, grow0, step, col, vcol);
        if constexpr (kBf16)
#pragma unroll
            for (int j = 0; j < NV; ++j) vop[j] = col_operand<NV>(vcol, j);

        if constexpr (kKind != kLocal) {
            // o += P v
            auto add = [&](int j, const U4 (&vo)[NV], const ColPart<IO, NV>& vw) {
                if constexpr (kBf16) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = P[i / 4][j][i % 4];
                    auto part = [&] {
                        const U4 w = next_part(x);
#pragma unroll
                        for (int v = 0; v < NV; ++v) O[j][v] = mfma(vo[v], w, O[j][v]);
                    };
#pragma unroll
                    for (int p = 0; p < kReadParts; ++p) part();
                } else {
#pragma unroll
                    for (int i = 0; i <= j; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int v = 0; v < NV; ++v) O[j][v] = mfma(vw.w[4 * i + r][v], P[i][j][r], O[j][v]);
                }
            };
            bool finite = true;
            if constexpr (kKind == kForward && kBf16) {
                S2 most = {0, 0};
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) most = __builtin_elementwise_max(most, __builtin_bit_cast(S2, vop[j][k] & 0x7fff7fffu));
                finite = most[0] < 0x7f80 && most[1] < 0x7f80;
            } else if constexpr (kKind == kForward) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
#pragma unroll
                    for (int j = 0; j < NV; ++j) finite = finite && __builtin_fabsf(vcol.w[k][j]) < __builtin_inff();
            }
            if (kKind != kForward || __builtin_expect(__all(finite), 1)) {
                add(0, vop, vcol);
                add(1, vop, vcol);
            } else {
                // a NaN or infinity among the values must not reach the tokens before it, as 0 times it would:
                // the product without them, then they alone, token by token
                U4 vo[NV];
                ColPart<IO, NV> vw;
                if constexpr (kBf16) {
#pragma unroll
                    for (int v = 0; v < NV; ++v)
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const uint32_t w = opaque(vop[v][m]);   // (else formed before the branch, for every chunk)
                            vo[v][m] = ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0xffffu) |
                                       ((w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0xffff0000u);
                        }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
#pragma unroll
                        for (int v = 0; v < NV; ++v) {
                            const float w = __uint_as_float(opaque(__float_as_uint(vcol.w[k][v])));
                            vw.w[k][v] = __builtin_fabsf(w) < __builtin_inff() ? w : 0.0f;
                        }
                }
                add(0, vo, vw);
                add(1, vo, vw);
                for (int s = 0; s < kChunk; ++s) {
                    RowPart<IO, NV> x;
                    TV::part(tv, s ^ flip, grp, x);
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
            // The output goes through a tile of its own, so that consecutive lanes write consecutive pieces of rows.
            wave_sync();
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float* p = reinterpret_cast<float*>(tr + (row0 + 16 * j * step) * TO::kRow) + 4 * NV * grp;
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int v = 0; v < NV; ++v) p[NV * r + v] = O[j][v][r];
            }
            wave_sync();
            const int64_t dst = uniform(reinterpret_cast<int64_t>(a.o) + mem * static_cast<int64_t>(o_ld) + h * a.V * oe);
            const auto ob = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(dst), 0,
                                                              static_cast<uint32_t>((cnt - 1) * o_ld + a.V * oe), kRsrcFlags);
            [[maybe_unused]] const auto wb = W.chunk(mem, kKind == kGradientDots ? cnt : 0);
            const uint32_t ox = opaque(o_at);
            [[maybe_unused]] const uint32_t wx = opaque(w_at);
#pragma unroll
            for (int k = 0; k < kChunk / kRows; ++k) {
                const int row = orow + k * kRows;
                const char* src = tr + row * TO::kRow + lane % kLanes * 32;
                float x[8];
                __builtin_memcpy(x, __builtin_assume_aligned(src, 16), 16);
                __builtin_memcpy(x + 4, __builtin_assume_aligned(src + 16, 16), 16);
                if constexpr (kKind == kGradientDots) {
                    // w . o, then the token's own pair
                    constexpr int kW = 8 * e / 16, nw = 16 / e;
                    auto value = [&](const U4 (&u)[kW], int c) {
                        if constexpr (kBf16) return (c & 1) ? bf16_hi(u[0][c / 2]) : bf16_lo(u[0][c / 2]);
                        else return __uint_as_float(u[c / 4][c % 4]);
                    };
                    U4 w[kW];
#pragma unroll
                    for (int q = 0; q < kW; ++q)
                        w[q] = load_piece<IO, kVec>(wb, !kVec ? wx + static_cast<uint32_t>(k * kRows) * W.ld : q == 0 || oc + nw < W.D ? wx + static_cast<uint32_t>(k * kRows) * W.ld + q * 16 : kOutside,
                                                    oc + q * nw, W.D);
                    float dot = 0.0f;
#pragma unroll
                    for (int c = 0; c < 8; ++c) dot = fmaf(x[c], value(w, c), dot);
#pragma unroll
                    for (int q = 1; q < kLanes; q *= 2) dot += __shfl_xor(dot, q);
                    if (lane % kLanes == 0 && row < cnt) a.dots[(static_cast<int64_t>(block) * a.tokens + mem + row) * a.H + h] = dot;
                    U4 v[kW];
#pragma unroll
                    for (int q = 0; q < kW; ++q) v[q] = *reinterpret_cast<const U4*>(tv + row * TV::kRow + lane % kLanes * 8 * e + q * 16);
                    const float p = same[row ^ flip];
#pragma unroll
                    for (int c = 0; c < 8; ++c) x[c] = fmaf(p, value(v, c), x[c]);
                }
                const uint32_t at = ox + static_cast<uint32_t>(k * kRows) * o_ld;
                if (!kBf16 || a.o_f32) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        if constexpr (kVec) {
                            // (in fp32 rows of whole pieces may end between the two)
                            U4 w;
                            __builtin_memcpy(&w, x + 4 * q, 16);
                            __builtin_amdgcn_raw_buffer_store_b128(w, ob, q == 0 || oc + 4 < a.V ? at + 16 * q : kOutside, 0, 0);
                        } else {
#pragma unroll
                            for (int c = 4 * q; c < 4 * q + 4; ++c)
                                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[c]), ob, oc + c < a.V ? at + (oc + c) * 4 : kOutside, 0, 0);
                        }
                    }
                } else if constexpr (kVec) {
                    const U4 w = {bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7])};
                    __builtin_amdgcn_raw_buffer_store_b128(w, ob, at, 0, kKind == kForward ? kKeep : kOnce);
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        __builtin_amdgcn_raw_buffer_store_b16(bf16_bits(x[c]), ob, oc + c < a.V ? at + (oc + c) * 2 : kOutside, 0, 0);
                }
            }
        }
        // S = e^{G_end} S + keys^T (values, decayed to the chunk's end). S is held over the decay since it was last scaled, so that
        // it need not be scaled in every chunk: the values are decayed to that point instead, which for more than 2^-16
        // costs no digits and stays in range.
        float2 end = make_float2(0.0f, 0.0f);
        const double after = scaled + total;
        scaled = after;
        if (!(after > -16.0 && after < 16.0)) {
            end = as_pair(after);
            scaled = 0.0;
            const float keep = fast_exp2(end.x + end.y);
#pragma unroll
            for (int i = 0; i < NK; ++i)
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) S[i][j][r] *= keep;
        }
        float out[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) out[k] = decay_between(end, sums[(k & 4) * 4 + 4 * grp + (k & 3)]) * a.key_scale;
        ColPart<IO, NK> kc;
        TK::state_columns(tk, grow0, step, col, kc);
        if constexpr (kBf16)
#pragma unroll
            for (int i = 0; i < NK; ++i) kop[i] = col_operand<NK>(kc, i);
        if constexpr (kBf16) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                float x[8];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    x[2 * q] = bf16_lo(vop[j][q]) * out[2 * q];
                    x[2 * q + 1] = bf16_hi(vop[j][q]) * out[2 * q + 1];
                }
                auto part = [&] {
                    const U4 w = next_part(x);
#pragma unroll
                    for (int i = 0; i < NK; ++i) S[i][j] = mfma(kop[i], w, S[i][j]);
                };
#pragma unroll
                for (int p = 0; p < kValueParts; ++p) part();
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const float x = vcol.w[k][j] * out[k];
#pragma unroll
                    for (int i = 0; i < NK; ++i) S[i][j] = mfma(kc.w[k][i], x, S[i][j]);
                }
        }
        if constexpr (kKind == kGradientDots) {
            // The border of two windows, between the rows of chunks e_border - 1 and e_border.
            constexpr int kPer = vimscan_host::kLinWindow / kChunk;
            const int e_border = desc ? chunks - 1 - m : m + 1;
            if (m + 1 < chunks && e_border % kPer == 0) {
                double decay = scaled;
                if (a.back) {
                    const int64_t tok = desc ? mem : mem + cnt - 1;
                    decay += log2_decay(a.ld_g ? a.g[tok * a.ld_g + h] : a.g[h]);
                }
                const float2 p = as_pair(decay);
                const float keep = fast_exp2(p.x + p.y);
                V4f* const mark = reinterpret_cast<V4f*>(a.marks) +
                                  (((sg.border + e_border / kPer - 1) * a.H + h) * a.blocks + block) * (64 * NK * NV) + lane;
                if (lin_lane_holds(lane, NK, NV, a.K, a.V - c0))
#pragma unroll
                    for (int i = 0; i < NK; ++i)
#pragma unroll
                        for (int j = 0; j < NV; ++j) {
                            V4f w;
#pragma unroll
                            for (int r = 0; r < 4; ++r) w[r] = S[i][j][r] * keep;
                            mark[(i * NV + j) * 64] = w;
                        }
            }
        }
    }

    // what is left: the state's scale; the decay of the last token, where decays were moved; the segment's or sequence's state
    {
        const float2 p = as_pair(scaled);
        const float keep = fast_exp2(p.x + p.y);
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[i][j][r] *= keep;
    }
    float rest_decay = 1.0f;
    if (a.back && n > 0) {
        const int64_t tok = desc ? sg.first : sg.first + n - 1;
        const double g = log2_decay(a.ld_g ? a.g[tok * a.ld_g + h] : a.g[h]);
        const float2 p = as_pair(g);
        rest_decay = fast_exp2(p.x + p.y);
        if (kKind == kLocal) all += g;
    }
    if constexpr (kKind == kGradientDots) {
        if (a.cdot) {
            const float* ep = lin_state(a.e, a.e_seg, sg.last, slot, sg.seq, a, h);
            float sum = 0.0f;
            if (ep)
                state_elements<NK, NV>(ep, a.K, a.V, a.e_row, a.e_col, grp, vc,
                    [&](int64_t at, auto&& place) {
                        const V4f w = *reinterpret_cast<const V4f*>(ep + at);
#pragma unroll
                        for (int k = 0; k < 4; ++k) place(k, [&](int i, int j, int r) { sum = fmaf(S[i][j][r], w[k], sum); });
                    },
                    [&](int64_t at, int i, int j, int r) { sum = fmaf(S[i][j][r], ep[at], sum); });
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
        state_elements<NK, NV>(dst, a.K, a.V, a.V, 1, grp, vc,
            [&](int64_t at, auto&& place) {
                V4f w;
#pragma unroll
                for (int k = 0; k < 4; ++k) place(k, [&](int i, int j, int r) { w[k] = S[i][j][r] * rest_decay; });
                *reinterpret_cast<V4f*>(dst + at) = w;
            },
            [&](int64_t at, int i, int j, int r) { dst[at] = S[i][j][r] * rest_decay; });
    }
}

// Queues a pass on a grid of its waves.
template <typename IO, int kKind>
void launch_lin_pass(const LinPasses& p, bool vec, hipStream_t s);

}  // namespace vimscan_dev

#endif  // VIMSCAN_LINATTN_DEVICE_H
