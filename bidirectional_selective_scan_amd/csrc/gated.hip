// Gated linear recurrence for AMD MI355X (gfx950): the forward pass over whole sequences, its
// backward pass and the single-token form (include/vimscan.h, vimscan_gated_*).
//
// Per channel: u = -c softplus(lam) sigmoid(r), a = e^u, m = sqrt(1 - a^2), h' = a h + m sigmoid(i) x.
//
// Execution design (gfx950, wave64). The tokens of a call are one stream of positions in walking
// order, whatever sequences they belong to; where a sequence starts, the state is replaced instead
// of carried over. A workgroup of 256 threads takes a tile of positions x 64 channels and reads it
// once: every thread holds the transitions and inputs of a few consecutive positions in registers,
// reduces them to the map h -> A h + H of its positions, the maps are composed across the rows of a
// wave (lane swaps), the waves (LDS) and the tiles (through the workspace, see below), and each
// thread then walks its positions from the state that enters them. So every element is read once and
// written once at any shape: one long sequence fills the chip as well as many short ones.
//  * Layout: V consecutive channels per lane (two, which are 4 bytes in bf16 and 8 in fp32, or one), 64 / V lanes over
//    the channels (rows of 128 or 256 bytes), the other lanes and waves over the positions.
//  * A map whose positions contain a sequence start does not depend on the entering state: A = 0, and
//    maps are applied and composed with the multiplication that gives 0 for a factor 0 whatever the
//    other one is, so that NaN or infinity in one sequence never reaches the next.
//  * Between tiles: a tile publishes its map before it waits for anything, then composes the maps of
//    the tiles before it in its group of kGatedGroup onto the state that the group before left, always
//    in this order (the same bits on every run); a group's last tile publishes the state it leaves.
//    Tiles wait only for tiles of lower workgroup ids, which the hardware starts first on each XCD, so
//    that waits are short. None depends on it: a workgroup that has waited for long (kWaitReads; other
//    work may hold the places that earlier tiles need, another such call on another stream among it)
//    walks the tiles before it itself, from the inputs, and then its own (fwd_alone, bwd_alone). So a
//    workgroup that has started ends by itself, whatever else runs, and as the walk takes the same
//    operations in the same order, the results are the same bits either way.
//  * Backward: the same with the positions' gradients walked the other way; the state before every
//    position is walked again from the states that the forward pass saved at every tile's first
//    position.

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

#include "block_device.h"
#include "block_plan.h"
#include "handover.h"
#include "vimscan.h"

namespace {

using namespace vimscan_dev;
using vimscan_host::GatedPlan;
using vimscan_host::kGatedBlock;
using vimscan_host::kGatedBwdTile;
using vimscan_host::kGatedFwdTile;
using vimscan_host::kGatedFwdTileSmall;
using vimscan_host::kGatedGroup;
using vimscan_host::kGatedStride;

struct GatedArgs {
    const void* x;
    const void* r;
    const void* i;
    int64_t ld_x, ld_r, ld_i;
    const float* lam;
    const float* h0;
    const int32_t* offsets;  // NULL: sequences of Lp tokens
    float c;
    int32_t N;               // tokens
    int32_t Lp;
    uint32_t lp_mul, lp_shift;  // position / Lp = position * lp_mul >> lp_shift (Lp > 0)
    int32_t D, nseq, ncb, tiles;
    int32_t rev;             // walk from the last token to the first
    void* y;
    float* h_last;
    float* states;
    // backward
    const void* dy;
    const float* dh_last;
    const float* states_in;
    void* dx;
    void* dr;
    void* di;
    int64_t ld_dy, ld_dx, ld_dr, ld_di;
    float* dlam;
    float* dh0;
    // workspace
    uint64_t* agg;           // [tile][2][width] maps handed over, width = 64 ncb
    uint64_t* inc;           // [group][2][width] the state a group leaves
    float* part;             // [tile][width] partial sums of dlam
    int32_t reads;           // reads of a value handed over before a workgroup goes on without it
};

// Walking positions: position p of the call is token p, or N - 1 - p walked from the end; sequence
// q in walking order is sequence q or nseq - 1 - q of the caller.
__device__ __forceinline__ int64_t seq_of(const GatedArgs& a, int q) { return a.rev ? a.nseq - 1 - q : q; }

// First position of sequence q in walking order (q = nseq: the end), inside 0..N whatever the
// offsets hold.
__device__ __forceinline__ int bound_of(const GatedArgs& a, int q) {
    if (!a.offsets) return q * a.Lp;
    const int o = a.rev ? a.offsets[a.nseq - q] : a.offsets[q];
    const int in = o < 0 ? 0 : o > a.N ? a.N : o;
    return a.rev ? a.N - in : in;
}

__device__ __forceinline__ int uniform_seq(const GatedArgs& a, int p) {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(p)) * a.lp_mul >> a.lp_shift);
}

// The last sequence of lo..hi that starts at or before position p (lo when none does): the one that
// holds p, empty ones being passed over.
__device__ __forceinline__ int seq_at(const GatedArgs& a, int p, int lo, int hi) {
    if (!a.offsets) return uniform_seq(a, p);
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (bound_of(a, mid) <= p) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The same over all sequences, for a position that the whole wave shares: 64 probes a round.
__device__ __forceinline__ int seq_at_wave(const GatedArgs& a, int p, int lane) {
    if (!a.offsets) return uniform_seq(a, p);
    int lo = 0, n = a.nseq;  // the answer is in lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 63) / 64;
        const int64_t probe = static_cast<int64_t>(lane + 1) * step;
        const bool before = probe < n && bound_of(a, lo + static_cast<int>(probe)) <= p;
        const int k = __popcll(__ballot(before)) * step;
        lo += k;
        n = n - k < step ? n - k : step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// The sequence boundaries among a wave's P positions (P <= 64): every wave finds its own, one position a
// lane, so that no barrier is needed.
struct WaveSeqs {
    uint64_t starts, ends;   // bit per position: the first, the last one of its sequence
    // row: the wave's place in LDS for the caller's sequence of each position, written only where there is
    // a boundary; lo: the sequence of the tile's first position. No bit is set past the stream's end; its
    // last position counts as an end whatever the offsets hold: the stores behind it hang on that.
    template <int P>
    __device__ __forceinline__ void find(const GatedArgs& a, int pw, int lo, int lane, int* row) {
        starts = ends = 0;
        const int pe = min(pw + P, a.N);
        if (pw >= a.N || (bound_of(a, lo) != pw && bound_of(a, lo + 1) > pe)) return;
        const int hi = a.offsets ? seq_at_wave(a, pe - 1, lane) : 0;
        const int p = pw + lane;
        const bool in = p < pe;
        const int q = in ? seq_at(a, p, lo, hi) : lo;
        if (lane < P) row[lane] = static_cast<int>(seq_of(a, q));
        starts = __ballot(in && bound_of(a, q) == p);
        ends = __ballot(in && (bound_of(a, q + 1) == p + 1 || p + 1 == a.N));
        asm volatile("" ::: "memory");  // the rows are read by this wave only, after they are written
    }
    // The bits of T positions from at on.
    template <int T>
    __device__ __forceinline__ static uint32_t bits(uint64_t m, int at) {
        return static_cast<uint32_t>(m >> at) & static_cast<uint32_t>((uint64_t(1) << T) - 1);
    }
};

// -c softplus(lam) log2(e), so that a = 2^(k2 sigmoid(r)). softplus in log2 units is
// max(w, 0) + log2(1 + p), w = lam log2(e), p = 2^-|w|; log2(1 + p) as log2(v) plus the first-order
// effect of rounding v = 1 + p (relative error below 2^-22 also where p is tiny).
__device__ __forceinline__ float decay_rate(float lam, float c) {
    const float w = lam * kLog2e;
    const float p = fast_exp2(-fabsf(w));
    const float v = 1.0f + p;
    const float rest = p - (v - 1.0f);
    return -c * (fmaxf(w, 0.0f) + fmaf(rest, kLog2e, fast_log2(v)));
}

// 1 - a^2 with a = 2^q, q <= 0: 1 - e^-t with t = -2 q ln 2. Small t by its series (the sixth power
// at t = 1/4 is 5e-8 of the result), written in q; larger t from a itself.
__device__ __forceinline__ float one_minus_sq(float q, float a) {
    constexpr double z = -2.0 * 0.693147180559945309417;
    constexpr float c1 = float(z), c2 = float(-z * z / 2), c3 = float(z * z * z / 6), c4 = float(-z * z * z * z / 24),
                    c5 = float(z * z * z * z * z / 120), c6 = float(-z * z * z * z * z * z / 720);
    // (two literals do not fit one instruction: one coefficient is kept in a register)
    float first = c5;
    asm("" : "+v"(first));
    float s = fmaf(q, c6, first);
    s = fmaf(q, s, c4);
    s = fmaf(q, s, c3);
    s = fmaf(q, s, c2);
    s = fmaf(q, s, c1);
    return q > float(0.25 / z) ? q * s : fmaf(-a, a, 1.0f);
}

// sigmoid(v) = 1 / (1 + e^-v)
__device__ __forceinline__ float sigmoid(float v) { return fast_rcp(1.0f + fast_exp2(-v * kLog2e)); }

// The same and 1 - sigmoid(v) = e / (1 + e), e = e^-v held below 2^126 (by the minimum that keeps a NaN: both
// are NaN then).
__device__ __forceinline__ float sigmoid2(float v, float* ns) {
    const float e = fast_exp2(__builtin_elementwise_minimum(-v * kLog2e, 126.0f));
    const float s = fast_rcp(1.0f + e);
    *ns = e * s;
    return s;
}

// Transition a and input gate m sigmoid(i) of a position.
__device__ __forceinline__ void gates(float r, float i, float k2, float* a, float* mg) {
    const float q = k2 * sigmoid(r);
    *a = fast_exp2(q);
    *mg = fast_sqrt(one_minus_sq(q, *a)) * sigmoid(i);
}

// What the backward pass takes of a position: a; m g; u a; g x a^2 u / m; 1 - sigmoid(r); 1 - sigmoid(i).
struct BackGates {
    float a, mg, ua, gm, ns, ng;
    __device__ __forceinline__ BackGates(float r, float i, float x, float k2) {
        const float q = k2 * sigmoid2(r, &ns);
        const float gx = sigmoid2(i, &ng);
        a = fast_exp2(q);
        const float m2 = one_minus_sq(q, a), u = q * kLn2;
        // 1 / m; where m^2 is below the normal numbers the hardware's rsq takes it for 0 and gives infinity:
        // m, below 1.1e-19 there, and its terms are taken as 0
        const float im = m2 >= 0x1p-126f ? fast_rsq(m2) : 0.0f;
        mg = m2 * im * gx;
        ua = u * a;
        gm = gx * x * (ua * a) * im;
    }
};

// The rows of a tile of one tensor as a buffer resource, rows in walking order. A position past the
// end of the stream, or a channel past the row's, takes an offset outside the resource: the hardware
// gives 0 for such a load and drops such a store.
constexpr uint32_t kOutside = 0x80000000u;

// The thread's T positions from tg * T on of a tile of TILE positions from p0.
template <typename IO, int TILE, int T>
struct TileRows {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t vo;             // the thread's lowest row in memory, and its channel
    uint32_t so, step;       // scalar offset of its first position, and from one to the next

    __device__ __forceinline__ void init(const GatedArgs& a, const void* base, int64_t ld, int p0, int tg, int c0) {
        const int64_t first = a.rev ? static_cast<int64_t>(a.N) - p0 - TILE : p0;  // the tile's lowest row
        const uint64_t at = reinterpret_cast<uint64_t>(base) + first * ld * static_cast<int64_t>(sizeof(IoElem<IO>));
        const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at));
        const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32));
        rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo), 0,
                                                 0x7fffffff, 0x00020000);
        const uint32_t row_bytes = static_cast<uint32_t>(ld) * sizeof(IoElem<IO>);
        const int row = (a.rev ? TILE / T - 1 - tg : tg) * T;
        vo = c0 < a.D && base ? row * row_bytes + c0 * static_cast<uint32_t>(sizeof(IoElem<IO>)) : kOutside;
        so = a.rev ? (T - 1) * row_bytes : 0;
        step = a.rev ? 0u - row_bytes : row_bytes;
    }
    __device__ __forceinline__ uint32_t at(bool in) const { return in ? vo : kOutside; }
};

// Cache policy of the rows' accesses. kOnce: the lines are not wanted again and are evicted first. Taken
// where every row starts on a line, so that no two workgroups share one: 65537 x 1536 bf16 forward 188 us
// instead of 201, 128 x 197 x 768 backward 67 instead of 73; where workgroups do share lines it makes them be
// fetched twice (32 x 1024 x 770: 81 us instead of 65).
constexpr int kPlain = 0, kOnce = 2;
template <typename IO, int V, int kPolicy>
__device__ __forceinline__ Raw<IO, V> ld_tile(__amdgpu_buffer_rsrc_t r, uint32_t vo, uint32_t so) {
    Raw<IO, V> o;
    if constexpr (sizeof(o) == 2) {
        const uint16_t w = __builtin_amdgcn_raw_buffer_load_b16(r, vo, so, kPolicy);
        __builtin_memcpy(&o, &w, 2);
    } else if constexpr (sizeof(o) == 4) {
        const uint32_t w = __builtin_amdgcn_raw_buffer_load_b32(r, vo, so, kPolicy);
        __builtin_memcpy(&o, &w, 4);
    } else {
        static_assert(sizeof(o) == 8, "one or two channels");
        const auto w = __builtin_amdgcn_raw_buffer_load_b64(r, vo, so, kPolicy);
        __builtin_memcpy(&o, &w, 8);
    }
    return o;
}
using U2 = uint32_t __attribute__((vector_size(8)));
template <typename IO, int V, int kPolicy>
__device__ __forceinline__ void st_tile(__amdgpu_buffer_rsrc_t r, uint32_t vo, uint32_t so, const float* v) {
    Raw<IO, V> o;
    o.set(v);
    if constexpr (sizeof(o) == 2) {
        uint16_t w;
        __builtin_memcpy(&w, &o, 2);
        __builtin_amdgcn_raw_buffer_store_b16(w, r, vo, so, kPolicy);
    } else if constexpr (sizeof(o) == 4) {
        uint32_t w;
        __builtin_memcpy(&w, &o, 4);
        __builtin_amdgcn_raw_buffer_store_b32(w, r, vo, so, kPolicy);
    } else {
        static_assert(sizeof(o) == 8, "one or two channels");
        U2 w;
        __builtin_memcpy(&w, &o, 8);
        __builtin_amdgcn_raw_buffer_store_b64(w, r, vo, so, kPolicy);
    }
}

// The product in which a factor 0 gives 0 whatever the other one is.
extern "C" __device__ float vimscan_mul_legacy(float, float) __asm("llvm.amdgcn.fmul.legacy");

// The map h -> A h + H of some consecutive positions; A = 0 where a sequence starts among them, and only
// there: a product of transitions that underflows is held at the least number above 0, so that NaN and
// infinity stay in the rest of their sequence (a finite state gets at most 5e-7 from it).
constexpr float kLeast = 0x1p-149f;
struct Map {
    float A, H;
    __device__ __forceinline__ float operator()(float h) const { return vimscan_mul_legacy(A, h) + H; }
};
__device__ __forceinline__ Map identity() { return {1.0f, 0.0f}; }
// f, then g.
__device__ __forceinline__ Map then(const Map& f, const Map& g) {
    return {fmaxf(vimscan_mul_legacy(f.A, g.A), fminf(fminf(f.A, g.A), kLeast)), g(f.H)};
}
__device__ __forceinline__ Map pick(bool c, const Map& f, const Map& g) { return {c ? f.A : g.A, c ? f.H : g.H}; }

// Composes the maps of a wave's position groups (64 / CL of them, CL lanes each): total of the wave,
// and before: the map of the groups before this lane's in walking order, or after it with kBack.
template <int CL, bool kBack>
__device__ __forceinline__ void scan_rows(const Map& f, int lane, Map* total, Map* before) {
    static_assert(CL == 32 || CL == 64, "one or two position groups in a wave");
    if constexpr (CL == 64) {
        *total = f;
        *before = identity();
    } else {
        Map lo, hi;
        swap32(f.A, &lo.A, &hi.A);
        swap32(f.H, &lo.H, &hi.H);
        const bool upper = lane & 32;
        *total = kBack ? then(hi, lo) : then(lo, hi);
        *before = kBack ? pick(upper, identity(), hi) : pick(upper, lo, identity());
    }
}

// Reads of a value handed over (about a microsecond each) before a workgroup goes on without it: some
// milliseconds, many times what a tile takes.
constexpr int kWaitReads = 1 << 12;
std::atomic<int> g_wait_reads{kWaitReads};
// Workgroups on this GPU that did.
__device__ unsigned long long g_alone;

// LDS of the hand-over.
struct ChainLds {
    int missing;                   // a wave went on without a value
    float2 wave[4][kGatedBlock];   // the maps of the waves
    float2 part[4][kGatedBlock];   // the maps of the tiles before this one, a quarter each
    float inc[kGatedBlock];        // the state that the group before left
};

// A value handed over: two 64-bit words (second words apart, so that a wave's are contiguous), the value and
// the value xor the dispatch's tag, each stored and loaded on its own (device-coherent, no order between
// them). A reader takes the value when the two differ by exactly this dispatch's tag, so words of earlier
// dispatches, arbitrary bytes and half a value never pass, the memory needs no clearing, and neither side
// waits for one access before the next: a value costs its reader one trip to memory after it was stored.
// w: the wave's first word (the same for all lanes).
__device__ __forceinline__ void hand_over(uint64_t* w, int64_t second, int lane, uint64_t tag, float x, float y) {
    const uint64_t v = __float_as_uint(x) | (static_cast<uint64_t>(__float_as_uint(y)) << 32);
    __hip_atomic_store(w + lane, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(w + second + lane, v ^ tag, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
struct Handed {
    uint64_t v, c;
    __device__ __forceinline__ void load(const uint64_t* w, int64_t second, int lane) {
        v = __hip_atomic_load(w + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        c = __hip_atomic_load(w + second + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __device__ __forceinline__ bool there(uint64_t tag) const { return (v ^ c) == tag; }
    // Loads until every lane's value is there; false when it was not in that many reads.
    __device__ __forceinline__ bool wait(const uint64_t* w, int64_t second, int lane, uint64_t tag, int reads) {
        for (int it = 0; it < reads; ++it) {
            load(w, second, lane);
            if (__all(there(tag))) return true;
            __builtin_amdgcn_s_sleep(1);
        }
        return false;
    }
    __device__ __forceinline__ float x() const { return __uint_as_float(static_cast<uint32_t>(v)); }
    __device__ __forceinline__ float y() const { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
};

// Hand-over along the chain: workgroup j of channel block cb publishes its tile's map (every one but
// the last, whatever the sequences: no wait depends on what the offsets hold) and gathers what comes
// in from tile first on (first == j: nothing comes in), or sets l.missing. Called by all threads between the
// barrier that completes l.wave and one that completes l.part and l.inc. kBack: the waves' maps compose from the
// last wave to the first.
template <bool kBack>
__device__ __forceinline__ Map tile_map(const ChainLds& l, int lane) {
    Map f = identity();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 w = l.wave[kBack ? 3 - k : k][lane];
        f = then(f, Map{w.x, w.y});
    }
    return f;
}
template <bool kBack>
__device__ __forceinline__ void chain_gather(const GatedArgs& a, ChainLds& l, int j, int cb, int first, uint64_t tag,
                                             int wave, int lane) {
    constexpr int kEach = kGatedGroup / 4;
    const int64_t width = static_cast<int64_t>(a.ncb) * kGatedBlock;
    const int64_t at = cb * kGatedBlock;
    if (wave == 3 && j + 1 < a.tiles) {
        const Map f = tile_map<kBack>(l, lane);
        hand_over(a.agg + 2 * j * width + at, width, lane, tag, f.A, f.H);
    }
    const int group = j / kGatedGroup, g0 = group * kGatedGroup;
    const bool from_group = first < g0;
    const int lo = (from_group ? g0 : first) + wave * kEach;   // this wave's tiles: lo .. lo + n - 1
    const int n = min(j - lo, kEach);
    const bool inc = from_group && wave == 0;
    Handed v[kEach];
    Map f = identity();
    bool all = true;
    // all loads first; then every value is waited for in turn
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        if (k < n) v[k].load(a.agg + 2 * (lo + k) * width + at, width, lane);
    if (wave == 0) {
        Handed h;
        h.v = 0;
        if (inc) all = h.wait(a.inc + 2 * (group - 1) * width + at, width, lane, tag, a.reads);
        l.inc[lane] = h.x();
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        if (k < n) {
            if (!__all(v[k].there(tag)))
                all = all && v[k].wait(a.agg + 2 * (lo + k) * width + at, width, lane, tag, a.reads);
            f = then(f, Map{v[k].x(), v[k].y()});
        }
    l.part[wave][lane] = make_float2(f.A, f.H);
    if (!all) l.missing = 1;
}
// The first tile of the backward pass that something comes in from to tile j, whose positions begin at p0: the
// one with the end of the sequence that goes on behind this one (j: none does).
__device__ __forceinline__ int first_back(const GatedArgs& a, int j, int p0, int lane) {
    const int next = p0 + kGatedBwdTile;
    if (next >= a.N) return j;
    const int q = seq_at_wave(a, next, lane);
    if (bound_of(a, q) == next) return j;
    return min(max(a.tiles - 1 - (bound_of(a, q + 1) - 1) / kGatedBwdTile, 0), j);
}
// What enters the tile in channel ch of the block (0 when nothing does).
__device__ __forceinline__ float chain_carry(const ChainLds& l, int ch) {
    float h = l.inc[ch];
#pragma unroll
    for (int k = 0; k < 4; ++k) h = Map{l.part[k][ch].x, l.part[k][ch].y}(h);
    return h;
}
// A group's last tile publishes the state it leaves.
template <bool kBack>
__device__ __forceinline__ void chain_leave(const GatedArgs& a, const ChainLds& l, int j, int cb, uint64_t tag, int wave,
                                            int lane) {
    if (wave != 0 || j + 1 >= a.tiles || j % kGatedGroup != kGatedGroup - 1) return;
    const int64_t width = static_cast<int64_t>(a.ncb) * kGatedBlock;
    const float h = tile_map<kBack>(l, lane)(chain_carry(l, lane));
    hand_over(a.inc + 2 * (j / kGatedGroup) * width + cb * kGatedBlock, width, lane, tag, h, 0.0f);
}

// Sequences without tokens: what comes out is what went in (0 without it). Shared out over the tiles.
__device__ __forceinline__ void pass_empty(const GatedArgs& a, const float* in, float* out, int j, int cb) {
    if (!out || (!a.offsets && a.N > 0)) return;
    const int ch = cb * kGatedBlock + (static_cast<int>(threadIdx.x) & 63);
    if (ch >= a.D) return;
    for (int64_t q = j * 4 + (threadIdx.x >> 6); q < a.nseq; q += static_cast<int64_t>(a.tiles) * 4) {
        const int k = static_cast<int>(q);
        if (a.N > 0 && bound_of(a, k + 1) > bound_of(a, k)) continue;
        const int64_t slot = seq_of(a, k) * a.D + ch;
        out[slot] = in ? in[slot] : 0.0f;
    }
}

// A value that the compiler fuses into no other operation.
__device__ __forceinline__ float rounded(float v) {
    asm("" : "+v"(v));
    return v;
}
// Pins values: they are computed before this point, not where they are used (which would keep what they
// are computed from in registers).
template <int T, int V>
__device__ __forceinline__ void pin_all(float (&a)[T][V]) {
#pragma unroll
    for (int k = 0; k < T; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) asm volatile("" : "+v"(a[k][v]));
}

// Makes the compiler take loaded values as new ones, so that what was computed from them before is not
// kept in registers for a later use.
template <int V>
__device__ __forceinline__ void forget(Raw<Bf16, V>& r) {
    if constexpr (V == 1) {
        uint32_t w = r.w;
        asm volatile("" : "+v"(w));
        r.w = static_cast<uint16_t>(w);
    } else {
        asm volatile("" : "+v"(r.w));
    }
}
template <int V>
__device__ __forceinline__ void forget(Raw<float, V>&) {}

// The initial state of the sequence that starts at a position (row: the caller's sequence), for the
// thread's channels from c0 on.
template <int V>
__device__ __forceinline__ void seq_value(const GatedArgs& a, const float* from, int row, int c0, float (&h)[V]) {
    const float* p = from + static_cast<int64_t>(row) * a.D + c0;
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = from && c0 < a.D ? p[v] : 0.0f;
}

// The kernel's arguments, read again where the hardware points at them: the slow path below reads each where it
// wants it, so that no register of the kernel is held for it (nor are indices: afresh makes one a new value to
// the compiler).
using ArgsAt = decltype(__builtin_amdgcn_kernarg_segment_ptr());
__device__ __forceinline__ const GatedArgs& args_again(ArgsAt at) {
    asm volatile("" : "+s"(at));
    return *(const GatedArgs*)at;
}
__device__ __forceinline__ int afresh_s(int v) {
    asm volatile("" : "+s"(v));
    return v;
}
__device__ __forceinline__ int afresh_v(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// The slow path of a workgroup whose wait took too long: each wave walks 64 channels, one a lane, element by
// element from the inputs, about a microsecond a position. A tile of TILE positions is 4 G runs of T, in the order
// of its threads. Measured, with every wait given up at once: 8 x 1025 x 768 bf16 1.3 ms forward, 2.0 backward; one
// sequence of 16384 x 768 22 and 41 ms. Its being there costs the calls that do not take it nothing that
// repeated timing shows above 1.5%.
template <typename IO, int V, int TILE>
struct Alone {
    static constexpr int CL = kGatedBlock / V, T = TILE * CL / 256, G = 64 / CL, kEach = kGatedGroup / 4;
    ArgsAt at;
    int c, lane;             // the lane's channel
    bool live;
    float k2;

    __device__ __forceinline__ Alone(ArgsAt args, int cb, int ln) : at(args), c(cb * kGatedBlock + ln), lane(ln) {
        const GatedArgs& a = args_again(at);
        live = c < a.D;
        k2 = decay_rate(a.lam[live ? c : 0], a.c);
    }

    __device__ __forceinline__ const GatedArgs& args() const { return args_again(at); }
    __device__ __forceinline__ int64_t row(const GatedArgs& a, int p) const { return a.rev ? a.N - 1 - p : p; }
    // An element of position p; 0 past the stream's end, in a channel past the row's and of an absent tensor.
    __device__ __forceinline__ float get(const void* base, int64_t ld, int p) const {
        const GatedArgs& a = args();
        Raw<IO, 1> v;
        v.zero();
        if (base && live && p < a.N) v.load(static_cast<const IoElem<IO>*>(base) + row(a, p) * ld + c);
        return v.get(0);
    }
    __device__ __forceinline__ void put(void* base, int64_t ld, int p, float x) const {
        const GatedArgs& a = args();
        Raw<IO, 1> v;
        v.set(&x);
        if (base && live && p < a.N) v.store(static_cast<IoElem<IO>*>(base) + row(a, p) * ld + c);
    }
    __device__ __forceinline__ float state(const float* from, int q) const {
        const GatedArgs& a = args();
        return from && live ? from[seq_of(a, q) * a.D + c] : 0.0f;
    }
    __device__ __forceinline__ bool starts(int p, int q) const {
        const GatedArgs& a = args();
        return p < a.N && bound_of(a, q) == p;
    }
    __device__ __forceinline__ bool ends(int p, int q) const {
        const GatedArgs& a = args();
        return p < a.N && (bound_of(a, q + 1) == p + 1 || p + 1 == a.N);
    }
    __device__ __forceinline__ int seq(int p) const {
        const GatedArgs& a = args();
        return seq_at_wave(a, min(p, a.N - 1), lane);
    }

    // The map of a run of T positions from pt on.
    __device__ __forceinline__ Map run_fwd(int pt) const {
        Map f = identity();
        bool cut = false;
#pragma unroll 1
        for (int p = pt; p < pt + T; ++p) {
            const GatedArgs& a = args();
            const int q = seq(p);
            if (starts(p, q)) {
                f.H = state(a.h0, q);
                cut = true;
            }
            float at, mg;
            gates(get(a.r, a.ld_r, p), get(a.i, a.ld_i, p), k2, &at, &mg);
            f.A *= at;
            f.H = fmaf(at, f.H, mg * get(a.x, a.ld_x, p));
        }
        f.A = cut ? 0.0f : fmaxf(f.A, kLeast);
        return f;
    }
    // The same as the backward kernel forms it (its gates keep the complements).
    __device__ __forceinline__ Map run_states(int pt) const {
        Map f = identity();
        bool cut = false;
#pragma unroll 1
        for (int p = pt; p < pt + T; ++p) {
            const GatedArgs& a = args();
            const int q = seq(p);
            if (starts(p, q)) {
                f.H = state(a.h0, q);
                cut = true;
            }
            const float x = get(a.x, a.ld_x, p);
            const BackGates g(get(a.r, a.ld_r, p), get(a.i, a.ld_i, p), x, k2);
            f.A *= g.a;
            f.H = fmaf(g.a, f.H, g.mg * x);
        }
        f.A = cut ? 0.0f : fmaxf(f.A, kLeast);
        return f;
    }
    // Whether a sequence starts or ends among a wave's positions from p on: the backward kernel's walks round a
    // product there that they fuse into the next sum elsewhere.
    __device__ __forceinline__ bool has_cuts(int p) const {
        bool any = false;
#pragma unroll 1
        for (int k = 0; k < T * G; ++k) {
            const int q = seq(p + k);
            any = any || starts(p + k, q) || ends(p + k, q);
        }
        return any;
    }
    // That of the gradient, walked from the run's end.
    __device__ __forceinline__ Map run_back(int pt, bool cuts) const {
        Map e = identity();
        float after = 1.0f;   // what e.H is still to be multiplied with: the decay of the position behind
        bool cut = false;
#pragma unroll 1
        for (int p = pt; p < pt + T; ++p) e.A *= decay(p);
#pragma unroll 1
        for (int p = pt + T - 1; p >= pt; --p) {
            const GatedArgs& a = args();
            const int q = seq(p);
            if (ends(p, q)) {
                e.H = state(a.dh_last, q);
                cut = true;
            }
            e.H = fmaf(after, e.H, get(a.dy, a.ld_dy, p));
            after = decay(p);
            if (cuts) {
                e.H = rounded(after * e.H);
                after = 1.0f;
            }
        }
        e.H = rounded(after * e.H);
        e.A = cut ? 0.0f : fmaxf(e.A, kLeast);
        return e;
    }
    __device__ __forceinline__ float decay(int p) const {
        const GatedArgs& a = args();
        float ns;
        return fast_exp2(k2 * sigmoid2(get(a.r, a.ld_r, p), &ns));
    }

    // What tile j (in walking order) hands over.
    template <bool kBack>
    __device__ __forceinline__ Map tile(int j) const {
        const int p0 = (kBack ? args().tiles - 1 - j : j) * TILE;
        Map all = identity();
#pragma unroll 1
        for (int w = 0; w < 4; ++w) {
            Map part = identity();
            const bool cuts = kBack && has_cuts(p0 + (3 - w) * G * T);
#pragma unroll 1
            for (int g = 0; g < G; ++g) {
                const int run = w * G + g;
                const Map f = kBack ? run_back(p0 + (4 * G - 1 - run) * T, cuts) : run_fwd(p0 + run * T);
                part = g == 0 ? f : then(part, f);
            }
            all = then(all, part);
        }
        return all;
    }

    // Fills l.part and l.inc for tile j as chain_gather does: wave 0 walks the groups before tile j's, from tile
    // first on, and then every wave its quarter of the group.
    template <bool kBack>
    __device__ __forceinline__ void gather(ChainLds& l, int j, int first, int wave) const {
        const int g0 = j / kGatedGroup * kGatedGroup;
        const int lo = (first < g0 ? g0 : first) + wave * kEach, end = min(j, lo + kEach);
        float h = 0.0f;
        Map f = identity();
        int quarters = 0;
#pragma unroll 1
        for (int t = wave == 0 && first < g0 ? first : lo; t < end; ++t) {
            const Map m = tile<kBack>(t);
            const bool last = t < lo && t % kGatedGroup == kGatedGroup - 1;
            if (!last) f = then(f, m);
            if (t >= lo) continue;
            // a quarter of a group before this one ends here, or the group does (empty quarters count too)
            if (!last && (t - max(first, t / kGatedGroup * kGatedGroup)) % kEach != kEach - 1) continue;
            do {
                h = f(h);
                f = identity();
            } while (++quarters < 4 && last);
            if (last) {
                h = m(h);
                quarters = 0;
            }
        }
        l.part[wave][lane] = make_float2(f.A, f.H);
        if (wave == 0) l.inc[lane] = h;
        if (wave == 0 && lane == 0) __hip_atomic_fetch_add(&g_alone, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
};

// The rest of k_gated_fwd behind the hand-over, without it. Called by all threads.
template <typename IO, int V, int TILE>
__device__ __forceinline__ void fwd_alone(ChainLds& l, int j, int cb, uint64_t tag) {
    using W = Alone<IO, V, TILE>;
    const int tid = afresh_v(static_cast<int>(threadIdx.x));
    const ArgsAt args = __builtin_amdgcn_kernarg_segment_ptr();
    const GatedArgs& a = args_again(args);
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    j = afresh_s(j);
    cb = afresh_s(cb);
    const W s(args, cb, lane);
    const int p0 = j * TILE, start = bound_of(a, s.seq(p0));
    s.template gather<false>(l, j, start >= p0 ? j : start / TILE, wave);
    __syncthreads();
    chain_leave<false>(a, l, j, cb, tag, wave, lane);
    float enter = chain_carry(l, lane);
#pragma unroll 1
    for (int w = 0; w < wave; ++w) enter = Map{l.wave[w][lane].x, l.wave[w][lane].y}(enter);
    Map before = identity();
#pragma unroll 1
    for (int g = 0; g < W::G; ++g) {
        const int pt = p0 + (wave * W::G + g) * W::T;
        float h = before(enter);
        if (a.states && s.live && pt < a.N && pt % kGatedStride == 0)
            a.states[static_cast<int64_t>(pt / kGatedStride) * a.D + s.c] = h;
        before = s.run_fwd(pt);
#pragma unroll 1
        for (int p = pt; p < min(pt + W::T, a.N); ++p) {
            const GatedArgs& a = s.args();
            const int q = s.seq(p);
            if (s.starts(p, q)) h = s.state(a.h0, q);
            float at, mg;
            gates(s.get(a.r, a.ld_r, p), s.get(a.i, a.ld_i, p), s.k2, &at, &mg);
            h = fmaf(at, h, mg * s.get(a.x, a.ld_x, p));
            s.put(a.y, a.D, p, h);
            if (a.h_last && s.live && s.ends(p, q)) a.h_last[seq_of(a, q) * a.D + s.c] = h;
        }
    }
    pass_empty(a, a.h0, a.h_last, j, cb);
}

// The rest of k_gated_bwd, likewise. fwd: the waves' maps of the states; park: T x 256 values.
template <typename IO, int V>
__device__ __forceinline__ void bwd_alone(ChainLds& l, int j, int cb, uint64_t tag, float2 (*fwd)[kGatedBlock], float* park) {
    using W = Alone<IO, V, kGatedBwdTile>;
    const int tid = afresh_v(static_cast<int>(threadIdx.x));
    const ArgsAt args = __builtin_amdgcn_kernarg_segment_ptr();
    const GatedArgs& a = args_again(args);
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    j = afresh_s(j);
    cb = afresh_s(cb);
    const W s(args, cb, lane);
    const int at = a.tiles - 1 - j, p0 = at * kGatedBwdTile;
    s.template gather<true>(l, j, first_back(a, j, p0, lane), wave);
    __syncthreads();
    chain_leave<true>(a, l, j, cb, tag, wave, lane);
    float h = a.states_in[static_cast<int64_t>(at) * a.D + (s.live ? s.c : 0)], d = chain_carry(l, lane), total = 0.0f;
#pragma unroll 1
    for (int w = 0; w < wave; ++w) h = Map{fwd[w][lane].x, fwd[w][lane].y}(h);
#pragma unroll 1
    for (int w = 3; w > wave; --w) d = Map{l.wave[w][lane].x, l.wave[w][lane].y}(d);
    float* mine = park + wave * W::T * 64 + lane;   // of position k: w / d
    const int from = p0 + wave * W::G * W::T;
    const bool cuts = s.has_cuts(from);
#pragma unroll 1
    for (int g = 0; g < W::G; ++g) {
        const int pt = from + g * W::T;
        float hk = (g == 0 ? identity() : s.run_states(from))(h);
        float da = 1.0f, dk = (g == W::G - 1 ? identity() : s.run_back(from + W::T, cuts))(d);
#pragma unroll 1
        for (int p = pt; p < pt + W::T; ++p) {
            const GatedArgs& a = s.args();
            const int q = s.seq(p);
            if (s.starts(p, q)) hk = s.state(a.h0, q);
            const float x = s.get(a.x, a.ld_x, p);
            const BackGates b(s.get(a.r, a.ld_r, p), s.get(a.i, a.ld_i, p), x, s.k2);
            mine[(p - pt) * 64] = fmaf(b.ua, hk, -b.gm);
            hk = fmaf(b.a, hk, b.mg * x);
        }
        float sum = 0.0f;
#pragma unroll 1
        for (int p = pt + W::T - 1; p >= pt; --p) {
            const GatedArgs& a = s.args();
            const int q = s.seq(p);
            if (s.ends(p, q)) {
                dk = s.state(a.dh_last, q);
                if (p == a.N - 1) sum = 0.0f;
            }
            const float x = s.get(a.x, a.ld_x, p);
            const BackGates b(s.get(a.r, a.ld_r, p), s.get(a.i, a.ld_i, p), x, s.k2);
            const float del = fmaf(da, dk, s.get(a.dy, a.ld_dy, p)), ua = mine[(p - pt) * 64], ox = del * b.mg;
            s.put(a.dx, a.ld_dx, p, ox);
            s.put(a.dr, a.ld_dr, p, del * ua * b.ns);
            s.put(a.di, a.ld_di, p, ox * x * b.ng);
            sum = fmaf(del, ua, sum);
            da = cuts ? 1.0f : b.a;
            dk = cuts ? rounded(b.a * del) : del;
            if (a.dh0 && s.live && s.starts(p, q)) a.dh0[seq_of(a, q) * a.D + s.c] = dk;
        }
        if (pt >= a.N || !s.live) sum = 0.0f;
        total = g == 0 ? sum : total + sum;
    }
    pass_empty(a, a.dh_last, a.dh0, j, cb);
    if (!a.dlam) return;
    __syncthreads();
    fwd[wave][lane].x = total;
    __syncthreads();
    if (wave == 0)
        a.part[static_cast<int64_t>(at) * a.ncb * kGatedBlock + cb * kGatedBlock + lane] =
            (fwd[0][lane].x + fwd[1][lane].x) + (fwd[2][lane].x + fwd[3][lane].x);
}

// Forward pass: a tile of TILE positions x 64 channels. The maps compose as (A2, H2)(A1, H1) = (A2 A1, A2 H1 +
// H2), so a tile needs only the state that enters it and no element is read twice. Measured: 1 x 65537 x
// 1536 bf16 188 us (805 MB, 4.3 TB/s), 8 x 1025 x 768 bf16 16.8 us, 128 x 197 x 768 bf16 with saved states 39
// us (4.0 TB/s), 33k x 384 fp32 packed 45 us (4.5 TB/s). Bound: in fp32 memory; in bf16 the hand-over's
// latency beside three exponentials, two reciprocals and a square root per element (as many tokens in sequences
// of 128, which hand nothing over: 166 us). Rows off cache lines: 32 x 1024 x 770 bf16 65 us (202 MB, 3.1 TB/s), as
// the halves of a line are wanted by workgroups of neighbouring ids, which run on different XCDs.
template <typename IO, int V, int TILE, bool kChain, int kPolicy>
__global__ __launch_bounds__(256, TILE < 128 ? 5 : sizeof(IoElem<IO>) == 2 && V > 1 ? 4 : 3) void k_gated_fwd(GatedArgs a) {
    constexpr int CL = kGatedBlock / V, TG = 256 / CL, T = TILE / TG;
    __shared__ ChainLds lds;
    constexpr int P = T * 64 / CL;  // positions of a wave
    __shared__ int rows[4][P];
    const int j = static_cast<int>(blockIdx.x) / a.ncb, cb = static_cast<int>(blockIdx.x) % a.ncb;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (a.N == 0) return pass_empty(a, a.h0, a.h_last, j, cb);
    const int cl = tid % CL, tg = tid / CL, c0 = cb * kGatedBlock + cl * V;
    const bool live = c0 < a.D;
    const int p0 = j * TILE, pt = p0 + tg * T;
    if (kChain && tid == 0) lds.missing = 0;

    float k2[V];
#pragma unroll
    for (int v = 0; v < V; ++v) k2[v] = a.lam[live ? c0 + v : 0];
    Raw<IO, V> xr[T], rr[T], ir[T];
    {
        TileRows<IO, TILE, T> x, r, i;
        r.init(a, a.r, a.ld_r, p0, tg, c0);
        i.init(a, a.i, a.ld_i, p0, tg, c0);
        x.init(a, a.x, a.ld_x, p0, tg, c0);
        if (p0 + TILE <= a.N) {
#pragma unroll
            for (int k = 0; k < T; ++k) {
                rr[k] = ld_tile<IO, V, kPolicy>(r.rsrc, r.vo, r.so + k * r.step);
                ir[k] = ld_tile<IO, V, kPolicy>(i.rsrc, i.vo, i.so + k * i.step);
                xr[k] = ld_tile<IO, V, kPolicy>(x.rsrc, x.vo, x.so + k * x.step);
            }
        } else {
#pragma unroll
            for (int k = 0; k < T; ++k) {
                rr[k] = ld_tile<IO, V, kPolicy>(r.rsrc, r.at(pt + k < a.N), r.so + k * r.step);
                ir[k] = ld_tile<IO, V, kPolicy>(i.rsrc, i.at(pt + k < a.N), i.so + k * i.step);
                xr[k] = ld_tile<IO, V, kPolicy>(x.rsrc, x.at(pt + k < a.N), x.so + k * x.step);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) k2[v] = decay_rate(k2[v], a.c);
    const int q0 = seq_at_wave(a, p0, lane), wt = lane / CL * T;  // wt: the thread's first position in its wave
    WaveSeqs ws;
    ws.find<P>(a, p0 + wave * P, q0, lane, rows[wave]);
    const uint32_t starts = WaveSeqs::bits<T>(ws.starts, wt), ends = WaveSeqs::bits<T>(ws.ends, wt);
    const bool cuts = (ws.starts | ws.ends) != 0;

    float av[T][V], bv[T][V];
    Map f[V], before[V];
#pragma unroll
    for (int k = 0; k < T; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float mg;
            gates(rr[k].get(v), ir[k].get(v), k2[v], &av[k][v], &mg);
            bv[k][v] = mg * xr[k].get(v);
        }
    pin_all(av);
    pin_all(bv);
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        h[v] = 0.0f;
        f[v].A = av[0][v];
    }
    if (!cuts) {
#pragma unroll
        for (int k = 0; k < T; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = fmaf(av[k][v], h[v], bv[k][v]);
    } else {
#pragma unroll
        for (int k = 0; k < T; ++k) {
            if (starts >> k & 1) seq_value(a, a.h0, rows[wave][wt + k], c0, h);
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = fmaf(av[k][v], h[v], bv[k][v]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 1; k < T; ++k) f[v].A *= av[k][v];
        f[v].H = h[v];
        f[v].A = starts ? 0.0f : fmaxf(f[v].A, kLeast);
        Map total;
        scan_rows<CL, false>(f[v], lane, &total, &before[v]);
        if (lane < CL) lds.wave[wave][lane * V + v] = make_float2(total.A, total.H);
    }
    __syncthreads();
    if constexpr (kChain) {
        const uint64_t tag = dispatch_tag();
        const int start = bound_of(a, q0);
        const int first = start >= p0 ? j : start / TILE;
        chain_gather<false>(a, lds, j, cb, first, tag, wave, lane);
        __syncthreads();
        if (__builtin_expect(lds.missing, 0)) return fwd_alone<IO, V, TILE>(lds, j, cb, tag);
        chain_leave<false>(a, lds, j, cb, tag, wave, lane);
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = chain_carry(lds, cl * V + v);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = 0.0f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        for (int w = 0; w < wave; ++w) h[v] = Map{lds.wave[w][cl * V + v].x, lds.wave[w][cl * V + v].y}(h[v]);
        h[v] = before[v](h[v]);
    }
    if (a.states && live && pt < a.N && pt % kGatedStride == 0) {
        float* dst = a.states + static_cast<int64_t>(pt / kGatedStride) * a.D + c0;
#pragma unroll
        for (int v = 0; v < V; ++v) dst[v] = h[v];
    }
    TileRows<IO, TILE, T> y;
    y.init(a, a.y, a.D, p0, tg, c0);
    if (!cuts) {
        // (also a wave past the stream's end comes here, without a boundary: its stores are dropped)
#pragma unroll
        for (int k = 0; k < T; ++k) {
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = fmaf(av[k][v], h[v], bv[k][v]);
            st_tile<IO, V, kPolicy>(y.rsrc, y.at(pt < a.N), y.so + k * y.step, h);
        }
    } else {
#pragma unroll
        for (int k = 0; k < T; ++k) {
            if (starts >> k & 1) seq_value(a, a.h0, rows[wave][wt + k], c0, h);
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = fmaf(av[k][v], h[v], bv[k][v]);
            st_tile<IO, V, kPolicy>(y.rsrc, y.at(pt + k < a.N), y.so + k * y.step, h);
            if (a.h_last && live && (ends >> k & 1)) {
                float* dst = a.h_last + static_cast<int64_t>(rows[wave][wt + k]) * a.D + c0;
#pragma unroll
                for (int v = 0; v < V; ++v) dst[v] = h[v];
            }
        }
    }
    pass_empty(a, a.h0, a.h_last, j, cb);
}

// Backward pass: a tile of kGatedBwdTile positions x 64 channels; workgroups take the tiles from the
// last to the first. With e the gradient that comes in behind a position (dh_last behind a sequence's
// last one), d = dy + e is the state's and a d goes on to the position before. With u, a, m as above, s = sigmoid(r),
// g = sigmoid(i): dx = d m g, di = d m x g (1 - g), w = d (u a h_prev - g x a^2 u / m), dr = w (1 - s),
// dlam = sigmoid(lam) / softplus(lam) sum w. A tile takes half the forward's positions: it holds four
// inputs and both walks. Measured: 128 x 197 x 768 bf16 65 us (271 MB, 4.2 TB/s), 33k x 384 fp32 packed 83 us
// (358 MB, 4.3 TB/s); rows off cache lines 32 x 1024 x 770 bf16 118 us (353 MB, 3.0 TB/s), single channels
// 16 x 1000 x 333 bf16 41 us (75 MB, 1.8 TB/s). Bound: the vector unit's instructions and the hand-over's latency together.
template <typename IO, int V, bool kChain, int kPolicy>
__global__ __launch_bounds__(256, sizeof(IoElem<IO>) == 2 && V > 1 ? 4 : 3) void k_gated_bwd(GatedArgs a) {
    constexpr int CL = kGatedBlock / V, TG = 256 / CL, T = kGatedBwdTile / TG;
    __shared__ ChainLds lds;
    constexpr int P = T * 64 / CL;  // positions of a wave
    __shared__ int rows[4][P];
    __shared__ float2 fwd[4][kGatedBlock];
    __shared__ __align__(16) float park[2 * T][256 * V];
    const int j = static_cast<int>(blockIdx.x) / a.ncb, cb = static_cast<int>(blockIdx.x) % a.ncb;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (a.N == 0) return pass_empty(a, a.dh_last, a.dh0, j, cb);
    const int tile = a.tiles - 1 - j;
    const int cl = tid % CL, tg = tid / CL, c0 = cb * kGatedBlock + cl * V;
    const bool live = c0 < a.D;
    const int p0 = tile * kGatedBwdTile, pt = p0 + tg * T;
    if (kChain && tid == 0) lds.missing = 0;

    float k2[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        k2[v] = a.lam[live ? c0 + v : 0];
        h[v] = a.states_in[static_cast<int64_t>(tile) * a.D + (live ? c0 + v : 0)];
    }
    Raw<IO, V> xr[T], rr[T], ir[T], gr[T];
    {
        TileRows<IO, kGatedBwdTile, T> x, r, i, g;
        r.init(a, a.r, a.ld_r, p0, tg, c0);
        i.init(a, a.i, a.ld_i, p0, tg, c0);
        x.init(a, a.x, a.ld_x, p0, tg, c0);
        g.init(a, a.dy, a.ld_dy, p0, tg, c0);
        if (p0 + kGatedBwdTile <= a.N) {
#pragma unroll
            for (int k = 0; k < T; ++k) {
                rr[k] = ld_tile<IO, V, kPolicy>(r.rsrc, r.vo, r.so + k * r.step);
                ir[k] = ld_tile<IO, V, kPolicy>(i.rsrc, i.vo, i.so + k * i.step);
                xr[k] = ld_tile<IO, V, kPolicy>(x.rsrc, x.vo, x.so + k * x.step);
                gr[k] = ld_tile<IO, V, kPolicy>(g.rsrc, g.vo, g.so + k * g.step);
            }
        } else {
#pragma unroll
            for (int k = 0; k < T; ++k) {
                rr[k] = ld_tile<IO, V, kPolicy>(r.rsrc, r.at(pt + k < a.N), r.so + k * r.step);
                ir[k] = ld_tile<IO, V, kPolicy>(i.rsrc, i.at(pt + k < a.N), i.so + k * i.step);
                xr[k] = ld_tile<IO, V, kPolicy>(x.rsrc, x.at(pt + k < a.N), x.so + k * x.step);
                gr[k] = ld_tile<IO, V, kPolicy>(g.rsrc, g.at(pt + k < a.N), g.so + k * g.step);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) k2[v] = decay_rate(k2[v], a.c);
    const int q0 = seq_at_wave(a, p0, lane), wt = lane / CL * T;  // wt: the thread's first position in its wave
    WaveSeqs ws;
    ws.find<P>(a, p0 + wave * P, q0, lane, rows[wave]);
    const uint32_t starts = WaveSeqs::bits<T>(ws.starts, wt), ends = WaveSeqs::bits<T>(ws.ends, wt);
    const bool cuts = (ws.starts | ws.ends) != 0;

    // per position: a; m g (of dx and the state's input); u a and g x a^2 u / m (of w). 1 - sigmoid(r)
    // and 1 - sigmoid(i), wanted at the end only, wait in LDS
    float av[T][V], mg[T][V], ua[T][V], gm[T][V];
#pragma unroll
    for (int k = 0; k < T; ++k) {
        float ns[V], ng[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const BackGates g(rr[k].get(v), ir[k].get(v), xr[k].get(v), k2[v]);
            av[k][v] = g.a;
            mg[k][v] = g.mg;
            ua[k][v] = g.ua;
            gm[k][v] = g.gm;
            ns[v] = g.ns;
            ng[v] = g.ng;
        }
        Raw<float, V> w;
        w.set(ns);
        w.store(&park[2 * k][tid * V]);
        w.set(ng);
        w.store(&park[2 * k + 1][tid * V]);
    }
    pin_all(av);
    pin_all(mg);
    pin_all(ua);
    pin_all(gm);
    Map f[V], e[V];
#pragma unroll
    for (int v = 0; v < V; ++v) f[v].H = e[v].H = 0.0f;
    if (!cuts) {
#pragma unroll
        for (int k = 0; k < T; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) f[v].H = fmaf(av[k][v], f[v].H, mg[k][v] * xr[k].get(v));
#pragma unroll
        for (int k = T - 1; k >= 0; --k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float own = gr[k].get(v);
                e[v].H = k == T - 1 ? own : fmaf(av[k == T - 1 ? k : k + 1][v], e[v].H, own);
            }
#pragma unroll
        for (int v = 0; v < V; ++v) e[v].H *= av[0][v];
    } else {
        float g[V];
#pragma unroll
        for (int k = 0; k < T; ++k) {
            if (starts >> k & 1) {
                seq_value(a, a.h0, rows[wave][wt + k], c0, g);
#pragma unroll
                for (int v = 0; v < V; ++v) f[v].H = g[v];
            }
#pragma unroll
            for (int v = 0; v < V; ++v) f[v].H = fmaf(av[k][v], f[v].H, mg[k][v] * xr[k].get(v));
        }
#pragma unroll
        for (int k = T - 1; k >= 0; --k) {
            if (ends >> k & 1) {
                seq_value(a, a.dh_last, rows[wave][wt + k], c0, g);
#pragma unroll
                for (int v = 0; v < V; ++v) e[v].H = g[v];
            }
#pragma unroll
            for (int v = 0; v < V; ++v) e[v].H = rounded(av[k][v] * (gr[k].get(v) + e[v].H));
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        f[v].A = av[0][v];
#pragma unroll
        for (int k = 1; k < T; ++k) f[v].A *= av[k][v];
        e[v].A = ends ? 0.0f : fmaxf(f[v].A, kLeast);
        f[v].A = starts ? 0.0f : fmaxf(f[v].A, kLeast);
    }
    Map fb[V], eb[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        Map total;
        scan_rows<CL, false>(f[v], lane, &total, &fb[v]);
        if (lane < CL) fwd[wave][lane * V + v] = make_float2(total.A, total.H);
        scan_rows<CL, true>(e[v], lane, &total, &eb[v]);
        if (lane < CL) lds.wave[wave][lane * V + v] = make_float2(total.A, total.H);
    }
    __syncthreads();
    // widening again is cheaper than keeping the widened values
#pragma unroll
    for (int k = 0; k < T; ++k) {
        forget(xr[k]);
        forget(gr[k]);
    }
    pin_all(mg);
    const uint64_t tag = kChain ? dispatch_tag() : 0;
    if constexpr (kChain) chain_gather<true>(a, lds, j, cb, first_back(a, j, p0, lane), tag, wave, lane);
    // the state before every position, meanwhile: ua becomes w / d
#pragma unroll
    for (int v = 0; v < V; ++v) {
        for (int w = 0; w < wave; ++w) h[v] = Map{fwd[w][cl * V + v].x, fwd[w][cl * V + v].y}(h[v]);
        h[v] = fb[v](h[v]);
    }
    if (!cuts) {
#pragma unroll
        for (int k = 0; k < T; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                ua[k][v] = fmaf(ua[k][v], h[v], -gm[k][v]);
                h[v] = fmaf(av[k][v], h[v], mg[k][v] * xr[k].get(v));
            }
    } else {
#pragma unroll
        for (int k = 0; k < T; ++k) {
            if (starts >> k & 1) seq_value(a, a.h0, rows[wave][wt + k], c0, h);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                ua[k][v] = fmaf(ua[k][v], h[v], -gm[k][v]);
                h[v] = fmaf(av[k][v], h[v], mg[k][v] * xr[k].get(v));
            }
        }
    }
#pragma unroll
    for (int k = 0; k < T; ++k) forget(xr[k]);
    float d[V], sum[V];
    if constexpr (kChain) {
        __syncthreads();
        if (__builtin_expect(lds.missing, 0)) return bwd_alone<IO, V>(lds, j, cb, tag, fwd, &park[0][0]);
        chain_leave<true>(a, lds, j, cb, tag, wave, lane);
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] = chain_carry(lds, cl * V + v);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] = 0.0f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        for (int w = 3; w > wave; --w) d[v] = Map{lds.wave[w][cl * V + v].x, lds.wave[w][cl * V + v].y}(d[v]);
        d[v] = eb[v](d[v]);
        sum[v] = 0.0f;
    }
    TileRows<IO, kGatedBwdTile, T> dx, dr, di;
    dx.init(a, a.dx, a.ld_dx, p0, tg, c0);
    dr.init(a, a.dr, a.ld_dr, p0, tg, c0);
    di.init(a, a.di, a.ld_di, p0, tg, c0);
    // the gradient's walk through position k, where what goes on to it is carry d; in: it is inside the stream
    auto walk = [&](int k, const float (&carry)[V], bool in) {
        float ox[V], orr[V], oi[V];
        Raw<float, V> ns, ng;
        ns.load(&park[2 * k][tid * V]);
        ng.load(&park[2 * k + 1][tid * V]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float del = fmaf(carry[v], d[v], gr[k].get(v));
            ox[v] = del * mg[k][v];
            oi[v] = ox[v] * xr[k].get(v) * ng.get(v);
            orr[v] = del * ua[k][v] * ns.get(v);
            sum[v] = fmaf(del, ua[k][v], sum[v]);
            d[v] = del;
        }
        st_tile<IO, V, kPolicy>(dx.rsrc, dx.at(in), dx.so + k * dx.step, ox);
        st_tile<IO, V, kPolicy>(dr.rsrc, dr.at(in), dr.so + k * dr.step, orr);
        st_tile<IO, V, kPolicy>(di.rsrc, di.at(in), di.so + k * di.step, oi);
    };
    float one[V];
#pragma unroll
    for (int v = 0; v < V; ++v) one[v] = 1.0f;
    if (!cuts) {
#pragma unroll
        for (int k = T - 1; k >= 0; --k) {
            if (k == T - 1) walk(k, one, pt < a.N);
            else walk(k, av[k + 1], pt < a.N);
        }
    } else {
#pragma unroll
        for (int k = T - 1; k >= 0; --k) {
            if (ends >> k & 1) {
                // behind the stream's end nothing counts for dlam (it may be NaN that came in from a tile)
                seq_value(a, a.dh_last, rows[wave][wt + k], c0, d);
#pragma unroll
                for (int v = 0; v < V; ++v) sum[v] = pt + k == a.N - 1 ? 0.0f : sum[v];
            }
            walk(k, one, pt + k < a.N);
#pragma unroll
            for (int v = 0; v < V; ++v) d[v] = rounded(av[k][v] * d[v]);
            if (a.dh0 && live && (starts >> k & 1)) {
                float* dst = a.dh0 + static_cast<int64_t>(rows[wave][wt + k]) * a.D + c0;
#pragma unroll
                for (int v = 0; v < V; ++v) dst[v] = d[v];
            }
        }
    }
    pass_empty(a, a.dh_last, a.dh0, j, cb);
    if (!a.dlam) return;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float p, q;
        sum[v] = pt < a.N && live ? sum[v] : 0.0f;
        if constexpr (CL < 64) {
            swap32(sum[v], &p, &q);
            sum[v] = p + q;
        }
    }
    __syncthreads();
    if (lane < CL) {
#pragma unroll
        for (int v = 0; v < V; ++v) fwd[wave][lane * V + v].x = sum[v];
    }
    __syncthreads();
    if (wave == 0)
        a.part[static_cast<int64_t>(tile) * a.ncb * kGatedBlock + cb * kGatedBlock + lane] =
            (fwd[0][lane].x + fwd[1][lane].x) + (fwd[2][lane].x + fwd[3][lane].x);
}

// dlam = sigmoid(lam) / softplus(lam) * the sum of the tiles' partial sums, in a fixed order. Latency
// bounds it: 4.7 us for 394 partials of 768 channels.
__global__ __launch_bounds__(1024) void k_gated_dlam(GatedArgs a, int parts) {
    const int c0 = static_cast<int>(blockIdx.x) * kColumns, d = c0 + static_cast<int>(threadIdx.x);
    const float sum = column_sum(a.part, parts, static_cast<int64_t>(a.ncb) * kGatedBlock, c0, a.D);
    if (threadIdx.x >= kColumns || d >= a.D) return;
    const float lam = a.lam[d];
    const float sp = decay_rate(lam, -kLn2);  // softplus(lam)
    // both tend to e^lam as lam goes to -infinity, where the ratio goes to 1
    const float ratio = sp > 0.0f ? fast_rcp(1.0f + fast_exp2(-lam * kLog2e)) / sp : 1.0f;
    a.dlam[d] = sum * ratio;
}

struct StepArgs {
    const void* x;
    const void* r;
    const void* i;
    int64_t ld_x, ld_r, ld_i;
    const float* lam;
    float c;
    float* state;
    int64_t nslots;
    const int32_t* slots_in;
    const int32_t* slots_out;
    void* y;
    int32_t D, batch, per_row;
};

// One token: h' = a h + m sigmoid(i) x, V channels a thread, a row of D takes per_row threads. A call's launch
// bounds it: 1 x 768 takes 2.4 us on the GPU and 3.7 us a call, 512 x 1536 bf16 4.8 us (12.6 MB).
template <typename IO, int V>
__global__ __launch_bounds__(256) void k_gated_step(StepArgs a) {
    const uint32_t t = blockIdx.x * 256u + threadIdx.x;
    const uint32_t b = t / static_cast<uint32_t>(a.per_row);
    const int d = static_cast<int>(t - b * static_cast<uint32_t>(a.per_row)) * V;
    if (b >= static_cast<uint32_t>(a.batch)) return;
    using E = IoElem<IO>;
    const int64_t from = a.slots_in ? a.slots_in[b] : static_cast<int64_t>(b);
    const int64_t to = a.slots_out ? a.slots_out[b] : from;
    Raw<IO, V> x, r, i, y;
    Raw<float, V> lam, s;
    x.load(static_cast<const E*>(a.x) + b * a.ld_x + d);
    r.load(static_cast<const E*>(a.r) + b * a.ld_r + d);
    i.load(static_cast<const E*>(a.i) + b * a.ld_i + d);
    lam.load(a.lam + d);
    const bool in = from >= 0 && from < a.nslots && to >= 0 && to < a.nslots;
    if (in) s.load(a.state + from * a.D + d);
    else s.zero();
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float at, mg;
        gates(r.get(v), i.get(v), decay_rate(lam.get(v), a.c), &at, &mg);
        h[v] = in ? fmaf(at, s.get(v), mg * x.get(v)) : 0.0f;
    }
    if (in) {
        s.set(h);
        s.store(a.state + to * a.D + d);
    }
    y.set(h);
    y.store(static_cast<E*>(a.y) + static_cast<int64_t>(b) * a.D + d);
}

GatedArgs common_args(const vimscan_gated* g, const vimscan_launch* l, const GatedPlan& p) {
    GatedArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = g->x;
    a.r = g->r;
    a.i = g->i;
    a.ld_x = g->ld_x;
    a.ld_r = g->ld_r;
    a.ld_i = g->ld_i;
    a.lam = g->lam;
    a.h0 = g->h0;
    a.offsets = g->offsets;
    a.c = g->c;
    a.N = static_cast<int32_t>(p.tokens);
    a.Lp = static_cast<int32_t>(p.Lp);
    if (p.Lp > 0) {
        // exact for positions below 2^31: lp_mul = floor(2^(31 + s) / Lp) + 1 with 2^(s - 1) < Lp <= 2^s
        int s = 0;
        while ((int64_t(1) << s) < p.Lp) ++s;
        a.lp_mul = static_cast<uint32_t>((uint64_t(1) << (31 + s)) / static_cast<uint64_t>(p.Lp) + 1);
        a.lp_shift = static_cast<uint32_t>(31 + s);
    }
    a.D = static_cast<int32_t>(l->d_inner);
    a.nseq = static_cast<int32_t>(p.nseq);
    a.ncb = static_cast<int32_t>(p.ncb);
    a.tiles = static_cast<int32_t>(p.tiles);
    char* ws = static_cast<char*>(l->workspace);
    if (p.chain) {
        a.agg = reinterpret_cast<uint64_t*>(ws);
        a.inc = reinterpret_cast<uint64_t*>(ws + p.off_inc);
    }
    a.part = p.ws > p.off_part ? reinterpret_cast<float*>(ws + p.off_part) : nullptr;
    a.rev = (l->flags & VIMSCAN_FLAG_REVERSE) ? 1 : 0;
    a.reads = g_wait_reads.load(std::memory_order_relaxed);
    return a;
}

// The caller's event pair around the call's kernels.
bool record(const vimscan_launch* l, int k) {
    if (!l->scan_events[0] || !l->scan_events[1]) return true;
    return hipEventRecord(static_cast<hipEvent_t>(l->scan_events[k]), static_cast<hipStream_t>(l->stream)) == hipSuccess;
}

// kVec channels per lane where every row of every tensor is aligned to them: half as many accesses as with one,
// of rows of 128 or 256 bytes a half wave. Measured at 128 x 197 x 768, two channels and one: bf16 37 and 44 us
// forward, 67 and 85 backward; fp32 59 and 65, 109 and 119.
constexpr int kVec = 2;

// Rows of one tensor, as far as the choice of a kernel goes.
struct RowsOf {
    const void* p;
    int64_t ld;
};
// Every tensor's rows start at multiples of bytes.
template <size_t N>
bool rows_at(const RowsOf (&rows)[N], size_t e, size_t bytes) {
    for (const RowsOf& r : rows)
        if (r.p && (reinterpret_cast<uintptr_t>(r.p) % bytes != 0 || static_cast<size_t>(r.ld) * e % bytes != 0)) return false;
    return true;
}

template <typename IO, int V, int TILE, int kPolicy>
void launch_fwd(const GatedArgs& a, const GatedPlan& p, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.wgs));
    if (p.chain) hipLaunchKernelGGL((k_gated_fwd<IO, V, TILE, true, kPolicy>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_gated_fwd<IO, V, TILE, false, kPolicy>), grid, dim3(256), 0, s, a);
}
template <typename IO>
void launch_fwd_any(const GatedArgs& a, const GatedPlan& p, hipStream_t s) {
    constexpr size_t e = sizeof(IoElem<IO>);
    const RowsOf rows[] = {{a.x, a.ld_x}, {a.r, a.ld_r}, {a.i, a.ld_i}, {a.y, a.D}};
    const bool vec = a.D % kVec == 0 && rows_at(rows, e, kVec * e), big = p.tile == kGatedFwdTile;
    // small calls do not gain from kOnce: their inputs are often in the caches still (8 x 1025 x 768 bf16 16.9
    // us, with it 17.1; 256 x 51 x 1536, 5,000 workgroups, 46.0 and 41.4)
    const bool once = rows_at(rows, e, 128) && (big || p.wgs >= 2048);
    if (vec && big && once) launch_fwd<IO, kVec, kGatedFwdTile, kOnce>(a, p, s);
    else if (vec && once) launch_fwd<IO, kVec, kGatedFwdTileSmall, kOnce>(a, p, s);
    else if (vec && big) launch_fwd<IO, kVec, kGatedFwdTile, kPlain>(a, p, s);
    else if (vec) launch_fwd<IO, kVec, kGatedFwdTileSmall, kPlain>(a, p, s);
    else if (big) launch_fwd<IO, 1, kGatedFwdTile, kPlain>(a, p, s);
    else launch_fwd<IO, 1, kGatedFwdTileSmall, kPlain>(a, p, s);
}

template <typename IO, int V, int kPolicy>
void launch_bwd(const GatedArgs& a, const GatedPlan& p, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.wgs));
    if (p.chain) hipLaunchKernelGGL((k_gated_bwd<IO, V, true, kPolicy>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_gated_bwd<IO, V, false, kPolicy>), grid, dim3(256), 0, s, a);
}
template <typename IO>
void launch_bwd_any(const GatedArgs& a, const GatedPlan& p, hipStream_t s) {
    constexpr size_t e = sizeof(IoElem<IO>);
    const RowsOf rows[] = {{a.x, a.ld_x},   {a.r, a.ld_r},   {a.i, a.ld_i},  {a.dy, a.ld_dy},
                           {a.dx, a.ld_dx}, {a.dr, a.ld_dr}, {a.di, a.ld_di}};
    if (a.D % kVec != 0 || !rows_at(rows, e, kVec * e)) launch_bwd<IO, 1, kPlain>(a, p, s);
    else if (rows_at(rows, e, 128)) launch_bwd<IO, kVec, kOnce>(a, p, s);
    else launch_bwd<IO, kVec, kPlain>(a, p, s);
}

}  // namespace

extern "C" {

int vimscan_gated_alone(uint64_t* count) {
    if (!count) return VIMSCAN_ERR_NULL;
    unsigned long long v = 0;
    if (hipMemcpyFromSymbol(&v, HIP_SYMBOL(g_alone), sizeof(v), 0, hipMemcpyDeviceToHost) != hipSuccess)
        return VIMSCAN_ERR_HIP;
    *count = static_cast<uint64_t>(v);
    return VIMSCAN_OK;
}

int vimscan_gated_wait_reads(int32_t reads) {
    if (reads < 0) return VIMSCAN_ERR_PARAM;
    g_wait_reads.store(reads, std::memory_order_relaxed);
    return VIMSCAN_OK;
}

int vimscan_gated_fwd(const vimscan_gated* g, int64_t seg_len, void* y, float* h_last, float* states,
                      const vimscan_launch* launch) {
    if (!g || !launch) return VIMSCAN_ERR_NULL;
    GatedPlan p;
    int rc = vimscan_host::make_gated_plan(launch, seg_len, g->offsets != nullptr, g->nseq, false, &p);
    if (rc != VIMSCAN_OK) return rc;
    rc = vimscan_host::check_gated_call(g, y, h_last, states, nullptr, launch, p);
    if (rc != VIMSCAN_OK) return rc;
    if (p.wgs == 0 || (p.tokens == 0 && !h_last)) return VIMSCAN_OK;
    GatedArgs a = common_args(g, launch, p);
    a.y = y;
    a.h_last = h_last;
    a.states = states;
    hipStream_t s = static_cast<hipStream_t>(launch->stream);
    if (!record(launch, 0)) return VIMSCAN_ERR_HIP;
    if (launch->io_dtype == VIMSCAN_F32) launch_fwd_any<float>(a, p, s);
    else launch_fwd_any<Bf16>(a, p, s);
    if (hipGetLastError() != hipSuccess || !record(launch, 1)) return VIMSCAN_ERR_HIP;
    return VIMSCAN_OK;
}

int vimscan_gated_bwd(const vimscan_gated* g, int64_t seg_len, const vimscan_gated_grad* grad,
                      const vimscan_launch* launch) {
    if (!g || !grad || !launch) return VIMSCAN_ERR_NULL;
    GatedPlan p;
    int rc = vimscan_host::make_gated_plan(launch, seg_len, g->offsets != nullptr, g->nseq, true, &p);
    if (rc != VIMSCAN_OK) return rc;
    rc = vimscan_host::check_gated_call(g, nullptr, nullptr, nullptr, grad, launch, p);
    if (rc != VIMSCAN_OK) return rc;
    if (launch->d_inner == 0) return VIMSCAN_OK;
    GatedArgs a = common_args(g, launch, p);
    a.dy = grad->dy;
    a.dh_last = grad->dh_last;
    a.states_in = grad->states;
    a.dx = grad->dx;
    a.dr = grad->dr;
    a.di = grad->di;
    a.ld_dy = grad->ld_dy;
    a.ld_dx = grad->ld_dx;
    a.ld_dr = grad->ld_dr;
    a.ld_di = grad->ld_di;
    a.dlam = grad->dlam;
    a.dh0 = grad->dh0;
    hipStream_t s = static_cast<hipStream_t>(launch->stream);
    if (!record(launch, 0)) return VIMSCAN_ERR_HIP;
    if (p.wgs > 0) {
        if (launch->io_dtype == VIMSCAN_F32) launch_bwd_any<float>(a, p, s);
        else launch_bwd_any<Bf16>(a, p, s);
    }
    if (a.dlam) {
        const unsigned blocks = static_cast<unsigned>((launch->d_inner + kColumns - 1) / kColumns);
        const int parts = p.tokens > 0 && p.wgs > 0 ? static_cast<int>(p.tiles) : 0;
        hipLaunchKernelGGL(k_gated_dlam, dim3(blocks), dim3(1024), 0, s, a, parts);
    }
    if (hipGetLastError() != hipSuccess || !record(launch, 1)) return VIMSCAN_ERR_HIP;
    return VIMSCAN_OK;
}

int vimscan_gated_step(const vimscan_gated* g, float* state, int64_t nslots, const int32_t* slots_in,
                       const int32_t* slots_out, void* y, const vimscan_launch* launch) {
    const int rc = vimscan_host::check_gated_step(g, state, nslots, slots_in, slots_out, y, launch);
    if (rc != VIMSCAN_OK) return rc;
    if (launch->batch == 0 || launch->d_inner == 0) return VIMSCAN_OK;
    StepArgs a;
    a.x = g->x;
    a.r = g->r;
    a.i = g->i;
    a.ld_x = g->ld_x;
    a.ld_r = g->ld_r;
    a.ld_i = g->ld_i;
    a.lam = g->lam;
    a.c = g->c;
    a.state = state;
    a.nslots = nslots;
    a.slots_in = slots_in;
    a.slots_out = slots_out;
    a.y = y;
    a.D = static_cast<int32_t>(launch->d_inner);
    a.batch = static_cast<int32_t>(launch->batch);
    hipStream_t s = static_cast<hipStream_t>(launch->stream);
    const bool f32 = launch->io_dtype == VIMSCAN_F32;
    const size_t e = f32 ? 4 : 2;
    const RowsOf rows[] = {{a.x, a.ld_x}, {a.r, a.ld_r}, {a.i, a.ld_i}, {y, launch->d_inner}};
    const bool vec = launch->d_inner % kVec == 0 && rows_at(rows, e, kVec * e) &&
                     reinterpret_cast<uintptr_t>(g->lam) % (4 * kVec) == 0 &&
                     reinterpret_cast<uintptr_t>(state) % (4 * kVec) == 0;
    a.per_row = static_cast<int32_t>(vec ? launch->d_inner / kVec : launch->d_inner);
    if (!record(launch, 0)) return VIMSCAN_ERR_HIP;
    const dim3 grid(static_cast<unsigned>((launch->batch * a.per_row + 255) / 256));
    if (vec) {
        if (f32) hipLaunchKernelGGL((k_gated_step<float, kVec>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((k_gated_step<Bf16, kVec>), grid, dim3(256), 0, s, a);
    } else {
        if (f32) hipLaunchKernelGGL((k_gated_step<float, 1>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((k_gated_step<Bf16, 1>), grid, dim3(256), 0, s, a);
    }
    if (hipGetLastError() != hipSuccess || !record(launch, 1)) return VIMSCAN_ERR_HIP;
    return VIMSCAN_OK;
}

}  // extern "C"
