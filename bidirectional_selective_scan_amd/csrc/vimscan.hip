// Bidirectional selective scan for AMD MI355X (gfx950): HIP kernels and the C ABI of
// include/vimscan.h.
//
// What is computed (Vision Mamba page, section 2.2; VSSD notes page, sections 4.1.2 and 4.2.1.3;
// Mamba2D page, "standard Mamba 1D formula"; SF-Mamba page, "Batch folding and periodic state
// reset"): for each (sequence, channel) a forward scan in token order and a backward scan in
// reverse token order over a 16-wide fp32 state, each discretised from its own parameters, read
// out with a skip term, summed and gated by SiLU(z).
//
// Execution design (gfx950, wave64):
//  * Folding: with a reset every seg_len tokens, the segments are independent sequences; in the
//    dense [batch][seqlen][.] layout a folded stream of B*T tokens is byte-for-byte the layout of
//    B sequences of T tokens, so the kernels index segments as sequences. No copy, no select.
//  * One workgroup = one chunk of one sequence x one or two blocks of 64 channels, two waves per
//    block: one runs the forward recurrence, the other the backward one, one channel per lane, the
//    16 states in VGPRs (forward only: every wave is a block of its own). A token's
//    B and C rows are the same for every channel of a sequence, so they are wave-uniform: the
//    chunk's B and C rows of both directions are staged once per workgroup in LDS as fp32
//    (bf16 widened on the way) and read as broadcasts. Nothing in the token loop goes through
//    the scalar memory path: scalar loads complete out of order, so a wait for any of them is a
//    wait for all, which left only one token of latency hiding for a row fetched from HBM.
//  * The two directions meet in the middle of the chunk: in the first half each wave parks its
//    branch output (forward for the first half of the chunk, backward for the second), then
//    after one barrier each wave finishes its own half, adds the parked output of the other
//    direction, applies the SiLU(z) gate and writes y once. Short chunks park in LDS; long ones
//    in a workspace region per workgroup, because an LDS park of a long chunk would leave too
//    few waves per SIMD to keep the VALU issuing (the scan is ALU-bound, not HBM-bound).
//  * Software pipelining: the state-independent part of a token (softplus, delta*x, the 16
//    transitions exp(delta*A)) is computed one token ahead, so it overlaps the dependent state
//    update of the current token; loads run several tokens ahead.
//  * Long sequences are cut into chunks (the associative form of the linear recurrence): per
//    chunk and direction the local end state from zero and the sum of delta over the chunk (the
//    chunk's transition product is exp(A * sum delta)) -- the chunk aggregate; folded in scan
//    order they give the state entering every chunk, from which the chunk is scanned with the
//    readout. Up to kFoldMaxChunks chunks per sequence (both directions or forward only) this is
//    one kernel: each workgroup computes its own chunk's aggregates, hands them to the other
//    chunks of its sequence through the workspace (k_bidir_chain, k_fwd_chain) and folds the
//    ones it receives.
//    Beyond that an aggregate pass, a combine kernel and the scan run as separate kernels.
//    Carries live in the caller's workspace.
//  * delta is kept in log2 units (softplus * log2 e), so the transitions are the hardware exp2
//    of delta2 * A; the state is then scaled by log2(e), which the C rows undo (they are staged
//    as C * ln 2). When a channel's A row is an arithmetic progression in n, the 16 transitions
//    are exp(delta*A0) * q^n with q = exp(delta*dA): two exponentials (one when A0 == dA, as in
//    the S4D-real initialisation A[d,n] = -(n+1)) and multiplies instead of 16 exponentials
//    (an exponential takes two VALU issue slots, an FMA one). A wave takes that path only when
//    every lane's row qualifies (an exact progression with A0 <= 0 and dA <= 0);
//    VIMSCAN_FLAG_GENERAL_DECAY turns it off.
//  * Workgroup ids are remapped so that consecutive logical workgroups (which share a
//    sequence's B/C rows) land on the same XCD and its L2.
//  * Variants of the same kernels (a template parameter): the directional convolution in front
//    of each direction (a register window of the previous raw inputs in walk order), and the scan
//    in a given token order (a step's token is looked up in the chunk's copy of the order in LDS;
//    chunks are ranges of steps, B and C rows are gathered into LDS in step order, so the park,
//    the meeting point and the chunk carries stay indexed by step).

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "handover.h"
#include "plan.h"
#include "vimscan.h"

namespace {

using vimscan_dev::dispatch_tag;
using vimscan_dev::kSpinLimit;
using vimscan_host::kFoldMaxChunks;
using vimscan_host::kMaxTaps;
using vimscan_host::kN;
using vimscan_host::kWave;
using Plan = vimscan_host::ScanPlan;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Bf16 {};  // tag for bf16 io

template <typename IO> struct IoTraits;
template <> struct IoTraits<float> {
    using elem = float;
    static constexpr int bytes = 4;
};
template <> struct IoTraits<Bf16> {
    using elem = uint16_t;
    static constexpr int bytes = 2;
};

__device__ __forceinline__ float fast_exp2(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float fast_log2(float v) { return __builtin_amdgcn_logf(v); }
__device__ __forceinline__ float fast_rcp(float v) { return __builtin_amdgcn_rcpf(v); }

// softplus(v) * log2(e) = log2(1 + 2^w), w = v log2 e. The scan keeps delta in these log2 units:
// the transitions are then 2^(A * delta2) with A as given, and the conversion back to natural
// units is folded into the C rows (C * ln 2, applied once when they are staged).
// Evaluated as max(w, 0) + log2(1 + p), p = 2^-|w| in (0, 1], which never forms 2^w for large w
// (no overflow, no threshold test). log2(1 + p) is taken as log2(v) + r log2(e), v = 1 + p rounded
// and r = p - (v - 1) its rounding error (exact): the correction is log2(1 + r / v) to first
// order, with 1/v dropped, which costs at most 2^-24.5 of the result (log2(1 + p) >= p on (0, 1]).
// Without it, log2(fl(1 + p)) alone is off by up to 2^-24 / p relative: 1e-4 at delta = 6e-4,
// and 0 below delta = 6e-8 -- visible wherever one token's delta * x dominates the state.
// Takes dt and bias * log2(e), so w is one fma.
__device__ __forceinline__ float softplus_log2(float dt, float bias2) {
    const float w = fmaf(dt, kLog2e, bias2);
    const float p = fast_exp2(-fabsf(w));
    const float v = 1.0f + p;
    const float r = p - (v - 1.0f);
    return fmaxf(w, 0.0f) + fmaf(r, kLog2e, fast_log2(v));
}

// silu(v) = v / (1 + e^-v)
__device__ __forceinline__ float silu(float v) { return v * fast_rcp(1.0f + fast_exp2(-v * kLog2e)); }

// Logical workgroup id for hardware id i of n: the hardware deals workgroups to the 8 XCDs
// round-robin; this hands each XCD one contiguous range of logical ids.
__device__ __forceinline__ int xcd_remap(int i, int n) {
    const int q = n >> 3, r = n & 7;
    const int x = i & 7, k = i >> 3;
    return (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + k;
}

// A chunk's rows of one [token][Di] tensor as a buffer resource: loads take the lane's channel
// offset from a VGPR and the token row offset from an SGPR, so no per-lane address arithmetic
// is spent per token. Every offset the kernels form lies inside the range.
// The address is wave-uniform by construction; passing it through readfirstlane makes that
// explicit, so the descriptor lands in SGPRs in every kernel variant.
template <typename T>
__device__ __forceinline__ T* uniform_ptr(T* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return reinterpret_cast<T*>((static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rsrc(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(uniform_ptr(base)), 0,
                                             static_cast<int>(__builtin_amdgcn_readfirstlane(bytes)), 0x00020000);
}
// Raw loads keep the bits as they are in memory (bf16 zero-extended); widening to fp32 happens
// where the value is used, so a prefetched load is not waited for until then.
__device__ __forceinline__ uint32_t ld_raw(float, __amdgpu_buffer_rsrc_t r, uint32_t vo, uint32_t so) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, vo, so, 0);
}
__device__ __forceinline__ uint32_t ld_raw(Bf16, __amdgpu_buffer_rsrc_t r, uint32_t vo, uint32_t so) {
    return static_cast<uint32_t>(__builtin_amdgcn_raw_buffer_load_b16(r, vo, so, 0));
}
// An fp32 ring value is copied into a register of its own when it is taken (as the bf16 shift
// does): the ring slot is then free for the refill the same step issues, where reusing the value in
// place would keep two generations of the ring live (about 30 more VGPRs, 2 waves per SIMD
// instead of 3).
__device__ __forceinline__ float widen(float, uint32_t raw) {
    uint32_t v;
    asm volatile("v_mov_b32 %0, %1" : "=v"(v) : "v"(raw));
    return __uint_as_float(v);
}
__device__ __forceinline__ float widen(Bf16, uint32_t raw) { return __uint_as_float(raw << 16); }
__device__ __forceinline__ void st_buf(float, __amdgpu_buffer_rsrc_t r, uint32_t vo, uint32_t so, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, vo, so, 0);
}
__device__ __forceinline__ void st_buf(Bf16, __amdgpu_buffer_rsrc_t r, uint32_t vo, uint32_t so, float v) {
    const __bf16 b = static_cast<__bf16>(v);  // round to nearest even (hardware conversion on gfx950)
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, b), r, vo, so, 0);
}

struct ScanArgs {
    const void* x;
    const void* dt;
    const void* z;
    const void* Bm[2];      // io-dtype rows as passed: [0] forward, [1] backward
    const void* Cm[2];
    const float* A[2];
    const float* D[2];
    const float* dtb[2];
    void* y;
    float* carry;  // chunked: [dir][seq][chunk][n][Di] states (x log2 e); pass 1 end states / pass 2 inputs
    float* dsum;   // chunked: [dir][seq][chunk][Di] sum of delta * log2(e) over the chunk
    float* parkg;  // park in global memory: [workgroup][T][64] (null: the park is in LDS)
    int Lp;        // tokens per independent sequence
    int Di;
    int nseq;
    int T;         // tokens per chunk
    int K;         // chunks per sequence
    int ncb;       // channel blocks of 64
    int subs;      // channel blocks per workgroup (1 or 2): 2 * subs waves per workgroup
    int general;   // 1: never use the arithmetic-progression transitions
    const float* cw[2];  // directional convolution taps [Di][conv_k] (vimscan_bidir_conv_fwd)
    const float* cb[2];  // its biases [Di]
    int conv_k;          // taps, 1..kMaxTaps; 0 without the convolution
    int uni;             // 1: forward only (vimscan_fwd): every wave of a workgroup is a channel block
    const int32_t* order;  // kOrdered: [nseq][Lp] the token each scan step visits (vimscan_bidir_order_fwd)
    uint64_t* tags;        // one-pass chunked (k_bidir_chain, k_fwd_chain): [dir][seq][chunk][ncb] tags; else null
};

// The directional convolution carries kMaxTaps taps (a layer with fewer taps is run with the
// missing ones at zero). Plans of up to kFoldMaxChunks chunks run as one kernel whose workgroups
// fold the aggregates of the chunks before theirs themselves (fold_carry), kFoldBatch chunks per
// round of loads.
constexpr int kFoldBatch = 4;

// What a scan kernel instance does besides the plain bidirectional scan.
enum Variant {
    kPlain = 0,     // raster order, x as given
    kWithConv = 1,  // the directional convolution + SiLU in front of each direction
    kOrdered = 2    // the tokens of every sequence visited in the order of ScanArgs::order
};

// The state-independent part of one token, computed a token ahead of its state update.
struct Prelude {
    float delta2, x;     // softplus(dt + bias) * log2(e); x (for the skip term)
    float u;             // delta2 * x (the walk against the scan order takes only delta2 and u)
    float e[kN];         // transitions exp(delta * A[d, n]) = 2^(delta2 * A[d, n])
    float ub[kN];        // inputs delta2 * x * B[n] (the state is kept scaled by log2(e))
};

// How a wave forms its 16 transitions (see Lane::prelude).
enum Decay { kGeneral = 0, kProgression = 1, kGeometric = 2 };

// A lane's A row in the form a walk uses it. The general form's 16 values are loaded when its
// walk starts, so they are not live through walks of the other forms (the register peak is then
// that of one form); the progression's two values come from the row the form vote read when the
// kernel started, so a walk of those forms starts without waiting for a load.
template <int kDecay> struct Rates;
template <> struct Rates<kGeneral> {
    float an[kN];  // A[d, n]
    __device__ __forceinline__ void load(const float* A, float, float) {
#pragma unroll
        for (int n = 0; n < kN; ++n) an[n] = A[n];
    }
};
template <> struct Rates<kProgression> {
    float a0, da;  // A[d, 0], A[d, 1] - A[d, 0]
    __device__ __forceinline__ void load(const float*, float a0_, float da_) {
        a0 = a0_;
        da = da_;
    }
};
template <> struct Rates<kGeometric> {
    float da;      // A[d, 1] - A[d, 0] (== A[d, 0])
    __device__ __forceinline__ void load(const float*, float, float da_) { da = da_; }
};

// Per-lane recurrence state of one direction over one channel.
struct Lane {
    float h[kN];    // state scaled by log2(e)
    float a0, da;       // A[d, 0], A[d, 1] - A[d, 0] (set by decay_form)
    float Dsum, bias2;  // D_f[d] + D_b[d] (the skip terms of both directions); dt_bias[d] * log2(e)
    float Dd;           // this direction's D[d] (with the convolution each direction has its own input)
    float ctap[kMaxTaps], cbias;  // convolution: ctap[j] weights the token j steps back in walk order

    // own_skip: the walk adds this direction's D[d] * u itself (the convolution, forward only).
    __device__ __forceinline__ void init(const ScanArgs& a, int dir, int dc, bool own_skip) {
        Dsum = a.D[0][dc] + a.D[1][dc];
        Dd = own_skip ? a.D[dir][dc] : 0.0f;
        bias2 = a.dtb[dir][dc] * kLog2e;
    }

    // Convolution taps of this direction: weight [d][K-1] is on the current token.
    __device__ __forceinline__ void init_conv(const ScanArgs& a, int dir, int dc) {
        const float* w = a.cw[dir] + static_cast<int64_t>(dc) * a.conv_k;
#pragma unroll
        for (int j = 0; j < kMaxTaps; ++j) ctap[j] = j < a.conv_k ? w[a.conv_k - 1 - j] : 0.0f;
        cbias = a.cb[dir][dc];
    }

    // The A row the transition-form vote reads, loaded whole (one memory round trip, no chain of
    // loads behind branches); the kernels issue it before the row staging, so its latency
    // overlaps the staging's.
    struct ARow {
        float r[kN];
    };
    __device__ __forceinline__ ARow load_arow(const ScanArgs& a, int dir, int dc) const {
        ARow row;
        const float* A = a.A[dir] + dc * kN;  // 4-byte aligned only
#pragma unroll
        for (int n = 0; n < kN; ++n) row.r[n] = A[n];
        return row;
    }

    // The transition form this wave uses: one form for all 64 lanes (a wave-wide vote). Keeps
    // A[d, 0] and A[d, 1] - A[d, 0] for the progression forms.
    // The factored forms take only rows that are exact arithmetic progressions in fp32 (A[n] ==
    // A0 + n*dA) and non-positive and non-increasing (A0 <= 0, dA <= 0): then e0 = 2^(delta2 A0)
    // is the largest transition and at most 1, q <= 1, and e0 q^n can underflow only where the
    // exact transition is itself below the smallest normal float. An ascending row would start the
    // chain at its smallest transition, which underflows to 0 (or meets q = inf) while the later
    // ones are still large; such rows take the general form.
    __device__ __forceinline__ int decay_form(const ScanArgs& a, const ARow& row) {
        a0 = row.r[0];
        da = row.r[1] - row.r[0];
        if (a.general) return kGeneral;
        bool ok = a0 <= 0.0f && da <= 0.0f;
#pragma unroll
        for (int n = 0; n < kN; ++n) ok &= (row.r[n] == row.r[0] + static_cast<float>(n) * da);
        if (!__all(ok)) return kGeneral;
        return __all(a0 == da) ? kGeometric : kProgression;
    }

    // Transition forms: kGeneral takes one exponential per state; kProgression uses
    // exp(delta*A0) * q^n for a row A0 + n*dA; kGeometric is the progression with A0 == dA, where
    // the transitions are q^(n+1) and the first exponential is q itself.
    template <int kDecay>
    __device__ __forceinline__ Prelude prelude(float xv, float dtv, const float (&Bv)[kN],
                                               const Rates<kDecay>& r) const {
        Prelude p;
        p.delta2 = softplus_log2(dtv, bias2);
        const float u = p.delta2 * xv;
        p.x = xv;
#pragma unroll
        for (int n = 0; n < kN; ++n) p.ub[n] = u * Bv[n];
        if constexpr (kDecay == kGeneral) {
#pragma unroll
            for (int n = 0; n < kN; ++n) p.e[n] = fast_exp2(p.delta2 * r.an[n]);
        } else {
            // e[n] = e0 * q^n along four independent chains of stride q^4
            const float q = fast_exp2(p.delta2 * r.da);
            const float q2 = q * q;
            const float q4 = q2 * q2;
            if constexpr (kDecay == kGeometric) {
                p.e[0] = q;
                p.e[1] = q2;
                p.e[2] = q2 * q;
                p.e[3] = q4;
            } else {
                p.e[0] = fast_exp2(p.delta2 * r.a0);
                p.e[1] = p.e[0] * q;
                p.e[2] = p.e[0] * q2;
                p.e[3] = p.e[1] * q2;
            }
#pragma unroll
            for (int n = 4; n < kN; ++n) p.e[n] = p.e[n - 4] * q4;
        }
        return p;
    }

    // State update h = e*h + delta2*x*B; returns the readout (C ln 2).h, i.e. C.h in natural
    // units (the skip terms D x of both directions are added once, where the outputs meet). Two
    // accumulation chains: the waves sharing a SIMD hide their latency, and one add joins them.
    template <bool kReadout>
    __device__ __forceinline__ float update(const Prelude& p, const float (&Cv)[kN]) {
        float acc[2] = {0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            h[n] = fmaf(h[n], p.e[n], p.ub[n]);
            if (kReadout) acc[n & 1] = fmaf(Cv[n], h[n], acc[n & 1]);
        }
        return acc[0] + acc[1];
    }

    // The chunk aggregate (the end state of the chunk's scan from a zero state) walked against
    // the scan order. A token t adds u_t B_t[n] times the transitions of every token after it in
    // scan order, prod_{s > t} 2^(delta2_s A[n]) = 2^(S A[n]) with S the sum of delta2 over those
    // tokens -- the tokens this walk has already passed, so S is the running delta sum itself.
    // The factored rows give 2^(S A[n]) = E Q^n (E = 2^(S A0), Q = 2^(S dA); geometric: E = Q)
    // and u enters at the head of that chain: c[n] = u E Q^n, h[n] += c[n] B[n], one product and
    // one fma per state where the scan-order walk needs three operations (its transition, the
    // product u B and the fma). Every transition comes straight from the exact suffix sum, not
    // from a running product.
    __device__ __forceinline__ Prelude prelude_rev(float xv, float dtv) const {
        Prelude p;
        p.delta2 = softplus_log2(dtv, bias2);
        p.x = xv;
        p.u = p.delta2 * xv;
        return p;
    }
    template <int kDecay>
    __device__ __forceinline__ void update_rev(const Prelude& p, const float (&Bv)[kN], const Rates<kDecay>& r,
                                               float S) {
        if constexpr (kDecay == kGeneral) {
#pragma unroll
            for (int n = 0; n < kN; ++n) h[n] = fmaf(p.u * fast_exp2(S * r.an[n]), Bv[n], h[n]);
        } else {
            const float Q = fast_exp2(S * r.da);
            float cn;
            if constexpr (kDecay == kGeometric) cn = p.u * Q;
            else cn = p.u * fast_exp2(S * r.a0);
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                h[n] = fmaf(cn, Bv[n], h[n]);
                if (n + 1 < kN) cn *= Q;
            }
        }
    }
};

struct WgCoords {
    int lid, seq, chunk, cb, lane, dir, sub, slot, d, dc, t0, t1;
    bool valid;
};

// One-pass chunked scan (kChain): the chunks of one (sequence, channel-block group) take
// consecutive workgroup ids, chunk fastest, in hardware order (no XCD remap): a workgroup waits only
// for the other chunks of its group, which the in-order dispatch has started or starts next.
template <bool kChain = false>
__device__ __forceinline__ WgCoords wg_coords(const ScanArgs& a, bool uni) {
    WgCoords c;
    const int lid = kChain ? static_cast<int>(blockIdx.x) : xcd_remap(static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    const int ncbw = (a.ncb + a.subs - 1) / a.subs;  // channel-block groups per sequence
    c.lid = lid;
    int cbw;
    if constexpr (kChain) {
        c.chunk = lid % a.K;
        const int rest = lid / a.K;
        cbw = rest % ncbw;
        c.seq = rest / ncbw;
    } else {
        cbw = lid % ncbw;
        const int rest = lid / ncbw;
        c.chunk = rest % a.K;
        c.seq = rest / a.K;
    }
    c.lane = static_cast<int>(threadIdx.x) & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    c.dir = uni ? 0 : wave & 1;
    c.sub = uni ? wave : wave >> 1;
    c.slot = lid * a.subs + c.sub;  // this wave pair's park region
    c.cb = cbw * a.subs + c.sub;    // may be past the last block when ncb is odd: y gets no stores
    c.d = c.cb * kWave + c.lane;
    c.valid = c.d < a.Di;
    c.dc = c.valid ? c.d : a.Di - 1;
    c.t0 = c.chunk * a.T;
    c.t1 = min(c.t0 + a.T, a.Lp);
    return c;
}

// What a token walk does with each token's readout.
enum WalkMode {
    kPark = 0,      // first half of a chunk: park this direction's output (LDS or global scratch)
    kFinish = 1,    // second half: add the other direction's parked output, gate, store y
    kAggregate = 2, // chunk pass 1: no readout, accumulate sum(delta)
    kOut = 3,       // forward only: gate and store every token (no park, no other direction)
    kAggRev = 4     // chunk pass 1 walked against the scan order (see Lane::update_rev)
};

// The register rings of a walk (see walk): raw x and dt of the steps ahead, z and the parked
// output of the steps it gates, and in a given order the tokens they hold.
constexpr int ring_depth(int var) { return var == kWithConv ? 5 : 6; }
template <int P> struct Ring {
    uint32_t xr[P], dr[P], zr[P], pr[P];
    int tx[P], tz[P];
};

// How a walk treats its rings: fill them and run (kRingFull); only fill them and return
// (kRingPrime: the kernels issue the first walk's ring loads before the row staging, whose latency
// they then share); run on rings already filled (kRingPrimed).
enum RingMode { kRingFull = 0, kRingPrime = 1, kRingPrimed = 2 };

// x of one token by its raw bits (bf16 zero-extended), from the full tensor.
template <typename IO>
__device__ __forceinline__ uint32_t ld_global_raw(const void* base, int64_t i) {
    if constexpr (IoTraits<IO>::bytes == 4) return __float_as_uint(static_cast<const float*>(base)[i]);
    else return static_cast<uint32_t>(static_cast<const uint16_t*>(base)[i]);
}

// Walk this wave's tokens k = kbeg..kend-1 of the chunk (forward: local token k; backward:
// local token len-1-k). Per step k: the prelude of token k+1 (including delta*x*B) is formed
// from a ring of prefetched x/dt values (refilled P tokens ahead) and the B row of token k+1,
// read from the chunk's rows in LDS; z and the parked value of token k come from their own ring;
// token k's state update and readout run on the prelude formed a step earlier, with the C row of
// token k read from LDS in the same step. Every prefetch index is clamped into the walk, so every
// load stays inside the chunk.
// With kConv each direction's input is u = silu(cbias + taps . x) over the current token and
// the three before it in walk order (a register window; at the walk's first step the window is
// loaded from the tokens before it, which may lie in the neighbouring chunk, and is zero
// outside the sequence).
template <typename IO, int kDecay, int kMode, bool kGlobalPark, int kVar, int kRing = kRingFull>
__device__ __forceinline__ void walk(const ScanArgs& a, const WgCoords& c, Lane& ln, float* lds_park,
                                     const float* lds_c, const float* lds_b, const int32_t* lds_ord, int kbeg,
                                     int kend, float& dsum, Ring<ring_depth(kVar)>& rg) {
    constexpr bool kConv = kVar == kWithConv;
    constexpr bool kOrd = kVar == kOrdered;
    static_assert(!(kOrd && kRing != kRingFull), "an ordered walk's tokens come from LDS: it fills its own rings");
    constexpr int P = ring_depth(kVar);  // ring depth (tokens prefetched ahead); the window takes the registers of one slot
    constexpr uint32_t e = IoTraits<IO>::bytes;
    constexpr bool kRev = kMode == kAggRev;
    constexpr bool kReadout = kMode != kAggregate && !kRev;
    static_assert(!(kRev && kConv), "the convolution's window follows the scan order");
    using E = typename IoTraits<IO>::elem;
    if (kbeg >= kend) return;
    const int len = c.t1 - c.t0;
    const int64_t row0 = static_cast<int64_t>(c.seq) * a.Lp + c.t0;  // first step (= token row) of the chunk
    // In a given order the chunk's steps visit tokens anywhere in the sequence: the buffers then
    // cover the whole sequence and every token row comes from the order.
    const int64_t rbase = kOrd ? static_cast<int64_t>(c.seq) * a.Lp : row0;
    const int64_t eoff = rbase * a.Di;
    const uint32_t rowb = static_cast<uint32_t>(a.Di) * e;           // bytes per token row
    const uint32_t span = static_cast<uint32_t>(kOrd ? a.Lp : len) * rowb;
    const __amdgpu_buffer_rsrc_t rx = chunk_rsrc(static_cast<const E*>(a.x) + eoff, span);
    const __amdgpu_buffer_rsrc_t rd = chunk_rsrc(static_cast<const E*>(a.dt) + eoff, span);
    const __amdgpu_buffer_rsrc_t rz = chunk_rsrc(static_cast<const E*>(a.z) + eoff, span);
    // A wave whose channel block lies past the last one (the spare part of the last workgroup)
    // gets an empty y range: the hardware drops its stores.
    const __amdgpu_buffer_rsrc_t ry = chunk_rsrc(static_cast<E*>(a.y) + eoff, c.cb < a.ncb ? span : 0u);
    const __amdgpu_buffer_rsrc_t rp =
        chunk_rsrc(kGlobalPark ? a.parkg + static_cast<int64_t>(c.slot) * a.T * kWave : nullptr,
                   static_cast<uint32_t>(a.T) * kWave * 4);
    const uint32_t vo = static_cast<uint32_t>(c.dc) * e;
    const uint32_t vp = static_cast<uint32_t>(c.lane) * 4;
    const int last = kend - 1;
    // Local token index of walk step k: k forward, len-1-k backward, as base + sign*k with
    // wave-uniform base and sign. Both directions run this same code: a separate instance per
    // direction puts two different hot loops on every CU and measured much slower.
    const int rdir = kRev ? 1 - c.dir : c.dir;  // the order of the walk
    const int sgn = 1 - 2 * rdir;
    const int tbase = rdir * (len - 1);
    auto lt = [&](int k) { return tbase + sgn * k; };
    // Token row (from rbase) of walk step min(k, last): the step itself, or in a given order the
    // token the order lists for it, read from the chunk's copy of the order in LDS (a broadcast
    // read; no scalar load in the loop) and clamped into the sequence (an order that is not a
    // permutation gives unspecified outputs but no access outside it).
    auto trow = [&](int k) -> int {
        const int st = lt(min(k, last));
        if constexpr (kOrd) return min(max(lds_ord[st], 0), a.Lp - 1);
        else return st;
    };
    auto toff = [&](int k) {  // token row byte offset of walk step min(k, last)
        return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(trow(k))) * rowb;
    };
    auto poff = [&](int k) {  // park byte offset of walk step min(k, last)
        return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(lt(min(k, last)))) * (kWave * 4);
    };

    auto tokoff = [&](int t) { return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(t)) * rowb; };
    // In a given order each step's token is looked up once, when its x and dt are requested, and
    // rides along the rings: tx[s] is the token whose x/dt slot s holds, tz[s] the one whose z
    // slot s holds (its y store offset). At the start of step kbeg + r, slot (r + i) % P of tx
    // holds step kbeg + r + i (i = 1..P-1) and slot r % P step kbeg + r + P.
    uint32_t (&xr)[P] = rg.xr;
    uint32_t (&dr)[P] = rg.dr;
    uint32_t (&zr)[P] = rg.zr;
    uint32_t (&pr)[P] = rg.pr;
    int (&tx)[P] = rg.tx;
    int (&tz)[P] = rg.tz;
    if constexpr (kRing != kRingPrimed) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            uint32_t so;
            if constexpr (kOrd) {
                tx[j] = tz[j] = trow(kbeg + j);
                so = tokoff(tx[j]);
            } else {
                so = toff(kbeg + j);
            }
            xr[j] = ld_raw(IO{}, rx, vo, so);
            dr[j] = ld_raw(IO{}, rd, vo, so);
            if (kMode == kFinish || kMode == kOut) {
                zr[j] = ld_raw(IO{}, rz, vo, so);
                pr[j] = (kMode == kFinish && kGlobalPark)
                            ? __builtin_amdgcn_raw_buffer_load_b32(rp, vp, poff(kbeg + j), 0)
                            : 0u;
            }
        }
    }
    if constexpr (kRing == kRingPrime) return;

    Rates<kDecay> rates;
    rates.load(a.A[c.dir] + c.dc * kN, ln.a0, ln.da);
    float xw[kMaxTaps - 1];  // raw x (widened) of walk steps k-1, k-2, k-3
    if (kConv) {
#pragma unroll
        for (int j = 1; j < kMaxTaps; ++j) {
            const int tok = __builtin_amdgcn_readfirstlane(c.t0 + lt(kbeg - j));  // in the sequence
            xw[j - 1] = (tok >= 0 && tok < a.Lp)
                            ? widen(IO{}, ld_global_raw<IO>(a.x, (static_cast<int64_t>(c.seq) * a.Lp + tok) * a.Di + c.dc))
                            : 0.0f;
        }
    }
    auto input = [&](float xv) -> float {  // this direction's input for token x, window shifted
        if (!kConv) return xv;
        float acc = fmaf(ln.ctap[0], xv, ln.cbias);
#pragma unroll
        for (int j = 1; j < kMaxTaps; ++j) acc = fmaf(ln.ctap[j], xw[j - 1], acc);
#pragma unroll
        for (int j = kMaxTaps - 2; j > 0; --j) xw[j] = xw[j - 1];
        xw[0] = xv;
        return silu(acc);
    };

    // B and C rows come from the chunk's copy in LDS (staged once per workgroup), read as
    // wave-uniform broadcasts at the start of the step that uses them: during step k the C row of
    // token k (its readout) and the B row of token k+1 (its prelude). Nothing is held across a
    // token boundary but the state, the next token's prelude and the register rings.
    float Bn[kN], Cv[kN];
    auto lds_row = [&](const float* rows, int k, float (&v)[kN]) {  // the row of walk step min(k, last)
        const float4* cp = reinterpret_cast<const float4*>(rows + lt(min(k, last)) * kN);
#pragma unroll
        for (int q = 0; q < kN / 4; ++q) {
            const float4 f = cp[q];
            v[4 * q] = f.x;
            v[4 * q + 1] = f.y;
            v[4 * q + 2] = f.z;
            v[4 * q + 3] = f.w;
        }
    };
    Prelude cur;
    if constexpr (kRev) {
        cur = ln.prelude_rev(widen(IO{}, xr[0]), widen(IO{}, dr[0]));
    } else {
        lds_row(lds_b, kbeg, Bn);
        cur = ln.template prelude<kDecay>(input(widen(IO{}, xr[0])), widen(IO{}, dr[0]), Bn, rates);
    }
    {
        uint32_t so;
        if constexpr (kOrd) {
            tx[0] = trow(kbeg + P);
            so = tokoff(tx[0]);
        } else {
            so = toff(kbeg + P);
        }
        xr[0] = ld_raw(IO{}, rx, vo, so);
        dr[0] = ld_raw(IO{}, rd, vo, so);
    }
    // In a given order the token of each refill is read from LDS a step before the refill that
    // uses it, so the lookup's latency is not on the path of the step's loads.
    int tla = kOrd ? trow(kbeg + 1 + P) : 0;

    auto body = [&](int kk, int j) {  // step kk, ring slot j = (kk - kbeg) % P
        const int jn = (j + 1) % P;
        const int tl = lt(kk);
        if (kReadout) lds_row(lds_c, kk, Cv);  // this token's C row
        lds_row(lds_b, kRev ? kk : kk + 1, Bn);  // next token's B row for its prelude (kRev: this token's)
        // Consume the ring slots before refilling them: the empty asm takes the widened values
        // and orders every load after it, so a refill can reuse its slot's register and the loop
        // needs no register copies (a copy would wait for the load just issued).
        const float xn = widen(IO{}, xr[jn]), dn = widen(IO{}, dr[jn]);
        float zv = 0.0f, pv = 0.0f;
        if (kMode == kFinish || kMode == kOut) {
            zv = widen(IO{}, zr[j]);
            pv = __uint_as_float(pr[j]);
        }
        asm volatile("" ::"v"(xn), "v"(dn), "v"(zv), "v"(pv) : "memory");
        {
            uint32_t so;
            if constexpr (kOrd) {
                tx[jn] = tla;  // step kk + 1 + P, looked up during the previous step
                so = tokoff(tx[jn]);
                tla = trow(kk + 2 + P);
            } else {
                so = toff(kk + 1 + P);
            }
            xr[jn] = ld_raw(IO{}, rx, vo, so);
            dr[jn] = ld_raw(IO{}, rd, vo, so);
        }
        int ytok = 0;  // kOrd: this step's token (its y store)
        if (kMode == kFinish || kMode == kOut) {
            uint32_t so;
            if constexpr (kOrd) {
                ytok = tz[j];
                tz[j] = tx[j];  // step kk + P
                so = tokoff(tz[j]);
            } else {
                so = toff(kk + P);
            }
            zr[j] = ld_raw(IO{}, rz, vo, so);
            if (kMode == kFinish && kGlobalPark) pr[j] = __builtin_amdgcn_raw_buffer_load_b32(rp, vp, poff(kk + P), 0);
        }
        Prelude nxt;  // next token's prelude
        if constexpr (kRev) nxt = ln.prelude_rev(xn, dn);
        else nxt = ln.template prelude<kDecay>(input(xn), dn, Bn, rates);
        if (kMode == kAggregate) dsum += cur.delta2;
        float yv = 0.0f;
        if constexpr (kRev) {
            ln.template update_rev<kDecay>(cur, Bn, rates, dsum);  // dsum: the suffix sum S so far
            dsum += cur.delta2;
        } else {
            yv = ln.template update<kReadout>(cur, Cv);
        }
        if (kConv && kReadout) yv = fmaf(ln.Dd, cur.x, yv);  // own skip term on own input u
        if (kMode == kPark) {
            if (kGlobalPark)
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(yv), rp, vp,
                                                      static_cast<uint32_t>(tl) * (kWave * 4), 0);
            else
                lds_park[tl * kWave + c.lane] = yv;
        }
        if (kMode == kFinish) {
            const float other = kGlobalPark ? pv : lds_park[tl * kWave + c.lane];
            // No branch on c.valid: a lane past d_inner in the last block runs channel
            // d_inner-1 on the same inputs and parameters, in the same wave (so with the same
            // transition form), and stores the same bits to the same element. Without the branch
            // the readout stays in the token's single basic block, where it interleaves with the
            // next token's prelude.
            const float ysum = kConv ? yv + other : fmaf(ln.Dsum, cur.x, yv + other);
            st_buf(IO{}, ry, vo, kOrd ? tokoff(ytok) : static_cast<uint32_t>(tl) * rowb, silu(zv) * ysum);
        }
        if (kMode == kOut)
            st_buf(IO{}, ry, vo, kOrd ? tokoff(ytok) : static_cast<uint32_t>(tl) * rowb,
                   silu(zv) * (kConv ? yv : fmaf(ln.Dd, cur.x, yv)));
        cur = nxt;
        // Token boundary: no instruction moves across it. Within a token the next prelude and
        // this update interleave freely; across tokens the scheduler would hoist preludes ahead
        // of the loads they wait for.
        __builtin_amdgcn_sched_barrier(0);
    };

    constexpr int U = P;  // steps per loop iteration: the ring depth (ring slots are compile-time indices)
    int k = kbeg;
    for (; k + U <= kend; k += U) {
#pragma unroll
        for (int j = 0; j < U; ++j) body(k + j, j % P);
    }
#pragma unroll
    for (int j = 0; j < U - 1; ++j)
        if (k + j < kend) body(k + j, j % P);
}

// The walk instance for this wave's transition form (wave-uniform).
template <typename IO, int kMode, bool kGlobalPark, int kVar, int kRing = kRingFull>
__device__ __forceinline__ void walk_as(int form, const ScanArgs& a, const WgCoords& c, Lane& ln, float* lds_park,
                                        const float* lds_c, const float* lds_b, const int32_t* lds_ord, int kbeg,
                                        int kend, float& dsum, Ring<ring_depth(kVar)>& rg) {
    if (form == kGeometric)
        walk<IO, kGeometric, kMode, kGlobalPark, kVar, kRing>(a, c, ln, lds_park, lds_c, lds_b, lds_ord, kbeg, kend,
                                                              dsum, rg);
    else if (form == kProgression)
        walk<IO, kProgression, kMode, kGlobalPark, kVar, kRing>(a, c, ln, lds_park, lds_c, lds_b, lds_ord, kbeg, kend,
                                                                dsum, rg);
    else
        walk<IO, kGeneral, kMode, kGlobalPark, kVar, kRing>(a, c, ln, lds_park, lds_c, lds_b, lds_ord, kbeg, kend,
                                                            dsum, rg);
}

// Issue the ring loads of a walk that starts at step kbeg (not in a given order).
template <typename IO, int kMode, bool kGlobalPark, int kVar>
__device__ __forceinline__ void prime_ring(const ScanArgs& a, const WgCoords& c, Lane& ln, int kbeg, int kend,
                                           Ring<ring_depth(kVar)>& rg) {
    float unused = 0.0f;
    walk<IO, kGeneral, kMode, kGlobalPark, kVar, kRingPrime>(a, c, ln, nullptr, nullptr, nullptr, nullptr, kbeg, kend,
                                                             unused, rg);
}

// Copy the chunk's rows into LDS as fp32: regions [C forward, C backward, B forward, B backward]
// of [T][16] each (forward only: [C, B]), C times ln 2 (the state is kept in log2 units), B as
// given; with withC false only the B regions, from region 0. Every row a walk reads then comes
// from LDS, so its waits never include a scalar load (those complete out of order, and a wait for
// one waits for every scalar load in flight). Each (matrix, direction) is one contiguous range of
// 32-bit words in memory; every thread issues all its loads before widening and storing, so the
// copy costs one memory round trip.
// Region reg of the staged rows (0 C forward, 1 C backward, 2 B forward, 3 B backward; forward
// only: 0 C, 1 B), chosen with selects (no run-time index into the kernel arguments).
__device__ __forceinline__ const void* region_rows(const ScanArgs& a, int reg, int ndir) {
    if (ndir == 1) return reg == 0 ? a.Cm[0] : a.Bm[0];
    return reg == 0 ? a.Cm[0] : reg == 1 ? a.Cm[1] : reg == 2 ? a.Bm[0] : a.Bm[1];
}

template <typename IO>
__device__ __forceinline__ void stage_rows(const ScanArgs& a, const WgCoords& c, float* lds, bool uni, bool withC) {
    constexpr int kU = IoTraits<IO>::bytes == 2 ? 7 : 4;       // words per region per thread and pass
    constexpr int kPerWord = 4 / IoTraits<IO>::bytes;          // values per 32-bit word
    using El = typename IoTraits<IO>::elem;
    const int len = c.t1 - c.t0;
    const int64_t off = (static_cast<int64_t>(c.seq) * a.Lp + c.t0) * kN;
    const int wpd = len * kN / kPerWord;                       // words per region
    const int ndir = uni ? 1 : 2;
    const int first = withC ? 0 : ndir;                        // first region: C forward, or B forward
    const int nreg = 2 * ndir - first;                         // regions staged (wave-uniform, 1..4)
    const uint32_t* src[4];                                    // their rows in memory
    float sc[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int reg = min(first + r, 2 * ndir - 1);
        src[r] = reinterpret_cast<const uint32_t*>(static_cast<const El*>(region_rows(a, reg, ndir)) + off);
        sc[r] = reg < ndir ? kLn2 : 1.0f;
    }
    const int nt = static_cast<int>(blockDim.x);
    // a pass moves the same kU word indices of every region: all loads are issued before any store
    for (int base = static_cast<int>(threadIdx.x); base < wpd; base += kU * nt) {
        uint32_t w[4][kU];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int i = base + u * nt;
                w[r][u] = (r < nreg && i < wpd) ? src[r][i] : 0u;
            }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int i = base + u * nt;
                if (r < nreg && i < wpd) {
                    float* dst = lds + r * a.T * kN + i * kPerWord;
                    if (kPerWord == 1) {
                        dst[0] = __uint_as_float(w[r][u]) * sc[r];
                    } else {
                        dst[0] = __uint_as_float(w[r][u] << 16) * sc[r];
                        dst[1] = __uint_as_float(w[r][u] & 0xffff0000u) * sc[r];
                    }
                }
            }
    }
}


// The C rows of both directions in registers (one pass of stage_rows' layout), for k_bidir_chain:
// loaded with the B rows and stored into LDS only after the aggregate walk, which reads B alone,
// so the walk starts after half the staging (high-res 63.2 -> 60.7 us per call).
template <typename IO>
struct CWords {
    static constexpr int kU = IoTraits<IO>::bytes == 2 ? 7 : 4;
    uint32_t w[2][kU];
};
template <typename IO>
__device__ __forceinline__ bool c_fits_one_pass(const ScanArgs& a, const WgCoords& c) {
    constexpr int kPerWord = 4 / IoTraits<IO>::bytes;
    const int len = c.t1 - c.t0;
    return len * kN / kPerWord <= CWords<IO>::kU * static_cast<int>(blockDim.x);
}
template <typename IO>
__device__ __forceinline__ void load_c_words(const ScanArgs& a, const WgCoords& c, CWords<IO>& cw) {
    constexpr int kU = CWords<IO>::kU;
    constexpr int kPerWord = 4 / IoTraits<IO>::bytes;
    using El = typename IoTraits<IO>::elem;
    const int len = c.t1 - c.t0;
    const int64_t off = (static_cast<int64_t>(c.seq) * a.Lp + c.t0) * kN;
    const int wpd = len * kN / kPerWord;
    const int nt = static_cast<int>(blockDim.x);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const El*>(a.Cm[r]) + off);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = static_cast<int>(threadIdx.x) + u * nt;
            cw.w[r][u] = i < wpd ? src[i] : 0u;
        }
    }
}
template <typename IO>
__device__ __forceinline__ void store_c_words(const ScanArgs& a, const WgCoords& c, float* lds, const CWords<IO>& cw) {
    constexpr int kU = CWords<IO>::kU;
    constexpr int kPerWord = 4 / IoTraits<IO>::bytes;
    const int len = c.t1 - c.t0;
    const int wpd = len * kN / kPerWord;
    const int nt = static_cast<int>(blockDim.x);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = static_cast<int>(threadIdx.x) + u * nt;
            if (i < wpd) {
                float* dst = lds + r * a.T * kN + i * kPerWord;
                if (kPerWord == 1) {
                    dst[0] = __uint_as_float(cw.w[r][u]) * kLn2;
                } else {
                    dst[0] = __uint_as_float(cw.w[r][u] << 16) * kLn2;
                    dst[1] = __uint_as_float(cw.w[r][u] & 0xffff0000u) * kLn2;
                }
            }
        }
}

// The same for a scan in a given order (both directions, C and B): the chunk's rows are gathered
// in step order (row k of a region is the row of the token the order lists for step t0 + k), so
// the walk reads them exactly as in raster order, and the chunk's order entries are copied after
// the rows (the walk's token lookups then read LDS). One thread per step: one lookup in the
// order, then the words of that token's row in every region as independent loads, so a chunk of
// up to blockDim.x steps costs two dependent memory round trips.
template <typename IO>
__device__ __forceinline__ void stage_rows_ordered(const ScanArgs& a, const WgCoords& c, float* lds, bool withC) {
    constexpr int kPerWord = 4 / IoTraits<IO>::bytes;
    constexpr int wpr = kN / kPerWord;  // words per row
    using El = typename IoTraits<IO>::elem;
    const int len = c.t1 - c.t0;
    const int64_t srow = static_cast<int64_t>(c.seq) * a.Lp;
    const int32_t* ord = a.order + srow + c.t0;
    const int first = withC ? 0 : 2;
    const int nreg = 4 - first;  // regions staged (wave-uniform)
    int32_t* lds_ord = reinterpret_cast<int32_t*>(lds + nreg * a.T * kN);  // after the rows
    for (int k = static_cast<int>(threadIdx.x); k < len; k += static_cast<int>(blockDim.x)) {
        const int32_t o = ord[k];
        lds_ord[k] = o;
        const int tok = min(max(static_cast<int>(o), 0), a.Lp - 1);
        uint32_t w[4][wpr];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (r < nreg) {
                const uint32_t* src = reinterpret_cast<const uint32_t*>(
                    static_cast<const El*>(region_rows(a, first + r, 2)) + (srow + tok) * kN);
#pragma unroll
                for (int q = 0; q < wpr; ++q) w[r][q] = src[q];
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (r < nreg) {
                const float sc = first + r < 2 ? kLn2 : 1.0f;
                float* dst = lds + r * a.T * kN + k * kN;
#pragma unroll
                for (int q = 0; q < wpr; ++q) {
                    if (kPerWord == 1) {
                        dst[q] = __uint_as_float(w[r][q]) * sc;
                    } else {
                        dst[2 * q] = __uint_as_float(w[r][q] << 16) * sc;
                        dst[2 * q + 1] = __uint_as_float(w[r][q] & 0xffff0000u) * sc;
                    }
                }
            }
        }
    }
}

// Main scan: one chunk of one sequence, 64 channels; wave 0 forward, wave 1 backward. The waves
// meet in the middle of the chunk through the park (LDS, or a global scratch region per
// workgroup when the chunk is long; see the file header).
// The state entering chunk `chunk` of direction dir, for the lane's channel dc (an = its A row): the chunk
// aggregates of the chunks before it in scan order folded in the carry combine's order and
// arithmetic (so bit for bit the combine's result). The loads go kFoldBatch chunks at a time, all
// issued together, clamped to a chunk whose aggregate exists; only the first cnt enter the fold.
// The aggregates are written by other workgroups of the same kernel (k_bidir_chain,
// k_fwd_chain): every load is a device-coherent one (an agent-scope atomic load), issued after
// wait_published.
__device__ __forceinline__ void fold_carry(const ScanArgs& a, int dir, int seq, int chunk, int dc, const float (&an)[kN],
                                           float (&h)[kN]) {
    auto ld = [](const float* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    const int64_t base = (static_cast<int64_t>(dir) * a.nseq + seq) * a.K;
    const int cnt = dir == 0 ? chunk : a.K - 1 - chunk;  // chunks before this one in scan order
#pragma unroll
    for (int n = 0; n < kN; ++n) h[n] = 0.0f;
    for (int j0 = 0; j0 < cnt; j0 += kFoldBatch) {
        float e[kFoldBatch][kN], sv[kFoldBatch];
#pragma unroll
        for (int j = 0; j < kFoldBatch; ++j) {
            const int k = dir == 0 ? min(j0 + j, a.K - 2) : max(a.K - 1 - j0 - j, 1);
            const int64_t slot = base + k;
            sv[j] = ld(a.dsum + slot * a.Di + dc);
#pragma unroll
            for (int n = 0; n < kN; ++n) e[j][n] = ld(a.carry + (slot * kN + n) * a.Di + dc);
        }
#pragma unroll
        for (int j = 0; j < kFoldBatch; ++j)
            if (j0 + j < cnt) {
#pragma unroll
                for (int n = 0; n < kN; ++n) h[n] = fmaf(fast_exp2(an[n] * sv[j]), h[n], e[j][n]);
            }
    }
}

template <typename IO, bool kCarry, bool kGlobalPark, int kVar>
__global__ __launch_bounds__(256) void k_bidir_scan(ScanArgs a) {
    constexpr bool kConv = kVar == kWithConv;
    // LDS: C and B rows [4][T][16]; in a given order the chunk's order [T]; the park [subs][T][64]
    // when in LDS
    extern __shared__ float lds[];
    const WgCoords c = wg_coords(a, false);
    const float* lds_c = lds + c.dir * a.T * kN;
    const float* lds_b = lds + (2 + c.dir) * a.T * kN;
    const int32_t* lds_ord = reinterpret_cast<const int32_t*>(lds + 4 * a.T * kN);
    float* lds_park = lds + 4 * a.T * kN + (kVar == kOrdered ? a.T : 0) + c.sub * a.T * kWave;
    const int len = c.t1 - c.t0;
    const int half = len >> 1;
    const int n1 = c.dir == 0 ? half : len - half;  // tokens this wave parks before the barrier
    Lane ln;
    ln.init(a, c.dir, c.dc, kConv);
    if (kConv) ln.init_conv(a, c.dir, c.dc);
    // Loads that need neither the staged rows nor one another are issued before the staging, so
    // their latency overlaps it: the first walk's rings (in raster order; a given order's tokens
    // come from the staged copy) and the A row of the transition-form vote.
    constexpr bool kPrime = kVar != kOrdered;
    Ring<ring_depth(kVar)> rg;
    if constexpr (kPrime) prime_ring<IO, kPark, kGlobalPark, kVar>(a, c, ln, 0, n1, rg);
    const Lane::ARow arow = ln.load_arow(a, c.dir, c.dc);
    if constexpr (kVar == kOrdered) stage_rows_ordered<IO>(a, c, lds, true);
    else stage_rows<IO>(a, c, lds, false, true);
    if (kCarry) {
        const float* src = a.carry + ((static_cast<int64_t>(c.dir) * a.nseq + c.seq) * a.K + c.chunk) * kN * a.Di;
#pragma unroll
        for (int n = 0; n < kN; ++n) ln.h[n] = src[n * static_cast<int64_t>(a.Di) + c.dc];
    } else {
#pragma unroll
        for (int n = 0; n < kN; ++n) ln.h[n] = 0.0f;
    }
    const int form = ln.decay_form(a, arow);
    float unused = 0.0f;
    __syncthreads();  // the rows are staged
    walk_as<IO, kPark, kGlobalPark, kVar, kPrime ? kRingPrimed : kRingFull>(form, a, c, ln, lds_park, lds_c, lds_b,
                                                                              lds_ord, 0, n1, unused, rg);
    __syncthreads();  // the park is complete (the barrier also orders the global park's stores)
    walk_as<IO, kFinish, kGlobalPark, kVar>(form, a, c, ln, lds_park, lds_c, lds_b, lds_ord, n1, len, unused, rg);
}

// Forward-only scan (vimscan_fwd): one chunk of one sequence, every wave a channel block of 64,
// all walking forward; each token is gated and stored at once (no park, no meeting point).
template <typename IO, bool kCarry>
__global__ __launch_bounds__(256) void k_fwd_scan(ScanArgs a) {
    extern __shared__ float lds[];  // the chunk's C rows [T][16], then its B rows [T][16]
    const WgCoords c = wg_coords(a, true);
    const int len = c.t1 - c.t0;
    Lane ln;
    ln.init(a, 0, c.dc, true);
    // the first walk's rings and the vote's A row go out before the staging (see k_bidir_scan)
    Ring<ring_depth(kPlain)> rg;
    prime_ring<IO, kOut, false, kPlain>(a, c, ln, 0, len, rg);
    const Lane::ARow arow = ln.load_arow(a, 0, c.dc);
    stage_rows<IO>(a, c, lds, true, true);
    if (kCarry) {
        const float* src = a.carry + (static_cast<int64_t>(c.seq) * a.K + c.chunk) * kN * a.Di;
#pragma unroll
        for (int n = 0; n < kN; ++n) ln.h[n] = src[n * static_cast<int64_t>(a.Di) + c.dc];
    } else {
#pragma unroll
        for (int n = 0; n < kN; ++n) ln.h[n] = 0.0f;
    }
    const int form = ln.decay_form(a, arow);
    float unused = 0.0f;
    __syncthreads();  // the rows are staged
    walk_as<IO, kOut, false, kPlain, kRingPrimed>(form, a, c, ln, nullptr, lds, lds + a.T * kN, nullptr, 0, len,
                                                  unused, rg);
}

// Pass 1 of the chunked scan: per chunk and direction, the end state of the chunk's local scan
// from a zero state, and the sum of delta over the chunk. The walk goes against the scan order
// (Lane::update_rev), except with the convolution, whose input window follows the scan order.
template <typename IO, int kVar>
__global__ __launch_bounds__(256) void k_chunk_aggregate(ScanArgs a) {
    constexpr bool kConv = kVar == kWithConv;
    constexpr int kAggMode = kConv ? kAggregate : kAggRev;
    extern __shared__ float lds[];  // the chunk's B rows [directions][T][16]; in a given order then the order [T]
    const WgCoords c = wg_coords(a, a.uni != 0);
    // The state after the last chunk in scan order (forward: the last chunk, backward: the first)
    // is never used, so that chunk's aggregate is not computed: its wave only helps stage the rows
    // and leaves after the barrier.
    const bool unused_chunk = c.chunk == (c.dir == 0 ? a.K - 1 : 0);
    const int len = c.t1 - c.t0;
    Lane ln;
    ln.init(a, c.dir, c.dc, false);
    if (kConv) ln.init_conv(a, c.dir, c.dc);
    // the walk's rings and the vote's A row go out before the staging (see k_bidir_scan)
    constexpr bool kPrime = kVar != kOrdered;
    Ring<ring_depth(kVar)> rg;
    if constexpr (kPrime) {
        if (!unused_chunk) prime_ring<IO, kAggMode, false, kVar>(a, c, ln, 0, len, rg);
    }
    const Lane::ARow arow = ln.load_arow(a, c.dir, c.dc);
    if constexpr (kVar == kOrdered) stage_rows_ordered<IO>(a, c, lds, false);
    else stage_rows<IO>(a, c, lds, a.uni != 0, false);
    __syncthreads();  // the rows are staged
    if (unused_chunk) return;  // no barrier follows
#pragma unroll
    for (int n = 0; n < kN; ++n) ln.h[n] = 0.0f;
    const int form = ln.decay_form(a, arow);
    float s = 0.0f;
    walk_as<IO, kAggMode, false, kVar, kPrime ? kRingPrimed : kRingFull>(
        form, a, c, ln, nullptr, nullptr, lds + c.dir * a.T * kN, reinterpret_cast<const int32_t*>(lds + 2 * a.T * kN),
        0, len, s, rg);
    if (c.valid) {
        const int64_t slot = (static_cast<int64_t>(c.dir) * a.nseq + c.seq) * a.K + c.chunk;
        float* dst = a.carry + slot * kN * a.Di;
#pragma unroll
        for (int n = 0; n < kN; ++n) dst[n * static_cast<int64_t>(a.Di) + c.d] = ln.h[n];
        a.dsum[slot * a.Di + c.d] = s;
    }
}

// One-pass chunked scan: the aggregate pass, the fold and the scan of k_chunk_aggregate and
// k_bidir_scan in one kernel, chunks handing their aggregates to the other chunks of their
// sequence through the workspace. Each workgroup stages its chunk's rows once, computes the
// aggregate of its chunk in both directions (the state after the chunk from a zero state, walked
// against the scan order as in k_chunk_aggregate), publishes it, waits until every chunk before it
// in scan order has published, folds those aggregates (fold_carry) and runs the scan from the
// folded state.
//
// Publication: a wave stores its aggregate and delta sum with device-coherent stores (agent-scope
// atomic stores, written through to where every XCD reads them), waits until all of them have
// completed, and only then stores the dispatch's tag in its tag word; a waiting wave reads the
// tag words of the aggregates it needs until all hold the tag, and only then issues its
// device-coherent loads of the aggregates. Both sides order their accesses by waiting for
// completion, not with agent-scope fences: such a fence writes back or invalidates the whole L2
// of the XCD, and with thousands of waves publishing that serialises the kernel (it measured
// several times slower than the two kernels it replaces). The tag is unique to the kernel dispatch (its
// packet index in its queue, mixed with the queue's address), so tag words left by earlier calls
// or holding arbitrary bytes never match it: the workspace needs no clearing between calls and no
// initial contents.
//
// Progress: a chunk waits only for the other chunks of its (sequence, channel-block group), whose
// workgroups have the neighbouring ids (wg_coords<true>), and it publishes before it waits. The
// hardware starts the workgroups of each XCD in increasing id order, so the chunks of the lowest
// group not yet complete are the first ones waiting on their XCDs; with room for at least
// kFoldMaxChunks workgroups per XCD (32 CUs, at least one workgroup each) all of them run at once
// and complete, and so on group by group. The wait is bounded all the same (kSpinLimit reads,
// about a second): past it the wave goes on, its output is unspecified, and it counts itself in
// g_wait_timeouts (vimscan_wait_timeouts).
// Waits of the one-kernel chunked scans on this GPU that ran past kSpinLimit since the library was
// loaded (none is expected: see the progress argument above).
__device__ unsigned long long g_wait_timeouts;

// The tag word of the aggregate of (dir, seq, chunk) for channel block cb.
__device__ __forceinline__ uint64_t* tag_word(const ScanArgs& a, int dir, int seq, int chunk, int cb) {
    return a.tags + ((static_cast<int64_t>(dir) * a.nseq + seq) * a.K + chunk) * a.ncb + cb;
}

// Wait until the aggregates of the chunks before `chunk` in scan order (for this wave's direction
// and channel block) are published: lane j reads the tag word of the j-th of them (at most
// kFoldMaxChunks - 1 < 64).
__device__ __forceinline__ void wait_published(const ScanArgs& a, const WgCoords& c, uint64_t tag) {
    const int cnt = c.dir == 0 ? c.chunk : a.K - 1 - c.chunk;
    if (cnt == 0) return;
    const bool mine = c.lane < cnt;
    const int k = mine ? (c.dir == 0 ? c.lane : a.K - 1 - c.lane) : c.chunk;
    const uint64_t* w = tag_word(a, c.dir, c.seq, k, c.cb);
    bool done = false;
    for (int it = 0; it < kSpinLimit && !done; ++it) {
        const bool ready = !mine || __hip_atomic_load(w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == tag;
        done = __all(ready);
        if (!done) __builtin_amdgcn_s_sleep(2);
    }
    if (!done && c.lane == 0)
        __hip_atomic_fetch_add(&g_wait_timeouts, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("" ::: "memory");  // the aggregate loads stay after the wait
}

template <typename IO, bool kGlobalPark, int kVar>
__global__ __launch_bounds__(256) void k_bidir_chain(ScanArgs a) {
    constexpr bool kConv = kVar == kWithConv;
    constexpr int kAggMode = kConv ? kAggregate : kAggRev;
    constexpr bool kPrime = kVar != kOrdered;
    // LDS as k_bidir_scan: C and B rows [4][T][16]; in a given order the chunk's order [T]; the
    // park [subs][T][64] when in LDS
    extern __shared__ float lds[];
    const WgCoords c = wg_coords<true>(a, false);
    const float* lds_c = lds + c.dir * a.T * kN;
    const float* lds_b = lds + (2 + c.dir) * a.T * kN;
    const int32_t* lds_ord = reinterpret_cast<const int32_t*>(lds + 4 * a.T * kN);
    float* lds_park = lds + 4 * a.T * kN + (kVar == kOrdered ? a.T : 0) + c.sub * a.T * kWave;
    const int len = c.t1 - c.t0;
    const int half = len >> 1;
    const int n1 = c.dir == 0 ? half : len - half;  // tokens this wave parks before the barrier
    // This wave's aggregate is used unless its chunk is the last in scan order; a wave past the
    // last channel block neither publishes nor waits.
    const bool live = c.cb < a.ncb;
    const bool publishes = live && c.chunk != (c.dir == 0 ? a.K - 1 : 0);
    const uint64_t tag = dispatch_tag();
    Lane ln;
    ln.init(a, c.dir, c.dc, kConv);
    if (kConv) ln.init_conv(a, c.dir, c.dc);
    Ring<ring_depth(kVar)> rg;
    if constexpr (kPrime) {
        if (publishes) prime_ring<IO, kAggMode, false, kVar>(a, c, ln, 0, len, rg);
    }
    int form;
    CWords<IO> cw;
    const bool late_c = kVar != kOrdered && c_fits_one_pass<IO>(a, c);
    {
        const Lane::ARow arow = ln.load_arow(a, c.dir, c.dc);
        if constexpr (kVar == kOrdered) {
            stage_rows_ordered<IO>(a, c, lds, true);
        } else if (late_c) {
            load_c_words<IO>(a, c, cw);
            stage_rows<IO>(a, c, lds + 2 * a.T * kN, false, false);
        } else {
            stage_rows<IO>(a, c, lds, false, true);
        }
        form = ln.decay_form(a, arow);
    }
    __syncthreads();  // the rows are staged (the C rows later when late_c)
    if (publishes) {
#pragma unroll
        for (int n = 0; n < kN; ++n) ln.h[n] = 0.0f;
        float s = 0.0f;
        walk_as<IO, kAggMode, false, kVar, kPrime ? kRingPrimed : kRingFull>(form, a, c, ln, nullptr, nullptr, lds_b,
                                                                            lds_ord, 0, len, s, rg);
        if (c.valid) {
            const int64_t slot = (static_cast<int64_t>(c.dir) * a.nseq + c.seq) * a.K + c.chunk;
            float* dst = a.carry + slot * kN * a.Di;
#pragma unroll
            for (int n = 0; n < kN; ++n)
                __hip_atomic_store(dst + n * static_cast<int64_t>(a.Di) + c.d, ln.h[n], __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(a.dsum + slot * a.Di + c.d, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // every store above has completed
        if (c.lane == 0)
            __hip_atomic_store(tag_word(a, c.dir, c.seq, c.chunk, c.cb), tag, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    if (kVar != kOrdered && late_c) {
        store_c_words<IO>(a, c, lds, cw);
        __syncthreads();  // the C rows are staged
    }
    if constexpr (kPrime) prime_ring<IO, kPark, kGlobalPark, kVar>(a, c, ln, 0, n1, rg);
    if (live) {
        wait_published(a, c, tag);
        const Lane::ARow arow = ln.load_arow(a, c.dir, c.dc);
        fold_carry(a, c.dir, c.seq, c.chunk, c.dc, arow.r, ln.h);
    } else {
#pragma unroll
        for (int n = 0; n < kN; ++n) ln.h[n] = 0.0f;
    }
    float unused = 0.0f;
    walk_as<IO, kPark, kGlobalPark, kVar, kPrime ? kRingPrimed : kRingFull>(form, a, c, ln, lds_park, lds_c, lds_b,
                                                                              lds_ord, 0, n1, unused, rg);
    __syncthreads();  // the park is complete (the barrier also orders the global park's stores)
    walk_as<IO, kFinish, kGlobalPark, kVar>(form, a, c, ln, lds_park, lds_c, lds_b, lds_ord, n1, len, unused, rg);
}

// Forward-only one-pass chunked scan (vimscan_fwd with 2..kFoldMaxChunks chunks): k_bidir_chain's
// aggregate walk, hand-over and fold in front of k_fwd_scan's walk; every wave a channel block.
template <typename IO>
__global__ __launch_bounds__(256) void k_fwd_chain(ScanArgs a) {
    extern __shared__ float lds[];  // the chunk's C rows [T][16], then its B rows [T][16]
    const WgCoords c = wg_coords<true>(a, true);
    const int len = c.t1 - c.t0;
    const bool live = c.cb < a.ncb;
    const bool publishes = live && c.chunk != a.K - 1;
    const uint64_t tag = dispatch_tag();
    Lane ln;
    ln.init(a, 0, c.dc, true);
    Ring<ring_depth(kPlain)> rg;
    if (publishes) prime_ring<IO, kAggRev, false, kPlain>(a, c, ln, 0, len, rg);
    int form;
    {
        const Lane::ARow arow = ln.load_arow(a, 0, c.dc);
        stage_rows<IO>(a, c, lds, true, true);
        form = ln.decay_form(a, arow);
    }
    __syncthreads();  // the rows are staged
    if (publishes) {
#pragma unroll
        for (int n = 0; n < kN; ++n) ln.h[n] = 0.0f;
        float s = 0.0f;
        walk_as<IO, kAggRev, false, kPlain, kRingPrimed>(form, a, c, ln, nullptr, nullptr, lds + a.T * kN, nullptr, 0,
                                                        len, s, rg);
        if (c.valid) {
            const int64_t slot = static_cast<int64_t>(c.seq) * a.K + c.chunk;
            float* dst = a.carry + slot * kN * a.Di;
#pragma unroll
            for (int n = 0; n < kN; ++n)
                __hip_atomic_store(dst + n * static_cast<int64_t>(a.Di) + c.d, ln.h[n], __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
            __hip_atomic_store(a.dsum + slot * a.Di + c.d, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // every store above has completed
        if (c.lane == 0)
            __hip_atomic_store(tag_word(a, 0, c.seq, c.chunk, c.cb), tag, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    prime_ring<IO, kOut, false, kPlain>(a, c, ln, 0, len, rg);
    if (live) {
        wait_published(a, c, tag);
        const Lane::ARow arow = ln.load_arow(a, 0, c.dc);
        fold_carry(a, 0, c.seq, c.chunk, c.dc, arow.r, ln.h);
    } else {
#pragma unroll
        for (int n = 0; n < kN; ++n) ln.h[n] = 0.0f;
    }
    float unused = 0.0f;
    walk_as<IO, kOut, false, kPlain, kRingPrimed>(form, a, c, ln, nullptr, lds, lds + a.T * kN, nullptr, 0, len,
                                                  unused, rg);
}

// Carry combine: for each (direction, sequence, state n, channel) fold the chunk aggregates in
// scan order; carry[chunk] is replaced by the state entering that chunk. The fold is the
// associative operator of the linear recurrence: (P1, e1) then (P2, e2) -> (P1 P2, P2 e1 + e2),
// with P = exp(A * sum delta) the chunk's transition product.
// Block: 256 threads = 64 channels x 4 states; grid (channel blocks x directions x sequences, 4)
// with the channel block fastest in x (x holds the large count: y and z are limited to 65535).
__global__ __launch_bounds__(256) void k_carry_combine(ScanArgs a) {
    const int bx = static_cast<int>(blockIdx.x);
    const int zz = bx / a.ncb;  // direction + 2 * sequence, or the sequence forward only
    const int d = (bx % a.ncb) * kWave + (static_cast<int>(threadIdx.x) & (kWave - 1));
    const int n = static_cast<int>(blockIdx.y) * 4 + (static_cast<int>(threadIdx.x) >> 6);
    const int dir = a.uni ? 0 : zz & 1;
    const int seq = a.uni ? zz : zz >> 1;
    if (d >= a.Di) return;
    const float an = a.A[dir][d * kN + n];
    const int64_t base = (static_cast<int64_t>(dir) * a.nseq + seq) * a.K;
    // Aggregates are read kB chunks at a time before any store (stores into the same workspace
    // would otherwise order every load after the previous store: one memory round trip per chunk).
    // The last chunk in scan order has no aggregate (its end state is never used): loads past the
    // second-to-last chunk are clamped to it, and the value is not used.
    constexpr int kB = 16;
    float H = 0.0f;
    for (int k0 = 0; k0 < a.K; k0 += kB) {
        float ev[kB], sv[kB];
#pragma unroll
        for (int j = 0; j < kB; ++j) {
            const int k = min(k0 + j, a.K - 2);  // K >= 2 when the combine runs
            const int64_t slot = base + (dir == 0 ? k : a.K - 1 - k);
            ev[j] = a.carry[(slot * kN + n) * a.Di + d];
            sv[j] = a.dsum[slot * a.Di + d];
        }
#pragma unroll
        for (int j = 0; j < kB; ++j) {
            const int k = k0 + j;
            if (k < a.K) {
                const int64_t slot = base + (dir == 0 ? k : a.K - 1 - k);
                a.carry[(slot * kN + n) * a.Di + d] = H;  // the state entering chunk k
                H = fmaf(fast_exp2(an * sv[j]), H, ev[j]);
            }
        }
    }
}

// Auxiliary-token swap after the scan (VIMSCAN_FLAG_AUX_SWAP): exchange the first and the last
// row of y in every sequence (segment). One thread per (sequence, channel); a 1-D grid of
// (channel group of 256) x sequences, channel group fastest.
template <typename IO>
__global__ __launch_bounds__(256) void k_aux_swap(ScanArgs a) {
    using E = typename IoTraits<IO>::elem;
    const int groups = (a.Di + 255) / 256;
    const int seq = static_cast<int>(blockIdx.x) / groups;
    const int d = (static_cast<int>(blockIdx.x) % groups) * 256 + static_cast<int>(threadIdx.x);
    if (d >= a.Di || a.Lp < 2) return;
    E* y = static_cast<E*>(a.y);
    const int64_t first = static_cast<int64_t>(seq) * a.Lp * a.Di + d;
    const int64_t last = first + static_cast<int64_t>(a.Lp - 1) * a.Di;
    const E v0 = y[first];
    y[first] = y[last];
    y[last] = v0;
}

// ------------------------------------------------------------------------------------------
// Host side

// Threads per workgroup: two waves (forward, backward) per channel block, or one forward only.
unsigned wg_threads(const Plan& p) { return static_cast<unsigned>((p.uni ? 64 : 128) * p.subs); }

template <typename IO, bool kGlobalPark, int kVar>
void launch_scan(const ScanArgs& a, const Plan& p, hipStream_t s, bool carry) {
    const dim3 grid(static_cast<unsigned>(p.wgs)), block(wg_threads(p));
    const size_t lds =
        (4 * p.T * kN + (kVar == kOrdered ? p.T : 0) + (kGlobalPark ? 0 : p.subs * p.T * kWave)) * sizeof(float);
    if (carry) hipLaunchKernelGGL((k_bidir_scan<IO, true, kGlobalPark, kVar>), grid, block, lds, s, a);
    else hipLaunchKernelGGL((k_bidir_scan<IO, false, kGlobalPark, kVar>), grid, block, lds, s, a);
}

template <typename IO, bool kGlobalPark, int kVar>
void launch_chain(const ScanArgs& a, const Plan& p, hipStream_t s) {
    const size_t lds =
        (4 * p.T * kN + (kVar == kOrdered ? p.T : 0) + (kGlobalPark ? 0 : p.subs * p.T * kWave)) * sizeof(float);
    hipLaunchKernelGGL((k_bidir_chain<IO, kGlobalPark, kVar>), dim3(static_cast<unsigned>(p.wgs)), dim3(wg_threads(p)),
                       lds, s, a);
}

template <typename IO, int kVar>
int launch_all(const ScanArgs& a, const Plan& p, hipStream_t s, hipEvent_t ev0, hipEvent_t ev1) {
    if (p.K > 1 && !p.chain) {
        const size_t lds = (static_cast<size_t>(p.uni ? 1 : 2) * p.T * kN + (kVar == kOrdered ? p.T : 0)) * sizeof(float);
        hipLaunchKernelGGL((k_chunk_aggregate<IO, kVar>), dim3(static_cast<unsigned>(p.wgs)), dim3(wg_threads(p)),
                           lds, s, a);
        const dim3 cgrid(static_cast<unsigned>(p.ncb * (p.uni ? 1 : 2) * p.nseq), 4);
        hipLaunchKernelGGL(k_carry_combine, cgrid, dim3(256), 0, s, a);
    }
    const bool timed = ev0 != nullptr && ev1 != nullptr;
    if (timed && hipEventRecord(ev0, s) != hipSuccess) return VIMSCAN_ERR_HIP;
    if (p.uni) {
        const size_t lds = 2 * static_cast<size_t>(p.T) * kN * sizeof(float);
        if (p.chain) hipLaunchKernelGGL((k_fwd_chain<IO>), dim3(static_cast<unsigned>(p.wgs)), dim3(wg_threads(p)),
                                        lds, s, a);
        else if (p.K > 1) hipLaunchKernelGGL((k_fwd_scan<IO, true>), dim3(static_cast<unsigned>(p.wgs)), dim3(wg_threads(p)),
                                        lds, s, a);
        else hipLaunchKernelGGL((k_fwd_scan<IO, false>), dim3(static_cast<unsigned>(p.wgs)), dim3(wg_threads(p)), lds,
                                s, a);
    } else if (p.chain) {
        if (p.park_global) launch_chain<IO, true, kVar>(a, p, s);
        else launch_chain<IO, false, kVar>(a, p, s);
    } else if (p.park_global) {
        launch_scan<IO, true, kVar>(a, p, s, p.K > 1);
    } else {
        launch_scan<IO, false, kVar>(a, p, s, p.K > 1);
    }
    if (hipGetLastError() != hipSuccess) return VIMSCAN_ERR_HIP;
    if (timed && hipEventRecord(ev1, s) != hipSuccess) return VIMSCAN_ERR_HIP;
    if (p.swap) {
        const dim3 sgrid(static_cast<unsigned>((a.Di + 255) / 256 * p.nseq));
        hipLaunchKernelGGL(k_aux_swap<IO>, sgrid, dim3(256), 0, s, a);
        if (hipGetLastError() != hipSuccess) return VIMSCAN_ERR_HIP;
    }
    return VIMSCAN_OK;
}

// Scratch of the allocation-free entry point (vimscan_bidir_fwd_noalloc): a static device array,
// one copy per GPU the library runs on, held until the process ends. In host code the array's name
// is not a device address; host code uses only the per-device address hipGetSymbolAddress gives.
static_assert(VIMSCAN_NOALLOC_SCRATCH_BYTES % 256 == 0, "scratch size");
static __device__ __align__(256) unsigned char scratch[VIMSCAN_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mutex;
void* g_scratch_addr[kMaxDevices];  // device address of `scratch` on each device, once looked up

// The current device's scratch address (looked up on the device's first use).
int scratch_address(void** out) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return VIMSCAN_ERR_HIP;
    std::lock_guard<std::mutex> lock(g_scratch_mutex);
    if (!g_scratch_addr[dev]) {
        void* p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return VIMSCAN_ERR_HIP;
        g_scratch_addr[dev] = p;
    }
    *out = g_scratch_addr[dev];
    return VIMSCAN_OK;
}

// Every entry point: conv is NULL without the convolution, order NULL in raster order (not both
// set). use_scratch: the workspace is the static scratch array (vimscan_bidir_fwd_noalloc), not
// launch->workspace.
int bidir_impl(const void* x, const void* dt, const void* z, const void* B_f, const void* C_f, const void* B_b,
               const void* C_b, const float* A_f, const float* A_b, const float* D_f, const float* D_b,
               const float* dt_bias_f, const float* dt_bias_b, const vimscan_conv* conv, const int32_t* order,
               int64_t seg_len, void* y, const vimscan_launch* launch, bool use_scratch = false) {
    if (!launch) return VIMSCAN_ERR_NULL;
    Plan p;
    int rc = vimscan_host::make_scan_plan(launch, seg_len, &p);
    if (rc != VIMSCAN_OK) return rc;
    // an empty call launches nothing; its pointers may be NULL (allocators return NULL for 0 bytes)
    if (launch->batch == 0 || launch->seqlen == 0 || launch->d_inner == 0) return VIMSCAN_OK;
    rc = vimscan_host::check_scan_call(x, dt, z, B_f, C_f, B_b, C_b, A_f, A_b, D_f, D_b, dt_bias_f, dt_bias_b, conv,
                                       order, y, launch, p, use_scratch);
    if (rc != VIMSCAN_OK) return rc;

    ScanArgs a;
    a.x = x;
    a.dt = dt;
    a.z = z;
    a.Bm[0] = B_f;
    a.Bm[1] = B_b;
    a.Cm[0] = C_f;
    a.Cm[1] = C_b;
    a.A[0] = A_f;
    a.A[1] = A_b;
    a.D[0] = D_f;
    a.D[1] = D_b;
    a.dtb[0] = dt_bias_f;
    a.dtb[1] = dt_bias_b;
    a.y = y;
    char* ws = static_cast<char*>(launch->workspace);
    if (use_scratch && p.ws > 0) {  // every argument check has passed: the first HIP call
        void* sp = nullptr;
        rc = scratch_address(&sp);
        if (rc != VIMSCAN_OK) return rc;
        ws = static_cast<char*>(sp);
    }
    a.carry = p.K > 1 ? reinterpret_cast<float*>(ws) : nullptr;
    a.dsum = p.K > 1 ? reinterpret_cast<float*>(ws + p.off_dsum) : nullptr;
    a.parkg = p.park_global ? reinterpret_cast<float*>(ws + p.off_park) : nullptr;
    a.tags = p.chain ? reinterpret_cast<uint64_t*>(ws + p.off_tags) : nullptr;
    a.Lp = static_cast<int>(p.Lp);
    a.Di = static_cast<int>(launch->d_inner);
    a.nseq = static_cast<int>(p.nseq);
    a.T = static_cast<int>(p.T);
    a.K = static_cast<int>(p.K);
    a.ncb = static_cast<int>(p.ncb);
    a.subs = static_cast<int>(p.subs);
    a.general = (launch->flags & VIMSCAN_FLAG_GENERAL_DECAY) ? 1 : 0;
    a.cw[0] = conv ? conv->w_f : nullptr;
    a.cw[1] = conv ? conv->w_b : nullptr;
    a.cb[0] = conv ? conv->bias_f : nullptr;
    a.cb[1] = conv ? conv->bias_b : nullptr;
    a.conv_k = conv ? static_cast<int>(conv->k) : 0;
    a.uni = p.uni ? 1 : 0;
    a.order = order;
    hipStream_t s = static_cast<hipStream_t>(launch->stream);
    hipEvent_t ev0 = static_cast<hipEvent_t>(launch->scan_events[0]);
    hipEvent_t ev1 = static_cast<hipEvent_t>(launch->scan_events[1]);
    if (conv)
        rc = launch->io_dtype == VIMSCAN_F32 ? launch_all<float, kWithConv>(a, p, s, ev0, ev1)
                                             : launch_all<Bf16, kWithConv>(a, p, s, ev0, ev1);
    else if (order)
        rc = launch->io_dtype == VIMSCAN_F32 ? launch_all<float, kOrdered>(a, p, s, ev0, ev1)
                                             : launch_all<Bf16, kOrdered>(a, p, s, ev0, ev1);
    else
        rc = launch->io_dtype == VIMSCAN_F32 ? launch_all<float, kPlain>(a, p, s, ev0, ev1)
                                             : launch_all<Bf16, kPlain>(a, p, s, ev0, ev1);
    return rc;
}

}  // namespace

extern "C" {

int vimscan_wait_timeouts(uint64_t* count) {
    if (!count) return VIMSCAN_ERR_NULL;
    unsigned long long v = 0;
    if (hipMemcpyFromSymbol(&v, HIP_SYMBOL(g_wait_timeouts), sizeof(v), 0, hipMemcpyDeviceToHost) != hipSuccess)
        return VIMSCAN_ERR_HIP;
    *count = static_cast<uint64_t>(v);
    return VIMSCAN_OK;
}

int vimscan_bidir_fwd(const void* x, const void* dt, const void* z, const void* B_f, const void* C_f,
                      const void* B_b, const void* C_b, const float* A_f, const float* A_b, const float* D_f,
                      const float* D_b, const float* dt_bias_f, const float* dt_bias_b, int64_t seg_len, void* y,
                      const vimscan_launch* launch) {
    if (launch && (launch->flags & VIMSCAN_FLAG_FORWARD_ONLY)) return VIMSCAN_ERR_FLAGS;
    return bidir_impl(x, dt, z, B_f, C_f, B_b, C_b, A_f, A_b, D_f, D_b, dt_bias_f, dt_bias_b, nullptr, nullptr, seg_len, y,
                      launch);
}

int vimscan_bidir_fwd_noalloc(const void* x, const void* dt, const void* z, const void* B_f, const void* C_f,
                              const void* B_b, const void* C_b, const float* A_f, const float* A_b, const float* D_f,
                              const float* D_b, const float* dt_bias_f, const float* dt_bias_b, int64_t seg_len,
                              void* y, const vimscan_launch* launch) {
    if (launch && (launch->flags & VIMSCAN_FLAG_FORWARD_ONLY)) return VIMSCAN_ERR_FLAGS;
    return bidir_impl(x, dt, z, B_f, C_f, B_b, C_b, A_f, A_b, D_f, D_b, dt_bias_f, dt_bias_b, nullptr, nullptr, seg_len, y,
                      launch, true);
}

int vimscan_fwd(const void* x, const void* dt, const void* z, const void* B, const void* C, const float* A,
                const float* D, const float* dt_bias, int64_t seg_len, void* y, const vimscan_launch* launch) {
    if (!launch) return VIMSCAN_ERR_NULL;
    vimscan_launch l = *launch;
    l.flags |= VIMSCAN_FLAG_FORWARD_ONLY;
    // the forward parameters fill both direction slots; the forward-only kernels read slot 0
    return bidir_impl(x, dt, z, B, C, B, C, A, A, D, D, dt_bias, dt_bias, nullptr, nullptr, seg_len, y, &l);
}

int vimscan_bidir_conv_fwd(const void* x, const vimscan_conv* conv, const void* dt, const void* z,
                           const void* B_f, const void* C_f, const void* B_b, const void* C_b, const float* A_f,
                           const float* A_b, const float* D_f, const float* D_b, const float* dt_bias_f,
                           const float* dt_bias_b, int64_t seg_len, void* y, const vimscan_launch* launch) {
    if (!launch || !conv) return VIMSCAN_ERR_NULL;
    if (launch->flags & VIMSCAN_FLAG_FORWARD_ONLY) return VIMSCAN_ERR_FLAGS;
    if (conv->k < 1 || conv->k > kMaxTaps) return VIMSCAN_ERR_CONV;
    return bidir_impl(x, dt, z, B_f, C_f, B_b, C_b, A_f, A_b, D_f, D_b, dt_bias_f, dt_bias_b, conv, nullptr, seg_len, y,
                      launch);
}

int vimscan_bidir_order_fwd(const void* x, const void* dt, const void* z, const void* B_f, const void* C_f,
                            const void* B_b, const void* C_b, const float* A_f, const float* A_b, const float* D_f,
                            const float* D_b, const float* dt_bias_f, const float* dt_bias_b, const int32_t* order,
                            int64_t seg_len, void* y, const vimscan_launch* launch) {
    if (!launch) return VIMSCAN_ERR_NULL;
    if (launch->flags & VIMSCAN_FLAG_FORWARD_ONLY) return VIMSCAN_ERR_FLAGS;
    const bool empty = launch->batch == 0 || launch->seqlen == 0 || launch->d_inner == 0;
    if (!order && !empty) return VIMSCAN_ERR_NULL;
    if (order && !vimscan_host::aligned(order, 4)) return VIMSCAN_ERR_ALIGN;
    return bidir_impl(x, dt, z, B_f, C_f, B_b, C_b, A_f, A_b, D_f, D_b, dt_bias_f, dt_bias_b, nullptr, order, seg_len,
                      y, launch);
}

}  // extern "C"
