// Linear attention with a decay for each head for AMD MI355X (gfx950): the entry points of include/vimscan.h
// (vimscan_linattn_*) and the kernels around the passes (linattn_device.h).
//
// Forward: one pass. Where sequences and heads alone do not fill the chip, or one may be far longer than the others, sequences are cut
// into segments: every segment's own state first (k_lin_pass, kLocal), a fold of those over the sequence (k_lin_fold), then the
// pass with every segment from its state.
// Backward: the same states, and those of the gradient from the other end; then three passes, for dq, dk and dv. With the decays' gradient
// the first two, which leave its terms, are one launch (128 x 197 x 12 heads of 64 x 64 bf16 160 us, 184 with a launch for each;
// packed 32 x up to 513 x 6 of 40 x 56 fp32 152, 164); without it all three where they are the same instance (101, 127; 117, 141).
// The decays' gradient is exp(g_t) <S_{t-1}, D_t> = sum over u = t .. e of (q_u . dq_u - k_u . dk_u) + the same behind e, where that is
// <S_e, E_e>, formed at the segment's end and at the borders of windows in it (k_lin_borders). The dq and dk passes leave
// the products q . dq and k . dk, without the pair of a token with itself, which is in both and cancels; k_lin_decay_grad adds them up.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>

#include "linattn_device.h"
#include "vimscan.h"

namespace vimscan_dev {

extern template void launch_lin_pass<Bf16, kLocal>(const LinPasses&, bool, hipStream_t);
extern template void launch_lin_pass<Bf16, kForward>(const LinPasses&, bool, hipStream_t);
extern template void launch_lin_pass<Bf16, kGradient>(const LinPasses&, bool, hipStream_t);
extern template void launch_lin_pass<Bf16, kGradientDots>(const LinPasses&, bool, hipStream_t);
extern template void launch_lin_pass<float, kLocal>(const LinPasses&, bool, hipStream_t);
extern template void launch_lin_pass<float, kForward>(const LinPasses&, bool, hipStream_t);
extern template void launch_lin_pass<float, kGradient>(const LinPasses&, bool, hipStream_t);
extern template void launch_lin_pass<float, kGradientDots>(const LinPasses&, bool, hipStream_t);

}  // namespace vimscan_dev

namespace {

using namespace vimscan_dev;
using vimscan_host::LinPlan;
constexpr int kWaves = 4;   // waves of the workgroups of the kernels here

constexpr int kFoldAhead = 8;
// Replaces every segment's own state but those at the sequence's edges by the state it starts from, in the order of the walk (from the
// end: from the last segment on): X = init; for each segment: its place <- X (the first starts from init itself), X = decay X + (what was
// there; of the last nothing is needed). One element a thread; a chain of loads bounds it, eight on their way at once: 42 segments of 24 heads
// of 64 x 64 (33 MB moved) 12 us.
__global__ __launch_bounds__(256) void k_lin_fold(LinArgs a, float* states, const float* tot, const float* init, int from_end) {
    const int64_t ks = static_cast<int64_t>(a.K) * a.V, per_seq = a.H * ks, all = a.nseq * per_seq;
    if (a.offsets && a.nseq <= 4096) {   // often no packed sequence is cut: one look at all of them
        bool any = false;
        for (int64_t seq = threadIdx.x; seq < a.nseq; seq += 256) {
            int64_t lo, hi;
            lin_bounds(a, seq, &lo, &hi);
            any = any || hi - lo > a.seg;
        }
        if (!__syncthreads_or(any)) return;
    }
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; t < all; t += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t seq = t / per_seq, at = t - seq * per_seq, h = at / ks;
        int64_t first = seq * a.segs, count = a.segs;
        if (a.offsets) {
            int64_t lo, hi;
            lin_bounds(a, seq, &lo, &hi);
            first = lin_base(a, seq);
            count = (hi - lo + a.seg - 1) / a.seg;
        }
        if (count < 2) continue;
        float x = init ? init[t] : 0.0f;
        const int64_t from = first + (from_end ? count - 1 : 0), step = from_end ? -1 : 1;
        for (int64_t j = 0; j < count; j += kFoldAhead) {
            // as many loads on their way at once
            float mine[kFoldAhead], dec[kFoldAhead];
#pragma unroll
            for (int k = 0; k < kFoldAhead; ++k) {
                const int64_t slot = from + (j + k < count - 1 ? j + k : count - 2) * step;
                mine[k] = states[slot * per_seq + at];
                dec[k] = tot[slot * a.H + h];
            }
#pragma unroll
            for (int k = 0; k < kFoldAhead; ++k)
                if (j + k < count) {
                    if (j + k > 0) states[(from + (j + k) * step) * per_seq + at] = x;
                    x = fmaf(dec[k], x, mine[k]);
                }
        }
    }
}

// The values at the borders of windows, exp(g_t) <S_{t-1}, D_t>: the product of what the passes of dq and dk left there. A wave
// a border, head and block (borders that no segment has are read and never asked for); memory bounds it: 128 x 12 borders of 64 x 64
// (50 MB) 9.5 us.
struct BorderArgs {
    const float* s;
    const float* e;
    float* out;
    int64_t count;
    int32_t K, V, blocks, NK, NV;
};
constexpr int64_t kMaxBorderWgs = 65536;
__global__ __launch_bounds__(64 * kWaves) void k_lin_borders(BorderArgs a) {
    const int lane = static_cast<int>(threadIdx.x) & 63, tiles = a.NK * a.NV;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * kWaves + (static_cast<int>(threadIdx.x) >> 6); at < a.count;
         at += static_cast<int64_t>(gridDim.x) * kWaves) {
        float sum = 0.0f;
        if (lin_lane_holds(lane, a.NK, a.NV, a.K, a.V - static_cast<int>(at % a.blocks) * 16 * a.NV)) {
            const V4f* s = reinterpret_cast<const V4f*>(a.s) + at * tiles * 64 + lane;
            const V4f* e = reinterpret_cast<const V4f*>(a.e) + at * tiles * 64 + lane;
#pragma unroll 4
            for (int t = 0; t < tiles; ++t) {
                const V4f x = s[t * 64], y = e[t * 64];
#pragma unroll
                for (int r = 0; r < 4; ++r) sum = fmaf(x[r], y[r], sum);
            }
        }
        sum = over_groups(sum);
        for (int m = 1; m < 16; m *= 2) sum += __shfl_xor(sum, m);
        if (lane == 0) a.out[at] = sum;
    }
}

struct DecayGradArgs {
    const float* rq;     // [blocks][tokens][H]: q . dq and k . dk, pairs of a token with itself left out
    const float* rk;
    const float* cdot;   // [slots][H][blocks]: <S, E> at the segment's end
    const float* bdot;   // [borders][H][blocks]: the same at the borders of its windows
    int32_t blocks;
    float* by_token;     // [tokens][H] or NULL
    float* by_head;      // [slots][H], the segments' sums, or NULL
};

// Below this log decay the factor is 0 in fp32 (half the least number is e^-103.97): the token's gradient is 0, and nothing behind the
// token reaches one before it.
constexpr float kNoFactor = -104.0f;

// dg_t = exp(g_t) <S_{t-1}, D_t>, of which the passes leave the values at the borders of windows: inside a window the sum of
// q . dq - k . dk from its end, over the value there. The sums hold pairs of tokens that both lie behind t, which cancel but for
// their rounding and for NaN and infinity: so they go no further than a window, and start anew where a factor is 0. In fp64 (they nearly
// cancel). A wave a segment and head, half of it a window: 128 x 197 x 12 heads 9.0 us, waves that wait for their loads.
__global__ __launch_bounds__(64 * kWaves) void k_lin_decay_grad(LinArgs a, DecayGradArgs d) {
    constexpr int kPer = vimscan_host::kLinWindow / kChunk;
    const int lane = static_cast<int>(threadIdx.x) & 63, half = lane >> 5, l = lane & 31;
    const int64_t task = static_cast<int64_t>(blockIdx.x) * kWaves + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    if (task >= a.slots * a.H) return;
    const int64_t slot = task / a.H, h = task - slot * a.H;
    const LinSegment sg = lin_segment(a, slot);
    double mine = 0.0;
    if (sg.valid) {
        const int64_t windows = (sg.n + kPer * kChunk - 1) / (kPer * kChunk);
        auto at_border = [&](int64_t window) {   // behind that window of rows
            double v = 0.0;
            for (int b = 0; b < d.blocks; ++b) v += d.bdot[((sg.border + window) * a.H + h) * d.blocks + b];
            return v;
        };
        for (int64_t m0 = 0; m0 < windows; m0 += 2) {
            const int64_t m = m0 + half;                       // window, from the walk's end
            const int64_t w = a.rev ? m : windows - 1 - m;     // in rows
            const bool there = m < windows;
            // every chunk's terms first: their loads overlap
            double v[kPer];
            int cut[kPer];   // a token without a factor is among those from the chunk's end on
            int64_t tok[kPer];
#pragma unroll
            for (int c = 0; c < kPer; ++c) {
                const int64_t row = w * (kPer * kChunk) + (a.rev ? c * kChunk + l : (kPer - c) * kChunk - 1 - l);
                tok[c] = there && row < sg.n ? sg.first + row : -1;
                v[c] = 0.0;
                cut[c] = 0;
                if (tok[c] >= 0) {
                    cut[c] = (a.ld_g ? a.g[tok[c] * a.ld_g + h] : a.g[h]) < kNoFactor;
                    if (!cut[c])
                        for (int b = 0; b < d.blocks; ++b) {
                            const int64_t k = (b * a.tokens + tok[c]) * a.H + h;
                            v[c] += static_cast<double>(d.rq[k]) - static_cast<double>(d.rk[k]);
                        }
                }
            }
            double behind = 0.0;   // the value behind the chunk
            if (there) {
                if (m > 0) behind = at_border(a.rev ? w - 1 : w);
                else
                    for (int b = 0; b < d.blocks; ++b) behind += d.cdot[task * d.blocks + b];
            }
#pragma unroll
            for (int c = 0; c < kPer; ++c) {
                const int own = cut[c];
                if (__any(own)) {
#pragma unroll
                    for (int s = 1; s < kChunk; s *= 2) {
                        const double before = __shfl_up(v[c], s, kChunk);
                        const int cut_before = __shfl_up(cut[c], s, kChunk);
                        if (l >= s && !cut[c]) {
                            v[c] += before;
                            cut[c] = cut_before;
                        }
                    }
                } else {
                    v[c] = half_wave_sums(v[c]);
                }
                if (!cut[c]) v[c] += behind;
                const double low = lane_value(v[c], kChunk - 1), high = lane_value(v[c], 2 * kChunk - 1);
                behind = half ? high : low;
                // (the token at the window's other border has the value there)
                if (c == kPer - 1 && l == kChunk - 1 && m + 1 < windows && !own) v[c] = at_border(a.rev ? w : w - 1);
                if (tok[c] >= 0) {
                    if (d.by_token) d.by_token[tok[c] * a.H + h] = static_cast<float>(v[c]);
                    mine += v[c];
                }
            }
        }
    }
    if (!d.by_head) return;
    for (int m = 1; m < 64; m *= 2) mine += __shfl_xor(mine, m);
    if (lane == 0) d.by_head[task] = static_cast<float>(mine);
}

// The gradient of a decay per head: the segments' sums in a fixed order. One workgroup a head.
__global__ __launch_bounds__(256) void k_lin_head_sum(const float* part, int64_t slots, int64_t H, float* out) {
    __shared__ double lds[256];
    const int tid = static_cast<int>(threadIdx.x);
    double s = 0.0;
    for (int64_t k = tid; k < slots; k += 256) s += part[k * H + blockIdx.x];
    lds[tid] = s;
    for (int m = 128; m > 0; m /= 2) {
        __syncthreads();
        if (tid < m) lds[tid] += lds[tid + m];
    }
    if (tid == 0) out[blockIdx.x] = static_cast<float>(lds[0]);
}

// Gradients of shared rows: the sum over the heads of a group, in their order, rounded once. 8681 tokens x 3 groups x 40, two heads each: 5.0 us.
template <typename IO>
__global__ __launch_bounds__(256) void k_lin_group_sum(const float* part, int64_t rows, int rep, int D, void* out) {
    const int64_t all = rows * D;   // rows: tokens x groups
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; t < all; t += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = t / D, c = t - row * D;
        const float* p = part + row * rep * D + c;
        float s = 0.0f;
        for (int r = 0; r < rep; ++r) s += p[static_cast<int64_t>(r) * D];
        Raw<IO, 1> o;
        o.set(&s);
        o.store(static_cast<IoElem<IO>*>(out) + t);
    }
}

// One token: S' = e^g S + k^T v, y = scale q S'. The states' traffic bounds it (8 bytes for 5 operations): 256 x 24 heads of 64 x 64
// (204 MB) 41.7 us, 4.9 TB/s, with states read and written past the caches, 45.4 through them. (Pools of up to 25 MB take the same either way,
// 1.6 MB 4.2 us, 6.3 MB 5.0, 25 MB 8.0. Larger ones that nothing else throws out of the memory-side cache between two tokens would be faster
// through it, 201 MB updated in place 68 and 60 us; a model's other layers do throw them out.) A workgroup takes a row's head and up to 4 CL of its value channels: CL lanes of V channels to a state row, the rows spread over the rest.
struct LinStepArgs {
    LinRows q, k, v;
    int32_t H, dk, dv, blocks;
    const float* g;
    int64_t ld_g;
    float scale;
    float* state;
    int64_t nslots;
    const int32_t* slots_in;
    const int32_t* slots_out;
    void* y;
};
template <typename IO, int V, int CL>
__global__ __launch_bounds__(256) void k_lin_step(LinStepArgs a) {
    using E = IoElem<IO>;
    constexpr int kRows = 256 / CL;
    __shared__ float lds[kWaves][CL][V];
    const int tid = static_cast<int>(threadIdx.x), cl = tid % CL, rg = tid / CL;
    const int64_t id = blockIdx.x;
    const int block = static_cast<int>(id % a.blocks);
    const int64_t rest = id / a.blocks, h = rest % a.H, b = rest / a.H;
    const int c = (block * CL + cl) * V;
    const int64_t from = a.slots_in ? a.slots_in[b] : b;
    const int64_t to = a.slots_out ? a.slots_out[b] : from;
    const bool in = from >= 0 && from < a.nslots && to >= 0 && to < a.nslots;
    const bool live = c < a.dv;
    float sum[V];
#pragma unroll
    for (int v = 0; v < V; ++v) sum[v] = 0.0f;
    if (in && live) {
        const int64_t ks = static_cast<int64_t>(a.dk) * a.dv;
        const float* src = a.state + (from * a.H + h) * ks + c;
        float* dst = a.state + (to * a.H + h) * ks + c;
        const E* q = static_cast<const E*>(a.q.p) + b * a.q.ld + h / a.q.div * a.q.hs;
        const E* k = static_cast<const E*>(a.k.p) + b * a.k.ld + h / a.k.div * a.k.hs;
        const E* vp = static_cast<const E*>(a.v.p) + b * a.v.ld + h * a.v.hs + c;
        const float2 g = as_pair(log2_decay(a.ld_g ? a.g[b * a.ld_g + h] : a.g[h]));
        const float dec = fast_exp2(g.x + g.y);
        float val[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            Raw<IO, 1> x;
            x.load(vp + v);
            val[v] = x.get(0);
        }
#pragma unroll 4
        for (int r = rg; r < a.dk; r += kRows) {
            Raw<float, V> s;
            load_any<true>(s, src + static_cast<int64_t>(r) * a.dv);
            Raw<IO, 1> qr, kr;
            qr.load(q + r);
            kr.load(k + r);
            float n[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                n[v] = fmaf(dec, s.get(v), kr.get(0) * val[v]);
                sum[v] = fmaf(qr.get(0), n[v], sum[v]);
            }
            s.set(n);
            store_any<true>(s, dst + static_cast<int64_t>(r) * a.dv);
        }
    }
    // over the wave's rows, then over the waves in their order
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int m = CL; m < 64; m *= 2) sum[v] += __shfl_xor(sum[v], m);
    const int wave = tid >> 6;
    if ((tid & 63) < CL)
#pragma unroll
        for (int v = 0; v < V; ++v) lds[wave][cl][v] = sum[v];
    __syncthreads();
    if (tid >= CL || !live) return;
    E* y = static_cast<E*>(a.y) + (b * a.H + h) * a.dv + c;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) s += lds[w][cl][v];
        s *= a.scale;
        Raw<IO, 1> o;
        o.set(&s);
        o.store(y + v);
    }
}

// ---------------------------------------------------------------------------------------------
// Host

LinArgs common_args(const vimscan_linattn* p, const vimscan_launch* l, const LinPlan& pl) {
    LinArgs a;
    std::memset(&a, 0, sizeof(a));
    a.H = static_cast<int32_t>(pl.H);
    a.g = p->log_decay;
    a.ld_g = p->ld_decay;
    a.offsets = p->offsets;
    a.tokens = pl.tokens;
    a.Lp = pl.Lp;
    a.seg = pl.seg > 0 ? pl.seg : 1;
    a.nseq = static_cast<int32_t>(pl.nseq);
    a.segs = static_cast<int32_t>(pl.segs);
    a.split = pl.split;
    a.rev = (l->flags & VIMSCAN_FLAG_REVERSE) ? 1 : 0;
    a.slots = pl.slots;
    a.seg_borders = static_cast<int32_t>(pl.seg_borders);
    // (q, k, v and one more array of v's size, against the 256 MB of the memory-side cache)
    const int64_t e = l->io_dtype == VIMSCAN_F32 ? 4 : 2;
    a.once = pl.tokens * e * (2 * pl.G * pl.dk + 2 * pl.H * pl.dv) > (int64_t(256) << 20);
    a.key_scale = a.out_scale = 1.0f;
    return a;
}

// The roles of a pass: reader, key, value. Its rows are not kept in the caches (kOnce) only where no other wave asks for their lines: a
// block of a head's outputs, a head of a group, the head beside it in a line of 128 bytes would fetch them from memory again.
void set_roles(int bytes, LinArgs* a, const LinRows& r, const LinRows& k, const LinRows& v, int64_t K, int64_t V) {
    a->r = r;
    a->k = k;
    a->v = v;
    a->K = static_cast<int32_t>(K);
    a->V = static_cast<int32_t>(V);
    a->blocks = static_cast<int32_t>(vimscan_host::lin_blocks(bytes, K, V));
    a->waves = a->slots * a->H * a->blocks;
    if (a->blocks > 1 || r.div > 1 || k.div > 1 || v.div > 1 || K * bytes % 128 != 0) a->once = 0;
}

void run_passes(int io, bool vec, LinKind kind, const LinPasses& p, hipStream_t s) {
    if (io == VIMSCAN_F32) {
        if (kind == kLocal) launch_lin_pass<float, kLocal>(p, vec, s);
        else if (kind == kForward) launch_lin_pass<float, kForward>(p, vec, s);
        else if (kind == kGradient) launch_lin_pass<float, kGradient>(p, vec, s);
        else launch_lin_pass<float, kGradientDots>(p, vec, s);
    } else {
        if (kind == kLocal) launch_lin_pass<Bf16, kLocal>(p, vec, s);
        else if (kind == kForward) launch_lin_pass<Bf16, kForward>(p, vec, s);
        else if (kind == kGradient) launch_lin_pass<Bf16, kGradient>(p, vec, s);
        else launch_lin_pass<Bf16, kGradientDots>(p, vec, s);
    }
}
void run_pass(int io, bool vec, LinKind kind, const LinArgs& a, hipStream_t s) {
    LinPasses p;
    std::memset(&p, 0, sizeof(p));
    p.count = 1;
    p.a[0] = a;
    run_passes(io, vec, kind, p, s);
}
unsigned some_blocks(int64_t elements) {
    const int64_t n = (elements + 255) / 256;
    return static_cast<unsigned>(n < 65536 ? n : 65536);
}

void run_fold(const LinArgs& a, float* states, const float* tot, const float* init, bool from_end, hipStream_t s) {
    const int64_t all = static_cast<int64_t>(a.nseq) * a.H * a.K * a.V;
    hipLaunchKernelGGL(k_lin_fold, dim3(some_blocks(all) < 2048 ? some_blocks(all) : 2048), dim3(256), 0, s, a, states, tot, init, from_end ? 1 : 0);
}

// Whether rows are whole pieces of 16 bytes that start at multiples of four bytes (the hardware takes those as they are). Else every array
// goes element by element, for which loads and stores bound the pass (bf16, forward and backward, us: 32 x 513 x 12 heads of 100 x 100
// 573 + 2042, of 104 x 104 92 + 445; 128 x 197 x 12 of 64 x 64 from an odd element on 176 + 609, else 46 + 160; of 20 x 20 99 + 275, of 24 x 24
// 37 + 110; fp32 64 x 513 x 8 of 30 x 30 97 + 316, of 32 x 32 69 + 201): pad heads to multiples of 8 (fp32: 4).
bool use_vectors(const vimscan_linattn* p, const vimscan_linattn_grad* g, const void* y, const LinPlan& pl, int io) {
    const int64_t n = io == VIMSCAN_F32 ? 4 : 8;
    if (pl.dk % n != 0 || pl.dv % n != 0) return false;
    if (io == VIMSCAN_F32) return true;
    auto by_words = [](const void* q, int64_t ld, int64_t hs) {
        return reinterpret_cast<uintptr_t>(q) % 4 == 0 && ld % 2 == 0 && hs % 2 == 0;
    };
    if (!by_words(p->q, p->ld_q, p->hs_q) || !by_words(p->k, p->ld_k, p->hs_k) || !by_words(p->v, p->ld_v, p->hs_v))
        return false;
    if (!g) return by_words(y, 0, 0);
    return by_words(g->dy, g->dy ? g->ld_dy : 0, g->dy ? g->hs_dy : 0) && by_words(g->dq, 0, 0) && by_words(g->dk, 0, 0) &&
           by_words(g->dv, 0, 0);
}

bool record(const vimscan_launch* l, int k) {
    if (!l->scan_events[0] || !l->scan_events[1]) return true;
    return hipEventRecord(static_cast<hipEvent_t>(l->scan_events[k]), static_cast<hipStream_t>(l->stream)) == hipSuccess;
}

}  // namespace

extern "C" {

int vimscan_linattn_fwd(const vimscan_linattn* p, int64_t seg_len, void* y, float* h_last, const vimscan_launch* launch) {
    if (!p || !launch) return VIMSCAN_ERR_NULL;
    LinPlan pl;
    int rc = vimscan_host::make_linattn_plan(launch, seg_len, p->heads, p->groups, p->offsets != nullptr, p->nseq, false, &pl);
    if (rc != VIMSCAN_OK) return rc;
    rc = vimscan_host::check_linattn_call(p, y, h_last, nullptr, launch, pl);
    if (rc != VIMSCAN_OK || pl.waves == 0) return rc;
    if (pl.tokens == 0 && !h_last) return VIMSCAN_OK;
    const int io = launch->io_dtype, bytes = io == VIMSCAN_F32 ? 4 : 2;
    const bool vec = use_vectors(p, nullptr, y, pl, io);
    const int32_t rep = static_cast<int32_t>(pl.H / pl.G);
    const LinRows q = {p->q, p->ld_q, p->hs_q, rep}, k = {p->k, p->ld_k, p->hs_k, rep}, v = {p->v, p->ld_v, p->hs_v, 1};
    char* ws = static_cast<char*>(launch->workspace);
    hipStream_t s = static_cast<hipStream_t>(launch->stream);
    LinArgs a = common_args(p, launch, pl);
    set_roles(bytes, &a, q, k, v, pl.dk, pl.dv);
    if (!record(launch, 0)) return VIMSCAN_ERR_HIP;
    a.s0 = p->h0;
    a.s0_row = pl.dv;
    a.s0_col = 1;
    if (pl.split) {
        float* states = reinterpret_cast<float*>(ws + pl.off_s);
        float* tot = reinterpret_cast<float*>(ws + pl.off_tot);
        LinArgs b = a;
        b.s_end = states;
        b.tot = tot;
        run_pass(io, vec, kLocal, b, s);
        run_fold(a, states, tot, p->h0, false, s);
        a.s0_seg = states;
    }
    a.out_scale = p->scale;
    a.o = y;
    a.s_end = h_last;
    run_pass(io, vec, kForward, a, s);
    if (hipGetLastError() != hipSuccess || !record(launch, 1)) return VIMSCAN_ERR_HIP;
    return VIMSCAN_OK;
}

int vimscan_linattn_bwd(const vimscan_linattn* p, int64_t seg_len, const vimscan_linattn_grad* grad,
                        const vimscan_launch* launch) {
    if (!p || !grad || !launch) return VIMSCAN_ERR_NULL;
    LinPlan pl;
    int rc = vimscan_host::make_linattn_plan(launch, seg_len, p->heads, p->groups, p->offsets != nullptr, p->nseq, true, &pl);
    if (rc != VIMSCAN_OK) return rc;
    rc = vimscan_host::check_linattn_call(p, nullptr, nullptr, grad, launch, pl);
    if (rc != VIMSCAN_OK) return rc;
    hipStream_t s = static_cast<hipStream_t>(launch->stream);
    const bool by_head = p->ld_decay == 0;
    const int bytes = launch->io_dtype == VIMSCAN_F32 ? 4 : 2;
    LinArgs a = common_args(p, launch, pl);
    if (pl.tokens == 0 && !(pl.waves > 0 && grad->dh0) && !(by_head && grad->dlog_decay)) return VIMSCAN_OK;
    if (!record(launch, 0)) return VIMSCAN_ERR_HIP;
    if (pl.tokens == 0) {
        // gradients of empty sequences' states, and of decays that no token has
        if (pl.waves > 0 && grad->dh0) {
            const LinRows none = {nullptr, 0, 0, 1};
            set_roles(bytes, &a, none, none, none, pl.dk, pl.dv);
            a.back = 1;
            a.s0 = grad->dh_last;
            a.s0_row = pl.dv;
            a.s0_col = 1;
            a.s_end = grad->dh0;
            run_pass(launch->io_dtype, true, kGradient, a, s);
        }
        if (by_head && grad->dlog_decay)
            hipLaunchKernelGGL(k_lin_head_sum, dim3(static_cast<unsigned>(pl.H)), dim3(256), 0, s,
                               static_cast<const float*>(nullptr), int64_t(0), pl.H, grad->dlog_decay);
        if (hipGetLastError() != hipSuccess || !record(launch, 1)) return VIMSCAN_ERR_HIP;
        return VIMSCAN_OK;
    }
    const int io = launch->io_dtype;
    const bool vec = use_vectors(p, grad, nullptr, pl, io);
    const int32_t rep = static_cast<int32_t>(pl.H / pl.G);
    const LinRows q = {p->q, p->ld_q, p->hs_q, rep}, k = {p->k, p->ld_k, p->hs_k, rep}, v = {p->v, p->ld_v, p->hs_v, 1};
    const LinRows dy = {grad->dy, grad->dy ? grad->ld_dy : 0, grad->dy ? grad->hs_dy : 0, 1};
    char* ws = static_cast<char*>(launch->workspace);
    auto at = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
    a.s0_row = pl.dv;
    a.s0_col = 1;
    if (pl.split) {
        LinArgs b = a;
        set_roles(bytes, &b, k, k, v, pl.dk, pl.dv);
        b.s_end = at(pl.off_s);
        b.tot = at(pl.off_tot);
        run_pass(io, vec, kLocal, b, s);
        run_fold(b, at(pl.off_s), at(pl.off_tot), p->h0, false, s);
        b = a;
        set_roles(bytes, &b, q, q, dy, pl.dk, pl.dv);
        b.back = 1;
        b.key_scale = p->scale;
        b.s_end = at(pl.off_e);
        b.tot = at(pl.off_tot);
        run_pass(io, vec, kLocal, b, s);
        run_fold(b, at(pl.off_e), at(pl.off_tot), grad->dh_last, true, s);
    }
    const bool decays = grad->dlog_decay != nullptr;
    const float* s_seg = pl.split ? at(pl.off_s) : nullptr;
    const float* e_seg = pl.split ? at(pl.off_e) : nullptr;
    const bool shared = rep > 1;
    LinArgs b = a;   // dq: forward, the state transposed
    set_roles(bytes, &b, dy, v, k, pl.dv, pl.dk);
    b.s0 = p->h0;
    b.s0_seg = s_seg;
    b.s0_row = 1;
    b.s0_col = pl.dv;
    b.out_scale = p->scale;
    b.o = shared ? at(pl.off_pq) : grad->dq;
    b.o_f32 = shared;
    if (decays) {
        b.w = q;
        b.dots = at(pl.off_rq);
        b.e = grad->dh_last;
        b.e_seg = e_seg;
        b.e_row = 1;
        b.e_col = pl.dv;
        b.cdot = at(pl.off_cd);
        b.marks = at(pl.off_ms);
    }
    const int32_t qblocks = b.blocks;
    LinPasses three;
    std::memset(&three, 0, sizeof(three));
    three.a[0] = b;
    b = a;           // dk: from the end, the gradient of the state transposed
    set_roles(bytes, &b, v, dy, q, pl.dv, pl.dk);
    b.back = 1;
    b.key_scale = p->scale;
    b.s0 = grad->dh_last;
    b.s0_seg = e_seg;
    b.s0_row = 1;
    b.s0_col = pl.dv;
    b.o = shared ? at(pl.off_pk) : grad->dk;
    b.o_f32 = shared;
    if (decays) {
        b.w = k;
        b.dots = at(pl.off_rk);
        b.marks = at(pl.off_me);
    }
    three.a[1] = b;
    b = a;           // dv, and the gradient of the state before the sequence
    set_roles(bytes, &b, k, q, dy, pl.dk, pl.dv);
    b.back = 1;
    b.key_scale = p->scale;
    b.s0 = grad->dh_last;
    b.s0_seg = e_seg;
    b.s_end = grad->dh0;
    b.o = grad->dv;
    three.a[2] = b;
    three.count = !decays && vimscan_host::lin_alike(bytes, pl.dk, pl.dv) ? 3 : 2;
    run_passes(io, vec, decays ? kGradientDots : kGradient, three, s);
    if (three.count == 2) run_pass(io, vec, kGradient, b, s);
    if (decays) {
        if (pl.borders > 0) {
            const BorderArgs c = {at(pl.off_ms), at(pl.off_me), at(pl.off_bd), pl.borders * pl.H * qblocks, static_cast<int32_t>(pl.dv),
                                  static_cast<int32_t>(pl.dk), qblocks, vimscan_host::lin_contract_tiles(pl.dv),
                                  vimscan_host::lin_output_tiles(bytes, pl.dv, pl.dk)};
            hipLaunchKernelGGL(k_lin_borders, dim3(static_cast<unsigned>(c.count < kMaxBorderWgs * kWaves ? (c.count + kWaves - 1) / kWaves : kMaxBorderWgs)),
                               dim3(64 * kWaves), 0, s, c);
        }
        DecayGradArgs d = {at(pl.off_rq), at(pl.off_rk), at(pl.off_cd), at(pl.off_bd), qblocks, by_head ? nullptr : grad->dlog_decay,
                           by_head ? at(pl.off_hs) : nullptr};
        const int64_t waves = pl.slots * pl.H;
        hipLaunchKernelGGL(k_lin_decay_grad, dim3(static_cast<unsigned>((waves + kWaves - 1) / kWaves)), dim3(64 * kWaves), 0, s,
                           b, d);
        if (by_head)
            hipLaunchKernelGGL(k_lin_head_sum, dim3(static_cast<unsigned>(pl.H)), dim3(256), 0, s, d.by_head, pl.slots, pl.H,
                               grad->dlog_decay);
    }
    if (shared) {
        const int64_t rows = pl.tokens * pl.G;
        const float* part[] = {at(pl.off_pq), at(pl.off_pk)};
        void* out[] = {grad->dq, grad->dk};
        for (int i = 0; i < 2; ++i) {
            const dim3 grid(some_blocks(rows * pl.dk));
            if (io == VIMSCAN_F32)
                hipLaunchKernelGGL(k_lin_group_sum<float>, grid, dim3(256), 0, s, part[i], rows, rep, static_cast<int>(pl.dk), out[i]);
            else
                hipLaunchKernelGGL(k_lin_group_sum<Bf16>, grid, dim3(256), 0, s, part[i], rows, rep, static_cast<int>(pl.dk), out[i]);
        }
    }
    if (hipGetLastError() != hipSuccess || !record(launch, 1)) return VIMSCAN_ERR_HIP;
    return VIMSCAN_OK;
}

int vimscan_linattn_step(const vimscan_linattn* p, float* state, int64_t nslots, const int32_t* slots_in,
                         const int32_t* slots_out, void* y, const vimscan_launch* launch) {
    const int rc = vimscan_host::check_linattn_step(p, state, nslots, slots_in, slots_out, y, launch);
    if (rc != VIMSCAN_OK) return rc;
    if (launch->batch == 0) return VIMSCAN_OK;
    const int64_t H = p->heads, dv = launch->d_inner / H;
    const int32_t rep = static_cast<int32_t>(H / p->groups);
    LinStepArgs a;
    a.q = {p->q, p->ld_q, p->hs_q, rep};
    a.k = {p->k, p->ld_k, p->hs_k, rep};
    a.v = {p->v, p->ld_v, p->hs_v, 1};
    a.H = static_cast<int32_t>(H);
    a.dk = static_cast<int32_t>(launch->d_state);
    a.dv = static_cast<int32_t>(dv);
    a.g = p->log_decay;
    a.ld_g = p->ld_decay;
    a.scale = p->scale;
    a.state = state;
    a.nslots = nslots;
    a.slots_in = slots_in;
    a.slots_out = slots_out;
    a.y = y;
    hipStream_t s = static_cast<hipStream_t>(launch->stream);
    if (!record(launch, 0)) return VIMSCAN_ERR_HIP;
    // four channels a lane where every state row starts at 16 bytes
    const bool vec = dv % 4 == 0 && reinterpret_cast<uintptr_t>(state) % 16 == 0;
    const int wide = !vec ? 64 : dv <= 16 ? 16 : dv <= 32 ? 32 : 64;   // channels of a workgroup
    a.blocks = static_cast<int32_t>((dv + wide - 1) / wide);
    const dim3 grid(static_cast<unsigned>(launch->batch * H * a.blocks));
    const bool f32 = launch->io_dtype == VIMSCAN_F32;
    auto run = [&](auto io) {
        using IO = decltype(io);
        if (!vec) hipLaunchKernelGGL((k_lin_step<IO, 1, 64>), grid, dim3(256), 0, s, a);
        else if (wide == 16) hipLaunchKernelGGL((k_lin_step<IO, 4, 4>), grid, dim3(256), 0, s, a);
        else if (wide == 32) hipLaunchKernelGGL((k_lin_step<IO, 4, 8>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((k_lin_step<IO, 4, 16>), grid, dim3(256), 0, s, a);
    };
    if (f32) run(float{});
    else run(Bf16{});
    if (hipGetLastError() != hipSuccess || !record(launch, 1)) return VIMSCAN_ERR_HIP;
    return VIMSCAN_OK;
}

}  // extern "C"
