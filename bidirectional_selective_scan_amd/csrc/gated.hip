// Gated linear recurrence for AMD MI355X (gfx950): the forward pass over whole sequences, its
// backward pass and the single-token form (include/vimscan.h, vimscan_gated_*).
//
// Per channel: u = -c softplus(lam) sigmoid(r), a = e^u, m = sqrt(1 - a^2), h' = a h + m sigmoid(i) x.

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>

#include "block_device.h"
#include "block_plan.h"
#include "vimscan.h"

namespace {

using namespace vimscan_dev;
using vimscan_host::GatedPlan;
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
    int64_t N;               // tokens
    int64_t Lp;
    int32_t D, nseq, ncb;
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
    float* part;             // [nseq][D] partial sums of dlam
};

// Walking positions: position p of the call is token p, or N - 1 - p walked from the end; sequence
// q in walking order is sequence q or nseq - 1 - q of the caller.
__device__ __forceinline__ int64_t token_of(const GatedArgs& a, int64_t p) { return a.rev ? a.N - 1 - p : p; }
__device__ __forceinline__ int64_t seq_of(const GatedArgs& a, int64_t q) { return a.rev ? a.nseq - 1 - q : q; }

// First position of sequence q in walking order (q = nseq: the end), inside 0..N whatever the
// offsets hold.
__device__ __forceinline__ int64_t bound_of(const GatedArgs& a, int64_t q) {
    if (!a.offsets) return q * a.Lp;
    const int64_t o = a.rev ? a.N - a.offsets[a.nseq - q] : a.offsets[q];
    return o < 0 ? 0 : o > a.N ? a.N : o;
}

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
// at t = 1/4 is 5e-8 of the result), larger t from a itself.
__device__ __forceinline__ float one_minus_sq(float q, float a) {
    const float t = -2.0f * kLn2 * q;
    float s = fmaf(t, -1.0f / 720.0f, 1.0f / 120.0f);
    s = fmaf(t, -s, 1.0f / 24.0f);
    s = fmaf(t, -s, 1.0f / 6.0f);
    s = fmaf(t, -s, 0.5f);
    s = fmaf(t, -s, 1.0f);
    return t < 0.25f ? t * s : fmaf(-a, a, 1.0f);
}

struct Gates {
    float s, ns;   // sigmoid(r) and 1 - sigmoid(r)
    float g, ng;   // sigmoid(i) and 1 - sigmoid(i)
    float q, a, m; // u log2(e), exp(u), sqrt(1 - a^2)
};

// sigmoid(v) = 1 / (1 + e), 1 - sigmoid(v) = e / (1 + e) with e = e^-v held below 2^126.
__device__ __forceinline__ void sigmoid2(float v, float* s, float* ns) {
    const float e = fast_exp2(fminf(-v * kLog2e, 126.0f));
    *s = fast_rcp(1.0f + e);
    *ns = e * *s;
}

__device__ __forceinline__ Gates gates(float r, float i, float k2) {
    Gates o;
    sigmoid2(r, &o.s, &o.ns);
    sigmoid2(i, &o.g, &o.ng);
    o.q = k2 * o.s;
    o.a = fast_exp2(o.q);
    o.m = fast_sqrt(one_minus_sq(o.q, o.a));
    return o;
}

template <typename IO>
__device__ __forceinline__ float ld(const void* p, int64_t k) {
    Raw<IO, 1> w;
    w.load(static_cast<const typename IoOf<IO>::elem*>(p) + k);
    return w.get(0);
}
template <typename IO>
__device__ __forceinline__ void st(void* p, int64_t k, float v) {
    Raw<IO, 1> w;
    w.set(&v);
    w.store(static_cast<typename IoOf<IO>::elem*>(p) + k);
}

// One wave per sequence and block of 64 channels, token by token.
template <typename IO>
__global__ __launch_bounds__(64) void k_gated_fwd(GatedArgs a) {
    const int64_t q = blockIdx.x / a.ncb;
    const int d = static_cast<int>(blockIdx.x % a.ncb) * 64 + static_cast<int>(threadIdx.x);
    if (d >= a.D) return;
    const int64_t slot = seq_of(a, q) * a.D + d;
    const int64_t p0 = bound_of(a, q), p1 = bound_of(a, q + 1);
    float h = a.h0 ? a.h0[slot] : 0.0f;
    if (p1 > p0) {
        const float k2 = decay_rate(a.lam[d], a.c);
        for (int64_t p = p0; p < p1; ++p) {
            const int64_t t = token_of(a, p);
            if (a.states && p % kGatedStride == 0) a.states[p / kGatedStride * a.D + d] = h;
            const Gates o = gates(ld<IO>(a.r, t * a.ld_r + d), ld<IO>(a.i, t * a.ld_i + d), k2);
            h = fmaf(o.a, h, o.m * o.g * ld<IO>(a.x, t * a.ld_x + d));
            st<IO>(a.y, t * a.D + d, h);
        }
    }
    if (a.h_last) a.h_last[slot] = h;
}

// The same division of the work, from the last group of kGatedStride positions to the first: the
// group's states are walked forward again from the saved one, then the gradient backward.
template <typename IO>
__global__ __launch_bounds__(64) void k_gated_bwd(GatedArgs a) {
    const int64_t q = blockIdx.x / a.ncb;
    const int d = static_cast<int>(blockIdx.x % a.ncb) * 64 + static_cast<int>(threadIdx.x);
    if (d >= a.D) return;
    const int64_t slot = seq_of(a, q) * a.D + d;
    const int64_t p0 = bound_of(a, q), p1 = bound_of(a, q + 1);
    float e = a.dh_last ? a.dh_last[slot] : 0.0f;
    float sum = 0.0f;
    if (p1 > p0) {
        const float k2 = decay_rate(a.lam[d], a.c);
        float before[kGatedStride];
        for (int64_t grp = (p1 - 1) / kGatedStride; grp >= p0 / kGatedStride; --grp) {
            const int64_t g0 = grp * kGatedStride;
            const int64_t lo = g0 > p0 ? g0 : p0, hi = g0 + kGatedStride < p1 ? g0 + kGatedStride : p1;
            float h = lo == p0 ? (a.h0 ? a.h0[slot] : 0.0f) : a.states_in[grp * a.D + d];
            for (int64_t p = lo; p < hi; ++p) {
                const int64_t t = token_of(a, p);
                before[p - g0] = h;
                const Gates o = gates(ld<IO>(a.r, t * a.ld_r + d), ld<IO>(a.i, t * a.ld_i + d), k2);
                h = fmaf(o.a, h, o.m * o.g * ld<IO>(a.x, t * a.ld_x + d));
            }
            for (int64_t p = hi - 1; p >= lo; --p) {
                const int64_t t = token_of(a, p);
                const Gates o = gates(ld<IO>(a.r, t * a.ld_r + d), ld<IO>(a.i, t * a.ld_i + d), k2);
                const float x = ld<IO>(a.x, t * a.ld_x + d);
                const float del = e + (a.dy ? ld<IO>(a.dy, t * a.ld_dy + d) : 0.0f);
                const float u = o.q * kLn2;
                const float um = o.m > 0.0f ? u * fast_rcp(o.m) : 0.0f;
                const float dx = del * o.m * o.g;
                const float w = del * (u * o.a * before[p - g0] - o.g * x * o.a * o.a * um);
                st<IO>(a.dx, t * a.ld_dx + d, dx);
                if (a.di) st<IO>(a.di, t * a.ld_di + d, dx * x * o.ng);
                if (a.dr) st<IO>(a.dr, t * a.ld_dr + d, w * o.ns);
                sum += w;
                e = o.a * del;
            }
        }
    }
    if (a.dh0) a.dh0[slot] = e;
    a.part[q * a.D + d] = sum;
}

// dlam = sigmoid(lam) / softplus(lam) * the sum of the partial sums, in their order.
__global__ __launch_bounds__(64) void k_gated_dlam(GatedArgs a, int64_t parts) {
    const int d = static_cast<int>(blockIdx.x) * 64 + static_cast<int>(threadIdx.x);
    if (d >= a.D) return;
    float sum = 0.0f;
    for (int64_t k = 0; k < parts; ++k) sum += a.part[k * a.D + d];
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
    int32_t D, ncb;
};

// One token: a wave per row and block of 64 channels.
template <typename IO>
__global__ __launch_bounds__(64) void k_gated_step(StepArgs a) {
    const int64_t b = blockIdx.x / a.ncb;
    const int d = static_cast<int>(blockIdx.x % a.ncb) * 64 + static_cast<int>(threadIdx.x);
    if (d >= a.D) return;
    const int64_t from = a.slots_in ? a.slots_in[b] : b;
    const int64_t to = a.slots_out ? a.slots_out[b] : from;
    float h = 0.0f;
    if (from >= 0 && from < a.nslots && to >= 0 && to < a.nslots) {
        const Gates o = gates(ld<IO>(a.r, b * a.ld_r + d), ld<IO>(a.i, b * a.ld_i + d), decay_rate(a.lam[d], a.c));
        h = fmaf(o.a, a.state[from * a.D + d], o.m * o.g * ld<IO>(a.x, b * a.ld_x + d));
        a.state[to * a.D + d] = h;
    }
    st<IO>(a.y, b * a.D + d, h);
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
    a.N = p.tokens;
    a.Lp = p.Lp;
    a.D = static_cast<int32_t>(l->d_inner);
    a.nseq = static_cast<int32_t>(p.nseq);
    a.ncb = static_cast<int32_t>(p.ncb);
    a.rev = (l->flags & VIMSCAN_FLAG_REVERSE) ? 1 : 0;
    return a;
}

// The caller's event pair around the call's kernels.
bool record(const vimscan_launch* l, int k) {
    if (!l->scan_events[0] || !l->scan_events[1]) return true;
    return hipEventRecord(static_cast<hipEvent_t>(l->scan_events[k]), static_cast<hipStream_t>(l->stream)) == hipSuccess;
}

}  // namespace

extern "C" {

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
    const dim3 grid(static_cast<unsigned>(p.wgs));
    if (launch->io_dtype == VIMSCAN_F32) hipLaunchKernelGGL(k_gated_fwd<float>, grid, dim3(64), 0, s, a);
    else hipLaunchKernelGGL(k_gated_fwd<Bf16>, grid, dim3(64), 0, s, a);
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
    a.part = static_cast<float*>(launch->workspace);
    hipStream_t s = static_cast<hipStream_t>(launch->stream);
    if (!record(launch, 0)) return VIMSCAN_ERR_HIP;
    if (p.wgs > 0) {
        const dim3 grid(static_cast<unsigned>(p.wgs));
        if (launch->io_dtype == VIMSCAN_F32) hipLaunchKernelGGL(k_gated_bwd<float>, grid, dim3(64), 0, s, a);
        else hipLaunchKernelGGL(k_gated_bwd<Bf16>, grid, dim3(64), 0, s, a);
    }
    if (a.dlam) {
        const unsigned blocks = static_cast<unsigned>((launch->d_inner + 63) / 64);
        hipLaunchKernelGGL(k_gated_dlam, dim3(blocks), dim3(64), 0, s, a, p.nseq);
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
    a.ncb = static_cast<int32_t>((launch->d_inner + 63) / 64);
    hipStream_t s = static_cast<hipStream_t>(launch->stream);
    if (!record(launch, 0)) return VIMSCAN_ERR_HIP;
    const dim3 grid(static_cast<unsigned>(launch->batch * a.ncb));
    if (launch->io_dtype == VIMSCAN_F32) hipLaunchKernelGGL(k_gated_step<float>, grid, dim3(64), 0, s, a);
    else hipLaunchKernelGGL(k_gated_step<Bf16>, grid, dim3(64), 0, s, a);
    if (hipGetLastError() != hipSuccess || !record(launch, 1)) return VIMSCAN_ERR_HIP;
    return VIMSCAN_OK;
}

}  // extern "C"
