// Block norm for AMD MI355X (gfx950): gate, post-norm, scaled residual and pre-norm of a row in one
// pass, and its backward pass (include/vimscan.h, vimscan_norm_*).

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>

#include "block_device.h"
#include "block_plan.h"
#include "vimscan.h"

namespace {

using namespace vimscan_dev;
using vimscan_host::NormPlan;

struct NormArgs {
    const void* x;
    const void* z;
    int64_t ld_x, ld_z;
    const float* w_post;
    const void* residual;
    const float* gamma;
    const float* w_pre;
    float eps, inv_d;
    int32_t D, res_f32, after;
    int64_t rows;
    void* sum;
    void* n;
    // backward
    const void* dsum;
    const void* dn;
    void* dx;
    void* dz;
    int64_t ld_dx, ld_dz;
    void* dres;
    float* dw[3];   // of w_post, gamma, w_pre
    float* part;    // [workgroup][3][D] partial weight gradients, NULL when none is wanted
};

// Sum over a wave, on the vector unit alone: within rows of 16 lanes by lane permutations of a quad and
// mirrors, across rows by lane swaps. Every lane gets the same bits.
template <int kCtrl>
__device__ __forceinline__ float add_dpp(float v) {
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), kCtrl, 0xf, 0xf, false));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = add_dpp<0xB1>(v);   // lane ^ 1
    v = add_dpp<0x4E>(v);   // lane ^ 2
    v = add_dpp<0x141>(v);  // half row mirrored
    v = add_dpp<0x140>(v);  // row mirrored
    float p, q;
    swap16(v, &p, &q);
    swap32(p + q, &p, &q);
    return p + q;
}

// Sums of two values over the W waves of a row, in the waves' order. Calls alternate between two slots:
// a slot is written again only after the barrier of the call between, which every wave reaches after
// its reads of that slot, so one barrier a call is enough.
template <int W>
__device__ __forceinline__ void row_sum(float* u, float* v, float2 (*lds)[W], int& slot, int wave) {
    *u = wave_sum(*u);
    *v = wave_sum(*v);
    if constexpr (W > 1) {
        slot ^= 1;
        if ((threadIdx.x & 63) == 0) lds[slot][wave] = make_float2(*u, *v);
        __syncthreads();
        float su = 0.0f, sv = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            su += lds[slot][k].x;
            sv += lds[slot][k].y;
        }
        *u = su;
        *v = sv;
    }
}

__device__ __forceinline__ float sigmoid(float v) { return fast_rcp(1.0f + fast_exp2(-v * kLog2e)); }

// How a row is spread: W waves, each lane NV vectors of V consecutive channels.
template <int V, int NV, int W> struct Spread {
    static constexpr int kThreads = W > 4 ? 64 * W : 256;
    static constexpr int kRows = kThreads / (64 * W);  // rows a workgroup works on at once
    __device__ __forceinline__ static int channel(int wave, int lane, int k) { return ((k * W + wave) * 64 + lane) * V; }
};

template <typename T, int V, int NV, typename S>
__device__ __forceinline__ void ld_row(const void* base, int64_t at, bool there, int D, int wave, int lane, Raw<T, V> (&o)[NV]) {
    const IoElem<T>* p = static_cast<const IoElem<T>*>(base) + at;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = S::channel(wave, lane, k);
        if (there && c < D) o[k].load(p + c);
        else o[k].zero();
    }
}
template <typename T, int V, int NV, typename S>
__device__ __forceinline__ void st_row(void* base, int64_t at, int D, int wave, int lane, const float (&v)[NV][V]) {
    IoElem<T>* p = static_cast<IoElem<T>*>(base) + at;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = S::channel(wave, lane, k);
        if (c < D) {
            Raw<T, V> o;
            o.set(v[k]);
            o.store(p + c);
        }
    }
}
// A weight's channels (1 where the weight is absent).
template <int V, int NV, typename S>
__device__ __forceinline__ void ld_weight(const float* w, int D, int wave, int lane, float (&o)[NV][V]) {
    Raw<float, V> r[NV];
    ld_row<float, V, NV, S>(w, 0, w != nullptr, D, wave, lane, r);
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) o[k][v] = w ? r[k].get(v) : 1.0f;
}

// Forward: a row stays in registers from its one read to its one write.
template <typename IO, typename RES, int V, int NV, int W>
__global__ __launch_bounds__((Spread<V, NV, W>::kThreads)) void k_norm_fwd(NormArgs a) {
    using S = Spread<V, NV, W>;
    __shared__ float2 lds[2][W];
    const int lane = static_cast<int>(threadIdx.x) & 63;
    const int w = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6), wave = w % W;
    float wp[NV][V], ga[NV][V], wn[NV][V];
    ld_weight<V, NV, S>(a.w_post, a.D, wave, lane, wp);
    ld_weight<V, NV, S>(a.gamma, a.D, wave, lane, ga);
    ld_weight<V, NV, S>(a.w_pre, a.D, wave, lane, wn);
    int slot = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * S::kRows + w / W; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * S::kRows) {
        Raw<IO, V> x[NV], z[NV];
        Raw<RES, V> r[NV];
        ld_row<IO, V, NV, S>(a.x, row * a.ld_x, true, a.D, wave, lane, x);
        ld_row<IO, V, NV, S>(a.z, row * a.ld_z, a.z != nullptr, a.D, wave, lane, z);
        ld_row<RES, V, NV, S>(a.residual, row * a.D, a.residual != nullptr, a.D, wave, lane, r);
        float s[NV][V];
        float ss = 0.0f, none = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[k][v] = x[k].get(v);
                if (a.z && !a.after) {
                    const float zv = z[k].get(v);
                    s[k][v] *= zv * sigmoid(zv);
                }
                ss = fmaf(s[k][v], s[k][v], ss);
            }
        float rho = 1.0f;
        if (a.w_post) {
            row_sum<W>(&ss, &none, lds, slot, wave);
            rho = fast_rsq(fmaf(ss, a.inv_d, a.eps));
        }
        ss = none = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[k][v] *= rho * wp[k][v];
                if (a.after) {
                    const float zv = z[k].get(v);
                    s[k][v] *= zv * sigmoid(zv);
                }
                s[k][v] = fmaf(s[k][v], ga[k][v], r[k].get(v));
                ss = fmaf(s[k][v], s[k][v], ss);
            }
        if (a.sum) st_row<RES, V, NV, S>(a.sum, row * a.D, a.D, wave, lane, s);
        if (!a.w_pre) continue;
        row_sum<W>(&ss, &none, lds, slot, wave);
        rho = fast_rsq(fmaf(ss, a.inv_d, a.eps));
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) s[k][v] *= rho * wn[k][v];
        st_row<IO, V, NV, S>(a.n, row * a.D, a.D, wave, lane, s);
    }
}

// Backward: the row's stages again from its inputs, then the gradients against them; the weights'
// gradients of a wave's rows stay in registers, are added up over the workgroup's waves at the end and
// left for k_norm_cols.
template <typename IO, typename RES, int V, int NV, int W>
__global__ __launch_bounds__((Spread<V, NV, W>::kThreads)) void k_norm_bwd(NormArgs a) {
    using S = Spread<V, NV, W>;
    __shared__ float2 lds[2][W];
    const int lane = static_cast<int>(threadIdx.x) & 63;
    const int w = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6), wave = w % W;
    float wp[NV][V], ga[NV][V], wn[NV][V];
    ld_weight<V, NV, S>(a.w_post, a.D, wave, lane, wp);
    ld_weight<V, NV, S>(a.gamma, a.D, wave, lane, ga);
    ld_weight<V, NV, S>(a.w_pre, a.D, wave, lane, wn);
    float dwp[NV][V], dga[NV][V], dwn[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) dwp[k][v] = dga[k][v] = dwn[k][v] = 0.0f;
    int slot = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * S::kRows + w / W; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * S::kRows) {
        Raw<IO, V> x[NV], z[NV], dn[NV];
        Raw<RES, V> r[NV], ds[NV];
        ld_row<IO, V, NV, S>(a.x, row * a.ld_x, true, a.D, wave, lane, x);
        ld_row<IO, V, NV, S>(a.z, row * a.ld_z, a.z != nullptr, a.D, wave, lane, z);
        ld_row<RES, V, NV, S>(a.residual, row * a.D, a.residual != nullptr, a.D, wave, lane, r);
        ld_row<IO, V, NV, S>(a.dn, row * a.D, a.dn != nullptr, a.D, wave, lane, dn);
        ld_row<RES, V, NV, S>(a.dsum, row * a.D, a.dsum != nullptr, a.D, wave, lane, ds);
        // val: the post-norm's input; s: the sum
        float val[NV][V], s[NV][V];
        float u = 0.0f, t = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                val[k][v] = x[k].get(v);
                if (a.z && !a.after) {
                    const float zv = z[k].get(v);
                    val[k][v] *= zv * sigmoid(zv);
                }
                u = fmaf(val[k][v], val[k][v], u);
            }
        float rho1 = 1.0f, rho2 = 0.0f, k2 = 0.0f;
        if (a.w_post) {
            row_sum<W>(&u, &t, lds, slot, wave);
            rho1 = fast_rsq(fmaf(u, a.inv_d, a.eps));
        }
        u = t = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float p = val[k][v] * rho1 * wp[k][v];
                if (a.after) {
                    const float zv = z[k].get(v);
                    p *= zv * sigmoid(zv);
                }
                s[k][v] = fmaf(p, ga[k][v], r[k].get(v));
                u = fmaf(s[k][v], s[k][v], u);
                t = fmaf(dn[k].get(v) * wn[k][v], s[k][v], t);
            }
        if (a.dn) {
            row_sum<W>(&u, &t, lds, slot, wave);
            rho2 = fast_rsq(fmaf(u, a.inv_d, a.eps));
            k2 = t * a.inv_d * rho2 * rho2 * rho2;
        }
        // from here s is the gradient of the sum
        u = t = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float g = dn[k].get(v);
                dwn[k][v] = fmaf(g, s[k][v] * rho2, dwn[k][v]);
                s[k][v] = ds[k].get(v) + fmaf(rho2 * g, wn[k][v], -s[k][v] * k2);
                const float q = val[k][v] * rho1 * wp[k][v], dp = s[k][v] * ga[k][v];
                float p = q, dq = dp;
                if (a.after) {
                    const float zv = z[k].get(v), gate = zv * sigmoid(zv);
                    p *= gate;
                    dq *= gate;
                }
                dga[k][v] = fmaf(p, s[k][v], dga[k][v]);
                dwp[k][v] = fmaf(dq, val[k][v] * rho1, dwp[k][v]);
                u = fmaf(dq * wp[k][v], val[k][v], u);
            }
        if (a.dres) st_row<RES, V, NV, S>(a.dres, row * a.D, a.D, wave, lane, s);
        float k1 = 0.0f;
        if (a.w_post) {
            row_sum<W>(&u, &t, lds, slot, wave);
            k1 = u * a.inv_d * rho1 * rho1 * rho1;
        }
        float dz[NV][V];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float dp = s[k][v] * ga[k][v];
                float gate = 1.0f, slope = 0.0f;
                if (a.z) {
                    const float zv = z[k].get(v), sg = sigmoid(zv);
                    gate = zv * sg;
                    slope = sg * fmaf(zv, 1.0f - sg, 1.0f);
                }
                const float dq = a.after ? dp * gate : dp;
                const float dv = fmaf(rho1 * dq, wp[k][v], -val[k][v] * k1);
                const float q = val[k][v] * rho1 * wp[k][v];
                dz[k][v] = (a.after ? dp * q : dv * x[k].get(v)) * slope;
                s[k][v] = a.after ? dv : dv * gate;
            }
        if (a.dx) st_row<IO, V, NV, S>(a.dx, row * a.ld_dx, a.D, wave, lane, s);
        if (a.dz) st_row<IO, V, NV, S>(a.dz, row * a.ld_dz, a.D, wave, lane, dz);
    }
    if (!a.part) return;
    float* part = a.part + static_cast<int64_t>(blockIdx.x) * 3 * a.D;
    if constexpr (S::kRows == 1) {
        st_row<float, V, NV, S>(part, 0, a.D, wave, lane, dwp);
        st_row<float, V, NV, S>(part, a.D, a.D, wave, lane, dga);
        st_row<float, V, NV, S>(part, 2 * a.D, a.D, wave, lane, dwn);
    } else {
        // the workgroup's waves in their order, one weight at a time
        __shared__ float col[NV * 64 * V];
        auto add_up = [&](float (&g)[NV][V], int which) {
            for (int turn = 0; turn < S::kRows; ++turn) {
                if (w == turn) {
#pragma unroll
                    for (int k = 0; k < NV; ++k)
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            float* p = col + (k * V + v) * 64 + lane;
                            if (turn > 0) g[k][v] += *p;
                            *p = g[k][v];
                        }
                    if (turn == S::kRows - 1) st_row<float, V, NV, S>(part, which * a.D, a.D, wave, lane, g);
                }
                __syncthreads();
            }
        };
        add_up(dwp, 0);
        add_up(dga, 1);
        add_up(dwn, 2);
    }
}

// The weight gradients: the workgroups' partial sums.
__global__ __launch_bounds__(1024) void k_norm_cols(NormArgs a, int parts) {
    float* dst = a.dw[blockIdx.y];
    if (!dst) return;
    const int c0 = static_cast<int>(blockIdx.x) * kColumns, c = c0 + static_cast<int>(threadIdx.x);
    const float s = column_sum(a.part + static_cast<int64_t>(blockIdx.y) * a.D, parts, 3 * static_cast<int64_t>(a.D), c0, a.D);
    if (threadIdx.x < kColumns && c < a.D) dst[c] = s;
}

// Wide loads where every row of every tensor, and every weight, is aligned to them.
bool by_four(const NormArgs& a, size_t e, size_t re) {
    auto ok = [](const void* p, int64_t ld, size_t size) {
        return !p || (reinterpret_cast<uintptr_t>(p) % (4 * size) == 0 && ld % 4 == 0);
    };
    const int64_t d = a.D;
    bool r = d % 4 == 0 && ok(a.x, a.ld_x, e) && ok(a.z, a.ld_z, e) && ok(a.n, d, e) && ok(a.dn, d, e) &&
             ok(a.dx, a.ld_dx, e) && ok(a.dz, a.ld_dz, e);
    const void* rs[] = {a.residual, a.sum, a.dsum, a.dres};
    for (const void* p : rs) r = r && ok(p, d, re);
    const void* ws[] = {a.w_post, a.gamma, a.w_pre};
    for (const void* p : ws) r = r && ok(p, d, 4);
    return r;
}

template <typename IO, typename RES, int V, int NV, int W>
void launch(const NormArgs& a, const NormPlan& p, bool back, hipStream_t s) {
    using S = Spread<V, NV, W>;
    const int64_t full = (a.rows + S::kRows - 1) / S::kRows;
    const dim3 grid(static_cast<unsigned>(full < p.wgs ? full : p.wgs)), block(S::kThreads);
    if (back) hipLaunchKernelGGL((k_norm_bwd<IO, RES, V, NV, W>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_norm_fwd<IO, RES, V, NV, W>), grid, block, 0, s, a);
    if (back && a.part)
        hipLaunchKernelGGL(k_norm_cols, dim3(static_cast<unsigned>((a.D + kColumns - 1) / kColumns), 3), dim3(1024), 0, s, a,
                           static_cast<int>(grid.x));
}

// The narrowest spread that holds the row.
template <typename IO, typename RES>
void launch_any(const NormArgs& a, const NormPlan& p, bool back, hipStream_t s) {
    const int d = a.D;
    if (by_four(a, sizeof(IoElem<IO>), sizeof(IoElem<RES>))) {
        if (d <= 256) launch<IO, RES, 4, 1, 1>(a, p, back, s);
        else if (d <= 512) launch<IO, RES, 4, 2, 1>(a, p, back, s);
        else if (d <= 768) launch<IO, RES, 4, 3, 1>(a, p, back, s);
        else if (d <= 1024) launch<IO, RES, 4, 4, 1>(a, p, back, s);
        else if (d <= 2048) launch<IO, RES, 4, 2, 4>(a, p, back, s);
        else if (d <= 4096) launch<IO, RES, 4, 4, 4>(a, p, back, s);
        else if (d <= 8192) launch<IO, RES, 4, 4, 8>(a, p, back, s);
        else if (d <= 16384) launch<IO, RES, 4, 4, 16>(a, p, back, s);
        else launch<IO, RES, 4, 8, 16>(a, p, back, s);
    } else {
        if (d <= 256) launch<IO, RES, 1, 4, 1>(a, p, back, s);
        else if (d <= 512) launch<IO, RES, 1, 8, 1>(a, p, back, s);
        else if (d <= 1024) launch<IO, RES, 1, 4, 4>(a, p, back, s);
        else if (d <= 2048) launch<IO, RES, 1, 8, 4>(a, p, back, s);
        else if (d <= 4096) launch<IO, RES, 1, 16, 4>(a, p, back, s);
        else if (d <= 8192) launch<IO, RES, 1, 16, 8>(a, p, back, s);
        else if (d <= 16384) launch<IO, RES, 1, 16, 16>(a, p, back, s);
        else launch<IO, RES, 1, 32, 16>(a, p, back, s);
    }
}

void launch_typed(const NormArgs& a, const NormPlan& p, int io, bool back, hipStream_t s) {
    if (io == VIMSCAN_F32) launch_any<float, float>(a, p, back, s);
    else if (a.res_f32) launch_any<Bf16, float>(a, p, back, s);
    else launch_any<Bf16, Bf16>(a, p, back, s);
}

// An empty backward pass: weight gradients of zero.
__global__ __launch_bounds__(64) void k_norm_zero(NormArgs a) {
    const int c = static_cast<int>(blockIdx.x) * 64 + static_cast<int>(threadIdx.x);
    if (c < a.D && a.dw[blockIdx.y]) a.dw[blockIdx.y][c] = 0.0f;
}

NormArgs common_args(const vimscan_norm* n, const vimscan_launch* l, const NormPlan& p) {
    NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = n->x;
    a.z = n->z;
    a.ld_x = n->ld_x;
    a.ld_z = n->ld_z;
    a.w_post = n->w_post;
    a.residual = n->residual;
    a.gamma = n->gamma;
    a.w_pre = n->w_pre;
    a.eps = n->eps;
    a.inv_d = 1.0f / static_cast<float>(p.D > 0 ? p.D : 1);
    a.D = static_cast<int32_t>(p.D);
    a.res_f32 = n->res_dtype == VIMSCAN_F32 ? 1 : 0;
    a.after = (l->flags & VIMSCAN_FLAG_GATE_AFTER) ? 1 : 0;
    a.rows = p.rows;
    return a;
}

bool record(const vimscan_launch* l, int k) {
    if (!l->scan_events[0] || !l->scan_events[1]) return true;
    return hipEventRecord(static_cast<hipEvent_t>(l->scan_events[k]), static_cast<hipStream_t>(l->stream)) == hipSuccess;
}

}  // namespace

extern "C" {

int vimscan_norm_fwd(const vimscan_norm* n, void* sum, void* out, const vimscan_launch* launch) {
    if (!n || !launch) return VIMSCAN_ERR_NULL;
    NormPlan p;
    int rc = vimscan_host::make_norm_plan(launch, false, &p);
    if (rc != VIMSCAN_OK) return rc;
    rc = vimscan_host::check_norm_call(n, sum, out, nullptr, launch, p);
    if (rc != VIMSCAN_OK || p.wgs == 0) return rc;
    NormArgs a = common_args(n, launch, p);
    a.sum = sum;
    a.n = out;
    hipStream_t s = static_cast<hipStream_t>(launch->stream);
    if (!record(launch, 0)) return VIMSCAN_ERR_HIP;
    launch_typed(a, p, launch->io_dtype, false, s);
    if (hipGetLastError() != hipSuccess || !record(launch, 1)) return VIMSCAN_ERR_HIP;
    return VIMSCAN_OK;
}

int vimscan_norm_bwd(const vimscan_norm* n, const vimscan_norm_grad* grad, const vimscan_launch* launch) {
    if (!n || !grad || !launch) return VIMSCAN_ERR_NULL;
    NormPlan p;
    int rc = vimscan_host::make_norm_plan(launch, true, &p);
    if (rc != VIMSCAN_OK) return rc;
    rc = vimscan_host::check_norm_call(n, nullptr, nullptr, grad, launch, p);
    if (rc != VIMSCAN_OK || p.D == 0) return rc;
    NormArgs a = common_args(n, launch, p);
    a.dsum = grad->dsum;
    a.dn = grad->dn;
    a.dx = grad->dx;
    a.dz = grad->dz;
    a.ld_dx = grad->ld_dx;
    a.ld_dz = grad->ld_dz;
    a.dres = grad->dresidual;
    a.dw[0] = grad->dw_post;
    a.dw[1] = grad->dgamma;
    a.dw[2] = grad->dw_pre;
    const bool weights = a.dw[0] || a.dw[1] || a.dw[2];
    a.part = weights ? static_cast<float*>(launch->workspace) : nullptr;
    hipStream_t s = static_cast<hipStream_t>(launch->stream);
    if (!record(launch, 0)) return VIMSCAN_ERR_HIP;
    if (p.wgs > 0) launch_typed(a, p, launch->io_dtype, true, s);
    else if (weights)
        hipLaunchKernelGGL(k_norm_zero, dim3(static_cast<unsigned>((p.D + 63) / 64), 3), dim3(64), 0, s, a);
    if (hipGetLastError() != hipSuccess || !record(launch, 1)) return VIMSCAN_ERR_HIP;
    return VIMSCAN_OK;
}

}  // extern "C"
