// Layer norm for AMD MI355X (gfx950): residual add and norm of a row in one pass, and its backward pass
// (include/vimscan.h, vimscan_layernorm_*).

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <iterator>

#include "block_device.h"
#include "block_plan.h"
#include "norm_rows.h"
#include "vimscan.h"

namespace {

using namespace vimscan_dev;
using vimscan_host::kNormBackward;
using vimscan_host::kNormForward;
using vimscan_host::kNormSingles;
using vimscan_host::NormPlan;

struct LayerNormArgs {
    const void* x;
    int64_t ld_x;
    const void* residual;
    const float* weight;
    const float* bias;
    float eps, inv_d;
    int32_t D, once;
    int64_t rows;
    void* sum;
    void* n;
    // backward
    const void* dsum;
    const void* dn;
    void* dx;
    int64_t ld_dx;
    void* dres;
    float* dw[2];   // of weight and bias
    float* part;    // [workgroup][2][D] partial weight gradients, NULL when none is wanted
};

// Outputs of calls that move more than kOnceBytes are written past the caches: there each line throws out another (768 channels bf16,
// us, kept and not: 25216 rows 43.3 and 40.2, 6272 rows 10.5 and 10.3; forward and backward 108.3 and 98.6, 33.4 and 28.8).
// Smaller ones are kept for whoever reads them next.
constexpr int64_t kOnceBytes = int64_t(32) << 20;
template <typename T, typename S>
__device__ __forceinline__ void st_out(bool once, void* base, int64_t at, int D, const float (&v)[S::NV][S::V]) {
    if (once) st_row<T, S, true>(base, at, D, v);
    else st_row<T, S>(base, at, D, v);
}

// A number that every lane of a row has: in a scalar register where registers are short (workgroups of 1024 threads; 4099 x 8192 bf16 forward
// and backward 136 us, 148 in vector registers; 13056 x 1531 fp32, in workgroups of 512, 94 and 92).
template <typename S>
__device__ __forceinline__ float of_row(float v) {
    if constexpr (S::W == 16) return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
    return v;
}

// The row minus its mean, and 1 / sqrt of its variance and eps: the mean first, then the squares about it (in
// registers, a second look costs no memory; the difference of two large sums would cost digits where the mean is large). The mean
// is rounded, which beside a small spread is as much as the output: what is left of it shows in the second look's sum. The norm of an
// element is then s x + y.
template <typename S>
__device__ __forceinline__ float2 center(const LayerNormArgs& a, float (&s)[S::NV][S::V], float2 (*lds)[S::W], int& slot, int wave) {
    float u = 0.0f, t = 0.0f;
#pragma unroll
    for (int k = 0; k < S::NV; ++k)
#pragma unroll
        for (int v = 0; v < S::V; ++v) u += s[k][v];
    row_sum<S::L, S::W>(&u, &t, lds, slot, wave);
    const float mean = of_row<S>(u * a.inv_d);
    u = t = 0.0f;
#pragma unroll
    for (int k = 0; k < S::NV; ++k)
#pragma unroll
        for (int v = 0; v < S::V; ++v) {
            // (channels past the row's are left out)
            s[k][v] = S::channel(k) + (S::kWhole ? 0 : v) < a.D ? s[k][v] - mean : 0.0f;
            u += s[k][v];
            t = fmaf(s[k][v], s[k][v], t);
        }
    row_sum<S::L, S::W>(&u, &t, lds, slot, wave);
    const float left = u * a.inv_d, rho = root_inverse(fmaxf(fmaf(t, a.inv_d, -left * left), 0.0f) + a.eps);
    return make_float2(of_row<S>(rho), of_row<S>(-left * rho));
}

// Forward: s = x + residual, n = (s - mean) rsq(var + eps) weight + bias. Memory bounds it: a row stays in registers from
// its one read to its one write, and the workgroups walk the rows so that the weights are read once per workgroup. 25216 x 768 bf16
// with an fp32 residual (232 MB): 40 us, 5.8 TB/s; 13056 x 1531 fp32 (160 MB, 4-byte accesses) 47 us, VALU busy 52%.
template <typename IO, typename RES, typename S>
__global__ __launch_bounds__(S::kThreads) void k_ln_fwd(LayerNormArgs a) {
    constexpr int NV = S::NV, V = S::V;
    __shared__ float2 lds[2][S::W];
    const int wave = S::wave();
    float w[NV][V], b[NV][V];
    ld_weight<S>(a.weight, a.D, w);
    ld_weight<S>(a.bias, a.D, b);
    int slot = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * S::kRows + S::row(); row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * S::kRows) {
        Raw<IO, V> x[NV];
        Raw<RES, V> r[NV];
        ld_row<IO, S>(a.x, row * a.ld_x, true, a.D, x);
        ld_row<RES, S>(a.residual, row * a.D, a.residual != nullptr, a.D, r);
        settle<IO, S>(a.D, x);
        settle<RES, S>(a.D, r);
        float s[NV][V];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) s[k][v] = x[k].get(v) + r[k].get(v);
        if (a.sum) st_out<RES, S>(a.once, a.sum, row * a.D, a.D, s);
        const float2 c = center<S>(a, s, lds, slot, wave);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) s[k][v] = fmaf(fmaf(s[k][v], c.x, c.y), w[k][v], a.bias ? b[k][v] : 0.0f);
        st_out<IO, S>(a.once, a.n, row * a.D, a.D, s);
    }
}

// Backward: the row's norm again from its inputs (cheaper than saved statistics), then with xh = (s - mean) rho and
// g = dn weight: ds = dsum + rho (g - mean g - xh mean(g xh)); dx = dresidual = ds. The weights' gradients, sums of dn xh
// and dn over the rows, stay with the thread over all its rows, are added up over the workgroup's rows at the end and left
// for k_ln_cols: no atomics, the same bits every time. Memory bounds it: 25216 x 768 bf16 (349 MB) 53 us, 6.5 TB/s (two thirds
// of it reads); 13056 x 1531 fp32 (240 MB) 65 us, VALU busy 64%.
template <typename IO, typename RES, typename S>
__global__ __launch_bounds__(S::kThreads) void k_ln_bwd(LayerNormArgs a) {
    constexpr int NV = S::NV, L = S::L, W = S::W, V = S::V;
    __shared__ float2 lds[2][W];
    const int wave = S::wave();
    // (a workgroup of 1024 threads has 128 registers a thread: there the weight is read again per row)
    constexpr bool kKeep = W < 16 || NV * V < 8;
    float w[NV][V];
    if constexpr (kKeep) ld_weight<S>(a.weight, a.D, w);
    // the weights' gradients: in registers, or each thread's in LDS where those are short and LDS holds them
    constexpr bool kInLds = !kKeep && S::kWidth <= 8192;
    float dw[NV][V], db[NV][V];
    __shared__ __align__(16) float sums[kInLds ? 2 : 1][kInLds ? NV : 1][kInLds ? S::kThreads : 1][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            dw[k][v] = db[k][v] = 0.0f;
            if constexpr (kInLds) sums[0][k][threadIdx.x][v] = sums[1][k][threadIdx.x][v] = 0.0f;
        }
    int slot = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * S::kRows + S::row(); row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * S::kRows) {
        Raw<IO, V> x[NV], dn[NV];
        Raw<RES, V> r[NV], ds[NV];
        ld_row<IO, S>(a.x, row * a.ld_x, true, a.D, x);
        ld_row<RES, S>(a.residual, row * a.D, a.residual != nullptr, a.D, r);
        ld_row<IO, S>(a.dn, row * a.D, a.dn != nullptr, a.D, dn);
        ld_row<RES, S>(a.dsum, row * a.D, a.dsum != nullptr, a.D, ds);
        settle<IO, S>(a.D, x);
        settle<RES, S>(a.D, r);
        settle<IO, S>(a.D, dn);
        settle<RES, S>(a.D, ds);
        float s[NV][V];
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) s[k][v] = x[k].get(v) + r[k].get(v);
        const float2 c = center<S>(a, s, lds, slot, wave);
        if constexpr (!kKeep) ld_weight<S>(a.weight, a.D, w);
        float u = 0.0f, t = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float d = dn[k].get(v), g = d * w[k][v];
                s[k][v] = fmaf(s[k][v], c.x, c.y);
                u += g;
                t = fmaf(g, s[k][v], t);
                if constexpr (kInLds) {
                    sums[0][k][threadIdx.x][v] = fmaf(d, s[k][v], sums[0][k][threadIdx.x][v]);
                    sums[1][k][threadIdx.x][v] += d;
                } else {
                    dw[k][v] = fmaf(d, s[k][v], dw[k][v]);
                    db[k][v] += d;
                }
            }
        row_sum<L, W>(&u, &t, lds, slot, wave);
        u = of_row<S>(u * a.inv_d);
        t = of_row<S>(t * a.inv_d);
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v)
                s[k][v] = fmaf(c.x, fmaf(-s[k][v], t, fmaf(dn[k].get(v), w[k][v], -u)), ds[k].get(v));
        if (a.dx) st_out<IO, S>(a.once, a.dx, row * a.ld_dx, a.D, s);
        if (a.dres) st_out<RES, S>(a.once, a.dres, row * a.D, a.D, s);
    }
    if (!a.part) return;
    float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.D;
    if constexpr (kInLds) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                dw[k][v] = sums[0][k][threadIdx.x][v];
                db[k][v] = sums[1][k][threadIdx.x][v];
            }
    }
    if constexpr (S::kRows == 1) {
        st_row<float, S>(part, 0, a.D, dw);
        st_row<float, S>(part, a.D, a.D, db);
    } else {
        // the rows of a wave, then the workgroup's four waves in their order
        constexpr int kWaves = S::kThreads / 64;
        const int me = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
        __shared__ float col[2][kWaves][NV * V][L];
        auto leave = [&](float (&g)[NV][V], int which) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float p, q;
                    if constexpr (L < 32) {
                        swap16(g[k][v], &p, &q);
                        g[k][v] = p + q;
                    }
                    if constexpr (L < 64) {
                        swap32(g[k][v], &p, &q);
                        g[k][v] = p + q;
                    }
                    if ((threadIdx.x & 63) < L) col[which][me][k * V + v][S::place()] = g[k][v];
                }
        };
        leave(dw, 0);
        leave(db, 1);
        __syncthreads();
        // one channel of one weight per thread and turn
        for (int i = static_cast<int>(threadIdx.x); i < 2 * S::kWidth; i += S::kThreads) {
            const int which = i / S::kWidth, c = i % S::kWidth;
            if (c >= a.D) continue;
            const int v = c % V, at = c / V % L, k = c / V / L;
            float sum = 0.0f;
#pragma unroll
            for (int m = 0; m < kWaves; ++m) sum += col[which][m][k * V + v][at];
            part[which * static_cast<int64_t>(a.D) + c] = sum;
        }
    }
}

// The weight gradients: the workgroups' partial sums, in a fixed order. 512 parts of 2 x 768 or 2 x 1531: 4.8 us, a launch and two
// rounds of loads.
__global__ __launch_bounds__(1024) void k_ln_cols(LayerNormArgs a, int parts) {
    float* dst = a.dw[blockIdx.y];
    if (!dst) return;
    const int c0 = static_cast<int>(blockIdx.x) * kColumns, c = c0 + static_cast<int>(threadIdx.x);
    const float s = column_sum(a.part + static_cast<int64_t>(blockIdx.y) * a.D, parts, 2 * static_cast<int64_t>(a.D), c0, a.D);
    if (threadIdx.x < kColumns && c < a.D) dst[c] = s;
}

// An empty backward pass: weight gradients of zero.
__global__ __launch_bounds__(64) void k_ln_zero(LayerNormArgs a) {
    const int c = static_cast<int>(blockIdx.x) * 64 + static_cast<int>(threadIdx.x);
    if (c < a.D && a.dw[blockIdx.y]) a.dw[blockIdx.y][c] = 0.0f;
}

template <typename IO, typename RES, bool kBack, typename S>
void launch(const LayerNormArgs& a, const NormPlan& p, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.wgs)), block(S::kThreads);
    if constexpr (kBack) {
        hipLaunchKernelGGL((k_ln_bwd<IO, RES, S>), grid, block, 0, s, a);
        if (a.part)
            hipLaunchKernelGGL(k_ln_cols, dim3(static_cast<unsigned>((a.D + kColumns - 1) / kColumns), 2), dim3(1024), 0, s,
                               a, static_cast<int>(grid.x));
    } else {
        hipLaunchKernelGGL((k_ln_fwd<IO, RES, S>), grid, block, 0, s, a);
    }
}

// The first of N spreads that holds the row.
template <typename IO, typename RES, bool kBack, bool kWhole, const NormSpread* kSpreads, size_t N, size_t I = 0>
void launch_first(const LayerNormArgs& a, const NormPlan& p, hipStream_t s) {
    constexpr NormSpread f = kSpreads[I];
    if constexpr (I + 1 < N) {
        if (a.D > f.width()) return launch_first<IO, RES, kBack, kWhole, kSpreads, N, I + 1>(a, p, s);
    }
    launch<IO, RES, kBack, Spread<f.nv, f.lanes, f.waves, f.vec, kWhole>>(a, p, s);
}
template <typename IO, typename RES, bool kWhole>
void launch_vectors(const LayerNormArgs& a, const NormPlan& p, bool back, hipStream_t s) {
    if (back) launch_first<IO, RES, true, kWhole, kNormBackward, std::size(kNormBackward)>(a, p, s);
    else launch_first<IO, RES, false, kWhole, kNormForward, std::size(kNormForward)>(a, p, s);
}
template <bool kBack>
void launch_singles(const LayerNormArgs& a, const NormPlan& p, hipStream_t s) {
    launch_first<float, float, kBack, true, kNormSingles, std::size(kNormSingles)>(a, p, s);
}

// Widths that are no multiple of four: bf16 vectors at any alignment, fp32 single channels (as for the block norm, whose
// launch gives both sides' times).
void launch_typed(const LayerNormArgs& a, const NormPlan& p, int io, bool res_f32, bool back, hipStream_t s) {
    const bool whole = a.D % 4 == 0;
    if (io == VIMSCAN_F32) {
        if (whole) launch_vectors<float, float, true>(a, p, back, s);
        else if (back) launch_singles<true>(a, p, s);
        else launch_singles<false>(a, p, s);
    } else if (res_f32) {
        if (whole) launch_vectors<Bf16, float, true>(a, p, back, s);
        else launch_vectors<Bf16, float, false>(a, p, back, s);
    } else {
        if (whole) launch_vectors<Bf16, Bf16, true>(a, p, back, s);
        else launch_vectors<Bf16, Bf16, false>(a, p, back, s);
    }
}

LayerNormArgs common_args(const vimscan_layernorm* n, const NormPlan& p) {
    LayerNormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = n->x;
    a.ld_x = n->ld_x;
    a.residual = n->residual;
    a.weight = n->weight;
    a.bias = n->bias;
    a.eps = n->eps;
    a.inv_d = 1.0f / static_cast<float>(p.D > 0 ? p.D : 1);
    a.D = static_cast<int32_t>(p.D);
    a.rows = p.rows;
    return a;
}

bool record(const vimscan_launch* l, int k) {
    if (!l->scan_events[0] || !l->scan_events[1]) return true;
    return hipEventRecord(static_cast<hipEvent_t>(l->scan_events[k]), static_cast<hipStream_t>(l->stream)) == hipSuccess;
}

}  // namespace

extern "C" {

int vimscan_layernorm_fwd(const vimscan_layernorm* p, void* sum, void* n, const vimscan_launch* launch) {
    if (!p || !launch) return VIMSCAN_ERR_NULL;
    NormPlan pl;
    int rc = vimscan_host::make_layernorm_plan(launch, false, &pl);
    if (rc != VIMSCAN_OK) return rc;
    rc = vimscan_host::check_layernorm_call(p, sum, n, nullptr, launch, pl);
    if (rc != VIMSCAN_OK || pl.wgs == 0) return rc;
    LayerNormArgs a = common_args(p, pl);
    a.sum = sum;
    a.n = n;
    const int64_t e = launch->io_dtype == VIMSCAN_F32 ? 4 : 2, re = p->res_dtype == VIMSCAN_F32 ? 4 : 2, size = pl.rows * pl.D;
    a.once = size * (2 * e + (p->residual ? re : 0) + (sum ? re : 0)) > kOnceBytes;
    hipStream_t s = static_cast<hipStream_t>(launch->stream);
    if (!record(launch, 0)) return VIMSCAN_ERR_HIP;
    launch_typed(a, pl, launch->io_dtype, p->res_dtype == VIMSCAN_F32, false, s);
    if (hipGetLastError() != hipSuccess || !record(launch, 1)) return VIMSCAN_ERR_HIP;
    return VIMSCAN_OK;
}

int vimscan_layernorm_bwd(const vimscan_layernorm* p, const vimscan_layernorm_grad* grad, const vimscan_launch* launch) {
    if (!p || !grad || !launch) return VIMSCAN_ERR_NULL;
    NormPlan pl;
    int rc = vimscan_host::make_layernorm_plan(launch, true, &pl);
    if (rc != VIMSCAN_OK) return rc;
    rc = vimscan_host::check_layernorm_call(p, nullptr, nullptr, grad, launch, pl);
    if (rc != VIMSCAN_OK || pl.D == 0) return rc;
    LayerNormArgs a = common_args(p, pl);
    a.dsum = grad->dsum;
    a.dn = grad->dn;
    a.dx = grad->dx;
    a.ld_dx = grad->ld_dx;
    a.dres = grad->dresidual;
    const int64_t e = launch->io_dtype == VIMSCAN_F32 ? 4 : 2, re = p->res_dtype == VIMSCAN_F32 ? 4 : 2, size = pl.rows * pl.D;
    a.once = size * (3 * e + (p->residual ? re : 0) + (grad->dsum ? re : 0) + (grad->dresidual ? re : 0)) > kOnceBytes;
    a.dw[0] = grad->dweight;
    a.dw[1] = grad->dbias;
    const bool weights = a.dw[0] || a.dw[1];
    a.part = weights ? static_cast<float*>(launch->workspace) : nullptr;
    hipStream_t s = static_cast<hipStream_t>(launch->stream);
    if (!record(launch, 0)) return VIMSCAN_ERR_HIP;
    if (pl.wgs > 0) launch_typed(a, pl, launch->io_dtype, p->res_dtype == VIMSCAN_F32, true, s);
    else if (weights)
        hipLaunchKernelGGL(k_ln_zero, dim3(static_cast<unsigned>((pl.D + 63) / 64), 2), dim3(64), 0, s, a);
    if (hipGetLastError() != hipSuccess || !record(launch, 1)) return VIMSCAN_ERR_HIP;
    return VIMSCAN_OK;
}

}  // extern "C"
