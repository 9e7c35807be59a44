// Block norm for AMD MI355X (gfx950): gate, post-norm, scaled residual and pre-norm of a row in one
// pass, and its backward pass (include/vimscan.h, vimscan_norm_*).

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <iterator>

#include "block_device.h"
#include "block_plan.h"
#include "vimscan.h"

namespace {

using namespace vimscan_dev;
using vimscan_host::kNormBackward;
using vimscan_host::kNormForward;
using vimscan_host::kNormSingles;
using vimscan_host::NormPlan;
using vimscan_host::NormSpread;

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

// Sum over L = 16, 32 or 64 lanes of a wave, on the vector unit alone: within rows of 16 lanes by lane
// permutations of a quad and mirrors, across rows by lane swaps. Every lane gets the same bits.
template <int kCtrl>
__device__ __forceinline__ float add_dpp(float v) {
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), kCtrl, 0xf, 0xf, false));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
    v = add_dpp<0xB1>(v);   // lane ^ 1
    v = add_dpp<0x4E>(v);   // lane ^ 2
    v = add_dpp<0x141>(v);  // half row mirrored
    v = add_dpp<0x140>(v);  // row mirrored
    float p, q;
    if constexpr (L > 16) {
        swap16(v, &p, &q);
        v = p + q;
    }
    if constexpr (L > 32) {
        swap32(v, &p, &q);
        v = p + q;
    }
    return v;
}

// Sums of two values over the W waves of a row, in the waves' order. Calls alternate between two slots:
// a slot is written again only after the barrier of the call between, which every wave reaches after
// its reads of that slot, so one barrier a call is enough.
template <int L, int W>
__device__ __forceinline__ void row_sum(float* u, float* v, float2 (*lds)[W], int& slot, int wave) {
    *u = lanes_sum<L>(*u);
    *v = lanes_sum<L>(*v);
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
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }

// A row spread over L lanes of a wave (W = 1) or W whole waves (L = 64), each lane NV vectors of V channels
// (NormSpread, whose tables say which widths take which). kWhole: the width is a multiple of V; otherwise a row's last vector is
// read as the row's last V elements and shifted into place once every load of the row has been issued
// (settle), and written by elements.
template <int NV_, int L_, int W_, int V_, bool kWhole_> struct Spread {
    static constexpr int NV = NV_, L = L_, W = W_, V = V_;
    static constexpr bool kWhole = kWhole_;
    static constexpr NormSpread kSpread{NV, L, W, V};
    static constexpr int kThreads = kSpread.threads(), kRows = kSpread.rows();
    static constexpr int kWidth = static_cast<int>(kSpread.width());
    static_assert(W == 1 || L == 64, "part of a wave, or whole waves");
    static_assert(V == 4 || kWhole, "single channels are always whole");
    // the thread's place in its row, and its row among the workgroup's
    __device__ __forceinline__ static int place() { return static_cast<int>(threadIdx.x) % (L * W); }
    __device__ __forceinline__ static int row() {
        const int r = static_cast<int>(threadIdx.x) / (L * W);
        return L == 64 ? __builtin_amdgcn_readfirstlane(r) : r;
    }
    __device__ __forceinline__ static int wave() { return W > 1 ? __builtin_amdgcn_readfirstlane(place() / 64) : 0; }
    __device__ __forceinline__ static int channel(int k) { return (k * (L * W) + place()) * V; }
};

template <typename T, typename S>
__device__ __forceinline__ void ld_row(const void* base, int64_t at, bool there, int D, Raw<T, S::V> (&o)[S::NV]) {
    constexpr int V = S::V;
    const IoElem<T>* p = static_cast<const IoElem<T>*>(base) + at;
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
        const int c = S::channel(k);
        o[k].zero();
        if constexpr (S::kWhole) {
            if (there && c < D) load_any(o[k], p + c);
        } else if (D >= V) {
            if (there && c < D) load_any(o[k], p + min(c, D - V));
        } else {
            if (there && c < D) load_some(o[k], p + c, D - c);
        }
    }
}
template <typename T, typename S>
__device__ __forceinline__ void settle(int D, Raw<T, S::V> (&o)[S::NV]) {
    constexpr int V = S::V;
    if constexpr (!S::kWhole) {
        if (D < V) return;
#pragma unroll
        for (int k = 0; k < S::NV; ++k) {
            const int c = S::channel(k);
            shift_down(o[k], c < D ? max(c + V - D, 0) : 0);
        }
    }
}
template <typename T, typename S>
__device__ __forceinline__ void st_row(void* base, int64_t at, int D, const float (&v)[S::NV][S::V]) {
    constexpr int V = S::V;
    IoElem<T>* p = static_cast<IoElem<T>*>(base) + at;
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
        const int c = S::channel(k);
        Raw<T, V> o;
        o.set(v[k]);
        if constexpr (S::kWhole) {
            if (c < D) store_any(o, p + c);
        } else {
            if (c + V <= D) store_any(o, p + c);
            else if (c < D) store_some(o, p + c, D - c);
        }
    }
}
// A weight's channels (1 where the weight is absent).
template <typename S>
__device__ __forceinline__ void ld_weight(const float* w, int D, float (&o)[S::NV][S::V]) {
    constexpr int V = S::V;
    Raw<float, V> r[S::NV];
    ld_row<float, S>(w, 0, w != nullptr, D, r);
    settle<float, S>(D, r);
#pragma unroll
    for (int k = 0; k < S::NV; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) o[k][v] = w ? r[k].get(v) : 1.0f;
}

// Forward: v = x (silu(z)), q = v rsq(mean v^2 + eps) w_post, s = residual + gamma q, n = s rsq(mean s^2 +
// eps) w_pre. Memory bounds it: a row stays in registers from its one read to its one write, and the
// workgroups walk the rows so that the weights are read once per workgroup and not per row. Measured: 25216
// x 768 bf16 with fp32 residuals 50 us (271 MB, 5.4 TB/s), 4099 x 8192 all bf16 49 us (269 MB, 5.5 TB/s),
// 13056 x 1531 fp32 48 us with a gate and no pre-norm (5.0 TB/s); a copy of 256 MiB reaches 5.4 TB/s. 1000 x 16384
// bf16 51 us (4.5 TB/s); past 16384 channels 72 to 216 registers spill: 500 x 32768 119 us (1.9 TB/s).
template <typename IO, typename RES, typename S>
__global__ __launch_bounds__(S::kThreads) void k_norm_fwd(NormArgs a) {
    constexpr int NV = S::NV, L = S::L, W = S::W, V = S::V;
    __shared__ float2 lds[2][W];
    const int wave = S::wave();
    float wp[NV][V], ga[NV][V], wn[NV][V];
    ld_weight<S>(a.w_post, a.D, wp);
    ld_weight<S>(a.gamma, a.D, ga);
    ld_weight<S>(a.w_pre, a.D, wn);
    int slot = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * S::kRows + S::row(); row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * S::kRows) {
        Raw<IO, V> x[NV], z[NV];
        Raw<RES, V> r[NV];
        ld_row<IO, S>(a.x, row * a.ld_x, true, a.D, x);
        ld_row<IO, S>(a.z, row * a.ld_z, a.z != nullptr, a.D, z);
        ld_row<RES, S>(a.residual, row * a.D, a.residual != nullptr, a.D, r);
        settle<IO, S>(a.D, x);
        settle<IO, S>(a.D, z);
        settle<RES, S>(a.D, r);
        float s[NV][V];
        float ss = 0.0f, none = 0.0f;
        // (the stages that are there or not are chosen outside the element loops: one branch a row)
        auto all = [](auto&& f) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) f(k, v);
        };
        all([&](int k, int v) { s[k][v] = x[k].get(v); });
        if (a.z && !a.after) all([&](int k, int v) { s[k][v] *= silu(z[k].get(v)); });
        all([&](int k, int v) { ss = fmaf(s[k][v], s[k][v], ss); });
        float rho = 1.0f;
        if (a.w_post) {
            row_sum<L, W>(&ss, &none, lds, slot, wave);
            rho = fast_rsq(fmaf(ss, a.inv_d, a.eps));
        }
        ss = none = 0.0f;
        all([&](int k, int v) { s[k][v] *= rho * wp[k][v]; });
        if (a.after) all([&](int k, int v) { s[k][v] *= silu(z[k].get(v)); });
        all([&](int k, int v) {
            s[k][v] = fmaf(s[k][v], ga[k][v], r[k].get(v));
            ss = fmaf(s[k][v], s[k][v], ss);
        });
        if (a.sum) st_row<RES, S>(a.sum, row * a.D, a.D, s);
        if (!a.w_pre) continue;
        row_sum<L, W>(&ss, &none, lds, slot, wave);
        rho = fast_rsq(fmaf(ss, a.inv_d, a.eps));
        all([&](int k, int v) { s[k][v] *= rho * wn[k][v]; });
        st_row<IO, S>(a.n, row * a.D, a.D, s);
    }
}

// Backward: the row's stages again from its inputs (reading them costs less than saved statistics and
// intermediates would), then the gradients against them. With g = dn w_pre: ds' = dsum + rho2 g - s rho2^3
// mean(g s); the post-norm's likewise; the gate's through silu' = sg (1 + z (1 - sg)). The weights' gradients
// of a thread's channels stay with the thread over all its rows, are added up over the workgroup's rows at
// the end and left for k_norm_cols: no atomics, the same bits every time. Memory bounds it up to 4096 channels:
// 25216 x 768 bf16 83 us (426 MB, 5.1 TB/s), 25216 x 1024 123 us (568 MB, 4.6 TB/s, one wave a SIMD: 256 registers),
// 13056 x 1531 fp32 84 us (400 MB, 4.7 TB/s). Past them a thread's registers are short (128 with 16 waves). LDS holds
// the weights' gradients up to 8192 channels: 4099 x 8192 all bf16 174 us (537 MB, 3.1 TB/s) against 243 with all in
// registers and spilled; widths there that are no multiple of 4 still spill 18 to 41 (4099 x 8191 bf16 294 us). Past
// 8192 every form spills 227 to 1229 registers, and scratch memory bounds it: 1000 x 16384 bf16 405 us (360 MB),
// 500 x 32768 882 us.
template <typename IO, typename RES, typename S>
__global__ __launch_bounds__(S::kThreads) void k_norm_bwd(NormArgs a) {
    constexpr int NV = S::NV, L = S::L, W = S::W, V = S::V;
    __shared__ float2 lds[2][W];
    const int wave = S::wave();
    // (a workgroup of 1024 threads has 128 registers a thread: there the weights are read again per stage)
    constexpr bool kKeep = W < 16 || NV * V < 8;
    float wp[NV][V], ga[NV][V], wn[NV][V];
    if constexpr (kKeep) {
        ld_weight<S>(a.w_post, a.D, wp);
        ld_weight<S>(a.gamma, a.D, ga);
        ld_weight<S>(a.w_pre, a.D, wn);
    }
    // the weights' gradients: in registers, or each thread's in LDS where those are short and LDS holds them
    constexpr bool kInLds = !kKeep && S::kWidth <= 8192;
    float dwp[NV][V], dga[NV][V], dwn[NV][V];
    __shared__ __align__(16) float sums[kInLds ? 3 : 1][kInLds ? NV : 1][kInLds ? S::kThreads : 1][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            dwp[k][v] = dga[k][v] = dwn[k][v] = 0.0f;
            if constexpr (kInLds) sums[0][k][threadIdx.x][v] = sums[1][k][threadIdx.x][v] = sums[2][k][threadIdx.x][v] = 0.0f;
        }
    auto add = [&](int which, float (&g)[NV][V], int k, int v, float a, float b) {
        if constexpr (kInLds) sums[which][k][threadIdx.x][v] = fmaf(a, b, sums[which][k][threadIdx.x][v]);
        else g[k][v] = fmaf(a, b, g[k][v]);
    };
    int slot = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * S::kRows + S::row(); row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * S::kRows) {
        Raw<IO, V> x[NV], z[NV], dn[NV];
        Raw<RES, V> r[NV], ds[NV];
        ld_row<IO, S>(a.x, row * a.ld_x, true, a.D, x);
        ld_row<IO, S>(a.z, row * a.ld_z, a.z != nullptr, a.D, z);
        ld_row<RES, S>(a.residual, row * a.D, a.residual != nullptr, a.D, r);
        ld_row<IO, S>(a.dn, row * a.D, a.dn != nullptr, a.D, dn);
        ld_row<RES, S>(a.dsum, row * a.D, a.dsum != nullptr, a.D, ds);
        settle<IO, S>(a.D, x);
        settle<IO, S>(a.D, z);
        settle<RES, S>(a.D, r);
        settle<IO, S>(a.D, dn);
        settle<RES, S>(a.D, ds);
        auto read_first = [&] {   // the weights of the stages up to the sum
            if constexpr (!kKeep) {
                ld_weight<S>(a.w_post, a.D, wp);
                ld_weight<S>(a.gamma, a.D, ga);
            }
        };
        auto read_last = [&] {    // that of the pre-norm
            if constexpr (!kKeep) ld_weight<S>(a.w_pre, a.D, wn);
        };
        // val: the post-norm's input; s: the sum
        float val[NV][V], s[NV][V];
        float u = 0.0f, t = 0.0f;
        auto all = [](auto&& f) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) f(k, v);
        };
        all([&](int k, int v) { val[k][v] = x[k].get(v); });
        if (a.z && !a.after) all([&](int k, int v) { val[k][v] *= silu(z[k].get(v)); });
        all([&](int k, int v) { u = fmaf(val[k][v], val[k][v], u); });
        float rho1 = 1.0f, rho2 = 0.0f, k2 = 0.0f;
        if (a.w_post) {
            row_sum<L, W>(&u, &t, lds, slot, wave);
            rho1 = fast_rsq(fmaf(u, a.inv_d, a.eps));
        }
        u = t = 0.0f;
        read_first();
        all([&](int k, int v) { s[k][v] = val[k][v] * rho1 * wp[k][v]; });
        if (a.after) all([&](int k, int v) { s[k][v] *= silu(z[k].get(v)); });
        all([&](int k, int v) { s[k][v] = fmaf(s[k][v], ga[k][v], r[k].get(v)); });
        if (a.dn) {
            read_last();
            all([&](int k, int v) {
                u = fmaf(s[k][v], s[k][v], u);
                t = fmaf(dn[k].get(v) * wn[k][v], s[k][v], t);
            });
            row_sum<L, W>(&u, &t, lds, slot, wave);
            rho2 = fast_rsq(fmaf(u, a.inv_d, a.eps));
            k2 = t * a.inv_d * rho2 * rho2 * rho2;
            read_last();
            // from here s is the gradient of the sum
            all([&](int k, int v) {
                const float g = dn[k].get(v) * rho2;
                add(2, dwn, k, v, g, s[k][v]);
                s[k][v] = ds[k].get(v) + fmaf(g, wn[k][v], -s[k][v] * k2);
            });
        } else {
            all([&](int k, int v) { s[k][v] = ds[k].get(v); });
        }
        u = t = 0.0f;
        read_first();
        // gradients of gamma and w_post; dq: of the post-norm's output
        if (a.after) {
            all([&](int k, int v) {
                const float gs = silu(z[k].get(v)) * s[k][v], vr = val[k][v] * rho1;
                const float dq = gs * ga[k][v];
                add(1, dga, k, v, vr * wp[k][v], gs);
                add(0, dwp, k, v, dq, vr);
                u = fmaf(dq * wp[k][v], val[k][v], u);
            });
        } else {
            all([&](int k, int v) {
                const float vr = val[k][v] * rho1, dq = s[k][v] * ga[k][v];
                add(1, dga, k, v, vr * wp[k][v], s[k][v]);
                add(0, dwp, k, v, dq, vr);
                u = fmaf(dq * wp[k][v], val[k][v], u);
            });
        }
        if (a.dres) st_row<RES, S>(a.dres, row * a.D, a.D, s);
        float k1 = 0.0f;
        if (a.w_post) {
            row_sum<L, W>(&u, &t, lds, slot, wave);
            k1 = u * a.inv_d * rho1 * rho1 * rho1;
        }
        read_first();
        // gradient of the post-norm's input: rho1 dq w_post - val k1 (dq itself without w_post)
        float dz[NV][V];
        if (!a.z) {
            all([&](int k, int v) { s[k][v] = fmaf(rho1 * s[k][v] * ga[k][v], wp[k][v], -val[k][v] * k1); });
        } else if (a.after) {
            all([&](int k, int v) {
                const float zv = z[k].get(v), sg = sigmoid(zv), dp = s[k][v] * ga[k][v], rw = rho1 * wp[k][v];
                dz[k][v] = dp * (val[k][v] * rw) * (sg * fmaf(zv, 1.0f - sg, 1.0f));
                s[k][v] = fmaf(dp * (zv * sg), rw, -val[k][v] * k1);
            });
        } else {
            all([&](int k, int v) {
                const float zv = z[k].get(v), sg = sigmoid(zv);
                const float dv = fmaf(rho1 * s[k][v] * ga[k][v], wp[k][v], -val[k][v] * k1);
                dz[k][v] = dv * x[k].get(v) * (sg * fmaf(zv, 1.0f - sg, 1.0f));
                s[k][v] = dv * (zv * sg);
            });
        }
        if (a.dx) st_row<IO, S>(a.dx, row * a.ld_dx, a.D, s);
        if (a.dz) st_row<IO, S>(a.dz, row * a.ld_dz, a.D, dz);
    }
    if (!a.part) return;
    float* part = a.part + static_cast<int64_t>(blockIdx.x) * 3 * a.D;
    if constexpr (kInLds) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                dwp[k][v] = sums[0][k][threadIdx.x][v];
                dga[k][v] = sums[1][k][threadIdx.x][v];
                dwn[k][v] = sums[2][k][threadIdx.x][v];
            }
    }
    if constexpr (S::kRows == 1) {
        st_row<float, S>(part, 0, a.D, dwp);
        st_row<float, S>(part, a.D, a.D, dga);
        st_row<float, S>(part, 2 * a.D, a.D, dwn);
    } else {
        // the rows of a wave, then the workgroup's four waves in their order
        constexpr int kWaves = S::kThreads / 64;
        const int w = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
        __shared__ float col[3][kWaves][NV * V][L];
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
                    if ((threadIdx.x & 63) < L) col[which][w][k * V + v][S::place()] = g[k][v];
                }
        };
        leave(dwp, 0);
        leave(dga, 1);
        leave(dwn, 2);
        __syncthreads();
        // one channel of one weight per thread and turn
        for (int n = static_cast<int>(threadIdx.x); n < 3 * S::kWidth; n += S::kThreads) {
            const int which = n / S::kWidth, c = n % S::kWidth;
            if (c >= a.D) continue;
            const int v = c % V, at = c / V % L, k = c / V / L;
            float sum = 0.0f;
#pragma unroll
            for (int t = 0; t < kWaves; ++t) sum += col[which][t][k * V + v][at];
            part[which * static_cast<int64_t>(a.D) + c] = sum;
        }
    }
}

// The weight gradients: the workgroups' partial sums, in a fixed order. Latency bounds it: 4.7 us for 512
// partials of 3 x 768.
__global__ __launch_bounds__(1024) void k_norm_cols(NormArgs a, int parts) {
    float* dst = a.dw[blockIdx.y];
    if (!dst) return;
    const int c0 = static_cast<int>(blockIdx.x) * kColumns, c = c0 + static_cast<int>(threadIdx.x);
    const float s = column_sum(a.part + static_cast<int64_t>(blockIdx.y) * a.D, parts, 3 * static_cast<int64_t>(a.D), c0, a.D);
    if (threadIdx.x < kColumns && c < a.D) dst[c] = s;
}

template <typename IO, typename RES, bool kBack, typename S>
void launch(const NormArgs& a, const NormPlan& p, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.wgs)), block(S::kThreads);
    if constexpr (kBack) {
        hipLaunchKernelGGL((k_norm_bwd<IO, RES, S>), grid, block, 0, s, a);
        if (a.part)
            hipLaunchKernelGGL(k_norm_cols, dim3(static_cast<unsigned>((a.D + kColumns - 1) / kColumns), 3), dim3(1024), 0, s,
                               a, static_cast<int>(grid.x));
    } else {
        hipLaunchKernelGGL((k_norm_fwd<IO, RES, S>), grid, block, 0, s, a);
    }
}

// The first of N spreads that holds the row.
template <typename IO, typename RES, bool kBack, bool kWhole, const NormSpread* kSpreads, size_t N, size_t I = 0>
void launch_first(const NormArgs& a, const NormPlan& p, hipStream_t s) {
    constexpr NormSpread f = kSpreads[I];
    if constexpr (I + 1 < N) {
        if (a.D > f.width()) return launch_first<IO, RES, kBack, kWhole, kSpreads, N, I + 1>(a, p, s);
    }
    launch<IO, RES, kBack, Spread<f.nv, f.lanes, f.waves, f.vec, kWhole>>(a, p, s);
}
template <typename IO, typename RES, bool kWhole>
void launch_vectors(const NormArgs& a, const NormPlan& p, bool back, hipStream_t s) {
    if (back) launch_first<IO, RES, true, kWhole, kNormBackward, std::size(kNormBackward)>(a, p, s);
    else launch_first<IO, RES, false, kWhole, kNormForward, std::size(kNormForward)>(a, p, s);
}
template <bool kBack>
void launch_singles(const NormArgs& a, const NormPlan& p, hipStream_t s) {
    launch_first<float, float, kBack, true, kNormSingles, std::size(kNormSingles)>(a, p, s);
}

// Widths that are no multiple of four: in bf16 vectors at any alignment are faster than single channels
// (13056 x 1531, all stages: 75 us against 120 forward, 119 against 190 backward; 54 and 92 at 1536), in fp32, where
// a single channel is a full access, they are slower (105 against 74 us, 161 against 132).
void launch_typed(const NormArgs& a, const NormPlan& p, int io, bool back, hipStream_t s) {
    const bool whole = a.D % 4 == 0;
    if (io == VIMSCAN_F32) {
        if (whole) launch_vectors<float, float, true>(a, p, back, s);
        else if (back) launch_singles<true>(a, p, s);
        else launch_singles<false>(a, p, s);
    } else if (a.res_f32) {
        if (whole) launch_vectors<Bf16, float, true>(a, p, back, s);
        else launch_vectors<Bf16, float, false>(a, p, back, s);
    } else {
        if (whole) launch_vectors<Bf16, Bf16, true>(a, p, back, s);
        else launch_vectors<Bf16, Bf16, false>(a, p, back, s);
    }
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
