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
template <typename IO>
__device__ __forceinline__ float ld_res(const NormArgs& a, const void* p, int64_t k) {
    return a.res_f32 ? ld<float>(p, k) : ld<IO>(p, k);
}
template <typename IO>
__device__ __forceinline__ void st_res(const NormArgs& a, void* p, int64_t k, float v) {
    if (a.res_f32) st<float>(p, k, v);
    else st<IO>(p, k, v);
}

// Sum over the 256 threads of a workgroup, in a fixed order.
__device__ __forceinline__ float wg_sum(float v, float* lds) {
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__device__ __forceinline__ float sigmoid(float v) { return fast_rcp(1.0f + fast_exp2(-v * kLog2e)); }

// One channel's way through the row: what the later stages need of it.
struct Chan {
    float x, gate, v, q, p, s;
};
template <typename IO>
__device__ __forceinline__ void stage_v(const NormArgs& a, int64_t row, int c, Chan& o) {
    o.x = ld<IO>(a.x, row * a.ld_x + c);
    o.gate = 1.0f;
    if (a.z) {
        const float z = ld<IO>(a.z, row * a.ld_z + c);
        o.gate = z * sigmoid(z);
    }
    o.v = a.after ? o.x : o.x * o.gate;
}
template <typename IO>
__device__ __forceinline__ void stage_s(const NormArgs& a, int64_t row, int c, float rho1, Chan& o) {
    o.q = a.w_post ? o.v * rho1 * a.w_post[c] : o.v;
    o.p = a.after ? o.q * o.gate : o.q;
    o.s = a.gamma ? o.p * a.gamma[c] : o.p;
    if (a.residual) o.s += ld_res<IO>(a, a.residual, row * a.D + c);
}

// A workgroup per row; every stage reads the row again.
template <typename IO>
__global__ __launch_bounds__(256) void k_norm_fwd(NormArgs a) {
    __shared__ float lds[4];
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        Chan o;
        float rho1 = 1.0f, rho2 = 0.0f;
        if (a.w_post) {
            float s = 0.0f;
            for (int c = threadIdx.x; c < a.D; c += 256) {
                stage_v<IO>(a, row, c, o);
                s = fmaf(o.v, o.v, s);
            }
            rho1 = fast_rsq(fmaf(wg_sum(s, lds), a.inv_d, a.eps));
        }
        if (a.w_pre) {
            float s = 0.0f;
            for (int c = threadIdx.x; c < a.D; c += 256) {
                stage_v<IO>(a, row, c, o);
                stage_s<IO>(a, row, c, rho1, o);
                s = fmaf(o.s, o.s, s);
            }
            rho2 = fast_rsq(fmaf(wg_sum(s, lds), a.inv_d, a.eps));
        }
        for (int c = threadIdx.x; c < a.D; c += 256) {
            stage_v<IO>(a, row, c, o);
            stage_s<IO>(a, row, c, rho1, o);
            if (a.sum) st_res<IO>(a, a.sum, row * a.D + c, o.s);
            if (a.w_pre) st<IO>(a.n, row * a.D + c, o.s * rho2 * a.w_pre[c]);
        }
    }
}

template <typename IO>
__global__ __launch_bounds__(256) void k_norm_bwd(NormArgs a) {
    __shared__ float lds[4];
    float* part = a.part ? a.part + static_cast<int64_t>(blockIdx.x) * 3 * a.D : nullptr;
    if (part)
        for (int c = threadIdx.x; c < 3 * a.D; c += 256) part[c] = 0.0f;
    __syncthreads();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        Chan o;
        float rho1 = 1.0f, rho2 = 0.0f, k2 = 0.0f;
        if (a.w_post) {
            float s = 0.0f;
            for (int c = threadIdx.x; c < a.D; c += 256) {
                stage_v<IO>(a, row, c, o);
                s = fmaf(o.v, o.v, s);
            }
            rho1 = fast_rsq(fmaf(wg_sum(s, lds), a.inv_d, a.eps));
        }
        if (a.dn) {
            float s = 0.0f, t = 0.0f;
            for (int c = threadIdx.x; c < a.D; c += 256) {
                stage_v<IO>(a, row, c, o);
                stage_s<IO>(a, row, c, rho1, o);
                s = fmaf(o.s, o.s, s);
                t = fmaf(ld<IO>(a.dn, row * a.D + c) * a.w_pre[c], o.s, t);
            }
            rho2 = fast_rsq(fmaf(wg_sum(s, lds), a.inv_d, a.eps));
            k2 = wg_sum(t, lds) * a.inv_d * rho2 * rho2 * rho2;
        }
        // gradient of s, then of q (the post-norm's output)
        auto grads = [&](int c, float& ds, float& dp, float& dq) {
            stage_v<IO>(a, row, c, o);
            stage_s<IO>(a, row, c, rho1, o);
            ds = a.dsum ? ld_res<IO>(a, a.dsum, row * a.D + c) : 0.0f;
            if (a.dn) ds += rho2 * ld<IO>(a.dn, row * a.D + c) * a.w_pre[c] - o.s * k2;
            dp = a.gamma ? ds * a.gamma[c] : ds;
            dq = a.after ? dp * o.gate : dp;
        };
        float k1 = 0.0f;
        if (a.w_post) {
            float t = 0.0f;
            for (int c = threadIdx.x; c < a.D; c += 256) {
                float ds, dp, dq;
                grads(c, ds, dp, dq);
                t = fmaf(dq * a.w_post[c], o.v, t);
            }
            k1 = wg_sum(t, lds) * a.inv_d * rho1 * rho1 * rho1;
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.D; c += 256) {
            float ds, dp, dq;
            grads(c, ds, dp, dq);
            const float dn = a.dn ? ld<IO>(a.dn, row * a.D + c) : 0.0f;
            const float dv = a.w_post ? rho1 * dq * a.w_post[c] - o.v * k1 : dq;
            const float zv = a.z ? ld<IO>(a.z, row * a.ld_z + c) : 0.0f;
            if (a.dres) st_res<IO>(a, a.dres, row * a.D + c, ds);
            if (a.dx) st<IO>(a.dx, row * a.ld_dx + c, a.after ? dv : dv * o.gate);
            if (a.dz) {
                const float sg = sigmoid(zv);
                const float slope = sg * fmaf(zv, 1.0f - sg, 1.0f);
                st<IO>(a.dz, row * a.ld_dz + c, (a.after ? dp * o.q : dv * o.x) * slope);
            }
            if (part) {
                part[c] += dq * o.v * rho1;
                part[a.D + c] += o.p * ds;
                part[2 * a.D + c] += dn * o.s * rho2;
            }
        }
        __syncthreads();
    }
}

// The weight gradients: the workgroups' partial sums in their order.
__global__ __launch_bounds__(64) void k_norm_cols(NormArgs a, int parts) {
    const int c = static_cast<int>(blockIdx.x) * 64 + static_cast<int>(threadIdx.x);
    float* dst = a.dw[blockIdx.y];
    if (c >= a.D || !dst) return;
    float s = 0.0f;
    for (int k = 0; k < parts; ++k) s += a.part[(static_cast<int64_t>(k) * 3 + blockIdx.y) * a.D + c];
    dst[c] = s;
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
    const dim3 grid(static_cast<unsigned>(p.wgs));
    if (launch->io_dtype == VIMSCAN_F32) hipLaunchKernelGGL(k_norm_fwd<float>, grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL(k_norm_fwd<Bf16>, grid, dim3(256), 0, s, a);
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
    if (p.wgs > 0) {
        const dim3 grid(static_cast<unsigned>(p.wgs));
        if (launch->io_dtype == VIMSCAN_F32) hipLaunchKernelGGL(k_norm_bwd<float>, grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL(k_norm_bwd<Bf16>, grid, dim3(256), 0, s, a);
    }
    if (weights) {
        const dim3 grid(static_cast<unsigned>((p.D + 63) / 64), 3);
        hipLaunchKernelGGL(k_norm_cols, grid, dim3(64), 0, s, a, static_cast<int>(p.wgs));
    }
    if (hipGetLastError() != hipSuccess || !record(launch, 1)) return VIMSCAN_ERR_HIP;
    return VIMSCAN_OK;
}

}  // extern "C"
