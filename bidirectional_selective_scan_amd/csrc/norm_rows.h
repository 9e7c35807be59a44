// Rows of norms in registers: how a row is spread over lanes and waves, its loads, stores and sums (blocknorm.hip, layernorm.hip).
#ifndef VIMSCAN_NORM_ROWS_H
#define VIMSCAN_NORM_ROWS_H

#include <hip/hip_runtime.h>

#include <cstdint>

#include "block_device.h"
#include "block_plan.h"

namespace vimscan_dev {

using vimscan_host::NormSpread;

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

// 1 / sqrt(v). The hardware's takes subnormal numbers, which a small eps alone may leave, for 0.
__device__ __forceinline__ float root_inverse(float v) {
    const bool tiny = v < 0x1p-126f;
    return fast_rsq(tiny ? v * 0x1p24f : v) * (tiny ? 0x1p12f : 1.0f);
}

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
// kOnce: past the caches (the lines are not kept).
template <typename T, typename S, bool kOnce = false>
__device__ __forceinline__ void st_row(void* base, int64_t at, int D, const float (&v)[S::NV][S::V]) {
    constexpr int V = S::V;
    IoElem<T>* p = static_cast<IoElem<T>*>(base) + at;
#pragma unroll
    for (int k = 0; k < S::NV; ++k) {
        const int c = S::channel(k);
        Raw<T, V> o;
        o.set(v[k]);
        if constexpr (S::kWhole) {
            if (c < D) store_any<kOnce>(o, p + c);
        } else {
            if (c + V <= D) store_any<kOnce>(o, p + c);
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

}  // namespace vimscan_dev

#endif  // VIMSCAN_NORM_ROWS_H
