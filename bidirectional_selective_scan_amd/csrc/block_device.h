// Device helpers shared by the recurrent block's kernels (gated.hip, blocknorm.hip).
#ifndef VIMSCAN_BLOCK_DEVICE_H
#define VIMSCAN_BLOCK_DEVICE_H

#include <hip/hip_runtime.h>

#include <cstdint>

namespace vimscan_dev {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Bf16 {};  // tag for bf16 io

template <typename IO> struct IoOf;
template <> struct IoOf<float> { using elem = float; };
template <> struct IoOf<Bf16> { using elem = uint16_t; };
template <typename IO> using IoElem = typename IoOf<IO>::elem;

__device__ __forceinline__ float fast_exp2(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float fast_log2(float v) { return __builtin_amdgcn_logf(v); }
__device__ __forceinline__ float fast_rcp(float v) { return __builtin_amdgcn_rcpf(v); }
__device__ __forceinline__ float fast_sqrt(float v) { return __builtin_amdgcn_sqrtf(v); }
__device__ __forceinline__ float fast_rsq(float v) { return __builtin_amdgcn_rsqf(v); }

// bf16 from fp32, to nearest even (the hardware conversion, two at a time).
__device__ __forceinline__ uint16_t bf16_bits(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
using F32x2 = float __attribute__((ext_vector_type(2)));
using Bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((F32x2{lo, hi}), Bf16x2));
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// V consecutive elements as they are in memory: one load of 2 to 16 bytes.
// The address is a multiple of the load's size.
template <typename IO, int V> struct Raw;
template <> struct Raw<Bf16, 1> {
    uint16_t w;
    __device__ __forceinline__ void load(const void* p) { w = *static_cast<const uint16_t*>(p); }
    __device__ __forceinline__ void zero() { w = 0; }
    __device__ __forceinline__ float get(int) const { return __uint_as_float(static_cast<uint32_t>(w) << 16); }
    __device__ __forceinline__ void set(const float* v) { w = bf16_bits(v[0]); }
    __device__ __forceinline__ void store(void* p) const { *static_cast<uint16_t*>(p) = w; }
};
template <> struct Raw<Bf16, 2> {
    uint32_t w;
    __device__ __forceinline__ void load(const void* p) { w = *static_cast<const uint32_t*>(p); }
    __device__ __forceinline__ void zero() { w = 0; }
    __device__ __forceinline__ float get(int k) const { return k ? bf16_hi(w) : bf16_lo(w); }
    __device__ __forceinline__ void set(const float* v) { w = bf16_pair(v[0], v[1]); }
    __device__ __forceinline__ void store(void* p) const { *static_cast<uint32_t*>(p) = w; }
};
template <> struct Raw<Bf16, 4> {
    uint2 w;
    __device__ __forceinline__ void load(const void* p) { w = *static_cast<const uint2*>(p); }
    __device__ __forceinline__ void zero() { w = make_uint2(0, 0); }
    __device__ __forceinline__ float get(int k) const {
        const uint32_t u = k < 2 ? w.x : w.y;
        return (k & 1) ? bf16_hi(u) : bf16_lo(u);
    }
    __device__ __forceinline__ void set(const float* v) { w = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])); }
    __device__ __forceinline__ void store(void* p) const { *static_cast<uint2*>(p) = w; }
};
template <> struct Raw<float, 1> {
    float w;
    __device__ __forceinline__ void load(const void* p) { w = *static_cast<const float*>(p); }
    __device__ __forceinline__ void zero() { w = 0.0f; }
    __device__ __forceinline__ float get(int) const { return w; }
    __device__ __forceinline__ void set(const float* v) { w = v[0]; }
    __device__ __forceinline__ void store(void* p) const { *static_cast<float*>(p) = w; }
};
template <> struct Raw<float, 2> {
    float2 w;
    __device__ __forceinline__ void load(const void* p) { w = *static_cast<const float2*>(p); }
    __device__ __forceinline__ void zero() { w = make_float2(0, 0); }
    __device__ __forceinline__ float get(int k) const { return k ? w.y : w.x; }
    __device__ __forceinline__ void set(const float* v) { w = make_float2(v[0], v[1]); }
    __device__ __forceinline__ void store(void* p) const { *static_cast<float2*>(p) = w; }
};
template <> struct Raw<float, 4> {
    float4 w;
    __device__ __forceinline__ void load(const void* p) { w = *static_cast<const float4*>(p); }
    __device__ __forceinline__ void zero() { w = make_float4(0, 0, 0, 0); }
    __device__ __forceinline__ float get(int k) const { return k == 0 ? w.x : k == 1 ? w.y : k == 2 ? w.z : w.w; }
    __device__ __forceinline__ void set(const float* v) { w = make_float4(v[0], v[1], v[2], v[3]); }
    __device__ __forceinline__ void store(void* p) const { *static_cast<float4*>(p) = w; }
};

// The same from and to any element address: the hardware takes a wide access at any alignment (the
// unaligned access mode of the HSA target), which memcpy tells the compiler.
template <typename IO, int V>
__device__ __forceinline__ void load_any(Raw<IO, V>& r, const IoElem<IO>* p) { __builtin_memcpy(&r, p, sizeof(r)); }
template <typename IO, int V>
__device__ __forceinline__ void store_any(const Raw<IO, V>& r, IoElem<IO>* p) { __builtin_memcpy(p, &r, sizeof(r)); }
// The first n < V elements.
template <typename IO, int V>
__device__ __forceinline__ void load_some(Raw<IO, V>& r, const IoElem<IO>* p, int n) {
    IoElem<IO> e[V];
#pragma unroll
    for (int k = 0; k < V; ++k) e[k] = k < n ? p[k] : IoElem<IO>(0);
    __builtin_memcpy(&r, e, sizeof(r));
}
// Elements n.. move to 0.., zeros behind them.
__device__ __forceinline__ void shift_down(Raw<Bf16, 4>& r, int n) {
    uint64_t w;
    __builtin_memcpy(&w, &r, 8);
    w >>= 16 * n;
    __builtin_memcpy(&r, &w, 8);
}
__device__ __forceinline__ void shift_down(Raw<float, 4>& r, int n) {
    const float4 w = r.w;
    r.w.x = n == 0 ? w.x : n == 1 ? w.y : n == 2 ? w.z : w.w;
    r.w.y = n == 0 ? w.y : n == 1 ? w.z : n == 2 ? w.w : 0.0f;
    r.w.z = n == 0 ? w.z : n == 1 ? w.w : 0.0f;
    r.w.w = n == 0 ? w.w : 0.0f;
}
template <typename IO, int V>
__device__ __forceinline__ void store_some(const Raw<IO, V>& r, IoElem<IO>* p, int n) {
    IoElem<IO> e[V];
    __builtin_memcpy(e, &r, sizeof(r));
#pragma unroll
    for (int k = 0; k < V; ++k)
        if (k < n) p[k] = e[k];
}

// Every lane's pair: the values of the even and the odd row of 16 lanes, or of the lower and the
// upper 32 lanes.
__device__ __forceinline__ void swap16(float v, float* even, float* odd) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    *even = __uint_as_float(r[0]);
    *odd = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap32(float v, float* lo, float* hi) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    *lo = __uint_as_float(r[0]);
    *hi = __uint_as_float(r[1]);
}

// Sum of column c0 + (lane of 16) over the rows of part, width elements apart, by a workgroup of 1024: each
// thread takes every 64th row of its column, then its wave's four row groups and the 16 waves are added, in a
// fixed order. The result is in threads 0..15 (0 in a column past cols). 16 columns to a workgroup: a few
// hundred rows of some hundred columns spread over dozens of workgroups, a few loads per thread.
constexpr int kColumns = 16;
__device__ __forceinline__ float column_sum(const float* part, int64_t rows, int64_t width, int c0, int cols) {
    __shared__ float lds[16][kColumns];
    const int tid = static_cast<int>(threadIdx.x), c = c0 + (tid & 15);
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int64_t k = tid >> 4; k < rows; k += 64) s += part[k * width + c];
    }
    float p, q;
    swap16(s, &p, &q);
    swap32(p + q, &p, &q);
    if ((tid & 63) < 16) lds[tid >> 6][tid & 15] = p + q;
    __syncthreads();
    s = 0.0f;
    if (tid < 16)
        for (int k = 0; k < 16; ++k) s += lds[k][tid];
    return s;
}

}  // namespace vimscan_dev

#endif  // VIMSCAN_BLOCK_DEVICE_H
