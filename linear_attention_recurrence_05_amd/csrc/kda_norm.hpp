// kda_norm.hpp -- what the norm kernels share: rows as 16-byte pieces, and the
// range in which a row's mean of squares is taken as fp32 gives it.
#pragma once

#include "kda_device.hpp"

namespace kda {

// Outside these means of squares (eps included) fp32 has lost squares to
// infinity, or some that count to its lower end, and the row is taken times
// 2^-80 or 2^80.  The sum of its squares is then within 2^103 or 2^67, and the
// mean at least 2^-32 or (eps being at least 2^-149) 2^11.
constexpr float kLeastMean = 0x1p-100f, kMostMean = 0x1.fffffep127f, kDown = 0x1p-80f;

__device__ __forceinline__ bool mean_in_range(float m) { return m >= kLeastMean && m <= kMostMean; }

template <typename E, int VE>
__device__ __forceinline__ void unpack(u32x4 v, float (&x)[VE]) {
    E e[VE];
    *reinterpret_cast<u32x4*>(e) = v;
#pragma unroll
    for (int i = 0; i < VE; ++i) x[i] = to_f32(e[i]);
}
template <typename E, int VE>
__device__ __forceinline__ u32x4 pack_row(const float (&x)[VE]) {
    if constexpr (sizeof(E) == 2)
        return __builtin_bit_cast(u32x4, pack8(f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]}));
    else
        return __builtin_bit_cast(u32x4, f32x4{x[0], x[1], x[2], x[3]});
}
template <typename E, int VE>
__device__ __forceinline__ void store_row(E* p, const float (&x)[VE]) {
    __builtin_nontemporal_store(pack_row<E, VE>(x), reinterpret_cast<u32x4*>(p));
}

// Sigmoid(z) and 1 - Sigmoid(z) = Sigmoid(-z), each without cancellation and
// without an overflow that matters.  For bf16 rows by the hardware's exp2 and
// reciprocal (1 ulp each, |z| 2^-24 from the product: eight instructions, where the
// full-range functions take forty and more and the norms become bound by them).
template <bool FAST>
__device__ __forceinline__ void sigmoids(float z, float& s, float& rest) {
    const float e = FAST ? fast_exp2(-fabsf(z) * kLog2e) : expf(-fabsf(z));
    const float big = FAST ? fast_rcp(1.0f + e) : 1.0f / (1.0f + e), small = e * big;
    s = z >= 0.f ? big : small;
    rest = z >= 0.f ? small : big;
}
template <bool FAST>
__device__ __forceinline__ float sigmoid(float z) {
    return FAST ? fast_rcp(1.0f + fast_exp2(-z * kLog2e)) : 1.0f / (1.0f + expf(-z));
}

// out[e] = sum over i of part[i][e], i = 0 .. n - 1, for e of `width` columns: 64
// columns a workgroup of 1024 threads, in fixed order.  Columns from `first` on go
// to `b`; a null array is not wanted.
__global__ __launch_bounds__(1024) void sum_parts_kernel(const float* __restrict__ part, int n, int width, int first,
                                                         float* __restrict__ a, float* __restrict__ b);

}  // namespace kda
