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
// without an overflow that matters.
__device__ __forceinline__ void sigmoids(float z, float& s, float& rest) {
    const float e = expf(-fabsf(z)), big = 1.0f / (1.0f + e), small = e * big;
    s = z >= 0.f ? big : small;
    rest = z >= 0.f ? small : big;
}

}  // namespace kda
