// kda_linear_frag.hpp -- matrix operands of the linear-attention kernels: eight
// values a lane, bf16 for one 16x16x32 MFMA or fp32 for eight 16x16x4 ones, so
// that one kernel text serves both element types.
#pragma once

#include "kda_device.hpp"

namespace kda {

// Eight values of a lane, of 32 along a contraction: lane group g = lane / 16
// holds eight of them (which ones is the caller's choice, the same for both
// operands).
template <typename E> struct Frag;
template <> struct Frag<bf16> { bf16x8 v; };
template <> struct Frag<float> { f32x4 lo, hi; };

__device__ __forceinline__ f32x4 mma(const Frag<bf16>& a, const Frag<bf16>& b, f32x4 c) {
    return mma_bf16_k32(a.v, b.v, c);
}
__device__ __forceinline__ f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = mma_f32_k4(a.lo[i], b.lo[i], c);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = mma_f32_k4(a.hi[i], b.hi[i], c);
    return c;
}

template <typename E> __device__ __forceinline__ Frag<E> to_frag(f32x4 lo, f32x4 hi);
template <> __device__ __forceinline__ Frag<bf16> to_frag<bf16>(f32x4 lo, f32x4 hi) { return {pack8(lo, hi)}; }
template <> __device__ __forceinline__ Frag<float> to_frag<float>(f32x4 lo, f32x4 hi) { return {lo, hi}; }

__device__ __forceinline__ void to_f32(const Frag<bf16>& a, f32x4& lo, f32x4& hi) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo[i] = (float)a.v[i];
        hi[i] = (float)a.v[4 + i];
    }
}
__device__ __forceinline__ void to_f32(const Frag<float>& a, f32x4& lo, f32x4& hi) {
    lo = a.lo;
    hi = a.hi;
}

// Eight consecutive elements of a row in LDS (16-byte aligned).
template <typename E> __device__ __forceinline__ Frag<E> row_frag(const E* p);
template <> __device__ __forceinline__ Frag<bf16> row_frag<bf16>(const bf16* p) {
    return {*reinterpret_cast<const bf16x8*>(p)};
}
template <> __device__ __forceinline__ Frag<float> row_frag<float>(const float* p) {
    return {*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4)};
}

// Lane (j, g) = 16 g + j: column `col(j)` of rows 4 g + {0..3} and 16 + 4 g +
// {0..3} of a [32][ld] tile in LDS, where col(j) = c0 + step (j / 4) + j % 4.
// bf16: two transposing reads, for which a lane names row j / 4 and column
// group j % 4 of its group's 4 x 16 block.
template <typename E>
__device__ __forceinline__ Frag<E> col_frag(const E* s, int ld, int c0, int step, int j, int g) {
    Frag<E> f;
    if constexpr (sizeof(E) == 2) {
        typedef __attribute__((address_space(3))) i16x4 lds4;
        const E* p = s + (4 * g + (j >> 2)) * ld + c0 + step * (j & 3);
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 16 * ld));
        f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
        const E* p = s + 4 * g * ld + c0 + step * (j >> 2) + (j & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f.lo[i] = p[i * ld];
            f.hi[i] = p[(16 + i) * ld];
        }
    }
    return f;
}

// x in fp32 as a sum of N terms of E: two bf16 hold 16 of its bits, three all 24,
// so a product with a bf16 operand keeps that accuracy; one fp32 is x itself.
template <int N>
__device__ __forceinline__ void split(f32x4 lo, f32x4 hi, Frag<bf16> (&out)[N]) {
#pragma unroll
    for (int s = 0; s < N; ++s) {
        out[s] = to_frag<bf16>(lo, hi);
        f32x4 a, b;
        to_f32(out[s], a, b);
        lo -= a;
        hi -= b;
    }
}
__device__ __forceinline__ void split(f32x4 lo, f32x4 hi, Frag<float> (&out)[1]) { out[0] = {lo, hi}; }

// A matrix operand as the sum of N bf16 terms (of decreasing size: each is what
// the ones before it leave, rounded).  Three hold an fp32 value's 24 bits.
template <int N> struct Terms { bf16x8 t[N]; };

// The products of the terms down to 2^-24 of the largest, small ones first: of
// two operands of three terms six of the nine, which is 2.7 times faster than
// the same contraction in 16x16x4 fp32 MFMAs.
template <int N, int M>
__device__ __forceinline__ f32x4 mma(const Terms<N>& a, const Terms<M>& b, f32x4 c) {
#pragma unroll
    for (int s = N + M - 2 < 2 ? N + M - 2 : 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (s - i >= 0 && s - i < M) c = mma_bf16_k32(a.t[i], b.t[s - i], c);
    return c;
}

template <int N>
__device__ __forceinline__ Terms<N> to_terms(f32x4 lo, f32x4 hi) {
    Terms<N> out;
#pragma unroll
    for (int s = 0; s < N; ++s) {
        out.t[s] = pack8(lo, hi);
        if (s + 1 < N) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] -= (float)out.t[s][i];
                hi[i] -= (float)out.t[s][4 + i];
            }
        }
    }
    return out;
}

template <int N>
__device__ __forceinline__ void to_f32(const Terms<N>& a, f32x4& lo, f32x4& hi) {
    lo = hi = zero4();
#pragma unroll
    for (int s = N - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] += (float)a.t[s][i];
            hi[i] += (float)a.t[s][4 + i];
        }
}

// row_frag and col_frag of a tile kept as N bf16 planes `plane` elements apart.
template <int N>
__device__ __forceinline__ Terms<N> row_terms(const bf16* p, int plane) {
    Terms<N> out;
#pragma unroll
    for (int s = 0; s < N; ++s) out.t[s] = row_frag<bf16>(p + s * plane).v;
    return out;
}
template <int N>
__device__ __forceinline__ Terms<N> col_terms(const bf16* p, int plane, int ld, int c0, int step, int j, int g) {
    Terms<N> out;
#pragma unroll
    for (int s = 0; s < N; ++s) out.t[s] = col_frag<bf16>(p + s * plane, ld, c0, step, j, g).v;
    return out;
}

}  // namespace kda
