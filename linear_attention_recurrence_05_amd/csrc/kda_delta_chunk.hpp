// kda_delta_chunk.hpp -- the chunk form of the gated delta rule, shared by the
// prefill and the gradients.  With C = 64 tokens of a chunk, S the state before
// them, G_i the sum of the chunk's log-decays up to token i, D_ij = exp(G_i - G_j)
// for i >= j and N = (K K^T) * D below the diagonal:
//   E  = (I + N diag(beta))^{-1} (V - e^G K S)        e_t of every token
//   O  = scale (e^G Q S + ((Q K^T) * D) diag(beta) E)
//   S' = e^{G_C} S + K^T diag(e^{G_C - G} beta) E
// Every exponent is <= 0 for g <= 0; G is summed in 64 bits and its differences are
// taken of two fp32 parts, so that a decay behind a far smaller one keeps its digits.
//
// What does not depend on the state, the inverse and the pairs' weights, is made
// first for all chunks at once (delta_pairs_kernel) and left in the workspace as
// the matrix operands that the state's chain reads, 16 bytes a lane.
#pragma once

#include "kda_delta.hpp"
#include "kda_device.hpp"
#include "kda_linear_frag.hpp"

namespace kda {

constexpr int kDeltaChunk = 64, kDeltaTiles = kDeltaChunk / 16;

// A chunk's block in the workspace.  An operand of one 16x16x32 MFMA is 64 lanes
// of 16 bytes; lane (j, g) holds row (or column) j, and along the contraction
// tokens 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3 of 32 tokens.  Of the lower
// triangular matrices six operands of 16 rows x 32 are not zero (lower()), of
// their transposes another six (upper()); each is N terms one after the other.
//   inv   lower, 3 terms   rows of (I + N diag(beta))^{-1}
//   pair  lower, NP terms  columns (queries) of scale ((Q K^T) * D diag(beta))^T
//   row   [64] e^{G_i}, [64] e^{G_C - G_j} beta_j, [64] e^{G_C - G_j}, [64] beta_j,
//         then e^{G_C} as a factor and what its rounding left out, relative to it
// and, for the gradients (BACK),
//   row   from [272] on p_i = scale q_i . k_i, from [336] on beta_i p_i
//   invt  upper, 3 terms   rows of ((I + diag(beta) N)^{-1})^T
//   pairt upper, 3 terms   rows (keys) of scale ((Q K^T) * D)^T
// all four of them without their diagonal (1, p_i beta_i, 1 and p_i), which the
// chains add: what a token takes from older tokens and later ones stays apart from
// what it has of itself, as dg needs it (kda_delta_backward.hip).
constexpr int kFragBytes = 1024;
__host__ __device__ constexpr int lower(int tile, int half) { return tile < 2 ? tile : 2 * tile - 2 + half; }
__host__ __device__ constexpr int upper(int tile, int half) { return tile < 2 ? 2 * tile + half : 2 + tile; }
template <int NP, bool BACK>
struct DeltaBlock {
    static constexpr int inv = 0, pair = inv + 18 * kFragBytes, row = pair + 6 * NP * kFragBytes;
    static constexpr int invt = row + (BACK ? 1600 : 1088), pairt = invt + 18 * kFragBytes;
    static constexpr int bytes = BACK ? pairt + 18 * kFragBytes : invt;
};
enum DeltaRow { kRowGrow = 0, kRowWrite = 64, kRowEnd = 128, kRowBeta = 192, kRowDecay = 256,   // floats from `row`
                kRowSelf = 272, kRowBetaSelf = 336 };

// Chunks c0 .. c1 - 1 of every sequence, block ((b H + h) (c1 - c0) + c - c0).
struct DeltaPairs {
    const void *q, *k;
    const float *g, *beta;
    float scale;
    StateIO S;          // its check tables
    const int* lens;
    char* blocks;
    int B, T, H, Hk, dk, c0, c1;
    bool is_bf16;
};
size_t delta_block_bytes(bool is_bf16, bool back);
hipError_t launch_delta_pairs(const DeltaPairs& a, bool back, hipStream_t stream);

__device__ __forceinline__ int seq_len(const int* lens, int b, int T) { return lens ? min(max(lens[b], 0), T) : T; }

// The factor e^{G_C} of a chunk, given as the block's pair: what each rounding
// leaves out goes into the next factor, so the factors' product stays the
// product however many chunks there are.
struct ChunkDecay {
    float left = 0.f;
    __device__ float operator()(float f, float rest) {
        const float d = f * (rest + left), got = f + d;
        left = got > 1e-30f ? (d - (got - f)) * fast_rcp(got) : 0.f;
        return got;
    }
};

// Workgroup x of units x tiles: a unit's tiles follow each other on one XCD
// (workgroups go round the eight), whose L2 then serves what they read in common.
__device__ __forceinline__ void unit_tile(int x, int units, int tiles, int& unit, int& tile) {
    const int whole = units / 8 * 8, rest = x - whole * tiles;
    unit = rest < 0 ? x / 8 / tiles * 8 + x % 8 : whole + rest / tiles;
    tile = rest < 0 ? x / 8 % tiles : rest % tiles;
}

// Two fp32 values rounded to bf16 in one word, which then hold what that leaves:
// the halves of the word are fp32 values as they stand.
__device__ __forceinline__ uint32_t take_pair(float& a, float& b) {
    const uint32_t w = __builtin_bit_cast(uint32_t, pack2(a, b));
    a -= __builtin_bit_cast(float, w << 16);
    b -= __builtin_bit_cast(float, w & 0xffff0000u);
    return w;
}
// to_terms with both values of a word taken from it (44 instructions for three terms
// of eight values, where a conversion of each value alone makes 60).
template <int N>
__device__ __forceinline__ Terms<N> split_terms(f32x4 lo, f32x4 hi) {
    Terms<N> out;
#pragma unroll
    for (int s = 0; s < N; ++s) {
        if (s + 1 < N) {
            float a[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = take_pair(a[2 * i], a[2 * i + 1]);
            out.t[s] = __builtin_bit_cast(bf16x8, w);
            lo = f32x4{a[0], a[1], a[2], a[3]};
            hi = f32x4{a[4], a[5], a[6], a[7]};
        } else {
            out.t[s] = pack8(lo, hi);
        }
    }
    return out;
}

// Eight consecutive elements of a row as loaded, 16 bytes of bf16 or 32 of fp32.
template <typename E> struct Raw;
template <> struct Raw<bf16> { u32x4 v; };
template <> struct Raw<float> { u32x4 v, w; };
template <typename E> __device__ __forceinline__ Raw<E> raw_load(Rsrc r, int off);
template <> __device__ __forceinline__ Raw<bf16> raw_load<bf16>(Rsrc r, int off) { return {buf_load<u32x4>(r, off)}; }
template <> __device__ __forceinline__ Raw<float> raw_load<float>(Rsrc r, int off) {
    return {buf_load<u32x4>(r, off), buf_load<u32x4>(r, off + 16)};
}
__device__ __forceinline__ Terms<1> raw_terms(const Raw<bf16>& r) { return {{__builtin_bit_cast(bf16x8, r.v)}}; }
__device__ __forceinline__ Terms<3> raw_terms(const Raw<float>& r) {
    return split_terms<3>(__builtin_bit_cast(f32x4, r.v), __builtin_bit_cast(f32x4, r.w));
}

// A 16-byte piece of a row to LDS: bf16 as it is, four fp32 values as their three
// terms, `plane` elements apart.
template <typename E>
__device__ __forceinline__ void put_piece(bf16* dst, int plane, u32x4 v, bool on = true) {
    if constexpr (sizeof(E) == 2) {
        if (on) *reinterpret_cast<u32x4*>(dst) = v;
    } else {
        f32x4 x = __builtin_bit_cast(f32x4, v);
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            const bf16x4 h = pack4(x);
            *reinterpret_cast<bf16x4*>(dst + s * plane) = h;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] -= (float)h[i];
        }
    }
}

// Four values as N terms to LDS, `plane` elements apart.
template <int N>
__device__ __forceinline__ void put_words(bf16* dst, int plane, f32x4 x) {
    float a[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
    for (int s = 0; s < N; ++s) {
        u32x2 w;
        w[0] = take_pair(a[0], a[1]);
        w[1] = take_pair(a[2], a[3]);
        *reinterpret_cast<u32x2*>(dst + s * plane) = w;
    }
}

// Stores of what another launch reads, past what L2 holds: they leave its lines to
// the operands that the tiles of a head share (the gradients' sweeps of B1 H32 T4096
// d128 take 381 us with them and 389 without, in turn; such loads, 521).
__device__ __forceinline__ void buf_stream_u32x4(Rsrc r, int off, u32x4 x) {
    __builtin_amdgcn_raw_buffer_store_b128(x, r, off, 0, 2);
}

// Four elements from a buffer, and eight streamed to it.
template <typename E>
__device__ __forceinline__ f32x4 buf_load4(Rsrc r, int off) {
    if constexpr (sizeof(E) == 4) {
        return __builtin_bit_cast(f32x4, buf_load<u32x4>(r, off));
    } else {
        const bf16x4 v = __builtin_bit_cast(bf16x4, buf_load<u32x2>(r, off));
        return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]};
    }
}
template <typename E>
__device__ __forceinline__ void buf_stream8(Rsrc r, int off, f32x4 lo, f32x4 hi) {
    if constexpr (sizeof(E) == 2) {
        buf_stream_u32x4(r, off, __builtin_bit_cast(u32x4, pack8(lo, hi)));
    } else {
        buf_stream_u32x4(r, off, __builtin_bit_cast(u32x4, lo));
        buf_stream_u32x4(r, off + 16, __builtin_bit_cast(u32x4, hi));
    }
}
__device__ __forceinline__ void store8(bf16* p, f32x4 lo, f32x4 hi) { *reinterpret_cast<bf16x8*>(p) = pack8(lo, hi); }
__device__ __forceinline__ void store8(float* p, f32x4 lo, f32x4 hi) {
    reinterpret_cast<f32x4*>(p)[0] = lo;
    reinterpret_cast<f32x4*>(p)[1] = hi;
}

// LDS of one wave: its writes are there for its reads.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// An offset past any buffer's end, also some KB further: such loads give zeros and
// such stores are dropped.
constexpr int kOffPast = -(1 << 16);

// Elements from one row of DK channels to the next in LDS: 16 banks on (of 64), so
// that the four rows of which col_terms reads every other 8 bytes with 16 lanes lie
// beside each other (with DK + 8 elements they met in the same banks four times).
template <int DK>
constexpr int kRowLd = DK == 32 ? 32 : DK + 32;

// mma, but of two operands of two terms without the product of both second ones
// (2^-18 of the largest).
template <int N, int M>
__device__ __forceinline__ f32x4 mma_top(const Terms<N>& a, const Terms<M>& b, f32x4 c) {
    if constexpr (N == 2 && M == 2) {
        c = mma_bf16_k32(a.t[0], b.t[1], c);
        c = mma_bf16_k32(a.t[1], b.t[0], c);
        return mma_bf16_k32(a.t[0], b.t[0], c);
    } else {
        return mma(a, b, c);
    }
}
// mma, but the largest product apart from the others: a sum of many products then
// rounds once, not six times, at its full size for each of them, and what it is added
// to once in all.  In the gradients' sweeps (fp32 B3 H8 T333, errors in norm): dg 6.0e-7
// -> 3.5e-7, dbeta 3.4e-7 -> 2.1e-7, dS0 4.4e-7 -> 1.5e-7, at the same time.
struct Sum2 {
    f32x4 big = zero4(), small = zero4();
    template <int N, int M>
    __device__ void add(const Terms<N>& a, const Terms<M>& b) {
#pragma unroll
        for (int s = N + M - 2 < 2 ? N + M - 2 : 2; s > 0; --s)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (s - i >= 0 && s - i < M) small = mma_bf16_k32(a.t[i], b.t[s - i], small);
        big = mma_bf16_k32(a.t[0], b.t[0], big);
    }
    __device__ f32x4 sum() const { return big + small; }
};
template <int N, int M>
__device__ __forceinline__ Terms<N> first_terms(const Terms<M>& a) {
    Terms<N> out;
#pragma unroll
    for (int i = 0; i < N; ++i) out.t[i] = a.t[i];
    return out;
}
// An operand kept in LDS as N fragments `step` bytes apart.
template <int N>
__device__ __forceinline__ Terms<N> frag_terms(const char* p, int step = kFragBytes) {
    Terms<N> out;
#pragma unroll
    for (int i = 0; i < N; ++i) out.t[i] = *reinterpret_cast<const bf16x8*>(p + i * step + lane_id() * 16);
    return out;
}
// N fragments of a block in the workspace (off kOffPast: zeros).
template <int N>
__device__ __forceinline__ Terms<N> load_terms(Rsrc r, int off) {
    Terms<N> out;
#pragma unroll
    for (int i = 0; i < N; ++i) out.t[i] = __builtin_bit_cast(bf16x8, buf_load<u32x4>(r, off + i * kFragBytes + lane_id() * 16));
    return out;
}
template <int CTRL>
__device__ __forceinline__ float dpp_move(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xF, 0xF, false));
}
// A tile of 16 x 16 (rows 4 g + i of column j, an accumulator's layout) as N terms
// to its half of an operand in LDS: half 0 is tokens 4 g .., half 1 16 + 4 g ..
template <int N>
__device__ __forceinline__ void put_half(char* frag, int half, f32x4 x) {
#pragma unroll
    for (int s = 0; s < N; ++s) {
        float a[4] = {x[0], x[1], x[2], x[3]};
        u32x2 w;
        w[0] = take_pair(a[0], a[1]);
        w[1] = take_pair(a[2], a[3]);
        *reinterpret_cast<u32x2*>(frag + s * kFragBytes + lane_id() * 16 + half * 8) = w;
        x = f32x4{a[0], a[1], a[2], a[3]};
    }
}
// The sums of x over the 16 lanes of a group, of x[i] in the lanes whose j % 4 is i:
// an accumulator's rows summed over its columns.
__device__ __forceinline__ float row_sums(f32x4 x, int j) {
    constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kRor4 = 0x124, kRor8 = 0x128;   // DPP controls
    const bool odd = j & 1, high = j & 2;
    const float a = (odd ? x[1] : x[0]) + dpp_move<kXor1>(odd ? x[0] : x[1]);
    const float b = (odd ? x[3] : x[2]) + dpp_move<kXor1>(odd ? x[2] : x[3]);
    float c = (high ? b : a) + dpp_move<kXor2>(high ? a : b);
    c += dpp_move<kRor4>(c);
    return c + dpp_move<kRor8>(c);
}
// What row_sums gives a lane the row of.
__device__ __forceinline__ float lane_row(f32x4 x, int j) {
    const float a = j & 1 ? x[1] : x[0], b = j & 1 ? x[3] : x[2];
    return j & 2 ? b : a;
}
// Column j of rows 4 g .. 4 g + 3 of a [16][ld] tile kept as N
// bf16 planes in LDS.
template <int N>
__device__ __forceinline__ f32x4 col4(const bf16* s, int plane, int ld, int j, int g) {
    typedef __attribute__((address_space(3))) i16x4 lds4;
    f32x4 x = zero4();
#pragma unroll
    for (int n = N - 1; n >= 0; --n) {
        const bf16* p = s + n * plane + (4 * g + (j >> 2)) * ld + 4 * (j & 3);
        const bf16x4 v = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] += (float)v[i];
    }
    return x;
}

}  // namespace kda
