// kda_delta_pairs.hip -- the parts of the gated delta rule's chunks that do not
// depend on the state (kda_delta_chunk.hpp): the inverse of the triangular system
// and the weights of pairs of tokens, as matrix operands in the workspace.
//
// One wave per chunk and head.  K K^T and Q K^T by MFMA with the decays applied
// in the accumulators.  The inverse: the two 16 x 16 blocks on the diagonal by
// substitution, a column a lane (stable for any beta in [0, 2] and keys of length
// 1, where a series in powers of N is not: repeated keys make its terms grow to
// thousands before they cancel), and the block below as -T22 A21 T11 in fp32 MFMA.
#include <algorithm>

#include "kda_delta_chunk.hpp"

namespace kda {

constexpr int kPairWaves = 4;
constexpr int kPairLd = 36;   // floats of a row of the 32 x 32 matrices in LDS

// Waves of a launch: more chunks loop.
constexpr long long kPairUnits = 1LL << 22;

// x of lane `from`, a double as two words
__device__ __forceinline__ double shfl_up_d(double x, int by) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __shfl_up((uint32_t)u, by), hi = __shfl_up((uint32_t)(u >> 32), by);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

template <typename E, int DK, int NP, bool BACK>
__global__ __launch_bounds__(kPairWaves * 64) void delta_pairs_kernel(DeltaPairs p) {
    using Blk = DeltaBlock<NP, BACK>;
    constexpr int C = kDeltaChunk, KM = DK / 32, NE = sizeof(E) == 2 ? 1 : 3, LD = kPairLd;
    __shared__ __align__(16) float s_a[kPairWaves][C * LD];                    // A, later its inverse
    __shared__ __align__(16) float s_b[kPairWaves][BACK ? C * LD : 4];        // the other system's
    __shared__ double s_G[kPairWaves][C];
    __shared__ float s_beta[kPairWaves][C];
    const int wave = wave_id(), lane = lane_id(), j = lane & 15, g = lane >> 4, W = p.c1 - p.c0;
    const long long all = (long long)p.B * W * p.H;
    for (long long at = (long long)blockIdx.x * kPairWaves + wave; at < all; at += (long long)gridDim.x * kPairWaves) {
        const int h = (int)(at % p.H), c = p.c0 + (int)(at / p.H % W), b = (int)(at / p.H / W);
        const int n = seq_len(p.lens, b, p.T), t0 = c * C, rows = min(C, n - t0);
        if (rows <= 0 || p.S.skip(b)) continue;                                // uniform over the wave
        char* blk = p.blocks + (((size_t)b * p.H + h) * W + (c - p.c0)) * Blk::bytes;
        // ---- decays and strengths
        const size_t gate = ((size_t)b * p.T + t0) * p.H + h;
        const int t = lane & 31;
        double G = 0;
        float beta = 0.f;
        if (t < rows) {
            G = (double)log_decay(p.g[gate + (size_t)t * p.H]);
            beta = p.beta[gate + (size_t)t * p.H];
        }
#pragma unroll
        for (int o = 1; o < C; o <<= 1) {
            const double up = shfl_up_d(G, o);
            if (t >= o) G += up;
        }
        float* A = s_a[wave];
        if (lane < C) {
            s_G[wave][t] = G;
            s_beta[wave][t] = beta;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const double GC = s_G[wave][C - 1];
        if (lane < C) {
            float* row = reinterpret_cast<float*>(blk + Blk::row);
            const float end = expf((float)(GC - G));
            row[t] = expf((float)G);
            row[C + t] = end * beta;
            if (t == 0) {
                const double f = exp(GC);
                const float ff = (float)f;
                row[2 * C] = ff;
                row[2 * C + 1] = f > 1e-30 ? (float)((f - (double)ff) / f) : 0.f;
            }
            if constexpr (BACK) {
                float* more = reinterpret_cast<float*>(blk + Blk::more);
                more[t] = end;
                more[C + t] = beta;
            }
        }
        // ---- K K^T and (K Q^T): rows are keys, columns the later token
        const int hk = h / (p.H / p.Hk), ld = p.Hk * DK * (int)sizeof(E);
        const size_t base = (((size_t)b * p.T + t0) * p.Hk + hk) * DK;
        const uint32_t bytes = (uint32_t)((rows - 1) * ld + DK * (int)sizeof(E));
        const Rsrc rk = make_rsrc((const E*)p.k + base, bytes), rq = make_rsrc((const E*)p.q + base, bytes);
        f32x4 kk[3], kq[3], qk[3];                                            // tiles (0,0), (0,1), (1,1): key, later
#pragma unroll
        for (int i = 0; i < 3; ++i) kk[i] = kq[i] = qk[i] = zero4();
#pragma unroll
        for (int m = 0; m < KM; ++m) {
            Terms<NE> x[2], y[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int off = 16 * q + j < rows ? (16 * q + j) * ld + (32 * m + 8 * g) * (int)sizeof(E) : kOffPast;
                x[q] = raw_terms(raw_load<E>(rk, off));
                y[q] = raw_terms(raw_load<E>(rq, off));
            }
            kk[0] = mma(x[0], x[0], kk[0]);
            kk[1] = mma(x[0], x[1], kk[1]);
            kk[2] = mma(x[1], x[1], kk[2]);
            kq[0] = mma(x[0], y[0], kq[0]);
            kq[1] = mma(x[0], y[1], kq[1]);
            kq[2] = mma(x[1], y[1], kq[2]);
            if constexpr (BACK) {
                qk[0] = mma(y[0], x[0], qk[0]);                                // rows: queries, columns: keys
                qk[1] = mma(y[1], x[0], qk[1]);
                qk[2] = mma(y[1], x[1], qk[2]);
            }
        }
        // ---- decays: key 16 a + 4 g + i, later token 16 b + j
        f32x4 bk[2];
        double Gk[2][4], Gl[2];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            Gl[a] = s_G[wave][16 * a + j];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                Gk[a][i] = s_G[wave][16 * a + 4 * g + i];
                bk[a][i] = s_beta[wave][16 * a + 4 * g + i];
            }
        }
        f32x4 P[3], Dt[3];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int d = j - 4 * g - i;                                       // later - key within a diagonal tile
            const float d00 = expf((float)fmin(Gl[0] - Gk[0][i], 0.0)), d01 = expf((float)fmin(Gl[1] - Gk[0][i], 0.0)),
                        d11 = expf((float)fmin(Gl[1] - Gk[1][i], 0.0));
            P[0][i] = d >= 0 ? p.scale * d00 * bk[0][i] * kq[0][i] : 0.f;
            P[1][i] = p.scale * d01 * bk[0][i] * kq[1][i];
            P[2][i] = d >= 0 ? p.scale * d11 * bk[1][i] * kq[2][i] : 0.f;
            Dt[0][i] = d > 0 ? d00 * kk[0][i] : 0.f;                           // N[later][key]
            Dt[1][i] = d01 * kk[1][i];
            Dt[2][i] = d > 0 ? d11 * kk[2][i] : 0.f;
        }
        const Terms<NP> w0 = to_terms<NP>(P[0], zero4()), w1 = to_terms<NP>(P[1], P[2]);
#pragma unroll
        for (int s = 0; s < NP; ++s) {
            bf16x8* dst = reinterpret_cast<bf16x8*>(blk + Blk::pair + 2 * s * kFragBytes) + lane;
            dst[0] = w0.t[s];
            dst[kFragBytes / 16] = w1.t[s];
        }
        if constexpr (BACK) {                                                  // row: key j, contraction: queries
            f32x4 X[3];
            // query 16 a + 4 g + i, key 16 b + j: later is the row here
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = 4 * g + i - j;
                X[0][i] = d >= 0 ? p.scale * expf((float)fmin(Gk[0][i] - Gl[0], 0.0)) * qk[0][i] : 0.f;
                X[1][i] = p.scale * expf((float)fmin(Gk[1][i] - Gl[0], 0.0)) * qk[1][i];
                X[2][i] = d >= 0 ? p.scale * expf((float)fmin(Gk[1][i] - Gl[1], 0.0)) * qk[2][i] : 0.f;
            }
            const Terms<3> t0f = to_terms<3>(X[0], X[1]), t1f = to_terms<3>(zero4(), X[2]);
#pragma unroll
            for (int s = 0; s < 3; ++s) {
                bf16x8* dst = reinterpret_cast<bf16x8*>(blk + Blk::pairt + 2 * s * kFragBytes) + lane;
                dst[0] = t0f.t[s];
                dst[kFragBytes / 16] = t1f.t[s];
            }
        }
        // ---- A = N diag(beta) (and diag(beta) N) in LDS, row: the later token
        auto put = [&](float* M, int row, int col, f32x4 v) { *reinterpret_cast<f32x4*>(M + row * LD + col) = v; };
        put(A, j, 4 * g, Dt[0] * bk[0]);
        put(A, 16 + j, 4 * g, Dt[1] * bk[0]);
        put(A, 16 + j, 16 + 4 * g, Dt[2] * bk[1]);
        if constexpr (BACK) {
            float* Bm = s_b[wave];
            const float b0 = s_beta[wave][j], b1 = s_beta[wave][16 + j];
            put(Bm, j, 4 * g, Dt[0] * b0);
            put(Bm, 16 + j, 4 * g, Dt[1] * b1);
            put(Bm, 16 + j, 16 + 4 * g, Dt[2] * b1);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        // ---- the diagonal blocks' inverses: lanes 0..15 block 0, 16..31 block 1
        // of A, 32..63 the same of the other system
        {
            const float* M = BACK && lane >= 32 ? s_b[wave] : A;
            const int o = 16 * (g & 1);
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float acc = r == j ? 1.f : 0.f;
                f32x4 a[4];
#pragma unroll
                for (int q = 0; q < (r + 3) / 4; ++q) a[q] = *reinterpret_cast<const f32x4*>(M + (o + r) * LD + o + 4 * q);
#pragma unroll
                for (int q = 0; q < r; ++q) acc -= a[q / 4][q % 4] * x[q];
                x[r] = acc;
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (BACK || lane < 32) {
                float* W_ = const_cast<float*>(M);
#pragma unroll
                for (int r = 0; r < 16; ++r) W_[(o + r) * LD + o + j] = x[r];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        // ---- the block below, and out: rows of the inverse, or (t) its columns
        auto finish = [&](float* M, int at_byte, bool transposed) {
            f32x4 X = zero4(), Y = zero4();                                    // A21 T11, then T22 of it
#pragma unroll
            for (int s = 0; s < 4; ++s) X = mma_f32_k4(M[(16 + j) * LD + 4 * g + s], M[(4 * g + s) * LD + j], X);
#pragma unroll
            for (int s = 0; s < 4; ++s) Y = mma_f32_k4(M[(16 + j) * LD + 16 + 4 * g + s], X[s], Y);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < 4; ++i) M[(16 + 4 * g + i) * LD + j] = -Y[i];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            f32x4 lo[2], hi[2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!transposed) {
                    lo[0][i] = M[j * LD + 4 * g + i];
                    hi[0][i] = 0.f;
                    lo[1][i] = M[(16 + j) * LD + 4 * g + i];
                    hi[1][i] = M[(16 + j) * LD + 16 + 4 * g + i];
                } else {
                    lo[0][i] = M[(4 * g + i) * LD + j];
                    hi[0][i] = M[(16 + 4 * g + i) * LD + j];
                    lo[1][i] = 0.f;
                    hi[1][i] = M[(16 + 4 * g + i) * LD + 16 + j];
                }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const Terms<3> f = to_terms<3>(lo[q], hi[q]);
#pragma unroll
                for (int s = 0; s < 3; ++s)
                    reinterpret_cast<bf16x8*>(blk + at_byte + (2 * s + q) * kFragBytes)[lane] = f.t[s];
            }
        };
        finish(A, Blk::inv, false);
        if constexpr (BACK) finish(s_b[wave], Blk::invt, true);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

size_t delta_block_bytes(bool is_bf16, bool back) {
    return is_bf16 ? (back ? DeltaBlock<3, true>::bytes : DeltaBlock<1, false>::bytes)
                   : (back ? DeltaBlock<3, true>::bytes : DeltaBlock<3, false>::bytes);
}

template <typename E, int NP, bool BACK>
static hipError_t launch_e(const DeltaPairs& a, hipStream_t stream) {
    const long long all = (long long)a.B * (a.c1 - a.c0) * a.H;
    const dim3 grid((unsigned)((std::min(all, kPairUnits) + kPairWaves - 1) / kPairWaves)), block(kPairWaves * 64);
    switch (a.dk) {
        case 32: hipLaunchKernelGGL((delta_pairs_kernel<E, 32, NP, BACK>), grid, block, 0, stream, a); break;
        case 64: hipLaunchKernelGGL((delta_pairs_kernel<E, 64, NP, BACK>), grid, block, 0, stream, a); break;
        default: hipLaunchKernelGGL((delta_pairs_kernel<E, 128, NP, BACK>), grid, block, 0, stream, a); break;
    }
    return hipGetLastError();
}

hipError_t launch_delta_pairs(const DeltaPairs& a, bool back, hipStream_t stream) {
    if (back) return a.is_bf16 ? launch_e<bf16, 3, true>(a, stream) : launch_e<float, 3, true>(a, stream);
    return a.is_bf16 ? launch_e<bf16, 1, false>(a, stream) : launch_e<float, 3, false>(a, stream);
}

}  // namespace kda
