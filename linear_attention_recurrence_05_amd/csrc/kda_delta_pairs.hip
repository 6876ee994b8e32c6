// kda_delta_pairs.hip -- the parts of the gated delta rule's chunks that do not
// depend on the state (kda_delta_chunk.hpp): the inverse of the triangular system
// and the weights of pairs of tokens, as matrix operands in the workspace.
//
// One workgroup of four waves per chunk and head; wave w has the 16 tokens of tile
// w.  K K^T and Q K^T by MFMA with the decays applied in the accumulators.  The
// inverse: the four 16 x 16 blocks on the diagonal by substitution, a column a lane
// (stable for any beta in [0, 2] and keys of length 1, where a series in powers of
// N is not: repeated keys make its terms grow to thousands before they cancel),
// then the blocks below as T_ll = -T_l A T_u in fp32 MFMA, first within 32 tokens,
// then across.
#include <algorithm>

#include "kda_delta_chunk.hpp"

namespace kda {

constexpr int kPairLd = 68;                     // floats of a row of the 64 x 64 matrices in LDS
constexpr long long kPairGroups = 1LL << 20;    // most workgroups of a launch: more chunks loop

// sum of x over the lanes up to this one
__device__ __forceinline__ double wave_scan(double x) {
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const double up = __shfl_up(x, o);
        if (lane_id() >= o) x += up;
    }
    return x;
}

template <typename E, int DK, int NP, bool BACK>
__global__ __launch_bounds__(256, 2) void delta_pairs_kernel(DeltaPairs p) {
    using Blk = DeltaBlock<NP, BACK>;
    constexpr int C = kDeltaChunk, KM = DK / 32, NE = sizeof(E) == 2 ? 1 : 3, ES = sizeof(E), LD = kPairLd;
    __shared__ __align__(16) float s_m[BACK ? 2 : 1][C * LD];   // N diag(beta), diag(beta) N; then their inverses
    __shared__ __align__(16) float s_hi[C], s_lo[C], s_beta[C];
    const int w = wave_id(), W = p.c1 - p.c0;
    const long long all = (long long)p.B * W * p.H;
    for (long long at = blockIdx.x; at < all; at += gridDim.x) {
        const int lane = fresh_lane_id(), j = lane & 15, g = lane >> 4;
        const int h = (int)(at % p.H), c = p.c0 + (int)(at / p.H % W), b = (int)(at / p.H / W);
        const int n = seq_len(p.lens, b, p.T), t0 = c * C, rows = min(C, n - t0);
        if (rows <= 0 || p.S.skip(b)) continue;                // uniform over the workgroup
        char* blk = p.blocks + (((size_t)b * p.H + h) * W + (c - p.c0)) * Blk::bytes;
        // ---- rows: K and Q of tile w
        const int hk = h / (p.H / p.Hk), ld = p.Hk * DK * ES;
        const size_t base = (((size_t)b * p.T + t0) * p.Hk + hk) * DK;
        const uint32_t bytes = (uint32_t)((rows - 1) * ld + DK * ES);
        const Rsrc rk = make_rsrc((const E*)p.k + base, bytes), rq = make_rsrc((const E*)p.q + base, bytes);
        auto row = [&](Rsrc r, int a, int m) {
            return raw_load<E>(r, 16 * a + j < rows ? (16 * a + j) * ld + (32 * m + 8 * g) * ES : kOffPast);
        };
        Raw<E> xw[KM], yw[KM];
#pragma unroll
        for (int m = 0; m < KM; ++m) {
            xw[m] = row(rk, w, m);
            yw[m] = row(rq, w, m);
        }
        // ---- decays and strengths
        double G = 0;
        float beta = 0.f;
        if (lane < rows) {
            const size_t gate = ((size_t)b * p.T + t0 + lane) * p.H + h;
            G = (double)log_decay(p.g[gate]);
            beta = p.beta[gate];
        }
        G = wave_scan(G);                                      // in every wave
        const double GC = __shfl(G, C - 1);
        __syncthreads();                                       // the last chunk is done with LDS
        if (w == 0) {
            s_hi[lane] = (float)G;
            s_lo[lane] = (float)(G - (double)(float)G);
            s_beta[lane] = beta;
        } else if (w == 1) {
            float* out = reinterpret_cast<float*>(blk + Blk::row);
            const float end = expf((float)(GC - G));
            out[kRowGrow + lane] = expf((float)G);
            out[kRowWrite + lane] = end * beta;
            out[kRowEnd + lane] = end;
            out[kRowBeta + lane] = beta;
            if (lane == 0) {
                const double f = exp(GC);
                const float ff = (float)f;
                out[kRowDecay] = ff;
                out[kRowDecay + 1] = f > 1e-30 ? (float)((f - (double)ff) / f) : 0.f;
            }
        }
        __syncthreads();
        // ---- tiles (key a, later token w): K K^T and K Q^T; (BACK) (query a, key w)
        f32x4 kk[kDeltaTiles], kq[kDeltaTiles], qk[kDeltaTiles];
#pragma unroll
        for (int a = 0; a < kDeltaTiles; ++a) {
            kk[a] = kq[a] = qk[a] = zero4();
            if (a < w) {
                Raw<E> x[KM];
#pragma unroll
                for (int m = 0; m < KM; ++m) x[m] = row(rk, a, m);
#pragma unroll
                for (int m = 0; m < KM; ++m) {
                    const Terms<NE> xa = raw_terms(x[m]);
                    kk[a] = mma(xa, raw_terms(xw[m]), kk[a]);
                    kq[a] = mma(xa, raw_terms(yw[m]), kq[a]);
                }
            } else if (a == w) {
#pragma unroll
                for (int m = 0; m < KM; ++m) {
                    const Terms<NE> xa = raw_terms(xw[m]), ya = raw_terms(yw[m]);
                    kk[a] = mma(xa, xa, kk[a]);
                    kq[a] = mma(xa, ya, kq[a]);
                    if constexpr (BACK) qk[a] = mma(ya, xa, qk[a]);
                }
            } else if (BACK) {
                Raw<E> y[KM];
#pragma unroll
                for (int m = 0; m < KM; ++m) y[m] = row(rq, a, m);
#pragma unroll
                for (int m = 0; m < KM; ++m) qk[a] = mma(raw_terms(y[m]), raw_terms(xw[m]), qk[a]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // ---- with their decays: to LDS (row: the later token), and the pairs' operands
        const float hi = s_hi[16 * w + j], lo = s_lo[16 * w + j], bl = s_beta[16 * w + j];
        f32x4 P[kDeltaTiles], X[kDeltaTiles];
#pragma unroll
        for (int a = 0; a < kDeltaTiles; ++a) {
            P[a] = X[a] = zero4();
            const f32x4 ghi = *reinterpret_cast<const f32x4*>(&s_hi[16 * a + 4 * g]),
                        glo = *reinterpret_cast<const f32x4*>(&s_lo[16 * a + 4 * g]);
            if (a <= w) {
                const f32x4 bk = *reinterpret_cast<const f32x4*>(&s_beta[16 * a + 4 * g]);
                f32x4 N0, N1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = 16 * (w - a) + j - 4 * g - i;   // later - key
                    const float D = d >= 0 ? __expf((hi - ghi[i]) + (lo - glo[i])) : 0.f;
                    P[a][i] = p.scale * D * bk[i] * kq[a][i];
                    const float N = d > 0 ? D * kk[a][i] : 0.f;
                    N0[i] = N * bk[i];
                    N1[i] = N * bl;
                }
                *reinterpret_cast<f32x4*>(&s_m[0][(16 * w + j) * LD + 16 * a + 4 * g]) = N0;
                if constexpr (BACK) *reinterpret_cast<f32x4*>(&s_m[BACK][(16 * w + j) * LD + 16 * a + 4 * g]) = N1;
            }
            if (BACK && a >= w) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = 16 * (a - w) + 4 * g + i - j;   // query - key
                    X[a][i] = d >= 0 ? p.scale * __expf((ghi[i] - hi) + (glo[i] - lo)) * qk[a][i] : 0.f;
                }
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (half <= w / 2) {
                const Terms<NP> f = to_terms<NP>(P[2 * half], P[2 * half + 1]);
#pragma unroll
                for (int s = 0; s < NP; ++s)
                    reinterpret_cast<bf16x8*>(blk + Blk::pair + (lower(w, half) * NP + s) * kFragBytes)[lane] = f.t[s];
            }
            if (BACK && half >= w / 2) {
                const Terms<3> f = to_terms<3>(X[2 * half], X[2 * half + 1]);
#pragma unroll
                for (int s = 0; s < 3; ++s)
                    reinterpret_cast<bf16x8*>(blk + Blk::pairt + (upper(w, half) * 3 + s) * kFragBytes)[lane] = f.t[s];
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_sched_barrier(0);
        // ---- the inverse of this wave's block on the diagonal: a column a lane
        // (lanes 16 .. 31 of the other system)
        {
            float* M = &s_m[BACK ? g & 1 : 0][(16 * w) * LD + 16 * w];
            float x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float acc = r == j ? 1.f : 0.f;
                f32x4 a[4];
                if (r % 4 == 0) __builtin_amdgcn_sched_barrier(0);   // else all rows are read first: 144 registers
#pragma unroll
                for (int q = 0; q < (r + 3) / 4; ++q) a[q] = *reinterpret_cast<const f32x4*>(M + r * LD + 4 * q);
#pragma unroll
                for (int q = 0; q < r; ++q) acc -= a[q / 4][q % 4] * x[q];
                x[r] = acc;
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (lane < (BACK ? 32 : 16)) {
#pragma unroll
                for (int r = 0; r < 16; ++r) M[r * LD + j] = x[r];
            }
        }
        __syncthreads();
        // ---- the blocks below: first (1, 0) and (3, 2), then the four of the lower
        // left quarter, a column of two to a wave.  An accumulator is the next
        // product's operand as it is (rows 4 g + s for both).
        auto tile = [&](const float* M, int r, int c, int s) { return M[(16 * r + j) * LD + 16 * c + 4 * g + s]; };
        auto column = [&](const float* M, int r, int c, int s) { return M[(16 * r + 4 * g + s) * LD + 16 * c + j]; };
        auto times = [&](const float* M, int r, int c, int c2, f32x4 acc) {   // block (r, c) times block (c, c2)
#pragma unroll
            for (int s = 0; s < 4; ++s) acc = mma_f32_k4(tile(M, r, c, s), column(M, c, c2, s), acc);
            __builtin_amdgcn_sched_barrier(0);
            return acc;
        };
        auto applied = [&](const float* M, int r, int c, f32x4 X, f32x4 acc) {   // block (r, c) times X
#pragma unroll
            for (int s = 0; s < 4; ++s) acc = mma_f32_k4(tile(M, r, c, s), X[s], acc);
            __builtin_amdgcn_sched_barrier(0);
            return acc;
        };
        auto put = [&](float* M, int r, int c, f32x4 X) {
#pragma unroll
            for (int i = 0; i < 4; ++i) M[(16 * r + 4 * g + i) * LD + 16 * c + j] = -X[i];
        };
        float* M = s_m[BACK ? w / 2 : 0];
        const bool busy = BACK || w < 2;
        const int e = w & 1;
        f32x4 X1 = zero4();
        if (busy) X1 = applied(M, 2 * e + 1, 2 * e + 1, times(M, 2 * e + 1, 2 * e, 2 * e, zero4()), zero4());
        if (busy) put(M, 2 * e + 1, 2 * e, X1);                // read by this wave alone so far
        __syncthreads();
        f32x4 X2 = zero4(), X3 = zero4();
        if (busy) {
            f32x4 a2, a3;
            if (e == 0) {
                a2 = times(M, 2, 1, 0, times(M, 2, 0, 0, zero4()));
                a3 = times(M, 3, 1, 0, times(M, 3, 0, 0, zero4()));
            } else {
                a2 = times(M, 2, 1, 1, zero4());
                a3 = times(M, 3, 1, 1, zero4());
            }
            X2 = applied(M, 2, 2, a2, zero4());
            X3 = applied(M, 3, 2, a2, applied(M, 3, 3, a3, zero4()));
        }
        __syncthreads();
        if (busy) {
            put(M, 2, e, X2);
            put(M, 3, e, X3);
        }
        __syncthreads();
        // ---- out: rows of the inverse, columns of the other one
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (half <= w / 2) {
                const float* row = &s_m[0][(16 * w + j) * LD + 32 * half + 4 * g];
                const f32x4 a = *reinterpret_cast<const f32x4*>(row);
                const f32x4 z = *reinterpret_cast<const f32x4*>(row + 16);
                const Terms<3> f = to_terms<3>(a, 2 * half + 1 <= w ? z : zero4());
#pragma unroll
                for (int s = 0; s < 3; ++s)
                    reinterpret_cast<bf16x8*>(blk + Blk::inv + (lower(w, half) * 3 + s) * kFragBytes)[lane] = f.t[s];
            }
            if (BACK && half >= w / 2) {
                f32x4 a = zero4(), z;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (2 * half >= w) a[i] = s_m[BACK][(32 * half + 4 * g + i) * LD + 16 * w + j];
                    z[i] = s_m[BACK][(32 * half + 16 + 4 * g + i) * LD + 16 * w + j];
                }
                const Terms<3> f = to_terms<3>(a, z);
#pragma unroll
                for (int s = 0; s < 3; ++s)
                    reinterpret_cast<bf16x8*>(blk + Blk::invt + (upper(w, half) * 3 + s) * kFragBytes)[lane] = f.t[s];
            }
        }
    }
}

size_t delta_block_bytes(bool is_bf16, bool back) {
    return back ? DeltaBlock<3, true>::bytes : is_bf16 ? DeltaBlock<1, false>::bytes : DeltaBlock<3, false>::bytes;
}

template <typename E, int NP, bool BACK>
static hipError_t launch_e(const DeltaPairs& a, hipStream_t stream) {
    const long long all = (long long)a.B * (a.c1 - a.c0) * a.H;
    const dim3 grid((unsigned)std::min(all, kPairGroups)), block(256);
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
