// kda_delta_pairs.hip -- the parts of the gated delta rule's chunks that do not
// depend on the state (kda_delta_chunk.hpp): the inverse of the triangular system
// and the weights of pairs of tokens, as matrix operands in the workspace.
//
// One wave per chunk and head.  K K^T and Q K^T by MFMA with the decays applied in the
// accumulators; N in LDS as its ten tiles of 16 x 16.  The inverse: the four tiles on
// the diagonal by substitution, a column a lane (stable for any beta in [0, 2] and keys
// of length 1, where a series in powers of N is not: repeated keys make its terms grow
// to thousands before they cancel), then those below, T_rc = -T_rr sum_q A_rq T_qc, in
// fp32 MFMA, in N's place.  (Four waves a chunk, each with 16 of its tokens, left three
// of four lanes idle in the substitution and two waves in the products below, and took
// three times as long.)  The 2,048 chunks of B1 H32 T4096 d128 bf16 take 24 us (64 MB
// written), with the gradients' operands 49 us, of which the 154 MB that they write are
// two thirds.  Two waves a SIMD, for the accumulators of up to three products; with the
// gradients' operands 12 to 24 registers of d_k 64 and 128 go through scratch.
#include <algorithm>

#include "kda_delta_chunk.hpp"

namespace kda {

constexpr int kTileLd = 20, kTileSize = 16 * kTileLd;   // floats of a row, of a tile in LDS
constexpr long long kPairGroups = 1LL << 20;            // most workgroups of a launch: more chunks loop

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
    constexpr int C = kDeltaChunk, NTL = kDeltaTiles, KM = DK / 32, NE = sizeof(E) == 2 ? 1 : 3, ES = sizeof(E), LD = kTileLd;
    constexpr int NB = NTL * (NTL + 1) / 2;                    // tiles on and below the diagonal
    __shared__ __align__(16) float s_n[4][NB * kTileSize], s_hi[4][C], s_lo[4][C], s_beta[4][C];
    const int wv = wave_id(), W = p.c1 - p.c0;
    float *N = s_n[wv], *sh = s_hi[wv], *sl = s_lo[wv], *sb = s_beta[wv];
    const unsigned all = (unsigned)(p.B * W * p.H);            // of blocks in memory: fewer than 2^31
    for (unsigned it = blockIdx.x * 4 + wv; it < all; it += gridDim.x * 4) {
        const int lane = fresh_lane_id(), j = lane & 15, g = lane >> 4;
        const unsigned per = (unsigned)p.H, win = (unsigned)W;
        const int h = (int)(it % per), c = p.c0 + (int)(it / per % win), b = (int)(it / per / win);
        const int n = seq_len(p.lens, b, p.T), t0 = c * C, rows = min(C, n - t0);
        if (rows <= 0 || p.S.skip(b)) continue;                // uniform over the wave
        char* blk = p.blocks + (((size_t)b * p.H + h) * W + (c - p.c0)) * Blk::bytes;
        const int hk = h / (p.H / p.Hk), ld = p.Hk * DK * ES;
        const size_t base = (((size_t)b * p.T + t0) * p.Hk + hk) * DK;
        const uint32_t bytes = (uint32_t)((rows - 1) * ld + DK * ES);
        const Rsrc rk = make_rsrc((const E*)p.k + base, bytes), rq = make_rsrc((const E*)p.q + base, bytes);
        auto row = [&](Rsrc r, int a, int m) {
            return raw_load<E>(r, 16 * a + j < rows ? (16 * a + j) * ld + (32 * m + 8 * g) * ES : kOffPast);
        };
        // ---- decays and strengths
        double G = 0;
        float beta = 0.f;
        if (lane < rows) {
            const size_t gate = ((size_t)b * p.T + t0 + lane) * p.H + h;
            G = (double)log_decay(p.g[gate]);
            beta = p.beta[gate];
        }
        G = wave_scan(G);
        const double GC = __shfl(G, C - 1);
        sh[lane] = (float)G;
        sl[lane] = (float)(G - (double)(float)G);
        sb[lane] = beta;
        {
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
        wave_fence();
        auto at = [](int r, int c_) { return r * (r + 1) / 2 + c_; };
        auto tile = [&](int r, int c_) { return N + at(r, c_) * kTileSize; };
        // ---- N = (K K^T) * D below the diagonal, row: the later token w
        f32x4 kh[NTL], kl[NTL];                                // of token 16 a + 4 g + i
#pragma unroll
        for (int a = 0; a < NTL; ++a) {
            kh[a] = *reinterpret_cast<const f32x4*>(&sh[16 * a + 4 * g]);
            kl[a] = *reinterpret_cast<const f32x4*>(&sl[16 * a + 4 * g]);
        }
        auto put_n = [&](const f32x4 (&kk)[NB]) {
#pragma unroll
            for (int w = 0; w < NTL; ++w) {
                const float hi = sh[16 * w + j], lo = sl[16 * w + j];
#pragma unroll
                for (int a = 0; a <= w; ++a) {
                    f32x4 v;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {              // a value, then a selection: no branch
                        const float x = __expf((hi - kh[a][i]) + (lo - kl[a][i])) * kk[at(w, a)][i];
                        v[i] = a < w || j - 4 * g - i > 0 ? x : 0.f;
                    }
                    *reinterpret_cast<f32x4*>(tile(w, a) + j * LD + 4 * g) = v;
                }
            }
        };
        // T = (I + N diag(beta))^{-1} in N's place, with the strengths in sb
        auto invert = [&] {
            // the tiles on the diagonal, one to 16 lanes: x = 1 - N diag(beta) x below it
            {
                float* M = N + (g * (g + 1) / 2 + g) * kTileSize;
                float x[16], y[16];                            // y: what later rows take of x
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    float acc = 0.f;
                    f32x4 a[4];
                    if (r % 4 == 0) __builtin_amdgcn_sched_barrier(0);   // else all rows are read first: 144 registers
#pragma unroll
                    for (int q = 0; q < (r + 3) / 4; ++q) a[q] = *reinterpret_cast<const f32x4*>(M + r * LD + 4 * q);
#pragma unroll
                    for (int q = 0; q < r; ++q) acc += a[q / 4][q % 4] * y[q];
                    x[r] = (r == j ? 1.f : 0.f) - acc;
                    y[r] = sb[16 * g + r] * x[r];
                }
                wave_fence();
#pragma unroll
                for (int r = 0; r < 16; ++r) M[r * LD + j] = x[r];
            }
            wave_fence();
            // those below, column by column: an accumulator is the next product's
            // operand as it is (rows 4 g + s for both)
            f32x4 kb[NTL];
#pragma unroll
            for (int a = 0; a < NTL; ++a) kb[a] = *reinterpret_cast<const f32x4*>(&sb[16 * a + 4 * g]);
            auto add = [&](int r, int q, int c_, f32x4 acc) {  // N_rq diag(beta) T_qc
                const f32x4 a = *reinterpret_cast<const f32x4*>(tile(r, q) + j * LD + 4 * g);
                const float* t = tile(q, c_) + 4 * g * LD + j;
#pragma unroll
                for (int s = 0; s < 4; ++s) acc = mma_f32_k4(a[s], t[s * LD] * kb[q][s], acc);
                return acc;
            };
            auto solve = [&](int r, int c_, f32x4 x) {         // T_rc = -T_rr x, in N_rc's place
                const f32x4 a = *reinterpret_cast<const f32x4*>(tile(r, r) + j * LD + 4 * g);
                f32x4 y = zero4();
#pragma unroll
                for (int s = 0; s < 4; ++s) y = mma_f32_k4(a[s], x[s], y);
                wave_fence();
#pragma unroll
                for (int i = 0; i < 4; ++i) tile(r, c_)[(4 * g + i) * LD + j] = -y[i];
                wave_fence();
            };
            solve(1, 0, add(1, 0, 0, zero4()));
            solve(2, 0, add(2, 1, 0, add(2, 0, 0, zero4())));
            solve(3, 0, add(3, 2, 0, add(3, 1, 0, add(3, 0, 0, zero4()))));
            solve(2, 1, add(2, 1, 1, zero4()));
            solve(3, 1, add(3, 2, 1, add(3, 1, 1, zero4())));
            solve(3, 2, add(3, 2, 2, zero4()));
        };
        {
            // bf16: every row of K and Q is loaded first, or (BACK) 32 channels ahead
            Raw<E> ak[KM][NTL], aq[KM][NTL];
            auto load = [&](int m) {
#pragma unroll
                for (int a = 0; a < NTL; ++a) {
                    ak[m][a] = row(rk, a, m);
                    aq[m][a] = row(rq, a, m);
                }
            };
            constexpr int AHEAD = NE != 1 ? 0 : BACK ? 1 : KM;
#pragma unroll
            for (int m = 0; m < AHEAD && m < KM; ++m) load(m);
            __builtin_amdgcn_sched_barrier(0);
            f32x4 kk[NB], kq[NB], qk[NB];                      // of the later token's tile and the key's
#pragma unroll
            for (int t = 0; t < NB; ++t) kk[t] = kq[t] = qk[t] = zero4();
#pragma unroll
            for (int m = 0; m < KM; ++m) {
                if (m + AHEAD < KM) load(m + AHEAD);
                if (NE == 1) __builtin_amdgcn_sched_barrier(0);
                Terms<NE> k[NTL];
#pragma unroll
                for (int a = 0; a < NTL; ++a) k[a] = raw_terms(ak[m][a]);
#pragma unroll
                for (int w = 0; w < NTL; ++w) {
                    const Terms<NE> q = raw_terms(aq[m][w]);
#pragma unroll
                    for (int a = 0; a <= w; ++a) {
                        kk[at(w, a)] = mma(k[a], k[w], kk[at(w, a)]);
                        kq[at(w, a)] = mma(k[a], q, kq[at(w, a)]);
                        if (BACK) qk[at(w, a)] = mma(q, k[a], qk[at(w, a)]);
                    }
                }
            }
            put_n(kk);
            // ---- the pairs: P's columns with the later token w's queries, P^T's rows
            // with the key w, its decays the other way round
#pragma unroll
            for (int w = 0; w < NTL; ++w) {
                const float hi = sh[16 * w + j], lo = sl[16 * w + j];
                f32x4 P[NTL];
#pragma unroll
                for (int a = 0; a < NTL; ++a) {
                    P[a] = zero4();
                    if (a > w) continue;
                    const f32x4 kb = *reinterpret_cast<const f32x4*>(&sb[16 * a + 4 * g]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = p.scale * __expf((hi - kh[a][i]) + (lo - kl[a][i])) * kb[i] * kq[at(w, a)][i];
                        P[a][i] = a < w || j - 4 * g - i >= (BACK ? 1 : 0) ? x : 0.f;
                    }
                }
                if constexpr (BACK) {                          // the diagonal, by the lane that has its element
                    float self = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) self = 4 * g + i == j ? p.scale * kq[at(w, w)][i] : self;
                    float* out = reinterpret_cast<float*>(blk + Blk::row) + 16 * w + j;
                    if (g == j >> 2) {
                        out[kRowSelf] = self;
                        out[kRowBetaSelf] = self * sb[16 * w + j];
                    }
                }
#pragma unroll
                for (int half = 0; half <= w / 2; ++half) {
                    const Terms<NP> f = split_terms<NP>(P[2 * half], P[2 * half + 1]);
#pragma unroll
                    for (int s = 0; s < NP; ++s)
                        reinterpret_cast<bf16x8*>(blk + Blk::pair + (lower(w, half) * NP + s) * kFragBytes)[lane] = f.t[s];
                }
            }
            if constexpr (BACK) {
#pragma unroll
                for (int w = 0; w < NTL; ++w) {
                    const float hi = sh[16 * w + j], lo = sl[16 * w + j];
                    f32x4 P[NTL];
#pragma unroll
                    for (int a = 0; a < NTL; ++a) {
                        P[a] = zero4();
                        if (a < w) continue;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float x = p.scale * __expf((kh[a][i] - hi) + (kl[a][i] - lo)) * qk[at(a, w)][i];
                            P[a][i] = a > w || 4 * g + i - j > 0 ? x : 0.f;
                        }
                    }
#pragma unroll
                    for (int half = w / 2; half < 2; ++half) {
                        const Terms<3> f = split_terms<3>(P[2 * half], P[2 * half + 1]);
#pragma unroll
                        for (int s = 0; s < 3; ++s)
                            reinterpret_cast<bf16x8*>(blk + Blk::pairt + (upper(w, half) * 3 + s) * kFragBytes)[lane] = f.t[s];
                    }
                }
            }
        }
        wave_fence();
        invert();
#pragma unroll
        for (int w = 0; w < NTL; ++w)
#pragma unroll
            for (int half = 0; half <= w / 2; ++half) {
                f32x4 lo = *reinterpret_cast<const f32x4*>(tile(w, 2 * half) + j * LD + 4 * g), hi = zero4();
                if (2 * half + 1 <= w) hi = *reinterpret_cast<const f32x4*>(tile(w, 2 * half + 1) + j * LD + 4 * g);
                if (BACK && w / 2 == half) {
                    f32x4& d = w % 2 ? hi : lo;
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[i] = 4 * g + i == j ? 0.f : d[i];
                }
                const Terms<3> f = split_terms<3>(lo, hi);
#pragma unroll
                for (int s = 0; s < 3; ++s)
                    reinterpret_cast<bf16x8*>(blk + Blk::inv + (lower(w, half) * 3 + s) * kFragBytes)[lane] = f.t[s];
            }
        // ---- the gradients' ((I + diag(beta) N)^{-1})^T: its element (t, r) is T_rt
        // beta_r / beta_t, whatever the strengths, for T_rt has beta_t as a factor.
        // Where one is (next to) zero the quotient is taken at 2^-60 instead, which
        // changes the others by less than a rounding.
        if constexpr (BACK) {
            const float least = 0x1p-60f;
            if (__any(lane < rows && fabsf(beta) < least)) {
                f32x4 kk[NB];
#pragma unroll
                for (int t = 0; t < NB; ++t) kk[t] = zero4();
#pragma unroll
                for (int m = 0; m < KM; ++m) {
                    Terms<NE> k[NTL];
#pragma unroll
                    for (int a = 0; a < NTL; ++a) k[a] = raw_terms(row(rk, a, m));
#pragma unroll
                    for (int w = 0; w < NTL; ++w)
#pragma unroll
                        for (int a = 0; a <= w; ++a) kk[at(w, a)] = mma(k[a], k[w], kk[at(w, a)]);
                }
                wave_fence();
                put_n(kk);
                sb[lane] = fabsf(beta) < least ? copysignf(least, beta) : beta;
                wave_fence();
                invert();
            }
#pragma unroll
            for (int w = 0; w < NTL; ++w) {
                const float own = sb[16 * w + j], over = own != 0.f ? 1.0f / own : 0.f;
#pragma unroll
                for (int half = w / 2; half < 2; ++half) {
                    f32x4 x[2] = {zero4(), zero4()};
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int r = 2 * half + y;
                        if (r < w) continue;
                        const f32x4 kb = *reinterpret_cast<const f32x4*>(&sb[16 * r + 4 * g]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float t = tile(r, w)[(4 * g + i) * LD + j];
                            x[y][i] = r == w && 4 * g + i == j ? 0.f : t * over * kb[i];
                        }
                    }
                    const Terms<3> f = split_terms<3>(x[0], x[1]);
#pragma unroll
                    for (int s = 0; s < 3; ++s)
                        reinterpret_cast<bf16x8*>(blk + Blk::invt + (upper(w, half) * 3 + s) * kFragBytes)[lane] = f.t[s];
                }
            }
        }
        wave_fence();
    }
}

size_t delta_block_bytes(bool is_bf16, bool back) {
    return back ? DeltaBlock<3, true>::bytes : is_bf16 ? DeltaBlock<2, false>::bytes : DeltaBlock<3, false>::bytes;
}

template <typename E, int NP, bool BACK>
static hipError_t launch_e(const DeltaPairs& a, hipStream_t stream) {
    const long long all = ((long long)a.B * (a.c1 - a.c0) * a.H + 3) / 4;
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
    return a.is_bf16 ? launch_e<bf16, 2, false>(a, stream) : launch_e<float, 3, false>(a, stream);
}

}  // namespace kda
