// kda_delta_backward.hip -- the gradients of the gated delta rule in chunk form
// (kda_delta_chunk.hpp).  With Y the gradient of the state behind a chunk, U =
// beta E, and dO taken times scale:
//   dU = P^T dO + e^{G_C - G} K Y,  P = (Q K^T) * D
//   Z  = ((I + diag(beta) N)^{-1})^T dU        the gradient of what a token writes
//   dv = R = beta Z,   dbeta = Z . E
//   Y' = e^{G_C} Y + Q^T (e^G dO) - K^T (e^G R)
// which is a chain over the chunks like the forward one, columns apart.  Scaling
// every decay from token t on scales what the outputs and the final state get out
// of the state before t, so that
//   dg_t = sum_{r >= t} (dO_r . o_r - dv_r . v_r) + <S_T, dS_T>
// which is taken from t to the next anchor, a chunk's end at which <S, Y> is
// formed anew: a sum over the whole sequence would carry its rounding along.
// The rest needs no chain and takes 64 tokens at a time, from the states and
// gradients that the two sweeps left:
//   dq = e^G dO S^T + ((dO U^T) * D) K
//   dk = e^{G_C - G} U Y^T - e^G R S^T + ((dO U^T) * D)^T Q - (X + X^T) K,
//   X  = (R U^T) * D below the diagonal
#include <algorithm>

#include "kda_delta_chain.hpp"

namespace kda {

struct DeltaReverse {
    const void *q, *k, *v;
    float scale;
    const float* dST;
    float* dS0;
    const int* lens;
    const char* blocks;
    void* dv_out;
    DeltaSweep sweep;
    int B, T, H, Hk, dk, dv;
};

// The chain from the last chunk to the first; as delta_chain_kernel: one workgroup
// per (b, h, 16 value columns), one wave for each 32 key channels of Y.
template <typename E, int DK>
__global__ __launch_bounds__(DK * 2, 2) void delta_reverse_kernel(DeltaReverse p) {
    constexpr int C = kDeltaChunk, KM = DK / 32, NT = DK * 2;
    constexpr int NE = sizeof(E) == 2 ? 1 : 3, ES = sizeof(E);
    using Blk = DeltaBlock<3, true>;
    constexpr int kFrom = Blk::row, kStage = Blk::bytes - kFrom;             // the block's part that is read here
    constexpr int LK = 40, LV = 24;
    constexpr int PB = kStage / 16, RB = (PB + NT - 1) / NT;
    constexpr int PR = ES, PV = C * PR, RV = (PV + NT - 1) / NT;             // pieces of 16 bytes of dO's rows, of its tile
    __shared__ __align__(16) bf16 s_k[KM][NE][C * LK], s_q[KM][NE][C * LK];
    __shared__ __align__(16) bf16 s_v[2][NE][C * LV];
    __shared__ __align__(16) char s_blk[2][kStage];
    __shared__ f32x4 s_part[KM > 1 ? 2 : 1][KM > 1 ? KM : 1][2][kWave];

    const int tiles = p.dv / 16, units = p.B * p.H;
    int unit, tile;
    unit_tile(blockIdx.x, units, tiles, unit, tile);
    const int b = unit / p.H, h = unit % p.H, hk = h / (p.H / p.Hk);
    const int n = seq_len(p.lens, b, p.T), c_end = (n + C - 1) / C;
    const int tid = threadIdx.x, kw = wave_id(), lane = lane_id(), j = lane & 15, g = lane >> 4;
    const DeltaSweep& sw = p.sweep;

    const size_t state = (size_t)DK * p.dv;
    f32x4 Y[2];
    {
        const float* in = p.dST ? p.dST + (size_t)unit * state : nullptr;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) Y[t][i] = in ? in[(size_t)(32 * kw + 8 * g + 4 * t + i) * p.dv + 16 * tile + j] : 0.f;
    }

    const int ldk = p.Hk * DK * ES, ldv = p.H * p.dv * ES;
    struct Own {
        Raw<E> k[2], q[2];
    };
    struct Common {
        u32x4 v[RV], blk[RB];
    };
    auto load_own = [&](int c, Own& x) {                     // chunks before the first load nothing
        const int rows = c >= 0 ? min(C, n - c * C) : 0;
        const size_t base = (((size_t)b * p.T + (size_t)max(c, 0) * C) * p.Hk + hk) * DK + 32 * kw;
        const uint32_t bytes = rows > 0 ? (uint32_t)((rows - 1) * ldk + 32 * ES) : 0;
        const Rsrc rk = make_rsrc((const E*)p.k + base, bytes), rq = make_rsrc((const E*)p.q + base, bytes);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int off = 16 * q + j < rows ? (16 * q + j) * ldk + 8 * g * ES : kOffPast;
            x.k[q] = raw_load<E>(rk, off);
            x.q[q] = raw_load<E>(rq, off);
        }
    };
    const char* blocks = p.blocks + (size_t)unit * sw.NC * Blk::bytes + kFrom;
    auto load_common = [&](int c, Common& x) {
        const int rows = c >= 0 ? min(C, n - c * C) : 0;
        const size_t base = (((size_t)b * p.T + (size_t)max(c, 0) * C) * p.H + h) * p.dv + 16 * tile;
        const Rsrc rv = make_rsrc((const E*)sw.dO + base, rows > 0 ? (uint32_t)((rows - 1) * ldv + 16 * ES) : 0);
        const Rsrc rb = make_rsrc(blocks + (size_t)max(c, 0) * Blk::bytes, rows > 0 ? kStage : 0);
#pragma unroll
        for (int i = 0; i < RV; ++i) {
            const int at = tid + i * NT, row = at / PR;
            x.v[i] = buf_load<u32x4>(rv, at < PV && row < rows ? row * ldv + at % PR * 16 : kOffPast);
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) x.blk[i] = buf_load<u32x4>(rb, tid + i * NT < PB ? (tid + i * NT) * 16 : kOffPast);
    };
    auto stage_common = [&](int buf, const Common& x) {
#pragma unroll
        for (int i = 0; i < RV; ++i) {
            const int at = tid + i * NT, row = at / PR;
            if (PV % NT == 0 || at < PV) put_piece<E>(&s_v[buf][0][row * LV + at % PR * (16 / ES)], C * LV, x.v[i]);
        }
#pragma unroll
        for (int i = 0; i < RB; ++i)
            if (PB % NT == 0 || tid + i * NT < PB) reinterpret_cast<u32x4*>(s_blk[buf])[tid + i * NT] = x.blk[i];
    };

    ChunkDecay decay;
    Own own[2];
    Common common;
    auto chunk = [&](auto set, int c) {
        constexpr int s = decltype(set)::value;
        Terms<NE> kt[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            kt[q] = raw_terms(own[s].k[q]);
            const Terms<NE> qt = raw_terms(own[s].q[q]);
#pragma unroll
            for (int i = 0; i < NE; ++i) {
                *reinterpret_cast<bf16x8*>(&s_k[kw][i][(16 * q + j) * LK + 8 * g]) = kt[q].t[i];
                *reinterpret_cast<bf16x8*>(&s_q[kw][i][(16 * q + j) * LK + 8 * g]) = qt.t[i];
            }
        }
        load_own(c - 2, own[s]);
        // what the outputs need, set out for early: v and e of token 16 q + j
        f32x4 v[2], e[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int t = c * C + 16 * q + j;
            v[q] = e[q] = zero4();
            if ((KM > 1 && kw != q) || t >= n) continue;
            load4((const E*)p.v + (((size_t)b * p.T + t) * p.H + h) * p.dv + 16 * tile + 4 * g, v[q]);
            const float* from = sw.e + (((size_t)unit * sw.NC + c) * p.dv + 16 * tile + 4 * g) * C + 16 * q + j;
#pragma unroll
            for (int i = 0; i < 4; ++i) e[q][i] = from[i * C];
        }
        if (c % kSuperChunks == kSuperChunks - 1 || c == c_end - 1) {
            E* dst = (E*)sw.Y + (((size_t)unit * sw.NS + c / kSuperChunks) * p.dv + 16 * tile + j) * DK + 32 * kw + 8 * g;
            store8(dst, Y[0], Y[1]);
        }
        if (c % kAnchorChunks == kAnchorChunks - 1 || c == c_end - 1) {
            const size_t at = (((size_t)unit * sw.NA + c / kAnchorChunks) * tiles + tile) * KM + kw;
            const f32x4* S = reinterpret_cast<const f32x4*>(sw.end) + at * 2 * kWave + lane;
            float d = 0.f;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) d += S[t * kWave][i] * Y[t][i];
#pragma unroll
            for (int o = 1; o < kWave; o <<= 1) d += __shfl_xor(d, o);
            if (lane == 0) sw.anchor[at] = d;
        }
        // K Y of this wave's channels
        const Terms<3> yf = to_terms<3>(Y[0], Y[1]);
        f32x4 x[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            x[q] = mma(kt[q], yf, zero4());
            if constexpr (KM > 1) s_part[s][kw][q][lane] = x[q];
        }
        __syncthreads();                                     // the parts are there, and this chunk's block and dO
        if constexpr (KM > 1) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                x[q] = s_part[s][0][q][lane];
#pragma unroll
                for (int w = 1; w < KM; ++w) x[q] += s_part[s][w][q][lane];
            }
        }
        const char* blk = s_blk[s] - kFrom;
        const float *row = reinterpret_cast<const float*>(blk + Blk::row), *more = reinterpret_cast<const float*>(blk + Blk::more);
        // dU, Z
        const Terms<NE> dOt = col_terms<NE>(&s_v[s][0][0], C * LV, LV, 0, 4, j, g);
        f32x4 u[2], z[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const f32x4 end = *reinterpret_cast<const f32x4*>(more + 16 * q + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[q][i] = end[i] * x[q][i];
            u[q] = mma(frag_terms<3>(blk + Blk::pairt + q * kFragBytes, 2 * kFragBytes), dOt, u[q]);
        }
        const Terms<3> ut = to_terms<3>(u[0], u[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) z[q] = mma(frag_terms<3>(blk + Blk::invt + q * kFragBytes, 2 * kFragBytes), ut, zero4());
        stage_common(1 - s, common);
        load_common(c - 2, common);
        // Y' = e^{G_C} Y + Q^T (e^G dO) - K^T (e^G beta Z)
        f32x4 dO[2], gq[2], gr[2];
        to_f32(dOt, dO[0], dO[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const f32x4 eg = *reinterpret_cast<const f32x4*>(row + 16 * q + 4 * g);
            const f32x4 beta = *reinterpret_cast<const f32x4*>(more + C + 16 * q + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                gq[q][i] = p.scale * eg[i] * dO[q][i];
                gr[q][i] = -eg[i] * (beta[i] * z[q][i]);
            }
        }
        const Terms<3> gqt = to_terms<3>(gq[0], gq[1]), grt = to_terms<3>(gr[0], gr[1]);
        const float f = decay(row[2 * C], row[2 * C + 1]);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            Y[t] = mma(col_terms<NE>(&s_q[kw][0][0], C * LK, LK, 4 * t, 8, j, g), gqt, f * Y[t]);
            Y[t] = mma(col_terms<NE>(&s_k[kw][0][0], C * LK, LK, 4 * t, 8, j, g), grt, Y[t]);
        }
        // out: Z once more with a token a lane, of the first two waves (the only
        // one's both) columns of tokens
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (KM > 1 && kw != q) continue;
            const f32x4 zt = mma(ut, frag_terms<3>(blk + Blk::invt + q * kFragBytes, 2 * kFragBytes), zero4());
            const float beta = more[C + 16 * q + j];
            const int t = c * C + 16 * q + j;
            f32x4 r;
            float d = 0.f, db = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r[i] = beta * zt[i];
                d += r[i] * v[q][i];
                db += zt[i] * e[q][i];
            }
            d += __shfl_xor(d, 16);
            d += __shfl_xor(d, 32);
            db += __shfl_xor(db, 16);
            db += __shfl_xor(db, 32);
            if (g == 0) {
                float* dot = sw.dot + ((size_t)tile * units + unit) * sw.NC * C + t;
                *dot -= d;
                dot[(size_t)tiles * units * sw.NC * C] = db;
            }
            if (t < n) {
                E* dst = (E*)p.dv_out + (((size_t)b * p.T + t) * p.H + h) * p.dv + 16 * tile + 4 * g;
                if constexpr (ES == 2)
                    *reinterpret_cast<bf16x4*>(dst) = pack4(r);
                else
                    *reinterpret_cast<f32x4*>(dst) = r;
            }
        }
    };

    if (c_end > 0) {
        constexpr std::integral_constant<int, 0> set0{};
        constexpr std::integral_constant<int, 1> set1{};
        load_common(c_end - 1, common);
        load_own(c_end - 1, own[0]);
        load_own(c_end - 2, own[1]);
        stage_common(0, common);
        load_common(c_end - 2, common);
        for (int c = c_end - 1;; c -= 2) {
            chunk(set0, c);
            if (c < 1) break;
            chunk(set1, c - 1);
            if (c < 2) break;
        }
    }
    if (p.dS0) {
        float* out = p.dS0 + (size_t)unit * state;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) out[(size_t)(32 * kw + 8 * g + 4 * t + i) * p.dv + 16 * tile + j] = Y[t][i];
    }
}

// ------------------------------------------------------------------ dq and dk

struct DeltaQK {
    const void *q, *k, *dv;
    const float *g, *beta;
    float scale;
    const int* lens;
    DeltaSweep sweep;
    void *dq, *dk;
    int B, T, H, Hk, dk_, dv_;
};

// One workgroup of four waves per superchunk of a head of q and k, over the heads
// that share it.  Over 32 value columns at a time, in LDS: S^T and Y^T [32][DK], dO
// and dv [64][32], U^T [32][64].  Wave m makes the products with S and Y of
// channels 32 m .. (transposed: a token a lane), and wave w the pairs of its 16
// tokens with all others, which then go through LDS as operands.
// With bf16 an operand is one bf16 term: what it leaves out is half a step on a
// part of the sum, beside the result's own rounding.
template <typename E, int DK>
__global__ __launch_bounds__(256) void delta_qk_kernel(DeltaQK p) {
    constexpr int NE = sizeof(E) == 2 ? 1 : 3, ES = sizeof(E), PE = 16 / ES, L = kSuperChunks * kDeltaChunk;
    constexpr int LS = DK + 8, LT = 32 + 8, LU = L + 8;      // padded rows
    constexpr int QS = 32 * LS, QT = L * LT, QU = 32 * LU, QK = L * LS;      // elements of a plane
    constexpr int kFrags = 3 * 4 * 2 * NE * kFragBytes;      // bytes of the pairs' operands
    constexpr int kStage1 = NE * (2 * QS + 2 * QT + QU) * 2, kStage2 = kFrags + NE * QK * 2;
    __shared__ __align__(16) char s_mem[kStage1 > kStage2 ? kStage1 : kStage2];
    __shared__ double s_G[L];
    __shared__ float s_eg[L], s_end[L], s_beta[L];
    bf16 *s_S = reinterpret_cast<bf16*>(s_mem), *s_Y = s_S + NE * QS, *s_O = s_Y + NE * QS, *s_R = s_O + NE * QT, *s_U = s_R + NE * QT;
    char* s_frag = s_mem;                                    // then, in the same place, the pairs and K or Q
    bf16* s_K = reinterpret_cast<bf16*>(s_mem + kFrags);
    const DeltaSweep& sw = p.sweep;
    const int sc = blockIdx.x / p.Hk % sw.NS, hk = blockIdx.x % p.Hk, b = blockIdx.x / p.Hk / sw.NS;
    const int n = seq_len(p.lens, b, p.T), t0 = sc * L, rows = min(L, n - t0);
    if (rows <= 0) return;
    const int tid = threadIdx.x, wave = wave_id(), lane = lane_id(), j = lane & 15, g = lane >> 4, G = p.H / p.Hk;
    const bool mine = wave < DK / 32;                        // this wave has channels
    const int chunks = (rows + kDeltaChunk - 1) / kDeltaChunk;
    f32x4 dq[2][4], dk[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) dq[t][r] = dk[t][r] = zero4();

    for (int hg = 0; hg < G; ++hg) {
        const int h = hk * G + hg, unit = b * p.H + h;
        __syncthreads();                                     // the last head is done with LDS
        if (wave == 0) {
            const size_t at = ((size_t)b * p.T + t0 + lane) * p.H + h;
            double s = lane < rows ? (double)log_decay(p.g[at]) : 0.0;
#pragma unroll
            for (int o = 1; o < L; o <<= 1) {
                const double up = __shfl_up(s, o);
                if (lane >= o) s += up;
            }
            const double end = __shfl(s, L - 1);
            s_G[lane] = s;
            s_eg[lane] = expf((float)s);
            s_end[lane] = expf((float)(end - s));
            s_beta[lane] = lane < rows ? p.beta[at] : 0.f;
        }
        __syncthreads();
        const E* gS = (const E*)sw.S + ((size_t)unit * sw.NS + sc) * p.dv_ * DK;
        const E* gY = (const E*)sw.Y + ((size_t)unit * sw.NS + sc) * p.dv_ * DK;
        const size_t tok = (((size_t)b * p.T + t0) * p.H + h) * p.dv_;
        const float* gE = sw.e + ((size_t)unit * sw.NC + kSuperChunks * sc) * p.dv_ * kDeltaChunk;
        f32x4 aq[2][4], as[2][4], ay[2][4], pr[4], xr[4], pd = zero4(), xd = zero4();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            pr[r] = xr[r] = zero4();
#pragma unroll
            for (int t = 0; t < 2; ++t) aq[t][r] = as[t][r] = ay[t][r] = zero4();
        }
        for (int c0 = 0; c0 < p.dv_; c0 += 32) {
            if (c0) __syncthreads();
            for (int i = tid; i < 32 * DK / PE; i += 256) {
                const int c = i / (DK / PE), ch = i % (DK / PE) * PE;
                put_piece<E>(s_S + c * LS + ch, QS, *reinterpret_cast<const u32x4*>(gS + (size_t)(c0 + c) * DK + ch));
                put_piece<E>(s_Y + c * LS + ch, QS, *reinterpret_cast<const u32x4*>(gY + (size_t)(c0 + c) * DK + ch));
            }
            for (int i = tid; i < L * 32 / PE; i += 256) {
                const int t = i / (32 / PE), c = i % (32 / PE) * PE;
                u32x4 x{}, y{};
                if (t < rows) {
                    const size_t at = tok + (size_t)t * p.H * p.dv_ + c0 + c;
                    x = *reinterpret_cast<const u32x4*>((const E*)sw.dO + at);
                    y = *reinterpret_cast<const u32x4*>((const E*)p.dv + at);
                }
                put_piece<E>(s_O + t * LT + c, QT, x);
                put_piece<E>(s_R + t * LT + c, QT, y);
            }
            for (int i = tid; i < 32 * L / 4; i += 256) {
                const int c = i / (L / 4), t = i % (L / 4) * 4, cc = t / kDeltaChunk;
                f32x4 u = zero4();
                if (cc < chunks) {
                    u = *reinterpret_cast<const f32x4*>(gE + ((size_t)cc * p.dv_ + c0 + c) * kDeltaChunk + t % kDeltaChunk);
#pragma unroll
                    for (int x = 0; x < 4; ++x) u[x] *= s_beta[t + x];
                }
#pragma unroll
                for (int s = 0; s < NE; ++s) {
                    const bf16x4 hi = pack4(u);
                    *reinterpret_cast<bf16x4*>(s_U + s * QU + c * LU + t) = hi;
#pragma unroll
                    for (int x = 0; x < 4; ++x) u[x] -= (float)hi[x];
                }
            }
            __syncthreads();
            // operands with a token a lane, value columns 4 g .. and 16 + 4 g ..
            auto tokens = [&](const bf16* s, int r) {
                Terms<NE> f;
#pragma unroll
                for (int x = 0; x < NE; ++x) {
                    const bf16* at = s + x * QT + (16 * r + j) * LT + 4 * g;
                    const bf16x4 lo = *reinterpret_cast<const bf16x4*>(at), hi = *reinterpret_cast<const bf16x4*>(at + 16);
                    f.t[x] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                }
                return f;
            };
            auto written = [&](int r) { return col_terms<NE>(s_U, QU, LU, 16 * r, 4, j, g); };
            const Terms<NE> Ow = tokens(s_O, wave), Rw = tokens(s_R, wave), Uw = written(wave);
            Terms<NE> Sf[2], Yf[2];
            if (mine) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    Sf[t] = col_terms<NE>(s_S, QS, LS, 32 * wave + 4 * t, 8, j, g);
                    Yf[t] = col_terms<NE>(s_Y, QS, LS, 32 * wave + 4 * t, 8, j, g);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const Terms<NE> O = tokens(s_O, r), R = tokens(s_R, r), U = written(r);
                if (mine) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        aq[t][r] = mma(Sf[t], O, aq[t][r]);
                        as[t][r] = mma(Sf[t], R, as[t][r]);
                        ay[t][r] = mma(Yf[t], U, ay[t][r]);
                    }
                }
                if (r <= wave) {                             // rows: what token r wrote, lane: the later one
                    pr[r] = mma(U, Ow, pr[r]);
                    xr[r] = mma(U, Rw, xr[r]);
                }
                if (r >= wave) {                             // rows: the later token, lane: what this one wrote
                    f32x4 &pp = r == wave ? pd : pr[r], &xx = r == wave ? xd : xr[r];
                    pp = mma(O, Uw, pp);
                    xx = mma(R, Uw, xx);
                }
            }
        }
        // ---- pairs with their decays, as operands with the output's token a lane:
        // (dO U^T)*D for dq, its transpose for dk, -(X + X^T) for dk
        f32x4 wq[4], wk[4], wx[4];
        const double Gw = s_G[16 * wave + j];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = 16 * (wave - r) + j - 4 * g - i;   // lane's token - row's token
                const float D = expf((float)fmin(d >= 0 ? Gw - s_G[16 * r + 4 * g + i] : s_G[16 * r + 4 * g + i] - Gw, 0.0));
                const float later = r == wave ? pd[i] : pr[r][i], xlater = r == wave ? xd[i] : xr[r][i];
                wq[r][i] = d >= 0 ? p.scale * D * pr[r][i] : 0.f;
                wk[r][i] = d <= 0 ? p.scale * D * later : 0.f;
                wx[r][i] = d > 0 ? -D * xr[r][i] : d < 0 ? -D * xlater : 0.f;
            }
        auto put = [&](int kind, const f32x4 (&w)[4]) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const Terms<NE> f = to_terms<NE>(w[2 * ks], w[2 * ks + 1]);
#pragma unroll
                for (int x = 0; x < NE; ++x)
                    reinterpret_cast<bf16x8*>(s_frag + (((kind * 4 + wave) * 2 + ks) * NE + x) * kFragBytes)[lane] = f.t[x];
            }
        };
        __syncthreads();                                     // every wave is done with the rows
        put(0, wq);
        put(1, wk);
        put(2, wx);
        if (mine) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float eg = s_eg[16 * r + j], end = s_end[16 * r + j], sq = p.scale * eg;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        dq[t][r][i] += sq * aq[t][r][i];
                        dk[t][r][i] += end * ay[t][r][i] - eg * as[t][r][i];
                    }
            }
        }
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {               // K, then Q
            __syncthreads();                                 // the pairs are there, K is used
            const E* from = (const E*)(pass ? p.q : p.k) + (((size_t)b * p.T + t0) * p.Hk + hk) * DK;
            for (int i = tid; i < L * DK / PE; i += 256) {
                const int t = i / (DK / PE), ch = i % (DK / PE) * PE;
                u32x4 x{};
                if (t < rows) x = *reinterpret_cast<const u32x4*>(from + (size_t)t * p.Hk * DK + ch);
                put_piece<E>(s_K + t * LS + ch, QK, x);
            }
            __syncthreads();
            if (!mine) continue;
            auto frag = [&](int kind, int r, int ks) { return frag_terms<NE>(s_frag + ((kind * 4 + r) * 2 + ks) * NE * kFragBytes, kFragBytes); };
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const Terms<NE> f = col_terms<NE>(s_K + 32 * ks * LS, QK, LS, 32 * wave + 4 * t, 8, j, g);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (pass == 0) {
                            if (ks <= r / 2) dq[t][r] = mma(f, frag(0, r, ks), dq[t][r]);
                            dk[t][r] = mma(f, frag(2, r, ks), dk[t][r]);
                        } else if (ks >= r / 2) {
                            dk[t][r] = mma(f, frag(1, r, ks), dk[t][r]);
                        }
                    }
                }
        }
    }
    if (!mine) return;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int t = 16 * r + j;
        if (t >= rows) continue;
        const size_t at = (((size_t)b * p.T + t0 + t) * p.Hk + hk) * DK + 32 * wave + 8 * g;
        store8((E*)p.dq + at, dq[0][r], dq[1][r]);
        store8((E*)p.dk + at, dk[0][r], dk[1][r]);
    }
}

// ------------------------------------------------------------------ dg and dbeta

// One wave per (b, h) and anchor: 256 tokens, four a lane, sums in 64 bits.
__global__ __launch_bounds__(256) void delta_gates_kernel(DeltaSweep sw, const int* __restrict__ lens, float* __restrict__ dg,
                                                          float* __restrict__ dbeta, int B, int T, int H, int tiles, int KM) {
    constexpr int N = kAnchorChunks * kDeltaChunk, PL = N / kWave;
    const long long all = (long long)B * H * sw.NA;
    const int lane = lane_id(), units = B * H;
    for (long long at = (long long)blockIdx.x * 4 + wave_id(); at < all; at += (long long)gridDim.x * 4) {
        const int unit = (int)(at % units), a = (int)(at / units), b = unit / H, h = unit % H;
        const int n = seq_len(lens, b, T), t0 = a * N + lane * PL;
        if (a * N >= n) continue;
        double x[PL], db[PL];
#pragma unroll
        for (int i = 0; i < PL; ++i) x[i] = db[i] = 0;
        const size_t plane = (size_t)units * sw.NC * kDeltaChunk;
        const float* dot = sw.dot + (size_t)unit * sw.NC * kDeltaChunk + t0;
        for (int t = 0; t < tiles; ++t)
#pragma unroll
            for (int i = 0; i < PL; ++i)
                if (t0 + i < n) {
                    x[i] += dot[t * plane + i];
                    db[i] += dot[(tiles + t) * plane + i];
                }
        double anchor = 0;
        for (int i = 0; i < tiles * KM; ++i) anchor += sw.anchor[((size_t)unit * sw.NA + a) * tiles * KM + i];
        double s = 0;
#pragma unroll
        for (int i = PL - 1; i >= 0; --i) x[i] = s += x[i];                    // to the end of the lane's tokens
        double behind = s;                                                    // then of the lanes behind
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            const double down = __shfl_down(behind, o);
            if (lane + o < kWave) behind += down;
        }
        behind += anchor - s;
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (t0 + i < n) {
                const size_t to = ((size_t)b * T + t0 + i) * H + h;
                dg[to] = (float)(x[i] + behind);
                dbeta[to] = (float)db[i];
            }
    }
}

// ------------------------------------------------------------------ launches

// Byte offsets of the workspace's regions, each 256-byte aligned.
struct DeltaBackLayout {
    size_t blocks, e, S, Y, end, anchor, dot, total;
    int NC, NS, NA;
};
static DeltaBackLayout back_layout(int B, int T, int H, int dk, int dv, bool is_bf16) {
    DeltaBackLayout l;
    l.NC = (T + kDeltaChunk - 1) / kDeltaChunk;
    l.NS = (l.NC + kSuperChunks - 1) / kSuperChunks;
    l.NA = (l.NC + kAnchorChunks - 1) / kAnchorChunks;
    const size_t units = (size_t)B * H, state = (size_t)dk * dv;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t from = at;
        at += (bytes + 255) / 256 * 256;
        return from;
    };
    l.blocks = take(units * l.NC * delta_block_bytes(is_bf16, true));
    l.e = take(units * l.NC * dv * kDeltaChunk * 4);
    l.S = take(units * l.NS * state * (is_bf16 ? 2 : 4));
    l.Y = take(units * l.NS * state * (is_bf16 ? 2 : 4));
    l.end = take(units * l.NA * state * 4);
    l.anchor = take(units * l.NA * (dv / 16) * (dk / 32) * 4);
    l.dot = take(2 * (size_t)(dv / 16) * units * l.NC * kDeltaChunk * 4);
    l.total = at;
    return l;
}

size_t delta_backward_ws_bytes(int B, int T, int H, int, int dk, int dv, bool is_bf16) {
    return back_layout(B, T, H, dk, dv, is_bf16).total;
}

template <typename E, int DK>
static hipError_t launch_k(const DeltaBackward& a, const DeltaReverse& r, const DeltaQK& x, hipStream_t stream) {
    hipLaunchKernelGGL((delta_reverse_kernel<E, DK>), dim3((unsigned)(a.B * a.H * (a.dv_ / 16))), dim3(DK * 2), 0, stream, r);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((delta_qk_kernel<E, DK>), dim3((unsigned)(a.B * a.Hk * r.sweep.NS)), dim3(256), 0, stream, x);
    return hipGetLastError();
}

template <typename E>
static hipError_t launch_e(const DeltaBackward& a, const DeltaReverse& r, const DeltaQK& x, hipStream_t stream) {
    switch (a.dk_) {
        case 32: return launch_k<E, 32>(a, r, x, stream);
        case 64: return launch_k<E, 64>(a, r, x, stream);
        default: return launch_k<E, 128>(a, r, x, stream);
    }
}

hipError_t launch_delta_backward(const DeltaBackward& a, void* ws, hipStream_t stream) {
    const DeltaBackLayout l = back_layout(a.B, a.T, a.H, a.dk_, a.dv_, a.is_bf16);
    char* w = (char*)ws;
    const DeltaSweep sw{a.dO, (float*)(w + l.e), w + l.S, w + l.Y, (float*)(w + l.end), (float*)(w + l.anchor), (float*)(w + l.dot),
                        l.NC, l.NS, l.NA};
    const StateIO S = dense_state(a.S0, nullptr);
    hipError_t e = launch_delta_pairs({a.q, a.k, a.g, a.beta, a.scale, S, a.lens, w + l.blocks, a.B, a.T, a.H, a.Hk, a.dk_, 0, l.NC,
                                       a.is_bf16}, true, stream);
    if (e != hipSuccess) return e;
    const DeltaChain c{a.q, a.k, a.v, a.scale, S, a.lens, w + l.blocks, nullptr, a.B, a.T, a.H, a.Hk, a.dk_, a.dv_, 0, l.NC, a.is_bf16, sw};
    if ((e = launch_delta_sweep(c, stream)) != hipSuccess) return e;
    const DeltaReverse r{a.q, a.k, a.v, a.scale, a.dST, a.dS0, a.lens, w + l.blocks, a.dv, sw, a.B, a.T, a.H, a.Hk, a.dk_, a.dv_};
    const DeltaQK x{a.q, a.k, a.dv, a.g, a.beta, a.scale, a.lens, sw, a.dq, a.dk, a.B, a.T, a.H, a.Hk, a.dk_, a.dv_};
    e = a.is_bf16 ? launch_e<bf16>(a, r, x, stream) : launch_e<float>(a, r, x, stream);
    if (e != hipSuccess) return e;
    const long long gates = ((long long)a.B * a.H * l.NA + 3) / 4;
    hipLaunchKernelGGL(delta_gates_kernel, dim3((unsigned)std::min<long long>(gates, 1 << 20)), dim3(256), 0, stream, sw, a.lens, a.dg,
                       a.dbeta, a.B, a.T, a.H, a.dv_ / 16, a.dk_ / 32);
    return hipGetLastError();
}

}  // namespace kda
