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

// The chain from the last chunk to the first, as delta_chain_kernel: one workgroup of
// four waves per (b, h, 16 value columns), wave w with Y's rows of key channels
// 32 w .. and the chunk's 16 tokens of tile w, three barriers a chunk:
//   K Y of the wave's channels for all tokens                                    |
//   dU of the wave's tokens, e^G dO                                              |
//   Z = the inverse's transpose times dU of the wave's tokens, -e^G beta Z; and Z
//   with a token a lane for what leaves the kernel                               |
//   Y's update from all tokens
template <typename E, int DK>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 2 : 1) void delta_reverse_kernel(DeltaReverse p) {
    constexpr int C = kDeltaChunk, KM = DK / 32, ES = sizeof(E), NE = ES == 2 ? 1 : 3;
    using Blk = DeltaBlock<3, true>;
    constexpr int LK = NE == 1 ? 40 : 32, LV = 24;           // padded rows in LDS
    __shared__ __align__(16) bf16 s_k[KM][NE][C * LK], s_q[KM][NE][C * LK];   // a wave's own channels
    __shared__ __align__(16) bf16 s_o[NE][C * LV];           // dO's tile
    __shared__ f32x4 s_part[KM][kDeltaTiles][kWave];
    __shared__ __align__(16) char s_d[2][3 * kFragBytes], s_gq[2][3 * kFragBytes], s_gr[2][3 * kFragBytes];

    const int tiles = p.dv / 16, units = p.B * p.H;
    int unit, tile;
    unit_tile(blockIdx.x, units, tiles, unit, tile);
    const int b = unit / p.H, h = unit % p.H, hk = h / (p.H / p.Hk);
    const int n = seq_len(p.lens, b, p.T), c_end = (n + C - 1) / C;
    const int w = wave_id(), lane = lane_id(), j = lane & 15, g = lane >> 4;
    const bool holds = KM == 4 || w < KM;                    // this wave has channels
    const DeltaSweep& sw = p.sweep;

    const size_t state = (size_t)DK * p.dv, at_state = (size_t)unit * state + (size_t)(32 * w + 8 * g) * p.dv + 16 * tile + j;
    f32x4 Y[2] = {zero4(), zero4()};
    if (holds && p.dST) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) Y[t][i] = p.dST[at_state + (size_t)(4 * t + i) * p.dv];
    }

    // ---- what a chunk reads.  Rows past the sequence's end, and chunks before the
    // first, give zeros.
    const int ldk = p.Hk * DK * ES, ldv = p.H * p.dv * ES;
    const size_t at_k = (((size_t)b * p.T) * p.Hk + hk) * DK * ES;
    const size_t at_v = (((size_t)b * p.T) * p.H + h) * p.dv * ES + (size_t)16 * tile * ES;
    const char* pb = p.blocks + (size_t)unit * sw.NC * Blk::bytes;
    auto rows_of = [&](int c) { return c >= 0 ? min(C, n - c * C) : 0; };
    auto rows_rsrc = [&](const void* base, size_t at, int c, int rows, int ld, int width) {
        return make_rsrc((const char*)base + at + (int64_t)max(c, 0) * C * ld, rows > 0 ? (uint32_t)((rows - 1) * ld + width) : 0);
    };
    auto blk_rsrc = [&](int c) { return make_rsrc(pb + (int64_t)max(c, 0) * Blk::bytes, c >= 0 ? Blk::bytes : 0); };
    Raw<E> rk[kDeltaTiles], rq[kDeltaTiles];
    u32x4 ro;
    f32x4 v, e, grow, end, beta, S[2];
    Terms<3> rt[2], rp[2];
    float beta_j, decay_f, decay_rest, dot;
    auto load_rows = [&](int c) {                            // K, Q and dO
        const int rows = rows_of(c);
        const Rsrc k = rows_rsrc(p.k, at_k, c, holds ? rows : 0, ldk, DK * ES), q = rows_rsrc(p.q, at_k, c, holds ? rows : 0, ldk, DK * ES);
#pragma unroll
        for (int a = 0; a < kDeltaTiles; ++a) {
            const int off = 16 * a + j < rows ? (16 * a + j) * ldk + (32 * w + 8 * g) * ES : kOffPast;
            rk[a] = raw_load<E>(k, off);
            rq[a] = raw_load<E>(q, off);
        }
        const int row = 16 * w + lane / ES;
        ro = buf_load<u32x4>(rows_rsrc(sw.dO, at_v, c, rows, ldv, 16 * ES),
                             lane < 16 * ES && row < rows ? row * ldv + lane % ES * 16 : kOffPast);
    };
    auto is_anchor = [&](int c) { return holds && c >= 0 && (c % kAnchorChunks == kAnchorChunks - 1 || c == c_end - 1); };
    auto anchor_at = [&](int c) { return (((size_t)unit * sw.NA + max(c, 0) / kAnchorChunks) * tiles + tile) * KM + (holds ? w : 0); };
    auto load_pair = [&](int c) {
        const Rsrc r = blk_rsrc(c);
#pragma unroll
        for (int x = 0; x < 2; ++x) rp[x] = load_terms<3>(r, x >= w / 2 ? Blk::pairt + upper(w, x) * 3 * kFragBytes : kOffPast);
        grow = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + (kRowGrow + 16 * w + 4 * g) * 4));
        end = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + (kRowEnd + 16 * w + 4 * g) * 4));
        const f32x4 d = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + kRowDecay * 4));
        decay_f = d[0];
        decay_rest = d[1];
        const Rsrc m = make_rsrc((const f32x4*)sw.end + anchor_at(c) * 2 * kWave, 2 * kWave * 16);
#pragma unroll
        for (int t = 0; t < 2; ++t)
            S[t] = __builtin_bit_cast(f32x4, buf_load<u32x4>(m, is_anchor(c) ? (t * kWave + lane) * 16 : kOffPast));
    };
    auto load_inv = [&](int c) {                             // and what the outputs take: v, e and dO . o of token 16 w + j
        const int rows = rows_of(c);
        const Rsrc r = blk_rsrc(c);
#pragma unroll
        for (int x = 0; x < 2; ++x) rt[x] = load_terms<3>(r, x >= w / 2 ? Blk::invt + upper(w, x) * 3 * kFragBytes : kOffPast);
        beta = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + (kRowBeta + 16 * w + 4 * g) * 4));
        beta_j = __builtin_bit_cast(float, buf_load<uint32_t>(r, Blk::row + (kRowBeta + 16 * w + j) * 4));
        v = buf_load4<E>(rows_rsrc(p.v, at_v, c, rows, ldv, 16 * ES), 16 * w + j < rows ? (16 * w + j) * ldv + 4 * g * ES : kOffPast);
        const Rsrc re = make_rsrc(sw.e + (((size_t)unit * sw.NC + max(c, 0)) * p.dv + 16 * tile) * C, c >= 0 ? 16 * C * 4 : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = __builtin_bit_cast(float, buf_load<uint32_t>(re, ((4 * g + i) * C + 16 * w + j) * 4));
        const Rsrc rd = make_rsrc(sw.dot + (((size_t)tile * units + unit) * sw.NC + max(c, 0)) * C, c >= 0 ? C * 4 : 0);
        dot = __builtin_bit_cast(float, buf_load<uint32_t>(rd, (16 * w + j) * 4));
    };

    ChunkDecay decay;
    load_rows(c_end - 1);                                    // in the loop's order, as in delta_chain_kernel
    __builtin_amdgcn_sched_barrier(0);
    load_pair(c_end - 1);
    __builtin_amdgcn_sched_barrier(0);
    load_inv(c_end - 1);
    __builtin_amdgcn_sched_barrier(0);
    for (int c = c_end - 1; c >= 0; --c) {
        const int rows = min(C, n - c * C);
        // ---- K Y of the wave's channels; Y itself, for dk, and at an anchor <S, Y>
        buf_store8<E>(make_rsrc((E*)sw.Y + (((size_t)unit * sw.NC + c) * p.dv + 16 * tile) * DK, 16 * DK * ES),
                      holds ? (j * DK + 32 * w + 8 * g) * ES : kOffPast, Y[0], Y[1]);
        float a = 0.f;
        if (is_anchor(c)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a += S[0][i] * Y[0][i] + S[1][i] * Y[1][i];
#pragma unroll
            for (int o = 1; o < kWave; o <<= 1) a += __shfl_xor(a, o);
        }
        buf_store_u32(make_rsrc(sw.anchor + anchor_at(c), 4), is_anchor(c) && lane == 0 ? 0 : kOffPast, __builtin_bit_cast(uint32_t, a));
        if (holds) {
            const Terms<3> yf = split_terms<3>(Y[0], Y[1]);
#pragma unroll
            for (int x = 0; x < kDeltaTiles; ++x) {
                const Terms<NE> kt = raw_terms(rk[x]), qt = raw_terms(rq[x]);
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    *reinterpret_cast<bf16x8*>(&s_k[w][i][(16 * x + j) * LK + 8 * g]) = kt.t[i];
                    *reinterpret_cast<bf16x8*>(&s_q[w][i][(16 * x + j) * LK + 8 * g]) = qt.t[i];
                }
                s_part[w][x][lane] = mma(kt, yf, zero4());
            }
        }
        put_piece<E>(&s_o[0][(16 * w + min(lane / ES, 15)) * LV + lane % ES * (16 / ES)], C * LV, ro, lane < 16 * ES);
        load_rows(c - 1);
        __syncthreads();
        // ---- dU of the wave's tokens; e^G dO
        f32x4 u = s_part[0][w][lane];
#pragma unroll
        for (int m = 1; m < KM; ++m) u += s_part[m][w][lane];
        u *= end;
        if (w < 2) u = mma(rp[0], col_terms<NE>(&s_o[0][0], C * LV, LV, 0, 4, j, g), u);
        u = mma(rp[1], col_terms<NE>(&s_o[0][32 * LV], C * LV, LV, 0, 4, j, g), u);
        put_half<3>(s_d[w >> 1], w & 1, u);
        put_half<3>(s_gq[w >> 1], w & 1, p.scale * grow * col4<NE>(&s_o[0][16 * w * LV], C * LV, LV, j, g));
        const f32x4 eg = grow;
        const float f = decay(decay_f, decay_rest);
        load_pair(c - 1);
        __syncthreads();
        // ---- Z of the wave's tokens, a column a lane and (zt) a token a lane
        const Terms<3> d1 = frag_terms<3>(s_d[1]);
        f32x4 z = mma(rt[1], d1, zero4()), zt = mma(d1, rt[1], zero4());
        if (w < 2) {
            const Terms<3> d0 = frag_terms<3>(s_d[0]);
            z = mma(rt[0], d0, z);
            zt = mma(d0, rt[0], zt);
        }
        put_half<3>(s_gr[w >> 1], w & 1, -eg * (beta * z));
        // ---- out: dv = beta Z; dO . o - dv . v, and dbeta = Z . E
        {
            const f32x4 r = beta_j * zt;
            float x = 0.f, db = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x += r[i] * v[i];
                db += zt[i] * e[i];
            }
            x += __shfl_xor(x, 16);
            x += __shfl_xor(x, 32);
            db += __shfl_xor(db, 16);
            db += __shfl_xor(db, 32);
            const int at = g == 0 ? (16 * w + j) * 4 : kOffPast;
            buf_store_u32(make_rsrc(sw.dot + (((size_t)tile * units + unit) * sw.NC + c) * C, C * 4), at, __builtin_bit_cast(uint32_t, dot - x));
            buf_store_u32(make_rsrc(sw.dot + (((size_t)(tiles + tile) * units + unit) * sw.NC + c) * C, C * 4), at,
                          __builtin_bit_cast(uint32_t, db));
            const Rsrc to = rows_rsrc(p.dv_out, at_v, c, rows, ldv, 16 * ES);
            const int off = 16 * w + j < rows ? (16 * w + j) * ldv + 4 * g * ES : kOffPast;
            if constexpr (ES == 2)
                buf_store_u32x2(to, off, __builtin_bit_cast(u32x2, pack4(r)));
            else
                buf_store_u32x4(to, off, __builtin_bit_cast(u32x4, r));
        }
        load_inv(c - 1);
        __syncthreads();
        // ---- Y' = e^{G_C} Y + Q^T (e^G dO) - K^T (e^G beta Z)
        if (holds) {
#pragma unroll
            for (int t = 0; t < 2; ++t) Y[t] *= f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const Terms<3> gq = frag_terms<3>(s_gq[x]), gr = frag_terms<3>(s_gr[x]);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    Y[t] = mma(col_terms<NE>(&s_q[w][0][32 * x * LK], C * LK, LK, 4 * t, 8, j, g), gq, Y[t]);
                    Y[t] = mma(col_terms<NE>(&s_k[w][0][32 * x * LK], C * LK, LK, 4 * t, 8, j, g), gr, Y[t]);
                }
            }
        }
    }
    if (holds && p.dS0) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) p.dS0[at_state + (size_t)(4 * t + i) * p.dv] = Y[t][i];
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

// One workgroup of eight waves per chunk of a head of q and k, over the heads that
// share it.  Over 64 value columns at a time (fp32: 32), in LDS: S^T and Y^T [64][DK],
// dO and dv [64][64], U^T [64][64], the next ones in flight.  Wave w makes the
// products with S and Y of channels 32 (w % 4) .. for two of the four token tiles
// (transposed: a token a lane), and of the tokens of tile w % 4 the pairs of dO
// (w < 4) or of R with all others, which then go through LDS as operands.
// With bf16 an operand is one bf16 term: what it leaves out is half a step on a
// part of the sum, beside the result's own rounding.
template <typename E, int DK>
__global__ __launch_bounds__(512, 2) void delta_qk_kernel(DeltaQK p) {
    constexpr int NE = sizeof(E) == 2 ? 1 : 3, ES = sizeof(E), PE = 16 / ES, L = kDeltaChunk, NT = 512;
    constexpr int CS = NE == 1 ? 64 : 32;                    // value columns at a time
    constexpr int LS = DK + 8, LT = CS + 8, LU = L + 8;      // padded rows
    constexpr int QS = CS * LS, QT = L * LT, QU = CS * LU, QK = L * LS;      // elements of a plane
    constexpr int kFrags = 3 * 4 * 2 * NE * kFragBytes;      // bytes of the pairs' operands
    constexpr int kStage1 = NE * (2 * QS + 2 * QT + QU) * 2, kStage2 = kFrags + NE * QK * 2;
    constexpr int RS = (CS * DK / PE + NT - 1) / NT, RT = (L * CS / PE + NT - 1) / NT, RU = (CS * L / 4 + NT - 1) / NT,
                  RK = (L * DK / PE + NT - 1) / NT;          // pieces of a thread
    __shared__ __align__(16) char s_mem[kStage1 > kStage2 ? kStage1 : kStage2];
    __shared__ __align__(16) float s_hi[L], s_lo[L], s_eg[L], s_end[L], s_beta[L];
    bf16 *s_S = reinterpret_cast<bf16*>(s_mem), *s_Y = s_S + NE * QS, *s_O = s_Y + NE * QS, *s_R = s_O + NE * QT, *s_U = s_R + NE * QT;
    char* s_frag = s_mem;                                    // then, in the same place, the pairs and K or Q
    bf16* s_K = reinterpret_cast<bf16*>(s_mem + kFrags);
    const DeltaSweep& sw = p.sweep;
    const int c = blockIdx.x / p.Hk % sw.NC, hk = blockIdx.x % p.Hk, b = blockIdx.x / p.Hk / sw.NC;
    const int n = seq_len(p.lens, b, p.T), t0 = c * L, rows = min(L, n - t0);
    if (rows <= 0) return;
    const int tid = threadIdx.x, wave = wave_id(), lane = lane_id(), j = lane & 15, g = lane >> 4, G = p.H / p.Hk;
    const int m = wave & 3, half = wave >> 2;                // channels 32 m .., token tiles 2 half ..; tokens of tile m, dO or R
    const bool mine = DK == 128 || m < DK / 32;              // this wave has channels
    f32x4 dq[2][2], dk[2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) dq[t][r] = dk[t][r] = zero4();

    for (int hg = 0; hg < G; ++hg) {
        const int h = hk * G + hg, unit = b * p.H + h;
        const Rsrc rS = make_rsrc((const E*)sw.S + ((size_t)unit * sw.NC + c) * p.dv_ * DK, (uint32_t)(p.dv_ * DK * ES));
        const Rsrc rY = make_rsrc((const E*)sw.Y + ((size_t)unit * sw.NC + c) * p.dv_ * DK, (uint32_t)(p.dv_ * DK * ES));
        const Rsrc rE = make_rsrc(sw.e + ((size_t)unit * sw.NC + c) * p.dv_ * L, (uint32_t)(p.dv_ * L * 4));
        const int ldv = p.H * p.dv_ * ES;
        const size_t tok = (((size_t)b * p.T + t0) * p.H + h) * p.dv_;
        const uint32_t tok_bytes = (uint32_t)((rows - 1) * ldv + p.dv_ * ES);
        const Rsrc rO = make_rsrc((const E*)sw.dO + tok, tok_bytes), rR = make_rsrc((const E*)p.dv + tok, tok_bytes);
        u32x4 xS[RS], xY[RS], xO[RT], xR[RT], xE[RU];
        auto load = [&](int c0) {                            // columns past the last: zeros
#pragma unroll
            for (int i = 0; i < RS; ++i) {
                const int at = (tid + i * NT) * 16 + c0 * DK * ES;
                const bool in = RS * NT * PE == CS * DK || tid + i * NT < CS * DK / PE;
                xS[i] = buf_load<u32x4>(rS, in ? at : kOffPast);
                xY[i] = buf_load<u32x4>(rY, in ? at : kOffPast);
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int t = (tid + i * NT) / (CS / PE), vc = c0 + (tid + i * NT) % (CS / PE) * PE;
                const int off = t < rows && vc < p.dv_ ? t * ldv + vc * ES : kOffPast;
                xO[i] = buf_load<u32x4>(rO, off);
                xR[i] = buf_load<u32x4>(rR, off);
            }
#pragma unroll
            for (int i = 0; i < RU; ++i) xE[i] = buf_load<u32x4>(rE, (tid + i * NT) * 16 + c0 * L * 4);
        };
        load(0);
        if (hg) __syncthreads();                             // the last head is done with LDS
        if (wave == 0) {
            const size_t at = ((size_t)b * p.T + t0 + lane) * p.H + h;
            double s = lane < rows ? (double)log_decay(p.g[at]) : 0.0;
#pragma unroll
            for (int o = 1; o < L; o <<= 1) {
                const double up = __shfl_up(s, o);
                if (lane >= o) s += up;
            }
            const double end = __shfl(s, L - 1);
            s_hi[lane] = (float)s;
            s_lo[lane] = (float)(s - (double)(float)s);
            s_eg[lane] = expf((float)s);
            s_end[lane] = expf((float)(end - s));
            s_beta[lane] = lane < rows ? p.beta[at] : 0.f;
        }
        __syncthreads();
        f32x4 aq[2][2], as[2][2], ay[2][2], pr[4], pd = zero4();
#pragma unroll
        for (int r = 0; r < 4; ++r) pr[r] = zero4();
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int t = 0; t < 2; ++t) aq[t][r] = as[t][r] = ay[t][r] = zero4();
        for (int c0 = 0; c0 < p.dv_; c0 += CS) {
            if (c0) __syncthreads();
#pragma unroll
            for (int i = 0; i < RS; ++i) {
                const int vc = (tid + i * NT) / (DK / PE), ch = (tid + i * NT) % (DK / PE) * PE;
                if (RS * NT * PE == CS * DK || vc < CS) {
                    put_piece<E>(s_S + vc * LS + ch, QS, xS[i]);
                    put_piece<E>(s_Y + vc * LS + ch, QS, xY[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int t = (tid + i * NT) / (CS / PE), vc = (tid + i * NT) % (CS / PE) * PE;
                put_piece<E>(s_O + t * LT + vc, QT, xO[i]);
                put_piece<E>(s_R + t * LT + vc, QT, xR[i]);
            }
#pragma unroll
            for (int i = 0; i < RU; ++i) {
                const int vc = (tid + i * NT) / (L / 4), t = (tid + i * NT) % (L / 4) * 4;
                f32x4 u = __builtin_bit_cast(f32x4, xE[i]) * *reinterpret_cast<const f32x4*>(&s_beta[t]);
#pragma unroll
                for (int s = 0; s < NE; ++s) {
                    const bf16x4 hi = pack4(u);
                    *reinterpret_cast<bf16x4*>(s_U + s * QU + vc * LU + t) = hi;
#pragma unroll
                    for (int x = 0; x < 4; ++x) u[x] -= (float)hi[x];
                }
            }
            __syncthreads();
            load(c0 + CS);
            // operands with a token a lane, value columns 32 k + 4 g .. and 32 k + 16 + 4 g ..
            auto tokens = [&](const bf16* s, int r, int k) {
                Terms<NE> f;
#pragma unroll
                for (int x = 0; x < NE; ++x) {
                    const bf16* at = s + x * QT + (16 * r + j) * LT + 32 * k + 4 * g;
                    const bf16x4 lo = *reinterpret_cast<const bf16x4*>(at), hi = *reinterpret_cast<const bf16x4*>(at + 16);
                    f.t[x] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                }
                return f;
            };
            auto written = [&](int r, int k) { return col_terms<NE>(s_U + 32 * k * LU, QU, LU, 16 * r, 4, j, g); };
#pragma unroll
            for (int k = 0; k < CS / 32; ++k) {
                if (c0 + 32 * k >= p.dv_) break;
                if (mine) {
                    Terms<NE> Sf[2], Yf[2];
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        Sf[t] = col_terms<NE>(s_S + 32 * k * LS, QS, LS, 32 * m + 4 * t, 8, j, g);
                        Yf[t] = col_terms<NE>(s_Y + 32 * k * LS, QS, LS, 32 * m + 4 * t, 8, j, g);
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const Terms<NE> O = tokens(s_O, 2 * half + r, k), R = tokens(s_R, 2 * half + r, k), U = written(2 * half + r, k);
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            aq[t][r] = mma(Sf[t], O, aq[t][r]);
                            as[t][r] = mma(Sf[t], R, as[t][r]);
                            ay[t][r] = mma(Yf[t], U, ay[t][r]);
                        }
                    }
                }
                const bf16* s_x = half ? s_R : s_O;
                const Terms<NE> Xw = tokens(s_x, m, k), Uw = written(m, k);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if (r <= m) pr[r] = mma(written(r, k), Xw, pr[r]);     // rows: what token r wrote, lane: the later one
                    if (r == m) pd = mma(Xw, Uw, pd);                      // rows: the later token, lane: what this one wrote
                    if (r > m) pr[r] = mma(tokens(s_x, r, k), Uw, pr[r]);
                }
            }
        }
        // ---- pairs with their decays, as operands with the output's token a lane:
        // (dO U^T)*D for dq, its transpose for dk, -(X + X^T) for dk
        f32x4 wa[4], wb[4];
        const float hi = s_hi[16 * m + j], lo = s_lo[16 * m + j];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const f32x4 rh = *reinterpret_cast<const f32x4*>(&s_hi[16 * r + 4 * g]), rl = *reinterpret_cast<const f32x4*>(&s_lo[16 * r + 4 * g]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = 16 * (m - r) + j - 4 * g - i;  // lane's token - row's token
                const float gap = (hi - rh[i]) + (lo - rl[i]), D = __expf(d >= 0 ? gap : -gap);
                const float later = r == m ? pd[i] : pr[r][i];
                if (half == 0) {
                    wa[r][i] = d >= 0 ? p.scale * D * pr[r][i] : 0.f;
                    wb[r][i] = d <= 0 ? p.scale * D * later : 0.f;
                } else {
                    wa[r][i] = d > 0 ? -D * pr[r][i] : d < 0 ? -D * later : 0.f;
                }
            }
        }
        auto put = [&](int kind, const f32x4 (&w)[4]) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                const Terms<NE> f = split_terms<NE>(w[2 * ks], w[2 * ks + 1]);
#pragma unroll
                for (int x = 0; x < NE; ++x)
                    reinterpret_cast<bf16x8*>(s_frag + (((kind * 4 + m) * 2 + ks) * NE + x) * kFragBytes)[lane] = f.t[x];
            }
        };
        const int ldk = p.Hk * DK * ES;
        const size_t row0 = (((size_t)b * p.T + t0) * p.Hk + hk) * DK;
        const uint32_t k_bytes = (uint32_t)((rows - 1) * ldk + DK * ES);
        const Rsrc rK = make_rsrc((const E*)p.k + row0, k_bytes), rQ = make_rsrc((const E*)p.q + row0, k_bytes);
        u32x4 xK[RK], xQ[RK];
#pragma unroll
        for (int i = 0; i < RK; ++i) {
            const int t = (tid + i * NT) / (DK / PE), ch = (tid + i * NT) % (DK / PE) * PE;
            const int off = t < rows ? t * ldk + ch * ES : kOffPast;
            xK[i] = buf_load<u32x4>(rK, off);
            xQ[i] = buf_load<u32x4>(rQ, off);
        }
        __syncthreads();                                     // every wave is done with the rows
        if (half == 0) {
            put(0, wa);
            put(1, wb);
        } else {
            put(2, wa);
        }
        if (mine) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int t16 = 16 * (2 * half + r) + j;
                const float eg = s_eg[t16], end = s_end[t16], sq = p.scale * eg;
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
            if (pass) __syncthreads();                       // K is used
#pragma unroll
            for (int i = 0; i < RK; ++i) {
                const int t = (tid + i * NT) / (DK / PE), ch = (tid + i * NT) % (DK / PE) * PE;
                if (RK * NT * PE == L * DK || t < L) put_piece<E>(s_K + t * LS + ch, QK, pass ? xQ[i] : xK[i]);
            }
            __syncthreads();                                 // with the pairs
            if (!mine) continue;
            auto frag = [&](int kind, int r, int ks) { return frag_terms<NE>(s_frag + ((kind * 4 + r) * 2 + ks) * NE * kFragBytes); };
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const Terms<NE> f = col_terms<NE>(s_K + 32 * ks * LS, QK, LS, 32 * m + 4 * t, 8, j, g);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int r = 2 * half + x;
                        if (pass == 0) {
                            if (ks <= half) dq[t][x] = mma(f, frag(0, r, ks), dq[t][x]);
                            dk[t][x] = mma(f, frag(2, r, ks), dk[t][x]);
                        } else if (ks >= half) {
                            dk[t][x] = mma(f, frag(1, r, ks), dk[t][x]);
                        }
                    }
                }
        }
    }
    if (!mine) return;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int t = 16 * (2 * half + r) + j;
        if (t >= rows) continue;
        const size_t at = (((size_t)b * p.T + t0 + t) * p.Hk + hk) * DK + 32 * m + 8 * g;
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
    int NC, NA;
};
static DeltaBackLayout back_layout(int B, int T, int H, int dk, int dv, bool is_bf16) {
    DeltaBackLayout l;
    l.NC = (T + kDeltaChunk - 1) / kDeltaChunk;
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
    l.S = take(units * l.NC * state * (is_bf16 ? 2 : 4));
    l.Y = take(units * l.NC * state * (is_bf16 ? 2 : 4));
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
    hipLaunchKernelGGL((delta_reverse_kernel<E, DK>), dim3((unsigned)(a.B * a.H * (a.dv_ / 16))), dim3(256), 0, stream, r);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((delta_qk_kernel<E, DK>), dim3((unsigned)(a.B * a.Hk * r.sweep.NC)), dim3(512), 0, stream, x);
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
                        l.NC, l.NA};
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
