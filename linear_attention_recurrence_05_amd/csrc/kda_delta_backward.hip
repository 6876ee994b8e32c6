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
// In each summand o holds p_r beta_r v_r of the token's own write (p = scale q . k)
// and dv holds beta_r p_r dO_r of its own output.  These cancel, and behind a strong
// decay they are all there is: left in, they cost dg its digits (of a head's norm 2e-5
// to 2e-4 with decays of e^-3, 5e-3 to 3e-2 with e^-10, many times it with e^-20, where
// it is 1e-6 to 8e-6 without them).  Without them a summand is
//   dO_r . (o'_r - beta_r p_r s_r) - beta_r y_r . v_r
// where o', s = S^T k and y = Y^T k are what the decayed state before r gives to the
// output and to the key, and the gradient behind r to the key: the first part is the
// forward sweep's, the second the reverse one's, and each has the decay of its token,
// or of the next, as a factor.  The sum is taken from t to the next anchor, a chunk's
// end at which <S, Y> is formed anew, for over a whole sequence it would carry its
// rounding along; there S is (I - beta k k^T) times the decayed state before the last
// token, whose y . v is left out, so that the anchor has its decay as a factor too.
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

// The chain from the last chunk to the first, as delta_chain: one workgroup of four
// waves per (b, h, 16 value columns), wave w with Y's rows of key channels
// 32 w .. and the chunk's 16 tokens of tile w, three barriers a chunk:
//   K Y of the wave's channels for all tokens                                    |
//   dU of the wave's tokens, e^G dO                                              |
//   Z = the inverse's transpose times dU of the wave's tokens, -e^G beta Z; and Z
//   with a token a lane for dv                                                   |
//   Y's update from all tokens
// P and the inverse come without their diagonal, so that y = Z - p dO, what later
// tokens alone give, is there before it is added.
template <typename E, int DK>
struct ReverseLds {
    static constexpr int C = kDeltaChunk, KM = DK / 32, NE = sizeof(E) == 2 ? 1 : 3;
    static constexpr int LK = NE == 1 ? 40 : 32, LV = 24;    // padded rows
    __align__(16) bf16 k[KM][NE][C * LK], q[KM][NE][C * LK]; // a wave's own channels
    __align__(16) bf16 o[NE][C * LV];                        // dO's tile
    __align__(16) bf16 v[4][NE][16 * LV];                    // a wave's own tokens of V
    f32x4 part[KM][kDeltaTiles][kWave];
    __align__(16) char d[2][3 * kFragBytes], gq[2][3 * kFragBytes], gr[2][3 * kFragBytes];
};
template <typename E, int DK>
__device__ __forceinline__ void delta_reverse(const DeltaReverse& p, int x, ReverseLds<E, DK>& s) {
    using Lds = ReverseLds<E, DK>;
    constexpr int C = kDeltaChunk, KM = DK / 32, ES = sizeof(E), NE = Lds::NE, LK = Lds::LK, LV = Lds::LV;
    using Blk = DeltaBlock<3, true>;
    const int tiles = p.dv / 16, units = p.B * p.H;
    int unit, tile;
    unit_tile(x, units, tiles, unit, tile);
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
    u32x4 ro, rv;
    f32x4 grow, end, beta, self;
    Terms<3> rt[2], rp[2];
    float beta_j, decay_f, decay_rest;
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
    auto is_anchor = [&](int c) { return c % kAnchorChunks == kAnchorChunks - 1 || c == c_end - 1; };
    auto anchor_at = [&](int c) { return (((size_t)unit * sw.NA + c / kAnchorChunks) * tiles + tile) * KM + (holds ? w : 0); };
    auto load_pair = [&](int c) {
        const Rsrc r = blk_rsrc(c);
#pragma unroll
        for (int x = 0; x < 2; ++x) rp[x] = load_terms<3>(r, x >= w / 2 ? Blk::pairt + upper(w, x) * 3 * kFragBytes : kOffPast);
        grow = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + (kRowGrow + 16 * w + 4 * g) * 4));
        end = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + (kRowEnd + 16 * w + 4 * g) * 4));
        self = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + (kRowSelf + 16 * w + 4 * g) * 4));
        const f32x4 d = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + kRowDecay * 4));
        decay_f = d[0];
        decay_rest = d[1];
    };
    auto load_inv = [&](int c) {                             // and V
        const int rows = rows_of(c);
        const Rsrc r = blk_rsrc(c);
#pragma unroll
        for (int x = 0; x < 2; ++x) rt[x] = load_terms<3>(r, x >= w / 2 ? Blk::invt + upper(w, x) * 3 * kFragBytes : kOffPast);
        beta = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + (kRowBeta + 16 * w + 4 * g) * 4));
        beta_j = __builtin_bit_cast(float, buf_load<uint32_t>(r, Blk::row + (kRowBeta + 16 * w + j) * 4));
        const int row = 16 * w + lane / ES;
        rv = buf_load<u32x4>(rows_rsrc(p.v, at_v, c, rows, ldv, 16 * ES),
                             lane < 16 * ES && row < rows ? row * ldv + lane % ES * 16 : kOffPast);
    };
    // the wave's tokens of their half of a chunk, as an operand
    Terms<1> own;
#pragma unroll
    for (int i = 0; i < 8; ++i) own.t[0][i] = (bf16)(i == 4 * (w & 1) + (j & 3) && g == j >> 2 ? 1.f : 0.f);

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
        buf_stream8<E>(make_rsrc((E*)sw.Y + (((size_t)unit * sw.NC + c) * p.dv + 16 * tile) * DK, 16 * DK * ES),
                      holds ? (j * DK + 32 * w + 8 * g) * ES : kOffPast, Y[0], Y[1]);
        const Rsrc ta = make_rsrc((f32x4*)sw.anchor + anchor_at(c) * 2 * kWave, 2 * kWave * 16);
#pragma unroll
        for (int t = 0; t < 2; ++t)
            buf_stream_u32x4(ta, holds && is_anchor(c) ? (t * kWave + lane) * 16 : kOffPast, __builtin_bit_cast(u32x4, Y[t]));
        if (holds) {
            const Terms<3> yf = split_terms<3>(Y[0], Y[1]);
#pragma unroll
            for (int x = 0; x < kDeltaTiles; ++x) {
                const Terms<NE> kt = raw_terms(rk[x]), qt = raw_terms(rq[x]);
#pragma unroll
                for (int i = 0; i < NE; ++i) {
                    *reinterpret_cast<bf16x8*>(&s.k[w][i][(16 * x + j) * LK + 8 * g]) = kt.t[i];
                    *reinterpret_cast<bf16x8*>(&s.q[w][i][(16 * x + j) * LK + 8 * g]) = qt.t[i];
                }
                s.part[w][x][lane] = mma(kt, yf, zero4());
            }
        }
        put_piece<E>(&s.o[0][(16 * w + min(lane / ES, 15)) * LV + lane % ES * (16 / ES)], C * LV, ro, lane < 16 * ES);
        load_rows(c - 1);
        __syncthreads();
        // ---- dU of the wave's tokens; e^G dO
        f32x4 u = s.part[0][w][lane];
#pragma unroll
        for (int m = 1; m < KM; ++m) u += s.part[m][w][lane];
        u *= end;
        if (w < 2) u = mma(rp[0], col_terms<NE>(&s.o[0][0], C * LV, LV, 0, 4, j, g), u);
        u = mma(rp[1], col_terms<NE>(&s.o[0][32 * LV], C * LV, LV, 0, 4, j, g), u);
        const f32x4 dO = col4<NE>(&s.o[0][16 * w * LV], C * LV, LV, j, g), p_own = self;
        f32x4 all;                                           // one rounding, not two
#pragma unroll
        for (int i = 0; i < 4; ++i) all[i] = u[i] + p_own[i] * dO[i];
        put_half<3>(s.d[w >> 1], w & 1, all);
        put_half<3>(s.gq[w >> 1], w & 1, p.scale * grow * dO);
        const f32x4 eg = grow;
        const float f = decay(decay_f, decay_rest);
        load_pair(c - 1);
        __syncthreads();
        // ---- Z of the wave's tokens, a column a lane and (zt) a token a lane
        const Terms<3> d1 = frag_terms<3>(s.d[1]);
        Sum2 ys;
        ys.add(rt[1], d1);
        f32x4 zt = mma(d1, rt[1], zero4());
        if (w < 2) {
            const Terms<3> d0 = frag_terms<3>(s.d[0]);
            ys.add(rt[0], d0);
            zt = mma(d0, rt[0], zt);
            zt = mma(d0, own, zt);
        } else {
            zt = mma(d1, own, zt);
        }
        put_piece<E>(&s.v[w][0][min(lane / ES, 15) * LV + lane % ES * (16 / ES)], 16 * LV, rv, lane < 16 * ES);
        wave_fence();
        const f32x4 y = u + ys.sum();
        f32x4 z;
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = y[i] + p_own[i] * dO[i];
        put_half<3>(s.gr[w >> 1], w & 1, -eg * (beta * z));
        // ---- out: Z; dv = beta Z; beta y . v
        {
            const Rsrc tz = make_rsrc(sw.z + (((size_t)unit * sw.NC + c) * p.dv + 16 * tile) * C, 16 * C * 4);
            buf_stream_u32x4(tz, (j * C + 16 * w + 4 * g) * 4, __builtin_bit_cast(u32x4, z));
            const f32x4 v = col4<NE>(&s.v[w][0][0], 16 * LV, LV, j, g);
            float x = lane_row(beta, j) * row_sums(v * y, j);   // of token 16 w + 4 g + j % 4
            if (is_anchor(c) && 16 * w + 4 * g + (j & 3) == rows - 1) x = 0.f;
            wave_fence();                                    // before the next chunk's v
            buf_store_u32(make_rsrc(sw.dot + (((size_t)(tiles + tile) * units + unit) * sw.NC + c) * C, C * 4),
                          j < 4 ? (16 * w + 4 * g + j) * 4 : kOffPast, __builtin_bit_cast(uint32_t, x));
            const f32x4 r = beta_j * zt;
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
            Sum2 sum[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const Terms<3> gq = frag_terms<3>(s.gq[x]), gr = frag_terms<3>(s.gr[x]);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    sum[t].add(col_terms<NE>(&s.q[w][0][32 * x * LK], C * LK, LK, 4 * t, 8, j, g), gq);
                    sum[t].add(col_terms<NE>(&s.k[w][0][32 * x * LK], C * LK, LK, 4 * t, 8, j, g), gr);
                }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) Y[t][i] = f * Y[t][i] + sum[t].sum()[i];
        }
    }
    if (holds && p.dS0) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) p.dS0[at_state + (size_t)(4 * t + i) * p.dv] = Y[t][i];
    }
}

// Both sweeps at once, for neither needs the other.  Where they leave CUs idle this
// hides the shorter one (fp32 B3 H8 T333 d64: 28 us against 23 and 28 one after the
// other); where each fills the device with a workgroup a CU, the other's waves issue
// while one's wait (B1 H32 T4096 d128 bf16: 373 us against 193 and 233; with every
// chunk's operands in L2 it was 285).  Eight waves a workgroup, which halve what
// a wave does, took 460 us there, for two of them find no registers beside each other.
template <typename E, int DK>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 2 : 1) void delta_sweeps_kernel(DeltaChain f, DeltaReverse r) {
    __shared__ union Lds {
        ChainLds<E, DK, true> f;
        ReverseLds<E, DK> r;
    } s;
    const int half = gridDim.x / 2;
    if ((int)blockIdx.x < half)
        delta_chain<E, DK, true>(f, blockIdx.x, s.f);
    else
        delta_reverse<E, DK>(r, blockIdx.x - half, s.r);
}

// ------------------------------------------------------------------ dq and dk

struct DeltaQK {
    const void *q, *k;
    const float *g, *beta;
    float scale;
    const int* lens;
    DeltaSweep sweep;
    void *dq, *dk;
    float *dbeta, *part;   // part: where heads share q and k, each one's dq and dk
    int B, T, H, Hk, dk_, dv_;
};

// One workgroup of eight waves per chunk and head.  Over 32 value columns at a time,
// in LDS: S^T and Y^T [32][DK], dO [64][32], U^T and R^T [32][64], the next ones in
// flight.  Wave w makes the products with S and Y of channels 32 (w % 4) .. for two
// of the four token tiles (transposed: a token a lane), and of the tokens of tile
// w % 4 the pairs of dO (w < 4) or of R with all others, which then go through LDS
// as operands.  dbeta = Z . E on the way.
// With bf16 U, R and the pairs' weights are two bf16 terms, S and Y one (what they
// leave out is half a step on a part of the sum, beside the result's own rounding:
// dq and dk are off by 2.1e-3 to 2.6e-3 of their norm, 1.7e-3 of it that rounding, more
// only where a large state is undone by the chunk's own tokens; with all of them one
// term they were off by 3.0e-3, with S and Y two by that rounding alone, for 628 us of
// the whole call instead of 551).  Bound by the latency of what it reads, 180 KB a chunk and
// head with one workgroup a CU: B1 H32 T4096 d128 takes 124 us, 3.2 TB/s.  32 columns
// of 64, with 168 registers (64 of them took 3 us more); two workgroups a CU (128
// registers) spilled and took 287 us.
template <typename E, int DK>
__global__ __launch_bounds__(512, 2) void delta_qk_kernel(DeltaQK p) {
    constexpr int NE = sizeof(E) == 2 ? 1 : 3, NU = NE == 1 ? 2 : 3, ES = sizeof(E), PE = 16 / ES, L = kDeltaChunk, NT = 512;
    constexpr int CS = 32;                                   // value columns at a time
    constexpr int LS = kRowLd<DK>, LT = CS + 8, LU = L + 8;  // padded rows
    constexpr int QS = CS * LS, QT = L * LT, QU = CS * LU, QK = L * LS;      // elements of a plane
    constexpr int kFrags = 3 * 4 * 2 * NU * kFragBytes;      // bytes of the pairs' operands
    constexpr int kStage1 = (NE * (2 * QS + QT) + NU * 2 * QU) * 2, kStage2 = kFrags + NE * QK * 2;
    constexpr int RS = (CS * DK / PE + NT - 1) / NT, RT = (L * CS / PE + NT - 1) / NT, RU = (CS * L / 4 + NT - 1) / NT,
                  RK = (L * DK / PE + NT - 1) / NT;          // pieces of a thread
    __shared__ __align__(16) char s_mem[kStage1 > kStage2 ? kStage1 : kStage2];
    __shared__ __align__(16) float s_hi[L], s_lo[L], s_eg[L], s_end[L], s_beta[L], s_db[8][L];
    bf16 *s_S = reinterpret_cast<bf16*>(s_mem), *s_Y = s_S + NE * QS, *s_O = s_Y + NE * QS, *s_U = s_O + NE * QT, *s_R = s_U + NU * QU;
    char* s_frag = s_mem;                                    // then, in the same place, the pairs and K or Q
    bf16* s_K = reinterpret_cast<bf16*>(s_mem + kFrags);
    const DeltaSweep& sw = p.sweep;
    const int h = blockIdx.x % p.H, c = blockIdx.x / p.H % sw.NC, b = blockIdx.x / p.H / sw.NC, hk = h / (p.H / p.Hk);
    const int n = seq_len(p.lens, b, p.T), t0 = c * L, rows = min(L, n - t0);
    if (rows <= 0) return;
    const int tid = threadIdx.x, wave = wave_id(), lane = lane_id(), j = lane & 15, g = lane >> 4;
    const int m = wave & 3, half = wave >> 2;                // channels 32 m .., token tiles 2 half ..; tokens of tile m, dO or R
    const bool mine = DK == 128 || m < DK / 32;              // this wave has channels
    const int unit = b * p.H + h;
    const Rsrc rS = make_rsrc((const E*)sw.S + ((size_t)unit * sw.NC + c) * p.dv_ * DK, (uint32_t)(p.dv_ * DK * ES));
    const Rsrc rY = make_rsrc((const E*)sw.Y + ((size_t)unit * sw.NC + c) * p.dv_ * DK, (uint32_t)(p.dv_ * DK * ES));
    const Rsrc rE = make_rsrc(sw.e + ((size_t)unit * sw.NC + c) * p.dv_ * L, (uint32_t)(p.dv_ * L * 4));
    const Rsrc rZ = make_rsrc(sw.z + ((size_t)unit * sw.NC + c) * p.dv_ * L, (uint32_t)(p.dv_ * L * 4));
    const int ldv = p.H * p.dv_ * ES;
    const size_t tok = (((size_t)b * p.T + t0) * p.H + h) * p.dv_;
    const uint32_t tok_bytes = (uint32_t)((rows - 1) * ldv + p.dv_ * ES);
    const Rsrc rO = make_rsrc((const E*)sw.dO + tok, tok_bytes);
    u32x4 xS[RS], xY[RS], xO[RT], xE[RU], xZ[RU];
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
            xO[i] = buf_load<u32x4>(rO, t < rows && vc < p.dv_ ? t * ldv + vc * ES : kOffPast);
        }
#pragma unroll
        for (int i = 0; i < RU; ++i) {
            xE[i] = buf_load<u32x4>(rE, (tid + i * NT) * 16 + c0 * L * 4);
            xZ[i] = buf_load<u32x4>(rZ, (tid + i * NT) * 16 + c0 * L * 4);
        }
    };
    load(0);
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
    f32x4 aq[2][2], as[2][2], ay[2][2], pr[4], pd = zero4(), db = zero4();
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
            if (RT * NT * PE == L * CS || t < L) put_piece<E>(s_O + t * LT + vc, QT, xO[i]);
        }
#pragma unroll
        for (int i = 0; i < RU; ++i) {
            const int vc = (tid + i * NT) / (L / 4), t = (tid + i * NT) % (L / 4) * 4;
            const f32x4 e = __builtin_bit_cast(f32x4, xE[i]), z = __builtin_bit_cast(f32x4, xZ[i]);
            const f32x4 beta = *reinterpret_cast<const f32x4*>(&s_beta[t]);
            db += e * z;
            put_words<NU>(s_U + vc * LU + t, QU, beta * e);
            put_words<NU>(s_R + vc * LU + t, QU, beta * z);
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
        auto columns = [&](const bf16* s, int r, int k) { return col_terms<NU>(s + 32 * k * LU, QU, LU, 16 * r, 4, j, g); };
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
                    const Terms<NE> O = tokens(s_O, 2 * half + r, k);
                    const Terms<NU> R = columns(s_R, 2 * half + r, k), U = columns(s_U, 2 * half + r, k);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        aq[t][r] = mma(Sf[t], O, aq[t][r]);
                        as[t][r] = mma(Sf[t], R, as[t][r]);
                        ay[t][r] = mma(Yf[t], U, ay[t][r]);
                    }
                }
            }
            auto pairs = [&](auto X) {
                const auto Xw = X(m);
                const Terms<NU> Uw = columns(s_U, m, k);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if (r <= m) pr[r] = mma_top(columns(s_U, r, k), Xw, pr[r]);    // rows: what token r wrote, lane: the later one
                    if (r == m) pd = mma_top(Xw, Uw, pd);                          // rows: the later token, lane: what this one wrote
                    if (r > m) pr[r] = mma_top(X(r), Uw, pr[r]);
                }
            };
            if (half)
                pairs([&](int r) { return columns(s_R, r, k); });
            else
                pairs([&](int r) { return tokens(s_O, r, k); });
        }
    }
    // ---- dbeta
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        db[i] += __shfl_xor(db[i], 16);
        db[i] += __shfl_xor(db[i], 32);
    }
    if (g == 0) *reinterpret_cast<f32x4*>(&s_db[wave][4 * j]) = db;
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
            const Terms<NU> f = split_terms<NU>(w[2 * ks], w[2 * ks + 1]);
#pragma unroll
            for (int x = 0; x < NU; ++x)
                reinterpret_cast<bf16x8*>(s_frag + (((kind * 4 + m) * 2 + ks) * NU + x) * kFragBytes)[lane] = f.t[x];
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
    if (tid < rows) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += s_db[i][tid];
        p.dbeta[((size_t)b * p.T + t0 + tid) * p.H + h] = s;
    }
    if (half == 0) {
        put(0, wa);
        put(1, wb);
    } else {
        put(2, wa);
    }
    // dq = scale e^G dO S^T, dk = e^{G_C - G} U Y^T - e^G R S^T, to which the pairs add
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int t16 = 16 * (2 * half + r) + j;
        const float eg = s_eg[t16], end = s_end[t16], sq = p.scale * eg;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                aq[t][r][i] *= sq;
                ay[t][r][i] = end * ay[t][r][i] - eg * as[t][r][i];
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
        auto frag = [&](int kind, int r, int ks) { return frag_terms<NU>(s_frag + ((kind * 4 + r) * 2 + ks) * NU * kFragBytes); };
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const Terms<NE> f = col_terms<NE>(s_K + 32 * ks * LS, QK, LS, 32 * m + 4 * t, 8, j, g);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = 2 * half + x;
                    if (pass == 0) {
                        if (ks <= half) aq[t][x] = mma(f, frag(0, r, ks), aq[t][x]);
                        ay[t][x] = mma(f, frag(2, r, ks), ay[t][x]);
                    } else if (ks >= half) {
                        ay[t][x] = mma(f, frag(1, r, ks), ay[t][x]);
                    }
                }
            }
    }
    if (!mine) return;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int t = 16 * (2 * half + r) + j;
        if (t >= rows) continue;
        if (p.part) {
            float* to = p.part + (((size_t)b * p.T + t0 + t) * p.H + h) * 2 * DK + 32 * m + 8 * g;
            store8(to, aq[0][r], aq[1][r]);
            store8(to + DK, ay[0][r], ay[1][r]);
        } else {
            const size_t at = (((size_t)b * p.T + t0 + t) * p.Hk + hk) * DK + 32 * m + 8 * g;
            store8((E*)p.dq + at, aq[0][r], aq[1][r]);
            store8((E*)p.dk + at, ay[0][r], ay[1][r]);
        }
    }
}

// The sum over the G heads that share one of q and k, four channels a thread.  (One
// workgroup for all of them left most CUs idle: fp32 B3 H8 over 2 T333 d64 took 57 us,
// now 16.5 and 4.6.)
template <typename E>
__global__ __launch_bounds__(256) void delta_qk_sum_kernel(DeltaQK p) {
    const int G = p.H / p.Hk, PR = p.dk_ / 2;                // pieces of a token's dq and dk
    const size_t all = (size_t)p.B * p.T * p.Hk * PR;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (size_t)gridDim.x * 256) {
        const int piece = (int)(i % PR), hk = (int)(i / PR % p.Hk);
        const size_t tok = i / PR / p.Hk;
        if ((int)(tok % p.T) >= seq_len(p.lens, (int)(tok / p.T), p.T)) continue;
        f32x4 s = zero4();
        for (int x = 0; x < G; ++x)
            s += *reinterpret_cast<const f32x4*>(p.part + ((tok * p.H + hk * G + x) * PR + piece) * 4);
        E* to = (E*)(piece < PR / 2 ? p.dq : p.dk) + (tok * p.Hk + hk) * p.dk_ + piece % (PR / 2) * 4;
        if constexpr (sizeof(E) == 2)
            *reinterpret_cast<bf16x4*>(to) = pack4(s);
        else
            *reinterpret_cast<f32x4*>(to) = s;
    }
}

// ------------------------------------------------------------------ dg

// One workgroup per (b, h) and anchor: 256 tokens, one a thread, sums in 64 bits.  At a
// token whose decay is zero in fp32 dg is zero, and the sums of tokens before it end.
__global__ __launch_bounds__(256) void delta_gates_kernel(DeltaSweep sw, const float* __restrict__ g, const int* __restrict__ lens,
                                                          float* __restrict__ dg, int B, int T, int H, int tiles, int state) {
    constexpr int N = kAnchorChunks * kDeltaChunk;
    static_assert(N == 256, "a token a thread");
    __shared__ double s_x[4], s_a[4];
    __shared__ int s_end[4];
    const int units = B * H, unit = (int)(blockIdx.x % units), a = (int)(blockIdx.x / units), b = unit / H, h = unit % H;
    const int n = seq_len(lens, b, T), t = a * N + threadIdx.x, lane = lane_id(), wave = wave_id();
    if (a * N >= n) return;
    // <S, Y> at the anchor
    const f32x4* S = reinterpret_cast<const f32x4*>(sw.end + ((size_t)unit * sw.NA + a) * state);
    const f32x4* Y = reinterpret_cast<const f32x4*>(sw.anchor + ((size_t)unit * sw.NA + a) * state);
    double dot = 0;
#pragma unroll 8
    for (int i = threadIdx.x; i < state / 4; i += N) {
        const f32x4 s = S[i], y = Y[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) dot += (double)s[e] * (double)y[e];
    }
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) dot += __shfl_xor(dot, o);
    // the token's summand, and the sum from it to the wave's end or a zero decay
    double x = 0;
    int end = 0;
    if (t < n) {
        const size_t plane = (size_t)units * sw.NC * kDeltaChunk;
        const float* at = sw.dot + (size_t)unit * sw.NC * kDeltaChunk + t;
#pragma unroll 4
        for (int i = 0; i < tiles; ++i) x += (double)at[i * plane] - (double)at[(tiles + i) * plane];
        end = expf(log_decay(g[((size_t)b * T + t) * H + h])) == 0.f;
        x = end ? 0.0 : x;
    }
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const double down = __shfl_down(x, o);
        const int then = __shfl_down(end, o);
        if (lane + o < kWave && !end) {
            x += down;
            end = then;
        }
    }
    if (lane == 0) {
        s_x[wave] = x;
        s_end[wave] = end;
        s_a[wave] = dot;
    }
    __syncthreads();
    for (int i = wave + 1; i < 4 && !end; ++i) {
        x += s_x[i];
        end = s_end[i];
    }
    if (!end) x += (s_a[0] + s_a[1]) + (s_a[2] + s_a[3]);
    if (t < n) dg[((size_t)b * T + t) * H + h] = (float)x;
}

// ------------------------------------------------------------------ launches

// Byte offsets of the workspace's regions, each 256-byte aligned.
struct DeltaBackLayout {
    size_t blocks, e, z, S, Y, end, anchor, dot, part, total;
    int NC, NA;
};

static DeltaBackLayout back_layout(int B, int T, int H, int Hk, int dk, int dv, bool is_bf16) {
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
    l.z = take(units * l.NC * dv * kDeltaChunk * 4);
    l.S = take(units * l.NC * state * (is_bf16 ? 2 : 4));
    l.Y = take(units * l.NC * state * (is_bf16 ? 2 : 4));
    l.end = take(units * l.NA * state * 4);
    l.anchor = take(units * l.NA * state * 4);
    l.dot = take(2 * (size_t)(dv / 16) * units * l.NC * kDeltaChunk * 4);
    l.part = take(H > Hk ? (size_t)B * T * H * 2 * dk * 4 : 0);
    l.total = at;
    return l;
}

size_t delta_backward_ws_bytes(int B, int T, int H, int Hk, int dk, int dv, bool is_bf16) {
    return back_layout(B, T, H, Hk, dk, dv, is_bf16).total;
}

template <typename E, int DK>
static hipError_t launch_k(const DeltaBackward& a, const DeltaChain& f, const DeltaReverse& r, const DeltaQK& x, hipStream_t stream) {
    hipLaunchKernelGGL((delta_sweeps_kernel<E, DK>), dim3((unsigned)(2 * a.B * a.H * (a.dv_ / 16))), dim3(256), 0, stream, f, r);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((delta_qk_kernel<E, DK>), dim3((unsigned)(a.B * a.H * r.sweep.NC)), dim3(512), 0, stream, x);
    if ((e = hipGetLastError()) != hipSuccess || !x.part) return e;
    const size_t pieces = (size_t)a.B * a.T * a.Hk * (DK / 2);
    hipLaunchKernelGGL((delta_qk_sum_kernel<E>), dim3((unsigned)std::min<size_t>((pieces + 255) / 256, 1 << 20)), dim3(256), 0, stream, x);
    return hipGetLastError();
}

template <typename E>
static hipError_t launch_e(const DeltaBackward& a, const DeltaChain& f, const DeltaReverse& r, const DeltaQK& x, hipStream_t stream) {
    switch (a.dk_) {
        case 32: return launch_k<E, 32>(a, f, r, x, stream);
        case 64: return launch_k<E, 64>(a, f, r, x, stream);
        default: return launch_k<E, 128>(a, f, r, x, stream);
    }
}

hipError_t launch_delta_backward(const DeltaBackward& a, void* ws, hipStream_t stream) {
    const DeltaBackLayout l = back_layout(a.B, a.T, a.H, a.Hk, a.dk_, a.dv_, a.is_bf16);
    char* w = (char*)ws;
    const DeltaSweep sw{a.dO, (float*)(w + l.e), (float*)(w + l.z), w + l.S, w + l.Y, (float*)(w + l.end), (float*)(w + l.anchor), (float*)(w + l.dot),
                        l.NC, l.NA};
    const StateIO S = dense_state(a.S0, nullptr);
    hipError_t e = launch_delta_pairs({a.q, a.k, a.g, a.beta, a.scale, S, a.lens, w + l.blocks, a.B, a.T, a.H, a.Hk, a.dk_, 0, l.NC,
                                       a.is_bf16}, true, stream);
    if (e != hipSuccess) return e;
    const DeltaChain c{a.q, a.k, a.v, a.scale, S, a.lens, w + l.blocks, nullptr, a.B, a.T, a.H, a.Hk, a.dk_, a.dv_, 0, l.NC, a.is_bf16, sw};
    const DeltaReverse r{a.q, a.k, a.v, a.scale, a.dST, a.dS0, a.lens, w + l.blocks, a.dv, sw, a.B, a.T, a.H, a.Hk, a.dk_, a.dv_};
    const DeltaQK x{a.q, a.k, a.g, a.beta, a.scale, a.lens, sw, a.dq, a.dk, a.dbeta,
                    a.H > a.Hk ? (float*)(w + l.part) : nullptr, a.B, a.T, a.H, a.Hk, a.dk_, a.dv_};
    e = a.is_bf16 ? launch_e<bf16>(a, c, r, x, stream) : launch_e<float>(a, c, r, x, stream);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(delta_gates_kernel, dim3((unsigned)(a.B * a.H * l.NA)), dim3(256), 0, stream, sw, a.g, a.lens, a.dg, a.B, a.T, a.H,
                       a.dv_ / 16, a.dk_ * a.dv_);
    return hipGetLastError();
}

}  // namespace kda
