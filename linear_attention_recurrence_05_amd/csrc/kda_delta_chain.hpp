// kda_delta_chain.hpp -- the state's chain over the chunks of the gated delta rule
// (kda_delta_chunk.hpp) for 16 value columns of one head: the prefill, or the
// gradients' forward sweep.
#pragma once

#include "kda_delta_chunk.hpp"

namespace kda {

// Chunks from one anchor <S, Y> of dg (kda_delta_backward.hip) to the next.  Twice as
// many cost dg a quarter of its accuracy (fp32 B3 T333: 6.5e-7 of the norm against
// 4.8e-7) for 8 us of 560 (B1 H32 T4096 bf16).
constexpr int kAnchorChunks = 4;

// What the gradients' sweeps leave in the workspace, for unit u = b H + h, chunk
// c of NC, anchor a of NA, column tile t of `tiles`:
//   e, z  [u][c][dv][64] fp32        e_t of every token, and its gradient Z
//   S, Y  [u][c][dv][dk] of E        the state before a chunk, and the gradient of
//                                    the one behind it, transposed
//   end, anchor  [u][a][t] state tiles   the state at an anchor, less what its last
//                                    token wrote of v, and its gradient, as the chains
//                                    hold them
//   dot   [2][t][u][64 NC] fp32      parts of dg's summands (kda_delta_backward.hip),
//                                    the forward sweep's and the reverse one's
struct DeltaSweep {
    const void* dO;
    float *e, *z;
    void *S, *Y;
    float *end, *anchor, *dot;
    int NC, NA;
};

// Chunks c0 .. c1 - 1 from the state S.in to S.out.
struct DeltaChain {
    const void *q, *k, *v;
    float scale;
    StateIO S;
    const int* lens;
    const char* blocks;     // of chunks c0 .. c1 - 1
    void* o;
    int B, T, H, Hk, dk, dv, c0, c1;
    bool is_bf16;
    DeltaSweep sweep;       // of the gradients' forward sweep, which leaves no o
};
// The prefill's chain by one workgroup per (b, h): bf16, dv = 128.
hipError_t launch_delta_wide(const DeltaChain& a, hipStream_t stream);

// One workgroup of four waves per (b, h, 16 value columns).  Wave w holds the
// state's rows of key channels 32 w .. (if there are as many), as two accumulator
// tiles whose rows are mapped to channels so that a lane's rows of both are eight
// consecutive channels: an operand of K S and Q S without a move.  It also has the
// chunk's 16 tokens of tile w.  A chunk goes through three barriers:
//   K S of the wave's channels for all tokens, and the channels' terms of S    |
//   R = V - e^G K S of the wave's tokens (the waves' parts summed in order), Q S |
//   E = inv R of the wave's tokens                                             |
//   the state's update from all tokens' E; o of the wave's tokens
// so that nothing is computed twice but the operands' reads from LDS.  A wave
// issues an instruction in about five cycles whatever it is, and what a chunk
// costs is their number (64 tokens: about 400) and the barriers.  Registers that a
// part has used are loaded for the next chunk at once, a chunk ahead.
// BACK: the gradients' forward sweep, which leaves e, the states and its part of dg's
// summands: of o and K S what older tokens give alone (the block's matrices have no
// diagonal there), with fp32's accuracy (three terms).
template <typename E, int DK, bool BACK>
struct ChainLds {
    static constexpr int C = kDeltaChunk, KM = DK / 32, NE = sizeof(E) == 2 ? 1 : 3;
    // Terms of the state in Q S, of E and of the pairs' weights in o.  With bf16 two of
    // each leave o its own rounding.  One of the weights would do with half a step on
    // each pair, and 6.5 us of B1 H32 T4096's 137 (70 of B8 H32 T8192's 1,320): 2.4e-3 of
    // the norm instead of 1.7e-3 for rows at random, but up to 9e-3 where queries and
    // keys have most of their length in common and the pairs' sum nearly cancels.
    static constexpr int NS = BACK || NE == 3 ? 3 : 2, NO = NS, NP = NS;
    static constexpr int LK = NE == 1 ? 40 : 32, LV = 24;    // padded rows
    __align__(16) bf16 k[KM][NE][C * LK];                    // a wave's own channels of K
    __align__(16) bf16 v[4][NE][16 * LV];                    // a wave's own tokens of V
    __align__(16) char S[KM][NS * kFragBytes];
    f32x4 part[KM][kDeltaTiles][kWave];
    __align__(16) char r[2][3 * kFragBytes], u[2][3 * kFragBytes], e[2][NO * kFragBytes];
    __align__(16) bf16 d[BACK ? 4 : 1][NE][16 * LV];         // a wave's own tokens of dO
    float write[16];                                         // beta v of an anchor's last token
};
template <typename E, int DK, bool BACK>
__device__ __forceinline__ void delta_chain(const DeltaChain& p, int x, ChainLds<E, DK, BACK>& s) {
    using Lds = ChainLds<E, DK, BACK>;
    constexpr int C = kDeltaChunk, KM = DK / 32, ES = sizeof(E), NE = Lds::NE, NS = Lds::NS, NO = Lds::NO, NP = Lds::NP;
    constexpr int LK = Lds::LK, LV = Lds::LV;
    using Blk = DeltaBlock<NP, BACK>;
    const int tiles = p.dv / 16, units = p.B * p.H;
    int unit, tile;
    unit_tile(x, units, tiles, unit, tile);
    const int b = unit / p.H, h = unit % p.H, hk = h / (p.H / p.Hk);
    if (p.S.skip(b)) return;
    const int n = seq_len(p.lens, b, p.T), c_end = min(p.c1, (n + C - 1) / C);
    const int w = wave_id(), lane = lane_id(), j = lane & 15, g = lane >> 4;
    const bool holds = KM == 4 || w < KM;                    // this wave has channels

    // ---- the state's rows: tile t, channel 32 w + 8 g + 4 t + i, column j
    const size_t state = (size_t)DK * p.dv, at_state = (size_t)(32 * w + 8 * g) * p.dv + 16 * tile + j;
    f32x4 M[2] = {zero4(), zero4()};
    if (holds && p.S.in) {
        const float* in = p.S.in + ((size_t)(p.S.in_slot ? p.S.in_slot[b] : b) * p.H + h) * state + at_state;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) M[t][i] = in[(size_t)(4 * t + i) * p.dv];
    }

    // ---- what a chunk reads.  Rows past the sequence's end, and chunks past the
    // last, give zeros.
    const int ldk = p.Hk * DK * ES, ldv = p.H * p.dv * ES;
    const char* pk = (const char*)p.k + (((size_t)b * p.T + (size_t)p.c0 * C) * p.Hk + hk) * DK * ES;
    const char* pq = (const char*)p.q + (((size_t)b * p.T + (size_t)p.c0 * C) * p.Hk + hk) * DK * ES;
    const size_t at_v = (((size_t)b * p.T + (size_t)p.c0 * C) * p.H + h) * p.dv * ES + (size_t)16 * tile * ES;
    const char* pb = p.blocks + (size_t)unit * (p.c1 - p.c0) * Blk::bytes;
    auto rows_of = [&](int c) { return c < c_end ? min(C, n - c * C) : 0; };
    auto rows_rsrc = [&](const char* base, int rows, int ld, int width) {
        return make_rsrc(base, rows > 0 ? (uint32_t)((rows - 1) * ld + width) : 0);
    };
    Raw<E> rk[kDeltaTiles], rq[KM];
    u32x4 rv;
    Terms<3> rt[2];
    Terms<NP> rp[2];
    f32x4 grow, write;
    float grow_j, decay_f, decay_rest;
    u32x4 rd = {0, 0, 0, 0};                                 // BACK: dO, as v
    f32x4 self = zero4();                                    // beta p of the wave's tokens
    auto load_k = [&](int c) {
        const int rows = rows_of(c);
        const Rsrc r = rows_rsrc(pk + (int64_t)(c - p.c0) * C * ldk, holds ? rows : 0, ldk, DK * ES);
#pragma unroll
        for (int a = 0; a < kDeltaTiles; ++a)
            rk[a] = raw_load<E>(r, 16 * a + j < rows ? (16 * a + j) * ldk + (32 * w + 8 * g) * ES : kOffPast);
    };
    auto load_qv = [&](int c) {
        const int rows = rows_of(c);
        const Rsrc r = rows_rsrc(pq + (int64_t)(c - p.c0) * C * ldk, rows, ldk, DK * ES);
        const int off = 16 * w + j < rows ? (16 * w + j) * ldk + 8 * g * ES : kOffPast;
#pragma unroll
        for (int m = 0; m < KM; ++m) rq[m] = raw_load<E>(r, off + 32 * m * ES);
        // v's tile of 16 rows of 16 elements: 16 bytes a lane (bf16: half the lanes)
        const Rsrc v = rows_rsrc((const char*)p.v + at_v + (int64_t)(c - p.c0) * C * ldv, rows, ldv, 16 * ES);
        const int row = 16 * w + lane / ES;
        const int at = lane < 16 * ES && row < rows ? row * ldv + lane % ES * 16 : kOffPast;
        rv = buf_load<u32x4>(v, at);
        if constexpr (BACK)
            rd = buf_load<u32x4>(rows_rsrc((const char*)p.sweep.dO + at_v + (int64_t)(c - p.c0) * C * ldv, rows, ldv, 16 * ES), at);
    };
    auto blk_rsrc = [&](int c) { return make_rsrc(pb + (int64_t)(c - p.c0) * Blk::bytes, c < c_end ? Blk::bytes : 0); };
    auto load_inv = [&](int c) {
        const Rsrc r = blk_rsrc(c);
#pragma unroll
        for (int x = 0; x < 2; ++x) rt[x] = load_terms<3>(r, x <= w / 2 ? Blk::inv + lower(w, x) * 3 * kFragBytes : kOffPast);
        write = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + (kRowWrite + 16 * w + 4 * g) * 4));
        if constexpr (BACK) self = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + (kRowBetaSelf + 16 * w + 4 * g) * 4));
    };
    auto load_pair = [&](int c) {
        const Rsrc r = blk_rsrc(c);
#pragma unroll
        for (int x = 0; x < 2; ++x) rp[x] = load_terms<NP>(r, x <= w / 2 ? Blk::pair + lower(w, x) * NP * kFragBytes : kOffPast);
        grow = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + (kRowGrow + 16 * w + 4 * g) * 4));
        grow_j = __builtin_bit_cast(float, buf_load<uint32_t>(r, Blk::row + (kRowGrow + 16 * w + j) * 4));
        const f32x4 d = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + kRowDecay * 4));
        decay_f = d[0];
        decay_rest = d[1];
    };

    ChunkDecay decay;
    // The first chunk's loads in the order of the loop's, or a wait there would be
    // for as many as the worse of the two orders asks (all of them).
    load_k(p.c0);
    __builtin_amdgcn_sched_barrier(0);
    load_qv(p.c0);
    __builtin_amdgcn_sched_barrier(0);
    load_inv(p.c0);
    __builtin_amdgcn_sched_barrier(0);
    load_pair(p.c0);
    __builtin_amdgcn_sched_barrier(0);
    for (int c = p.c0; c < c_end; ++c) {
        const int rows = min(C, n - c * C);
        const DeltaSweep& sw = p.sweep;
        // ---- K S of the wave's channels, and the channels' terms of S
        if constexpr (BACK) {
            const Rsrc to = make_rsrc((E*)sw.S + (((size_t)unit * sw.NC + c) * p.dv + 16 * tile) * DK, 16 * DK * ES);
            buf_stream8<E>(to, holds ? (j * DK + 32 * w + 8 * g) * ES : kOffPast, M[0], M[1]);
        }
        if (holds) {
            const Terms<3> sf = split_terms<3>(M[0], M[1]);
#pragma unroll
            for (int i = 0; i < NS; ++i) reinterpret_cast<bf16x8*>(s.S[w] + i * kFragBytes)[lane] = sf.t[i];
#pragma unroll
            for (int a = 0; a < kDeltaTiles; ++a) {
                const Terms<NE> kt = raw_terms(rk[a]);
#pragma unroll
                for (int i = 0; i < NE; ++i) *reinterpret_cast<bf16x8*>(&s.k[w][i][(16 * a + j) * LK + 8 * g]) = kt.t[i];
                s.part[w][a][lane] = mma(kt, sf, zero4());
            }
        }
        put_piece<E>(&s.v[w][0][min(lane / ES, 15) * LV + lane % ES * (16 / ES)], 16 * LV, rv, lane < 16 * ES);
        if constexpr (BACK)
            put_piece<E>(&s.d[w][0][min(lane / ES, 15) * LV + lane % ES * (16 / ES)], 16 * LV, rd, lane < 16 * ES);
        load_k(c + 1);
        __syncthreads();
        // ---- R of the wave's tokens; Q S
        f32x4 R = s.part[0][w][lane];
#pragma unroll
        for (int m = 1; m < KM; ++m) R += s.part[m][w][lane];
        const f32x4 v = col4<NE>(&s.v[w][0][0], 16 * LV, LV, j, g);
        f32x4 ks = zero4(), dO = zero4(), dO_t = zero4();    // BACK: K S, dO of rows 4 g + i, and of token 16 w + j
        if constexpr (BACK) {
            ks = grow * R;
            dO = col4<NE>(&s.d[w][0][0], 16 * LV, LV, j, g);
#pragma unroll
            for (int x = NE - 1; x >= 0; --x) {
                const bf16x4 t = *reinterpret_cast<const bf16x4*>(&s.d[w][x][j * LV + 4 * g]);
#pragma unroll
                for (int i = 0; i < 4; ++i) dO_t[i] += (float)t[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) R[i] = v[i] - grow[i] * R[i];
        put_half<3>(s.r[w >> 1], w & 1, R);
        f32x4 o = zero4();                                   // rows: columns 4 g + i, column: token 16 w + j
#pragma unroll
        for (int m = 0; m < KM; ++m) o = mma(frag_terms<NS>(s.S[m]), raw_terms(rq[m]), o);
        load_qv(c + 1);
        __syncthreads();
        // ---- E of the wave's tokens
        f32x4 e;
        float dot = 0.f;
        if constexpr (BACK) {
            Sum2 x;
            x.add(rt[0], frag_terms<3>(s.r[0]));
            if (w >= 2) x.add(rt[1], frag_terms<3>(s.r[1]));
            ks -= x.sum();                                   // all that older tokens give
            e = x.sum() + R;
            dot = lane_row(self, j) * row_sums(dO * ks, j);  // of token 16 w + 4 g + j % 4
        } else {
            e = mma(rt[0], frag_terms<3>(s.r[0]), zero4());
            if (w >= 2) e = mma(rt[1], frag_terms<3>(s.r[1]), e);
        }
        put_half<NO>(s.e[w >> 1], w & 1, e);
        if constexpr (BACK) {
            const Rsrc to = make_rsrc(sw.e + (((size_t)unit * sw.NC + c) * p.dv + 16 * tile) * C, 16 * C * 4);
            buf_stream_u32x4(to, (j * C + 16 * w + 4 * g) * 4, __builtin_bit_cast(u32x4, e));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] *= write[i];
        const bool anchor = BACK && (c % kAnchorChunks == kAnchorChunks - 1 || c == c_end - 1);
        if (anchor) {                                        // its last token's v is written behind
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (16 * w + 4 * g + i != rows - 1) continue;
                e[i] = -write[i] * ks[i];
                s.write[j] = write[i] * v[i];
            }
        }
        put_half<3>(s.u[w >> 1], w & 1, e);
        load_inv(c + 1);
        __syncthreads();
        // ---- the state's update; o of the wave's tokens
        const float f = decay(decay_f, decay_rest);
        if (BACK && holds) {
            Sum2 sum[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const Terms<3> u = frag_terms<3>(s.u[x]);
#pragma unroll
                for (int t = 0; t < 2; ++t) sum[t].add(col_terms<NE>(&s.k[w][0][32 * x * LK], C * LK, LK, 4 * t, 8, j, g), u);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) M[t][i] = f * M[t][i] + sum[t].sum()[i];
        } else if (holds) {
#pragma unroll
            for (int t = 0; t < 2; ++t) M[t] *= f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const Terms<3> u = frag_terms<3>(s.u[x]);
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    M[t] = mma(col_terms<NE>(&s.k[w][0][32 * x * LK], C * LK, LK, 4 * t, 8, j, g), u, M[t]);
            }
        }
        o *= p.scale * grow_j;
        o = mma_top(frag_terms<NO>(s.e[0]), rp[0], o);
        if (w >= 2) o = mma_top(frag_terms<NO>(s.e[1]), rp[1], o);
        if constexpr (BACK) {
            float own = 0.f;                                 // dO . o of token 16 w + j
#pragma unroll
            for (int i = 0; i < 4; ++i) own += dO_t[i] * o[i];
            own += __shfl_xor(own, 16);
            own += __shfl_xor(own, 32);
            own -= __shfl(dot, 16 * (j >> 2) + (j & 3));
            const Rsrc to = make_rsrc(sw.dot + (((size_t)tile * units + unit) * sw.NC + c) * C, C * 4);
            buf_store_u32(to, g == 0 ? (16 * w + j) * 4 : kOffPast, __builtin_bit_cast(uint32_t, own));
            if (anchor && holds) {
                const Rsrc tm = make_rsrc((f32x4*)sw.end + ((((size_t)unit * sw.NA + c / kAnchorChunks) * tiles + tile) * KM + w) * 2 * kWave,
                                          2 * kWave * 16);
                f32x4 k[2] = {zero4(), zero4()};             // the last token's key
#pragma unroll
                for (int x = NE - 1; x >= 0; --x) {
                    const bf16x8 kx = *reinterpret_cast<const bf16x8*>(&s.k[w][x][(rows - 1) * LK + 8 * g]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) k[i / 4][i % 4] += (float)kx[i];
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    buf_stream_u32x4(tm, (t * kWave + lane) * 16, __builtin_bit_cast(u32x4, M[t]));
                    M[t] += s.write[j] * k[t];
                }
            }
        } else {
            const Rsrc to = rows_rsrc((char*)p.o + at_v + (int64_t)(c - p.c0) * C * ldv, rows, ldv, 16 * ES);
            const int off = 16 * w + j < rows ? (16 * w + j) * ldv + 4 * g * ES : kOffPast;
            if constexpr (ES == 2)
                buf_store_u32x2(to, off, __builtin_bit_cast(u32x2, pack4(o)));
            else
                buf_store_u32x4(to, off, __builtin_bit_cast(u32x4, o));
        }
        load_pair(c + 1);
    }
    if (holds && p.S.out) {
        float* out = p.S.out + ((size_t)(p.S.out_slot ? p.S.out_slot[b] : b) * p.H + h) * state + at_state;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) out[(size_t)(4 * t + i) * p.dv] = M[t][i];
    }
}

}  // namespace kda
