// kda_delta.hip -- the gated delta rule over a sequence in chunk form
// (kda_delta_chunk.hpp): the chain of states over the chunks.
#include <algorithm>

#include "kda_delta_chain.hpp"

namespace kda {

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
// BACK: the gradients' forward sweep, which leaves e, the states and the parts of
// dO . o, whose sum over the sequence needs o with fp32's accuracy (three terms).
template <typename E, int DK, bool BACK>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 2 : 1) void delta_chain_kernel(DeltaChain p) {
    constexpr int C = kDeltaChunk, KM = DK / 32, ES = sizeof(E), NE = ES == 2 ? 1 : 3;
    // Terms of the state in Q S, of E and of the pairs' weights in o.  With bf16 two,
    // two and one leave the weights' rounding alone beside o's own.
    constexpr int NS = BACK || ES == 4 ? 3 : 2, NO = NS, NP = BACK || ES == 4 ? 3 : 1;
    using Blk = DeltaBlock<NP, BACK>;
    constexpr int LK = NE == 1 ? 40 : 32, LV = 24;           // padded rows in LDS
    __shared__ __align__(16) bf16 s_k[KM][NE][C * LK];       // a wave's own channels of K
    __shared__ __align__(16) bf16 s_v[4][NE][16 * LV];       // a wave's own tokens of V
    __shared__ __align__(16) char s_S[KM][NS * kFragBytes];
    __shared__ f32x4 s_part[KM][kDeltaTiles][kWave];
    __shared__ __align__(16) char s_r[2][3 * kFragBytes], s_u[2][3 * kFragBytes], s_e[2][NO * kFragBytes];

    const int tiles = p.dv / 16, units = p.B * p.H;
    int unit, tile;
    unit_tile(blockIdx.x, units, tiles, unit, tile);
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
    f32x4 dO = zero4();
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
        rv = buf_load<u32x4>(v, lane < 16 * ES && row < rows ? row * ldv + lane % ES * 16 : kOffPast);
        if constexpr (BACK) {
            const Rsrc d = rows_rsrc((const char*)p.sweep.dO + at_v + (int64_t)(c - p.c0) * C * ldv, rows, ldv, 16 * ES);
            dO = buf_load4<E>(d, 16 * w + j < rows ? (16 * w + j) * ldv + 4 * g * ES : kOffPast);
        }
    };
    auto blk_rsrc = [&](int c) { return make_rsrc(pb + (int64_t)(c - p.c0) * Blk::bytes, c < c_end ? Blk::bytes : 0); };
    auto load_inv = [&](int c) {
        const Rsrc r = blk_rsrc(c);
#pragma unroll
        for (int x = 0; x < 2; ++x) rt[x] = load_terms<3>(r, x <= w / 2 ? Blk::inv + lower(w, x) * 3 * kFragBytes : kOffPast);
        write = __builtin_bit_cast(f32x4, buf_load<u32x4>(r, Blk::row + (kRowWrite + 16 * w + 4 * g) * 4));
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
            buf_store8<E>(to, holds ? (j * DK + 32 * w + 8 * g) * ES : kOffPast, M[0], M[1]);
        }
        if (holds) {
            const Terms<3> sf = split_terms<3>(M[0], M[1]);
#pragma unroll
            for (int s = 0; s < NS; ++s) reinterpret_cast<bf16x8*>(s_S[w] + s * kFragBytes)[lane] = sf.t[s];
#pragma unroll
            for (int a = 0; a < kDeltaTiles; ++a) {
                const Terms<NE> kt = raw_terms(rk[a]);
#pragma unroll
                for (int i = 0; i < NE; ++i) *reinterpret_cast<bf16x8*>(&s_k[w][i][(16 * a + j) * LK + 8 * g]) = kt.t[i];
                s_part[w][a][lane] = mma(kt, sf, zero4());
            }
        }
        put_piece<E>(&s_v[w][0][min(lane / ES, 15) * LV + lane % ES * (16 / ES)], 16 * LV, rv, lane < 16 * ES);
        load_k(c + 1);
        __syncthreads();
        // ---- R of the wave's tokens; Q S
        f32x4 R = s_part[0][w][lane];
#pragma unroll
        for (int m = 1; m < KM; ++m) R += s_part[m][w][lane];
        const f32x4 v = col4<NE>(&s_v[w][0][0], 16 * LV, LV, j, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) R[i] = v[i] - grow[i] * R[i];
        put_half<3>(s_r[w >> 1], w & 1, R);
        f32x4 o = zero4();                                   // rows: columns 4 g + i, column: token 16 w + j
#pragma unroll
        for (int m = 0; m < KM; ++m) o = mma(frag_terms<NS>(s_S[m]), raw_terms(rq[m]), o);
        const f32x4 d = dO;
        load_qv(c + 1);
        __syncthreads();
        // ---- E of the wave's tokens
        f32x4 e = mma(rt[0], frag_terms<3>(s_r[0]), zero4());
        if (w >= 2) e = mma(rt[1], frag_terms<3>(s_r[1]), e);
        put_half<NO>(s_e[w >> 1], w & 1, e);
        if constexpr (BACK) {
            const Rsrc to = make_rsrc(sw.e + (((size_t)unit * sw.NC + c) * p.dv + 16 * tile) * C, 16 * C * 4);
            buf_store_u32x4(to, (j * C + 16 * w + 4 * g) * 4, __builtin_bit_cast(u32x4, e));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] *= write[i];
        put_half<3>(s_u[w >> 1], w & 1, e);
        load_inv(c + 1);
        __syncthreads();
        // ---- the state's update; o of the wave's tokens
        const float f = decay(decay_f, decay_rest);
        if (holds) {
#pragma unroll
            for (int t = 0; t < 2; ++t) M[t] *= f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const Terms<3> u = frag_terms<3>(s_u[x]);
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    M[t] = mma(col_terms<NE>(&s_k[w][0][32 * x * LK], C * LK, LK, 4 * t, 8, j, g), u, M[t]);
            }
        }
        o *= p.scale * grow_j;
        o = mma(frag_terms<NO>(s_e[0]), rp[0], o);
        if (w >= 2) o = mma(frag_terms<NO>(s_e[1]), rp[1], o);
        if constexpr (BACK) {
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) dot += d[i] * o[i];
            dot += __shfl_xor(dot, 16);
            dot += __shfl_xor(dot, 32);
            const Rsrc to = make_rsrc(sw.dot + (((size_t)tile * units + unit) * sw.NC + c) * C, C * 4);
            buf_store_u32(to, g == 0 ? (16 * w + j) * 4 : kOffPast, __builtin_bit_cast(uint32_t, dot));
            const bool anchor = holds && (c % kAnchorChunks == kAnchorChunks - 1 || c == c_end - 1);
            const Rsrc tm = make_rsrc((f32x4*)sw.end + ((((size_t)unit * sw.NA + c / kAnchorChunks) * tiles + tile) * KM + w) * 2 * kWave,
                                      2 * kWave * 16);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                buf_store_u32x4(tm, anchor ? (t * kWave + lane) * 16 : kOffPast, __builtin_bit_cast(u32x4, M[t]));
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

// Chunks whose blocks the workspace holds at a time: longer sequences run window
// by window, the state carried in the workspace.
constexpr size_t kDeltaWindowBytes = (size_t)192 << 20;

// From so many heads of bf16 rows on a workgroup takes a whole one
// (delta_wide_kernel), where fewer leave more than half of the device idle.  d 128,
// T 4096, wide against eight workgroups of 16 columns: 64 heads 402 and 308 us, 128
// heads 484 and 615 us, 256 heads 676 and 1,236 us.
constexpr int kWideUnits = 128;

struct DeltaWindows {
    int chunks, len, n;      // chunks of a sequence, of a window, windows
    size_t blocks, carry;    // bytes
};
static DeltaWindows windows(int B, int T, int H, int dk, int dv, bool is_bf16) {
    const size_t units = (size_t)B * H, blk = delta_block_bytes(is_bf16, false);
    DeltaWindows w;
    w.chunks = (T + kDeltaChunk - 1) / kDeltaChunk;
    w.len = (int)std::min<size_t>(w.chunks, std::max<size_t>(8, kDeltaWindowBytes / (units * blk)));
    w.n = (w.chunks + w.len - 1) / w.len;
    w.len = (w.chunks + w.n - 1) / w.n;
    w.blocks = (units * w.len * blk + 255) / 256 * 256;
    w.carry = w.n > 1 ? units * dk * dv * sizeof(float) : 0;
    return w;
}

size_t delta_prefill_ws_bytes(int B, int T, int H, int dk, int dv, bool is_bf16) {
    const DeltaWindows w = windows(B, T, H, dk, dv, is_bf16);
    return w.blocks + w.carry;
}

template <typename E, bool BACK>
static hipError_t launch_chain(const DeltaChain& a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * a.H * (a.dv / 16)));
    switch (a.dk) {
        case 32: hipLaunchKernelGGL((delta_chain_kernel<E, 32, BACK>), grid, dim3(256), 0, stream, a); break;
        case 64: hipLaunchKernelGGL((delta_chain_kernel<E, 64, BACK>), grid, dim3(256), 0, stream, a); break;
        default: hipLaunchKernelGGL((delta_chain_kernel<E, 128, BACK>), grid, dim3(256), 0, stream, a); break;
    }
    return hipGetLastError();
}

hipError_t launch_delta_sweep(const DeltaChain& a, hipStream_t stream) {
    return a.is_bf16 ? launch_chain<bf16, true>(a, stream) : launch_chain<float, true>(a, stream);
}

hipError_t launch_delta_prefill(const DeltaPrefill& a, void* ws, hipStream_t stream) {
    const DeltaWindows w = windows(a.B, a.T, a.H, a.dk, a.dv, a.is_bf16);
    const bool wide = a.is_bf16 && a.dv == 128 && a.B * a.H >= kWideUnits;
    char* blocks = (char*)ws;
    float* carry = w.n > 1 ? (float*)(blocks + w.blocks) : nullptr;
    for (int i = 0; i < w.n; ++i) {
        const int c0 = i * w.len, c1 = std::min(w.chunks, c0 + w.len);
        StateIO S = a.S;
        if (i > 0) S.in = carry, S.in_slot = nullptr;
        if (i + 1 < w.n) S.out = carry, S.out_slot = nullptr;
        hipError_t e = launch_delta_pairs({a.q, a.k, a.g, a.beta, a.scale, S, a.lens, blocks, a.B, a.T, a.H, a.Hk, a.dk, c0, c1,
                                           a.is_bf16}, false, stream);
        if (e != hipSuccess) return e;
        const DeltaChain c{a.q, a.k, a.v, a.scale, S, a.lens, blocks, a.o, a.B, a.T, a.H, a.Hk, a.dk, a.dv, c0, c1, a.is_bf16, {}};
        e = wide ? launch_delta_wide(c, stream) : a.is_bf16 ? launch_chain<bf16, false>(c, stream) : launch_chain<float, false>(c, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace kda
