// kda_delta.hip -- the gated delta rule over a sequence in chunk form
// (kda_delta_chunk.hpp): the chain of states over the chunks.
#include <algorithm>

#include "kda_delta_chain.hpp"

namespace kda {

// One workgroup per (b, h, 16 value columns), one wave for each 32 key channels:
// the wave holds their part of the state [DK, 16] as two accumulator tiles, whose
// rows are mapped to channels so that a lane's rows of both are eight consecutive
// channels: the tiles are then an operand of K S and of Q S without a move.  The
// waves' parts of K S (and of Q S, for o) are summed through LDS, in order, the one
// barrier of a chunk; E and its scaled form are made by every wave, whose own
// channels of the state they then update.
// BACK: the gradients' forward sweep, which leaves e, the states and the parts of
// dO . o, whose sum over the sequence needs o with fp32's accuracy (three terms).
template <typename E, int DK, bool BACK>
__global__ __launch_bounds__(DK * 2, 2) void delta_chain_kernel(DeltaChain p) {
    constexpr int C = kDeltaChunk, KM = DK / 32, NT = DK * 2;
    constexpr int NE = sizeof(E) == 2 ? 1 : 3, NP = BACK ? 3 : NE, ES = sizeof(E);
    using Blk = DeltaBlock<NP, BACK>;
    constexpr int LK = 40, LV = 24;                          // padded rows of the K slice and of v in LDS
    constexpr int kStage = BACK ? Blk::row + 512 : Blk::bytes;     // the block's part that is read here
    constexpr int PB = kStage / 16, RB = (PB + NT - 1) / NT;   // pieces of a block, a thread's
    constexpr int PV = C * 16 * ES / 16, RV = (PV + NT - 1) / NT;  // pieces of v's tile
    __shared__ __align__(16) bf16 s_k[KM][NE][C * LK];
    __shared__ __align__(16) bf16 s_v[2][NE][C * LV];
    __shared__ __align__(16) char s_blk[2][kStage];
    __shared__ f32x4 s_part[KM > 1 ? 2 : 1][KM > 1 ? KM : 1][4][kWave];

    const int tiles = p.dv / 16, units = p.B * p.H;
    int unit, tile;
    unit_tile(blockIdx.x, units, tiles, unit, tile);
    const int b = unit / p.H, h = unit % p.H, hk = h / (p.H / p.Hk);
    if (p.S.skip(b)) return;
    const int n = seq_len(p.lens, b, p.T), c_end = min(p.c1, (n + C - 1) / C);
    const int tid = threadIdx.x, kw = wave_id(), lane = lane_id(), j = lane & 15, g = lane >> 4;

    // ---- the state's rows: tile t, channel 32 kw + 8 g + 4 t + i, column j
    const size_t state = (size_t)DK * p.dv;
    f32x4 M[2];
    {
        const float* in = p.S.in ? p.S.in + ((size_t)(p.S.in_slot ? p.S.in_slot[b] : b) * p.H + h) * state : nullptr;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) M[t][i] = in ? in[(size_t)(32 * kw + 8 * g + 4 * t + i) * p.dv + 16 * tile + j] : 0.f;
    }

    // ---- rows of chunk c: K and Q as operands (row 16 q + j, this wave's
    // channels), v's tile and the block for all waves
    const int ldk = p.Hk * DK * ES, ldv = p.H * p.dv * ES;
    struct Own {
        Raw<E> k[2], q[2];
    };
    struct Common {
        u32x4 v[RV], blk[RB];
    };
    // Chunks past the end load nothing: every offset is past the buffer.
    auto load_own = [&](int c, Own& x) {
        const int rows = c < c_end ? min(C, n - c * C) : 0;
        const size_t base = (((size_t)b * p.T + (size_t)c * C) * p.Hk + hk) * DK + 32 * kw;
        const uint32_t bytes = rows > 0 ? (uint32_t)((rows - 1) * ldk + 32 * ES) : 0;
        const Rsrc rk = make_rsrc((const E*)p.k + base, bytes), rq = make_rsrc((const E*)p.q + base, bytes);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int off = 16 * q + j < rows ? (16 * q + j) * ldk + 8 * g * ES : kOffPast;
            x.k[q] = raw_load<E>(rk, off);
            x.q[q] = raw_load<E>(rq, off);
        }
    };
    const char* blocks = p.blocks + (size_t)unit * (p.c1 - p.c0) * Blk::bytes;
    auto load_common = [&](int c, Common& x) {
        const int rows = c < c_end ? min(C, n - c * C) : 0;
        const size_t base = (((size_t)b * p.T + (size_t)c * C) * p.H + h) * p.dv + 16 * tile;
        const Rsrc rv = make_rsrc((const E*)p.v + base, rows > 0 ? (uint32_t)((rows - 1) * ldv + 16 * ES) : 0);
        const Rsrc rb = make_rsrc(blocks + (size_t)(c - p.c0) * Blk::bytes, rows > 0 ? kStage : 0);
        constexpr int PR = ES;                               // 16-byte pieces of a row of 16 elements
#pragma unroll
        for (int i = 0; i < RV; ++i) {
            const int at = tid + i * NT, row = at / PR;
            x.v[i] = buf_load<u32x4>(rv, at < PV && row < rows ? row * ldv + at % PR * 16 : kOffPast);
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) x.blk[i] = buf_load<u32x4>(rb, tid + i * NT < PB ? (tid + i * NT) * 16 : kOffPast);
    };
    auto stage_common = [&](int buf, const Common& x) {
        constexpr int PR = ES;
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
        Terms<NE> kt[2], qt[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            kt[q] = raw_terms(own[s].k[q]);
            qt[q] = raw_terms(own[s].q[q]);
#pragma unroll
            for (int i = 0; i < NE; ++i) *reinterpret_cast<bf16x8*>(&s_k[kw][i][(16 * q + j) * LK + 8 * g]) = kt[q].t[i];
        }
        load_own(c + 2, own[s]);
        const DeltaSweep& sw = p.sweep;
        if (BACK && c % kSuperChunks == 0) {
            E* dst = (E*)sw.S + (((size_t)unit * sw.NS + c / kSuperChunks) * p.dv + 16 * tile + j) * DK + 32 * kw + 8 * g;
            store8(dst, M[0], M[1]);
        }
        f32x4 dO[2];                                         // set out for early
        if constexpr (BACK) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int t = c * C + 16 * q + j;
                dO[q] = zero4();
                if ((KM == 1 || kw == q) && t < n)
                    load4((const E*)sw.dO + (((size_t)b * p.T + t) * p.H + h) * p.dv + 16 * tile + 4 * g, dO[q]);
            }
        }
        // K S (rows: tokens) and (Q S)^T (columns: tokens) of this wave's channels
        const Terms<3> sf = to_terms<3>(M[0], M[1]);
        f32x4 ks[2], qs[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            ks[q] = mma(kt[q], sf, zero4());
            qs[q] = mma(first_terms<NP>(sf), qt[q], zero4());
        }
        if constexpr (KM > 1) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                s_part[s][kw][q][lane] = ks[q];
                s_part[s][kw][2 + q][lane] = qs[q];
            }
        }
        __syncthreads();                                     // the parts are there, and this chunk's block and v
        if constexpr (KM > 1) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                ks[q] = s_part[s][0][q][lane];
#pragma unroll
                for (int w = 1; w < KM; ++w) ks[q] += s_part[s][w][q][lane];
            }
        }
        const char* blk = s_blk[s];
        const float* row = reinterpret_cast<const float*>(blk + Blk::row);
        // R = V - e^G K S, E = inv R
        const Terms<NE> vt = col_terms<NE>(&s_v[s][0][0], C * LV, LV, 0, 4, j, g);
        f32x4 R[2], e[2];
        to_f32(vt, R[0], R[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const f32x4 eg = *reinterpret_cast<const f32x4*>(row + 16 * q + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) R[q][i] -= eg[i] * ks[q][i];
        }
        const Terms<3> rt = to_terms<3>(R[0], R[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) e[q] = mma(frag_terms<3>(blk + Blk::inv + q * kFragBytes, 2 * kFragBytes), rt, zero4());
        stage_common(1 - s, common);
        load_common(c + 2, common);
        // S' = e^{G_C} S + K^T (e^{G_C - G} beta E)
        f32x4 u[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const f32x4 w = *reinterpret_cast<const f32x4*>(row + C + 16 * q + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) u[q][i] = w[i] * e[q][i];
        }
        const Terms<3> ut = to_terms<3>(u[0], u[1]);
        const float f = decay(row[2 * C], row[2 * C + 1]);
#pragma unroll
        for (int t = 0; t < 2; ++t)
            M[t] = mma(col_terms<NE>(&s_k[kw][0][0], C * LK, LK, 4 * t, 8, j, g), ut, f * M[t]);
        if constexpr (BACK) {
            if (kw == KM - 1) {                              // every wave has E
                f32x4* dst = reinterpret_cast<f32x4*>(sw.e + (((size_t)unit * sw.NC + c) * p.dv + 16 * tile + j) * C) + g;
                dst[0] = e[0];
                dst[4] = e[1];
            }
            if (c % kAnchorChunks == kAnchorChunks - 1 || c == c_end - 1) {
                f32x4* dst = reinterpret_cast<f32x4*>(sw.end) +
                             ((((size_t)unit * sw.NA + c / kAnchorChunks) * tiles + tile) * KM + kw) * 2 * kWave + lane;
                dst[0] = M[0];
                dst[kWave] = M[1];
            }
        }
        // o: the waves' first two (the only one's both) columns of tokens
        const Terms<NP> et = to_terms<NP>(e[0], e[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (KM > 1 && kw != q) continue;
            f32x4 o = qs[q];
            if constexpr (KM > 1) {
                o = s_part[s][0][2 + q][lane];
#pragma unroll
                for (int w = 1; w < KM; ++w) o += s_part[s][w][2 + q][lane];
            }
            o = mma(et, frag_terms<NP>(blk + Blk::pair + q * kFragBytes, 2 * kFragBytes), (p.scale * row[16 * q + j]) * o);
            const int t = c * C + 16 * q + j;
            if constexpr (BACK) {
                float d = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) d += dO[q][i] * o[i];
                d += __shfl_xor(d, 16);
                d += __shfl_xor(d, 32);
                if (g == 0) sw.dot[((size_t)tile * units + unit) * sw.NC * C + t] = d;
            } else if (t < n) {
                E* dst = (E*)p.o + (((size_t)b * p.T + t) * p.H + h) * p.dv + 16 * tile + 4 * g;
                if constexpr (ES == 2)
                    *reinterpret_cast<bf16x4*>(dst) = pack4(o);
                else
                    *reinterpret_cast<f32x4*>(dst) = o;
            }
        }
    };

    if (p.c0 < c_end) {
        constexpr std::integral_constant<int, 0> set0{};
        constexpr std::integral_constant<int, 1> set1{};
        load_common(p.c0, common);
        load_own(p.c0, own[0]);
        load_own(p.c0 + 1, own[1]);
        stage_common(0, common);
        load_common(p.c0 + 1, common);
        for (int c = p.c0;; c += 2) {
            chunk(set0, c);
            if (c + 1 >= c_end) break;
            chunk(set1, c + 1);
            if (c + 2 >= c_end) break;
        }
    }
    if (p.S.out) {
        float* out = p.S.out + ((size_t)(p.S.out_slot ? p.S.out_slot[b] : b) * p.H + h) * state;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) out[(size_t)(32 * kw + 8 * g + 4 * t + i) * p.dv + 16 * tile + j] = M[t][i];
    }
}

// Chunks whose blocks the workspace holds at a time: longer sequences run window
// by window, the state carried in the workspace.
constexpr size_t kDeltaWindowBytes = (size_t)192 << 20;

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
        case 32: hipLaunchKernelGGL((delta_chain_kernel<E, 32, BACK>), grid, dim3(64), 0, stream, a); break;
        case 64: hipLaunchKernelGGL((delta_chain_kernel<E, 64, BACK>), grid, dim3(128), 0, stream, a); break;
        default: hipLaunchKernelGGL((delta_chain_kernel<E, 128, BACK>), grid, dim3(256), 0, stream, a); break;
    }
    return hipGetLastError();
}

hipError_t launch_delta_sweep(const DeltaChain& a, hipStream_t stream) {
    return a.is_bf16 ? launch_chain<bf16, true>(a, stream) : launch_chain<float, true>(a, stream);
}

hipError_t launch_delta_prefill(const DeltaPrefill& a, void* ws, hipStream_t stream) {
    const DeltaWindows w = windows(a.B, a.T, a.H, a.dk, a.dv, a.is_bf16);
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
        e = a.is_bf16 ? launch_chain<bf16, false>(c, stream) : launch_chain<float, false>(c, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace kda
