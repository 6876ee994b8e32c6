// kda_delta_wide.hip -- the chain of states of the gated delta rule
// (kda_delta_chunk.hpp) for batches whose heads fill the device: one workgroup per
// (b, h), one wave for each 16 value columns.
//
// A wave holds its columns' whole state [DK, 16] in accumulators and needs no other
// wave: K, Q and the chunk's block are staged in LDS for all of them, in two buffers,
// one barrier a chunk, and V by each wave for itself.  Against delta_chain_kernel,
// which divides a chunk among four waves, nothing but the staged rows passes through
// LDS, so that the CU's waves fill its issue slots: 2.2 KB of LDS a token and 16
// columns against 2.7, and no exchange.
#include <algorithm>

#include "kda_delta_chain.hpp"

namespace kda {

template <int DK, int DV>
__global__ __launch_bounds__(DV * 4, 2) void delta_wide_kernel(DeltaChain p) {
    typedef bf16 E;
    constexpr int C = kDeltaChunk, KM = DK / 32, NT = DV * 4, NS = 2, NO = 2, ES = 2;
    using Blk = DeltaBlock<2, false>;
    // Padded rows of K: 12 (mod 16) banks apart, so that both 16 rows of 16 bytes and
    // the transposing reads of 8-byte groups spread over the banks.
    constexpr int LK = DK + 24, LQ = DK + 8, LV = 24;
    constexpr int PK = C * DK / 8, PB = Blk::bytes / 16;    // 16-byte pieces
    constexpr int RK = (PK + NT - 1) / NT, RV = 2, RB = (PB + NT - 1) / NT;   // of a thread
    static_assert(PK % NT == 0 || PK < NT, "pieces");
    __shared__ __align__(16) bf16 s_k[2][C * LK], s_q[2][C * LQ], s_v[DV / 16][C * LV];
    __shared__ __align__(16) char s_blk[2][Blk::bytes];

    const int unit = blockIdx.x, b = unit / p.H, h = unit % p.H, hk = h / (p.H / p.Hk);
    if (p.S.skip(b)) return;
    const int n = seq_len(p.lens, b, p.T), c_end = min(p.c1, (n + C - 1) / C);
    const int tid = threadIdx.x, w = wave_id(), lane = lane_id(), j = lane & 15, g = lane >> 4;

    // ---- the state: tile t, channel 32 (t / 2) + 8 g + 4 (t % 2) + i, column 16 w + j
    f32x4 M[2 * KM];
    {
        const float* in = p.S.in ? p.S.in + ((size_t)(p.S.in_slot ? p.S.in_slot[b] : b) * p.H + h) * (DK * DV) : nullptr;
#pragma unroll
        for (int t = 0; t < 2 * KM; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) M[t][i] = in ? in[(32 * (t >> 1) + 8 * g + 4 * (t & 1) + i) * DV + 16 * w + j] : 0.f;
    }

    const int ldk = p.Hk * DK * ES, ldv = p.H * DV * ES;
    const size_t at_k = (((size_t)b * p.T + (size_t)p.c0 * C) * p.Hk + hk) * DK * ES;
    const size_t at_v = (((size_t)b * p.T + (size_t)p.c0 * C) * p.H + h) * DV * ES;
    const char* pb = p.blocks + (size_t)unit * (p.c1 - p.c0) * Blk::bytes;
    auto rows_rsrc = [&](const void* base, size_t at, int c, int rows, int ld, int width) {
        return make_rsrc((const char*)base + at + (int64_t)(c - p.c0) * C * ld, rows > 0 ? (uint32_t)((rows - 1) * ld + width) : 0);
    };
    u32x4 xk[RK], xq[RK], xv[RV], xb[RB];
    auto load = [&](int c) {                                 // rows and chunks past the end: zeros
        const int rows = c < c_end ? min(C, n - c * C) : 0;
        const Rsrc k = rows_rsrc(p.k, at_k, c, rows, ldk, DK * ES), q = rows_rsrc(p.q, at_k, c, rows, ldk, DK * ES),
                   v = rows_rsrc(p.v, at_v, c, rows, ldv, DV * ES);
        const Rsrc r = make_rsrc(pb + (int64_t)(c - p.c0) * Blk::bytes, rows > 0 ? Blk::bytes : 0);
#pragma unroll
        for (int i = 0; i < RK; ++i) {
            const int row = (tid + i * NT) / (DK / 8), off = row < rows ? row * ldk + (tid + i * NT) % (DK / 8) * 16 : kOffPast;
            xk[i] = buf_load<u32x4>(k, off);
            xq[i] = buf_load<u32x4>(q, off);
        }
#pragma unroll
        for (int i = 0; i < RV; ++i) {
            const int row = 32 * i + lane / 2;               // the wave's own columns
            xv[i] = buf_load<u32x4>(v, row < rows ? row * ldv + (32 * w + lane % 2 * 16) : kOffPast);
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) xb[i] = buf_load<u32x4>(r, (tid + i * NT) * 16);
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < RK; ++i) {
            const int row = (tid + i * NT) / (DK / 8), col = (tid + i * NT) % (DK / 8) * 8;
            if (PK < NT && row >= C) continue;
            *reinterpret_cast<u32x4*>(&s_k[buf][row * LK + col]) = xk[i];
            *reinterpret_cast<u32x4*>(&s_q[buf][row * LQ + col]) = xq[i];
        }
#pragma unroll
        for (int i = 0; i < RB; ++i)
            if (PB % NT == 0 || tid + i * NT < PB) reinterpret_cast<u32x4*>(s_blk[buf])[tid + i * NT] = xb[i];
    };

    auto stage_v = [&] {
#pragma unroll
        for (int i = 0; i < RV; ++i) *reinterpret_cast<u32x4*>(&s_v[w][(32 * i + lane / 2) * LV + lane % 2 * 8]) = xv[i];
    };

    ChunkDecay decay;
    load(p.c0);
    stage_v();
    stage(0);
    load(p.c0 + 1);
    int buf = 0;
    for (int c = p.c0; c < c_end; ++c, buf ^= 1) {
        const int rows = min(C, n - c * C);
        __syncthreads();                                     // this chunk is staged, the last one read
        f32x4 v[kDeltaTiles];                                // the wave's own columns, whose place the next chunk's take
#pragma unroll
        for (int a = 0; a < kDeltaTiles; ++a) v[a] = col4<1>(&s_v[w][16 * a * LV], 0, LV, j, g);
        wave_fence();
        stage_v();
        stage(buf ^ 1);
        load(c + 2);
        __builtin_amdgcn_sched_barrier(0);                   // not later: they have this chunk's time to come
        const bf16 *sk = s_k[buf], *sq = s_q[buf];
        const char* blk = s_blk[buf];
        const float* row = reinterpret_cast<const float*>(blk + Blk::row);
        // K S (rows: tokens) and (Q S)^T (columns: tokens)
        f32x4 ks[kDeltaTiles], o[kDeltaTiles];
#pragma unroll
        for (int a = 0; a < kDeltaTiles; ++a) ks[a] = o[a] = zero4();
#pragma unroll
        for (int m = 0; m < KM; ++m) {
            const Terms<3> sf = split_terms<3>(M[2 * m], M[2 * m + 1]);
#pragma unroll
            for (int a = 0; a < kDeltaTiles; ++a) {
                const Terms<1> kt = row_terms<1>(sk + (16 * a + j) * LK + 32 * m + 8 * g, 0),
                               qt = row_terms<1>(sq + (16 * a + j) * LQ + 32 * m + 8 * g, 0);
                ks[a] = mma(kt, sf, ks[a]);
                o[a] = mma(first_terms<NS>(sf), qt, o[a]);
            }
        }
        // R = V - e^G K S, E = inv R
        Terms<3> rt[2];
#pragma unroll
        for (int a = 0; a < kDeltaTiles; ++a) {
            const f32x4 eg = *reinterpret_cast<const f32x4*>(row + kRowGrow + 16 * a + 4 * g);
            const float eo = p.scale * row[kRowGrow + 16 * a + j];
#pragma unroll
            for (int i = 0; i < 4; ++i) ks[a][i] = v[a][i] - eg[i] * ks[a][i];
            o[a] *= eo;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) rt[x] = split_terms<3>(ks[2 * x], ks[2 * x + 1]);
        f32x4 e[kDeltaTiles];
#pragma unroll
        for (int a = 0; a < kDeltaTiles; ++a) {
            e[a] = zero4();
#pragma unroll
            for (int x = 0; x <= a / 2; ++x) e[a] = mma(frag_terms<3>(blk + Blk::inv + lower(a, x) * 3 * kFragBytes), rt[x], e[a]);
        }
        // o, stored a row of four columns a lane
        Terms<NO> et[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) et[x] = split_terms<NO>(e[2 * x], e[2 * x + 1]);
        const Rsrc to = rows_rsrc(p.o, at_v, c, rows, ldv, DV * ES);
#pragma unroll
        for (int a = 0; a < kDeltaTiles; ++a) {
#pragma unroll
            for (int x = 0; x <= a / 2; ++x) o[a] = mma_top(et[x], frag_terms<2>(blk + Blk::pair + lower(a, x) * 2 * kFragBytes), o[a]);
            const int off = 16 * a + j < rows ? (16 * a + j) * ldv + (16 * w + 4 * g) * ES : kOffPast;
            buf_store_u32x2(to, off, __builtin_bit_cast(u32x2, pack4(o[a])));
        }
        // S' = e^{G_C} S + K^T (e^{G_C - G} beta E)
        Terms<3> ut[2];
#pragma unroll
        for (int a = 0; a < kDeltaTiles; ++a) {
            const f32x4 wr = *reinterpret_cast<const f32x4*>(row + kRowWrite + 16 * a + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) e[a][i] *= wr[i];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) ut[x] = split_terms<3>(e[2 * x], e[2 * x + 1]);
        const float f = decay(row[kRowDecay], row[kRowDecay + 1]);
#pragma unroll
        for (int t = 0; t < 2 * KM; ++t) {
            M[t] *= f;
#pragma unroll
            for (int x = 0; x < 2; ++x)
                M[t] = mma(col_terms<1>(sk + 32 * x * LK, 0, LK, 32 * (t >> 1) + 4 * (t & 1), 8, j, g), ut[x], M[t]);
        }
    }
    if (p.S.out) {
        float* out = p.S.out + ((size_t)(p.S.out_slot ? p.S.out_slot[b] : b) * p.H + h) * (DK * DV);
#pragma unroll
        for (int t = 0; t < 2 * KM; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) out[(32 * (t >> 1) + 8 * g + 4 * (t & 1) + i) * DV + 16 * w + j] = M[t][i];
    }
}

hipError_t launch_delta_wide(const DeltaChain& a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * a.H)), block(512);
    switch (a.dk) {
        case 32: hipLaunchKernelGGL((delta_wide_kernel<32, 128>), grid, block, 0, stream, a); break;
        case 64: hipLaunchKernelGGL((delta_wide_kernel<64, 128>), grid, block, 0, stream, a); break;
        default: hipLaunchKernelGGL((delta_wide_kernel<128, 128>), grid, block, 0, stream, a); break;
    }
    return hipGetLastError();
}

}  // namespace kda
