// kda_linear.hip -- linear attention with a decay for each head: the prefill
// and its gradients, all made of one pass (LinearPass in kda_linear.hpp).
//
// Forward: x = q, y = k, u = v.  The gradients are the same recurrence with
// other tensors in its places, since with R_t = scale q_t dO_t^T + Y_{t+1},
// Y_t = a R_t (Y_n = dS_T):
//   dq_t = scale S_t dO_t  : forward, x = dO, y = v, u = k, on S^T
//   dv_t = R_t^T k_t       : reverse, x = k, y = q, u = dO, on R
//   dk_t = R_t v_t         : reverse, x = v, y = dO, u = q, on R^T
//
// Chunk form, with C = 32 steps r = 0 .. c - 1 of a chunk (c < C in the last
// one), M the state at its start and f = 1 in a reverse pass, else 0:
//   out_r = so [ a^{r + 1 - f} M^T x_r + su sum_{j <= r} a^{r - j} (x_r . y_j) u_j ]
//   M    <- a^c M + su sum_j a^{c - 1 - j + f} y_j u_j^T
// (a reverse pass takes its steps from the last token to the first and its
// state is Y, decayed already.)  Every weight is a power of a with an exponent
// >= 0, formed as exp of the product, so nothing overflows for g <= 0 and no
// error builds up along a chunk.
#include <algorithm>
#include <cmath>

#include "kda_device.hpp"
#include "kda_linear.hpp"
#include "kda_linear_frag.hpp"

namespace kda {

constexpr int kLinChunk = 32;

// ------------------------------------------------------------------ the pass

// Segments of a sequence run side by side: a first launch leaves in the
// workspace what each segment but the last adds to a zero state, the second
// starts every segment from the initial state and the ones before it.
struct LinearSegs {
    int R, len;  // segments of a sequence, their length in steps (a multiple of 32)
};

// Up to three passes of the same sizes in one launch (the gradients), each
// with its workspace [unit][R][DA * DB]: R - 1 segments' states, then the
// initial one, each as [DA / 4][DB] quads of rows (16 bytes a lane).  The first
// launch runs the passes before `state`; a pass with ws_t reads the states of
// another one, of [DB, DA], transposed.
struct LinearJob {
    LinearPass pass[3];
    float* ws[3];
    bool ws_t[3];
    int passes, state, shared;   // shared: heads that share one of q and k
    LinearSegs segs;
};

// One workgroup per (b, h, segment), one wave for each NC tiles of 16
// columns of the state [DA, DB] in registers (MFMA accumulator layout).  A
// state tile pair in that layout is an operand of M^T x without a move: rows
// are mapped to channels so that a lane's rows of two tiles are eight
// consecutive channels.  x, y and u of a chunk are staged in LDS (two buffers,
// one barrier a chunk, the chunk after the next in flight in registers).  The
// pair weights are computed transposed (keys x queries) by every wave, which
// makes the product with u take them straight from the accumulators.
// Matrix operands are sums of bf16 terms: x, y and u are one if bf16, three if
// fp32; NP is the number for the state and the pair weights in their products
// with x and u (see launch_job_d).  STATE: only the state of a segment
// from zero, into the workspace.
// What bounds it: where every CU has a workgroup, its instructions and its rows
// alike (B8 H32 T8192 d128 bf16 in 479 us: one wave a SIMD issues in 57 % of its
// cycles, VALU 42 %, and waits in 20 %, the matrix cores are busy in 33 %; 2.19 GB
// at 4.6 TB/s, a large copy's rate, where the decode step reaches 5.85); where
// sequences are few or short, a chunk's own chain (stage, products, barrier: 1.4
// us, of which MFMA and VALU issue fill two thirds).
template <typename E, int DA, int DB, int NC, int NP, bool STATE>
__global__ __launch_bounds__(DB / NC * 4, 2) void linear_chunk_kernel(LinearJob job) {
    constexpr int C = kLinChunk, NT = DB / NC * 4, KM = DA / 32;
    constexpr int NE = sizeof(E) == 2 ? 1 : 3;               // bf16 terms of x, y and u
    constexpr int PE = 16 / sizeof(E);                       // elements of 16 bytes
    // Padded LDS rows.  bf16: rows 12 (mod 16) banks apart for x and y, so that
    // both 16 rows of 16 bytes and the transposing reads of 8-byte groups 16
    // bytes apart spread over the banks; 8 (mod 16) apart for u.  fp32, as three
    // bf16 planes: what fits the LDS.
    constexpr int LA = DA + (NE == 1 ? 24 : 8), LB = DB + (NE == 1 ? 16 : 8);
    constexpr int QA = C * LA, QB = C * LB;                  // elements of a plane
    constexpr int PA = C * DA / PE, PB = C * DB / PE;        // 16-byte pieces of a tile
    constexpr int RA = (PA + NT - 1) / NT, RB = (PB + NT - 1) / NT;
    static_assert(DB % (16 * NC) == 0, "waves cover the columns");
    __shared__ __align__(16) bf16 s_x[STATE ? 1 : 2][STATE ? 8 : NE * QA];
    __shared__ __align__(16) bf16 s_y[2][NE * QA], s_u[2][NE * QB];

    const LinearSegs segs = job.segs;
    const int units = job.pass[0].B * job.pass[0].H, nseg = STATE ? segs.R - 1 : segs.R;
    // The heads that share q and k, and the passes, of one segment follow each
    // other on one XCD (workgroups go round the eight), whose L2 then serves what
    // they read in common.
    const int near = job.shared * (STATE ? job.state : job.passes), groups = units / job.shared * nseg;
    const int whole = groups / 8 * 8, x = blockIdx.x, rest = x - whole * near;
    const int group = rest < 0 ? x / 8 / near * 8 + x % 8 : whole + rest / near;
    const int at = rest < 0 ? x / 8 % near : rest % near, role = at / job.shared;
    const int seg = group / (units / job.shared), unit = group % (units / job.shared) * job.shared + at % job.shared;
    const LinearPass& p = job.pass[role];
    const int b = unit / p.H, h = unit % p.H;
    if (p.S.skip(b)) return;
    const int n = p.lens ? min(max(p.lens[b], 0), p.T) : p.T;
    const int s0 = seg * segs.len;
    if (s0 >= n && !(seg == 0)) return;
    const int s1 = min(n, s0 + segs.len);
    const bool last = s1 == n;
    if (STATE && last) return;                               // nothing follows it
    const int tid = threadIdx.x, wave = wave_id(), lane = lane_id(), j = lane & 15, g = lane >> 4;
    const int hx = h / (p.H / p.x.n), hy = h / (p.H / p.y.n), hu = h / (p.H / p.u.n), ho = h / (p.H / p.n_out);
    const float lg = log_decay(p.g[h]);
    const int rev = p.reverse ? 1 : 0;

    // columns of this lane: tile ct of the wave, lane column j
    const int cbase = wave * NC * 16, cstep = 4 * NC;
    auto col = [&](int ct) { return cbase + cstep * (j >> 2) + 4 * ct + (j & 3); };

    // ---- the state at the segment's start.  The final state may go where the
    // initial one came from, so with several segments only the first launch
    // reads that, and copies it.
    auto slot = [&](int m) { return job.ws[role] + ((size_t)unit * segs.R + m) * (DA * DB); };
    // quad of rows of tile t in a slot, and the same rows of its transposed form
    auto quad = [&](float* w, int t, int ct) -> f32x4& {
        return reinterpret_cast<f32x4*>(w)[(8 * (t >> 1) + 2 * g + (t & 1)) * DB + col(ct)];
    };
    auto quad_t = [&](const float* w, int t, int ct) {
        const int c = col(ct), row = 32 * (t >> 1) + 8 * g + 4 * (t & 1);
        const float* q = w + ((size_t)(c >> 2) * DA + row) * 4 + (c & 3);
        return f32x4{q[0], q[4], q[8], q[12]};
    };
    const bool direct = STATE || (seg == 0 && last);
    const float* in = p.S.in && (STATE ? seg == 0 : direct)
                          ? p.S.in + ((size_t)(p.S.in_slot ? p.S.in_slot[b] : b) * p.H + h) * (DA * DB) : nullptr;
    f32x4 M[2 * KM][NC];
#pragma unroll
    for (int t = 0; t < 2 * KM; ++t)
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ch = 32 * (t >> 1) + 8 * g + 4 * (t & 1) + i;
                M[t][ct][i] = in ? in[p.in_t ? col(ct) * DA + ch : ch * DB + col(ct)] : 0.f;
            }
            if (STATE) {
                if (in) quad(slot(segs.R - 1), t, ct) = M[t][ct];
                M[t][ct] = zero4();
            }
        }
    if (!direct) {
        const float as = expf(lg * (float)segs.len);
        auto start = [&](auto transposed) {
            auto add = [&](int m, float keep) {
                float* w = slot(m);
#pragma unroll
                for (int t = 0; t < 2 * KM; ++t)
#pragma unroll
                    for (int ct = 0; ct < NC; ++ct)
                        M[t][ct] = keep * M[t][ct] + (decltype(transposed)::value ? quad_t(w, t, ct) : quad(w, t, ct));
            };
            if (p.S.in) add(segs.R - 1, 0.f);
            for (int m = 0; m < seg; ++m) add(m, as);
        };
        if (job.ws_t[role])
            start(std::true_type{});
        else
            start(std::false_type{});
    }

    // ---- weights of a chunk of c steps
    float wd[4], wo[4], wi[2], wu[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int d = j - 4 * g - i;                         // query - key within a 16 x 16 block
        wd[i] = d >= 0 ? p.so * p.su * expf(lg * (float)d) : 0.f;
        wo[i] = p.so * p.su * expf(lg * (float)(16 + d));
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) wi[q] = p.so * expf(lg * (float)(16 * q + j + 1 - rev));
    // a^c as an fp32 factor: the part of a^c that each rounding leaves out goes
    // into the next chunk's factor, so the factors' product stays a^{steps}
    // however many chunks there are.
    double ac = 0, ac_inv = 0, ac_left = 0;
    auto chunk_weights = [&](int c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int left = c - 1 - ((i & 4) * 4 + 4 * g + (i & 3));
            wu[i] = left >= 0 ? p.su * expf(lg * (float)(left + rev)) : 0.f;
        }
        ac = exp((double)lg * c);
        ac_inv = ac > 1e-30 ? 1.0 / ac : 0.0;
    };
    auto chunk_decay = [&]() {
        const double want = ac + ac * ac_left;
        const float f = (float)want;
        ac_left = (want - (double)f) * ac_inv;
        return f;
    };

    // ---- rows of a chunk in step order.  Thread offsets within a chunk are
    // constant; the chunk's base (for a reverse pass 32 tokens below its first
    // step, which may lie before the tensor) moves on.  Rows past the chunk's
    // end get an offset past the buffer's: zero.
    struct Rows {
        const char* base;
        int64_t step;
        uint32_t bytes;
        int ld;
    };
    const int os = p.out_f32 ? 4 : (int)sizeof(E);           // bytes of an element of out
    auto rows_of = [&](const void* ptr, int heads, int head, int d, int es) {
        const int ld = heads * d * es;
        const int64_t t0 = (int64_t)b * p.T + (rev ? n - s0 - C : s0);
        return Rows{(const char*)ptr + t0 * ld + (int64_t)head * d * es, (rev ? -C : C) * (int64_t)ld,
                    (uint32_t)((C - 1) * ld + d * es), ld};
    };
    auto row_off = [&](int row, int ld) { return (rev ? C - 1 - row : row) * ld; };
    constexpr int kPast = -16;                               // an offset past any buffer's end
    Rows X = rows_of(p.x.p, p.x.n, hx, DA, sizeof(E)), Y = rows_of(p.y.p, p.y.n, hy, DA, sizeof(E)),
         U = rows_of(p.u.p, p.u.n, hu, DB, sizeof(E)), Out = rows_of(p.out, p.n_out, ho, DB, os);
    auto row_of = [&](int i, int d) { return (tid + i * NT) / (d / PE); };
    int ox[RA], oy[RA], ou[RB], oo[2];
#pragma unroll
    for (int i = 0; i < RA; ++i) {
        ox[i] = row_off(row_of(i, DA), X.ld) + (tid + i * NT) % (DA / PE) * 16;
        oy[i] = row_off(row_of(i, DA), Y.ld) + (tid + i * NT) % (DA / PE) * 16;
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) ou[i] = row_off(row_of(i, DB), U.ld) + (tid + i * NT) % (DB / PE) * 16;
#pragma unroll
    for (int q = 0; q < 2; ++q) oo[q] = row_off(16 * q + j, Out.ld) + (cbase + cstep * g) * os;

    u32x4 rx[RA], ry[RA], ru[RB];
    // The next chunk, of c steps.  Past the last one (c <= 0) every offset is
    // past the buffer: the loads are issued all the same, so that the number in
    // flight is known at every wait (a branch around them made each wait one
    // for the youngest load: 1.6 us a chunk).
    auto load = [&](int c) {
        const Rsrc x = make_rsrc(X.base, X.bytes), y = make_rsrc(Y.base, Y.bytes), u = make_rsrc(U.base, U.bytes);
#pragma unroll
        for (int i = 0; i < RA; ++i) {
            const bool in = row_of(i, DA) < c;
            if (!STATE) rx[i] = buf_load<u32x4>(x, in ? ox[i] : kPast);
            ry[i] = buf_load<u32x4>(y, in ? oy[i] : kPast);
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) ru[i] = buf_load<u32x4>(u, row_of(i, DB) < c ? ou[i] : kPast);
        X.base += X.step;
        Y.base += Y.step;
        U.base += U.step;
    };
    // A 16-byte piece to LDS: bf16 as it is, four fp32 values as their terms.
    auto put = [](bf16* dst, int plane, u32x4 v) {
        if constexpr (NE == 1) {
            *reinterpret_cast<u32x4*>(dst) = v;
        } else {
            f32x4 x = __builtin_bit_cast(f32x4, v);
#pragma unroll
            for (int s = 0; s < NE; ++s) {
                const bf16x4 h = pack4(x);
                *reinterpret_cast<bf16x4*>(dst + s * plane) = h;
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] -= (float)h[i];
            }
        }
    };
    auto stage = [&](auto set) {
        constexpr int buf = decltype(set)::value;
#pragma unroll
        for (int i = 0; i < RA; ++i) {
            const int at = row_of(i, DA) * LA + (tid + i * NT) % (DA / PE) * PE;
            if (PA % NT == 0 || tid + i * NT < PA) {
                if (!STATE) put(&s_x[STATE ? 0 : buf][at], QA, rx[i]);
                put(&s_y[buf][at], QA, ry[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const int at = row_of(i, DB) * LB + (tid + i * NT) % (DB / PE) * PE;
            if (PB % NT == 0 || tid + i * NT < PB) put(&s_u[buf][at], QB, ru[i]);
        }
    };

    // One chunk from LDS buffer k; the next is staged into the other buffer and
    // the one after it set out for.
    auto chunk = [&](auto set, int s) {
        constexpr int k = decltype(set)::value;
        constexpr std::integral_constant<int, 1 - k> other{};
        const int c = min(C, s1 - s);
        __syncthreads();                                     // this chunk is staged, the last one read
        stage(other);
        load(s1 - s - 2 * C);
        if (c < C) chunk_weights(c);
        const bf16 *sx = s_x[STATE ? 0 : k], *sy = s_y[k], *su = s_u[k];
        Terms<NE> uf[NC];
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) uf[ct] = col_terms<NE>(su, QB, LB, cbase + 4 * ct, cstep, j, g);
        if constexpr (!STATE) {
            f32x4 p00 = zero4(), p01 = zero4(), p11 = zero4(), o[NC][2];
#pragma unroll
            for (int ct = 0; ct < NC; ++ct) o[ct][0] = o[ct][1] = zero4();
#pragma unroll
            for (int m = 0; m < KM; ++m) {
                const int e = 32 * m + 8 * g;
                const Terms<NE> x0 = row_terms<NE>(sx + j * LA + e, QA), x1 = row_terms<NE>(sx + (16 + j) * LA + e, QA);
                const Terms<NE> y0 = row_terms<NE>(sy + j * LA + e, QA), y1 = row_terms<NE>(sy + (16 + j) * LA + e, QA);
                p00 = mma(y0, x0, p00);
                p01 = mma(y0, x1, p01);
                p11 = mma(y1, x1, p11);
#pragma unroll
                for (int ct = 0; ct < NC; ++ct) {
                    const Terms<NP> mf = to_terms<NP>(M[2 * m][ct], M[2 * m + 1][ct]);
                    o[ct][0] = mma(mf, x0, o[ct][0]);
                    o[ct][1] = mma(mf, x1, o[ct][1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p00[i] *= wd[i];
                p01[i] *= wo[i];
                p11[i] *= wd[i];
            }
            const Terms<NP> w0 = to_terms<NP>(p00, zero4()), w1 = to_terms<NP>(p01, p11);
            const Rsrc out = make_rsrc(Out.base, Out.bytes);
            Out.base += Out.step;
#pragma unroll
            for (int ct = 0; ct < NC; ++ct) {
                o[ct][0] = mma(uf[ct], w0, wi[0] * o[ct][0]);
                o[ct][1] = mma(uf[ct], w1, wi[1] * o[ct][1]);
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int off = 16 * q + j < c ? oo[q] : kPast;
                if (os == 2) {
                    if constexpr (NC == 2) {
                        buf_store_u32x4(out, off, __builtin_bit_cast(u32x4, pack8(o[0][q], o[1][q])));
                    } else {
                        buf_store_u32x2(out, off, __builtin_bit_cast(u32x2, pack4(o[0][q])));
                    }
                } else {
#pragma unroll
                    for (int ct = 0; ct < NC; ++ct)
                        buf_store_u32x4(out, off == kPast ? kPast : off + 16 * ct, __builtin_bit_cast(u32x4, o[ct][q]));
                }
            }
        }
        Terms<3> us[NC];                                     // the state keeps fp32's accuracy
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) {
            f32x4 lo, hi;
            to_f32(uf[ct], lo, hi);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] *= wu[i];
                hi[i] *= wu[4 + i];
            }
            us[ct] = to_terms<3>(lo, hi);
        }
        const float f = chunk_decay();
#pragma unroll
        for (int t = 0; t < 2 * KM; ++t) {
            const Terms<NE> yt = col_terms<NE>(sy, QA, LA, 32 * (t >> 1) + 4 * (t & 1), 8, j, g);
#pragma unroll
            for (int ct = 0; ct < NC; ++ct) {
                M[t][ct] = mma(yt, us[ct], f * M[t][ct]);
            }
        }
    };

    if (s0 < s1) {
        constexpr std::integral_constant<int, 0> set0{};
        constexpr std::integral_constant<int, 1> set1{};
        chunk_weights(C);
        load(s1 - s0);
        stage(set0);
        load(s1 - s0 - C);
        for (int s = s0;; s += 2 * C) {
            chunk(set0, s);
            if (s + C >= s1) break;
            chunk(set1, s + C);
            if (s + 2 * C >= s1) break;
        }
    }

    if constexpr (STATE) {
        float* w = slot(seg);
#pragma unroll
        for (int t = 0; t < 2 * KM; ++t)
#pragma unroll
            for (int ct = 0; ct < NC; ++ct) quad(w, t, ct) = M[t][ct];
    } else if (last && p.S.out) {
        float* out = p.S.out + ((size_t)(p.S.out_slot ? p.S.out_slot[b] : b) * p.H + h) * (DA * DB);
#pragma unroll
        for (int t = 0; t < 2 * KM; ++t)
#pragma unroll
            for (int ct = 0; ct < NC; ++ct)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    out[(32 * (t >> 1) + 8 * g + 4 * (t & 1) + i) * DB + col(ct)] = M[t][ct][i];
    }
}

// dq[row, hk], then dk: the sum of src[row, h] over the heads h that share hk,
// in order.  src: dq's then dk's, each fp32 [rows, H, d]; count elements each.
template <typename E>
__global__ __launch_bounds__(256) void linear_share_kernel(const float* __restrict__ src, E* __restrict__ dq,
                                                           E* __restrict__ dk, const int* __restrict__ lens, int T,
                                                           int Hk, int G, int d, size_t count) {
    for (size_t at = (size_t)blockIdx.x * 256 + threadIdx.x; at < 2 * count; at += (size_t)gridDim.x * 256) {
        const size_t i = at < count ? at : at - count;
        const size_t tok = i / ((size_t)Hk * d), rest = i % ((size_t)Hk * d);
        if (lens && (int)(tok % T) >= lens[tok / T]) continue;
        const int hk = (int)(rest / d), e = (int)(rest % d);
        const float* from = src + (at < count ? 0 : count * G) + (tok * Hk * G + (size_t)hk * G) * d + e;
        float s = 0.f;
        for (int j = 0; j < G; ++j) s += from[j * d];
        (at < count ? dq : dk)[i] = from_f32<E>(s);
    }
}

// ------------------------------------------------------------------ launches

// Column tiles a wave holds.  128 columns as eight waves of one tile or four of
// two: eight hide a chunk's latencies better (B1 H32 T1024 bf16 30 against 34
// us), four form the pair weights half as often, which counts where every CU has
// work throughout (B8 H32 T8192 519 against 492 us, gradients of B1 H32 T4096 165
// against 151).
static int wave_tiles(int passes, int B, int H, int db) {
    return db == 128 && (long long)B * H * passes >= 96 ? 2 : 1;
}

// Segments of a sequence.  One segment leaves CUs idle where there are few
// (b, h); R of them cost a first launch over the tokens, and every workgroup
// of the second reads the states before its own.  The estimate below, in us,
// is taken for each R and the least wins.  Its constants are measured: a chunk
// takes `out` us in the second launch and `state` us in the first where each CU
// has one workgroup, 0.3 of that more for another on the CU (eight waves fit;
// fp32's LDS takes one workgroup), and workgroups beyond that wait for a round
// of their own; a launch takes no less than its rows at 5.2 TB/s, and as much
// longer as the busiest CU has more than its share; the first one takes 6 us of
// its own, and the states move at 8 TB/s.  Of a padded batch three quarters of the
// workgroups are taken to have tokens.  B1 H32 T4096 d128 bf16: 197 us
// with one segment, 93 with 4, 62 with 8, 92 with 10; its gradients: 204 with one,
// 134 with 4, 116 with 5, 139 with 6; B8 H32 T8192: 477 with one, 636 with 2; B4 H16
// T2048 fp32: 328 with one, 156 with 4, 202 with 16.
static LinearSegs segments(int passes, int states, int B, int T, int H, int da, int db, bool is_bf16, bool padded) {
    const double units = (double)B * H * passes * (padded ? 0.75 : 1.0), size = da * db / 16384.0;
    const double out = is_bf16 ? 0.7 + 0.7 * size : 1.1 + 4.0 * size;
    const double state = is_bf16 ? 0.4 + 0.35 * size : 0.7 + 2.0 * size;
    const double token = units * T * (da + db) * (is_bf16 ? 2 : 4) / 5.2e6;   // us to move y and u, or x and out
    const int fit = is_bf16 ? 8 * 16 * wave_tiles(passes, B, H, db) / db : 1;
    auto busy = [&](double groups) {
        const double round = 256.0 * fit, rounds = std::floor(groups / round), rest = groups - rounds * round;
        return rounds * (1 + 0.3 * (fit - 1)) + (rest > 0 ? 1 + 0.3 * (std::ceil(rest / 256) - 1) : 0);
    };
    LinearSegs best{1, (T + kLinChunk - 1) / kLinChunk * kLinChunk};
    double least = 0;
    for (int r = 1; r <= 32; ++r) {
        const int chunks = ((T + r - 1) / r + kLinChunk - 1) / kLinChunk, len = chunks * kLinChunk;
        const int R = (T + len - 1) / len;
        if (R != r) continue;
        const double share = units * R / 256;
        double us = std::max(chunks * out * busy(units * R), 2 * token * std::max(1.0, std::ceil(share) / share));
        if (R > 1)
            us += 6 + std::max(chunks * state * busy(units * states / passes * (R - 1)), token * states / passes * (R - 1) / R) +
                  units * da * db * 4 * (0.5 * R * (R - 1) + 2 * R) / 8e6;
        if (r == 1 || us < least) {
            least = us;
            best = {R, len};
        }
    }
    return best;
}

// Workspace of one pass's segments, for a batch padded or not.
static size_t segs_bytes(int passes, int states, int B, int T, int H, int da, int db, bool is_bf16) {
    const int R = std::max(segments(passes, states, B, T, H, da, db, is_bf16, false).R,
                           segments(passes, states, B, T, H, da, db, is_bf16, true).R);
    return R > 1 ? (size_t)B * H * R * da * db * sizeof(float) : 0;
}

template <typename E, int DA, int DB, int NC, int NP>
static hipError_t launch_job_n(const LinearJob& job, hipStream_t stream) {
    const unsigned units = (unsigned)(job.pass[0].B * job.pass[0].H);
    const dim3 block(DB / NC * 4);
    if (job.segs.R > 1) {
        hipLaunchKernelGGL((linear_chunk_kernel<E, DA, DB, NC, 1, true>), dim3(units * job.state * (job.segs.R - 1)), block,
                           0, stream, job);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((linear_chunk_kernel<E, DA, DB, NC, NP, false>), dim3(units * job.passes * job.segs.R), block, 0,
                       stream, job);
    return hipGetLastError();
}

// bf16: the state and the pair weights enter their products as one bf16 term
// each, which leaves half a step of bf16 on each part of the output's sum
// beside its own rounding (2.3e-3 of the norm against 1.7e-3).  A second term
// removes that and costs a fifth and more of a chunk's arithmetic (everywhere: B1
// H32 T4096 75 against 64 us, B8 H32 T8192 617 against 487, gradients of B1 H32
// T4096 150 against 124), which only a pass of a few chunks and one tile a wave,
// latency for the most part, has to spare: with two tiles a wave the CUs are
// full, whatever the length.  So a sequence's rounding depends on the batch.
template <typename E, int DA, int DB>
static hipError_t launch_job_d(const LinearJob& job, hipStream_t stream) {
    constexpr int NP = sizeof(E) == 2 ? 1 : 3;
    if constexpr (DB == 128) {
        if (wave_tiles(job.passes, job.pass[0].B, job.pass[0].H, DB) == 2)
            return launch_job_n<E, DA, DB, 2, NP>(job, stream);
    }
    if constexpr (sizeof(E) == 2) {
        if (job.segs.len <= 4 * kLinChunk) return launch_job_n<E, DA, DB, 1, 2>(job, stream);
    }
    return launch_job_n<E, DA, DB, 1, NP>(job, stream);
}

template <typename E, int DA>
static hipError_t launch_job_a(const LinearJob& job, hipStream_t stream) {
    switch (job.pass[0].db) {
        case 32: return launch_job_d<E, DA, 32>(job, stream);
        case 64: return launch_job_d<E, DA, 64>(job, stream);
        default: return launch_job_d<E, DA, 128>(job, stream);
    }
}

template <typename E>
static hipError_t launch_job_e(const LinearJob& job, hipStream_t stream) {
    switch (job.pass[0].da) {
        case 32: return launch_job_a<E, 32>(job, stream);
        case 64: return launch_job_a<E, 64>(job, stream);
        default: return launch_job_a<E, 128>(job, stream);
    }
}

static hipError_t launch_job(const LinearJob& job, hipStream_t stream) {
    return job.pass[0].is_bf16 ? launch_job_e<bf16>(job, stream) : launch_job_e<float>(job, stream);
}

size_t linear_prefill_ws_bytes(int B, int T, int H, int da, int db, bool is_bf16) {
    return segs_bytes(1, 1, B, T, H, da, db, is_bf16);
}

hipError_t launch_linear_prefill(const LinearPass& p, void* ws, hipStream_t stream) {
    return launch_job(LinearJob{{p}, {(float*)ws}, {}, 1, 1, p.H / p.x.n, segments(1, 1, p.B, p.T, p.H, p.da, p.db, p.is_bf16, p.lens != nullptr)}, stream);
}

// The segment states of S and of R, then (shared heads) dq and dk of every
// head in fp32, summed afterwards.
size_t linear_backward_ws_bytes(int B, int T, int H, int Hk, int dk, int dv, bool is_bf16) {
    return 2 * segs_bytes(3, 2, B, T, H, dk, dv, is_bf16) + (H == Hk ? 0 : 2 * (size_t)B * T * H * dk * sizeof(float));
}

hipError_t launch_linear_backward(const LinearBackward& a, void* ws, hipStream_t stream) {
    const bool shared = a.H != a.Hk;
    const int n = shared ? a.H : a.Hk;
    const size_t seg_bytes = segs_bytes(3, 2, a.B, a.T, a.H, a.dk_, a.dv_, a.is_bf16);
    float *seg_s = (float*)ws, *seg_r = (float*)((char*)ws + seg_bytes), *part = (float*)((char*)ws + 2 * seg_bytes);
    const size_t rows = (size_t)a.B * a.T;
    const LinearPass dq{{a.dO, a.H}, {a.v, a.H}, {a.k, a.Hk}, shared ? part : a.dq, n, shared || !a.is_bf16, a.g,
                        a.scale, 1.0f, dense_state(a.S0, nullptr), true, a.lens, false, a.B, a.T, a.H, a.dv_, a.dk_,
                        a.is_bf16};
    const LinearPass dk{{a.v, a.H}, {a.dO, a.H}, {a.q, a.Hk}, shared ? part + rows * a.H * a.dk_ : a.dk, n,
                        shared || !a.is_bf16, a.g, 1.0f, a.scale, dense_state(a.dST, nullptr), true, a.lens, true,
                        a.B, a.T, a.H, a.dv_, a.dk_, a.is_bf16};
    const LinearPass dv{{a.k, a.Hk}, {a.q, a.Hk}, {a.dO, a.H}, a.dv, a.H, !a.is_bf16, a.g, 1.0f, a.scale,
                        dense_state(a.dST, a.dS0), false, a.lens, true, a.B, a.T, a.H, a.dk_, a.dv_, a.is_bf16};
    // dk's states are dv's, transposed
    const LinearSegs segs = segments(3, 2, a.B, a.T, a.H, a.dk_, a.dv_, a.is_bf16, a.lens != nullptr);
    hipError_t e;
    if (a.dk_ == a.dv_) {                                    // one launch for the three
        e = launch_job(LinearJob{{dq, dv, dk}, {seg_s, seg_r, seg_r}, {false, false, true}, 3, 2, a.H / a.Hk, segs}, stream);
    } else if ((e = launch_job(LinearJob{{dv}, {seg_r}, {}, 1, 1, a.H / a.Hk, segs}, stream)) == hipSuccess) {
        e = launch_job(LinearJob{{dq, dk}, {seg_s, seg_r}, {false, true}, 2, 1, a.H / a.Hk, segs}, stream);
    }
    if (e != hipSuccess) return e;
    if (!shared) return hipSuccess;
    const size_t count = rows * a.Hk * a.dk_;
    const dim3 grid((unsigned)std::min<size_t>((2 * count + 255) / 256, 1 << 14));
    if (a.is_bf16)
        hipLaunchKernelGGL((linear_share_kernel<bf16>), grid, dim3(256), 0, stream, part, (bf16*)a.dq, (bf16*)a.dk,
                           a.lens, a.T, a.Hk, a.H / a.Hk, a.dk_, count);
    else
        hipLaunchKernelGGL((linear_share_kernel<float>), grid, dim3(256), 0, stream, part, (float*)a.dq, (float*)a.dk,
                           a.lens, a.T, a.Hk, a.H / a.Hk, a.dk_, count);
    return hipGetLastError();
}

}  // namespace kda
