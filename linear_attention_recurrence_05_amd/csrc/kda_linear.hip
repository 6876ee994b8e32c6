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

#include "kda_device.hpp"
#include "kda_linear.hpp"

namespace kda {

constexpr int kLinChunk = 32;

// ------------------------------------------------------------------ operands

// Eight values of a lane, of 32 along a contraction: lane group g = lane / 16
// holds eight of them (which ones is the caller's choice, the same for both
// operands).
template <typename E> struct Frag;
template <> struct Frag<bf16> { bf16x8 v; };
template <> struct Frag<float> { f32x4 lo, hi; };

__device__ __forceinline__ f32x4 mma(const Frag<bf16>& a, const Frag<bf16>& b, f32x4 c) {
    return mma_bf16_k32(a.v, b.v, c);
}
__device__ __forceinline__ f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = mma_f32_k4(a.lo[i], b.lo[i], c);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = mma_f32_k4(a.hi[i], b.hi[i], c);
    return c;
}

template <typename E> __device__ __forceinline__ Frag<E> to_frag(f32x4 lo, f32x4 hi);
template <> __device__ __forceinline__ Frag<bf16> to_frag<bf16>(f32x4 lo, f32x4 hi) { return {pack8(lo, hi)}; }
template <> __device__ __forceinline__ Frag<float> to_frag<float>(f32x4 lo, f32x4 hi) { return {lo, hi}; }

__device__ __forceinline__ void to_f32(const Frag<bf16>& a, f32x4& lo, f32x4& hi) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo[i] = (float)a.v[i];
        hi[i] = (float)a.v[4 + i];
    }
}
__device__ __forceinline__ void to_f32(const Frag<float>& a, f32x4& lo, f32x4& hi) {
    lo = a.lo;
    hi = a.hi;
}

// Eight consecutive elements of a row in LDS (16-byte aligned).
template <typename E> __device__ __forceinline__ Frag<E> row_frag(const E* p);
template <> __device__ __forceinline__ Frag<bf16> row_frag<bf16>(const bf16* p) {
    return {*reinterpret_cast<const bf16x8*>(p)};
}
template <> __device__ __forceinline__ Frag<float> row_frag<float>(const float* p) {
    return {*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4)};
}

// Lane (j, g) = 16 g + j: column `col(j)` of rows 4 g + {0..3} and 16 + 4 g +
// {0..3} of a [32][ld] tile in LDS, where col(j) = c0 + step (j / 4) + j % 4.
// bf16: two transposing reads, for which a lane names row j / 4 and column
// group j % 4 of its group's 4 x 16 block.
template <typename E>
__device__ __forceinline__ Frag<E> col_frag(const E* s, int ld, int c0, int step, int j, int g) {
    Frag<E> f;
    if constexpr (sizeof(E) == 2) {
        typedef __attribute__((address_space(3))) i16x4 lds4;
        const E* p = s + (4 * g + (j >> 2)) * ld + c0 + step * (j & 3);
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p);
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 16 * ld));
        f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
        const E* p = s + 4 * g * ld + c0 + step * (j >> 2) + (j & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f.lo[i] = p[i * ld];
            f.hi[i] = p[(16 + i) * ld];
        }
    }
    return f;
}

// x in fp32 as a sum of bf16 terms: three hold its 24 bits, so a product with
// a bf16 operand keeps fp32's accuracy.
__device__ __forceinline__ void split(f32x4 lo, f32x4 hi, Frag<bf16> (&out)[3]) {
#pragma unroll
    for (int s = 0; s < 3; ++s) {
        out[s] = to_frag<bf16>(lo, hi);
        f32x4 a, b;
        to_f32(out[s], a, b);
        lo -= a;
        hi -= b;
    }
}
__device__ __forceinline__ void split(f32x4 lo, f32x4 hi, Frag<float> (&out)[1]) { out[0] = {lo, hi}; }

// ------------------------------------------------------------------ the pass

// Segments of a sequence run side by side: a first launch leaves in the
// workspace what each segment but the last adds to a zero state, the second
// starts every segment from the initial state and the ones before it.
struct LinearSegs {
    float* ws;   // [unit][R][DA * DB]: R - 1 segments' states, then the initial one
    int R, len;  // segments of a sequence, their length in steps (a multiple of 32)
};

// One workgroup per (b, h, segment); NW waves, each with NC tiles of 16
// columns of the state [DA, DB] in registers (MFMA accumulator layout).  A
// state tile pair in that layout is an operand of M^T x without a move: rows
// are mapped to channels so that a lane's rows of two tiles are eight
// consecutive channels.  x, y and u of a chunk are staged in LDS (two buffers,
// one barrier a chunk, the chunk after the next in flight in registers).  The
// pair weights are computed transposed (keys x queries) by every wave, which
// makes the product with u take them straight from the accumulators.
// STATE: only the state of a segment from zero, into the workspace.
template <typename E, typename O, int DA, int DB, int NW, int NC, bool STATE>
__global__ __launch_bounds__(NW * 64, 2) void linear_chunk_kernel(LinearPass p, LinearSegs segs) {
    constexpr int C = kLinChunk, NT = NW * 64, KM = DA / 32, NS = sizeof(E) == 2 ? 3 : 1;
    constexpr int PE = 16 / sizeof(E);                       // elements of 16 bytes
    constexpr int LA = DA + PE, LB = DB + PE;                // padded LDS rows
    constexpr int PA = C * DA / PE, PB = C * DB / PE;        // 16-byte pieces of a tile
    constexpr int RA = (PA + NT - 1) / NT, RB = (PB + NT - 1) / NT;
    static_assert(NW * NC * 16 == DB, "waves cover the columns");
    __shared__ __align__(16) E s_x[STATE ? 1 : 2][STATE ? 8 : C * LA];
    __shared__ __align__(16) E s_y[2][C * LA], s_u[2][C * LB];

    const int units = p.B * p.H;
    const int unit = blockIdx.x % units, seg = blockIdx.x / units;
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
    auto slot = [&](int m) {
        return reinterpret_cast<f32x4*>(segs.ws + ((size_t)unit * segs.R + m) * (DA * DB)) + wave * 2 * KM * NC * 64 + lane;
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
                if (in) slot(segs.R - 1)[(t * NC + ct) * 64] = M[t][ct];
                M[t][ct] = zero4();
            }
        }
    if (!direct) {
        const float as = expf(lg * (float)segs.len);
        if (p.S.in) {
            const f32x4* w = slot(segs.R - 1);
#pragma unroll
            for (int t = 0; t < 2 * KM; ++t)
#pragma unroll
                for (int ct = 0; ct < NC; ++ct) M[t][ct] = w[(t * NC + ct) * 64];
        }
        for (int m = 0; m < seg; ++m) {
            const f32x4* w = slot(m);
#pragma unroll
            for (int t = 0; t < 2 * KM; ++t)
#pragma unroll
                for (int ct = 0; ct < NC; ++ct) M[t][ct] = as * M[t][ct] + w[(t * NC + ct) * 64];
        }
    }

    // ---- weights of a chunk of c steps
    float wd[4], wo[4], wi[2], wu[8], ac, ac_lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int d = j - 4 * g - i;                         // query - key within a 16 x 16 block
        wd[i] = d >= 0 ? p.so * p.su * expf(lg * (float)d) : 0.f;
        wo[i] = p.so * p.su * expf(lg * (float)(16 + d));
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) wi[q] = p.so * expf(lg * (float)(16 * q + j + 1 - rev));
    auto chunk_weights = [&](int c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int left = c - 1 - ((i & 4) * 4 + 4 * g + (i & 3));
            wu[i] = left >= 0 ? p.su * expf(lg * (float)(left + rev)) : 0.f;
        }
        const double d = exp((double)lg * c);                // in two parts: their product with M
        ac = (float)d;                                       // is a^c M to fp32, chunk after chunk
        ac_lo = (float)(d - (double)ac);
    };

    // ---- loads of a chunk: rows in step order, zero past its end
    u32x4 rx[RA], ry[RA], ru[RB];
    auto load = [&](int s) {
        const int c = min(C, s1 - s);
        const size_t t0 = (size_t)b * p.T + (rev ? n - s - c : s);
        auto rsrc = [&](const HeadTensor& t, int head, int d) {
            const int ld = t.n * d * (int)sizeof(E);
            return make_rsrc((const char*)t.p + t0 * ld + (size_t)head * d * sizeof(E), (c - 1) * (uint32_t)ld + d * sizeof(E));
        };
        auto tile = [&](Rsrc r, int ld, int d, int i) {
            const int at = tid + i * NT, row = at / (d / PE), piece = at % (d / PE);
            const int off = (rev ? c - 1 - row : row) * ld + piece * 16;
            return buf_load<u32x4>(r, row < c ? off : -1 << 4);
        };
        const Rsrc x = rsrc(p.x, hx, DA), y = rsrc(p.y, hy, DA), u = rsrc(p.u, hu, DB);
#pragma unroll
        for (int i = 0; i < RA; ++i) {
            if (!STATE) rx[i] = tile(x, p.x.n * DA * (int)sizeof(E), DA, i);
            ry[i] = tile(y, p.y.n * DA * (int)sizeof(E), DA, i);
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) ru[i] = tile(u, p.u.n * DB * (int)sizeof(E), DB, i);
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < RA; ++i) {
            const int at = tid + i * NT, row = at / (DA / PE), piece = at % (DA / PE);
            if (PA % NT == 0 || at < PA) {
                if (!STATE) *reinterpret_cast<u32x4*>(&s_x[buf][row * LA + piece * PE]) = rx[i];
                *reinterpret_cast<u32x4*>(&s_y[buf][row * LA + piece * PE]) = ry[i];
            }
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const int at = tid + i * NT, row = at / (DB / PE), piece = at % (DB / PE);
            if (PB % NT == 0 || at < PB) *reinterpret_cast<u32x4*>(&s_u[buf][row * LB + piece * PE]) = ru[i];
        }
    };

    if (s0 < s1) {
        load(s0);
        stage(0);
        if (s0 + C < s1) load(s0 + C);
        chunk_weights(C);
    }
    int buf = 0;
    for (int s = s0; s < s1; s += C, buf ^= 1) {
        const int c = min(C, s1 - s);
        __syncthreads();                                     // this chunk is staged, the last one read
        if (s + C < s1) {
            stage(buf ^ 1);
            if (s + 2 * C < s1) load(s + 2 * C);
        }
        if (c < C) chunk_weights(c);
        const E *X = s_x[STATE ? 0 : buf], *Y = s_y[buf], *U = s_u[buf];
        Frag<E> uf[NC];
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) uf[ct] = col_frag<E>(U, LB, cbase + 4 * ct, cstep, j, g);
        if constexpr (!STATE) {
            f32x4 p00 = zero4(), p01 = zero4(), p11 = zero4(), o[NC][2];
#pragma unroll
            for (int ct = 0; ct < NC; ++ct) o[ct][0] = o[ct][1] = zero4();
#pragma unroll
            for (int m = 0; m < KM; ++m) {
                const int e = 32 * m + 8 * g;
                const Frag<E> x0 = row_frag<E>(X + j * LA + e), x1 = row_frag<E>(X + (16 + j) * LA + e);
                const Frag<E> y0 = row_frag<E>(Y + j * LA + e), y1 = row_frag<E>(Y + (16 + j) * LA + e);
                p00 = mma(y0, x0, p00);
                p01 = mma(y0, x1, p01);
                p11 = mma(y1, x1, p11);
#pragma unroll
                for (int ct = 0; ct < NC; ++ct) {
                    // the state rounded once to E for its product with x
                    const Frag<E> mf = to_frag<E>(M[2 * m][ct], M[2 * m + 1][ct]);
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
            // the pair weights rounded once to E for their product with u
            const Frag<E> w0 = to_frag<E>(p00, zero4()), w1 = to_frag<E>(p01, p11);
#pragma unroll
            for (int ct = 0; ct < NC; ++ct) {
                o[ct][0] = mma(uf[ct], w0, wi[0] * o[ct][0]);
                o[ct][1] = mma(uf[ct], w1, wi[1] * o[ct][1]);
            }
            const size_t t0 = (size_t)b * p.T + (rev ? n - s - c : s);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int r = 16 * q + j;
                if (r < c) {
                    O* dst = (O*)p.out + ((t0 + (rev ? c - 1 - r : r)) * p.n_out + ho) * DB + cbase + cstep * g;
#pragma unroll
                    for (int ct = 0; ct < NC; ++ct) {
                        if constexpr (sizeof(O) == 2)
                            *reinterpret_cast<bf16x4*>(dst + 4 * ct) = pack4(o[ct][q]);
                        else
                            *reinterpret_cast<f32x4*>(dst + 4 * ct) = o[ct][q];
                    }
                }
            }
        }
        Frag<E> us[NC][NS];
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) {
            f32x4 lo, hi;
            to_f32(uf[ct], lo, hi);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo[i] *= wu[i];
                hi[i] *= wu[4 + i];
            }
            split(lo, hi, us[ct]);
        }
#pragma unroll
        for (int t = 0; t < 2 * KM; ++t) {
            const Frag<E> yt = col_frag<E>(Y, LA, 32 * (t >> 1) + 4 * (t & 1), 8, j, g);
#pragma unroll
            for (int ct = 0; ct < NC; ++ct) {
                f32x4 acc = M[t][ct] * ac_lo + M[t][ct] * ac;
#pragma unroll
                for (int k = 0; k < NS; ++k) acc = mma(yt, us[ct][k], acc);
                M[t][ct] = acc;
            }
        }
    }

    if constexpr (STATE) {
        f32x4* w = slot(seg);
#pragma unroll
        for (int t = 0; t < 2 * KM; ++t)
#pragma unroll
            for (int ct = 0; ct < NC; ++ct) w[(t * NC + ct) * 64] = M[t][ct];
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

// dst[row, hk] = the sum of src[row, h] over the heads h that share hk, in
// order.  src fp32 [rows, H, d].
template <typename E>
__global__ __launch_bounds__(256) void linear_share_kernel(const float* __restrict__ src, E* __restrict__ dst,
                                                           const int* __restrict__ lens, int T, int Hk, int G,
                                                           int d, size_t count) {
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (size_t)gridDim.x * 256) {
        const size_t tok = i / ((size_t)Hk * d), rest = i % ((size_t)Hk * d);
        if (lens && (int)(tok % T) >= lens[tok / T]) continue;
        const int hk = (int)(rest / d), e = (int)(rest % d);
        float s = 0.f;
        for (int j = 0; j < G; ++j) s += src[(tok * Hk * G + (size_t)hk * G + j) * d + e];
        dst[i] = from_f32<E>(s);
    }
}

// ------------------------------------------------------------------ launches

// Segments of a sequence: as many as give the device 512 workgroups (two for
// each CU), of 256 steps at least.
static LinearSegs segments(int B, int T, int H, void* ws) {
    const long long units = (long long)B * H;
    int R = (int)((512 + units - 1) / units);
    R = std::min({R, std::max(1, T / 256), 16});
    int len = (T + R - 1) / R;
    len = (len + kLinChunk - 1) / kLinChunk * kLinChunk;
    R = (T + len - 1) / len;
    return {(float*)ws, R, len};
}

size_t linear_prefill_ws_bytes(int B, int T, int H, int da, int db, bool is_bf16) {
    const int R = segments(B, T, H, nullptr).R;
    return R > 1 ? (size_t)B * H * R * da * db * sizeof(float) : 0;
}

template <typename E, typename O, int DA, int DB>
static hipError_t launch_pass_d(const LinearPass& p, void* ws, hipStream_t stream) {
    constexpr int NW = DB == 32 ? 2 : 4, NC = DB / 16 / NW;
    const LinearSegs s = segments(p.B, p.T, p.H, ws);
    const unsigned units = (unsigned)(p.B * p.H);
    if (s.R > 1) {
        hipLaunchKernelGGL((linear_chunk_kernel<E, O, DA, DB, NW, NC, true>), dim3(units * (s.R - 1)),
                           dim3(NW * 64), 0, stream, p, s);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((linear_chunk_kernel<E, O, DA, DB, NW, NC, false>), dim3(units * s.R), dim3(NW * 64), 0,
                       stream, p, s);
    return hipGetLastError();
}

template <typename E, typename O, int DA>
static hipError_t launch_pass_a(const LinearPass& p, void* ws, hipStream_t stream) {
    switch (p.db) {
        case 32: return launch_pass_d<E, O, DA, 32>(p, ws, stream);
        case 64: return launch_pass_d<E, O, DA, 64>(p, ws, stream);
        default: return launch_pass_d<E, O, DA, 128>(p, ws, stream);
    }
}

template <typename E, typename O>
static hipError_t launch_pass_e(const LinearPass& p, void* ws, hipStream_t stream) {
    switch (p.da) {
        case 32: return launch_pass_a<E, O, 32>(p, ws, stream);
        case 64: return launch_pass_a<E, O, 64>(p, ws, stream);
        default: return launch_pass_a<E, O, 128>(p, ws, stream);
    }
}

static hipError_t launch_pass(const LinearPass& p, void* ws, hipStream_t stream) {
    if (!p.is_bf16) return launch_pass_e<float, float>(p, ws, stream);
    return p.out_f32 ? launch_pass_e<bf16, float>(p, ws, stream) : launch_pass_e<bf16, bf16>(p, ws, stream);
}

hipError_t launch_linear_prefill(const LinearPass& p, void* ws, hipStream_t stream) {
    return launch_pass(p, ws, stream);
}

// The segments' states, then (shared heads) dq or dk of every head in fp32,
// summed afterwards.
size_t linear_backward_ws_bytes(int B, int T, int H, int Hk, int dk, int dv, bool is_bf16) {
    return linear_prefill_ws_bytes(B, T, H, dk, dv, is_bf16) +
           (H == Hk ? 0 : (size_t)B * T * H * dk * sizeof(float));
}

static hipError_t launch_share(const LinearBackward& a, const float* src, void* dst, hipStream_t stream) {
    const size_t count = (size_t)a.B * a.T * a.Hk * a.dk_;
    const dim3 grid((unsigned)std::min<size_t>((count + 255) / 256, 1 << 14));
    if (a.is_bf16)
        hipLaunchKernelGGL((linear_share_kernel<bf16>), grid, dim3(256), 0, stream, src, (bf16*)dst, a.lens, a.T,
                           a.Hk, a.H / a.Hk, a.dk_, count);
    else
        hipLaunchKernelGGL((linear_share_kernel<float>), grid, dim3(256), 0, stream, src, (float*)dst, a.lens, a.T,
                           a.Hk, a.H / a.Hk, a.dk_, count);
    return hipGetLastError();
}

hipError_t launch_linear_backward(const LinearBackward& a, void* ws, hipStream_t stream) {
    const bool shared = a.H != a.Hk;
    const int n = shared ? a.H : a.Hk;
    float* part = (float*)((char*)ws + linear_prefill_ws_bytes(a.B, a.T, a.H, a.dk_, a.dv_, a.is_bf16));
    LinearPass dq{{a.dO, a.H}, {a.v, a.H}, {a.k, a.Hk}, shared ? part : a.dq, n, shared, a.g, a.scale, 1.0f,
                  dense_state(a.S0, nullptr), true, a.lens, false, a.B, a.T, a.H, a.dv_, a.dk_, a.is_bf16};
    LinearPass dv{{a.k, a.Hk}, {a.q, a.Hk}, {a.dO, a.H}, a.dv, a.H, false, a.g, 1.0f, a.scale,
                  dense_state(a.dST, a.dS0), false, a.lens, true, a.B, a.T, a.H, a.dk_, a.dv_, a.is_bf16};
    LinearPass dk{{a.v, a.H}, {a.dO, a.H}, {a.q, a.Hk}, shared ? part : a.dk, n, shared, a.g, 1.0f, a.scale,
                  dense_state(a.dST, nullptr), true, a.lens, true, a.B, a.T, a.H, a.dv_, a.dk_, a.is_bf16};
    hipError_t e;
    if ((e = launch_pass(dq, ws, stream)) != hipSuccess) return e;
    if (shared && (e = launch_share(a, part, a.dq, stream)) != hipSuccess) return e;
    if ((e = launch_pass(dv, ws, stream)) != hipSuccess) return e;
    if ((e = launch_pass(dk, ws, stream)) != hipSuccess) return e;
    if (shared && (e = launch_share(a, part, a.dk, stream)) != hipSuccess) return e;
    return hipSuccess;
}

}  // namespace kda
