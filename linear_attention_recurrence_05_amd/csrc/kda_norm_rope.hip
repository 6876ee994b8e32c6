// kda_norm_rope.hip -- the norm of each head's queries and keys with the
// position rotation in the same pass, and its gradients.
//   n = x r,  r = (c sum x^2 + eps)^{-1/2};  u = w n;  y = Rot(angle) u
//   du = Rot(-angle) dy;  dw = sum du n;  dn = w du;
//   dx = r (dn - c n (n . dn))
//
// Bound, over many heads, by the one read and one write of the rows (4096 tokens
// of 32 + 32 heads, bf16, d 128: 26 us, 5.1 TB/s).  A workgroup takes a token at a
// time: its cos and sin are formed once, in LDS, and serve all heads of q and k.
// With few heads most of its row places stay empty (65,536 tokens of 1 + 1 heads of
// 32: 53 us, 0.3 TB/s), and the gradients' three or four tokens a workgroup do not
// fill the device's memory (2002 tokens of 32 + 8 heads: 19 us, 3.3 TB/s).
// A row lies in d / VE neighbouring lanes of 16 bytes each, so a
// wave reads and writes 1 KB at a time, sums within the row's lanes, and gets
// the other element of a pair from the same lane (interleaved), from a lane
// rot / 2 elements away (halves of whole lanes), or through LDS (any other rot).
#include <algorithm>

#include "kda_device.hpp"
#include "kda_linear.hpp"

namespace kda {

// Most workgroups of a launch; more tokens loop, with the next rows in flight
// (4096 tokens of H 32 + 32, bf16, d 128: 26 us forward with 1024, 35 with 512, 28
// with 4096; 2002 tokens of H 32 + 8 backward, each workgroup leaving a partial
// weight gradient: 22 us with 512 to 768, 25 with 1024, 28 with 256).
constexpr int kNormGroups = 1024, kNormBwdGroups = 768;

// Outside these means of squares (eps included) fp32 has lost squares to
// infinity, or some that count to its lower end, and the row is taken times
// 2^-80 or 2^80.  The sum of its squares is then within 2^103 or 2^67, and the
// mean at least 2^-32 or (eps being at least 2^-149) 2^11.
constexpr float kLeastMean = 0x1p-100f, kMostMean = 0x1.fffffep127f, kDown = 0x1p-80f;

// cos and sin of pos * f.  The product is formed and reduced to a turn in
// 64 bits: at position 10^6 a product in fp32 would be off by 0.03 radians.
__device__ __forceinline__ void angle(int pos, float f, float& c, float& s) {
    double turns = (double)pos * (double)f * 0.15915494309189533577;
    turns -= rint(turns);
    sincosf((float)(turns * 6.28318530717958647693), &s, &c);
}

// How a lane gets the other elements of its pairs.
enum class Pairs { kNone, kLane, kLaneAny, kShuffle, kLds };

template <typename E, int VE>
__device__ __forceinline__ void unpack(u32x4 v, float (&x)[VE]) {
    E e[VE];
    *reinterpret_cast<u32x4*>(e) = v;
#pragma unroll
    for (int i = 0; i < VE; ++i) x[i] = to_f32(e[i]);
}
template <typename E, int VE>
__device__ __forceinline__ void store_row(E* p, const float (&x)[VE]) {
    u32x4 v;
    if constexpr (sizeof(E) == 2)
        v = __builtin_bit_cast(u32x4, pack8(f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]}));
    else
        v = __builtin_bit_cast(u32x4, f32x4{x[0], x[1], x[2], x[3]});
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
}

// N consecutive floats of LDS (N of 2, 4 or 8, aligned to min(N, 4) of them).
template <int N>
__device__ __forceinline__ void copy(float (&x)[N], const float* p) {
    typedef float vec __attribute__((ext_vector_type(N < 4 ? N : 4)));
#pragma unroll
    for (int i = 0; i < N; i += N < 4 ? N : 4) *reinterpret_cast<vec*>(&x[i]) = *reinterpret_cast<const vec*>(p + i);
}

template <typename E, int D, bool BWD, Pairs PAIRS>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormRope p, float* __restrict__ part) {
    constexpr int VE = 16 / sizeof(E), LR = D / VE, RW = kWave / LR;   // lanes of a row, rows of a wave
    __shared__ __align__(16) float s_cos[2][D / 2], s_sin[2][D / 2];
    __shared__ __align__(16) float s_x[PAIRS == Pairs::kLds ? 256 * VE : 4];
    __shared__ float s_dw[BWD ? 2 * D * (256 / LR) : 1];
    const int tid = threadIdx.x, lr = tid % LR, e0 = lr * VE, half = p.rot / 2;
    const float c = p.rms ? 1.0f / (float)D : 1.0f;
    float wq[VE], wk[VE], dwq[VE], dwk[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) {
        wq[i] = p.w_q ? p.w_q[e0 + i] : 1.0f;
        wk[i] = p.w_k ? p.w_k[e0 + i] : 1.0f;
        dwq[i] = dwk[i] = 0.f;
    }
    const int64_t tokens = (int64_t)p.B * p.T;
    // rows 0 .. H - 1 are q's heads, the rest k's; the rows of one wave step end
    // at H so that a step has one weight
    // (a scalar wave index makes the choice of q or k a branch: 2 us faster
    // forward, 4 slower backward)
    const int wave = BWD ? tid / kWave : wave_id(), steps_q = (p.H + RW - 1) / RW, steps = steps_q + (p.Hk + RW - 1) / RW;
    struct Row {
        u32x4 x, dy;
        size_t off;
        bool in;
    };
    auto fetch = [&](int64_t tok, int step) {                 // this lane's part of its row of a step
        Row r{};
        if (tok >= tokens || step >= steps) return r;
        const bool isk = step >= steps_q;
        const int head = (isk ? step - steps_q : step) * RW + tid % kWave / LR, heads = isk ? p.Hk : p.H;
        r.in = head < heads;
        r.off = ((size_t)tok * heads + (r.in ? head : 0)) * D + e0;
        r.x = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>((const E*)(isk ? p.k : p.q) + r.off));
        if (BWD) r.dy = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>((const E*)(isk ? p.dy_k : p.dy_q) + r.off));
        return r;
    };
    // The last wave (whose steps are the fewest) forms the next token's angles
    // while the others use this one's; every wave has its next step's rows in
    // flight.
    const bool turns = PAIRS != Pairs::kNone && wave == 3 && tid % kWave < half;
    const float freq = turns ? p.inv_freq[tid % kWave] : 0.f;
    auto angles = [&](int64_t tok, int buf) {
        if (turns && tok < tokens) {
            float cs, sn;
            angle(p.positions[tok], freq, cs, sn);
            s_cos[buf][tid % kWave] = cs;
            s_sin[buf][tid % kWave] = BWD ? -sn : sn;
        }
    };
    Row next = fetch(blockIdx.x, wave);
    angles(blockIdx.x, 0);
    int buf = 0;
    for (int64_t tok = blockIdx.x; tok < tokens; tok += gridDim.x, buf ^= 1) {
        if (PAIRS != Pairs::kNone) __syncthreads();           // this token's angles are there, the last one's used
        angles(tok + gridDim.x, buf ^ 1);
        const float *s_c = s_cos[buf], *s_s = s_sin[buf];
        for (int step = wave; step < steps; step += 4) {
            const bool isk = step >= steps_q;
            const Row row = next;
            next = step + 4 < steps ? fetch(tok, step + 4) : fetch(tok + gridDim.x, wave);
            const bool in = row.in;
            const size_t off = row.off;
            float x[VE], u[VE];
            unpack<E, VE>(row.x, x);
            if (BWD) unpack<E, VE>(row.dy, u);
            auto mean = [&](float eps) {                      // the same in all lanes of a row
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < VE; ++i) sum += x[i] * x[i];
#pragma unroll
                for (int o = 1; o < LR; o <<= 1) sum += __shfl_xor(sum, o);
                return c * sum + eps;
            };
            float m = mean(p.eps), scale = 1.0f;
            const bool scaled = __any(!(m >= kLeastMean && m <= kMostMean));   // some row of the wave's
            if (__builtin_expect(scaled, false)) {            // from here on x is the row times scale
                if (!(m >= kLeastMean && m <= kMostMean)) scale = m > 1.0f ? kDown : 1.0f / kDown;
#pragma unroll
                for (int i = 0; i < VE; ++i) x[i] *= scale;
                m = mean(p.eps * scale * scale);
            }
            const float r = 1.0f / sqrtf(m);
            if (!BWD) {
#pragma unroll
                for (int i = 0; i < VE; ++i) u[i] = x[i] * r * (isk ? wk[i] : wq[i]);
            }
            if constexpr (PAIRS == Pairs::kLane) {            // rot is a multiple of VE
                if (e0 < p.rot) {
                    float cs[VE / 2], sn[VE / 2];
                    copy<VE / 2>(cs, &s_c[e0 / 2]);
                    copy<VE / 2>(sn, &s_s[e0 / 2]);
#pragma unroll
                    for (int i = 0; i < VE; i += 2) {
                        const float a = u[i], b = u[i + 1];
                        u[i] = a * cs[i / 2] - b * sn[i / 2];
                        u[i + 1] = b * cs[i / 2] + a * sn[i / 2];
                    }
                }
            } else if constexpr (PAIRS == Pairs::kLaneAny) {
#pragma unroll
                for (int i = 0; i < VE; i += 2) {
                    if (e0 + i < p.rot) {
                        const float cs = s_c[(e0 + i) / 2], sn = s_s[(e0 + i) / 2], a = u[i], b = u[i + 1];
                        u[i] = a * cs - b * sn;
                        u[i + 1] = b * cs + a * sn;
                    }
                }
            } else if constexpr (PAIRS != Pairs::kNone) {     // halves: e and e +- half
                float other[VE];
                const bool first = e0 < half;
                if constexpr (PAIRS == Pairs::kShuffle) {     // half is a multiple of VE
                    const int from = lane_id() + (e0 < p.rot ? (first ? half : -half) / VE : 0);
#pragma unroll
                    for (int i = 0; i < VE; ++i) other[i] = __shfl(u[i], from);
                    if (e0 < p.rot) {
                        const int pr = first ? e0 : e0 - half;
                        float cs[VE], sn[VE];
                        copy<VE>(cs, &s_c[pr]);
                        copy<VE>(sn, &s_s[pr]);
#pragma unroll
                        for (int i = 0; i < VE; ++i) u[i] = u[i] * cs[i] + (first ? -other[i] : other[i]) * sn[i];
                    }
                } else {                                      // within the wave's own part of LDS
                    float* part_row = s_x + tid / LR * D;
#pragma unroll
                    for (int i = 0; i < VE; ++i) part_row[e0 + i] = u[i];
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        const int e = e0 + i;
                        if (e >= p.rot) continue;
                        const bool lo = e < half;
                        const int pr = lo ? e : e - half;
                        const float o = part_row[lo ? e + half : pr];
                        u[i] = u[i] * s_c[pr] + (lo ? -o : o) * s_s[pr];
                    }
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                }
            }
            if (BWD) {
                // of n = r x throughout: products of dy with x may overflow where
                // the gradient does not
                float dot = 0.f;
                const float keep = in ? r : 0.f;
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    x[i] *= keep;
                    const float dw = u[i] * x[i];
                    if (isk) dwk[i] += dw; else dwq[i] += dw;
                    u[i] *= isk ? wk[i] : wq[i];
                    dot += u[i] * x[i];
                }
#pragma unroll
                for (int o = 1; o < LR; o <<= 1) dot += __shfl_xor(dot, o);
                dot *= c;
#pragma unroll
                for (int i = 0; i < VE; ++i) u[i] = r * (u[i] - dot * x[i]);
                if (__builtin_expect(scaled, false)) {
#pragma unroll
                    for (int i = 0; i < VE; ++i) u[i] *= scale;
                }
            }
            if (in) store_row<E, VE>((E*)(isk ? p.y_k : p.y_q) + off, u);
        }
    }
    if (BWD && part) {                                        // this workgroup's dw_q, dw_k
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            s_dw[tid / LR * 2 * D + e0 + i] = dwq[i];
            s_dw[tid / LR * 2 * D + D + e0 + i] = dwk[i];
        }
        __syncthreads();
        for (int e = tid; e < 2 * D; e += 256) {
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < 256 / LR; ++w) t += s_dw[w * 2 * D + e];
            part[(size_t)blockIdx.x * 2 * D + e] = t;
        }
    }
}

// The sum of the workgroups' partial weight gradients, 16 columns a workgroup.
__global__ __launch_bounds__(256) void norm_rope_dw_kernel(const float* __restrict__ part, int n, int d,
                                                           float* __restrict__ dw_q, float* __restrict__ dw_k) {
    __shared__ float s_t[16][17];
    const int e = blockIdx.x * 16 + threadIdx.x % 16, row = threadIdx.x / 16;
    float t = 0.f;
#pragma unroll 16
    for (int i = row; i < n; i += 16) t += part[(size_t)i * 2 * d + e];
    s_t[row][threadIdx.x % 16] = t;
    __syncthreads();
    if (row == 0) {
#pragma unroll
        for (int i = 1; i < 16; ++i) t += s_t[i][threadIdx.x];
        float* dw = e < d ? dw_q : dw_k;
        if (dw) dw[e % d] = t;
    }
}

template <typename E, int D, bool BWD>
static hipError_t launch_d(const NormRope& a, float* part, int groups, hipStream_t stream) {
    constexpr int VE = 16 / sizeof(E);
    const Pairs pairs = a.rot == 0 ? Pairs::kNone
                        : a.interleaved ? (a.rot % VE == 0 ? Pairs::kLane : Pairs::kLaneAny)
                        : (a.rot / 2) % VE == 0 ? Pairs::kShuffle : Pairs::kLds;
    const dim3 grid((unsigned)groups), block(256);
    switch (pairs) {
        case Pairs::kNone: hipLaunchKernelGGL((norm_rope_kernel<E, D, BWD, Pairs::kNone>), grid, block, 0, stream, a, part); break;
        case Pairs::kLane: hipLaunchKernelGGL((norm_rope_kernel<E, D, BWD, Pairs::kLane>), grid, block, 0, stream, a, part); break;
        case Pairs::kLaneAny: hipLaunchKernelGGL((norm_rope_kernel<E, D, BWD, Pairs::kLaneAny>), grid, block, 0, stream, a, part); break;
        case Pairs::kShuffle: hipLaunchKernelGGL((norm_rope_kernel<E, D, BWD, Pairs::kShuffle>), grid, block, 0, stream, a, part); break;
        case Pairs::kLds: hipLaunchKernelGGL((norm_rope_kernel<E, D, BWD, Pairs::kLds>), grid, block, 0, stream, a, part); break;
    }
    return hipGetLastError();
}

template <bool BWD>
static hipError_t launch_any(const NormRope& a, float* part, int groups, hipStream_t stream) {
    switch (a.d) {
        case 32: return a.is_bf16 ? launch_d<bf16, 32, BWD>(a, part, groups, stream) : launch_d<float, 32, BWD>(a, part, groups, stream);
        case 64: return a.is_bf16 ? launch_d<bf16, 64, BWD>(a, part, groups, stream) : launch_d<float, 64, BWD>(a, part, groups, stream);
        default: return a.is_bf16 ? launch_d<bf16, 128, BWD>(a, part, groups, stream) : launch_d<float, 128, BWD>(a, part, groups, stream);
    }
}

static int norm_groups(int B, int T, int most) { return (int)std::min<int64_t>((int64_t)B * T, most); }

hipError_t launch_norm_rope(const NormRope& a, hipStream_t stream) {
    return launch_any<false>(a, nullptr, norm_groups(a.B, a.T, kNormGroups), stream);
}

size_t norm_rope_backward_ws_bytes(int B, int T, int H, int Hk, int d) {
    return (size_t)norm_groups(B, T, kNormBwdGroups) * 2 * d * sizeof(float);
}

hipError_t launch_norm_rope_backward(const NormRope& a, void* ws, hipStream_t stream) {
    const bool dw = a.dw_q || a.dw_k;
    const int groups = norm_groups(a.B, a.T, kNormBwdGroups);
    hipError_t e = launch_any<true>(a, dw ? (float*)ws : nullptr, groups, stream);
    if (e != hipSuccess || !dw) return e;
    hipLaunchKernelGGL(norm_rope_dw_kernel, dim3(2 * a.d / 16), dim3(256), 0, stream, (const float*)ws, groups, a.d,
                       a.dw_q, a.dw_k);
    return hipGetLastError();
}

}  // namespace kda
