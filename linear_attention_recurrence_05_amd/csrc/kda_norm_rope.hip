// kda_norm_rope.hip -- the norm of each head's queries and keys with the
// position rotation in the same pass, and its gradients.
//   n = x r,  r = (c sum x^2 + eps)^{-1/2};  u = w n;  y = Rot(angle) u
//   du = Rot(-angle) dy;  dw = sum du n;  dn = w du;
//   dx = r dn - c r^3 x (x . dn)
//
// Bound by the one read and one write of the rows.  A workgroup takes a token
// at a time: its cos and sin are formed once, in LDS, and serve all heads of
// q and k.  A row lies in d / VE neighbouring lanes of 16 bytes each, so a
// wave reads and writes 1 KB at a time, sums within the row's lanes, and gets
// the other element of a pair from the same lane (interleaved), from a lane
// rot / 2 elements away (halves of whole lanes), or through LDS (any other rot).
#include <algorithm>

#include "kda_device.hpp"
#include "kda_linear.hpp"

namespace kda {

constexpr int kNormMaxGroups = 2048;   // workgroups of a launch (8 a CU); more tokens loop
constexpr int kNormDwGroups = 512;     // the same where each leaves a partial weight gradient

// cos and sin of pos * f.  The product is formed and reduced to a turn in
// 64 bits: at position 10^6 a product in fp32 would be off by 0.03 radians.
__device__ __forceinline__ void angle(int pos, float f, float& c, float& s) {
    double turns = (double)pos * (double)f * 0.15915494309189533577;
    turns -= rint(turns);
    sincosf((float)(turns * 6.28318530717958647693), &s, &c);
}

// How a lane gets the other elements of its pairs.
enum class Pairs { kNone, kLane, kShuffle, kLds };

template <typename E, int VE>
__device__ __forceinline__ void load_row(const E* p, float (&x)[VE]) {
    E e[VE];
    *reinterpret_cast<u32x4*>(e) = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
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

template <typename E, int D, bool BWD, Pairs PAIRS>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormRope p, float* __restrict__ part) {
    constexpr int VE = 16 / sizeof(E), LR = D / VE, RW = kWave / LR;   // lanes of a row, rows of a wave
    __shared__ __align__(16) float s_c[D / 2], s_s[D / 2];
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
    for (int64_t tok = blockIdx.x; tok < tokens; tok += gridDim.x) {
        if (PAIRS != Pairs::kNone) {
            __syncthreads();                                  // the last token's angles are used
            if (tid < half) {
                float cs, sn;
                angle(p.positions[tok], p.inv_freq[tid], cs, sn);
                s_c[tid] = cs;
                s_s[tid] = BWD ? -sn : sn;
            }
            __syncthreads();
        }
        // rows 0 .. H - 1 are q's heads, the rest k's; the rows of one wave step
        // end at H so that a step has one weight
        const int steps_q = (p.H + RW - 1) / RW, steps = steps_q + (p.Hk + RW - 1) / RW;
        for (int step = tid / kWave; step < steps; step += 4) {
            const bool isk = step >= steps_q;
            const int head = (isk ? step - steps_q : step) * RW + tid % kWave / LR, heads = isk ? p.Hk : p.H;
            const bool in = head < heads;
            const size_t off = ((size_t)tok * heads + (in ? head : 0)) * D + e0;
            float x[VE], u[VE];
            load_row<E, VE>((const E*)(isk ? p.k : p.q) + off, x);
            if (BWD) load_row<E, VE>((const E*)(isk ? p.dy_k : p.dy_q) + off, u);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < VE; ++i) sum += x[i] * x[i];
#pragma unroll
            for (int o = 1; o < LR; o <<= 1) sum += __shfl_xor(sum, o);
            const float r = 1.0f / sqrtf(c * sum + p.eps);
            if (!BWD) {
#pragma unroll
                for (int i = 0; i < VE; ++i) u[i] = x[i] * r * (isk ? wk[i] : wq[i]);
            }
            if constexpr (PAIRS == Pairs::kLane) {
                if (e0 < p.rot) {
#pragma unroll
                    for (int i = 0; i < VE; i += 2) {
                        if (e0 + i >= p.rot) break;
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
#pragma unroll
                        for (int i = 0; i < VE; ++i)
                            u[i] = u[i] * s_c[pr + i] + (first ? -other[i] : other[i]) * s_s[pr + i];
                    }
                } else {                                      // within the wave's own part of LDS
                    float* row = s_x + tid / LR * D;
#pragma unroll
                    for (int i = 0; i < VE; ++i) row[e0 + i] = u[i];
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        const int e = e0 + i;
                        if (e >= p.rot) continue;
                        const bool lo = e < half;
                        const int pr = lo ? e : e - half;
                        const float o = row[lo ? e + half : pr];
                        u[i] = u[i] * s_c[pr] + (lo ? -o : o) * s_s[pr];
                    }
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                }
            }
            if (BWD) {
                float dot = 0.f;
                const float keep = in ? r : 0.f;
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const float dw = u[i] * x[i] * keep;
                    if (isk) dwk[i] += dw; else dwq[i] += dw;
                    u[i] *= isk ? wk[i] : wq[i];
                    dot += u[i] * x[i];
                }
#pragma unroll
                for (int o = 1; o < LR; o <<= 1) dot += __shfl_xor(dot, o);
                const float f = c * r * r * dot;
#pragma unroll
                for (int i = 0; i < VE; ++i) u[i] = r * (u[i] - f * x[i]);
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
#pragma unroll 4
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
                        : a.interleaved ? Pairs::kLane
                        : (a.rot / 2) % VE == 0 ? Pairs::kShuffle : Pairs::kLds;
    const dim3 grid((unsigned)groups), block(256);
    switch (pairs) {
        case Pairs::kNone: hipLaunchKernelGGL((norm_rope_kernel<E, D, BWD, Pairs::kNone>), grid, block, 0, stream, a, part); break;
        case Pairs::kLane: hipLaunchKernelGGL((norm_rope_kernel<E, D, BWD, Pairs::kLane>), grid, block, 0, stream, a, part); break;
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
    return launch_any<false>(a, nullptr, norm_groups(a.B, a.T, kNormMaxGroups), stream);
}

size_t norm_rope_backward_ws_bytes(int B, int T, int H, int Hk, int d) {
    return (size_t)norm_groups(B, T, kNormDwGroups) * 2 * d * sizeof(float);
}

hipError_t launch_norm_rope_backward(const NormRope& a, void* ws, hipStream_t stream) {
    const bool dw = a.dw_q || a.dw_k;
    const int groups = norm_groups(a.B, a.T, dw ? kNormDwGroups : kNormMaxGroups);
    hipError_t e = launch_any<true>(a, dw ? (float*)ws : nullptr, groups, stream);
    if (e != hipSuccess || !dw) return e;
    hipLaunchKernelGGL(norm_rope_dw_kernel, dim3(2 * a.d / 16), dim3(256), 0, stream, (const float*)ws, groups, a.d,
                       a.dw_q, a.dw_k);
    return hipGetLastError();
}

}  // namespace kda
