// kda_block_norm.hip -- between two blocks: the block's output y normed (or
// not), weighted, gated and scaled, added to the residual stream r, and the norm
// that the next block reads; and the gradients.
//   m = y r_y or y,  u = s Sigmoid(z) w_y m,  h = r + u,  n = w_n h r_h
//   with r_x = (mean x^2 + eps)^{-1/2}
//   dr = dh + r_h (t - k mean(k t)),  k = h r_h, t = w_n dn;   dw_n = sum dn k
//   du = s dr;  dw_y = sum du a m;  dz = du w_y m a (1 - a);  t_y = du a w_y
//   dy = r_y (t_y - m mean(m t_y)) or t_y
// n is formed of h before its rounding; the gradients of h as it was stored.
//
// Bound by the one read and one write of the rows.  A row is held in registers,
// as up to NV pieces of 16 bytes in each of TPR threads: one wave (four rows a
// workgroup, no LDS), 256 or 1024 threads, which sum through LDS in fixed order.
#include <algorithm>

#include "kda_delta.hpp"
#include "kda_norm.hpp"

namespace kda {

// Most workgroups of a launch; more rows loop.  Each row slot of the gradients'
// workgroups leaves partial weight gradients.
constexpr int kBlockGroups = 4096, kBlockBwdGroups = 512;

// Sums over a row's TPR threads, the same in all of them.  With more than one
// wave, a call uses buffer `at` of LDS, which the call after the next may reuse.
template <int TPR>
struct RowSum {
    static constexpr int W = TPR / kWave;
    float (*s)[W][2];   // [3][W][2]
    int at = 0;
    __device__ void operator()(float& a, float& b) {
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            a += __shfl_xor(a, o);
            b += __shfl_xor(b, o);
        }
        if constexpr (W > 1) {
            if (lane_id() == 0) {
                s[at][threadIdx.x / kWave][0] = a;
                s[at][threadIdx.x / kWave][1] = b;
            }
            __syncthreads();
            a = b = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                a += s[at][i][0];
                b += s[at][i][1];
            }
            at = at == 2 ? 0 : at + 1;
        }
    }
};

template <typename E, int TPR, int NV, bool BWD>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void block_norm_kernel(BlockNorm p, float* __restrict__ part) {
    constexpr int VE = 16 / sizeof(E), NT = TPR < 256 ? 256 : TPR, RPW = NT / TPR;
    __shared__ float s_sum[3][TPR / kWave][2];
    RowSum<TPR> sum{s_sum};
    const int t = threadIdx.x % TPR, slot = TPR < 256 ? wave_id() : 0, pieces = p.D / VE;
    const float inv = 1.0f / (float)p.D;
    auto load = [&](const void* base, size_t row, int v, float (&x)[VE]) {
        unpack<E, VE>(__builtin_nontemporal_load(reinterpret_cast<const u32x4*>((const E*)base + row * p.D) + v * TPR + t), x);
    };
    auto store = [&](void* base, size_t row, int v, const float (&x)[VE]) {
        store_row<E, VE>((E*)base + row * p.D + (size_t)(v * TPR + t) * VE, x);
    };
    auto weight = [&](const float* w, int v, float (&x)[VE]) {
#pragma unroll
        for (int i = 0; i < VE; i += 4)
            *reinterpret_cast<f32x4*>(&x[i]) = *reinterpret_cast<const f32x4*>(w + (size_t)(v * TPR + t) * VE + i);
    };
    auto has = [&](int v) { return v * TPR + t < pieces; };
    // r of the row in x, which is taken times `scale` where its squares leave fp32
    auto norm = [&](float (&x)[NV][VE], float& scale) {
        auto mean = [&](float eps) {
            float a = 0.f, b = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < VE; ++i) a += x[v][i] * x[v][i];
            sum(a, b);
            return a * inv + eps;
        };
        float m = mean(p.eps);
        scale = 1.0f;
        if (__builtin_expect(!mean_in_range(m), false)) {    // the same for the whole row
            scale = m > 1.0f ? kDown : 1.0f / kDown;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < VE; ++i) x[v][i] *= scale;
            m = mean(p.eps * scale * scale);
        }
        return 1.0f / sqrtf(m);
    };
    float dwy[BWD ? NV : 1][VE], dwn[BWD ? NV : 1][VE];
#pragma unroll
    for (int v = 0; v < (BWD ? NV : 1); ++v)
#pragma unroll
        for (int i = 0; i < VE; ++i) dwy[v][i] = dwn[v][i] = 0.f;
    for (long long row = (long long)blockIdx.x * RPW + slot; row < p.rows; row += (long long)gridDim.x * RPW) {
        float y[NV][VE], h[NV][VE], scale;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < VE; ++i) y[v][i] = h[v][i] = 0.f;
        if (p.y) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (has(v)) load(p.y, row, v, y[v]);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (has(v)) load(BWD ? p.h_in : p.r, row, v, h[v]);
        float ry = 1.0f, yscale = 1.0f;
        if (p.norm_y) ry = norm(y, yscale);
        if constexpr (!BWD) {
            if (p.y) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    if (!has(v)) continue;
                    float w[VE], z[VE];
                    if (p.w_y) weight(p.w_y, v, w);
                    if (p.z) load(p.z, row, v, z);
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        float u = y[v][i] * ry, s, rest;
                        if (p.w_y) u *= w[i];
                        if (p.z) {
                            sigmoids(z[i], s, rest);
                            u *= s;
                        }
                        h[v][i] += p.scale * u;
                    }
                    store(p.h, row, v, h[v]);
                }
            }
            const float r = norm(h, scale);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!has(v)) continue;
                float w[VE];
                if (p.w_n) weight(p.w_n, v, w);
#pragma unroll
                for (int i = 0; i < VE; ++i) h[v][i] *= p.w_n ? r * w[i] : r;
                store(p.n, row, v, h[v]);
            }
        } else {
            const float r = norm(h, scale);
            float t1[NV][VE], dot = 0.f, none = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
#pragma unroll
                for (int i = 0; i < VE; ++i) t1[v][i] = 0.f;
                if (!has(v)) continue;
                float w[VE];
                load(p.dn, row, v, t1[v]);
                if (p.w_n) weight(p.w_n, v, w);
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    h[v][i] *= r;
                    dwn[v][i] += t1[v][i] * h[v][i];
                    if (p.w_n) t1[v][i] *= w[i];
                    dot += t1[v][i] * h[v][i];
                }
            }
            sum(dot, none);
            dot *= inv;
            float dot_y = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!has(v)) continue;
                float x[VE], w[VE], z[VE], dz[VE];
                if (p.dh) load(p.dh, row, v, x);
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const float g = scale * (r * (t1[v][i] - dot * h[v][i]));
                    t1[v][i] = p.dh ? x[i] + g : g;
                }
                store(p.dr, row, v, t1[v]);
                if (!p.y) continue;
                if (p.w_y) weight(p.w_y, v, w);
                if (p.z) load(p.z, row, v, z);
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const float du = p.scale * t1[v][i];
                    float s = 1.0f, rest = 0.f;
                    y[v][i] *= ry;
                    if (p.z) sigmoids(z[i], s, rest);
                    dwy[v][i] += du * s * y[v][i];
                    float dm = du * s;
                    if (p.w_y) dm *= w[i];
                    dz[i] = dm * y[v][i] * rest;
                    dot_y += dm * y[v][i];
                    t1[v][i] = dm;
                }
                if (p.z) store(p.dz, row, v, dz);
            }
            if (p.y) {
                if (p.norm_y) {
                    sum(dot_y, none);
                    dot_y *= inv;
                }
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    if (!has(v)) continue;
                    if (p.norm_y) {
#pragma unroll
                        for (int i = 0; i < VE; ++i) t1[v][i] = yscale * (ry * (t1[v][i] - dot_y * y[v][i]));
                    }
                    store(p.dy, row, v, t1[v]);
                }
            }
        }
    }
    if (BWD && part) {
        float* at = part + ((size_t)blockIdx.x * RPW + slot) * 2 * p.D;
#pragma unroll
        for (int v = 0; v < (BWD ? NV : 1); ++v) {
            if (!has(v)) continue;
#pragma unroll
            for (int i = 0; i < VE; i += 4) {
                const size_t e = (size_t)(v * TPR + t) * VE + i;
                *reinterpret_cast<f32x4*>(at + e) = *reinterpret_cast<const f32x4*>(&dwy[v][i]);
                *reinterpret_cast<f32x4*>(at + p.D + e) = *reinterpret_cast<const f32x4*>(&dwn[v][i]);
            }
        }
    }
}

// The sum of the row slots' partial weight gradients, 16 columns a workgroup.
__global__ __launch_bounds__(256) void block_norm_dw_kernel(const float* __restrict__ part, int n, int D,
                                                            float* __restrict__ dw_y, float* __restrict__ dw_n) {
    __shared__ float s_t[16][17];
    const int e = blockIdx.x * 16 + threadIdx.x % 16, row = threadIdx.x / 16;
    float t = 0.f;
#pragma unroll 16
    for (int i = row; i < n; i += 16) t += part[(size_t)i * 2 * D + e];
    s_t[row][threadIdx.x % 16] = t;
    __syncthreads();
    if (row == 0) {
#pragma unroll
        for (int i = 1; i < 16; ++i) t += s_t[i][threadIdx.x];
        float* dw = e < D ? dw_y : dw_n;
        if (dw) dw[e < D ? e : e - D] = t;
    }
}

// Threads of a row and pieces of a thread: up to four pieces each.
struct BlockShape {
    int tpr, nv;
};
static BlockShape block_shape(int D, bool is_bf16) {
    const int pieces = D / (is_bf16 ? 8 : 4), tpr = pieces <= 256 ? 64 : pieces <= 1024 ? 256 : 1024;
    const int nv = (pieces + tpr - 1) / tpr;
    return {tpr, nv > 2 ? 4 : nv};
}
static int block_groups(long long rows, int tpr, int most) {
    const int rpw = tpr < 256 ? 256 / tpr : 1;
    return (int)std::min<long long>((rows + rpw - 1) / rpw, most);
}
static int block_slots(long long rows, int tpr) {   // partial weight gradients
    return block_groups(rows, tpr, kBlockBwdGroups) * (tpr < 256 ? 256 / tpr : 1);
}

template <typename E, bool BWD, int TPR, int NV>
static hipError_t launch_v(const BlockNorm& a, float* part, hipStream_t stream) {
    const dim3 grid((unsigned)block_groups(a.rows, TPR, BWD ? kBlockBwdGroups : kBlockGroups)), block(TPR < 256 ? 256 : TPR);
    hipLaunchKernelGGL((block_norm_kernel<E, TPR, NV, BWD>), grid, block, 0, stream, a, part);
    return hipGetLastError();
}

template <typename E, bool BWD, int TPR>
static hipError_t launch_t(const BlockNorm& a, float* part, int nv, hipStream_t stream) {
    if constexpr (TPR == 64) {
        if (nv == 1) return launch_v<E, BWD, TPR, 1>(a, part, stream);
    }
    return nv == 2 ? launch_v<E, BWD, TPR, 2>(a, part, stream) : launch_v<E, BWD, TPR, 4>(a, part, stream);
}

template <typename E, bool BWD>
static hipError_t launch_e(const BlockNorm& a, float* part, hipStream_t stream) {
    const BlockShape s = block_shape(a.D, sizeof(E) == 2);
    switch (s.tpr) {
        case 64: return launch_t<E, BWD, 64>(a, part, s.nv, stream);
        case 256: return launch_t<E, BWD, 256>(a, part, s.nv, stream);
        default: return launch_t<E, BWD, 1024>(a, part, s.nv, stream);
    }
}

hipError_t launch_block_norm(const BlockNorm& a, hipStream_t stream) {
    return a.is_bf16 ? launch_e<bf16, false>(a, nullptr, stream) : launch_e<float, false>(a, nullptr, stream);
}

size_t block_norm_backward_ws_bytes(long long rows, int D, bool is_bf16) {
    return (size_t)block_slots(rows, block_shape(D, is_bf16).tpr) * 2 * D * sizeof(float);
}

hipError_t launch_block_norm_backward(const BlockNorm& a, void* ws, hipStream_t stream) {
    float* part = a.dw_y || a.dw_n ? (float*)ws : nullptr;
    const hipError_t e = a.is_bf16 ? launch_e<bf16, true>(a, part, stream) : launch_e<float, true>(a, part, stream);
    if (e != hipSuccess || !part) return e;
    hipLaunchKernelGGL(block_norm_dw_kernel, dim3(2 * a.D / 16), dim3(256), 0, stream, part,
                       block_slots(a.rows, block_shape(a.D, a.is_bf16).tpr), a.D, a.dw_y, a.dw_n);
    return hipGetLastError();
}

}  // namespace kda
