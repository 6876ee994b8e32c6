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
// workgroup, no LDS) or a workgroup, which sums through LDS in fixed order.  A
// workgroup takes several rows, with the next one's pieces in flight and the
// weights, twice a bf16 row's bytes each, in registers throughout: 4,096 bf16 rows
// of 7,168 with norm, gate and weights take 52 us, 5.7 TB/s (85 us with one row of
// a workgroup after the other and the weights read for each), the gradients of
// 2,002 rows of 4,096 take 38.5 us (57.5 us), of 8,192 rows of 512 24 us (30 us with
// a partial weight gradient for each row of a workgroup).  Of the widest rows they take
// 126 us for 2,002 bf16 ones of 16,384, 4.2 TB/s (236 with spills), 113 us for 1,000 fp32
// ones (198).
#include <algorithm>

#include "kda_delta.hpp"
#include "kda_norm.hpp"

namespace kda {

// Waves of a launch at most, about as many as a device holds: more rows loop.
constexpr int kBlockWaves = 4096;

// Sums over a row's TPR threads, the same in all of them.  With more than one
// wave, a call uses buffer `at` of LDS, which the call after the next may reuse.
template <int TPR>
struct RowSum {
    static constexpr int W = TPR / kWave;
    float* s;   // [2][W]
    int at = 0;
    __device__ float operator()(float a) {
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) a += __shfl_xor(a, o);
        if constexpr (W > 1) {
            if (lane_id() == 0) s[at * W + threadIdx.x / kWave] = a;
            __syncthreads();
            a = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) a += s[at * W + i];
            at ^= 1;
        }
        return a;
    }
};

template <typename E, int TPR, int NV, bool BWD>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void block_norm_kernel(BlockNorm p, float* __restrict__ part) {
    constexpr int VE = 16 / sizeof(E), NT = TPR < 256 ? 256 : TPR, RPW = NT / TPR;
    constexpr bool FAST = sizeof(E) == 2;
    constexpr bool AHEAD = TPR < 1024;   // 1,024 threads have half the registers
    // Sixteen elements a thread do not leave room for their weights and for the sums of
    // the weights' gradients in 128 registers (120 and 151 of them were spilled): such
    // rows read the weights again, from L2, and keep the sums in LDS, each thread its own
    // columns; of fp32 rows z and dh are loaded where they are used.
    constexpr bool LEAN = BWD && TPR == 1024 && NV * VE > 8, LATE = LEAN && sizeof(E) == 4;
    __shared__ float s_sum[2 * TPR / kWave];
    RowSum<TPR> sum{s_sum};
    const int t = threadIdx.x % TPR, slot = TPR < 256 ? wave_id() : 0, pieces = p.D / VE;
    const float inv = 1.0f / (float)p.D;
    auto has = [&](int v) { return v * TPR + t < pieces; };
    __shared__ __align__(16) float s_lean[LEAN ? 2 : 1][LEAN ? TPR * NV * VE : 1];
    constexpr int NW = LEAN ? 1 : NV;
    float wy[NW][VE], wn[NW][VE];
    auto weights = [&](const float* w, int v, float (&x)[VE]) {
#pragma unroll
        for (int i = 0; i < VE; i += 4) {
            const size_t e = (size_t)(v * TPR + t) * VE + i;
            *reinterpret_cast<f32x4*>(&x[i]) = w && has(v) ? *reinterpret_cast<const f32x4*>(w + e) : f32x4{1.f, 1.f, 1.f, 1.f};
        }
    };
    if constexpr (!LEAN) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            weights(p.w_y, v, wy[v]);
            weights(p.w_n, v, wn[v]);
        }
    }
    struct Row {
        u32x4 y[NV], h[NV], z[NV], dn[BWD ? NV : 1], dh[BWD ? NV : 1];
    };
    auto fetch = [&](long long row, Row& x) {                // pieces that are absent: zeros
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const bool in = row < p.rows && has(v);
            const size_t at = ((size_t)row * p.D) / VE + v * TPR + t;
            auto get = [&](const void* base) {
                return base && in ? __builtin_nontemporal_load((const u32x4*)base + at) : u32x4{0, 0, 0, 0};
            };
            x.y[v] = get(p.y);
            x.h[v] = get(BWD ? p.h_in : p.r);
            if constexpr (!LATE) x.z[v] = get(p.z);
            if constexpr (BWD) {
                x.dn[v] = get(p.dn);
                if constexpr (!LATE) x.dh[v] = get(p.dh);
            }
        }
    };
    auto late = [&](const void* base, long long row, int v) {
        const size_t at = ((size_t)row * p.D) / VE + v * TPR + t;
        return base && has(v) ? __builtin_nontemporal_load((const u32x4*)base + at) : u32x4{0, 0, 0, 0};
    };
    auto store = [&](void* base, long long row, int v, const float (&x)[VE]) {
        store_row<E, VE>((E*)base + (size_t)row * p.D + (size_t)(v * TPR + t) * VE, x);
    };
    // r of the row in x, which is taken times `scale` where its squares leave fp32
    auto norm = [&](float (&x)[NV][VE], float& scale) {
        auto mean = [&](float eps) {
            float a = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < VE; ++i) a += x[v][i] * x[v][i];
            return sum(a) * inv + eps;
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
    float dwy[BWD ? NW : 1][VE], dwn[BWD ? NW : 1][VE];      // LEAN: of the piece at hand
#pragma unroll
    for (int v = 0; v < (BWD ? NW : 1); ++v)
#pragma unroll
        for (int i = 0; i < VE; ++i) dwy[v][i] = dwn[v][i] = 0.f;
    auto to_lds = [&](int of, int v, float (&x)[VE]) {       // adds x to piece v's sums, and clears it
#pragma unroll
        for (int i = 0; i < VE; i += 4) {
            if (part) *reinterpret_cast<f32x4*>(&s_lean[of][(v * TPR + t) * VE + i]) += *reinterpret_cast<const f32x4*>(&x[i]);
            *reinterpret_cast<f32x4*>(&x[i]) = zero4();
        }
    };
    if constexpr (LEAN) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < VE; i += 4)
                *reinterpret_cast<f32x4*>(&s_lean[0][(v * TPR + t) * VE + i]) = *reinterpret_cast<f32x4*>(&s_lean[1][(v * TPR + t) * VE + i]) = zero4();
    }
    const long long step = (long long)gridDim.x * RPW;
    long long row = (long long)blockIdx.x * RPW + slot;
    Row next;
    if constexpr (AHEAD) fetch(row, next);
    for (; row < p.rows; row += step) {
        if constexpr (!AHEAD) fetch(row, next);
        const Row cur = next;
        if constexpr (AHEAD) fetch(row + step, next);
        float y[NV][VE], h[NV][VE], scale;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            unpack<E, VE>(cur.y[v], y[v]);
            unpack<E, VE>(cur.h[v], h[v]);
        }
        float ry = 1.0f, yscale = 1.0f;
        if (p.norm_y) ry = norm(y, yscale);
        if constexpr (!BWD) {
            if (p.y) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    float z[VE];
                    unpack<E, VE>(cur.z[v], z);
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        // the factors first: y, and y w_y, may be beyond fp32 where u is not
                        float c = p.scale * wy[v][i];
                        if (p.z) c *= sigmoid<FAST>(z[i]);
                        h[v][i] += y[v][i] * ry * c;
                    }
                    if (has(v)) store(p.h, row, v, h[v]);
                }
            }
            const float r = norm(h, scale);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
#pragma unroll
                for (int i = 0; i < VE; ++i) h[v][i] *= r * wn[v][i];
                if (has(v)) store(p.n, row, v, h[v]);
            }
        } else {
            const float r = norm(h, scale);
            float g[NV][VE], dot = 0.f, dot_y = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int k = LEAN ? 0 : v;
                unpack<E, VE>(cur.dn[v], g[v]);
                if constexpr (LEAN) weights(p.w_n, v, wn[0]);
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    h[v][i] *= r;
                    dwn[k][i] += g[v][i] * h[v][i];
                    g[v][i] *= wn[k][i];
                    dot += g[v][i] * h[v][i];
                }
                if constexpr (LEAN) to_lds(1, v, dwn[0]);
            }
            dot = sum(dot) * inv;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float x[VE], z[VE], dz[VE];
                unpack<E, VE>(LATE ? late(p.dh, row, v) : cur.dh[v], x);
#pragma unroll
                for (int i = 0; i < VE; ++i) g[v][i] = x[i] + scale * (r * (g[v][i] - dot * h[v][i]));
                if (has(v)) store(p.dr, row, v, g[v]);
                if (!p.y) continue;
                const int k = LEAN ? 0 : v;
                unpack<E, VE>(LATE ? late(p.z, row, v) : cur.z[v], z);
                if constexpr (LEAN) weights(p.w_y, v, wy[0]);
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    float s = 1.0f, rest = 0.f;
                    if (p.z) sigmoids<FAST>(z[i], s, rest);
                    y[v][i] *= ry;
                    const float du = p.scale * g[v][i] * s;
                    dwy[k][i] += du * y[v][i];
                    const float dm = du * wy[k][i];
                    dz[i] = dm * rest * y[v][i];             // in this order, as above
                    dot_y += dm * y[v][i];
                    g[v][i] = dm;
                }
                if constexpr (LEAN) to_lds(0, v, dwy[0]);
                if (p.z && has(v)) store(p.dz, row, v, dz);
            }
            if (p.y) {
                if (p.norm_y) dot_y = sum(dot_y) * inv;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    if (p.norm_y) {
#pragma unroll
                        for (int i = 0; i < VE; ++i) g[v][i] = yscale * (ry * (g[v][i] - dot_y * y[v][i]));
                    }
                    if (has(v)) store(p.dy, row, v, g[v]);
                }
            }
        }
    }
    if constexpr (BWD) {
        if (!part) return;
        float* to = part + (size_t)blockIdx.x * 2 * p.D;
        if constexpr (RPW > 1) {                             // of the workgroup's rows, in order
            constexpr int W = TPR * NV * VE;                 // >= D
            __shared__ __align__(16) float s_dw[RPW][2][W];
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < VE; i += 4) {
                    const int e = (v * TPR + t) * VE + i;
                    *reinterpret_cast<f32x4*>(&s_dw[slot][0][e]) = *reinterpret_cast<const f32x4*>(&dwy[v][i]);
                    *reinterpret_cast<f32x4*>(&s_dw[slot][1][e]) = *reinterpret_cast<const f32x4*>(&dwn[v][i]);
                }
            __syncthreads();
            for (int e = threadIdx.x; e < 2 * p.D; e += NT) {
                const int of = e >= p.D, col = e - of * p.D;
                float x = s_dw[0][of][col];
#pragma unroll
                for (int r = 1; r < RPW; ++r) x += s_dw[r][of][col];
                to[e] = x;
            }
        } else {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                if (!has(v)) continue;
#pragma unroll
                for (int i = 0; i < VE; i += 4) {
                    const size_t e = (size_t)(v * TPR + t) * VE + i;
                    *reinterpret_cast<f32x4*>(to + e) = *reinterpret_cast<const f32x4*>(LEAN ? &s_lean[0][e] : &dwy[LEAN ? 0 : v][i]);
                    *reinterpret_cast<f32x4*>(to + p.D + e) = *reinterpret_cast<const f32x4*>(LEAN ? &s_lean[1][e] : &dwn[LEAN ? 0 : v][i]);
                }
            }
        }
    }
}

// Threads of a row, so that each has at most two pieces of it (of the widest fp32
// rows four).
static int block_threads(int D, bool is_bf16) {
    const int pieces = D / (is_bf16 ? 8 : 4);
    return pieces <= 128 ? 64 : pieces <= 512 ? 256 : pieces <= 1024 ? 512 : 1024;
}
static int block_groups(long long rows, int tpr, int most_waves) {
    const int rpw = tpr < 256 ? 256 / tpr : 1, waves = std::max(tpr, 256) / kWave;
    return (int)std::min<long long>((rows + rpw - 1) / rpw, most_waves / waves);
}
// Of the gradients as many as a device holds: half as many waves with two pieces a
// thread (228 registers) as with one (120), but for rows of 1,024 threads, which have
// 128 registers whatever they hold.  Each leaves partial weight gradients.
static int block_bwd_groups(long long rows, int D, bool is_bf16) {
    const int tpr = block_threads(D, is_bf16);
    return block_groups(rows, tpr, D / (is_bf16 ? 8 : 4) <= tpr || tpr == 1024 ? kBlockWaves : kBlockWaves / 2);
}

template <typename E, bool BWD, int TPR, int NV>
static hipError_t launch_v(const BlockNorm& a, float* part, hipStream_t stream) {
    const dim3 grid((unsigned)(BWD ? block_bwd_groups(a.rows, a.D, a.is_bf16) : block_groups(a.rows, TPR, kBlockWaves))), block(TPR < 256 ? 256 : TPR);
    hipLaunchKernelGGL((block_norm_kernel<E, TPR, NV, BWD>), grid, block, 0, stream, a, part);
    return hipGetLastError();
}

template <typename E, bool BWD>
static hipError_t launch_e(const BlockNorm& a, float* part, hipStream_t stream) {
    const int pieces = a.D / (sizeof(E) == 2 ? 8 : 4), tpr = block_threads(a.D, sizeof(E) == 2);
    switch (tpr) {
        case 64: return pieces <= 64 ? launch_v<E, BWD, 64, 1>(a, part, stream) : launch_v<E, BWD, 64, 2>(a, part, stream);
        case 256: return pieces <= 256 ? launch_v<E, BWD, 256, 1>(a, part, stream) : launch_v<E, BWD, 256, 2>(a, part, stream);
        case 512: return launch_v<E, BWD, 512, 2>(a, part, stream);
        default:
            if constexpr (sizeof(E) == 4) {
                if (pieces > 2048) return launch_v<E, BWD, 1024, 4>(a, part, stream);
            }
            return launch_v<E, BWD, 1024, 2>(a, part, stream);
    }
}

hipError_t launch_block_norm(const BlockNorm& a, hipStream_t stream) {
    return a.is_bf16 ? launch_e<bf16, false>(a, nullptr, stream) : launch_e<float, false>(a, nullptr, stream);
}

size_t block_norm_backward_ws_bytes(long long rows, int D, bool is_bf16) {
    return (size_t)block_bwd_groups(rows, D, is_bf16) * 2 * D * sizeof(float);
}

hipError_t launch_block_norm_backward(const BlockNorm& a, void* ws, hipStream_t stream) {
    float* part = a.dw_y || a.dw_n ? (float*)ws : nullptr;
    const hipError_t e = a.is_bf16 ? launch_e<bf16, true>(a, part, stream) : launch_e<float, true>(a, part, stream);
    if (e != hipSuccess || !part) return e;
    hipLaunchKernelGGL(sum_parts_kernel, dim3((2 * a.D + 63) / 64), dim3(1024), 0, stream, part,
                       block_bwd_groups(a.rows, a.D, a.is_bf16), 2 * a.D, a.D, a.dw_y, a.dw_n);
    return hipGetLastError();
}

}  // namespace kda
