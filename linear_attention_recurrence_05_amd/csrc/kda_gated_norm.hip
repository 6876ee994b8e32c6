// kda_gated_norm.hip -- the norm of each head's output row under its gate, and
// its gradients.
//   n = x r,  r = (mean x^2 + eps)^{-1/2};  y = a(z) w n,  a = Sigmoid or SiLU
//   dw = sum dy a n;  dz = dy w n a'(z);  dn = dy a w;  dx = r (dn - n mean(n dn))
//
// Bound by the one read and one write of the rows.  A row lies in d / VE
// neighbouring lanes of 16 bytes each; a wave reads and writes 1 KB at a time
// and sums within the row's lanes, and the next rows are in flight.  With expf and
// a full division the gate bound it instead: 131,072 bf16 rows of 128 took 26.8 us;
// with the hardware's exp2 and reciprocal 20.4 us, 4.9 TB/s, as a large copy does.
#include <algorithm>

#include "kda_delta.hpp"
#include "kda_norm.hpp"

namespace kda {

// Most workgroups of a launch; more rows loop.  Each workgroup of the gradients
// leaves a partial weight gradient: of bf16 rows of 128, 512 / 1,024 / 2,048 of them
// take 18.8 / 18.8 / 22.6 us for 32,032 rows and 123 / 125 / 126 us for 524,288.
constexpr int kGatedGroups = 2048, kGatedBwdGroups = 1024;

template <typename E, int D, bool BWD, bool SILU>
__global__ __launch_bounds__(256) void gated_norm_kernel(GatedNorm p, float* __restrict__ part) {
    constexpr int VE = 16 / sizeof(E), LR = D / VE, RW = 256 / LR;   // lanes of a row, rows of a workgroup
    __shared__ float s_dw[BWD ? RW : 1][D];
    const int tid = threadIdx.x, e0 = tid % LR * VE;
    float w[VE], dw[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) {
        w[i] = p.w ? p.w[e0 + i] : 1.0f;
        dw[i] = 0.f;
    }
    struct Row {
        u32x4 x, z, dy;
    };
    auto fetch = [&](long long row) {                        // this lane's piece of a row
        Row r{};
        if (row >= p.rows) return r;
        const size_t off = (size_t)row * D + e0;
        r.x = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>((const E*)p.x + off));
        r.z = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>((const E*)p.z + off));
        if (BWD) r.dy = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>((const E*)p.dy + off));
        return r;
    };
    const long long step = (long long)gridDim.x * RW;
    long long row = (long long)blockIdx.x * RW + tid / LR;
    Row next = fetch(row);
    for (; row - tid / LR < p.rows; row += step) {           // the wave's rows end together
        const Row cur = next;
        next = fetch(row + step);
        float x[VE], z[VE];
        unpack<E, VE>(cur.x, x);
        unpack<E, VE>(cur.z, z);
        auto mean = [&](float eps) {                         // the same in all lanes of a row
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < VE; ++i) sum += x[i] * x[i];
#pragma unroll
            for (int o = 1; o < LR; o <<= 1) sum += __shfl_xor(sum, o);
            return sum * (1.0f / (float)D) + eps;
        };
        float m = mean(p.eps), scale = 1.0f;
        const bool scaled = __any(!mean_in_range(m));
        if (__builtin_expect(scaled, false)) {               // from here on x is the row times scale
            if (!mean_in_range(m)) scale = m > 1.0f ? kDown : 1.0f / kDown;
#pragma unroll
            for (int i = 0; i < VE; ++i) x[i] *= scale;
            m = mean(p.eps * scale * scale);
        }
        const float r = 1.0f / sqrtf(m);
        float dy[VE], dot = 0.f;
        if (BWD) unpack<E, VE>(cur.dy, dy);
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            x[i] *= r;                                       // n
            if (!BWD) {
                const float s = sigmoid<sizeof(E) == 2>(z[i]);
                x[i] *= (SILU ? z[i] * s : s) * w[i];
            } else {
                float s, rest;
                sigmoids<sizeof(E) == 2>(z[i], s, rest);
                const float a = SILU ? z[i] * s : s;
                const float da = SILU ? s * (1.0f + z[i] * rest) : s * rest;
                z[i] = dy[i] * x[i] * w[i] * da;             // dz
                dy[i] *= a;
                dw[i] += row < p.rows ? dy[i] * x[i] : 0.f;
                dy[i] *= w[i];                               // dn
                dot += dy[i] * x[i];
            }
        }
        if (BWD) {
#pragma unroll
            for (int o = 1; o < LR; o <<= 1) dot += __shfl_xor(dot, o);
            dot *= 1.0f / (float)D;
#pragma unroll
            for (int i = 0; i < VE; ++i) x[i] = r * (dy[i] - dot * x[i]);
            if (__builtin_expect(scaled, false)) {
#pragma unroll
                for (int i = 0; i < VE; ++i) x[i] *= scale;
            }
        }
        if (row < p.rows) {
            const size_t off = (size_t)row * D + e0;
            store_row<E, VE>((E*)p.y + off, x);
            if (BWD) store_row<E, VE>((E*)p.dz + off, z);
        }
    }
    if (BWD && part) {                                       // this workgroup's dw
#pragma unroll
        for (int i = 0; i < VE; ++i) s_dw[tid / LR][e0 + i] = dw[i];
        __syncthreads();
        for (int e = tid; e < D; e += 256) {
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < RW; ++i) t += s_dw[i][e];
            part[(size_t)blockIdx.x * D + e] = t;
        }
    }
}

__global__ __launch_bounds__(1024) void sum_parts_kernel(const float* __restrict__ part, int n, int width, int first,
                                                         float* __restrict__ a, float* __restrict__ b) {
    __shared__ float s_t[16][64];
    const int e = blockIdx.x * 64 + lane_id(), row = threadIdx.x / 64;
    float t = 0.f;
    if (e < width) {
#pragma unroll 16
        for (int i = row; i < n; i += 16) t += part[(size_t)i * width + e];
    }
    s_t[row][lane_id()] = t;
    __syncthreads();
    if (row == 0 && e < width) {
#pragma unroll
        for (int i = 1; i < 16; ++i) t += s_t[i][lane_id()];
        float* to = e < first ? a : b;
        if (to) to[e < first ? e : e - first] = t;
    }
}

static int gated_groups(long long rows, int d, bool is_bf16, int most) {
    const int per = 256 / (d / (is_bf16 ? 8 : 4));
    return (int)std::min<long long>((rows + per - 1) / per, most);
}

template <typename E, int D, bool BWD>
static hipError_t launch_d(const GatedNorm& a, float* part, hipStream_t stream) {
    const dim3 grid((unsigned)gated_groups(a.rows, D, sizeof(E) == 2, BWD ? kGatedBwdGroups : kGatedGroups)), block(256);
    if (a.silu)
        hipLaunchKernelGGL((gated_norm_kernel<E, D, BWD, true>), grid, block, 0, stream, a, part);
    else
        hipLaunchKernelGGL((gated_norm_kernel<E, D, BWD, false>), grid, block, 0, stream, a, part);
    return hipGetLastError();
}

template <bool BWD>
static hipError_t launch_any(const GatedNorm& a, float* part, hipStream_t stream) {
    switch (a.d) {
        case 32: return a.is_bf16 ? launch_d<bf16, 32, BWD>(a, part, stream) : launch_d<float, 32, BWD>(a, part, stream);
        case 64: return a.is_bf16 ? launch_d<bf16, 64, BWD>(a, part, stream) : launch_d<float, 64, BWD>(a, part, stream);
        default: return a.is_bf16 ? launch_d<bf16, 128, BWD>(a, part, stream) : launch_d<float, 128, BWD>(a, part, stream);
    }
}

hipError_t launch_gated_norm(const GatedNorm& a, hipStream_t stream) { return launch_any<false>(a, nullptr, stream); }

size_t gated_norm_backward_ws_bytes(long long rows, int d) {   // of fp32's groups: the most
    return (size_t)gated_groups(rows, d, false, kGatedBwdGroups) * d * sizeof(float);
}

hipError_t launch_gated_norm_backward(const GatedNorm& a, void* ws, hipStream_t stream) {
    hipError_t e = launch_any<true>(a, a.dw ? (float*)ws : nullptr, stream);
    if (e != hipSuccess || !a.dw) return e;
    hipLaunchKernelGGL(sum_parts_kernel, dim3((a.d + 63) / 64), dim3(1024), 0, stream, (const float*)ws,
                       gated_groups(a.rows, a.d, a.is_bf16, kGatedBwdGroups), a.d, a.d, a.dw, nullptr);
    return hipGetLastError();
}

}  // namespace kda
