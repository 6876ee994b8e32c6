// kda_norm_rope.hip -- the norm of each head's queries and keys with the
// position rotation in the same pass, and its gradients.
//   n = x r,  r = (c sum x^2 + eps)^{-1/2};  u = w n;  y = Rot(angle) u
//   du = Rot(-angle) dy;  dw = sum du n;  dn = w du;
//   dx = r dn - c r^3 x (x . dn)
#include "kda_device.hpp"
#include "kda_linear.hpp"

namespace kda {

// cos and sin of pos * f.  The product is formed and reduced to a turn in
// 64 bits: at position 10^6 a product in fp32 would be off by 0.03 radians.
__device__ __forceinline__ void angle(int pos, float f, float& c, float& s) {
    double turns = (double)pos * (double)f * 0.15915494309189533577;
    turns -= rint(turns);
    sincosf((float)(turns * 6.28318530717958647693), &s, &c);
}

// Element index of the other of e's pair, and the pair's index; e < rot.
__device__ __forceinline__ int pair_of(int e, int rot, bool il, int& other) {
    const int half = rot / 2;
    if (il) {
        other = e ^ 1;
        return e >> 1;
    }
    other = e < half ? e + half : e - half;
    return e < half ? e : e - half;
}

// One wave per row; a workgroup per token.
template <typename E, bool BWD>
__global__ __launch_bounds__(256) void norm_rope_kernel(NormRope p, float* __restrict__ part) {
    __shared__ float s_c[64], s_s[64], s_u[4][128], s_dw[4][2][128];
    const int tok = blockIdx.x, wave = wave_id(), lane = lane_id();
    const int d = p.d, half = p.rot / 2;
    const float c = p.rms ? 1.0f / (float)d : 1.0f;
    if ((int)threadIdx.x < half) {
        float cs, sn;
        angle(p.positions[tok], p.inv_freq[threadIdx.x], cs, sn);
        s_c[threadIdx.x] = cs;
        s_s[threadIdx.x] = BWD ? -sn : sn;
    }
    for (int e = lane; e < 128; e += kWave) s_dw[wave][0][e] = s_dw[wave][1][e] = 0.f;
    __syncthreads();
    for (int row = wave; row < p.H + p.Hk; row += 4) {
        const bool isk = row >= p.H;
        const size_t off = isk ? ((size_t)tok * p.Hk + row - p.H) * d : ((size_t)tok * p.H + row) * d;
        const E* x = (const E*)(isk ? p.k : p.q) + off;
        const E* dy = (const E*)(isk ? p.dy_k : p.dy_q) + off;
        const float* w = isk ? p.w_k : p.w_q;
        E* y = (E*)(isk ? p.y_k : p.y_q) + off;
        float xv[2], sum = 0.f;
        for (int i = 0; i < 2; ++i) {
            const int e = lane + 64 * i;
            xv[i] = e < d ? to_f32(x[e]) : 0.f;
            sum += xv[i] * xv[i];
            if (e < d) s_u[wave][e] = BWD ? to_f32(dy[e]) : xv[i];
        }
        for (int o = 1; o < kWave; o <<= 1) sum += __shfl_xor(sum, o);
        const float r = 1.0f / sqrtf(c * sum + p.eps);
        if (!BWD) {
            for (int i = 0; i < 2; ++i) {
                const int e = lane + 64 * i;
                if (e < d) s_u[wave][e] = xv[i] * r * (w ? w[e] : 1.0f);
            }
        }
        __builtin_amdgcn_wave_barrier();
        __threadfence_block();
        float dn[2], dot = 0.f;
        for (int i = 0; i < 2; ++i) {
            const int e = lane + 64 * i;
            dn[i] = 0.f;
            if (e >= d) continue;
            float u = s_u[wave][e];
            if (e < p.rot) {
                int other;
                const int j = pair_of(e, p.rot, p.interleaved, other);
                const bool first = p.interleaved ? (e & 1) == 0 : e < half;
                u = u * s_c[j] + (first ? -1.f : 1.f) * s_u[wave][other] * s_s[j];
            }
            if (!BWD) {
                y[e] = from_f32<E>(u);
            } else {
                s_dw[wave][isk][e] += u * xv[i] * r;
                dn[i] = u * (w ? w[e] : 1.0f);
                dot += dn[i] * xv[i];
            }
        }
        if (BWD) {
            for (int o = 1; o < kWave; o <<= 1) dot += __shfl_xor(dot, o);
            for (int i = 0; i < 2; ++i) {
                const int e = lane + 64 * i;
                if (e < d) y[e] = from_f32<E>(r * dn[i] - c * r * r * r * xv[i] * dot);
            }
        }
        __builtin_amdgcn_wave_barrier();
        __threadfence_block();
    }
    if (BWD && part) {
        __syncthreads();
        for (int e = threadIdx.x; e < 2 * d; e += 256) {
            float t = 0.f;
            for (int v = 0; v < 4; ++v) t += s_dw[v][e / d][e % d];
            part[(size_t)tok * 2 * d + e] = t;
        }
    }
}

__global__ __launch_bounds__(64) void norm_rope_dw_kernel(const float* __restrict__ part, size_t n, int d,
                                                          float* __restrict__ dw_q, float* __restrict__ dw_k) {
    const int e = blockIdx.x;   // 0 .. 2 d - 1
    float t = 0.f;
    for (size_t i = threadIdx.x; i < n; i += 64) t += part[i * 2 * d + e];
    for (int o = 1; o < kWave; o <<= 1) t += __shfl_xor(t, o);
    float* dw = e < d ? dw_q : dw_k;
    if (threadIdx.x == 0 && dw) dw[e % d] = t;
}

hipError_t launch_norm_rope(const NormRope& a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * a.T));
    if (a.is_bf16)
        hipLaunchKernelGGL((norm_rope_kernel<bf16, false>), grid, dim3(256), 0, stream, a, (float*)nullptr);
    else
        hipLaunchKernelGGL((norm_rope_kernel<float, false>), grid, dim3(256), 0, stream, a, (float*)nullptr);
    return hipGetLastError();
}

size_t norm_rope_backward_ws_bytes(int B, int T, int H, int Hk, int d) {
    return (size_t)B * T * 2 * d * sizeof(float);
}

hipError_t launch_norm_rope_backward(const NormRope& a, void* ws, hipStream_t stream) {
    const bool dw = a.dw_q || a.dw_k;
    const dim3 grid((unsigned)(a.B * a.T));
    float* part = dw ? (float*)ws : nullptr;
    if (a.is_bf16)
        hipLaunchKernelGGL((norm_rope_kernel<bf16, true>), grid, dim3(256), 0, stream, a, part);
    else
        hipLaunchKernelGGL((norm_rope_kernel<float, true>), grid, dim3(256), 0, stream, a, part);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !dw) return e;
    hipLaunchKernelGGL(norm_rope_dw_kernel, dim3(2 * a.d), dim3(64), 0, stream, part, (size_t)a.B * a.T, a.d, a.dw_q,
                       a.dw_k);
    return hipGetLastError();
}

}  // namespace kda
