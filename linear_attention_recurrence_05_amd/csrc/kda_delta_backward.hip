// kda_delta_backward.hip -- the gradients of the gated delta rule, token by token.  One workgroup of 256 threads per (b, h): thread tid holds column
// tid % DV of DK / (256 / DV) rows of the state.
#include <algorithm>

#include "kda_delta.hpp"
#include "kda_device.hpp"

namespace kda {

template <typename E, int DK, int DV>
struct Tok {
    static constexpr int NT = 256, RG = NT / DV, R = DK / RG;   // row groups, rows of a thread
    float S[R];

    static __device__ int col() { return threadIdx.x % DV; }
    static __device__ int row0() { return (int)(threadIdx.x / DV) * R; }
    __device__ void load(const float* p) {
        for (int i = 0; i < R; ++i) S[i] = p ? p[(row0() + i) * DV + col()] : 0.f;
    }
    __device__ void store(float* p) const {
        for (int i = 0; i < R; ++i) p[(row0() + i) * DV + col()] = S[i];
    }
    // sum over the rows of x[row] S[row][col], in every thread of the column
    __device__ float down(const float* x, float* s_red) const {
        float t = 0.f;
        for (int i = 0; i < R; ++i) t += x[row0() + i] * S[i];
        s_red[threadIdx.x] = t;
        __syncthreads();
        t = 0.f;
        for (int i = 0; i < RG; ++i) t += s_red[i * DV + col()];
        __syncthreads();
        return t;
    }
    // sum over the columns of S[row][col] y (y this column's), into out[row]
    __device__ void across(float y, float* out, float* s_part) const {   // s_part [4][DK]
        constexpr int W = DV < 64 ? DV : 64;
        const int wave = threadIdx.x / 64;
        for (int i = 0; i < R; ++i) {
            float t = S[i] * y;
            for (int o = 1; o < W; o <<= 1) t += __shfl_xor(t, o);
            if (threadIdx.x % W == 0) s_part[(DV > 64 ? wave % 2 : 0) * DK + row0() + i] = t;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < DK; i += NT) out[i] = s_part[i] + (DV > 64 ? s_part[DK + i] : 0.f);
        __syncthreads();
    }
    // sum of x over the columns (x the same in all row groups), in every thread
    static __device__ float all(float x, float* s_red) {
        s_red[threadIdx.x] = x;
        __syncthreads();
        float t = 0.f;
        for (int i = 0; i < DV; ++i) t += s_red[i];
        __syncthreads();
        return t;
    }
};

// Three passes over the sequence: forward (E, the token sums of dO . o, dq and
// what the old state gives dk once dv is known needs a third), reverse (dv,
// dbeta, dg, dk's first part), forward again (dk's second part).
// ws: E [B, T, H, DV], then dq and dk of every head [B, T, H, DK], all fp32.
template <typename E, int DK, int DV>
__global__ __launch_bounds__(256) void delta_backward_kernel(DeltaBackward p, float* ws) {
    using K = Tok<E, DK, DV>;
    __shared__ float s_q[DK], s_k[DK], s_red[256], s_part[4 * DK], s_out[DK];
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H, hk = h / (p.H / p.Hk);
    const int n = p.lens ? min(max(p.lens[b], 0), p.T) : p.T;
    const size_t toks = (size_t)p.B * p.T * p.H;
    float *we = ws, *wq = ws + toks * DV, *wk = wq + toks * DK;
    const float* S0 = p.S0 ? p.S0 + (size_t)blockIdx.x * DK * DV : nullptr;
    auto at = [&](int t) { return ((size_t)b * p.T + t) * p.H + h; };
    auto rows = [&](int t) {
        const size_t qk = (((size_t)b * p.T + t) * p.Hk + hk) * DK;
        for (int i = threadIdx.x; i < DK; i += 256) {
            s_q[i] = to_f32(((const E*)p.q)[qk + i]);
            s_k[i] = to_f32(((const E*)p.k)[qk + i]);
        }
        __syncthreads();
    };
    K st;
    st.load(S0);
    for (int t = 0; t < n; ++t) {
        rows(t);
        const float a = expf(log_decay(p.g[at(t)])), beta = p.beta[at(t)];
        for (int i = 0; i < K::R; ++i) st.S[i] *= a;
        const float e = to_f32(((const E*)p.v)[at(t) * DV + K::col()]) - st.down(s_k, s_red);
        if (K::row0() == 0) we[at(t) * DV + K::col()] = e;
        for (int i = 0; i < K::R; ++i) st.S[i] += s_k[K::row0() + i] * (beta * e);
        const float dO = p.scale * to_f32(((const E*)p.dO)[at(t) * DV + K::col()]);
        const float dot = K::all(dO * st.down(s_q, s_red), s_red);
        if (threadIdx.x == 0) p.dg[at(t)] = dot;
        st.across(dO, s_out, s_part);
        for (int i = threadIdx.x; i < DK; i += 256) wq[at(t) * DK + i] = s_out[i];
        __syncthreads();
    }
    K Y;
    Y.load(p.dST ? p.dST + (size_t)blockIdx.x * DK * DV : nullptr);
    float end = 0.f;
    for (int i = 0; i < K::R; ++i) end += st.S[i] * Y.S[i];
    s_red[threadIdx.x] = end;
    __syncthreads();
    double run = 0;
    for (int i = 0; i < 256; ++i) run += s_red[i];
    __syncthreads();
    for (int t = n - 1; t >= 0; --t) {
        rows(t);
        const float a = expf(log_decay(p.g[at(t)])), beta = p.beta[at(t)];
        const float e = we[at(t) * DV + K::col()], dO = p.scale * to_f32(((const E*)p.dO)[at(t) * DV + K::col()]);
        for (int i = 0; i < K::R; ++i) Y.S[i] += s_q[K::row0() + i] * dO;
        const float z = Y.down(s_k, s_red), dv = beta * z;
        const float db = K::all(z * e, s_red), vdot = K::all(dv * to_f32(((const E*)p.v)[at(t) * DV + K::col()]), s_red);
        Y.across(beta * e, s_out, s_part);
        for (int i = threadIdx.x; i < DK; i += 256) wk[at(t) * DK + i] = s_out[i];
        run += (double)p.dg[at(t)] - vdot;
        __syncthreads();
        if (threadIdx.x == 0) {
            p.dg[at(t)] = (float)run;
            p.dbeta[at(t)] = db;
        }
        if (K::row0() == 0) {
            ((E*)p.dv)[at(t) * DV + K::col()] = from_f32<E>(dv);
            we[at(t) * DV + K::col()] = dv;
        }
        for (int i = 0; i < K::R; ++i) Y.S[i] = a * (Y.S[i] - s_k[K::row0() + i] * dv);
        __syncthreads();
    }
    if (p.dS0) Y.store(p.dS0 + (size_t)blockIdx.x * DK * DV);
    __syncthreads();
    st.load(S0);
    for (int t = 0; t < n; ++t) {
        rows(t);
        const float a = expf(log_decay(p.g[at(t)])), beta = p.beta[at(t)];
        for (int i = 0; i < K::R; ++i) st.S[i] *= a;
        st.across(we[at(t) * DV + K::col()], s_out, s_part);
        for (int i = threadIdx.x; i < DK; i += 256) wk[at(t) * DK + i] -= s_out[i];
        const float e = to_f32(((const E*)p.v)[at(t) * DV + K::col()]) - st.down(s_k, s_red);
        for (int i = 0; i < K::R; ++i) st.S[i] += s_k[K::row0() + i] * (beta * e);
        __syncthreads();
    }
}

template <typename E>
__global__ __launch_bounds__(256) void delta_share_kernel(const float* __restrict__ src, E* __restrict__ dq,
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

#define KDA_BY_SIZE(E, K, V, CALL)                                             \
    switch (K * 256 + V) {                                                     \
        case 32 * 256 + 32: CALL(E, 32, 32); break;                            \
        case 32 * 256 + 64: CALL(E, 32, 64); break;                            \
        case 32 * 256 + 128: CALL(E, 32, 128); break;                          \
        case 64 * 256 + 32: CALL(E, 64, 32); break;                            \
        case 64 * 256 + 64: CALL(E, 64, 64); break;                            \
        case 64 * 256 + 128: CALL(E, 64, 128); break;                          \
        case 128 * 256 + 32: CALL(E, 128, 32); break;                          \
        case 128 * 256 + 64: CALL(E, 128, 64); break;                          \
        default: CALL(E, 128, 128); break;                                     \
    }

size_t delta_backward_ws_bytes(int B, int T, int H, int, int dk, int dv, bool) {
    return (size_t)B * T * H * (dv + 2 * dk) * sizeof(float);
}

hipError_t launch_delta_backward(const DeltaBackward& a, void* ws, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * a.H)), block(256);
#define CALL(E, K, V) hipLaunchKernelGGL((delta_backward_kernel<E, K, V>), grid, block, 0, stream, a, (float*)ws)
    if (a.is_bf16) KDA_BY_SIZE(bf16, a.dk_, a.dv_, CALL) else KDA_BY_SIZE(float, a.dk_, a.dv_, CALL)
#undef CALL
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const size_t count = (size_t)a.B * a.T * a.Hk * a.dk_;
    const float* part = (const float*)ws + (size_t)a.B * a.T * a.H * a.dv_;
    const dim3 sgrid((unsigned)std::min<size_t>((2 * count + 255) / 256, 1 << 14));
    if (a.is_bf16)
        hipLaunchKernelGGL((delta_share_kernel<bf16>), sgrid, dim3(256), 0, stream, part, (bf16*)a.dq, (bf16*)a.dk,
                           a.lens, a.T, a.Hk, a.H / a.Hk, a.dk_, count);
    else
        hipLaunchKernelGGL((delta_share_kernel<float>), sgrid, dim3(256), 0, stream, part, (float*)a.dq, (float*)a.dk,
                           a.lens, a.T, a.Hk, a.H / a.Hk, a.dk_, count);
    return hipGetLastError();
}

}  // namespace kda
