// kda_linear.hip -- linear attention with a decay for each head: the prefill
// and its gradients, all made of one pass (LinearPass in kda_linear.hpp).
//
// Forward: x = q, y = k, u = v.  The gradients are the same recurrence with
// other tensors in its places, since with R_t = scale q_t dO_t^T + Y_{t+1},
// Y_t = a R_t (Y_n = dS_T):
//   dq_t = scale S_t dO_t  : forward, x = dO, y = v, u = k, on S^T
//   dv_t = R_t^T k_t       : reverse, x = k, y = q, u = dO, on R
//   dk_t = R_t v_t         : reverse, x = v, y = dO, u = q, on R^T
#include "kda_device.hpp"
#include "kda_linear.hpp"

namespace kda {

// The state of unit (b, h) in a StateIO of [da, db] states.
__device__ __forceinline__ size_t state_off(int row, int h, int H, int n) {
    return ((size_t)row * H + h) * (size_t)n;
}

// Token by token: one workgroup per (b, h), each thread one column of the
// state in registers, the token's x and y rows in LDS.
template <typename E, typename O, int DA, int DB>
__global__ __launch_bounds__(DB < 64 ? 64 : DB) void linear_tokens_kernel(LinearPass p) {
    constexpr int NT = DB < 64 ? 64 : DB;
    __shared__ float s_x[DA], s_y[DA];
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H, c = threadIdx.x;
    if (p.S.skip(b)) return;
    const int n = p.lens ? min(max(p.lens[b], 0), p.T) : p.T;
    const float a = expf(fmaxf(p.g[h], kMinLogDecay));
    const int hx = h / (p.H / p.x.n), hy = h / (p.H / p.y.n), hu = h / (p.H / p.u.n),
              ho = h / (p.H / p.n_out);
    const bool col = c < DB;
    float M[DA];
    const float* in = p.S.in ? p.S.in + state_off(p.S.in_slot ? p.S.in_slot[b] : b, h, p.H, DA * DB) : nullptr;
#pragma unroll
    for (int i = 0; i < DA; ++i) M[i] = in && col ? in[p.in_t ? c * DA + i : i * DB + c] : 0.f;
    for (int s = 0; s < n; ++s) {
        const size_t t = (size_t)b * p.T + (p.reverse ? n - 1 - s : s);
        __syncthreads();
        for (int i = c; i < DA; i += NT) {
            s_x[i] = to_f32(((const E*)p.x.p)[(t * p.x.n + hx) * DA + i]);
            s_y[i] = to_f32(((const E*)p.y.p)[(t * p.y.n + hy) * DA + i]);
        }
        __syncthreads();
        if (!col) continue;
        const float u = p.su * to_f32(((const E*)p.u.p)[(t * p.u.n + hu) * DB + c]);
        float o = 0.f;
#pragma unroll
        for (int i = 0; i < DA; ++i) {
            if (!p.reverse) M[i] *= a;
            M[i] += s_y[i] * u;
            o += s_x[i] * M[i];
            if (p.reverse) M[i] *= a;
        }
        ((O*)p.out)[(t * p.n_out + ho) * DB + c] = from_f32<O>(p.so * o);
    }
    if (p.S.out && col) {
        float* out = p.S.out + state_off(p.S.out_slot ? p.S.out_slot[b] : b, h, p.H, DA * DB);
#pragma unroll
        for (int i = 0; i < DA; ++i) out[i * DB + c] = M[i];
    }
}

// dst[row, hk] = the sum of src[row, h] over the heads h that share hk, in
// order.  src fp32 [rows, H, d].
template <typename E>
__global__ __launch_bounds__(256) void linear_share_kernel(const float* __restrict__ src, E* __restrict__ dst,
                                                           const int* __restrict__ lens, int T, int Hk, int G,
                                                           int d, size_t count) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= count) return;
    const size_t tok = i / ((size_t)Hk * d), rest = i % ((size_t)Hk * d);
    if (lens && (int)(tok % T) >= lens[tok / T]) return;
    const int hk = (int)(rest / d), e = (int)(rest % d);
    float s = 0.f;
    for (int j = 0; j < G; ++j) s += src[(tok * Hk * G + (size_t)hk * G + j) * d + e];
    dst[i] = from_f32<E>(s);
}

template <typename E, typename O, int DA>
static hipError_t launch_tokens_a(const LinearPass& p, hipStream_t stream) {
    const dim3 grid((unsigned)(p.B * p.H));
    switch (p.db) {
        case 32: hipLaunchKernelGGL((linear_tokens_kernel<E, O, DA, 32>), grid, dim3(64), 0, stream, p); break;
        case 64: hipLaunchKernelGGL((linear_tokens_kernel<E, O, DA, 64>), grid, dim3(64), 0, stream, p); break;
        default: hipLaunchKernelGGL((linear_tokens_kernel<E, O, DA, 128>), grid, dim3(128), 0, stream, p); break;
    }
    return hipGetLastError();
}

template <typename E, typename O>
static hipError_t launch_tokens_e(const LinearPass& p, hipStream_t stream) {
    switch (p.da) {
        case 32: return launch_tokens_a<E, O, 32>(p, stream);
        case 64: return launch_tokens_a<E, O, 64>(p, stream);
        default: return launch_tokens_a<E, O, 128>(p, stream);
    }
}

static hipError_t launch_pass(const LinearPass& p, hipStream_t stream) {
    if (!p.is_bf16) return launch_tokens_e<float, float>(p, stream);
    return p.out_f32 ? launch_tokens_e<bf16, float>(p, stream) : launch_tokens_e<bf16, bf16>(p, stream);
}

size_t linear_prefill_ws_bytes(int B, int T, int H, int da, int db, bool is_bf16) { return 0; }

hipError_t launch_linear_prefill(const LinearPass& p, void* ws, hipStream_t stream) {
    return launch_pass(p, stream);
}

// Shared heads: dq and dk of every head in fp32, summed afterwards.
size_t linear_backward_ws_bytes(int B, int T, int H, int Hk, int dk, int dv, bool is_bf16) {
    return H == Hk ? 0 : (size_t)B * T * H * dk * sizeof(float);
}

static hipError_t launch_share(const LinearBackward& a, const float* src, void* dst, hipStream_t stream) {
    const size_t count = (size_t)a.B * a.T * a.Hk * a.dk_;
    const dim3 grid((unsigned)((count + 255) / 256));
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
    LinearPass dq{{a.dO, a.H}, {a.v, a.H}, {a.k, a.Hk}, shared ? ws : a.dq, n, shared, a.g, a.scale, 1.0f,
                  dense_state(a.S0, nullptr), true, a.lens, false, a.B, a.T, a.H, a.dv_, a.dk_, a.is_bf16};
    LinearPass dv{{a.k, a.Hk}, {a.q, a.Hk}, {a.dO, a.H}, a.dv, a.H, false, a.g, 1.0f, a.scale,
                  dense_state(a.dST, a.dS0), false, a.lens, true, a.B, a.T, a.H, a.dk_, a.dv_, a.is_bf16};
    LinearPass dk{{a.v, a.H}, {a.dO, a.H}, {a.q, a.Hk}, shared ? ws : a.dk, n, shared, a.g, 1.0f, a.scale,
                  dense_state(a.dST, nullptr), true, a.lens, true, a.B, a.T, a.H, a.dv_, a.dk_, a.is_bf16};
    hipError_t e;
    if ((e = launch_pass(dq, stream)) != hipSuccess) return e;
    if (shared && (e = launch_share(a, (const float*)ws, a.dq, stream)) != hipSuccess) return e;
    if ((e = launch_pass(dv, stream)) != hipSuccess) return e;
    if ((e = launch_pass(dk, stream)) != hipSuccess) return e;
    if (shared && (e = launch_share(a, (const float*)ws, a.dk, stream)) != hipSuccess) return e;
    return hipSuccess;
}

}  // namespace kda
