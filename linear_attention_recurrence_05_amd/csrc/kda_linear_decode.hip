// kda_linear_decode.hip -- one token of linear attention with a decay for each
// head, the state updated in place:
//   S <- a S + k v^T,   o = scale S^T q.
#include "kda_device.hpp"
#include "kda_linear.hpp"

namespace kda {

template <typename E, int DK, int DV>
__global__ __launch_bounds__(256) void linear_decode_kernel(LinearDecode p) {
    constexpr int CG = DV / 4;              // groups of 4 columns
    constexpr int RG = 256 / CG;            // row groups
    __shared__ float s_q[DK], s_k[DK];
    __shared__ f32x4 s_red[RG][CG];
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H, tid = threadIdx.x;
    if (p.S.skip(b)) return;
    const size_t unit = (size_t)b * p.H + h;
    const size_t row = (size_t)b * p.Hk + h / (p.H / p.Hk);
    const float a = expf(log_decay(p.g[h]));
    for (int i = tid; i < DK; i += 256) {
        s_q[i] = to_f32(((const E*)p.q)[row * DK + i]);
        s_k[i] = to_f32(((const E*)p.k)[row * DK + i]);
    }
    const int cg = tid % CG, rg = tid / CG;
    f32x4 v;
    for (int x = 0; x < 4; ++x) v[x] = to_f32(((const E*)p.v)[unit * DV + 4 * cg + x]);
    f32x4* S = (f32x4*)(p.S.out + ((size_t)(p.S.out_slot ? p.S.out_slot[b] : b) * p.H + h) * DK * DV);
    __syncthreads();
    f32x4 o = zero4();
    for (int c = rg; c < DK; c += RG) {
        const f32x4 s = a * S[c * CG + cg] + s_k[c] * v;
        S[c * CG + cg] = s;
        o += s_q[c] * s;
    }
    s_red[rg][cg] = o;
    __syncthreads();
    if (tid < CG) {
        f32x4 t = s_red[0][tid];
        for (int r = 1; r < RG; ++r) t += s_red[r][tid];
        for (int x = 0; x < 4; ++x) ((E*)p.o)[unit * DV + 4 * tid + x] = from_f32<E>(p.scale * t[x]);
    }
}

template <typename E, int DK>
static hipError_t launch_k(const LinearDecode& a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * a.H)), block(256);
    switch (a.dv) {
        case 32: hipLaunchKernelGGL((linear_decode_kernel<E, DK, 32>), grid, block, 0, stream, a); break;
        case 64: hipLaunchKernelGGL((linear_decode_kernel<E, DK, 64>), grid, block, 0, stream, a); break;
        default: hipLaunchKernelGGL((linear_decode_kernel<E, DK, 128>), grid, block, 0, stream, a); break;
    }
    return hipGetLastError();
}

template <typename E>
static hipError_t launch_e(const LinearDecode& a, hipStream_t stream) {
    switch (a.dk) {
        case 32: return launch_k<E, 32>(a, stream);
        case 64: return launch_k<E, 64>(a, stream);
        default: return launch_k<E, 128>(a, stream);
    }
}

hipError_t launch_linear_decode(const LinearDecode& a, hipStream_t stream) {
    return a.is_bf16 ? launch_e<bf16>(a, stream) : launch_e<float>(a, stream);
}

}  // namespace kda
