// kda_linear_decode.hip -- one token of linear attention with a decay for each
// head, the state updated in place:
//   S <- a S + k v^T,   o = scale S^T q.
//
// Bound by the one read and one write of S (8 d_k d_v bytes against 4 d_k d_v
// flops): B = 256, H = 32, d = 128 in 183 us, 5.9 TB/s.  A workgroup holds one
// (b, h), each thread four columns of up to eight rows: all loads of S are in
// flight before the first is used, the update needs no reduction and is stored
// at once, and only o is summed over the rows (within the wave, then through
// LDS, in fixed order).  Two units a workgroup took 187 us, plain instead of
// non-temporal stores 197.
#include "kda_device.hpp"
#include "kda_linear.hpp"

namespace kda {

template <int DK, int DV>
constexpr int decode_threads() { return DK * DV / 32 < 64 ? 64 : DK * DV / 32; }

template <typename E, int DK, int DV>
__global__ __launch_bounds__((decode_threads<DK, DV>())) void linear_decode_kernel(LinearDecode p) {
    constexpr int NT = decode_threads<DK, DV>(), NWAVE = NT / kWave;
    constexpr int CG = DV / 4, RG = NT / CG, RPT = DK / RG;
    __shared__ float s_q[DK], s_k[DK];
    __shared__ __align__(16) float s_v[DV];
    __shared__ f32x4 s_red[NWAVE][CG];
    const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG, wave = tid / kWave, lane = tid % kWave;
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H;
    const int row = p.S.out_slot ? p.S.out_slot[b] : b;
    if (p.S.out_slot && (unsigned)row >= (unsigned)p.S.n_slots) return;
    f32x4* S = (f32x4*)(p.S.out + ((size_t)row * p.H + h) * (DK * DV));
    f32x4 st[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) st[i] = __builtin_nontemporal_load(&S[(rg + RG * i) * CG + cg]);
    const size_t qk = ((size_t)b * p.Hk + h / (p.H / p.Hk)) * DK, vo = (size_t)blockIdx.x * DV;
    for (int e = tid; e < 2 * DK + DV; e += NT) {
        if (e < DK)
            s_q[e] = to_f32(((const E*)p.q)[qk + e]);
        else if (e < 2 * DK)
            s_k[e - DK] = to_f32(((const E*)p.k)[qk + e - DK]);
        else
            s_v[e - 2 * DK] = to_f32(((const E*)p.v)[vo + e - 2 * DK]);
    }
    __syncthreads();
    const float a = expf(log_decay(p.g[h]));
    const f32x4 v = *reinterpret_cast<const f32x4*>(&s_v[4 * cg]);
    f32x4 o = zero4();
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int c = rg + RG * i;
        const f32x4 s = a * st[i] + s_k[c] * v;
        __builtin_nontemporal_store(s, &S[c * CG + cg]);
        o += s_q[c] * s;
    }
#pragma unroll
    for (int off = CG; off < kWave; off <<= 1)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[x] += __shfl_xor(o[x], off);
    if (lane < CG) s_red[wave][lane] = o;
    __syncthreads();
    if (tid < CG) {
        o = s_red[0][tid];
#pragma unroll
        for (int w = 1; w < NWAVE; ++w) o += s_red[w][tid];
        o *= p.scale;
        E* dst = (E*)p.o + vo + 4 * tid;
        if constexpr (sizeof(E) == 2)
            *reinterpret_cast<bf16x4*>(dst) = pack4(o);
        else
            *reinterpret_cast<f32x4*>(dst) = o;
    }
}

template <typename E, int DK, int DV>
static hipError_t launch_kv(const LinearDecode& a, hipStream_t stream) {
    hipLaunchKernelGGL((linear_decode_kernel<E, DK, DV>), dim3((unsigned)(a.B * a.H)), dim3(decode_threads<DK, DV>()), 0,
                       stream, a);
    return hipGetLastError();
}

template <typename E, int DK>
static hipError_t launch_k(const LinearDecode& a, hipStream_t stream) {
    switch (a.dv) {
        case 32: return launch_kv<E, DK, 32>(a, stream);
        case 64: return launch_kv<E, DK, 64>(a, stream);
        default: return launch_kv<E, DK, 128>(a, stream);
    }
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
