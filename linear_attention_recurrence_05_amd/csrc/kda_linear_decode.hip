// kda_linear_decode.hip -- one token of linear attention with a decay for each
// head, the state updated in place:
//   S <- a S + k v^T,   o = scale S^T q.
//
// Bound by the one read and one write of S (8 d_k d_v bytes against 4 d_k d_v
// flops).  A workgroup holds U units (b, h), each thread four columns of up to
// eight rows of every unit: all loads of S are in flight before the first is
// used, the update needs no reduction and is stored at once, and only o is
// summed over the rows (within the wave, then through LDS, in fixed order).
#include "kda_device.hpp"
#include "kda_linear.hpp"

namespace kda {

template <int DK, int DV>
constexpr int decode_threads() { return DK * DV / 32 < 64 ? 64 : DK * DV / 32; }

template <typename E, int DK, int DV, int U>
__global__ __launch_bounds__((decode_threads<DK, DV>())) void linear_decode_kernel(LinearDecode p) {
    constexpr int NT = decode_threads<DK, DV>(), NWAVE = NT / kWave;
    constexpr int CG = DV / 4, RG = NT / CG, RPT = DK / RG;
    __shared__ float s_q[U][DK], s_k[U][DK];
    __shared__ __align__(16) float s_v[U][DV];
    __shared__ f32x4 s_red[U][NWAVE][CG];
    const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG, wave = tid / kWave, lane = tid % kWave;
    const int units = p.B * p.H;
    f32x4 st[U][RPT];
    f32x4* S[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int unit = blockIdx.x * U + u;
        on[u] = unit < units;                                 // uniform over the workgroup
        const int b = on[u] ? unit / p.H : 0, h = unit % p.H;
        int row = b;
        if (p.S.out_slot) {
            row = p.S.out_slot[b];
            on[u] = on[u] && (unsigned)row < (unsigned)p.S.n_slots;
        }
        if (!on[u]) continue;
        S[u] = (f32x4*)(p.S.out + ((size_t)row * p.H + h) * (DK * DV));
#pragma unroll
        for (int i = 0; i < RPT; ++i) st[u][i] = __builtin_nontemporal_load(&S[u][(rg + RG * i) * CG + cg]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (!on[u]) continue;
        const int unit = blockIdx.x * U + u, b = unit / p.H, h = unit % p.H;
        const size_t qk = ((size_t)b * p.Hk + h / (p.H / p.Hk)) * DK, vo = (size_t)unit * DV;
        for (int e = tid; e < 2 * DK + DV; e += NT) {
            if (e < DK)
                s_q[u][e] = to_f32(((const E*)p.q)[qk + e]);
            else if (e < 2 * DK)
                s_k[u][e - DK] = to_f32(((const E*)p.k)[qk + e - DK]);
            else
                s_v[u][e - 2 * DK] = to_f32(((const E*)p.v)[vo + e - 2 * DK]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (!on[u]) continue;
        const float a = expf(log_decay(p.g[(blockIdx.x * U + u) % p.H]));
        const f32x4 v = *reinterpret_cast<const f32x4*>(&s_v[u][4 * cg]);
        f32x4 o = zero4();
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int c = rg + RG * i;
            const f32x4 s = a * st[u][i] + s_k[u][c] * v;
            __builtin_nontemporal_store(s, &S[u][c * CG + cg]);
            o += s_q[u][c] * s;
        }
#pragma unroll
        for (int off = CG; off < kWave; off <<= 1)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[x] += __shfl_xor(o[x], off);
        if (lane < CG) s_red[u][wave][lane] = o;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (!on[u] || tid >= CG) continue;
        f32x4 o = s_red[u][0][tid];
#pragma unroll
        for (int w = 1; w < NWAVE; ++w) o += s_red[u][w][tid];
        E* dst = (E*)p.o + (size_t)(blockIdx.x * U + u) * DV + 4 * tid;
        if constexpr (sizeof(E) == 2)
            *reinterpret_cast<bf16x4*>(dst) = pack4(p.scale * o);
        else
            *reinterpret_cast<f32x4*>(dst) = p.scale * o;
    }
}

template <typename E, int DK, int DV>
static hipError_t launch_kv(const LinearDecode& a, hipStream_t stream) {
    constexpr int NT = decode_threads<DK, DV>();
    const int units = a.B * a.H;
    if (units >= 1024)
        hipLaunchKernelGGL((linear_decode_kernel<E, DK, DV, 2>), dim3((unsigned)((units + 1) / 2)), dim3(NT), 0, stream, a);
    else
        hipLaunchKernelGGL((linear_decode_kernel<E, DK, DV, 1>), dim3((unsigned)units), dim3(NT), 0, stream, a);
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
