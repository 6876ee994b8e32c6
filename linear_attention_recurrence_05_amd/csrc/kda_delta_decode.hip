// kda_delta_decode.hip -- one token of the gated delta rule, the state updated
// in place.  With S' = a S (a = exp(g)):
//   p = S'^T k,  r = S'^T q,  e = beta (v - p),
//   S <- S' + k e^T,   o = scale (r + (q . k) e)      (= scale S^T q)
//
// Bound by the one read and one write of S (8 d_k d_v bytes against 7 d_k d_v
// flops).  A workgroup holds one (b, h), each thread four columns of up to eight
// rows: all loads of S are in flight before the first is used, both reductions
// come from the same read (within the wave, then through LDS, in fixed order),
// and the state is written from registers.
#include "kda_delta.hpp"
#include "kda_device.hpp"

namespace kda {

template <int DK, int DV>
constexpr int delta_threads() { return DK * DV / 32 < 64 ? 64 : DK * DV / 32; }

template <typename E, int DK, int DV>
__global__ __launch_bounds__((delta_threads<DK, DV>())) void delta_decode_kernel(DeltaDecode p) {
    constexpr int NT = delta_threads<DK, DV>(), NWAVE = NT / kWave;
    constexpr int CG = DV / 4, RG = NT / CG, RPT = DK / RG;
    static_assert(DK % RG == 0 && CG <= kWave, "layout");
    __shared__ float s_q[DK], s_k[DK];
    __shared__ __align__(16) float s_v[DV];
    __shared__ f32x4 s_p[NWAVE][CG], s_r[NWAVE][CG];
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
    const float a = expf(log_decay(p.g[blockIdx.x])), beta = p.beta[blockIdx.x];
    __syncthreads();
    f32x4 pk = zero4(), rq = zero4();
    float qk_dot = 0.f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int c = rg + RG * i;
        const float kc = s_k[c], qc = s_q[c];
        st[i] *= a;
        pk += kc * st[i];
        rq += qc * st[i];
        qk_dot += qc * kc;                                   // this thread's rows
    }
#pragma unroll
    for (int off = CG; off < kWave; off <<= 1) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            pk[x] += __shfl_xor(pk[x], off);
            rq[x] += __shfl_xor(rq[x], off);
        }
        qk_dot += __shfl_xor(qk_dot, off);
    }
    __shared__ float s_d[NWAVE];
    if (lane < CG) {
        s_p[wave][lane] = pk;
        s_r[wave][lane] = rq;
    }
    if (lane == 0) s_d[wave] = qk_dot;
    __syncthreads();
    pk = s_p[0][cg];
#pragma unroll
    for (int w = 1; w < NWAVE; ++w) pk += s_p[w][cg];
    const f32x4 e = beta * (*reinterpret_cast<const f32x4*>(&s_v[4 * cg]) - pk);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int c = rg + RG * i;
        __builtin_nontemporal_store(st[i] + s_k[c] * e, &S[c * CG + cg]);
    }
    if (rg == 0) {
        f32x4 o = s_r[0][cg];
        float d = s_d[0];
#pragma unroll
        for (int w = 1; w < NWAVE; ++w) {
            o += s_r[w][cg];
            d += s_d[w];
        }
        o = p.scale * (o + d * e);
        E* dst = (E*)p.o + vo + 4 * cg;
        if constexpr (sizeof(E) == 2)
            *reinterpret_cast<bf16x4*>(dst) = pack4(o);
        else
            *reinterpret_cast<f32x4*>(dst) = o;
    }
}

template <typename E, int DK, int DV>
static hipError_t launch_kv(const DeltaDecode& a, hipStream_t stream) {
    hipLaunchKernelGGL((delta_decode_kernel<E, DK, DV>), dim3((unsigned)(a.B * a.H)), dim3(delta_threads<DK, DV>()), 0,
                       stream, a);
    return hipGetLastError();
}

template <typename E, int DK>
static hipError_t launch_k(const DeltaDecode& a, hipStream_t stream) {
    switch (a.dv) {
        case 32: return launch_kv<E, DK, 32>(a, stream);
        case 64: return launch_kv<E, DK, 64>(a, stream);
        default: return launch_kv<E, DK, 128>(a, stream);
    }
}

template <typename E>
static hipError_t launch_e(const DeltaDecode& a, hipStream_t stream) {
    switch (a.dk) {
        case 32: return launch_k<E, 32>(a, stream);
        case 64: return launch_k<E, 64>(a, stream);
        default: return launch_k<E, 128>(a, stream);
    }
}

hipError_t launch_delta_decode(const DeltaDecode& a, hipStream_t stream) {
    return a.is_bf16 ? launch_e<bf16>(a, stream) : launch_e<float>(a, stream);
}

}  // namespace kda
