// kda_linear_tree.hip -- linear attention for a tree of drafted tokens over the
// states, and the commit of its accepted path.
//
// With n_i the nodes from the state S to node i, i included, the state after
// i is a^{n_i} S + sum over j on the path of a^{n_i - n_j} k_j v_j^T, so
//   o_i = scale (a^{n_i} S^T q_i + sum_j a^{n_i - n_j} (q_i . k_j) v_j):
// S is read once for all nodes and no state of a node is ever formed.
#include "kda_device.hpp"
#include "kda_linear.hpp"

namespace kda {

constexpr int kTree = 64;   // KDA_MAX_TREE_TOKENS: one lane of a wave per node

// The path of node `lane` as a set of nodes (itself included), 0 for an
// absent one: every lane's set starts as {itself} and takes in the set of the
// next node above it, which doubles the covered length of the path; six rounds
// cover 64 nodes.  Called by one whole wave.
__device__ __forceinline__ uint64_t tree_path(const int* __restrict__ parent, int T) {
    const int lane = lane_id();
    int up = lane < T ? parent[lane] : -2;
    bool bad = up < -1 || up >= lane;         // absent: no earlier node
    uint64_t set = 1ull << lane;
    int top = bad ? -1 : up;                  // the next node above the set (-1: S)
#pragma unroll
    for (int r = 0; r < 6; ++r) {
        const int from = top < 0 ? lane : top;
        const uint32_t lo = __shfl((uint32_t)set, from), hi = __shfl((uint32_t)(set >> 32), from);
        const int next = __shfl(top, from);
        const int above_bad = __shfl((int)bad, from);
        if (top >= 0) {
            set |= ((uint64_t)hi << 32) | lo;
            bad = bad || above_bad;
            top = next;
        }
    }
    return bad ? 0 : set;
}

// One workgroup per (b, h), a thread per value column; node by node.
template <typename E, int DK, int DV>
__global__ __launch_bounds__(DV < 64 ? 64 : DV) void linear_tree_kernel(LinearTree p) {
    constexpr int NT = DV < 64 ? 64 : DV;
    __shared__ uint64_t s_path[kTree];
    __shared__ float s_q[DK], s_w[kTree];
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H, c = threadIdx.x;
    if (p.S.skip(b)) return;
    const int hk = h / (p.H / p.Hk);
    const float g = log_decay(p.g[h]);
    if (c < kWave) s_path[c] = tree_path(p.parent + (size_t)b * p.T, p.T);
    const float* S = p.S.in + ((size_t)(p.S.in_slot ? p.S.in_slot[b] : b) * p.H + h) * DK * DV;
    for (int i = 0; i < p.T; ++i) {
        const size_t tok = (size_t)b * p.T + i;
        __syncthreads();
        for (int e = c; e < DK; e += NT) s_q[e] = to_f32(((const E*)p.q)[(tok * p.Hk + hk) * DK + e]);
        __syncthreads();
        const uint64_t path = s_path[i];
        if (c < kTree) {
            float w = 0.f;
            if (path >> c & 1) {
                for (int e = 0; e < DK; ++e)
                    w += s_q[e] * to_f32(((const E*)p.k)[(((size_t)b * p.T + c) * p.Hk + hk) * DK + e]);
                w *= expf(g * (float)(__popcll(path) - __popcll(s_path[c])));
            }
            s_w[c] = w;
        }
        __syncthreads();
        if (c >= DV) continue;
        float o = 0.f;
        if (path) {
            for (int e = 0; e < DK; ++e) o += s_q[e] * S[e * DV + c];
            o *= expf(g * (float)__popcll(path));
            for (int j = 0; j <= i; ++j)
                if (path >> j & 1)
                    o += s_w[j] * to_f32(((const E*)p.v)[(((size_t)b * p.T + j) * p.H + h) * DV + c]);
        }
        ((E*)p.o)[(tok * p.H + h) * DV + c] = from_f32<E>(p.scale * o);
    }
}

template <typename E, int DK, int DV>
__global__ __launch_bounds__(256) void linear_commit_kernel(LinearTree p) {
    constexpr int CG = DV / 4, RG = 256 / CG;
    __shared__ uint64_t s_path[kTree];
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H, tid = threadIdx.x;
    if (p.S.skip(b)) return;
    const int x = p.accepted[b];
    if (x < -1 || x >= p.T) return;
    const int hk = h / (p.H / p.Hk);
    const float g = log_decay(p.g[h]);
    if (tid < kWave) s_path[tid] = tree_path(p.parent + (size_t)b * p.T, p.T);
    __syncthreads();
    const uint64_t path = x < 0 ? 0 : s_path[x];
    if (x >= 0 && path == 0) return;
    const int n = __popcll(path), cg = tid % CG, rg = tid / CG;
    const f32x4* S = (const f32x4*)(p.S.in + ((size_t)(p.S.in_slot ? p.S.in_slot[b] : b) * p.H + h) * DK * DV);
    f32x4* So = (f32x4*)(p.S.out + ((size_t)(p.S.out_slot ? p.S.out_slot[b] : b) * p.H + h) * DK * DV);
    const float an = expf(g * (float)n);
    for (int c = rg; c < DK; c += RG) {
        f32x4 s = S[c * CG + cg];
        if (n) s *= an;
        for (uint64_t rest = path; rest; rest &= rest - 1) {
            const int j = __ffsll((unsigned long long)rest) - 1;
            const size_t tok = (size_t)b * p.T + j;
            const float kj = to_f32(((const E*)p.k)[(tok * p.Hk + hk) * DK + c]) *
                             expf(g * (float)(n - __popcll(s_path[j])));
            for (int e = 0; e < 4; ++e)
                s[e] += kj * to_f32(((const E*)p.v)[(tok * p.H + h) * DV + 4 * cg + e]);
        }
        So[c * CG + cg] = s;
    }
}

template <typename E, int DK, int DV>
static hipError_t launch_kv(const LinearTree& a, bool commit, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * a.H));
    if (commit)
        hipLaunchKernelGGL((linear_commit_kernel<E, DK, DV>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((linear_tree_kernel<E, DK, DV>), grid, dim3(DV < 64 ? 64 : DV), 0, stream, a);
    return hipGetLastError();
}

template <typename E, int DK>
static hipError_t launch_k(const LinearTree& a, bool commit, hipStream_t stream) {
    switch (a.dv) {
        case 32: return launch_kv<E, DK, 32>(a, commit, stream);
        case 64: return launch_kv<E, DK, 64>(a, commit, stream);
        default: return launch_kv<E, DK, 128>(a, commit, stream);
    }
}

template <typename E>
static hipError_t launch_e(const LinearTree& a, bool commit, hipStream_t stream) {
    switch (a.dk) {
        case 32: return launch_k<E, 32>(a, commit, stream);
        case 64: return launch_k<E, 64>(a, commit, stream);
        default: return launch_k<E, 128>(a, commit, stream);
    }
}

hipError_t launch_linear_tree(const LinearTree& a, hipStream_t stream) {
    return a.is_bf16 ? launch_e<bf16>(a, false, stream) : launch_e<float>(a, false, stream);
}

hipError_t launch_linear_commit(const LinearTree& a, hipStream_t stream) {
    return a.is_bf16 ? launch_e<bf16>(a, true, stream) : launch_e<float>(a, true, stream);
}

}  // namespace kda
