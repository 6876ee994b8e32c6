// kda_linear_tree.hip -- linear attention for a tree of drafted tokens over the
// states, and the commit of its accepted path.
//
// With n_i the nodes from the state S to node i, i included, the state after
// i is a^{n_i} S + sum over j on the path of a^{n_i - n_j} k_j v_j^T, so
//   o_i = scale (a^{n_i} S^T q_i + sum_j a^{n_i - n_j} (q_i . k_j) v_j):
// S is read once for all nodes and no state of a node is ever formed.  Both
// kernels are bound by that one pass over S (and the commit's write).
#include "kda_device.hpp"
#include "kda_linear.hpp"
#include "kda_linear_frag.hpp"

namespace kda {

constexpr int kTree = 64;   // KDA_MAX_TREE_TOKENS: one lane of a wave per node

// The path of node `lane` as a set of nodes (itself included), 0 for an
// absent one: every lane's set starts as {itself} and takes in the set of the
// next node above it, which doubles the covered length of the path; six rounds
// cover 64 nodes.  Called by one whole wave.
__device__ __forceinline__ uint64_t tree_path(const int* __restrict__ parent, int T) {
    const int lane = lane_id();
    const int up = lane < T ? parent[lane] : -2;
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

// Tiles of 16 value columns that a wave holds.  Of 128 columns two: four waves
// form the pair weights and read the keys half as often as eight, and rows of S
// come in whole 128-byte lines (B64 H32 d128 bf16, T64: 50 against 79 us; T16: 33
// against 35; B2 T13: 6.5 both).  Of 64 columns one (B64 T64: 37 against 40 us).
template <int DV> constexpr int tree_tiles() { return DV == 128 ? 2 : 1; }

// One workgroup per (b, h), one wave per NC tiles of value columns.  A wave's
// slab of S is the operand of S^T q straight from its loads; q, k
// and v of the nodes lie in LDS, rows of absent nodes as zeros (they may hold
// anything).  The weights of 32 keys for 16 queries are formed transposed by
// every wave, so that they are the operand of the product with v as they are.
// TN: nodes rounded up to 32 (the LDS taken).  NS: terms of E that the state and
// the pair weights are split into for their products.  bf16 takes two, which
// leaves only the output's own rounding, where the device is not full anyway,
// and one, half a bf16 step on each part of the sum, where it is (B64 H32 T64
// d128: 50 against 58 us; with its commit 94 against 98).  Three waves a SIMD, so three workgroups of 53 KB of
// LDS a CU, where the registers suffice: B64 H32 T64 moves 267 MB in 43 us with
// its inputs cached in part (50 among others).
template <typename E, int DK, int DV, int TN, int NS>
__global__ __launch_bounds__(DV * 4 / tree_tiles<DV>(), DV == 128 && sizeof(E) == 2 && NS == 1 ? 3 : 2) void linear_tree_kernel(LinearTree p) {
    constexpr int NC = tree_tiles<DV>(), NT = DV * 4 / NC, KM = DK / 32, PE = 16 / sizeof(E);
    constexpr int LK = DK + PE, LV = DV + PE;                 // padded LDS rows
    constexpr int PK = TN * DK / PE, PV = TN * DV / PE;       // 16-byte pieces
    constexpr int RK = (PK + NT - 1) / NT, RV = (PV + NT - 1) / NT;
    __shared__ __align__(16) E s_q[TN * LK], s_k[TN * LK], s_v[TN * LV];
    __shared__ __align__(16) float s_n[TN];
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H;
    if (p.S.skip(b)) return;
    const int tid = threadIdx.x, wave = wave_id(), lane = lane_id(), j = lane & 15, g = lane >> 4;
    const int hk = h / (p.H / p.Hk), T = p.T, cbase = wave * NC * 16;

    const float* S = p.S.in + ((size_t)(p.S.in_slot ? p.S.in_slot[b] : b) * p.H + h) * (DK * DV);
    float st[NC][KM][8];                                      // tile ct: columns cbase + NC j + ct
#pragma unroll
    for (int m = 0; m < KM; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float* at = S + (32 * m + 8 * g + i) * DV + cbase + NC * j;
            if constexpr (NC == 2) {
                const f32x2 x = *reinterpret_cast<const f32x2*>(at);
                st[0][m][i] = x[0];
                st[1][m][i] = x[1];
            } else {
                st[0][m][i] = *at;
            }
        }
    const size_t t0 = (size_t)b * T;
    const uint64_t path = tree_path(p.parent + t0, T);        // of node `lane`
    const uint64_t live = __ballot(path != 0);
    {
        u32x4 rq[RK], rk[RK], rv[RV];
        const u32x4 none = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < RK; ++i) {
            const int at = tid + i * NT, row = at / (DK / PE), e = at % (DK / PE) * PE;
            const bool in = at < PK && row < T;
            const size_t off = ((t0 + (in ? row : 0)) * p.Hk + hk) * DK + e;
            rq[i] = *reinterpret_cast<const u32x4*>((const E*)p.q + off);
            rk[i] = *reinterpret_cast<const u32x4*>((const E*)p.k + off);
        }
#pragma unroll
        for (int i = 0; i < RV; ++i) {
            const int at = tid + i * NT, row = at / (DV / PE), e = at % (DV / PE) * PE;
            const bool in = at < PV && row < T;
            rv[i] = *reinterpret_cast<const u32x4*>((const E*)p.v + ((t0 + (in ? row : 0)) * p.H + h) * DV + e);
        }
#pragma unroll
        for (int i = 0; i < RK; ++i) {
            const int at = tid + i * NT, row = at / (DK / PE), e = at % (DK / PE) * PE;
            if (PK % NT == 0 || at < PK) {
                const bool in = live >> row & 1;
                *reinterpret_cast<u32x4*>(&s_q[row * LK + e]) = in ? rq[i] : none;
                *reinterpret_cast<u32x4*>(&s_k[row * LK + e]) = in ? rk[i] : none;
            }
        }
#pragma unroll
        for (int i = 0; i < RV; ++i) {
            const int at = tid + i * NT, row = at / (DV / PE), e = at % (DV / PE) * PE;
            if (PV % NT == 0 || at < PV) {
                const u32x4 v = live >> row & 1 ? rv[i] : none;
                if constexpr (NC == 1) {
                    *reinterpret_cast<u32x4*>(&s_v[row * LV + e]) = v;
                } else {                                      // of 32 columns the even ones, then the odd ones
                    E* dst = &s_v[row * LV + (e & ~31) + (e & 31) / 2];
                    u32x2 even, odd;
                    if constexpr (sizeof(E) == 2) {
                        even = u32x2{(v[0] & 0xffff) | v[1] << 16, (v[2] & 0xffff) | v[3] << 16};
                        odd = u32x2{v[0] >> 16 | (v[1] & 0xffff0000), v[2] >> 16 | (v[3] & 0xffff0000)};
                    } else {
                        even = u32x2{v[0], v[2]};
                        odd = u32x2{v[1], v[3]};
                    }
                    *reinterpret_cast<u32x2*>(dst) = even;
                    *reinterpret_cast<u32x2*>(dst + 16) = odd;
                }
            }
        }
    }
    if (wave == 0 && lane < TN) s_n[lane] = (float)__popcll(path);
    __syncthreads();

    const float lg = log_decay(p.g[h]);
    Frag<E> sf[NC][KM][NS];
#pragma unroll
    for (int ct = 0; ct < NC; ++ct)
#pragma unroll
        for (int m = 0; m < KM; ++m) {
            const float* x = st[ct][m];
            split(f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]}, sf[ct][m]);
        }
    for (int qt = 0; qt * 16 < T; ++qt) {                     // 16 queries: lane j has query 16 qt + j
        const int q = 16 * qt + j;
        const float nq = s_n[q];
        const uint32_t path_lo = __shfl((uint32_t)path, q), path_hi = __shfl((uint32_t)(path >> 32), q);
        Frag<E> x[KM];
        f32x4 o[NC];
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) o[ct] = zero4();
#pragma unroll
        for (int m = 0; m < KM; ++m) {
            x[m] = row_frag<E>(&s_q[q * LK + 32 * m + 8 * g]);
#pragma unroll
            for (int ct = 0; ct < NC; ++ct)
#pragma unroll
                for (int s = 0; s < NS; ++s) o[ct] = mma(sf[ct][m][s], x[m], o[ct]);
        }
#pragma unroll
        for (int ct = 0; ct < NC; ++ct) o[ct] *= p.scale * expf(lg * nq);
#pragma unroll
        for (int kb = 0; kb < TN / 32; ++kb) {                // 32 keys
            if (2 * kb > qt) break;
            const uint32_t bits = kb ? path_hi : path_lo;
            f32x4 w[2];
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                w[kt] = zero4();
                if (2 * kb + kt > qt) continue;               // keys behind the queries
#pragma unroll
                for (int m = 0; m < KM; ++m)
                    w[kt] = mma(row_frag<E>(&s_k[(32 * kb + 16 * kt + j) * LK + 32 * m + 8 * g]), x[m], w[kt]);
                const f32x4 nk = *reinterpret_cast<const f32x4*>(&s_n[32 * kb + 16 * kt + 4 * g]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[kt][i] = bits >> (16 * kt + 4 * g + i) & 1 ? w[kt][i] * (p.scale * expf(lg * (nq - nk[i]))) : 0.f;
            }
            Frag<E> wf[NS];
            split(w[0], w[1], wf);
#pragma unroll
            for (int ct = 0; ct < NC; ++ct) {
                const Frag<E> vf = col_frag<E>(&s_v[32 * kb * LV], LV, cbase + 16 * ct, 4, j, g);
#pragma unroll
                for (int s = 0; s < NS; ++s) o[ct] = mma(vf, wf[s], o[ct]);
            }
        }
        if (q < T) {
            float y[4 * NC];                                  // columns in order
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int ct = 0; ct < NC; ++ct) y[NC * i + ct] = nq == 0.f ? 0.f : o[ct][i];
            E* dst = (E*)p.o + ((t0 + q) * p.H + h) * DV + cbase + 4 * NC * g;
            if constexpr (sizeof(E) == 2 && NC == 2) {
                *reinterpret_cast<bf16x8*>(dst) = pack8(f32x4{y[0], y[1], y[2], y[3]}, f32x4{y[4], y[5], y[6], y[7]});
            } else {
#pragma unroll
                for (int i = 0; i < 4 * NC; i += 4) {
                    const f32x4 part = {y[i], y[i + 1], y[i + 2], y[i + 3]};
                    if constexpr (sizeof(E) == 2)
                        *reinterpret_cast<bf16x4*>(dst + i) = pack4(part);
                    else
                        *reinterpret_cast<f32x4*>(dst + i) = part;
                }
            }
        }
    }
}

// One workgroup per (b, h); a thread holds 4 columns of RPT rows of S, read
// before the path is known.  The path's k (weighted) and v pass through LDS in
// blocks of kPathBlock nodes.
constexpr int kPathBlock = 16;
template <typename E, int DK, int DV>
__global__ __launch_bounds__(DK * DV / 32 < 64 ? 64 : DK * DV / 32) void linear_commit_kernel(LinearTree p) {
    constexpr int NT = DK * DV / 32 < 64 ? 64 : DK * DV / 32;
    constexpr int CG = DV / 4, RG = NT / CG, RPT = DK / RG;
    __shared__ __align__(16) float s_k[kPathBlock][DK], s_v[kPathBlock][DV];
    __shared__ int s_node[kTree];                             // the path's nodes in order
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H, tid = threadIdx.x;
    if (p.S.skip(b)) return;
    const int cg = tid % CG, rg = tid / CG, hk = h / (p.H / p.Hk), x = p.accepted[b];
    if (x < -1 || x >= p.T) return;
    const f32x4* S = (const f32x4*)(p.S.in + ((size_t)(p.S.in_slot ? p.S.in_slot[b] : b) * p.H + h) * (DK * DV));
    f32x4* So = (f32x4*)(p.S.out + ((size_t)(p.S.out_slot ? p.S.out_slot[b] : b) * p.H + h) * (DK * DV));
    f32x4 st[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) st[i] = __builtin_nontemporal_load(&S[(rg + RG * i) * CG + cg]);
    // every wave finds the path by itself
    const size_t t0 = (size_t)b * p.T;
    const uint64_t all = tree_path(p.parent + t0, p.T);
    const int from = x < 0 ? 0 : x;
    const uint64_t found = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(all >> 32), from) << 32) |
                    (uint32_t)__builtin_amdgcn_readlane((int)all, from);
    const uint64_t path = x < 0 ? 0 : found;
    if (x >= 0 && path == 0) return;                          // absent (uniform over the workgroup)
    const int n = __popcll(path);
    const float lg = log_decay(p.g[h]);
    if (n > 0) {
        const float an = expf(lg * (float)n);
#pragma unroll
        for (int i = 0; i < RPT; ++i) st[i] *= an;
    }
    const int me = lane_id();
    if (wave_id() == 0 && (path >> me & 1)) s_node[__popcll(path & ((1ull << me) - 1))] = me;
    constexpr int PE = 16 / sizeof(E), PR = (DK + DV) / PE;   // 16-byte pieces of a node's k and v
    for (int n0 = 0; n0 < n; n0 += kPathBlock) {
        const int nb = min(kPathBlock, n - n0);
        __syncthreads();
        for (int at = tid; at < nb * PR; at += NT) {
            const int s = at / PR, e = at % PR * PE, node = s_node[n0 + s];
            const bool isk = e < DK;
            const E* src = isk ? (const E*)p.k + ((t0 + node) * p.Hk + hk) * DK + e
                               : (const E*)p.v + ((t0 + node) * p.H + h) * DV + e - DK;
            float* dst = isk ? &s_k[s][e] : &s_v[s][e - DK];
            const float w = isk ? expf(lg * (float)(n - 1 - n0 - s)) : 1.0f;
            E x[PE];
            *reinterpret_cast<u32x4*>(x) = *reinterpret_cast<const u32x4*>(src);
#pragma unroll
            for (int i = 0; i < PE; ++i) dst[i] = w * to_f32(x[i]);
        }
        __syncthreads();
        for (int s = 0; s < nb; ++s) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(&s_v[s][4 * cg]);
#pragma unroll
            for (int i = 0; i < RPT; ++i) st[i] += s_k[s][rg + RG * i] * v;
        }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) __builtin_nontemporal_store(st[i], &So[(rg + RG * i) * CG + cg]);
}

template <typename E, int DK, int DV, int NS>
static void launch_tree(const LinearTree& a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * a.H)), block(DV * 4 / tree_tiles<DV>());
    if (a.T <= 32)
        hipLaunchKernelGGL((linear_tree_kernel<E, DK, DV, 32, NS>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((linear_tree_kernel<E, DK, DV, 64, NS>), grid, block, 0, stream, a);
}

template <typename E, int DK, int DV>
static hipError_t launch_kv(const LinearTree& a, bool commit, hipStream_t stream) {
    constexpr int NT = DK * DV / 32 < 64 ? 64 : DK * DV / 32;
    const dim3 grid((unsigned)(a.B * a.H));
    if (commit)
        hipLaunchKernelGGL((linear_commit_kernel<E, DK, DV>), grid, dim3(NT), 0, stream, a);
    else if (sizeof(E) == 2 && grid.x < 512)
        launch_tree<E, DK, DV, sizeof(E) == 2 ? 2 : 1>(a, stream);
    else
        launch_tree<E, DK, DV, 1>(a, stream);
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
