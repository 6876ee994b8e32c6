// kda_delta.hip -- the gated delta rule over a sequence in chunk form
// (kda_delta_chunk.hpp): the chain of states over the chunks.
#include <algorithm>

#include "kda_delta_chain.hpp"

namespace kda {

template <typename E, int DK>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 2 : 1) void delta_chain_kernel(DeltaChain p) {
    __shared__ ChainLds<E, DK, false> s;
    delta_chain<E, DK, false>(p, blockIdx.x, s);
}

// Chunks whose blocks the workspace holds at a time: longer sequences run window
// by window, the state carried in the workspace.  Half as much, which the last-level
// cache holds, costs more in launches than it saves, and twice as much saves no more
// than 3 %: H32 d128 bf16, 192 / 384 / 768 MiB, B4 T4096 505 / 490 / 489 us, B8 T8192
// 1,367 / 1,340 / 1,303, B1 T32768 1,215 / 1,192 / 1,174.  At least eight chunks: 2 GiB
// for 8,192 heads.
constexpr size_t kDeltaWindowBytes = (size_t)384 << 20;

// From so many heads of bf16 rows on a workgroup takes a whole one
// (delta_wide_kernel), where fewer leave more than half of the device idle.  Wide
// against eight workgroups of 16 columns, d_v 128, d_k 128 / 64 / 32, us: T 4096, 64
// heads 425 / 293 / 251 and 285 / 201 / 179, 96 heads 459 / 324 / 288 and 435 / 342 /
// 295, 128 heads 488 / 346 / 313 and 569 / 455 / 403, 256 heads 671 / 502 / 435 and
// 1,139 / 891 / 768; T 512, 128 heads 66 / 51 / 46 and 69 / 56 / 50; T 100, 128 heads
// 32 / 26 / 23 and 34 / 28 / 25.  Fewer value columns would leave a workgroup two or
// four waves, and fp32's three terms of K and Q need twice the LDS there is.
constexpr int kWideUnits = 128;

struct DeltaWindows {
    int chunks, len, n;      // chunks of a sequence, of a window, windows
    size_t blocks, carry;    // bytes
};
static DeltaWindows windows(int B, int T, int H, int dk, int dv, bool is_bf16) {
    const size_t units = (size_t)B * H, blk = delta_block_bytes(is_bf16, false);
    DeltaWindows w;
    w.chunks = (T + kDeltaChunk - 1) / kDeltaChunk;
    w.len = (int)std::min<size_t>(w.chunks, std::max<size_t>(8, kDeltaWindowBytes / (units * blk)));
    w.n = (w.chunks + w.len - 1) / w.len;
    w.len = (w.chunks + w.n - 1) / w.n;
    w.blocks = (units * w.len * blk + 255) / 256 * 256;
    w.carry = w.n > 1 ? units * dk * dv * sizeof(float) : 0;
    return w;
}

size_t delta_prefill_ws_bytes(int B, int T, int H, int dk, int dv, bool is_bf16) {
    const DeltaWindows w = windows(B, T, H, dk, dv, is_bf16);
    return w.blocks + w.carry;
}

template <typename E>
static hipError_t launch_chain(const DeltaChain& a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.B * a.H * (a.dv / 16)));
    switch (a.dk) {
        case 32: hipLaunchKernelGGL((delta_chain_kernel<E, 32>), grid, dim3(256), 0, stream, a); break;
        case 64: hipLaunchKernelGGL((delta_chain_kernel<E, 64>), grid, dim3(256), 0, stream, a); break;
        default: hipLaunchKernelGGL((delta_chain_kernel<E, 128>), grid, dim3(256), 0, stream, a); break;
    }
    return hipGetLastError();
}

hipError_t launch_delta_prefill(const DeltaPrefill& a, void* ws, hipStream_t stream) {
    const DeltaWindows w = windows(a.B, a.T, a.H, a.dk, a.dv, a.is_bf16);
    const bool wide = a.is_bf16 && a.dv == 128 && a.B * a.H >= kWideUnits;
    char* blocks = (char*)ws;
    float* carry = w.n > 1 ? (float*)(blocks + w.blocks) : nullptr;
    for (int i = 0; i < w.n; ++i) {
        const int c0 = i * w.len, c1 = std::min(w.chunks, c0 + w.len);
        StateIO S = a.S;
        if (i > 0) S.in = carry, S.in_slot = nullptr;
        if (i + 1 < w.n) S.out = carry, S.out_slot = nullptr;
        hipError_t e = launch_delta_pairs({a.q, a.k, a.g, a.beta, a.scale, S, a.lens, blocks, a.B, a.T, a.H, a.Hk, a.dk, c0, c1,
                                           a.is_bf16}, false, stream);
        if (e != hipSuccess) return e;
        const DeltaChain c{a.q, a.k, a.v, a.scale, S, a.lens, blocks, a.o, a.B, a.T, a.H, a.Hk, a.dk, a.dv, c0, c1, a.is_bf16, {}};
        e = wide ? launch_delta_wide(c, stream) : a.is_bf16 ? launch_chain<bf16>(c, stream) : launch_chain<float>(c, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace kda
