// kda_delta_chain.hpp -- the state's chain over the chunks of the gated delta rule
// (kda_delta_chunk.hpp) for 16 value columns of one head: the prefill, or the
// gradients' forward sweep.
#pragma once

#include "kda_delta_chunk.hpp"

namespace kda {

// Chunks from one anchor <S, Y> of dg (kda_delta_backward.hip) to the next.
constexpr int kAnchorChunks = 4;

// What the gradients' sweeps leave in the workspace, for unit u = b H + h, chunk
// c of NC, anchor a of NA, column tile t of `tiles`:
//   e     [u][c][dv][64] fp32        e_t of every token
//   S, Y  [u][c][dv][dk] of E        the state before a chunk, and the gradient of
//                                    the one behind it, transposed
//   end   [u][a][t] state tiles      the state at an anchor, as the chain holds it
//   anchor[u][a][t][DK / 32] fp32    parts of <S, Y>
//   dot   [2][t][u][64 NC] fp32      parts of dO . o - dv . v, and of dbeta
struct DeltaSweep {
    const void* dO;
    float* e;
    void *S, *Y;
    float *end, *anchor, *dot;
    int NC, NA;
};

// Chunks c0 .. c1 - 1 from the state S.in to S.out.
struct DeltaChain {
    const void *q, *k, *v;
    float scale;
    StateIO S;
    const int* lens;
    const char* blocks;     // of chunks c0 .. c1 - 1
    void* o;
    int B, T, H, Hk, dk, dv, c0, c1;
    bool is_bf16;
    DeltaSweep sweep;       // of the gradients' forward sweep, which leaves no o
};
hipError_t launch_delta_sweep(const DeltaChain& a, hipStream_t stream);
// The prefill's chain by one workgroup per (b, h): bf16, dv = 128.
hipError_t launch_delta_wide(const DeltaChain& a, hipStream_t stream);

}  // namespace kda
