// kda_delta_chain.hpp -- the state's chain over the chunks of the gated delta rule
// (kda_delta_chunk.hpp) for 16 value columns of one head: the prefill, or the
// gradients' forward sweep.
#pragma once

#include "kda_delta_chunk.hpp"

namespace kda {

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
};

}  // namespace kda
