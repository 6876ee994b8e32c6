// kda_delta.hpp -- launchers of the gated delta rule with a decay and a write
// strength for each token and head, and of the norms around it, shared between
// their C ABI (kda_delta_api.hip) and the kernel files.  Arguments reaching
// these functions have been validated by the ABI layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "kda_linear.hpp"

namespace kda {

// Most sequences x heads of a delta-rule call: eight workgroups of up to 512
// threads each, and a launch holds fewer than 2^32 threads.
constexpr long long kDeltaMaxUnits = 1LL << 19;

struct DeltaPrefill {
    const void *q, *k, *v;
    const float *g, *beta;
    float scale;
    StateIO S;
    const int* lens;
    void* o;
    int B, T, H, Hk, dk, dv;
    bool is_bf16;
};
size_t delta_prefill_ws_bytes(int B, int T, int H, int dk, int dv, bool is_bf16);
hipError_t launch_delta_prefill(const DeltaPrefill& a, void* ws, hipStream_t stream);

struct DeltaBackward {
    const void *q, *k, *v;
    const float *g, *beta;
    float scale;
    const float* S0;
    const int* lens;
    const void* dO;
    const float* dST;
    void *dq, *dk, *dv;
    float *dg, *dbeta, *dS0;
    int B, T, H, Hk, dk_, dv_;
    bool is_bf16;
};
size_t delta_backward_ws_bytes(int B, int T, int H, int Hk, int dk, int dv, bool is_bf16);
hipError_t launch_delta_backward(const DeltaBackward& a, void* ws, hipStream_t stream);

struct DeltaDecode {
    const void *q, *k, *v;
    const float *g, *beta;
    float scale;
    StateIO S;   // in place
    void* o;
    int B, H, Hk, dk, dv;
    bool is_bf16;
};
hipError_t launch_delta_decode(const DeltaDecode& a, hipStream_t stream);

// y = act(z) w x (mean(x^2) + eps)^{-1/2} over rows of d elements, and its
// gradients (dy set; y is dx).
struct GatedNorm {
    const void *x, *z;
    const float* w;
    bool silu;
    float eps;
    const void* dy;
    void *y, *dz;
    float* dw;
    long long rows;
    int d;
    bool is_bf16;
};
hipError_t launch_gated_norm(const GatedNorm& a, hipStream_t stream);
size_t gated_norm_backward_ws_bytes(long long rows, int d);
hipError_t launch_gated_norm_backward(const GatedNorm& a, void* ws, hipStream_t stream);

// u = scale sigmoid(z) w_y (y or its norm), h = r + u, n = w_n norm(h) over
// rows of D elements; gradients with h the stored sum (dn set).
struct BlockNorm {
    const void *y, *z;
    const float* w_y;
    const void* r;
    const float* w_n;
    bool norm_y;
    float scale, eps;
    void *h, *n;                       // forward outputs (h may be null without y)
    const void *h_in, *dn, *dh;        // backward
    void *dr, *dy, *dz;
    float *dw_y, *dw_n;
    long long rows;
    int D;
    bool is_bf16;
};
hipError_t launch_block_norm(const BlockNorm& a, hipStream_t stream);
size_t block_norm_backward_ws_bytes(long long rows, int D, bool is_bf16);
hipError_t launch_block_norm_backward(const BlockNorm& a, void* ws, hipStream_t stream);

}  // namespace kda
