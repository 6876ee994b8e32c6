// kda_linear.hpp -- launchers of the linear-attention, tree and norm kernels,
// shared between their C ABI (kda_linear_api.hip) and the kernel files.
// Arguments reaching these functions have been validated by the ABI layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>

#include "kda_launch.hpp"

namespace kda {

// Log-decays below this are taken as this: exp of it, and of any multiple, is
// exactly 0 in fp32, and 0 times it is 0 (0 times -infinity would be NaN).
constexpr float kMinLogDecay = -1e4f;
__device__ __forceinline__ float log_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }   // NaN stays

// One tensor [B, T, n, d] that the H heads of a pass read or write; head h of
// the pass uses head h / (H / n).
struct HeadTensor {
    const void* p;
    int n;
};

// One pass of the recurrence over every sequence, from which the forward and
// each gradient are made.  Tokens t = 0 .. n - 1 (forward) or n - 1 .. 0
// (reverse), n = lens[b] or T, state M [da, db]:
//   forward:  M <- a M + su y_t u_t^T,  out_t = so M^T x_t
//   reverse:  M <- M + su y_t u_t^T,    out_t = so M^T x_t,  M <- a M
// x, y have rows of da elements, u and out of db.  M starts from the state
// `S.in` (null: zero), read transposed if in_t, and ends in `S.out`.
// out is of the inputs' element type, or fp32 if out_f32.
struct LinearPass {
    HeadTensor x, y, u;
    void* out;
    int n_out;
    bool out_f32;
    const float* g;
    float so, su;
    StateIO S;
    bool in_t;
    const int* lens;
    bool reverse;
    int B, T, H, da, db;
    bool is_bf16;
};

struct LinearBackward {
    const void *q, *k, *v;
    const float* g;
    float scale;
    const float* S0;
    const int* lens;
    const void* dO;
    const float* dST;
    void *dq, *dk, *dv;
    float* dS0;
    int B, T, H, Hk, dk_, dv_;
    bool is_bf16;
};

size_t linear_prefill_ws_bytes(int B, int T, int H, int da, int db, bool is_bf16);
hipError_t launch_linear_prefill(const LinearPass& p, void* ws, hipStream_t stream);
size_t linear_backward_ws_bytes(int B, int T, int H, int Hk, int dk, int dv, bool is_bf16);
hipError_t launch_linear_backward(const LinearBackward& a, void* ws, hipStream_t stream);

struct LinearDecode {
    const void *q, *k, *v;
    const float* g;
    float scale;
    StateIO S;   // in place
    void* o;
    int B, H, Hk, dk, dv;
    bool is_bf16;
};
hipError_t launch_linear_decode(const LinearDecode& a, hipStream_t stream);

// The tree's outputs (q, o set) or the commit of its accepted path (q, o
// null; S.out and accepted set).
struct LinearTree {
    const void *q, *k, *v;
    const float* g;
    float scale;
    StateIO S;
    const int *parent, *accepted;
    void* o;
    int B, T, H, Hk, dk, dv;
    bool is_bf16;
};
hipError_t launch_linear_tree(const LinearTree& a, hipStream_t stream);
hipError_t launch_linear_commit(const LinearTree& a, hipStream_t stream);

struct NormRope {
    const void *q, *k;
    const float *w_q, *w_k;
    const int* positions;
    const float* inv_freq;
    bool rms;
    float eps;
    int rot;
    bool interleaved;
    const void *dy_q, *dy_k;   // backward
    void *y_q, *y_k;           // outputs (backward: dq, dk)
    float *dw_q, *dw_k;        // backward, may be null
    int B, T, H, Hk, d;
    bool is_bf16;
};
hipError_t launch_norm_rope(const NormRope& a, hipStream_t stream);
size_t norm_rope_backward_ws_bytes(int B, int T, int H, int Hk, int d);
hipError_t launch_norm_rope_backward(const NormRope& a, void* ws, hipStream_t stream);

}  // namespace kda
