// kda_call.hpp -- the argument checks that the linear-attention, delta-rule and
// norm entry points share: sizes, element types, pools, and the pointers of a
// call with what may overlap.  All on the host, before any HIP call.
#pragma once

#include <cmath>
#include <cstring>

#include "kda_host.hpp"
#include "kda_launch.hpp"

namespace kda {
namespace host {

inline bool head_size_ok(int d) { return d == 32 || d == 64 || d == 128; }

inline kda_status check_dtype(kda_dtype dt) {
    if (dt != KDA_F32 && dt != KDA_BF16) return fail(KDA_ERR_UNSUPPORTED, "dtype %d is not KDA_F32 or KDA_BF16", (int)dt);
    return KDA_OK;
}

// Most (b, h) of a linear-attention call: one workgroup of up to 512 threads
// each, in the gradients three of up to 256 (so many are never split into
// segments), and a launch holds fewer than 2^32 threads.
constexpr long long kMaxUnits = 1LL << 22;

// Sizes of a linear-attention call, in elements.
struct Sizes {
    size_t qk, vo, state, tok;   // q or k; v or o; all states; tokens B * T
};

inline kda_status check_sizes(int B, int T, int H, int H_k, int d_k, int d_v, kda_dtype dt, float scale,
                       Sizes& n) {
    kda_status s = check_dtype(dt);
    if (s != KDA_OK) return s;
    if (!head_size_ok(d_k) || !head_size_ok(d_v))
        return fail(KDA_ERR_UNSUPPORTED, "(d_k, d_v) = (%d, %d); supported: 32, 64 and 128 each", d_k, d_v);
    if (!std::isfinite(scale)) return fail(KDA_ERR_INVALID_VALUE, "scale = %g is not finite", (double)scale);
    size_t nel, ntok;
    if ((s = check_shape(B, T, H, d_k > d_v ? d_k : d_v, nel, ntok)) != KDA_OK) return s;
    if ((long long)B * H > kMaxUnits)
        return fail(KDA_ERR_INVALID_SHAPE, "B*H = %lld is too large (limit 2^22)", (long long)B * H);
    if (H_k < 1 || H_k > H || H % H_k != 0)
        return fail(KDA_ERR_INVALID_SHAPE, "H_k=%d must divide H=%d", H_k, H);
    n.tok = (size_t)B * T;
    n.qk = n.tok * H_k * d_k;
    n.vo = n.tok * H * d_v;
    n.state = (size_t)B * H * d_k * d_v;
    return KDA_OK;
}

inline kda_status check_pool(int n_slots, int H) {
    if (n_slots < 1) return fail(KDA_ERR_INVALID_SHAPE, "n_slots=%d must be >= 1", n_slots);
    if ((long long)n_slots * H > (1LL << 26))
        return fail(KDA_ERR_INVALID_SHAPE, "n_slots*H = %lld is too large", (long long)n_slots * H);
    return KDA_OK;
}

// One pointer of a call.  Outputs (and the workspace) may overlap no other
// range, but for the one input that an output may equal exactly (in place):
// another input given the same address would be overwritten before it is read.
struct Ptr {
    const char* name;
    const void* p;
    size_t bytes;
    unsigned align;
    bool required;
    bool output;
    const char* same;   // the name of the input this output may equal exactly (null: none)
};

inline kda_status check_call(const Ptr* r, int n) {
    for (int i = 0; i < n; ++i) {
        if (!r[i].p) {
            if (r[i].required) return fail(KDA_ERR_NULL_POINTER, "%s is NULL", r[i].name);
            continue;
        }
        if (!aligned(r[i].p, r[i].align))
            return fail(KDA_ERR_MISALIGNED, "%s is not %u-byte aligned", r[i].name, r[i].align);
    }
    for (int out = 0; out < n; ++out) {
        if (!r[out].output) continue;
        for (int i = 0; i < n; ++i) {
            if (i == out || (r[out].same && r[i].p == r[out].p && !std::strcmp(r[i].name, r[out].same))) continue;
            if (overlap(Range{r[out].name, r[out].p, r[out].bytes, 1},
                        Range{r[i].name, r[i].p, r[i].bytes, 1}))
                return fail(KDA_ERR_ALIASING, "%s overlaps %s", r[out].name, r[i].name);
        }
    }
    return KDA_OK;
}

inline kda_status check_workspace(size_t have, size_t need) {
    if (have < need)
        return fail(KDA_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", have, need);
    return KDA_OK;
}

inline kda::StateIO pool_state(float* pool, int n_slots, const int* in, const int* out) {
    return kda::StateIO{in ? pool : nullptr, in, out ? pool : nullptr, out, in, out, n_slots};
}

}  // namespace host
}  // namespace kda
