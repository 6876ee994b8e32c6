// kda_host.hpp -- host-side helpers shared by the entry points: the status and
// detail string of the last error on this thread, and the checks of pointers,
// ranges and sizes that every call makes before any HIP call.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <string>

#include "../../include/kda.h"

namespace kda {
namespace host {

inline thread_local std::string g_last_error;

inline kda_status fail(kda_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_last_error = buf;
    return s;
}

inline kda_status ok() {
    g_last_error.clear();
    return KDA_OK;
}

struct Range {
    const char* name;
    const void* p;
    size_t bytes;
    unsigned align;   // required alignment in bytes
};

inline bool overlap(const Range& a, const Range& b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// Longest sequence: chunk counts and token offsets are formed in 32-bit ints.
constexpr int kMaxT = 1 << 30;

inline bool aligned(const void* p, unsigned a) { return ((uintptr_t)p & (uintptr_t)(a - 1)) == 0; }

// Checks a list of tensor ranges for NULL (when required) and alignment.
inline kda_status check_ptrs(const Range* r, int n, const bool* required) {
    for (int i = 0; i < n; ++i) {
        if (!r[i].p) {
            if (required[i]) return fail(KDA_ERR_NULL_POINTER, "%s is NULL", r[i].name);
            continue;
        }
        if (!aligned(r[i].p, r[i].align))
            return fail(KDA_ERR_MISALIGNED, "%s is not %u-byte aligned", r[i].name, r[i].align);
    }
    return KDA_OK;
}

inline kda_status hip_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return ok();
    return fail(KDA_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// Shape check shared by prefill-style calls; returns element counts.
inline kda_status check_shape(int B, int T, int H, int d, size_t& n_tok_el, size_t& n_tok) {
    if (B < 1 || T < 1 || H < 1) return fail(KDA_ERR_INVALID_SHAPE, "B=%d T=%d H=%d must all be >= 1", B, T, H);
    if (T > kMaxT) return fail(KDA_ERR_INVALID_SHAPE, "T=%d is too large (limit 2^30)", T);
    const unsigned long long tok = (unsigned long long)B * (unsigned long long)T * (unsigned long long)H;
    if ((long long)B * H > (1LL << 26) || tok > (1ULL << 40))
        return fail(KDA_ERR_INVALID_SHAPE, "B*T*H = %llu is too large", tok);
    if ((long long)H * d > (1LL << 24))
        return fail(KDA_ERR_INVALID_SHAPE, "H*d = %lld is too large (limit 2^24)", (long long)H * d);
    n_tok = (size_t)tok;
    n_tok_el = n_tok * (size_t)d;
    return KDA_OK;
}

}  // namespace host
}  // namespace kda
