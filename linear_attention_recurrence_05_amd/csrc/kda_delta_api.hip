// kda_delta_api.hip -- the C ABI of the delta-rule and norm entry points of
// include/kda.h: argument validation (entirely on the host, before any HIP
// call) and dispatch to the kernel launchers.
#include "kda_call.hpp"
#include "kda_delta.hpp"

namespace {

using namespace kda::host;

kda_status check_delta(int B, int T, int H, int H_k, int d_k, int d_v, kda_dtype dt, float scale, Sizes& n) {
    const kda_status s = check_sizes(B, T, H, H_k, d_k, d_v, dt, scale, n);
    if (s != KDA_OK) return s;
    if ((long long)B * H > kda::kDeltaMaxUnits)
        return fail(KDA_ERR_INVALID_SHAPE, "B*H = %lld is too large (limit 2^19)", (long long)B * H);
    // 64 tokens of a head lie within 2^30 bytes
    if ((long long)H * (d_k > d_v ? d_k : d_v) > (1LL << 22))
        return fail(KDA_ERR_INVALID_SHAPE, "H*d = %lld is too large (limit 2^22)", (long long)H * (d_k > d_v ? d_k : d_v));
    return KDA_OK;
}

// kda_delta_prefill and kda_delta_prefill_paged (pool set).
kda_status prefill(const char* where, const void* q, const void* k, const void* v, const float* g,
                   const float* beta, float scale, const float* S0, float* S_T, float* pool,
                   int n_slots, const int* slots_in, const int* slots_out, bool paged,
                   const int* lens, void* o, int B, int T, int H, int H_k, int d_k, int d_v,
                   kda_dtype dt, void* ws, size_t ws_bytes, void* stream) {
    Sizes n;
    kda_status s = check_delta(B, T, H, H_k, d_k, d_v, dt, scale, n);
    if (s != KDA_OK || (paged && (s = check_pool(n_slots, H)) != KDA_OK)) return s;
    const size_t es = dt == KDA_BF16 ? 2 : 4;
    const size_t need = kda::delta_prefill_ws_bytes(B, T, H, d_k, d_v, dt == KDA_BF16);
    const size_t pool_bytes = paged ? (size_t)n_slots * H * d_k * d_v * 4 : 0;
    const Ptr r[] = {{"q", q, n.qk * es, 16, true, false, nullptr},
                     {"k", k, n.qk * es, 16, true, false, nullptr},
                     {"v", v, n.vo * es, 16, true, false, nullptr},
                     {"g", g, n.tok * H * 4, 4, true, false, nullptr},
                     {"beta", beta, n.tok * H * 4, 4, true, false, nullptr},
                     {"S0", S0, n.state * 4, 16, false, false, nullptr},
                     {"lens", lens, (size_t)B * 4, 4, false, false, nullptr},
                     {"slots_in", slots_in, (size_t)B * 4, 4, false, false, nullptr},
                     {"slots_out", slots_out, (size_t)B * 4, 4, false, false, nullptr},
                     {"pool", pool, pool_bytes, 16, paged, true, nullptr},
                     {"o", o, n.vo * es, 16, true, true, nullptr},
                     {"S_T", S_T, n.state * 4, 16, false, true, "S0"},
                     {"workspace", ws, need, 16, need > 0, true, nullptr}};
    if ((s = check_call(r, 13)) != KDA_OK || (s = check_workspace(ws_bytes, need)) != KDA_OK) return s;
    const kda::DeltaPrefill a{q, k, v, g, beta, scale,
                              paged ? pool_state(pool, n_slots, slots_in, slots_out)
                                    : kda::dense_state(S0, S_T),
                              lens, o, B, T, H, H_k, d_k, d_v, dt == KDA_BF16};
    return hip_status(kda::launch_delta_prefill(a, ws, (hipStream_t)stream), where);
}

kda_status decode(const char* where, const void* q, const void* k, const void* v, const float* g,
                  const float* beta, float scale, float* S, int n_slots, const int* slots,
                  bool paged, void* o, int B, int H, int H_k, int d_k, int d_v, kda_dtype dt,
                  void* stream) {
    Sizes n;
    kda_status s = check_delta(B, 1, H, H_k, d_k, d_v, dt, scale, n);
    if (s != KDA_OK || (paged && (s = check_pool(n_slots, H)) != KDA_OK)) return s;
    const size_t es = dt == KDA_BF16 ? 2 : 4;
    const size_t S_bytes = paged ? (size_t)n_slots * H * d_k * d_v * 4 : n.state * 4;
    const Ptr r[] = {{"q", q, n.qk * es, 16, true, false, nullptr},
                     {"k", k, n.qk * es, 16, true, false, nullptr},
                     {"v", v, n.vo * es, 16, true, false, nullptr},
                     {"g", g, n.tok * H * 4, 4, true, false, nullptr},
                     {"beta", beta, n.tok * H * 4, 4, true, false, nullptr},
                     {"slots", slots, (size_t)B * 4, 4, paged, false, nullptr},
                     {paged ? "pool" : "S", S, S_bytes, 16, true, true, nullptr},
                     {"o", o, n.vo * es, 16, true, true, nullptr}};
    if ((s = check_call(r, 8)) != KDA_OK) return s;
    const kda::DeltaDecode a{q, k, v, g, beta, scale,
                             paged ? pool_state(S, n_slots, slots, slots) : kda::dense_state(S, S),
                             o, B, H, H_k, d_k, d_v, dt == KDA_BF16};
    return hip_status(kda::launch_delta_decode(a, (hipStream_t)stream), where);
}

kda_status check_eps(float eps) {
    if (!std::isfinite(eps) || eps <= 0.0f)
        return fail(KDA_ERR_INVALID_VALUE, "eps = %g must be finite and > 0", (double)eps);
    return KDA_OK;
}

kda_status check_rows(long long rows, long long d) {
    if (rows < 1) return fail(KDA_ERR_INVALID_SHAPE, "rows=%lld must be >= 1", rows);
    if (rows > (1LL << 40) / d) return fail(KDA_ERR_INVALID_SHAPE, "rows=%lld of %lld elements are too many (limit 2^40 elements)", rows, d);
    return KDA_OK;
}

kda_status check_gated(long long rows, int d, kda_dtype dt, int act, float eps) {
    kda_status s = check_dtype(dt);
    if (s != KDA_OK) return s;
    if (!head_size_ok(d)) return fail(KDA_ERR_UNSUPPORTED, "d = %d; supported: 32, 64, 128", d);
    if ((s = check_rows(rows, d)) != KDA_OK) return s;
    if (act != KDA_GATE_SIGMOID && act != KDA_GATE_SILU)
        return fail(KDA_ERR_INVALID_VALUE, "act %d is not KDA_GATE_SIGMOID or KDA_GATE_SILU", act);
    return check_eps(eps);
}

kda_status check_block(long long rows, int D, kda_dtype dt, int norm_y, float scale, float eps) {
    kda_status s = check_dtype(dt);
    if (s != KDA_OK) return s;
    if (D < 8 || D > KDA_MAX_NORM_WIDTH || D % 8 != 0)
        return fail(KDA_ERR_UNSUPPORTED, "D = %d; supported: multiples of 8 in [8, %d]", D, KDA_MAX_NORM_WIDTH);
    if ((s = check_rows(rows, D)) != KDA_OK) return s;
    if (norm_y != 0 && norm_y != 1) return fail(KDA_ERR_INVALID_VALUE, "norm_y = %d is not 0 or 1", norm_y);
    if (!std::isfinite(scale)) return fail(KDA_ERR_INVALID_VALUE, "scale = %g is not finite", (double)scale);
    return check_eps(eps);
}

}  // namespace

extern "C" {

size_t kda_delta_prefill_workspace_bytes(int B, int T, int H, int H_k, int d_k, int d_v,
                                         kda_dtype dt) {
    Sizes n;
    if (check_delta(B, T, H, H_k, d_k, d_v, dt, 1.0f, n) != KDA_OK) return 0;
    return kda::delta_prefill_ws_bytes(B, T, H, d_k, d_v, dt == KDA_BF16);
}

kda_status kda_delta_prefill(const void* q, const void* k, const void* v, const float* g,
                             const float* beta, float scale, const float* S0, const int* lens,
                             void* o, float* S_T, int B, int T, int H, int H_k, int d_k, int d_v,
                             kda_dtype dt, void* workspace, size_t workspace_bytes, void* stream) {
    return prefill("kda_delta_prefill launch", q, k, v, g, beta, scale, S0, S_T, nullptr, 0,
                   nullptr, nullptr, false, lens, o, B, T, H, H_k, d_k, d_v, dt, workspace,
                   workspace_bytes, stream);
}

kda_status kda_delta_prefill_paged(const void* q, const void* k, const void* v, const float* g,
                                   const float* beta, float scale, float* pool, int n_slots,
                                   const int* slots_in, const int* slots_out, const int* lens,
                                   void* o, int B, int T, int H, int H_k, int d_k, int d_v,
                                   kda_dtype dt, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    return prefill("kda_delta_prefill_paged launch", q, k, v, g, beta, scale, nullptr, nullptr,
                   pool, n_slots, slots_in, slots_out, true, lens, o, B, T, H, H_k, d_k, d_v, dt,
                   workspace, workspace_bytes, stream);
}

size_t kda_delta_backward_workspace_bytes(int B, int T, int H, int H_k, int d_k, int d_v,
                                          kda_dtype dt) {
    Sizes n;
    if (check_delta(B, T, H, H_k, d_k, d_v, dt, 1.0f, n) != KDA_OK) return 0;
    return kda::delta_backward_ws_bytes(B, T, H, H_k, d_k, d_v, dt == KDA_BF16);
}

kda_status kda_delta_backward(const void* q, const void* k, const void* v, const float* g,
                              const float* beta, float scale, const float* S0, const int* lens,
                              const void* dO, const float* dS_T, void* dq, void* dk, void* dv,
                              float* dg, float* dbeta, float* dS0, int B, int T, int H, int H_k,
                              int d_k, int d_v, kda_dtype dt, void* workspace,
                              size_t workspace_bytes, void* stream) {
    Sizes n;
    kda_status s = check_delta(B, T, H, H_k, d_k, d_v, dt, scale, n);
    if (s != KDA_OK) return s;
    const size_t es = dt == KDA_BF16 ? 2 : 4, gates = n.tok * H * 4;
    const size_t need = kda::delta_backward_ws_bytes(B, T, H, H_k, d_k, d_v, dt == KDA_BF16);
    const Ptr r[] = {{"q", q, n.qk * es, 16, true, false, nullptr},
                     {"k", k, n.qk * es, 16, true, false, nullptr},
                     {"v", v, n.vo * es, 16, true, false, nullptr},
                     {"g", g, gates, 4, true, false, nullptr},
                     {"beta", beta, gates, 4, true, false, nullptr},
                     {"S0", S0, n.state * 4, 16, false, false, nullptr},
                     {"lens", lens, (size_t)B * 4, 4, false, false, nullptr},
                     {"dO", dO, n.vo * es, 16, true, false, nullptr},
                     {"dS_T", dS_T, n.state * 4, 16, false, false, nullptr},
                     {"dq", dq, n.qk * es, 16, true, true, nullptr},
                     {"dk", dk, n.qk * es, 16, true, true, nullptr},
                     {"dv", dv, n.vo * es, 16, true, true, nullptr},
                     {"dg", dg, gates, 4, true, true, nullptr},
                     {"dbeta", dbeta, gates, 4, true, true, nullptr},
                     {"dS0", dS0, n.state * 4, 16, false, true, nullptr},
                     {"workspace", workspace, need, 16, need > 0, true, nullptr}};
    if ((s = check_call(r, 16)) != KDA_OK || (s = check_workspace(workspace_bytes, need)) != KDA_OK)
        return s;
    const kda::DeltaBackward a{q, k, v, g, beta, scale, S0, lens, dO, dS_T, dq, dk, dv, dg, dbeta,
                               dS0, B, T, H, H_k, d_k, d_v, dt == KDA_BF16};
    return hip_status(kda::launch_delta_backward(a, workspace, (hipStream_t)stream),
                      "kda_delta_backward launch");
}

kda_status kda_delta_decode_step(const void* q, const void* k, const void* v, const float* g,
                                 const float* beta, float scale, float* S, void* o, int B, int H,
                                 int H_k, int d_k, int d_v, kda_dtype dt, void* stream) {
    return decode("kda_delta_decode_step launch", q, k, v, g, beta, scale, S, 0, nullptr, false, o,
                  B, H, H_k, d_k, d_v, dt, stream);
}

kda_status kda_delta_decode_step_paged(const void* q, const void* k, const void* v, const float* g,
                                       const float* beta, float scale, float* pool, int n_slots,
                                       const int* slots, void* o, int B, int H, int H_k, int d_k,
                                       int d_v, kda_dtype dt, void* stream) {
    return decode("kda_delta_decode_step_paged launch", q, k, v, g, beta, scale, pool, n_slots,
                  slots, true, o, B, H, H_k, d_k, d_v, dt, stream);
}

kda_status kda_gated_norm(const void* x, const void* z, const float* w, int act, float eps, void* y,
                          long long rows, int d, kda_dtype dt, void* stream) {
    kda_status s = check_gated(rows, d, dt, act, eps);
    if (s != KDA_OK) return s;
    const size_t n = (size_t)rows * d * (dt == KDA_BF16 ? 2 : 4);
    const Ptr r[] = {{"x", x, n, 16, true, false, nullptr},
                     {"z", z, n, 16, true, false, nullptr},
                     {"w", w, (size_t)d * 4, 4, false, false, nullptr},
                     {"y", y, n, 16, true, true, "x"}};
    if ((s = check_call(r, 4)) != KDA_OK) return s;
    const kda::GatedNorm a{x, z, w, act == KDA_GATE_SILU, eps, nullptr, y, nullptr, nullptr, rows, d,
                           dt == KDA_BF16};
    return hip_status(kda::launch_gated_norm(a, (hipStream_t)stream), "kda_gated_norm launch");
}

size_t kda_gated_norm_backward_workspace_bytes(long long rows, int d, kda_dtype dt) {
    if (check_gated(rows, d, dt, KDA_GATE_SILU, 1.0f) != KDA_OK) return 0;
    return kda::gated_norm_backward_ws_bytes(rows, d);
}

kda_status kda_gated_norm_backward(const void* x, const void* z, const float* w, int act, float eps,
                                   const void* dy, void* dx, void* dz, float* dw, long long rows,
                                   int d, kda_dtype dt, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    kda_status s = check_gated(rows, d, dt, act, eps);
    if (s != KDA_OK) return s;
    const size_t n = (size_t)rows * d * (dt == KDA_BF16 ? 2 : 4);
    const size_t need = dw ? kda::gated_norm_backward_ws_bytes(rows, d) : 0;
    const Ptr r[] = {{"x", x, n, 16, true, false, nullptr},
                     {"z", z, n, 16, true, false, nullptr},
                     {"w", w, (size_t)d * 4, 4, dw != nullptr, false, nullptr},
                     {"dy", dy, n, 16, true, false, nullptr},
                     {"dx", dx, n, 16, true, true, "dy"},
                     {"dz", dz, n, 16, true, true, nullptr},
                     {"dw", dw, (size_t)d * 4, 4, false, true, nullptr},
                     {"workspace", workspace, need, 16, need > 0, true, nullptr}};
    if ((s = check_call(r, 8)) != KDA_OK || (s = check_workspace(workspace_bytes, need)) != KDA_OK)
        return s;
    const kda::GatedNorm a{x, z, w, act == KDA_GATE_SILU, eps, dy, dx, dz, dw, rows, d, dt == KDA_BF16};
    return hip_status(kda::launch_gated_norm_backward(a, workspace, (hipStream_t)stream),
                      "kda_gated_norm_backward launch");
}

kda_status kda_block_norm(const void* y, const void* z, const float* w_y, const void* r,
                          const float* w_n, int norm_y, float scale, float eps, void* h, void* n,
                          long long rows, int D, kda_dtype dt, void* stream) {
    kda_status s = check_block(rows, D, dt, norm_y, scale, eps);
    if (s != KDA_OK) return s;
    if (!y && (z || w_y || h || norm_y))
        return fail(KDA_ERR_INVALID_VALUE, "z, w_y, h and norm_y belong to y, which is NULL");
    const size_t bytes = (size_t)rows * D * (dt == KDA_BF16 ? 2 : 4), w = (size_t)D * 4;
    const Ptr p[] = {{"y", y, bytes, 16, false, false, nullptr},
                     {"z", z, bytes, 16, false, false, nullptr},
                     {"w_y", w_y, w, 16, false, false, nullptr},
                     {"r", r, bytes, 16, true, false, nullptr},
                     {"w_n", w_n, w, 16, false, false, nullptr},
                     {"h", h, bytes, 16, y != nullptr, true, "r"},
                     {"n", n, bytes, 16, true, true, y ? "y" : "r"}};
    if ((s = check_call(p, 7)) != KDA_OK) return s;
    const kda::BlockNorm a{y, z, w_y, r, w_n, norm_y == 1, scale, eps, h, n, nullptr, nullptr,
                           nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, rows, D,
                           dt == KDA_BF16};
    return hip_status(kda::launch_block_norm(a, (hipStream_t)stream), "kda_block_norm launch");
}

size_t kda_block_norm_backward_workspace_bytes(long long rows, int D, kda_dtype dt) {
    if (check_block(rows, D, dt, 0, 1.0f, 1.0f) != KDA_OK) return 0;
    return kda::block_norm_backward_ws_bytes(rows, D, dt == KDA_BF16);
}

kda_status kda_block_norm_backward(const void* y, const void* z, const float* w_y, const void* h,
                                   const float* w_n, int norm_y, float scale, float eps,
                                   const void* dn, const void* dh, void* dr, void* dy, void* dz,
                                   float* dw_y, float* dw_n, long long rows, int D, kda_dtype dt,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    kda_status s = check_block(rows, D, dt, norm_y, scale, eps);
    if (s != KDA_OK) return s;
    if (!y && (z || w_y || dy || dz || dw_y || norm_y))
        return fail(KDA_ERR_INVALID_VALUE, "z, w_y, dy, dz, dw_y and norm_y belong to y, which is NULL");
    if (!z && dz) return fail(KDA_ERR_INVALID_VALUE, "dz belongs to z, which is NULL");
    const size_t bytes = (size_t)rows * D * (dt == KDA_BF16 ? 2 : 4), w = (size_t)D * 4;
    const size_t need = dw_y || dw_n ? kda::block_norm_backward_ws_bytes(rows, D, dt == KDA_BF16) : 0;
    const Ptr p[] = {{"y", y, bytes, 16, false, false, nullptr},
                     {"z", z, bytes, 16, false, false, nullptr},
                     {"w_y", w_y, w, 16, dw_y != nullptr, false, nullptr},
                     {"h", h, bytes, 16, true, false, nullptr},
                     {"w_n", w_n, w, 16, dw_n != nullptr, false, nullptr},
                     {"dn", dn, bytes, 16, true, false, nullptr},
                     {"dh", dh, bytes, 16, false, false, nullptr},
                     {"dr", dr, bytes, 16, true, true, "dh"},
                     {"dy", dy, bytes, 16, y != nullptr, true, nullptr},
                     {"dz", dz, bytes, 16, z != nullptr, true, nullptr},
                     {"dw_y", dw_y, w, 16, false, true, nullptr},
                     {"dw_n", dw_n, w, 16, false, true, nullptr},
                     {"workspace", workspace, need, 16, need > 0, true, nullptr}};
    if ((s = check_call(p, 13)) != KDA_OK || (s = check_workspace(workspace_bytes, need)) != KDA_OK)
        return s;
    const kda::BlockNorm a{y, z, w_y, nullptr, w_n, norm_y == 1, scale, eps, nullptr, nullptr, h, dn,
                           dh, dr, dy, dz, dw_y, dw_n, rows, D, dt == KDA_BF16};
    return hip_status(kda::launch_block_norm_backward(a, workspace, (hipStream_t)stream),
                      "kda_block_norm_backward launch");
}

}  // extern "C"
