// kda_linear_api.hip -- the C ABI of the linear-attention, tree and norm entry
// points of include/kda.h: argument validation (entirely on the host, before
// any HIP call) and dispatch to the kernel launchers.
#include "kda_call.hpp"
#include "kda_linear.hpp"

namespace {

using namespace kda::host;

// kda_linear_prefill and kda_linear_prefill_paged (pool set).
kda_status prefill(const char* where, const void* q, const void* k, const void* v, const float* g,
                   float scale, const float* S0, float* S_T, float* pool, int n_slots,
                   const int* slots_in, const int* slots_out, bool paged, const int* lens, void* o,
                   int B, int T, int H, int H_k, int d_k, int d_v, kda_dtype dt, void* ws,
                   size_t ws_bytes, void* stream) {
    Sizes n;
    kda_status s = check_sizes(B, T, H, H_k, d_k, d_v, dt, scale, n);
    if (s != KDA_OK || (paged && (s = check_pool(n_slots, H)) != KDA_OK)) return s;
    const size_t es = dt == KDA_BF16 ? 2 : 4;
    const size_t need = kda::linear_prefill_ws_bytes(B, T, H, d_k, d_v, dt == KDA_BF16);
    const size_t pool_bytes = paged ? (size_t)n_slots * H * d_k * d_v * 4 : 0;
    const Ptr r[] = {{"q", q, n.qk * es, 16, true, false, nullptr},
                     {"k", k, n.qk * es, 16, true, false, nullptr},
                     {"v", v, n.vo * es, 16, true, false, nullptr},
                     {"g", g, (size_t)H * 4, 4, true, false, nullptr},
                     {"S0", S0, n.state * 4, 16, false, false, nullptr},
                     {"lens", lens, (size_t)B * 4, 4, false, false, nullptr},
                     {"slots_in", slots_in, (size_t)B * 4, 4, false, false, nullptr},
                     {"slots_out", slots_out, (size_t)B * 4, 4, false, false, nullptr},
                     {"pool", pool, pool_bytes, 16, paged, true, nullptr},
                     {"o", o, n.vo * es, 16, true, true, nullptr},
                     {"S_T", S_T, n.state * 4, 16, false, true, "S0"},
                     {"workspace", ws, need, 16, need > 0, true, nullptr}};
    if ((s = check_call(r, 12)) != KDA_OK || (s = check_workspace(ws_bytes, need)) != KDA_OK) return s;
    const kda::LinearPass p{{q, H_k}, {k, H_k}, {v, H}, o, H, dt == KDA_F32, g, scale, 1.0f,
                            paged ? pool_state(pool, n_slots, slots_in, slots_out)
                                  : kda::dense_state(S0, S_T),
                            false, lens, false, B, T, H, d_k, d_v, dt == KDA_BF16};
    return hip_status(kda::launch_linear_prefill(p, ws, (hipStream_t)stream), where);
}

kda_status decode(const char* where, const void* q, const void* k, const void* v, const float* g,
                  float scale, float* S, int n_slots, const int* slots, bool paged, void* o, int B,
                  int H, int H_k, int d_k, int d_v, kda_dtype dt, void* stream) {
    Sizes n;
    kda_status s = check_sizes(B, 1, H, H_k, d_k, d_v, dt, scale, n);
    if (s != KDA_OK || (paged && (s = check_pool(n_slots, H)) != KDA_OK)) return s;
    const size_t es = dt == KDA_BF16 ? 2 : 4;
    const size_t S_bytes = paged ? (size_t)n_slots * H * d_k * d_v * 4 : n.state * 4;
    const Ptr r[] = {{"q", q, n.qk * es, 16, true, false, nullptr},
                     {"k", k, n.qk * es, 16, true, false, nullptr},
                     {"v", v, n.vo * es, 16, true, false, nullptr},
                     {"g", g, (size_t)H * 4, 4, true, false, nullptr},
                     {"slots", slots, (size_t)B * 4, 4, paged, false, nullptr},
                     {paged ? "pool" : "S", S, S_bytes, 16, true, true, nullptr},
                     {"o", o, n.vo * es, 16, true, true, nullptr}};
    if ((s = check_call(r, 7)) != KDA_OK) return s;
    const kda::LinearDecode a{q, k, v, g, scale,
                              paged ? pool_state(S, n_slots, slots, slots) : kda::dense_state(S, S),
                              o, B, H, H_k, d_k, d_v, dt == KDA_BF16};
    return hip_status(kda::launch_linear_decode(a, (hipStream_t)stream), where);
}

kda_status check_tree_tokens(int T) {
    if (T < 1 || T > KDA_MAX_TREE_TOKENS)
        return fail(KDA_ERR_INVALID_SHAPE, "T=%d outside [1, %d]", T, KDA_MAX_TREE_TOKENS);
    return KDA_OK;
}

kda_status tree(const char* where, const void* q, const void* k, const void* v, const float* g,
                float scale, const float* S, int n_slots, const int* slots, bool paged,
                const int* parent, void* o, int B, int T, int H, int H_k, int d_k, int d_v,
                kda_dtype dt, void* stream) {
    Sizes n;
    kda_status s = check_sizes(B, T, H, H_k, d_k, d_v, dt, scale, n);
    if (s != KDA_OK || (s = check_tree_tokens(T)) != KDA_OK ||
        (paged && (s = check_pool(n_slots, H)) != KDA_OK))
        return s;
    const size_t es = dt == KDA_BF16 ? 2 : 4;
    const size_t S_bytes = paged ? (size_t)n_slots * H * d_k * d_v * 4 : n.state * 4;
    const Ptr r[] = {{"q", q, n.qk * es, 16, true, false, nullptr},
                     {"k", k, n.qk * es, 16, true, false, nullptr},
                     {"v", v, n.vo * es, 16, true, false, nullptr},
                     {"g", g, (size_t)H * 4, 4, true, false, nullptr},
                     {"slots", slots, (size_t)B * 4, 4, paged, false, nullptr},
                     {paged ? "pool" : "S", S, S_bytes, 16, true, false, nullptr},
                     {"parent", parent, n.tok * 4, 4, true, false, nullptr},
                     {"o", o, n.vo * es, 16, true, true, nullptr}};
    if ((s = check_call(r, 8)) != KDA_OK) return s;
    kda::StateIO io = paged ? pool_state(const_cast<float*>(S), n_slots, slots, nullptr)
                            : kda::dense_state(S, nullptr);
    const kda::LinearTree a{q, k, v, g, scale, io, parent, nullptr, o, B, T, H, H_k, d_k, d_v,
                            dt == KDA_BF16};
    return hip_status(kda::launch_linear_tree(a, (hipStream_t)stream), where);
}

kda_status commit(const char* where, const void* k, const void* v, const float* g,
                  const int* parent, const int* accepted, const float* S, float* S_out,
                  int n_slots, const int* slots_in, const int* slots_out, bool paged, int B, int T,
                  int H, int H_k, int d_k, int d_v, kda_dtype dt, void* stream) {
    Sizes n;
    kda_status s = check_sizes(B, T, H, H_k, d_k, d_v, dt, 1.0f, n);
    if (s != KDA_OK || (s = check_tree_tokens(T)) != KDA_OK ||
        (paged && (s = check_pool(n_slots, H)) != KDA_OK))
        return s;
    const size_t es = dt == KDA_BF16 ? 2 : 4;
    const size_t S_bytes = paged ? (size_t)n_slots * H * d_k * d_v * 4 : n.state * 4;
    const Ptr r[] = {{"k", k, n.qk * es, 16, true, false, nullptr},
                     {"v", v, n.vo * es, 16, true, false, nullptr},
                     {"g", g, (size_t)H * 4, 4, true, false, nullptr},
                     {"parent", parent, n.tok * 4, 4, true, false, nullptr},
                     {"accepted", accepted, (size_t)B * 4, 4, true, false, nullptr},
                     {"slots_in", slots_in, (size_t)B * 4, 4, paged, false, nullptr},
                     {"slots_out", slots_out, (size_t)B * 4, 4, paged, false, nullptr},
                     {"S", paged ? nullptr : S, n.state * 4, 16, !paged, false, nullptr},
                     {paged ? "pool" : "S_out", S_out, S_bytes, 16, true, true, paged ? nullptr : "S"}};
    if ((s = check_call(r, 9)) != KDA_OK) return s;
    kda::StateIO io = paged ? pool_state(S_out, n_slots, slots_in, slots_out) : kda::dense_state(S, S_out);
    const kda::LinearTree a{nullptr, k, v, g, 1.0f, io, parent, accepted, nullptr, B, T, H, H_k,
                            d_k, d_v, dt == KDA_BF16};
    return hip_status(kda::launch_linear_commit(a, (hipStream_t)stream), where);
}

kda_status check_norm(int B, int T, int H, int H_k, int d, kda_dtype dt, int norm, float eps,
                      int rot, int interleaved, size_t& nq, size_t& nk) {
    kda_status s = check_dtype(dt);
    if (s != KDA_OK) return s;
    if (!head_size_ok(d)) return fail(KDA_ERR_UNSUPPORTED, "d = %d; supported: 32, 64, 128", d);
    size_t ntok;
    if ((s = check_shape(B, T, H, d, nq, ntok)) != KDA_OK) return s;
    if ((s = check_shape(B, T, H_k, d, nk, ntok)) != KDA_OK) return s;
    if (norm != KDA_NORM_L2 && norm != KDA_NORM_RMS)
        return fail(KDA_ERR_INVALID_VALUE, "norm %d is not KDA_NORM_L2 or KDA_NORM_RMS", norm);
    if (!std::isfinite(eps) || eps <= 0.0f)
        return fail(KDA_ERR_INVALID_VALUE, "eps = %g must be finite and > 0", (double)eps);
    if (rot < 0 || rot > d || rot % 2 != 0)
        return fail(KDA_ERR_INVALID_VALUE, "rot = %d must be even and in [0, d = %d]", rot, d);
    if (interleaved != 0 && interleaved != 1)
        return fail(KDA_ERR_INVALID_VALUE, "interleaved = %d is not 0 or 1", interleaved);
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_linear_prefill_workspace_bytes(int B, int T, int H, int H_k, int d_k, int d_v,
                                          kda_dtype dt) {
    Sizes n;
    if (check_sizes(B, T, H, H_k, d_k, d_v, dt, 1.0f, n) != KDA_OK) return 0;
    return kda::linear_prefill_ws_bytes(B, T, H, d_k, d_v, dt == KDA_BF16);
}

kda_status kda_linear_prefill(const void* q, const void* k, const void* v, const float* g,
                              float scale, const float* S0, const int* lens, void* o, float* S_T,
                              int B, int T, int H, int H_k, int d_k, int d_v, kda_dtype dt,
                              void* workspace, size_t workspace_bytes, void* stream) {
    return prefill("kda_linear_prefill launch", q, k, v, g, scale, S0, S_T, nullptr, 0, nullptr,
                   nullptr, false, lens, o, B, T, H, H_k, d_k, d_v, dt, workspace, workspace_bytes,
                   stream);
}

kda_status kda_linear_prefill_paged(const void* q, const void* k, const void* v, const float* g,
                                    float scale, float* pool, int n_slots, const int* slots_in,
                                    const int* slots_out, const int* lens, void* o, int B, int T,
                                    int H, int H_k, int d_k, int d_v, kda_dtype dt,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    return prefill("kda_linear_prefill_paged launch", q, k, v, g, scale, nullptr, nullptr, pool,
                   n_slots, slots_in, slots_out, true, lens, o, B, T, H, H_k, d_k, d_v, dt,
                   workspace, workspace_bytes, stream);
}

size_t kda_linear_backward_workspace_bytes(int B, int T, int H, int H_k, int d_k, int d_v,
                                           kda_dtype dt) {
    Sizes n;
    if (check_sizes(B, T, H, H_k, d_k, d_v, dt, 1.0f, n) != KDA_OK) return 0;
    return kda::linear_backward_ws_bytes(B, T, H, H_k, d_k, d_v, dt == KDA_BF16);
}

kda_status kda_linear_backward(const void* q, const void* k, const void* v, const float* g,
                               float scale, const float* S0, const int* lens, const void* dO,
                               const float* dS_T, void* dq, void* dk, void* dv, float* dS0, int B,
                               int T, int H, int H_k, int d_k, int d_v, kda_dtype dt,
                               void* workspace, size_t workspace_bytes, void* stream) {
    Sizes n;
    kda_status s = check_sizes(B, T, H, H_k, d_k, d_v, dt, scale, n);
    if (s != KDA_OK) return s;
    const size_t es = dt == KDA_BF16 ? 2 : 4;
    const size_t need = kda::linear_backward_ws_bytes(B, T, H, H_k, d_k, d_v, dt == KDA_BF16);
    const Ptr r[] = {{"q", q, n.qk * es, 16, true, false, nullptr},
                     {"k", k, n.qk * es, 16, true, false, nullptr},
                     {"v", v, n.vo * es, 16, true, false, nullptr},
                     {"g", g, (size_t)H * 4, 4, true, false, nullptr},
                     {"S0", S0, n.state * 4, 16, false, false, nullptr},
                     {"lens", lens, (size_t)B * 4, 4, false, false, nullptr},
                     {"dO", dO, n.vo * es, 16, true, false, nullptr},
                     {"dS_T", dS_T, n.state * 4, 16, false, false, nullptr},
                     {"dq", dq, n.qk * es, 16, true, true, nullptr},
                     {"dk", dk, n.qk * es, 16, true, true, nullptr},
                     {"dv", dv, n.vo * es, 16, true, true, nullptr},
                     {"dS0", dS0, n.state * 4, 16, false, true, nullptr},
                     {"workspace", workspace, need, 16, need > 0, true, nullptr}};
    if ((s = check_call(r, 13)) != KDA_OK || (s = check_workspace(workspace_bytes, need)) != KDA_OK)
        return s;
    const kda::LinearBackward a{q, k, v, g, scale, S0, lens, dO, dS_T, dq, dk, dv, dS0,
                                B, T, H, H_k, d_k, d_v, dt == KDA_BF16};
    return hip_status(kda::launch_linear_backward(a, workspace, (hipStream_t)stream),
                      "kda_linear_backward launch");
}

kda_status kda_linear_decode_step(const void* q, const void* k, const void* v, const float* g,
                                  float scale, float* S, void* o, int B, int H, int H_k, int d_k,
                                  int d_v, kda_dtype dt, void* stream) {
    return decode("kda_linear_decode_step launch", q, k, v, g, scale, S, 0, nullptr, false, o, B,
                  H, H_k, d_k, d_v, dt, stream);
}

kda_status kda_linear_decode_step_paged(const void* q, const void* k, const void* v,
                                        const float* g, float scale, float* pool, int n_slots,
                                        const int* slots, void* o, int B, int H, int H_k, int d_k,
                                        int d_v, kda_dtype dt, void* stream) {
    return decode("kda_linear_decode_step_paged launch", q, k, v, g, scale, pool, n_slots, slots,
                  true, o, B, H, H_k, d_k, d_v, dt, stream);
}

kda_status kda_linear_tree(const void* q, const void* k, const void* v, const float* g,
                           float scale, const float* S, const int* parent, void* o, int B, int T,
                           int H, int H_k, int d_k, int d_v, kda_dtype dt, void* stream) {
    return tree("kda_linear_tree launch", q, k, v, g, scale, S, 0, nullptr, false, parent, o, B, T,
                H, H_k, d_k, d_v, dt, stream);
}

kda_status kda_linear_tree_paged(const void* q, const void* k, const void* v, const float* g,
                                 float scale, const float* pool, int n_slots, const int* slots,
                                 const int* parent, void* o, int B, int T, int H, int H_k, int d_k,
                                 int d_v, kda_dtype dt, void* stream) {
    return tree("kda_linear_tree_paged launch", q, k, v, g, scale, pool, n_slots, slots, true,
                parent, o, B, T, H, H_k, d_k, d_v, dt, stream);
}

kda_status kda_linear_tree_commit(const void* k, const void* v, const float* g, const int* parent,
                                  const int* accepted, const float* S, float* S_out, int B, int T,
                                  int H, int H_k, int d_k, int d_v, kda_dtype dt, void* stream) {
    return commit("kda_linear_tree_commit launch", k, v, g, parent, accepted, S, S_out, 0, nullptr,
                  nullptr, false, B, T, H, H_k, d_k, d_v, dt, stream);
}

kda_status kda_linear_tree_commit_paged(const void* k, const void* v, const float* g,
                                        const int* parent, const int* accepted, float* pool,
                                        int n_slots, const int* slots_in, const int* slots_out,
                                        int B, int T, int H, int H_k, int d_k, int d_v,
                                        kda_dtype dt, void* stream) {
    return commit("kda_linear_tree_commit_paged launch", k, v, g, parent, accepted, nullptr, pool,
                  n_slots, slots_in, slots_out, true, B, T, H, H_k, d_k, d_v, dt, stream);
}

kda_status kda_qk_norm_rope(const void* q, const void* k, const float* w_q, const float* w_k,
                            const int* positions, const float* inv_freq, int norm, float eps,
                            int rot, int interleaved, void* y_q, void* y_k, int B, int T, int H,
                            int H_k, int d, kda_dtype dt, void* stream) {
    size_t nq, nk;
    kda_status s = check_norm(B, T, H, H_k, d, dt, norm, eps, rot, interleaved, nq, nk);
    if (s != KDA_OK) return s;
    const size_t es = dt == KDA_BF16 ? 2 : 4, w = (size_t)d * 4;
    const Ptr r[] = {{"q", q, nq * es, 16, true, false, nullptr},
                     {"k", k, nk * es, 16, true, false, nullptr},
                     {"w_q", w_q, w, 4, false, false, nullptr},
                     {"w_k", w_k, w, 4, false, false, nullptr},
                     {"positions", positions, (size_t)B * T * 4, 4, rot > 0, false, nullptr},
                     {"inv_freq", inv_freq, (size_t)rot * 2, 4, rot > 0, false, nullptr},
                     {"y_q", y_q, nq * es, 16, true, true, "q"},
                     {"y_k", y_k, nk * es, 16, true, true, "k"}};
    if ((s = check_call(r, 8)) != KDA_OK) return s;
    const kda::NormRope a{q, k, w_q, w_k, positions, inv_freq, norm == KDA_NORM_RMS, eps, rot,
                          interleaved == 1, nullptr, nullptr, y_q, y_k, nullptr, nullptr,
                          B, T, H, H_k, d, dt == KDA_BF16};
    return hip_status(kda::launch_norm_rope(a, (hipStream_t)stream), "kda_qk_norm_rope launch");
}

size_t kda_qk_norm_rope_backward_workspace_bytes(int B, int T, int H, int H_k, int d,
                                                 kda_dtype dt) {
    size_t nq, nk;
    if (check_norm(B, T, H, H_k, d, dt, KDA_NORM_RMS, 1.0f, 0, 0, nq, nk) != KDA_OK) return 0;
    return kda::norm_rope_backward_ws_bytes(B, T, H, H_k, d);
}

kda_status kda_qk_norm_rope_backward(const void* q, const void* k, const float* w_q,
                                     const float* w_k, const int* positions,
                                     const float* inv_freq, int norm, float eps, int rot,
                                     int interleaved, const void* dy_q, const void* dy_k, void* dq,
                                     void* dk, float* dw_q, float* dw_k, int B, int T, int H,
                                     int H_k, int d, kda_dtype dt, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    size_t nq, nk;
    kda_status s = check_norm(B, T, H, H_k, d, dt, norm, eps, rot, interleaved, nq, nk);
    if (s != KDA_OK) return s;
    const size_t need = dw_q || dw_k ? kda::norm_rope_backward_ws_bytes(B, T, H, H_k, d) : 0;
    const size_t es = dt == KDA_BF16 ? 2 : 4, w = (size_t)d * 4;
    const Ptr r[] = {{"q", q, nq * es, 16, true, false, nullptr},
                     {"k", k, nk * es, 16, true, false, nullptr},
                     {"w_q", w_q, w, 4, dw_q != nullptr, false, nullptr},
                     {"w_k", w_k, w, 4, dw_k != nullptr, false, nullptr},
                     {"positions", positions, (size_t)B * T * 4, 4, rot > 0, false, nullptr},
                     {"inv_freq", inv_freq, (size_t)rot * 2, 4, rot > 0, false, nullptr},
                     {"dy_q", dy_q, nq * es, 16, true, false, nullptr},
                     {"dy_k", dy_k, nk * es, 16, true, false, nullptr},
                     {"dq", dq, nq * es, 16, true, true, "dy_q"},
                     {"dk", dk, nk * es, 16, true, true, "dy_k"},
                     {"dw_q", dw_q, w, 4, false, true, nullptr},
                     {"dw_k", dw_k, w, 4, false, true, nullptr},
                     {"workspace", workspace, need, 16, need > 0, true, nullptr}};
    if ((s = check_call(r, 13)) != KDA_OK || (s = check_workspace(workspace_bytes, need)) != KDA_OK)
        return s;
    const kda::NormRope a{q, k, w_q, w_k, positions, inv_freq, norm == KDA_NORM_RMS, eps, rot,
                          interleaved == 1, dy_q, dy_k, dq, dk, dw_q, dw_k,
                          B, T, H, H_k, d, dt == KDA_BF16};
    return hip_status(kda::launch_norm_rope_backward(a, workspace, (hipStream_t)stream),
                      "kda_qk_norm_rope_backward launch");
}

}  // extern "C"
