// block_capi.cpp -- the exported C ABI of the feed-forward operators
// (include/q4_block.h): argument validation and the launches.
//
// Every check runs on the host before any HIP call, so a rejected call
// enqueues nothing and the checks work on a machine without a GPU.
#include "q4_block.h"

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "block_common.hpp"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 30;
// N and K: a panel of 32 rows of an operand image stays below 2^32 bytes
constexpr int64_t kMaxSum = int64_t(1) << 25;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int need(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!p) return Q4_ERR_NULL;
    for (const void* p : ps)
        if (!aligned16(p)) return Q4_ERR_ALIGN;
    return Q4_OK;
}
int optional(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!aligned16(p)) return Q4_ERR_ALIGN;
    return Q4_OK;
}

bool fmt_ok(int fmt) { return fmt == Q4_FMT_Q4_0 || fmt == Q4_FMT_AFFINE4 || fmt == Q4_FMT_AFFINE8; }
bool act_ok(int act) { return act >= Q4_ACT_NONE && act <= Q4_ACT_RELU; }
bool norm_ok(int norm) { return norm >= Q4_NORM_NONE && norm <= Q4_NORM_LAYER; }

int format_wf(int fmt) {
    return fmt == Q4_FMT_Q4_0 ? q4::WF_Q4_0 : fmt == Q4_FMT_AFFINE4 ? q4::WF_AFFINE4 : q4::WF_AFFINE8;
}

int check_product(int fmt, int act, int64_t M, int64_t N, int64_t K) {
    if (!fmt_ok(fmt) || !act_ok(act)) return Q4_ERR_ARG;
    if (M < 0 || N < 0 || K <= 0 || M > kMaxDim || N > kMaxSum || K > kMaxSum) return Q4_ERR_SHAPE;
    if (K % (fmt == Q4_FMT_Q4_0 ? 32 : 64) != 0) return Q4_ERR_SHAPE;
    return Q4_OK;
}

int check_planes(int fmt, const void* q, const void* s, const void* b) {
    const int rc = need({q, s});
    return rc || fmt == Q4_FMT_Q4_0 ? rc : need({b});
}

int check_workspace(const void* ws, int64_t have, int64_t want) {
    if (want <= 0) return Q4_OK;
    if (!ws || have < want) return Q4_ERR_WORKSPACE;
    return aligned16(ws) ? Q4_OK : Q4_ERR_ALIGN;
}

int hip_status(hipError_t e) { return e == hipSuccess ? Q4_OK : Q4_ERR_HIP; }
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

int64_t forward_bytes(int fmt, int nmat, int dtype, int64_t M, int64_t N, int64_t K) {
    if (dtype != Q4_BF16 && dtype != Q4_F16) return 0;
    if (check_product(fmt, Q4_ACT_NONE, M, N, K) != Q4_OK || M == 0 || N == 0) return 0;
    return q4::linear_workspace_bytes(format_wf(fmt), nmat, dtype, M, N, K);
}
int64_t backward_bytes(int fmt, int nmat, int64_t M, int64_t N, int64_t K) {
    if (check_product(fmt, Q4_ACT_NONE, M, N, K) != Q4_OK || M == 0 || N == 0) return 0;
    return q4::linear_grad_workspace_bytes(format_wf(fmt), nmat, M, N, K);
}

}  // namespace

extern "C" {

// ---- linear --------------------------------------------------------------------

int64_t q4_linear_workspace_size(int fmt, int dtype, int64_t M, int64_t N, int64_t K) {
    return forward_bytes(fmt, 1, dtype, M, N, K);
}

int q4_linear(int fmt, const uint8_t* w_q, const uint16_t* w_s, const uint16_t* w_b, const void* bias, int act,
              const void* residual, const void* x, int dtype, void* y, void* pre, int64_t M, int64_t N, int64_t K,
              void* workspace, int64_t workspace_bytes, void* stream) {
    if (dtype != Q4_BF16 && dtype != Q4_F16) return Q4_ERR_DTYPE;
    int rc = check_product(fmt, act, M, N, K);
    if (rc) return rc;
    if (M == 0 || N == 0) return Q4_OK;
    if ((rc = check_planes(fmt, w_q, w_s, w_b)) || (rc = need({x, y})) || (rc = optional({bias, residual, pre}))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, forward_bytes(fmt, 1, dtype, M, N, K)))) return rc;
    q4::LinearArgs a{};
    a.wf = format_wf(fmt);
    a.nmat = 1;
    a.act = act;
    a.dtype = dtype;
    a.w[0] = {w_q, w_s, w_b};
    a.bias[0] = bias;
    a.residual = residual;
    a.x = x;
    a.y = y;
    a.pre[0] = pre;
    a.M = M;
    a.N = N;
    a.K = K;
    return hip_status(q4::launch_linear(a, workspace, as_stream(stream)));
}

int64_t q4_linear_backward_workspace_size(int fmt, int64_t M, int64_t N, int64_t K) {
    return backward_bytes(fmt, 1, M, N, K);
}

int q4_linear_backward(int fmt, const uint8_t* w_q, const uint16_t* w_s, const uint16_t* w_b, int act,
                       const void* pre, const void* dy, int dtype, void* dx, void* dz, float* dbias, int64_t M,
                       int64_t N, int64_t K, void* workspace, int64_t workspace_bytes, void* stream) {
    if (dtype != Q4_BF16) return Q4_ERR_DTYPE;
    int rc = check_product(fmt, act, M, N, K);
    if (rc) return rc;
    if (act == Q4_ACT_NONE && dz) return Q4_ERR_ARG;
    if (M == 0 || N == 0) return Q4_OK;
    if ((rc = check_planes(fmt, w_q, w_s, w_b)) || (rc = need({dy, dx})) || (rc = optional({pre, dz, dbias}))) return rc;
    if (act != Q4_ACT_NONE && !pre) return Q4_ERR_NULL;
    if ((rc = check_workspace(workspace, workspace_bytes, backward_bytes(fmt, 1, M, N, K)))) return rc;
    q4::LinearGradArgs a{};
    a.wf = format_wf(fmt);
    a.nmat = 1;
    a.act = act;
    a.w[0] = {w_q, w_s, w_b};
    a.pre[0] = act != Q4_ACT_NONE ? pre : nullptr;
    a.dy = dy;
    a.dx = dx;
    a.dz[0] = dz;
    a.dbias[0] = dbias;
    a.M = M;
    a.N = N;
    a.K = K;
    return hip_status(q4::launch_linear_grad(a, workspace, as_stream(stream)));
}

// ---- gated ---------------------------------------------------------------------

int64_t q4_gated_workspace_size(int fmt, int dtype, int64_t M, int64_t N, int64_t K) {
    return forward_bytes(fmt, 2, dtype, M, N, K);
}

int q4_gated(int fmt, const uint8_t* gate_q, const uint16_t* gate_s, const uint16_t* gate_b, const uint8_t* up_q,
             const uint16_t* up_s, const uint16_t* up_b, const void* gate_bias, const void* up_bias, int act,
             const void* x, int dtype, void* h, void* gate_pre, void* up_pre, int64_t M, int64_t N, int64_t K,
             void* workspace, int64_t workspace_bytes, void* stream) {
    if (dtype != Q4_BF16 && dtype != Q4_F16) return Q4_ERR_DTYPE;
    int rc = check_product(fmt, act, M, N, K);
    if (rc) return rc;
    if ((gate_pre == nullptr) != (up_pre == nullptr)) return Q4_ERR_ARG;
    if (M == 0 || N == 0) return Q4_OK;
    if ((rc = check_planes(fmt, gate_q, gate_s, gate_b)) || (rc = check_planes(fmt, up_q, up_s, up_b)) ||
        (rc = need({x, h})) || (rc = optional({gate_bias, up_bias, gate_pre, up_pre})))
        return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, forward_bytes(fmt, 2, dtype, M, N, K)))) return rc;
    q4::LinearArgs a{};
    a.wf = format_wf(fmt);
    a.nmat = 2;
    a.act = act;
    a.dtype = dtype;
    a.w[0] = {gate_q, gate_s, gate_b};
    a.w[1] = {up_q, up_s, up_b};
    a.bias[0] = gate_bias;
    a.bias[1] = up_bias;
    a.x = x;
    a.y = h;
    a.pre[0] = gate_pre;
    a.pre[1] = up_pre;
    a.M = M;
    a.N = N;
    a.K = K;
    return hip_status(q4::launch_linear(a, workspace, as_stream(stream)));
}

int64_t q4_gated_backward_workspace_size(int fmt, int64_t M, int64_t N, int64_t K) {
    return backward_bytes(fmt, 2, M, N, K);
}

int q4_gated_backward(int fmt, const uint8_t* gate_q, const uint16_t* gate_s, const uint16_t* gate_b,
                      const uint8_t* up_q, const uint16_t* up_s, const uint16_t* up_b, int act,
                      const void* gate_pre, const void* up_pre, const void* dh, int dtype, void* dx, void* dgate,
                      void* dup, float* dgate_bias, float* dup_bias, int64_t M, int64_t N, int64_t K,
                      void* workspace, int64_t workspace_bytes, void* stream) {
    if (dtype != Q4_BF16) return Q4_ERR_DTYPE;
    int rc = check_product(fmt, act, M, N, K);
    if (rc) return rc;
    if (M == 0 || N == 0) return Q4_OK;
    if ((rc = check_planes(fmt, gate_q, gate_s, gate_b)) || (rc = check_planes(fmt, up_q, up_s, up_b)) ||
        (rc = need({gate_pre, up_pre, dh, dx})) || (rc = optional({dgate, dup, dgate_bias, dup_bias})))
        return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, backward_bytes(fmt, 2, M, N, K)))) return rc;
    q4::LinearGradArgs a{};
    a.wf = format_wf(fmt);
    a.nmat = 2;
    a.act = act;
    a.w[0] = {gate_q, gate_s, gate_b};
    a.w[1] = {up_q, up_s, up_b};
    a.pre[0] = gate_pre;
    a.pre[1] = up_pre;
    a.dy = dh;
    a.dx = dx;
    a.dz[0] = dgate;
    a.dz[1] = dup;
    a.dbias[0] = dgate_bias;
    a.dbias[1] = dup_bias;
    a.M = M;
    a.N = N;
    a.K = K;
    return hip_status(q4::launch_linear_grad(a, workspace, as_stream(stream)));
}

// ---- norms ---------------------------------------------------------------------

static int check_norm(int dtype, int r_dtype, int64_t M, int64_t D, int64_t gate_rows, float scale, int post_norm,
                      int pre_norm) {
    if (dtype != Q4_BF16 && dtype != Q4_F16 && dtype != Q4_F32) return Q4_ERR_DTYPE;
    if (r_dtype != dtype && r_dtype != Q4_F32) return Q4_ERR_DTYPE;
    if (M < 0 || D < 0 || M > kMaxDim || D > Q4_NORM_MAX_D) return Q4_ERR_SHAPE;
    if (!norm_ok(post_norm) || !norm_ok(pre_norm) || !std::isfinite(scale)) return Q4_ERR_ARG;
    if (gate_rows < 1 && M > 0) return Q4_ERR_ARG;
    return Q4_OK;
}

int block_norm(const void* y, const void* r, int dtype, int r_dtype, int64_t M, int64_t D, int post_norm,
               const void* post_weight, const void* post_bias, const void* gate, int64_t gate_rows, float scale,
               int pre_norm, const void* pre_weight, const void* pre_bias, float eps, void* r_out, void* n,
               float* stats, void* stream) {
    int rc = check_norm(dtype, r_dtype, M, D, gate_rows, scale, post_norm, pre_norm);
    if (rc) return rc;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return Q4_ERR_ARG;
    if (post_norm == Q4_NORM_NONE && (post_weight || post_bias)) return Q4_ERR_ARG;
    if (pre_norm == Q4_NORM_NONE && (pre_weight || pre_bias || n)) return Q4_ERR_ARG;
    if (M == 0 || D == 0) return Q4_OK;
    if (!y && (post_norm != Q4_NORM_NONE || gate || r_out)) return Q4_ERR_ARG;
    if ((rc = need({r})) || (y && (rc = need({r_out}))) || (pre_norm != Q4_NORM_NONE && (rc = need({n}))) ||
        (rc = optional({y, post_weight, post_bias, gate, pre_weight, pre_bias, stats})))
        return rc;
    q4::NormArgs a{};
    a.dtype = dtype;
    a.r_dtype = r_dtype;
    a.post = post_norm;
    a.pre = pre_norm;
    a.y = y;
    a.r = r;
    a.post_w = post_weight;
    a.post_b = post_bias;
    a.gate = gate;
    a.pre_w = pre_weight;
    a.pre_b = pre_bias;
    a.r_out = r_out;
    a.n = n;
    a.stats = stats;
    a.M = M;
    a.D = D;
    a.gate_rows = gate_rows;
    a.scale = scale;
    a.eps = eps;
    return hip_status(q4::launch_block_norm(a, as_stream(stream)));
}

int64_t block_norm_backward_workspace_size(int64_t M, int64_t D, int64_t gate_rows) {
    if (M <= 0 || D <= 0 || M > kMaxDim || D > Q4_NORM_MAX_D || gate_rows < 1) return 0;
    return q4::norm_grad_workspace_bytes(M, D, gate_rows);
}

int block_norm_backward(const void* y, const void* r_out, const float* stats, const void* dn, const void* dr_out,
                        int dtype, int r_dtype, int64_t M, int64_t D, int post_norm, const void* post_weight,
                        const void* post_bias, const void* gate, int64_t gate_rows, float scale, int pre_norm,
                        const void* pre_weight, void* dr, void* dy, void* dgate, float* pre_dw, float* pre_db,
                        float* post_dw, float* post_db, void* workspace, int64_t workspace_bytes, void* stream) {
    int rc = check_norm(dtype, r_dtype, M, D, gate_rows, scale, post_norm, pre_norm);
    if (rc) return rc;
    if (post_norm == Q4_NORM_NONE && (post_weight || post_bias || post_dw || post_db)) return Q4_ERR_ARG;
    if (pre_norm == Q4_NORM_NONE && (pre_weight || pre_dw || pre_db || dn)) return Q4_ERR_ARG;
    if (!gate && dgate) return Q4_ERR_ARG;
    if (M == 0 || D == 0) return Q4_OK;
    if (!y && (post_norm != Q4_NORM_NONE || gate || dy)) return Q4_ERR_ARG;
    if ((rc = need({r_out, stats, dr})) || (y && (rc = need({dy}))) || (pre_norm != Q4_NORM_NONE && (rc = need({dn}))) ||
        (!dn && (rc = need({dr_out}))) ||
        (rc = optional({y, dr_out, post_weight, post_bias, gate, pre_weight, dgate, pre_dw, pre_db, post_dw, post_db})))
        return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, q4::norm_grad_workspace_bytes(M, D, gate_rows)))) return rc;
    q4::NormGradArgs a{};
    a.dtype = dtype;
    a.r_dtype = r_dtype;
    a.post = post_norm;
    a.pre = pre_norm;
    a.y = y;
    a.r_out = r_out;
    a.stats = stats;
    a.dn = dn;
    a.dr_out = dr_out;
    a.post_w = post_weight;
    a.post_b = post_bias;
    a.gate = gate;
    a.pre_w = pre_weight;
    a.dr = dr;
    a.dy = dy;
    a.dgate = dgate;
    a.pre_dw = pre_dw;
    a.pre_db = pre_db;
    a.post_dw = post_dw;
    a.post_db = post_db;
    a.M = M;
    a.D = D;
    a.gate_rows = gate_rows;
    a.scale = scale;
    return hip_status(q4::launch_block_norm_grad(a, workspace, as_stream(stream)));
}

}  // extern "C"
