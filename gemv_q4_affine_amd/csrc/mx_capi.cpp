// mx_capi.cpp -- the exported C ABI of the operators on microscaled numbers
// (include/q4_mx.h): argument validation and the launches.
//
// Every check runs on the host before any HIP call, so a rejected call
// enqueues nothing and the checks work on a machine without a GPU.
#include "q4_mx.h"

#include <cmath>
#include <cstdint>

#include "capi_checks.hpp"
#include "mx_common.hpp"

namespace {

using namespace q4::checks;

bool mx_type_ok(int type) { return type == Q4_MXFP4 || type == Q4_MXFP8; }
bool dtype16(int dtype) { return dtype == Q4_BF16 || dtype == Q4_F16; }

int check_product(int act, int64_t M, int64_t N, int64_t K) {
    if (!act_ok(act)) return Q4_ERR_ARG;
    if (M < 0 || N < 0 || K <= 0 || K % 32 != 0 || M > kMaxDim || N > kMaxSum || K > kMaxSum) return Q4_ERR_SHAPE;
    return Q4_OK;
}
int check_x(int x_type, int dtype) {
    if (!dtype16(dtype)) return Q4_ERR_DTYPE;
    return mx_type_ok(x_type) || x_type == dtype ? Q4_OK : Q4_ERR_DTYPE;
}
// x of an MX type has scales, a 16-bit one none.
int check_x_planes(int x_type, const void* x, const void* x_s) {
    if (mx_type_ok(x_type)) return need({x, x_s});
    return x_s ? Q4_ERR_ARG : need({x});
}

int64_t forward_bytes(int x_type, int nmat, int64_t M, int64_t N, int64_t K) {
    if (!mx_type_ok(x_type) && !dtype16(x_type)) return 0;
    if (check_product(Q4_ACT_NONE, M, N, K) != Q4_OK || M == 0 || N == 0) return 0;
    return q4::mx_linear_workspace_bytes(x_type, nmat, M, N, K);
}
int64_t backward_bytes(int nmat, int64_t M, int64_t N, int64_t K) {
    if (check_product(Q4_ACT_NONE, M, N, K) != Q4_OK || M == 0 || N == 0) return 0;
    return q4::linear_grad_workspace_bytes(q4::WF_MXFP4, nmat, M, N, K);
}

q4::QuantW planes(const uint8_t* q, const uint8_t* s) { return {q, reinterpret_cast<const uint16_t*>(s), nullptr}; }

int check_mx_plane_call(const void* v, int dtype, int type, const void* codes, const void* scales, int64_t M, int64_t K) {
    if (dtype != Q4_F32 && !dtype16(dtype)) return Q4_ERR_DTYPE;
    if (!mx_type_ok(type)) return Q4_ERR_DTYPE;
    if (M < 0 || M > kMaxDim || K <= 0 || K > kMaxDim || K % 32 != 0) return Q4_ERR_SHAPE;
    return M == 0 ? Q4_OK : need({v, codes, scales});
}

}  // namespace

extern "C" {

int mx_quantize(const void* v, int dtype, int type, uint8_t* codes, uint8_t* scales, int64_t M, int64_t K, void* stream) {
    const int rc = check_mx_plane_call(v, dtype, type, codes, scales, M, K);
    if (rc || M == 0) return rc;
    return hip_status(q4::launch_mx_quantize(v, dtype, type, codes, scales, M, K, as_stream(stream)));
}

int mx_dequantize(int type, const uint8_t* codes, const uint8_t* scales, void* v, int dtype, int64_t M, int64_t K,
                  void* stream) {
    const int rc = check_mx_plane_call(v, dtype, type, codes, scales, M, K);
    if (rc || M == 0) return rc;
    return hip_status(q4::launch_mx_dequantize(type, codes, scales, v, dtype, M, K, as_stream(stream)));
}

int64_t mx_linear_workspace_size(int x_type, int64_t M, int64_t N, int64_t K) { return forward_bytes(x_type, 1, M, N, K); }

int mx_linear(const uint8_t* w_q, const uint8_t* w_s, const void* bias, int act, const void* residual, int x_type,
              const void* x, const uint8_t* x_s, int dtype, void* y, void* pre, int64_t M, int64_t N, int64_t K,
              void* workspace, int64_t workspace_bytes, void* stream) {
    int rc = check_x(x_type, dtype);
    if (rc || (rc = check_product(act, M, N, K))) return rc;
    if (M == 0 || N == 0) return Q4_OK;
    if ((rc = need({w_q, w_s, y})) || (rc = check_x_planes(x_type, x, x_s)) || (rc = optional({bias, residual, pre}))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, forward_bytes(x_type, 1, M, N, K)))) return rc;
    q4::MxLinearArgs p{};
    p.x_type = x_type;
    p.x_s = x_s;
    p.a.wf = q4::WF_MXFP4;
    p.a.nmat = 1;
    p.a.act = act;
    p.a.dtype = dtype;
    p.a.w[0] = planes(w_q, w_s);
    p.a.bias[0] = bias;
    p.a.residual = residual;
    p.a.x = x;
    p.a.y = y;
    p.a.pre[0] = pre;
    p.a.M = M;
    p.a.N = N;
    p.a.K = K;
    return hip_status(q4::launch_mx_linear(p, workspace, as_stream(stream)));
}

int64_t mx_linear_backward_workspace_size(int64_t M, int64_t N, int64_t K) { return backward_bytes(1, M, N, K); }

int mx_linear_backward(const uint8_t* w_q, const uint8_t* w_s, int act, const void* pre, const void* dy, int dtype,
                       void* dx, void* dz, float* dbias, int64_t M, int64_t N, int64_t K, void* workspace,
                       int64_t workspace_bytes, void* stream) {
    if (dtype != Q4_BF16) return Q4_ERR_DTYPE;
    int rc = check_product(act, M, N, K);
    if (rc) return rc;
    if (act == Q4_ACT_NONE && dz) return Q4_ERR_ARG;
    if (M == 0 || N == 0) return Q4_OK;
    if ((rc = need({w_q, w_s, dy, dx})) || (rc = optional({pre, dz, dbias}))) return rc;
    if (act != Q4_ACT_NONE && !pre) return Q4_ERR_NULL;
    if ((rc = check_workspace(workspace, workspace_bytes, backward_bytes(1, M, N, K)))) return rc;
    q4::LinearGradArgs a{};
    a.wf = q4::WF_MXFP4;
    a.nmat = 1;
    a.act = act;
    a.w[0] = planes(w_q, w_s);
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

int64_t mx_gated_workspace_size(int x_type, int64_t M, int64_t N, int64_t K) { return forward_bytes(x_type, 2, M, N, K); }

int mx_gated(const uint8_t* gate_q, const uint8_t* gate_s, const uint8_t* up_q, const uint8_t* up_s,
             const void* gate_bias, const void* up_bias, int act, int x_type, const void* x, const uint8_t* x_s,
             int dtype, void* h, void* gate_pre, void* up_pre, int64_t M, int64_t N, int64_t K, void* workspace,
             int64_t workspace_bytes, void* stream) {
    int rc = check_x(x_type, dtype);
    if (rc || (rc = check_product(act, M, N, K))) return rc;
    if ((gate_pre == nullptr) != (up_pre == nullptr)) return Q4_ERR_ARG;
    if (M == 0 || N == 0) return Q4_OK;
    if ((rc = need({gate_q, gate_s, up_q, up_s, h})) || (rc = check_x_planes(x_type, x, x_s)) ||
        (rc = optional({gate_bias, up_bias, gate_pre, up_pre})))
        return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, forward_bytes(x_type, 2, M, N, K)))) return rc;
    q4::MxLinearArgs p{};
    p.x_type = x_type;
    p.x_s = x_s;
    p.a.wf = q4::WF_MXFP4;
    p.a.nmat = 2;
    p.a.act = act;
    p.a.dtype = dtype;
    p.a.w[0] = planes(gate_q, gate_s);
    p.a.w[1] = planes(up_q, up_s);
    p.a.bias[0] = gate_bias;
    p.a.bias[1] = up_bias;
    p.a.x = x;
    p.a.y = h;
    p.a.pre[0] = gate_pre;
    p.a.pre[1] = up_pre;
    p.a.M = M;
    p.a.N = N;
    p.a.K = K;
    return hip_status(q4::launch_mx_linear(p, workspace, as_stream(stream)));
}

int64_t mx_gated_backward_workspace_size(int64_t M, int64_t N, int64_t K) { return backward_bytes(2, M, N, K); }

int mx_gated_backward(const uint8_t* gate_q, const uint8_t* gate_s, const uint8_t* up_q, const uint8_t* up_s, int act,
                      const void* gate_pre, const void* up_pre, const void* dh, int dtype, void* dx, void* dgate,
                      void* dup, float* dgate_bias, float* dup_bias, int64_t M, int64_t N, int64_t K,
                      void* workspace, int64_t workspace_bytes, void* stream) {
    if (dtype != Q4_BF16) return Q4_ERR_DTYPE;
    int rc = check_product(act, M, N, K);
    if (rc) return rc;
    if (M == 0 || N == 0) return Q4_OK;
    if ((rc = need({gate_q, gate_s, up_q, up_s, gate_pre, up_pre, dh, dx})) ||
        (rc = optional({dgate, dup, dgate_bias, dup_bias})))
        return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, backward_bytes(2, M, N, K)))) return rc;
    q4::LinearGradArgs a{};
    a.wf = q4::WF_MXFP4;
    a.nmat = 2;
    a.act = act;
    a.w[0] = planes(gate_q, gate_s);
    a.w[1] = planes(up_q, up_s);
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

int block_norm_mx(const void* y, const void* r, int dtype, int r_dtype, int64_t M, int64_t D, int post_norm,
                  const void* post_weight, const void* post_bias, const void* gate, int64_t gate_rows, float scale,
                  int pre_norm, const void* pre_weight, const void* pre_bias, float eps, void* r_out, int n_type,
                  uint8_t* n_codes, uint8_t* n_scales, float* stats, void* stream) {
    int rc = check_norm(dtype, r_dtype, M, D, gate_rows, scale, post_norm, pre_norm);
    if (rc) return rc;
    if (!mx_type_ok(n_type)) return Q4_ERR_DTYPE;
    if (D % 32 != 0) return Q4_ERR_SHAPE;
    if (!(eps > 0.0f) || !std::isfinite(eps) || pre_norm == Q4_NORM_NONE) return Q4_ERR_ARG;
    if (post_norm == Q4_NORM_NONE && (post_weight || post_bias)) return Q4_ERR_ARG;
    if (M == 0 || D == 0) return Q4_OK;
    if (!y && (post_norm != Q4_NORM_NONE || gate || r_out)) return Q4_ERR_ARG;
    if ((rc = need({r, n_codes, n_scales})) || (y && (rc = need({r_out}))) ||
        (rc = optional({y, post_weight, post_bias, gate, pre_weight, pre_bias, stats})))
        return rc;
    q4::MxNormArgs p{};
    p.n_type = n_type;
    p.codes = n_codes;
    p.scales = n_scales;
    q4::NormArgs& a = p.norm;
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
    a.stats = stats;
    a.M = M;
    a.D = D;
    a.gate_rows = gate_rows;
    a.scale = scale;
    a.eps = eps;
    return hip_status(q4::launch_block_norm_mx(p, as_stream(stream)));
}

}  // extern "C"
