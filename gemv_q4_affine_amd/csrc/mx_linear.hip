// mx_linear.hip -- mx_linear and mx_gated: which kernels a call takes.
#include "mx_few.hpp"
#include "mx_tile.hpp"

namespace q4 {

namespace {

bool is_mx(int x_type) { return x_type == XT_MXFP4 || x_type == XT_MXFP8; }

}  // namespace

int64_t mx_linear_workspace_bytes(int x_type, int nmat, int64_t M, int64_t N, int64_t K) {
    if (mx_few_takes(x_type, nmat, M, N, K)) return 0;
    return is_mx(x_type) ? mx_tile_workspace_bytes(x_type, nmat, M, N, K) : linear_workspace_bytes(WF_MXFP4, nmat, x_type, M, N, K);
}

hipError_t launch_mx_linear(const MxLinearArgs& p, void* workspace, hipStream_t s) {
    if (mx_few_takes(p.x_type, p.a.nmat, p.a.M, p.a.N, p.a.K)) return launch_mx_few(p, s);
    return is_mx(p.x_type) ? launch_mx_tile(p, epilogue_args(p.a), workspace, s) : launch_linear(p.a, workspace, s);
}

}  // namespace q4
