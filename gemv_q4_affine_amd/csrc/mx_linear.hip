// mx_linear.hip -- mx_linear and mx_gated: which kernels a call takes.
#include "mx_tile.hpp"

namespace q4 {

namespace {

// Value k of a row of x, without its block's scale.
__device__ __forceinline__ float x_value(const MxLinearArgs& p, int64_t m, int64_t k) {
    const int64_t i = m * p.a.K + k;
    const uint8_t* q = static_cast<const uint8_t*>(p.a.x);
    if (p.x_type == XT_MXFP4) {
        const f32x2_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((uint32_t)q[i >> 1], 1.0f, 0);
        return v[i & 1];
    }
    if (p.x_type == XT_MXFP8) return __builtin_amdgcn_cvt_f32_fp8((int)q[i], 0);
    return load_elem(p.a.x, p.a.dtype, i);
}

__global__ __launch_bounds__(256) void k_mx_plain(const MxLinearArgs p) {
    const LinearArgs& a = p.a;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= a.M * a.N) return;
    const int64_t m = id / a.N, n = id % a.N;
    float z[2] = {0.0f, 0.0f};
    for (int64_t b = 0; b < a.K / 32; b++)
        for (int t = 0; t < a.nmat; t++) {
            // the scales' product: either alone may leave binary32's range
            const int ws = reinterpret_cast<const uint8_t*>(a.w[t].s)[n * (a.K / 32) + b];
            const int xs = p.x_s ? p.x_s[m * (a.K / 32) + b] : 127;
            float d = ws == 255 || xs == 255 ? __builtin_nanf("") : 0.0f;
            for (int e = 0; e < 32; e += 2) {
                const f32x2_t w = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4((uint32_t)a.w[t].q[(n * a.K + b * 32 + e) >> 1], 1.0f, 0);
                d = fmaf(w[0], x_value(p, m, b * 32 + e), d);
                d = fmaf(w[1], x_value(p, m, b * 32 + e + 1), d);
            }
            z[t] += ldexpf(d, ws + xs - 254);
        }
    for (int t = 0; t < a.nmat; t++) {
        if (a.bias[t]) z[t] += load_elem(a.bias[t], a.dtype, n);
        if (a.pre[t]) store_elem(a.pre[t], a.dtype, id, z[t]);
    }
    float zs[1] = {z[0]}, none[1];
    activate_all<false>(a.act, zs, zs, none);
    float y = zs[0];
    if (a.nmat == 2) y *= z[1];
    if (a.residual) y += load_elem(a.residual, a.dtype, id);
    store_elem(a.y, a.dtype, id, y);
}

constexpr int64_t kFewMaxM = 64;

bool is_mx(int x_type) { return x_type == XT_MXFP4 || x_type == XT_MXFP8; }

EpilogueArgs epilogue_args(const LinearArgs& a) {
    EpilogueArgs e{};
    e.act = a.act;
    e.dtype = a.dtype;
    e.M = a.M;
    e.N = a.N;
    for (int i = 0; i < 2; i++) {
        e.bias[i] = a.bias[i];
        e.pre[i] = a.pre[i];
    }
    e.residual = a.residual;
    e.y = a.y;
    return e;
}

}  // namespace

int64_t mx_linear_workspace_bytes(int x_type, int nmat, int64_t M, int64_t N, int64_t K) {
    if (M <= kFewMaxM) return 0;
    return is_mx(x_type) ? mx_tile_workspace_bytes(x_type, nmat, M, N, K) : linear_workspace_bytes(WF_MXFP4, nmat, x_type, M, N, K);
}

hipError_t launch_mx_linear(const MxLinearArgs& p, void* workspace, hipStream_t s) {
    if (p.a.M > kFewMaxM)
        return is_mx(p.x_type) ? launch_mx_tile(p, epilogue_args(p.a), workspace, s) : launch_linear(p.a, workspace, s);
    const int64_t blocks = (p.a.M * p.a.N + 255) / 256;
    if (!launchable(blocks, 256)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_mx_plain, dim3((unsigned)blocks), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace q4
