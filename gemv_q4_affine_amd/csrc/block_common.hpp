// block_common.hpp -- what the feed-forward operators' kernels share: typed
// loads and stores, the activations and their derivatives, the argument
// records, and the launchers that block_capi.cpp calls after it has validated
// every argument.
#pragma once

#include "device_common.hpp"
#include "kernels.hpp"

namespace q4 {

// codes of Q4_ACT_* and Q4_NORM_* (include/q4_block.h)
enum : int { ACT_NONE = 0, ACT_SILU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_RELU = 4 };
enum : int { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };

// A quantised matrix: Q4_0 (q = qs, s = d), affine 4-bit or 8-bit (codes,
// scales, biases), WF_* of kernels.hpp.
struct QuantW {
    const uint8_t* q;
    const uint16_t* s;
    const uint16_t* b;
};

// y = act(x W^T + bias) + residual; nmat == 2: h = act(x W0^T + bias0) *
// (x W1^T + bias1), with pre[1] the second projection.
struct LinearArgs {
    int wf, nmat, act, dtype;
    QuantW w[2];
    const void* bias[2];
    const void* residual;
    const void* x;
    void* y;
    void* pre[2];
    int64_t M, N, K;
};
// Gradients of the same: pre[] are inputs, dz[] and dbias[] outputs.
struct LinearGradArgs {
    int wf, nmat, act;
    QuantW w[2];
    const void* pre[2];
    const void* dy;
    void* dx;
    void* dz[2];
    float* dbias[2];
    int64_t M, N, K;
};
int64_t linear_workspace_bytes(int wf, int nmat, int dtype, int64_t M, int64_t N, int64_t K);
hipError_t launch_linear(const LinearArgs& a, void* workspace, hipStream_t s);
int64_t linear_grad_workspace_bytes(int wf, int nmat, int64_t M, int64_t N, int64_t K);
hipError_t launch_linear_grad(const LinearGradArgs& a, void* workspace, hipStream_t s);

struct NormArgs {
    int dtype, r_dtype, post, pre;
    const void* y;
    const void* r;
    const void* post_w;
    const void* post_b;
    const void* gate;
    const void* pre_w;
    const void* pre_b;
    void* r_out;
    void* n;
    float* stats;
    int64_t M, D, gate_rows;
    float scale, eps;
};
struct NormGradArgs {
    int dtype, r_dtype, post, pre;
    const void* y;
    const void* r_out;
    const float* stats;
    const void* dn;
    const void* dr_out;
    const void* post_w;
    const void* post_b;
    const void* gate;
    const void* pre_w;
    void* dr;
    void* dy;
    void* dgate;
    float* pre_dw;
    float* pre_db;
    float* post_dw;
    float* post_db;
    int64_t M, D, gate_rows;
    float scale;
};
hipError_t launch_block_norm(const NormArgs& a, hipStream_t s);
int64_t norm_grad_workspace_bytes(int64_t M, int64_t D, int64_t gate_rows);
hipError_t launch_block_norm_grad(const NormGradArgs& a, void* workspace, hipStream_t s);

// One direct-to-LDS copy: lane l's 16 bytes at src + voff land at LDS address
// m0 + 16 l.  Inline assembly, so that the compiler does not take it for an LDS
// store and wait for every copy in flight before each read; the kernels' own
// waits order the copies with the reads.  No register receives data.
__device__ __forceinline__ void copy_unit(const uint8_t* src, uint32_t voff, uint32_t m0) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(voff), "s"(src), "s"(m0)
                 : "memory", "m0");
}

// ---- typed element access ----------------------------------------------------

__device__ __forceinline__ float load_elem(const void* p, int dt, int64_t i) {
    if (dt == DT_F32) return static_cast<const float*>(p)[i];
    const uint16_t h = static_cast<const uint16_t*>(p)[i];
    return dt == DT_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
}
__device__ __forceinline__ void store_elem(void* p, int dt, int64_t i, float v) {
    if (dt == DT_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = (uint16_t)(dt == DT_BF16 ? f32_to_bf16(v) : f32_to_f16_rne(v));
}

// ---- activations ---------------------------------------------------------------
//
// In binary32 on the hardware exponential and reciprocal (about 1 ulp each):
//   silu       z s(z),  slope s + z s (1 - s),  s(z) = 1 / (1 + exp(-z))
//   gelu       z F(z),  slope F + z f(z), F the normal distribution function:
//              F(-|z|) = erfc(|z| / sqrt 2) / 2 by Abramowitz & Stegun 7.1.26,
//              (a1 t + .. + a5 t^5) exp(-x^2) with t = 1 / (1 + p x), absolute
//              error 1.5e-7, whose exp(-x^2) = exp(-z^2 / 2) is also f's
//   gelu_tanh  (1 + tanh v) / 2 = s(2 v), so z s(2v) has no cancellation for
//              negative z
__device__ __forceinline__ float fast_exp(float v) { return __builtin_amdgcn_exp2f(v * 1.44269504088896f); }
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + fast_exp(-v)); }

// Activation ACT of z, and with GRAD its derivative in `slope`.
template <int ACT, bool GRAD>
__device__ __forceinline__ float activate(float z, float& slope) {
    if constexpr (ACT == ACT_SILU) {
        const float s = sigmoid(z);
        if constexpr (GRAD) slope = fmaf(z, s * (1.0f - s), s);
        return z * s;
    } else if constexpr (ACT == ACT_GELU) {
        const float x = fabsf(z) * 0.707106781186548f;
        const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, x, 1.0f));
        const float e = fast_exp(-x * x);
        float q = fmaf(t, 1.061405429f, -1.453152027f);
        q = fmaf(t, q, 1.421413741f);
        q = fmaf(t, q, -0.284496736f);
        q = fmaf(t, q, 0.254829592f);
        q = 0.5f * q * t * e;                     // F(-|z|)
        const float F = z < 0.0f ? q : 1.0f - q;
        if constexpr (GRAD) slope = fmaf(z * 0.398942280401433f, e, F);
        return z * F;
    } else if constexpr (ACT == ACT_GELU_TANH) {
        constexpr float c = 1.59576912160573f;     // 2 sqrt(2 / pi)
        const float z2 = z * z;
        const float s = sigmoid(c * z * fmaf(0.044715f, z2, 1.0f));
        if constexpr (GRAD) {
            // s (1 - s) is zero from |z| = 16 on (and far before), where the cubic may overflow later
            const float b = __builtin_amdgcn_fmed3f(z, -16.0f, 16.0f);
            slope = fmaf(b * c * fmaf(0.134145f, b * b, 1.0f), s * (1.0f - s), s);
        }
        return z * s;
    } else if constexpr (ACT == ACT_RELU) {
        if constexpr (GRAD) slope = z > 0.0f ? 1.0f : 0.0f;
        return z < 0.0f ? 0.0f : z;        // a NaN stays one
    } else {
        if constexpr (GRAD) slope = 1.0f;
        return z;
    }
}
// N values at once: one branch on the activation, then independent chains (a
// branch at every value kept eight exponentials from overlapping).
template <int ACT, bool GRAD, int N>
__device__ __forceinline__ void activate_as(const float (&z)[N], float (&v)[N], float (&slope)[N]) {
#pragma unroll
    for (int e = 0; e < N; e++) v[e] = activate<ACT, GRAD>(z[e], slope[e]);
}
template <bool GRAD, int N>
__device__ __forceinline__ void activate_all(int act, const float (&z)[N], float (&v)[N], float (&slope)[N]) {
    switch (act) {
        case ACT_SILU: activate_as<ACT_SILU, GRAD>(z, v, slope); break;
        case ACT_GELU: activate_as<ACT_GELU, GRAD>(z, v, slope); break;
        case ACT_GELU_TANH: activate_as<ACT_GELU_TANH, GRAD>(z, v, slope); break;
        case ACT_RELU: activate_as<ACT_RELU, GRAD>(z, v, slope); break;
        default: activate_as<ACT_NONE, GRAD>(z, v, slope);
    }
}

}  // namespace q4
