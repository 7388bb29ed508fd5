// mx_common.hpp -- what the kernels on microscaled (MX) numbers share: the type
// codes, scales, the rounding to codes, the argument records and the launchers
// that mx_capi.cpp calls after it has validated every argument.
#pragma once

#include "block_common.hpp"

namespace q4 {

// codes of Q4_MXFP4 and Q4_MXFP8 (include/q4_mx.h), beside DT_BF16 and DT_F16
enum : int { XT_MXFP4 = 8, XT_MXFP8 = 9 };

hipError_t launch_mx_quantize(const void* v, int dtype, int type, uint8_t* codes, uint8_t* scales, int64_t M, int64_t K,
                              hipStream_t s);
hipError_t launch_mx_dequantize(int type, const uint8_t* codes, const uint8_t* scales, void* v, int dtype, int64_t M,
                                int64_t K, hipStream_t s);

struct MxNormArgs {
    NormArgs norm;             // n unused
    int n_type;
    uint8_t* codes;
    uint8_t* scales;
};
hipError_t launch_block_norm_mx(const MxNormArgs& a, hipStream_t s);

// The product of LinearArgs with x of x_type (MX: planes a.x and x_s) and W in
// MXFP4 (w[].q codes, w[].s its scales' bytes).
struct MxLinearArgs {
    LinearArgs a;              // wf WF_MXFP4
    int x_type;
    const uint8_t* x_s;
};
int64_t mx_linear_workspace_bytes(int x_type, int nmat, int64_t M, int64_t N, int64_t K);
hipError_t launch_mx_linear(const MxLinearArgs& a, void* workspace, hipStream_t s);

// ---- scales and codes ---------------------------------------------------------------

// 2^(s - 127) in binary32: exponent s, but for the ends (subnormal, NaN).
__device__ __forceinline__ float mx_scale(uint32_t s) {
    return __uint_as_float(s == 0u ? 0x00400000u : s == 255u ? 0x7FC00000u : s << 23);
}

// The scale byte of a block from the largest |value|'s bits: its exponent less
// e, at least 0; 255 where it is an infinity or a NaN.
template <int TYPE>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
    constexpr uint32_t e = TYPE == XT_MXFP4 ? 2u : 8u;
    const uint32_t x = amax >> 23;
    return x == 255u ? 255u : x > e ? x - e : 0u;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Eight values to codes under a block's scale byte: one dword (4 bits) or two.
// The hardware's conversions divide by the scale's power of two and round to
// nearest even; the 4-bit one saturates, the 8-bit one makes a NaN of what
// lies past 448, so that its values are cut first.
typedef short i16x2_t __attribute__((ext_vector_type(2)));
template <int TYPE>
__device__ __forceinline__ u32x2_t mx_codes8(const float (&v)[8], uint32_t scale_byte) {
    if (scale_byte == 255u) return u32x2_t{0u, 0u};
    const float s = mx_scale(scale_byte);
    u32x2_t r = {0u, 0u};
    if constexpr (TYPE == XT_MXFP4) {
        uint32_t q = 0u;
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], s, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], s, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], s, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], s, 3);
        r[0] = q;
    } else {
        const float top = 448.0f * s;
        float c[8];
#pragma unroll
        for (int e = 0; e < 8; e++) c[e] = __builtin_amdgcn_fmed3f(v[e], -top, top);
#pragma unroll
        for (int h = 0; h < 2; h++) {
            i16x2_t q = {0, 0};
            q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, c[4 * h], c[4 * h + 1], s, false);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(q, c[4 * h + 2], c[4 * h + 3], s, true);
            r[h] = __builtin_bit_cast(uint32_t, q);
        }
    }
    return r;
}

// The eight codes of a word times a quarter of their scale in bfloat16, exact under any:
// 2^-130, the least, is a subnormal number of it, and 6 * 2^125 the largest.
__device__ __forceinline__ u32x4_t bf16_quarters(uint32_t w, float s) {
    const float f = 0.25f * s;
    auto pair = [&](f32x2_t v) __attribute__((always_inline)) {
        const f32x2_t t = {v[0] * f, v[1] * f};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(t, bf16x2_t));
    };
    return u32x4_t{pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0)), pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1)),
                   pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2)), pair(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3))};
}

// Maximum over the four lanes of an aligned quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    uint32_t t = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false);
    v = t > v ? t : v;
    t = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false);
    return t > v ? t : v;
}

}  // namespace q4
