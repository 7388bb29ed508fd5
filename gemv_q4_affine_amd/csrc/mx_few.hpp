// mx_few.hpp -- the few-row product on MXFP4 weights (mx_few.hip).
#pragma once

#include "mx_common.hpp"
#include "mx_few_plan.hpp"

namespace q4 {

// Whether a product goes to launch_mx_few, else to the tile products (mx_tile.hip,
// linear.hip: 16-bit x there must have more than 64 rows).
bool mx_few_takes(int x_type, int nmat, int64_t M, int64_t N, int64_t K);

hipError_t launch_mx_few(const MxLinearArgs& a, hipStream_t s);

// 16-bit x: W's codes are multiplied in bfloat16, which holds them under every scale up to
// 2^125; under 2^126 and 2^127 the largest codes are past its range.  Such a block counts as
// one under 2^-127 (2^-253 of its terms, and what an infinity or a NaN in x makes of them) and
// sets `past`; its terms are added from quarters of them.
__device__ __forceinline__ bool past_bf16(uint32_t scale_byte) { return scale_byte == 253u || scale_byte == 254u; }
__device__ __forceinline__ float bf16_scale(uint32_t s, bool& past) {
    past |= s >= 253u;                         // (a NaN scale adds nothing there)
    return __uint_as_float(s - 1u >= 252u ? (s == 255u ? 0x7FC00000u : 0x00400000u) : s << 23);
}
// Pair B of the eight 4-bit codes of a word times such a scale, in bfloat16 (exact).
template <int B>
__device__ __forceinline__ uint32_t bf16_pair(uint32_t w, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, B));
}

// 16-bit values with zeros in the place of infinities and NaN.
template <int DT>
__device__ __forceinline__ u32x4_t finite16(const u32x4_t& v) {
    constexpr uint32_t top = DT == DT_BF16 ? 0x7F80u : 0x7C00u;
    u32x4_t r;
#pragma unroll
    for (int e = 0; e < 4; e++)
        r[e] = ((v[e] & top) == top ? 0u : v[e] & 0xFFFFu) | ((v[e] >> 16 & top) == top ? 0u : v[e] & 0xFFFF0000u);
    return r;
}

// Binary16 values as the sums of two bfloat16 ones: the upper 8 bits, and what
// they leave of the 11 (nothing of an infinity or a NaN).
__device__ __forceinline__ void split_f16(const u32x4_t& v, u32x4_t& hi, u32x4_t& lo) {
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const float a = f16_to_f32(v[e] & 0xFFFFu), b = f16_to_f32(v[e] >> 16);
        // cut to 8 bits: what is left has 3 and fits too
        const uint32_t ha = __float_as_uint(a) & 0xFFFF0000u, hb = __float_as_uint(b) & 0xFFFF0000u;
        const float la = a - __uint_as_float(ha), lb = b - __uint_as_float(hb);
        hi[e] = (ha >> 16) | hb;
        const uint32_t ra = la == la ? __float_as_uint(la) : 0u, rb = lb == lb ? __float_as_uint(lb) : 0u;
        lo[e] = (ra >> 16) | (rb & 0xFFFF0000u);
    }
}

}  // namespace q4
