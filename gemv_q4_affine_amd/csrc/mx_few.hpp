// mx_few.hpp -- the few-row product on MXFP4 weights (mx_few.hip).
#pragma once

#include "mx_common.hpp"

namespace q4 {

// Whether a product goes to launch_mx_few, else to the tile products (mx_tile.hip,
// linear.hip: 16-bit x there must have more than 64 rows).
bool mx_few_takes(int x_type, int nmat, int64_t M, int64_t N, int64_t K);

// Waves of a workgroup along the sum and along the rows of W, row tiles of a wave.
struct MxFewPlan {
    int kw, rw, r;
};
hipError_t launch_mx_few(const MxLinearArgs& a, hipStream_t s);

// Pair B of the eight 4-bit codes of a word times its scale, in bfloat16 (exact).
template <int B>
__device__ __forceinline__ uint32_t bf16_pair(uint32_t w, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, B));
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
