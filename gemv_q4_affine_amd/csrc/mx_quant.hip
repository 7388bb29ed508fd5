// mx_quant.hip -- mx_quantize and mx_dequantize.
//
// A lane takes eight consecutive values, four lanes a block of 32: the block's
// largest |value| is the maximum of the magnitudes' bit patterns (which also
// orders infinities and NaNs above every number) over the quad.  Eight values a
// lane make a wave's reads and writes whole lines in both directions, and the
// conversions are the hardware's, four instructions a lane.  Bound by memory, one read
// and one write of each value: 12288 x 4096 bfloat16 to 4 bits 19.6 us and back
// 19.4 (127 MB, 6.5 TB/s, part of it from the last-level cache; a large copy moves 5.2),
// 1001 x 8192 to 8 bits 5.0 (25 MB).
#include "mx_common.hpp"
#include "tile_image.hpp"

namespace q4 {

namespace {

template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
    if constexpr (DT == DT_F32) {
        const floatx4_t* q = reinterpret_cast<const floatx4_t*>(static_cast<const float*>(p) + i);
        const floatx4_t lo = q[0], hi = q[1];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            v[e] = lo[e];
            v[4 + e] = hi[e];
        }
    } else {
        unpack8(DT, load8_raw<true>(p, i, 8), v);
    }
}

constexpr int kThreads = 256;

// Pieces of eight values: thread, + the grid's threads ..; `pieces` is a
// multiple of four and so is the grid's step, so a quad's lanes share a block.
template <int DT, int TYPE>
__global__ __launch_bounds__(kThreads) void k_mx_quantize(const void* __restrict__ v, int64_t pieces,
                                                          uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    for (int64_t p = (int64_t)blockIdx.x * kThreads + threadIdx.x; p < pieces; p += (int64_t)gridDim.x * kThreads) {
        float f[8];
        load8<DT>(v, p * 8, f);
        uint32_t top = 0u;
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const uint32_t b = abs_bits(f[e]);
            top = b > top ? b : top;
        }
        const uint32_t s = mx_scale_byte<TYPE>(quad_max(top));
        const u32x2_t q = mx_codes8<TYPE>(f, s);
        if constexpr (TYPE == XT_MXFP4) reinterpret_cast<uint32_t*>(codes)[p] = q[0];
        else reinterpret_cast<u32x2_t*>(codes)[p] = q;
        if ((p & 3) == 0) scales[p >> 2] = (uint8_t)s;
    }
}

template <int DT, int TYPE>
__global__ __launch_bounds__(kThreads) void k_mx_dequantize(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t pieces,
                                                            void* __restrict__ v) {
    for (int64_t p = (int64_t)blockIdx.x * kThreads + threadIdx.x; p < pieces; p += (int64_t)gridDim.x * kThreads) {
        const float s = mx_scale(scales[p >> 2]);
        float f[8];
        f32x2_t t[4];
        // unscaled first: the conversion's own scaling may flush what binary32 still holds
        if constexpr (TYPE == XT_MXFP4) {
            const uint32_t q = reinterpret_cast<const uint32_t*>(codes)[p];
            t[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0);
            t[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1);
            t[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2);
            t[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
        } else {
            const u32x2_t q = reinterpret_cast<const u32x2_t*>(codes)[p];
            t[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[0], 1.0f, false);
            t[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[0], 1.0f, true);
            t[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[1], 1.0f, false);
            t[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q[1], 1.0f, true);
        }
#pragma unroll
        for (int e = 0; e < 8; e++) f[e] = t[e >> 1][e & 1] * s;
        if constexpr (DT == DT_F32) {
            floatx4_t* o = reinterpret_cast<floatx4_t*>(static_cast<float*>(v) + p * 8);
            o[0] = floatx4_t{f[0], f[1], f[2], f[3]};
            o[1] = floatx4_t{f[4], f[5], f[6], f[7]};
        } else {
            reinterpret_cast<u32x4_t*>(v)[p] = pack8(DT, f);
        }
    }
}

unsigned grid_of(int64_t pieces) {
    const int64_t blocks = (pieces + kThreads - 1) / kThreads, most = (int64_t)current_cu_count() * 32;
    return (unsigned)(blocks < most ? blocks : most);
}

template <int DT>
void quantize_t(const void* v, int type, uint8_t* codes, uint8_t* scales, int64_t pieces, hipStream_t s) {
    auto k = type == XT_MXFP4 ? k_mx_quantize<DT, XT_MXFP4> : k_mx_quantize<DT, XT_MXFP8>;
    hipLaunchKernelGGL(k, dim3(grid_of(pieces)), dim3(kThreads), 0, s, v, pieces, codes, scales);
}
template <int DT>
void dequantize_t(int type, const uint8_t* codes, const uint8_t* scales, void* v, int64_t pieces, hipStream_t s) {
    auto k = type == XT_MXFP4 ? k_mx_dequantize<DT, XT_MXFP4> : k_mx_dequantize<DT, XT_MXFP8>;
    hipLaunchKernelGGL(k, dim3(grid_of(pieces)), dim3(kThreads), 0, s, codes, scales, pieces, v);
}

}  // namespace

hipError_t launch_mx_quantize(const void* v, int dtype, int type, uint8_t* codes, uint8_t* scales, int64_t M, int64_t K,
                              hipStream_t s) {
    const int64_t pieces = M * (K / 8);
    if (dtype == DT_F32) quantize_t<DT_F32>(v, type, codes, scales, pieces, s);
    else if (dtype == DT_BF16) quantize_t<DT_BF16>(v, type, codes, scales, pieces, s);
    else quantize_t<DT_F16>(v, type, codes, scales, pieces, s);
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(int type, const uint8_t* codes, const uint8_t* scales, void* v, int dtype, int64_t M,
                                int64_t K, hipStream_t s) {
    const int64_t pieces = M * (K / 8);
    if (dtype == DT_F32) dequantize_t<DT_F32>(type, codes, scales, v, pieces, s);
    else if (dtype == DT_BF16) dequantize_t<DT_BF16>(type, codes, scales, v, pieces, s);
    else dequantize_t<DT_F16>(type, codes, scales, v, pieces, s);
    return hipGetLastError();
}

}  // namespace q4
