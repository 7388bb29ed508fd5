// tile_image.hpp -- the 16-bit operand images of the dense matrix-core
// product (tile_gemm.hip) and the packers' device helpers (tile_pack.hip).
//
// An image holds the rows of an operand (weights or activations), in binary16 or
// bfloat16, in the order in which v_mfma_f32_32x32x16_f16 (_bf16) reads them.  Rows go in panels of 32, the
// summed index k in slices of 16; the unit of panel p and slice s is 1 KiB:
// lane l's 16 bytes are row 32 p + (l & 31), k = 16 s + 8 (l >> 5) .. + 7.
// Units of a panel are contiguous (slices first), so
//   * a direct-to-LDS copy moves one unit with one instruction,
//   * a wave reads an operand fragment with one ds_read_b128 at lane * 16: no
//     bank conflict, no address arithmetic, and
//   * a tile of any number of panels finds its data without repacking.
// The slice count is even (k padded to 32 with zeros on both operands).
#pragma once

#include "block_common.hpp"
#include "gemm_common.hpp"
#include "launch_limits.hpp"

namespace q4 {

constexpr int kUnit = 1024;                 // bytes of a unit

// Slices of a sum over K terms.
inline int64_t image_slices(int64_t K) { return (K + 31) / 32 * 2; }

// Epilogue of the product (one of them is chosen at compile time).
enum : int {
    EPI_LINEAR = 0,    // y = act(z + bias) + residual, pre = z + bias
    EPI_GATED = 1,     // panels alternate gate, up: h = act(g + bias0) * (u + bias1)
    EPI_PARTIAL = 2    // binary32 sums of a part of the slices, joined by a kernel of their own
};

struct EpilogueArgs {
    int act, dtype;
    int64_t M, N;              // of the output
    const void* bias[2];
    const void* residual;
    void* y;
    void* pre[2];
    // MXFP4: a scale byte for each row of the weights' image (padded to whole panels), which holds
    // it under 2^13 in the place of 2^(byte - 127).  Null: as they are.
    const uint8_t* w_scale[2];
};
constexpr int kRowScale = 127 + 13;
inline EpilogueArgs epilogue_args(const LinearArgs& a) {
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

// The bias gradients: sums over groups of rows, [groups][nmat][N], joined in order
// into the columns of out (null: none).
struct SumsArgs {
    const float* sums;
    int64_t groups, N;
    int nmat;
    float* out[2];
};

// One product Z[m][n] = sum_k X[m][k] W[n][k] over two images.
struct TileArgs {
    const uint8_t* wimg;
    const uint8_t* ximg;
    const int8_t* xexp;        // row m of the x image holds x * 2^xexp[m] (null: see unit)
    bool bf16;                 // images in bfloat16 (no xexp), else in binary16
    int64_t slices;            // of both images
    int64_t w_panels, x_panels;
    int parts;                 // parts of the slices (EPI_PARTIAL), else 1
    float* part;               // [parts][M][N'] sums as they were added up, N' = w_panels * 32
    float unit;                // of them where there is no xexp
    EpilogueArgs epi;
    SumsArgs sums;             // nmat 0: none; joined with the parts
};

// The plan of a product: tile shape (panels of a wave: a workgroup's tile is
// 2 NT x 2 MT panels) and the parts the sum is split into.
struct TilePlan {
    int nt, mt, parts;
};
TilePlan plan_tiles(int nmat, int64_t M, int64_t N, int64_t K);
int64_t partial_bytes(const TilePlan& p, int64_t M, int64_t w_panels);

hipError_t launch_tile_gemm(const TilePlan& p, int nmat, const TileArgs& a, hipStream_t s);
// The parts of a split sum, joined, and the epilogue.
hipError_t launch_tile_join(int nmat, const TileArgs& a, hipStream_t s);
// The weights as rows n (image of W) or as rows k (image of W^T, summed over
// n); `mats` matrices side by side: panels alternate (rows n) or slices follow
// each other (rows k).
enum : int {
    IMG_F16 = 0,       // in binary16
    IMG_REST = 1,      // rows n: after K terms the roundings' remainders; the activations' image then holds its rows twice
    IMG_ROWS = 2,      // MXFP4: a power of two for each row, from `scales`, into scales.out
    IMG_QUARTER = 3    // MXFP4, rows n: quarters in bfloat16
};
// The largest scale bytes of MXFP4 weights, for IMG_ROWS: found beside the packing of the
// activations or gradients, which comes first.
struct ScaleArgs {
    const uint8_t* s[2];
    int mats;                  // 0: none
    int64_t N, nb;             // rows, scales of a row
    uint8_t* out;              // rows n: of row n of matrix i at i * panels * 32 + n; rows k: of block k / 32 at k
    int parts;                 // rows k: parts that the rows are taken in, at most kScaleParts
    uint8_t* part;             // [parts][nb], largest byte + 1 (0: NaNs only)
};
constexpr int kScaleParts = 16;
int scale_parts(int64_t M, int64_t nb);       // beside a gradient of M rows
hipError_t launch_pack_weights(int wf, int mats, const QuantW* w, int64_t N, int64_t K, bool transposed, int form,
                               const ScaleArgs& scales, uint8_t* img, hipStream_t s);
// dtype DT_BF16 and no xexp: the rows as they are, in bfloat16.
hipError_t launch_pack_x(const void* x, int dtype, int64_t M, int64_t K, bool twice, uint8_t* img, int8_t* xexp,
                         const ScaleArgs& scales, hipStream_t s);
// dz of every projection: the image, the dz outputs and the column sums.
int64_t grad_sums_bytes(int nmat, int64_t M, int64_t N);
hipError_t launch_pack_dz(const LinearGradArgs& a, uint8_t* img, int8_t* xexp, float* sums, const ScaleArgs& scales,
                          hipStream_t s);
// What launch_pack_dz leaves in `sums` to be joined, by launch_join_sums or with a split product's parts.
SumsArgs sums_args(const LinearGradArgs& a, const float* sums);
hipError_t launch_join_sums(const SumsArgs& a, hipStream_t s);

// ---- eight values at a time ----------------------------------------------------

// Eight consecutive 16-bit values, `left` of them inside the tensor (>= 8: one
// 16-byte access), the others zero.  VEC: rows are 16-byte aligned and `left`
// is 8 or at most 0; else an access is aligned to its elements only, which
// global memory takes too.
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
template <bool VEC>
__device__ __forceinline__ u32x4_t load8_raw(const void* p, int64_t i, int left) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if (VEC) return left > 0 ? *reinterpret_cast<const u32x4_t*>(q) : u32x4_t{0u, 0u, 0u, 0u};
    if (left >= 8) return *reinterpret_cast<const u32x4_any_t*>(q);
    u32x4_t r = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; e++)
        if (e < left) r[e >> 1] |= (uint32_t)q[e] << (16 * (e & 1));
    return r;
}
__device__ __forceinline__ void unpack8(int dt, const u32x4_t& r, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 4; e++) {
        if (dt == DT_BF16) {
            v[2 * e] = __uint_as_float(r[e] << 16);
            v[2 * e + 1] = __uint_as_float(r[e] & 0xFFFF0000u);
        } else {
            v[2 * e] = f16_to_f32(r[e] & 0xFFFFu);
            v[2 * e + 1] = f16_to_f32(r[e] >> 16);
        }
    }
}
// Two binary32 values rounded to nearest even into a pair of 16-bit ones.
__device__ __forceinline__ uint32_t pack2(int dt, float a, float b) {
    const f32x2_t f = {a, b};
    if (dt == DT_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, half2_t));
}
__device__ __forceinline__ u32x4_t pack8(int dt, const float (&v)[8]) {
    u32x4_t r;
#pragma unroll
    for (int e = 0; e < 4; e++) r[e] = pack2(dt, v[2 * e], v[2 * e + 1]);
    return r;
}
template <bool VEC>
__device__ __forceinline__ void store8(void* p, int64_t i, int left, const u32x4_t& r) {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    if (VEC) {
        if (left > 0) *reinterpret_cast<u32x4_t*>(q) = r;
        return;
    }
    if (left >= 8) {
        *reinterpret_cast<u32x4_any_t*>(q) = r;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; e++)
        if (e < left) q[e] = (uint16_t)(r[e >> 1] >> (16 * (e & 1)));
}

// Eight sums times 2^e and their columns' powers of two (in one step: halfway they may leave the range).
__device__ __forceinline__ void unscale8(const u32x2_t& bytes, int e, float (&v)[8]) {
#pragma unroll
    for (int t = 0; t < 8; t++) v[t] = ldexpf(v[t], (int)((bytes[t >> 2] >> (8 * (t & 3))) & 0xFFu) - kRowScale + e);
}

// The epilogue of eight consecutive columns n .. n + 7 of row m (`left` of
// them inside the output): z, and for EPI_GATED the second projection z2.
// Residual and y may be the same tensor: each element is read before it is
// written, by the same lane.
template <int EPI, bool VEC>
__device__ __forceinline__ void epilogue8(const EpilogueArgs& a, int64_t m, int64_t n, float (&z)[8], float (&z2)[8]) {
    const int left = (int)(a.N - n < 8 ? a.N - n : 8);
    const int64_t o = m * a.N + n;
    float t[8];
    if (a.bias[0]) {
        unpack8(a.dtype, load8_raw<VEC>(a.bias[0], n, left), t);
#pragma unroll
        for (int e = 0; e < 8; e++) z[e] += t[e];
    }
    if (a.pre[0]) store8<VEC>(a.pre[0], o, left, pack8(a.dtype, z));
    if constexpr (EPI == EPI_GATED) {
        if (a.bias[1]) {
            unpack8(a.dtype, load8_raw<VEC>(a.bias[1], n, left), t);
#pragma unroll
            for (int e = 0; e < 8; e++) z2[e] += t[e];
        }
        if (a.pre[1]) store8<VEC>(a.pre[1], o, left, pack8(a.dtype, z2));
    }
    if (a.act != ACT_NONE) activate_all<false>(a.act, z, z, t);
    if constexpr (EPI == EPI_GATED) {
#pragma unroll
        for (int e = 0; e < 8; e++) z[e] *= z2[e];
    }
    if (a.residual) {
        unpack8(a.dtype, load8_raw<VEC>(a.residual, o, left), t);
#pragma unroll
        for (int e = 0; e < 8; e++) z[e] += t[e];
    }
    store8<VEC>(a.y, o, left, pack8(a.dtype, z));
}

}  // namespace q4
