// tile_pack.hip -- the packers of the dense product's operand images
// (tile_image.hpp): weights dequantised to binary16, by rows or transposed;
// activations and gradients scaled to binary16 row by row.  MXFP4 weights against
// bfloat16 activations are images in bfloat16, the activations as they are.  All are bound by
// memory (a quantised matrix read, two bytes a weight written).
#include "mx_common.hpp"
#include "tile_image.hpp"

namespace q4 {

// ---- weights ---------------------------------------------------------------------
//
// Dequantised exactly in binary32 ((q - 8) d has 15 bits, q s + b one rounding)
// and rounded once to binary16.  MXFP4, whose scales may be any power of two:
//   IMG_QUARTER  a quarter of each, which bfloat16 holds exactly under any scale;
//   IMG_ROWS     binary16, the scales of a row (of W^T: of 32 rows, which share them) multiplied
//                by the power of two that brings the largest to 2^13: exact from 2^-36 of it on.

// Codes as binary32: byte e of w (8-bit), or its low / high nibble.
template <int E>
__device__ __forceinline__ float byte_f32(uint32_t w) { return (float)((w >> (8 * E)) & 0xFFu); }

template <int WF>
struct RowScale {
    float s, b;
    __device__ __forceinline__ float operator()(float q) const {
        return WF == WF_Q4_0 ? (q - 8.0f) * s : __builtin_fmaf(q, s, b);
    }
};
// MXFP4: a block's scale byte s in a row whose largest is `most`; the eight codes of a word as
// four pairs of binary16.
__device__ __forceinline__ float scale_below(int s, int most) {
    const int to = s - most + kRowScale;
    return mx_scale(s == 255 ? 255u : to < 1 ? 1u : (uint32_t)to);
}
__device__ __forceinline__ u32x4_t mx_pairs(uint32_t w, float s) {
    return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 0)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 1)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 2)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, 3))};
}
template <int WF>
__device__ __forceinline__ RowScale<WF> row_scale(const QuantW& w, int64_t n, int64_t blk32, int64_t K) {
    if constexpr (WF == WF_Q4_0) {
        return {f16_to_f32(w.s[n * (K / 32) + blk32]), 0.0f};
    } else if constexpr (WF == WF_MXFP4) {
        return {mx_scale(reinterpret_cast<const uint8_t*>(w.s)[n * (K / 32) + blk32]), 0.0f};
    } else {
        const int64_t g = n * (K / 64) + (blk32 >> 1);
        return {bf16_to_f32(w.s[g]), bf16_to_f32(w.b[g])};
    }
}

// Image of W: a wave takes a panel's 32 rows by 128 bytes of codes (256 weights;
// 128 at 8 bits).  Direct-to-LDS copies of 8 rows by 128 contiguous bytes (a load
// whose neighbouring lanes lie on different rows asks for 64 separate pieces),
// the pieces of 16 bytes placed by an XOR with the row; then lane (row j, half h)
// takes whole blocks of 32 weights, block 2 t + h in pass t, and writes each as
// its four 16-byte pieces: for one piece 32 lanes write 512 contiguous bytes.
// IMG_REST: the image has twice the slices, and the second half holds what the
// rounding to binary16 left of each weight (see launch_linear).
// Measured: two 12288 x 4096 Q4_0 matrices 44 us, 57 MB read and 201 MB written.
template <int WF, int FORM>
__global__ __launch_bounds__(256) void k_pack_weights(QuantW w0, QuantW w1, int mats, int N, int64_t K, int64_t slices,
                                                      int64_t kgroups, const ScaleArgs scales, uint8_t* __restrict__ img) {
    constexpr int kBlocks = WF == WF_AFFINE8 ? 4 : 8;        // of 32 weights, in a wave's 128 bytes of a row
    constexpr int kPieces = 8 / kBlocks;                     // 16-byte pieces of a block
    __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * 32 * 128];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), j = lane & 31, h = lane >> 5;
    const int64_t panel = blockIdx.x / kgroups;
    const QuantW w = mats == 2 && (panel & 1) ? w1 : w0;
    const int64_t first = panel / mats * 32, in = N - 1 - first;
    const int64_t nb = K / 32, b0 = (blockIdx.x % kgroups * 4 + wave) * kBlocks;
    if (b0 >= nb) return;                                    // no barrier below: a wave's LDS is its own
    const uint32_t row_q = (uint32_t)(WF == WF_AFFINE8 ? K : K / 2), last = row_q / 16 - 1;
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds) +
                          (uint32_t)wave * 4096;
#pragma unroll
    for (int c = 0; c < 4; c++) {
        // rows past N repeat the last one (their outputs are never stored), pieces
        // past the row its last (never written)
        const uint32_t r = (uint32_t)(8 * c + (lane >> 3)), row = r < (uint32_t)in ? r : (uint32_t)in;
        const uint32_t p = (uint32_t)b0 * kPieces + ((uint32_t)(lane & 7) ^ (r & 7u));
        copy_unit(w.q + first * row_q, row * row_q + (p < last ? p : last) * 16u, lds0 + c * 1024);
    }
    const int64_t n = first + (j < in ? j : in);
    RowScale<WF> sc[kBlocks / 2];
    int most = 0;
    if constexpr (FORM == IMG_ROWS) most = scales.out[(mats == 2 && (panel & 1) ? ((int64_t)N + 31) / 32 * 32 : 0) + n];
#pragma unroll
    for (int t = 0; t < kBlocks / 2; t++) {
        int64_t b = b0 + 2 * t + h;
        b = b < nb ? b : nb - 1;
        if constexpr (FORM == IMG_ROWS) {
            sc[t] = {scale_below(reinterpret_cast<const uint8_t*>(w.s)[n * nb + b], most), 0.0f};
        } else {
            sc[t] = row_scale<WF>(w, n, b, K);
        }
    }
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    Q4_WAIT_VMCNT(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
#pragma unroll
    for (int t = 0; t < kBlocks / 2; t++) {
        const int64_t b = b0 + 2 * t + h;
        if (b >= nb) continue;
        u32x4_t raw[kPieces];
#pragma unroll
        for (int e = 0; e < kPieces; e++)
            raw[e] = *reinterpret_cast<const u32x4_t*>(lds + wave * 4096 + j * 128 + ((((2 * t + h) * kPieces + e) ^ (j & 7)) * 16));
        uint8_t* out = img + (panel * slices + 2 * b) * kUnit + j * 16;
#pragma unroll
        for (int c = 0; c < 4; c++) {        // elements 8 c .. 8 c + 7: slice c / 2, half c % 2
            if constexpr (WF == WF_MXFP4) {
                *reinterpret_cast<u32x4_t*>(out + (c >> 1) * kUnit + (c & 1) * 512) =
                    FORM == IMG_QUARTER ? bf16_quarters(raw[0][c], sc[t].s) : mx_pairs(raw[0][c], sc[t].s);
                continue;
            }
            float f[8];
            uint32_t lo, hi;
            if constexpr (WF == WF_AFFINE8) {
                lo = raw[c >> 1][2 * (c & 1)];
                hi = raw[c >> 1][2 * (c & 1) + 1];
            } else if constexpr (WF == WF_Q4_0) {
                // elements 0..15 low nibbles, 16..31 high nibbles of bytes 0..15
                lo = (raw[0][2 * (c & 1)] >> (c < 2 ? 0 : 4)) & 0x0F0F0F0Fu;
                hi = (raw[0][2 * (c & 1) + 1] >> (c < 2 ? 0 : 4)) & 0x0F0F0F0Fu;
            } else {
                // byte i: elements 2 i (low nibble) and 2 i + 1
                lo = raw[0][c] & 0x0F0F0F0Fu;
                hi = (raw[0][c] >> 4) & 0x0F0F0F0Fu;
            }
            constexpr bool kPairs = WF == WF_AFFINE4;
            f[0] = byte_f32<0>(lo); f[kPairs ? 2 : 1] = byte_f32<1>(lo); f[kPairs ? 4 : 2] = byte_f32<2>(lo); f[kPairs ? 6 : 3] = byte_f32<3>(lo);
            f[kPairs ? 1 : 4] = byte_f32<0>(hi); f[kPairs ? 3 : 5] = byte_f32<1>(hi); f[kPairs ? 5 : 6] = byte_f32<2>(hi); f[7] = byte_f32<3>(hi);
#pragma unroll
            for (int e = 0; e < 8; e++) f[e] = sc[t](f[e]);
            const u32x4_t v = pack8(DT_F16, f);
            *reinterpret_cast<u32x4_t*>(out + (c >> 1) * kUnit + (c & 1) * 512) = v;
            if constexpr (FORM == IMG_REST) {
                float rounded[8];
                unpack8(DT_F16, v, rounded);
#pragma unroll
                for (int e = 0; e < 8; e++) f[e] -= rounded[e];
                *reinterpret_cast<u32x4_t*>(out + (slices / 2 + (c >> 1)) * kUnit + (c & 1) * 512) = pack8(DT_F16, f);
            }
        }
    }
}

// Image of W^T (rows k, summed over n; n past N are zeros): a workgroup takes 64
// rows n by kTileK weights.  A thread loads one 32-bit word of codes from each
// of eight consecutive rows (a row's words over consecutive lanes: 128
// contiguous bytes) and holds the codes of 8 n for 8 (4) k: eight (four)
// 16-byte pieces of the image.  They change places in LDS, where a panel's four
// units lie as in memory, and leave as whole units.
template <int WF>
__global__ __launch_bounds__(256) void k_pack_weights_t(QuantW w0, QuantW w1, int N, int64_t K, int64_t slices,
                                                        int64_t ktiles, int64_t ntiles, const ScaleArgs scales,
                                                        uint8_t* __restrict__ img) {
    constexpr int kPer = WF == WF_AFFINE8 ? 4 : 8;           // weights of a code word
    constexpr int kTileK = 32 * kPer;
    constexpr int kTilePanels = kTileK / 32;
    constexpr int kPanelB = 4 * kUnit + 16;                  // the 16 spread the panels over the banks
    __shared__ __attribute__((aligned(16))) uint8_t lds[kTilePanels * kPanelB];
    const int tid = threadIdx.x, word = tid & 31, o = tid >> 5;       // code word of the tile's row, octet of rows
    const int64_t kt = blockIdx.x % ktiles, rest = blockIdx.x / ktiles;
    const int64_t nt = rest % ntiles;
    const int mat = (int)(rest / ntiles);
    const QuantW w = mat ? w1 : w0;
    const int64_t k0 = kt * kTileK + word * kPer;            // this word's first position, in code order
    const int64_t n0 = nt * 64 + o * 8;
    constexpr int kWordsPerBlk = 32 / kPer;                  // of a block of 32
    const int p = word / kWordsPerBlk, wb = word % kWordsPerBlk;
    const int64_t blk = k0 / 32, nb = K / 32;
    const bool in_k = blk < nb;
    uint32_t raw[8];
    RowScale<WF> sc[8];
    // MXFP4: the tile's eight columns of scales and their parts' largest, a byte a thread
    __shared__ __attribute__((aligned(16))) uint8_t parts[8][kScaleParts];
    if (WF == WF_MXFP4 && tid < 8 * kScaleParts) {
        const int64_t b = kt * 8 + tid / kScaleParts, part = tid % kScaleParts;
        parts[0][tid] = scales.part[(part < scales.parts ? part : scales.parts - 1) * nb + (b < nb ? b : nb - 1)];
    }
    int byte[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int64_t n = n0 + i < N ? n0 + i : N - 1, b = in_k ? blk : nb - 1;
        raw[i] = *reinterpret_cast<const uint32_t*>(w.q + (n * nb + b) * (128 / kPer) + wb * 4);
        if constexpr (WF == WF_MXFP4) byte[i] = reinterpret_cast<const uint8_t*>(w.s)[n * nb + b];
        else sc[i] = row_scale<WF>(w, n, b, K);
    }
    if constexpr (WF == WF_MXFP4) {
        __syncthreads();
        const u32x4_t all = *reinterpret_cast<const u32x4_t*>(parts[p]);
        int most = 0;
#pragma unroll
        for (int i = 0; i < kScaleParts; i++) {
            const int m = (int)(all[i >> 2] >> (8 * (i & 3)) & 0xFFu);
            most = m > most ? m : most;
        }
        most = most > 0 ? most - 1 : 0;
        if (nt == 0 && mat == 0 && o == 0 && in_k)
            *reinterpret_cast<u32x2_t*>(scales.out + k0) = u32x2_t{most * 0x01010101u, most * 0x01010101u};
#pragma unroll
        for (int i = 0; i < 8; i++) sc[i] = {scale_below(byte[i], most), 0.0f};
    }
#pragma unroll
    for (int i = 0; i < 8; i++)
        if (!in_k || n0 + i >= N) {
            sc[i].s = 0.0f;
            sc[i].b = 0.0f;
            raw[i] = 0u;
        }
    uint8_t* base = lds + p * kPanelB + (o >> 1) * kUnit + (o & 1) * 512;
    auto put = [&](int j, auto code) __attribute__((always_inline)) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = sc[i](code(raw[i]));
        *reinterpret_cast<u32x4_t*>(base + j * 16) = pack8(DT_F16, f);
    };
    if constexpr (WF == WF_MXFP4) {
        // elements 8 wb .. + 7 of the eight rows, two rows to a word
        u32x4_t pair[8];
#pragma unroll
        for (int i = 0; i < 8; i++) pair[i] = mx_pairs(raw[i], sc[i].s);
#pragma unroll
        for (int e = 0; e < 8; e++) {
            u32x4_t v;
#pragma unroll
            for (int i = 0; i < 4; i++)
                v[i] = __builtin_amdgcn_perm(pair[2 * i + 1][e >> 1], pair[2 * i][e >> 1], e & 1 ? 0x07060302u : 0x05040100u);
            *reinterpret_cast<u32x4_t*>(base + (8 * wb + e) * 16) = v;
        }
    } else if constexpr (WF == WF_AFFINE8) {
        put(4 * wb + 0, [](uint32_t v) { return byte_f32<0>(v); });
        put(4 * wb + 1, [](uint32_t v) { return byte_f32<1>(v); });
        put(4 * wb + 2, [](uint32_t v) { return byte_f32<2>(v); });
        put(4 * wb + 3, [](uint32_t v) { return byte_f32<3>(v); });
    } else {
        // Q4_0: byte i of word wb holds elements 4 wb + i and 16 + 4 wb + i;
        // affine: elements 8 wb + 2 i and 8 wb + 2 i + 1
        constexpr int kStep = WF == WF_Q4_0 ? 1 : 2, kHigh = WF == WF_Q4_0 ? 16 : 1;
        const int j0 = WF == WF_Q4_0 ? 4 * wb : 8 * wb;
        put(j0 + 0 * kStep, [](uint32_t v) { return byte_f32<0>(v & 0x0F0F0F0Fu); });
        put(j0 + 1 * kStep, [](uint32_t v) { return byte_f32<1>(v & 0x0F0F0F0Fu); });
        put(j0 + 2 * kStep, [](uint32_t v) { return byte_f32<2>(v & 0x0F0F0F0Fu); });
        put(j0 + 3 * kStep, [](uint32_t v) { return byte_f32<3>(v & 0x0F0F0F0Fu); });
        put(j0 + 0 * kStep + kHigh, [](uint32_t v) { return byte_f32<0>((v >> 4) & 0x0F0F0F0Fu); });
        put(j0 + 1 * kStep + kHigh, [](uint32_t v) { return byte_f32<1>((v >> 4) & 0x0F0F0F0Fu); });
        put(j0 + 2 * kStep + kHigh, [](uint32_t v) { return byte_f32<2>((v >> 4) & 0x0F0F0F0Fu); });
        put(j0 + 3 * kStep + kHigh, [](uint32_t v) { return byte_f32<3>((v >> 4) & 0x0F0F0F0Fu); });
    }
    __syncthreads();
    const int64_t mat_slices = ((int64_t)N + 31) / 32 * 2;
#pragma unroll
    for (int t = 0; t < kTilePanels; t++) {                  // a wave writes one unit of the panel
        const int64_t panel = kt * kTilePanels + t, sl = nt * 4 + (tid >> 6);
        if (panel * 32 >= K || sl >= mat_slices) continue;
        *reinterpret_cast<u32x4_t*>(img + (panel * slices + mat * mat_slices + sl) * kUnit + (tid & 63) * 16) =
            *reinterpret_cast<const u32x4_t*>(lds + t * kPanelB + tid * 16);
    }
}

template <int WF>
static hipError_t pack_weights_t(int mats, const QuantW* w, int64_t N, int64_t K, bool transposed, int form,
                                 const ScaleArgs& scales, uint8_t* img, hipStream_t s) {
    if (!transposed) {
        constexpr int kGroupK = WF == WF_AFFINE8 ? 512 : 1024;
        const int64_t kgroups = (K + kGroupK - 1) / kGroupK, blocks = (N + 31) / 32 * mats * kgroups;
        if (!launchable(blocks, 256)) return hipErrorInvalidValue;
        constexpr bool kMx = WF == WF_MXFP4;
        auto k = form == IMG_REST || form == IMG_ROWS ? k_pack_weights<WF, kMx ? IMG_ROWS : IMG_REST>
                                                      : k_pack_weights<WF, kMx ? IMG_QUARTER : IMG_F16>;
        hipLaunchKernelGGL(k, dim3((unsigned)blocks), dim3(256), 0, s, w[0], w[mats - 1], mats, (int)N, K,
                           image_slices(K) * (form == IMG_REST ? 2 : 1), kgroups, scales, img);
    } else {
        constexpr int kTileK = WF == WF_AFFINE8 ? 128 : 256;
        const int64_t ktiles = (K + kTileK - 1) / kTileK, ntiles = (N + 63) / 64, blocks = ktiles * ntiles * mats;
        if (!launchable(blocks, 256)) return hipErrorInvalidValue;
        hipLaunchKernelGGL((k_pack_weights_t<WF>), dim3((unsigned)blocks), dim3(256), 0, s, w[0], w[mats - 1], (int)N, K,
                           image_slices(N) * mats, ktiles, ntiles, scales, img);
    }
    return hipGetLastError();
}

hipError_t launch_pack_weights(int wf, int mats, const QuantW* w, int64_t N, int64_t K, bool transposed, int form,
                               const ScaleArgs& scales, uint8_t* img, hipStream_t s) {
    if (wf == WF_Q4_0) return pack_weights_t<WF_Q4_0>(mats, w, N, K, transposed, form, scales, img, s);
    if (wf == WF_AFFINE4) return pack_weights_t<WF_AFFINE4>(mats, w, N, K, transposed, form, scales, img, s);
    if (wf == WF_MXFP4) return pack_weights_t<WF_MXFP4>(mats, w, N, K, transposed, form, scales, img, s);
    return pack_weights_t<WF_AFFINE8>(mats, w, N, K, transposed, form, scales, img, s);
}

// ---- the largest scales of MXFP4 weights ---------------------------------------------
//
// By the first workgroups of the launches below, 16 scales a load (a launch of its own for as
// few bytes, k_mx_scales, takes 3.4 us).  As byte + 1, so that a NaN (255) is 0 and counts for nothing, pairs of bytes as
// 16-bit numbers.
constexpr int kPackThreads = 1024;

typedef u32x4_t u32x4_b __attribute__((aligned(1)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void take_pair(u16x2_t& most, uint32_t pair) {
    most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2_t, (pair + 0x00010001u) & 0x00FF00FFu));
}

// Of rows: eight lanes a row.
constexpr int kScaleRows = kPackThreads / 8;
static unsigned row_scale_blocks(const ScaleArgs& a) {       // (at most 2^26 rows: 2^19 workgroups)
    return (unsigned)(((a.N + 31) / 32 * 32 * a.mats + kScaleRows - 1) / kScaleRows);
}
__device__ __forceinline__ void row_scales(const ScaleArgs& a, unsigned block) {
    const int64_t np = (a.N + 31) / 32 * 32, id = (int64_t)block * kScaleRows + threadIdx.x / 8;
    if (id >= np * a.mats) return;
    const int64_t n = id % np, last = n < a.N ? n : a.N - 1;
    const uint8_t* row = a.s[id / np] + last * a.nb;
    const int t = threadIdx.x & 7;
    u16x2_t most = {0, 0};
    for (int64_t i = t * 16; i + 16 <= a.nb; i += 128) {
        const u32x4_t v = *reinterpret_cast<const u32x4_b*>(row + i);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            take_pair(most, v[e] & 0x00FF00FFu);
            take_pair(most, v[e] >> 8 & 0x00FF00FFu);
        }
    }
    for (int64_t i = a.nb / 16 * 16 + t; i < a.nb; i += 8) take_pair(most, row[i]);
    int m = most[0] > most[1] ? most[0] : most[1];
#pragma unroll
    for (int d = 1; d < 8; d *= 2) {
        const int o = __shfl_xor(m, d, 64);
        m = o > m ? o : m;
    }
    if (t == 0) a.out[id] = (uint8_t)(m > 0 ? m - 1 : 0);
}

// Of columns of scales, over part `block % parts` of the rows of all matrices: a
// workgroup takes 128 columns, eight lanes of 16 of them a row.
static unsigned column_scale_blocks(const ScaleArgs& a) {    // (at most 2^20 columns: 2^17 workgroups)
    return a.mats > 0 ? (unsigned)((a.nb + 127) / 128 * a.parts) : 0u;
}
__device__ __forceinline__ void column_scales(const ScaleArgs& a, unsigned block) {
    __shared__ __attribute__((aligned(16))) uint8_t red[kPackThreads / 64][128];
    const int part = (int)(block % a.parts), t = threadIdx.x & 7;
    const int64_t group = block / a.parts * 128, c = group + t * 16, rows = a.N * a.mats;
    const int64_t r1 = rows * (part + 1) / a.parts;
    // what a load of 16 would read past the row lies in front of it; less than 16 come one by one
    const int64_t from = c + 16 <= a.nb ? c : a.nb - 16;
    u16x2_t most[8] = {};
    if (c < a.nb)
#pragma unroll 4
        for (int64_t r = rows * part / a.parts + threadIdx.x / 8; r < r1; r += kPackThreads / 8) {
            const uint8_t* row = r < a.N ? a.s[0] + r * a.nb : a.s[1] + (r - a.N) * a.nb;
            u32x4_t v = {~0u, ~0u, ~0u, ~0u};
            if (from >= 0) {
                v = *reinterpret_cast<const u32x4_b*>(row + from);
            } else {
#pragma unroll
                for (int e = 0; e < 16; e++)
                    if (from + e >= 0) v[e >> 2] ^= (uint32_t)(row[from + e] ^ 0xFFu) << (8 * (e & 3));
            }
#pragma unroll
            for (int e = 0; e < 4; e++) {
                take_pair(most[2 * e], v[e] & 0x00FF00FFu);
                take_pair(most[2 * e + 1], v[e] >> 8 & 0x00FF00FFu);
            }
        }
    // over the wave's eight rows, then over the waves
    u32x4_t all;
#pragma unroll
    for (int e = 0; e < 4; e++) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int d = 8; d < 64; d *= 2)
                most[2 * e + h] = __builtin_elementwise_max(
                    most[2 * e + h], __builtin_bit_cast(u16x2_t, __shfl_xor(__builtin_bit_cast(int, most[2 * e + h]), d, 64)));
        all[e] = __builtin_bit_cast(uint32_t, most[2 * e]) | __builtin_bit_cast(uint32_t, most[2 * e + 1]) << 8;
    }
    if ((threadIdx.x & 63) < 8) *reinterpret_cast<u32x4_t*>(&red[threadIdx.x >> 6][t * 16]) = all;
    __syncthreads();
    if (threadIdx.x < 128 && group + threadIdx.x < a.nb) {
        // a column's byte in its lane's 16
        const int lane = threadIdx.x / 16;
        const int64_t lc = group + lane * 16, lf = lc + 16 <= a.nb ? lc : a.nb - 16;
        const int at = lane * 16 + (int)(group + threadIdx.x - lf);
        int m = 0;
        for (int w = 0; w < kPackThreads / 64; w++) m = red[w][at] > m ? red[w][at] : m;
        a.part[part * a.nb + group + threadIdx.x] = (uint8_t)m;
    }
}

// ---- rows of activations and gradients ----------------------------------------------
//
// A row is multiplied by the power of two 2^e that brings its largest |value|
// into [2^14, 2^15) and rounded to binary16: the whole bfloat16 range fits, and
// values down to 2^-29 of the row's largest keep binary16's 11 bits (bfloat16
// values: exact).  The product's epilogue takes 2^-e off again.  A workgroup
// takes eight rows, so that a piece's eight rows are 128 contiguous bytes of
// the image (four where eight would leave CUs idle); it reads them twice, the
// second time from cache.  `twice`: the image holds the row twice, for weights
// in two halves.  Measured: 2048 x 4096 10 us, 2048 x 12288 19 us (5.3 TB/s).

constexpr float kLargest = 3.4028234663852886e38f;

// Of a row's largest |value| (NaNs left out).
__device__ __forceinline__ int row_exponent(float mx) {
    if (!(mx > 0.0f)) return 0;
    if (mx > kLargest) return -113;        // an infinity: no finite value beside it becomes one
    const int e = 14 - (__builtin_amdgcn_frexp_expf(mx) - 1);
    return e < -113 ? -113 : e > 127 ? 127 : e;
}

// Maximum over the lanes and waves that hold the same row (lane % ROWS).
template <int ROWS>
__device__ __forceinline__ float rows_max(float mx, float (*red)[8]) {
#pragma unroll
    for (int d = ROWS; d < 64; d *= 2) mx = fmaxf(mx, __shfl_xor(mx, d, 64));
    const int lane = threadIdx.x & 63;
    if (lane < ROWS) red[threadIdx.x >> 6][lane] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPackThreads / 64; w++) mx = fmaxf(mx, red[w][lane % ROWS]);
    return mx;
}

__device__ __forceinline__ uint8_t* piece(uint8_t* img, int64_t m, int64_t slices, int64_t c) {
    return img + (m / 32 * slices + (c >> 1)) * kUnit + (c & 1) * 512 + (m & 31) * 16;
}

__device__ __forceinline__ float max8(const float (&v)[8], float mx) {
#pragma unroll
    for (int e = 0; e < 8; e++) mx = fmaxf(mx, fabsf(v[e]));
    return mx;
}

// AS_IS: bfloat16 rows, copied.
template <int ROWS, bool AS_IS>
__global__ __launch_bounds__(kPackThreads) void k_pack_rows(const void* __restrict__ x, int dtype, int64_t M, int64_t K,
                                                            int64_t slices, int twice, uint8_t* __restrict__ img,
                                                            int8_t* __restrict__ xexp, const ScaleArgs scales,
                                                            const unsigned scale_blocks) {
    if (blockIdx.x < scale_blocks) {
        row_scales(scales, blockIdx.x);
        return;
    }
    __shared__ float red[kPackThreads / 64][8];
    const int lane = threadIdx.x & 63;
    constexpr int kStride = kPackThreads / ROWS;
    const int64_t m = (int64_t)(blockIdx.x - scale_blocks) * ROWS + lane % ROWS, c0 = (threadIdx.x >> 6) * (64 / ROWS) + lane / ROWS;
    const int64_t row = (m < M ? m : M - 1) * K, chunks = K / 8;          // K % 32 == 0
    if constexpr (AS_IS) {
        if (m < M)
            for (int64_t c = c0; c < chunks; c += kStride)
                *reinterpret_cast<u32x4_t*>(piece(img, m, slices, c)) = load8_raw<true>(x, row + c * 8, 8);
        return;
    }
    float v[8], mx = 0.0f;
    for (int64_t c = c0; c < chunks; c += kStride) {
        unpack8(dtype, load8_raw<true>(x, row + c * 8, 8), v);
        mx = max8(v, mx);
    }
    int e = row_exponent(rows_max<ROWS>(mx, red));
    if (scales.mats > 0 && e < 0) e = 0;                     // binary16 rows against scaled weights: exact
    const float scale = ldexpf(1.0f, e);
    if (m < M) {
        for (int64_t c = c0; c < chunks; c += kStride) {
            unpack8(dtype, load8_raw<true>(x, row + c * 8, 8), v);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] *= scale;
            const u32x4_t p = pack8(DT_F16, v);
            *reinterpret_cast<u32x4_t*>(piece(img, m, slices, c)) = p;
            if (twice) {
                // an infinity counts in the first half only: a remainder may be zero
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] = fabsf(v[i]) <= kLargest ? v[i] : 0.0f;
                *reinterpret_cast<u32x4_t*>(piece(img, m, slices, c + chunks)) = pack8(DT_F16, v);
            }
        }
        if (threadIdx.x < ROWS) xexp[m] = (int8_t)e;
    }
}

// Rows of a workgroup: four where eight would leave CUs idle.
static int pack_rows(int64_t M) { return M > 8 * (current_cu_count() - 1) ? 8 : 4; }
// Rows of a launch: a thread for each 1/128 row stays below a launch's 2^32
// (whole panels, and whole groups of rows).
constexpr int64_t kLaunchRows = int64_t(1) << 24;

hipError_t launch_pack_x(const void* x, int dtype, int64_t M, int64_t K, bool twice, uint8_t* img, int8_t* xexp,
                         const ScaleArgs& scales, hipStream_t s) {
    const int rows = pack_rows(M);
    const int64_t slices = image_slices(K) * (twice ? 2 : 1);
    const bool as_is = !xexp;
    auto k = rows == 8 ? (as_is ? k_pack_rows<8, true> : k_pack_rows<8, false>)
                       : (as_is ? k_pack_rows<4, true> : k_pack_rows<4, false>);
    unsigned scale_blocks = row_scale_blocks(scales);
    for (int64_t m = 0; m < M; m += kLaunchRows, scale_blocks = 0) {
        const int64_t count = M - m < kLaunchRows ? M - m : kLaunchRows;
        const unsigned row_blocks = (unsigned)((count + rows - 1) / rows);
        if (!launchable((int64_t)row_blocks + scale_blocks, kPackThreads)) return hipErrorInvalidValue;
        hipLaunchKernelGGL(k, dim3(row_blocks + scale_blocks), dim3(kPackThreads), 0, s,
                           static_cast<const char*>(x) + m * K * 2, dtype, count, K, slices, twice ? 1 : 0,
                           img + m / 32 * slices * kUnit, as_is ? nullptr : xexp + m, scales, scale_blocks);
    }
    return hipGetLastError();
}

// dz of the projections: the same image (the projections' slices follow each
// other), the dz outputs rounded from the same binary32 values, and the sums of
// the workgroup's rows, joined by k_join_sums (or with a split product's parts) in a fixed order.
template <bool VEC>
__device__ __forceinline__ void load_dz(const LinearGradArgs& a, int64_t o, int left, float (&dz)[2][8]) {
    unpack8(DT_BF16, load8_raw<VEC>(a.dy, o, left), dz[0]);
    if (a.pre[0]) {
        float g[8], slope[8];
        unpack8(DT_BF16, load8_raw<VEC>(a.pre[0], o, left), g);
        if (a.nmat == 2) {
            float u[8];
            unpack8(DT_BF16, load8_raw<VEC>(a.pre[1], o, left), u);
            activate_all<true>(a.act, g, g, slope);
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float dh = dz[0][e];
                dz[0][e] = dh * u[e] * slope[e];
                dz[1][e] = dh * g[e];
            }
        } else {
            activate_all<true>(a.act, g, g, slope);
#pragma unroll
            for (int e = 0; e < 8; e++) dz[0][e] *= slope[e];
        }
    }
    // past the row's end: zeros in the image, whatever the derivative of zeros is
    if (left < 8) {
#pragma unroll
        for (int e = 0; e < 8; e++)
            if (e >= left) dz[0][e] = dz[1][e] = 0.0f;
    }
}

template <bool VEC, int ROWS>
__global__ __launch_bounds__(kPackThreads) void k_pack_dz(const LinearGradArgs a, int64_t slices, uint8_t* __restrict__ img,
                                                          int8_t* __restrict__ xexp, float* __restrict__ sums,
                                                          const ScaleArgs scales, const unsigned scale_blocks) {
    if (blockIdx.x < scale_blocks) {
        column_scales(scales, blockIdx.x);
        return;
    }
    const int64_t group = blockIdx.x - scale_blocks;
    __shared__ float red[kPackThreads / 64][8];
    const int lane = threadIdx.x & 63;
    constexpr int kStride = kPackThreads / ROWS;
    const int64_t m = group * ROWS + lane % ROWS, c0 = (threadIdx.x >> 6) * (64 / ROWS) + lane / ROWS;
    const int64_t row = (m < a.M ? m : a.M - 1) * a.N, chunks = slices * 2;      // of one projection, padded
    float dz[2][8], mx = 0.0f;
    auto left_of = [&](int64_t c) { return (int)(a.N - c * 8 < 8 ? a.N - c * 8 : 8); };
    // The exponent of the row's largest |dz| needs all of dz first.  Instead of
    // computing it twice, the largest |dy| gives a guess (to 2^8) that holds if
    // the largest |dz| then lies in [2^-2, 2^15), where binary16 keeps its bits;
    // the rows that miss it write the image again.
    for (int64_t c = c0; c * 8 < a.N; c += kStride) {
        unpack8(DT_BF16, load8_raw<VEC>(a.dy, row + c * 8, left_of(c)), dz[0]);
        mx = max8(dz[0], mx);
    }
    const bool exact = !a.pre[0];                            // dz is dy
    int e = row_exponent(rows_max<ROWS>(mx, red));
    if (!exact) e = e - 7 < -113 ? -113 : e - 7;
    const bool live = m < a.M;
    for (bool again = false;; again = true) {
        const float scale = ldexpf(1.0f, e);
        mx = 0.0f;
        for (int64_t c = c0; c < chunks; c += kStride) {
            const int left = left_of(c);
            load_dz<VEC>(a, row + (left > 0 ? c * 8 : 0), left, dz);
            mx = max8(dz[0], mx);
            if (a.nmat == 2) mx = max8(dz[1], mx);
#pragma unroll
            for (int i = 0; i < 2; i++) {
                if (i >= a.nmat) break;
                float v[8];
#pragma unroll
                for (int t = 0; t < 8; t++) v[t] = dz[i][t];
                if (live) {
                    if (a.dz[i] && left > 0 && !again) store8<VEC>(a.dz[i], row + c * 8, left, pack8(DT_BF16, v));
                    float sv[8];
#pragma unroll
                    for (int t = 0; t < 8; t++) sv[t] = v[t] * scale;
                    *reinterpret_cast<u32x4_t*>(piece(img, m, slices * a.nmat, c + i * chunks)) = pack8(DT_F16, sv);
                }
                if (a.dbias[i] && !again) {
#pragma unroll
                    for (int t = 0; t < 8; t++) {
                        float q = live ? v[t] : 0.0f;
#pragma unroll
                        for (int d = 1; d < ROWS; d *= 2) q += __shfl_xor(q, d, 64);
                        v[t] = q;
                    }
                    // lane r of the rows stores columns c * 8 + r, + ROWS ..
#pragma unroll
                    for (int t0 = 0; t0 < 8; t0 += ROWS) {
                        float mine = v[t0];
#pragma unroll
                        for (int t = 1; t < ROWS; t++) mine = lane % ROWS == t ? v[t0 + t] : mine;
                        const int col = t0 + lane % ROWS;
                        if (col < left) sums[(group * a.nmat + i) * a.N + c * 8 + col] = mine;
                    }
                }
            }
        }
        if (exact || again) break;
        __syncthreads();                                     // `red` is read no more
        mx = rows_max<ROWS>(mx, red);
        const int at = mx > 0.0f && mx <= kLargest ? __builtin_amdgcn_frexp_expf(mx) - 1 + e : 0;
        const bool miss = at < -2 || at >= 15 || (mx > kLargest && e > -113);
        if (miss) e = row_exponent(mx);
        if (!__syncthreads_or(miss)) break;
    }
    if (threadIdx.x < ROWS && live) xexp[m] = (int8_t)e;
}

// Columns of the sums of row groups, in order: a workgroup takes 64 columns of a
// projection, its sixteen waves a sixteenth of the groups each.
__global__ __launch_bounds__(1024) void k_join_sums(const float* __restrict__ sums, int64_t groups, int nmat, int64_t N,
                                                    float* __restrict__ out0, float* __restrict__ out1) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = blockIdx.y;
    const int64_t n = (int64_t)blockIdx.x * 64 + lane;
    float* out = i ? out1 : out0;
    if (!out) return;
    const int64_t last = groups * (wave + 1) / 16;
    float t = 0.0f;
    if (n < N)
#pragma unroll 8
        for (int64_t g = groups * wave / 16; g < last; g++) t += sums[(g * nmat + i) * N + n];
    red[wave][lane] = t;
    __syncthreads();
    if (wave == 0 && n < N) {
        for (int w = 1; w < 16; w++) t += red[w][lane];
        out[n] = t;
    }
}

// A gradient's workgroup fills a CU: where the last round over the CUs leaves room for four
// parts or more, they fit in there (1001 x 8192 x 2048: 14.8 us, without them
// 14.2, with 16 parts, a round more, 16.9).
int scale_parts(int64_t M, int64_t nb) {
    const int64_t cus = current_cu_count(), rows = pack_rows(M), blocks = (M + rows - 1) / rows, groups = (nb + 127) / 128;
    const int64_t room = (cus - blocks % cus) / groups;
    return (int)(room >= 4 && room < kScaleParts ? room : kScaleParts);
}

int64_t grad_sums_bytes(int nmat, int64_t M, int64_t N) { return (M + pack_rows(M) - 1) / pack_rows(M) * nmat * N * 4; }

hipError_t launch_pack_dz(const LinearGradArgs& a, uint8_t* img, int8_t* xexp, float* sums, const ScaleArgs& scales,
                          hipStream_t s) {
    const int rows = pack_rows(a.M);
    const int64_t slices = image_slices(a.N);
    auto k = a.N % 8 == 0 ? (rows == 8 ? k_pack_dz<true, 8> : k_pack_dz<true, 4>)
                          : (rows == 8 ? k_pack_dz<false, 8> : k_pack_dz<false, 4>);
    unsigned scale_blocks = column_scale_blocks(scales);
    for (int64_t m = 0; m < a.M; m += kLaunchRows, scale_blocks = 0) {
        LinearGradArgs t = a;
        auto from = [&](const void* p) { return p ? const_cast<char*>(static_cast<const char*>(p)) + m * a.N * 2 : nullptr; };
        t.M = a.M - m < kLaunchRows ? a.M - m : kLaunchRows;
        t.dy = from(a.dy);
        for (int i = 0; i < 2; i++) {
            t.pre[i] = from(a.pre[i]);
            t.dz[i] = from(a.dz[i]);
        }
        const unsigned row_blocks = (unsigned)((t.M + rows - 1) / rows);
        if (!launchable((int64_t)row_blocks + scale_blocks, kPackThreads)) return hipErrorInvalidValue;
        hipLaunchKernelGGL(k, dim3(row_blocks + scale_blocks), dim3(kPackThreads), 0, s, t, slices,
                           img + m / 32 * slices * a.nmat * kUnit, xexp + m, sums + m / rows * a.nmat * a.N, scales, scale_blocks);
    }
    return hipGetLastError();
}

SumsArgs sums_args(const LinearGradArgs& a, const float* sums) {
    const int rows = pack_rows(a.M);
    SumsArgs t{};
    t.sums = sums;
    t.groups = (a.M + rows - 1) / rows;
    t.N = a.N;
    t.nmat = a.dbias[0] || a.dbias[1] ? a.nmat : 0;
    t.out[0] = a.dbias[0];
    t.out[1] = a.dbias[1];
    return t;
}

hipError_t launch_join_sums(const SumsArgs& a, hipStream_t s) {
    if (a.nmat == 0) return hipSuccess;
    hipLaunchKernelGGL(k_join_sums, dim3((unsigned)((a.N + 63) / 64), a.nmat), dim3(1024), 0, s, a.sums, a.groups, a.nmat, a.N,
                       a.out[0], a.out[1]);
    return hipGetLastError();
}

}  // namespace q4
