// linear_few.hpp -- q4_linear and q4_gated at few rows (decode, small batches):
// the weights are streamed once, straight from their planes into registers, and
// never rounded.
//
// Mathematics.  A 16x16x32 MFMA multiplies 16 rows of x with 32 weights of each
// of 16 columns, given as codes: the scale of a block (group) is taken out of
// its sum,
//   Q4_0    y += d (sum x (128 + q) - 136 sum x)       per block of 32
//   affine  y += s sum x q + b sum x                    per group of 64
// with bfloat16 x: 128 + q (4 bits) or q (8 bits) is exact in bfloat16, and the
// subtracted multiple of sum x is the MFMA's accumulator input, itself one MFMA
// of x against a constant that serves every column.  All of these operands carry
// a factor 2^-14 (8 bits: 2^-15), taken off the joined sum again: a block's
// sums then stay in binary32's range for every x (64 terms of 255 x 2^-15, 143 x
// 2^-14 or 128 x 2^-14), and the products' bits are the same.  With binary16 x the codes
// are q - 8 and q themselves.  Products are exact, sums binary32: the result
// differs from the exact one by binary32 summation and the output's rounding.
//
// Layout.  The MFMA wants 16 rows of W across neighbouring lanes; memory wants
// neighbouring lanes on one row: read in the MFMA's order a load touches 64
// separate pieces (12 us for 28 MB, its address processing the bound).  So the
// codes go through LDS: a step is 128 bytes of each of a tile's 16 rows (256
// weights at 4 bits, 128 at 8), two direct-to-LDS copies of 8 rows by 128
// contiguous bytes, pieces of 16 bytes placed by an XOR with the row so that a
// wave's reads (lane j = lane & 15, g = lane >> 4: row j, pieces g and 4 + g) meet
// no bank twice.  The scales of a step are 16 bytes a row, loaded by one lane a
// row and passed through LDS too; x lies in LDS in the fragments' order, a slice
// of K at a time.
//
// At 4 bits a lane then holds block 4 c + g whole, where the MFMA of block t
// wants dword g of block 4 c + t: a 4 x 4 transposition over the four g, four
// lane swaps (v_permlane32_swap, v_permlane16_swap).  Up to four rows (DIAG) it
// falls away: row 4 m + b of the MFMA's A operand holds x of row m in the lanes
// g = b only, zeros elsewhere, so the four MFMAs of a chunk sum dwords 0 .. 3 of
// every lane's own block and row 4 m + b of the result is the whole sum of block
// b: four scaled additions a chunk and column instead of sixteen.  At 8 bits the
// MFMA's k order follows the load (a group has one scale).
//
// The waves of a workgroup take steps in turn, each its next one in flight while
// it multiplies, and add their sums through LDS in wave order (deterministic).
// For q4_gated the tiles come in pairs, gate and up of the same 16 columns.  A
// long sum over few columns is split over workgroups (FewSplit) and joined.
//
// Bound: up to four rows by round trips to memory, with one step of a wave in flight;
// above them by vector work, 16 to 18 instructions beside each MFMA, and by x through
// LDS.  Measured, Q4_0, N = 12288, K = 4096: one row 9.7 us (28.3 MB, 2.9 TB/s; with no loads
// at all 4.4), 16 rows 13.8 (2.1 TB/s), 32 rows 19.0; affine 8, one row 16.3; the
// gated pair 18.0, 23.2 and 41.5.
#pragma once

#include "block_common.hpp"
#include "gemm_common.hpp"

namespace q4 {

namespace few {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef u32x4_t u32x4_u __attribute__((aligned(2)));
typedef u32x2_t u32x2_u __attribute__((aligned(2)));
typedef uint32_t u32_u __attribute__((aligned(2)));

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
// Dword r of lane row g's 16 bytes -> dword g of lane row r's.
__device__ __forceinline__ void transpose4(u32x4_t& q) {
    uint32_t a = q[0], b = q[1], c = q[2], d = q[3];
    swap32(a, c);
    swap32(b, d);
    swap16(a, b);
    swap16(c, d);
    q = u32x4_t{a, b, c, d};
}

template <int XDT>
__device__ __forceinline__ floatx4_t mfma16(const u32x4_t& x, const u32x4_t& w, const floatx4_t& c) {
    if constexpr (XDT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x), __builtin_bit_cast(bf16x8_t, w), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, x), __builtin_bit_cast(half8_t, w), c, 0,
                                                      0, 0);
}

// The factor of the codes and offsets beside bfloat16 x is 2^-this (see above).
template <int WF, int XDT> constexpr int kDown = XDT != DT_BF16 ? 0 : WF == WF_AFFINE8 ? 15 : 14;
// A constant of them, twice: the bfloat16 bits of c 2^-this (exponents subtract).
template <int WF> constexpr uint32_t lowered(uint32_t bits) { return (bits - (kDown<WF, DT_BF16> << 7)) * 0x10001u; }

// Eight codes of a dword, in the pair order (byte 0, byte 2), (1, 3) of the low
// nibbles, then of the high ones: bfloat16 (128 + q) 2^-14, binary16 q - SUB.
template <int XDT, int SUB>
__device__ __forceinline__ u32x4_t nibbles(uint32_t w, uint32_t mask) {
    const uint32_t base = XDT == DT_BF16 ? lowered<WF_Q4_0>(0x4300u) : 0x64006400u;
    u32x4_t r;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const int shift = e == 0 ? 0 : e == 1 ? 8 : e == 2 ? 4 : 12;
        const uint32_t v = ((w >> shift) & mask) | base;
        if constexpr (XDT == DT_BF16) {
            r[e] = v;
        } else {
            const uint32_t off = SUB == 8 ? 0xE408E408u : 0xE400E400u;          // -1032, -1024
            const half2_t h = __builtin_bit_cast(half2_t, v) + __builtin_bit_cast(half2_t, off);
            r[e] = __builtin_bit_cast(uint32_t, h);
        }
    }
    return r;
}
// Eight 8-bit codes, exact in either type, in order (bfloat16: q 2^-15; the
// subtraction from the exponent saturates, so that a zero stays one).
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
template <int XDT>
__device__ __forceinline__ u32x4_t bytes8(uint32_t lo, uint32_t hi) {
    u32x4_t r;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const uint32_t w = e < 2 ? lo : hi;
        const f32x2_t f = {(float)((w >> (16 * (e & 1))) & 0xFFu), (float)((w >> (16 * (e & 1) + 8)) & 0xFFu)};
        if constexpr (XDT == DT_BF16)
            r[e] = __builtin_bit_cast(uint32_t, __builtin_elementwise_sub_sat(
                                                    __builtin_bit_cast(u16x2_t, __builtin_convertvector(f, bf16x2_t)),
                                                    __builtin_bit_cast(u16x2_t, (kDown<WF_AFFINE8, DT_BF16> << 7) * 0x10001u)));
        else r[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, half2_t));
    }
    return r;
}

}  // namespace few

// A sum split over workgroups: part blockIdx.y takes `per` steps and leaves its
// sums in rows of `np` values (the order of k_tile_join), unrounded and with
// their factor 2^-kDown.
struct FewSplit {
    float* part;          // null: one part, the epilogue here
    int64_t rows, np;     // rows of a part (of the whole call)
    int per, x_shift;
};

// Output n of a row x whose sum z over k0 <= k < k1 came out as NaN.  The sums
// above hold an infinite x with either sign (x (128 + q) - 136 x, s x q + b x), so
// that one infinity already gives a NaN; the infinite terms w x themselves
// decide what the sum is.  Without any z stays.  Reached by spoilt rows only.
template <int WF>
__device__ __forceinline__ float spoilt_sum(const QuantW& w, const uint16_t* x, int xdt, int64_t n, int64_t K, int k0, int k1,
                                            float z) {
    const uint32_t top = xdt == DT_BF16 ? 0x7F80u : 0x7C00u;
    float t = 0.0f;
    bool any = false;
#pragma unroll 1
    for (int k = k0; k < k1 && t == t; k += 8) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(x + k);
#pragma unroll 1
        for (int e = 0; e < 8; e++) {
            const uint32_t h = (v[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
            if ((h & top) != top) continue;
            const int64_t at = n * K + k + e;
            float q;
            if constexpr (WF == WF_AFFINE8) q = (float)w.q[at];
            else if constexpr (WF == WF_AFFINE4) q = (float)((w.q[at / 2] >> (4 * (at & 1))) & 15u);
            else q = (float)((w.q[at / 32 * 16 + (at & 15)] >> (at & 16 ? 4 : 0)) & 15u) - 8.0f;
            const float wk = WF == WF_Q4_0 ? q * f16_to_f32(w.s[at / 32])
                                           : __builtin_fmaf(q, bf16_to_f32(w.s[at / 64]), bf16_to_f32(w.b[at / 64]));
            t = __builtin_fmaf(wk, xdt == DT_BF16 ? bf16_to_f32(h) : f16_to_f32(h), t);
            any = true;
        }
    }
    return any ? t : z;
}

// Waves and LDS of a variant.  What is in flight on a CU is a step a wave: up to
// four rows a workgroup has eight waves, above them four, so that two workgroups
// with their x share a CU, or eight where there is but one workgroup a CU.
template <int WAVES, bool DIAG> constexpr int few_x() { return DIAG ? 32 << 10 : WAVES << 13; }      // x

template <int WF, int XDT, int MT, int NT, bool GATED, bool DIAG, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 2) void k_linear_few(const LinearArgs a, const FewSplit split) {
    using namespace few;
    static_assert(!DIAG || MT == 1, "a form for few rows");
    constexpr bool kBlocks = DIAG && WF != WF_AFFINE8;       // the block-diagonal x (see above)
    constexpr int kMaxWaves = WAVES, kX = few_x<WAVES, DIAG>();
    constexpr int kTile = DIAG ? 4 * 16 : MT * 16 * 16;
    constexpr int kStepB = 2048, kScaleB = 256;              // codes and scales of a tile and step
    constexpr int kStep = WF == WF_AFFINE8 ? 128 : 256;      // weights of a row and step
    constexpr int kRing = kMaxWaves * NT * kStepB, kScales = kMaxWaves * NT * kScaleB;
    static_assert(kMaxWaves * NT * kTile * 4 <= kRing, "the sums fit where the codes were");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing + kScales + kX + 64];
    uint8_t* xs = lds + kRing + kScales;
    float* red = reinterpret_cast<float*>(lds);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6, x_shift = split.x_shift, x_rows = 1 << x_shift;
    const int j = lane & 15, g = lane >> 4;
    const int K = (int)a.K, N = (int)a.N, M = (int)a.M;
    const int nb = K / 32, s0 = (int)blockIdx.y * split.per, left_steps = (K + kStep - 1) / kStep - s0;
    const int steps = left_steps < split.per ? left_steps : split.per;     // of this part, counted from s0
    constexpr int kCols = GATED ? NT / 2 : NT;              // column tiles of 16 outputs
    const int n0 = (int)blockIdx.x * kCols * 16;

    // ---- a step's loads.  Tile t, row i of it; rows past N repeat the last one
    // (never stored), pieces past the row's end its last (x is zero there) ----
    const uint32_t row_q = (uint32_t)(WF == WF_AFFINE8 ? K : K / 2), row_s = (uint32_t)(WF == WF_Q4_0 ? nb : K / 64);
    auto tile_first = [&](int t) __attribute__((always_inline)) {
        const int first = n0 + (GATED ? t >> 1 : t) * 16;
        return first < N ? first : N - 1;
    };
    auto tile_w = [&](int t) -> const QuantW& { return a.w[GATED ? t & 1 : 0]; };
    uint32_t copy_row[2];                                    // this lane's rows in the two copies
#pragma unroll
    for (int h = 0; h < 2; h++) copy_row[h] = (uint32_t)(8 * h + (lane >> 3));
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds) +
                          (uint32_t)wave * NT * kStepB;
    constexpr int kSL = (NT + 3) / 4;                        // scale loads: lane = tile * 16 + row
    u32x4_t sc[kSL];
    auto request = [&](int step) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const int first = tile_first(t), in = N - 1 - first;
            const uint8_t* base = tile_w(t).q + (int64_t)first * row_q;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const uint32_t row = copy_row[h] < (uint32_t)in ? copy_row[h] : (uint32_t)in;
                const uint32_t p = (uint32_t)(s0 + step) * 8u + ((uint32_t)(lane & 7) ^ (copy_row[h] & 7u)), last = row_q / 16 - 1;
                copy_unit(base, row * row_q + (p < last ? p : last) * 16u, lds0 + t * kStepB + h * 1024);
            }
        }
#pragma unroll
        for (int e = 0; e < kSL; e++) {
            int t = e * 4 + g;
            t = t < NT ? t : NT - 1;
            const QuantW& w = GATED ? a.w[t & 1] : a.w[0];
            int n = n0 + (GATED ? t >> 1 : t) * 16 + j;
            n = n < N ? n : N - 1;
            const int64_t at = (int64_t)n * row_s;
            constexpr int kPer = WF == WF_Q4_0 ? 8 : kStep / 64;        // scales of a row and step
            const int first = (s0 + step) * kPer;
            if (first + kPer <= (int)row_s) {
                if constexpr (WF == WF_Q4_0) {
                    sc[e] = *reinterpret_cast<const u32x4_u*>(w.s + at + first);
                } else if constexpr (WF == WF_AFFINE4) {
                    const u32x2_t s = *reinterpret_cast<const u32x2_u*>(w.s + at + first), b = *reinterpret_cast<const u32x2_u*>(w.b + at + first);
                    sc[e] = u32x4_t{s[0], s[1], b[0], b[1]};
                } else {
                    sc[e] = u32x4_t{*reinterpret_cast<const u32_u*>(w.s + at + first), 0u, *reinterpret_cast<const u32_u*>(w.b + at + first), 0u};
                }
            } else {
                // the last step of a K that is no multiple of it: one by one, zeros past the end
                u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int i = 0; i < kPer; i++)
                    if (first + i < (int)row_s) {
                        v[i >> 1] |= (uint32_t)w.s[at + first + i] << (16 * (i & 1));
                        if constexpr (WF != WF_Q4_0) v[2 + (i >> 1)] |= (uint32_t)w.b[at + first + i] << (16 * (i & 1));
                    }
                sc[e] = v;
            }
        }
    };

    // ---- x in LDS: [chunk of 128 k][MFMA][row][g][16 bytes], blocks past K zeros.
    // Piece u of that order, of chunk c: its load, and its place. ----
    auto x_piece = [&](int c, int u) __attribute__((always_inline)) {
        const uint16_t* x = static_cast<const uint16_t*>(a.x);
        const int gg = u & 3, m = (u >> 2) & (x_rows - 1), b = 4 * (s0 * (kStep / 128) + c) + ((u >> (2 + x_shift)) & 3);     // block of 32
        u32x4_t v = {0u, 0u, 0u, 0u};
        if (b < nb) {
            const uint16_t* p = x + (int64_t)(m < M ? m : M - 1) * K;
            if constexpr (WF == WF_Q4_0) {
                // elements 4 g .. + 3 and 16 + 4 g .. + 3
                const u32x2_t lo = *reinterpret_cast<const u32x2_t*>(p + b * 32 + 4 * gg);
                const u32x2_t hi = *reinterpret_cast<const u32x2_t*>(p + b * 32 + 16 + 4 * gg);
                v = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
            } else if constexpr (WF == WF_AFFINE4) {
                v = *reinterpret_cast<const u32x4_t*>(p + b * 32 + 8 * gg);
            } else {
                v = *reinterpret_cast<const u32x4_t*>(p + (b & ~1) * 32 + 16 * gg + 8 * (b & 1));
            }
        }
        return v;
    };
    auto x_put = [&](int u, const u32x4_t& v) __attribute__((always_inline)) {
        u32x4_t o = v;
        if constexpr (WF == WF_Q4_0)          // nibble pairs (0, 2), (1, 3) of either half
            o = u32x4_t{__builtin_amdgcn_perm(v[1], v[0], 0x05040100u), __builtin_amdgcn_perm(v[1], v[0], 0x07060302u),
                        __builtin_amdgcn_perm(v[3], v[2], 0x05040100u), __builtin_amdgcn_perm(v[3], v[2], 0x07060302u)};
        if constexpr (WF == WF_AFFINE4)       // byte i holds elements 2 i and 2 i + 1: pairs (0, 4), (2, 6), (1, 5), (3, 7)
            o = u32x4_t{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x05040100u),
                        __builtin_amdgcn_perm(v[2], v[0], 0x07060302u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
        *reinterpret_cast<u32x4_t*>(xs + u * 16) = o;
    };
    int xat[MT];                                             // this lane's piece of an MFMA's x
#pragma unroll
    for (int i = 0; i < MT; i++) xat[i] = ((i * 16 + j < x_rows ? i * 16 + j : x_rows - 1) * 4 + g) * 16;

    floatx4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[i][t] = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t mask = 0x000F000Fu;
    asm volatile("" : "+v"(mask));           // in a register: one v_and_or_b32 a pair
    const floatx4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
    auto splat = [](uint32_t v) { return u32x4_t{v, v, v, v}; };

    // kBlocks: this lane's row of A is 4 m + b; its x, or the zeros after the slice
    const bool diag = (j & 3) == g && (j >> 2) < x_rows;
    const int diag_at = ((j & 3) * x_rows + (j >> 2)) * 64;
    if (threadIdx.x < 16) reinterpret_cast<uint32_t*>(xs + kX)[threadIdx.x] = 0u;

    // A chunk of 128 k: codes q (8 bits: two pieces) and scales of every tile, x
    // chunk `local` of the slice in LDS.  Scale e of the chunk (of its blocks at
    // Q4_0, of its groups else) and bias e.
    struct Codes {
        u32x4_t q[WF == WF_AFFINE8 ? 2 : 1];
        uint32_t s[2];
    };
    auto scale = [](const Codes& c, int e) __attribute__((always_inline)) {
        if constexpr (WF == WF_Q4_0) return f16_to_f32((c.s[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
        else return bf16_to_f32((c.s[0] >> (16 * e)) & 0xFFFFu);
    };
    auto bias = [](const Codes& c, int e) __attribute__((always_inline)) { return bf16_to_f32((c.s[1] >> (16 * e)) & 0xFFFFu); };
    auto compute = [&](Codes (&w)[NT], int local) __attribute__((always_inline)) {
        u32x4_t x[MT][4];
        if constexpr (kBlocks) {
            const uint8_t* p = diag ? xs + local * 4 * x_rows * 64 + diag_at : xs + kX;
#pragma unroll
            for (int r = 0; r < 4; r++) x[0][r] = *reinterpret_cast<const u32x4_t*>(p + r * 16);
            // Q4_0: codes less 8; affine: the sums of x for the group's bias too
            constexpr bool kOffset = XDT == DT_BF16;
            const uint32_t one = WF == WF_Q4_0 ? lowered<WF>(0xC308u) : kOffset ? lowered<WF>(0xC300u) : 0x3C003C00u;
            floatx4_t cs = zero;
            if (kOffset || WF == WF_AFFINE4) {
#pragma unroll
                for (int r = 0; r < 4; r++) cs = mfma16<XDT>(x[0][r], splat(one), cs);
            }
#pragma unroll
            for (int n = 0; n < NT; n++) {
                floatx4_t v = kOffset ? cs : zero;
#pragma unroll
                for (int r = 0; r < 4; r++) v = mfma16<XDT>(x[0][r], nibbles<XDT, WF == WF_Q4_0 ? 8 : 0>(w[n].q[0][r], mask), v);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    if constexpr (WF == WF_Q4_0) acc[0][n][e] = fmaf(scale(w[n], e), v[e], acc[0][n][e]);
                    else
                        acc[0][n][e] = fmaf(bias(w[n], e >> 1) * (kOffset ? -0.0078125f : 1.0f), cs[e],
                                            fmaf(scale(w[n], e >> 1), v[e], acc[0][n][e]));
                }
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int t = 0; t < 4; t++)
                x[i][t] = *reinterpret_cast<const u32x4_t*>(xs + (local * 4 + t) * x_rows * 64 + xat[i]);
        if constexpr (WF == WF_Q4_0) {
#pragma unroll
            for (int n = 0; n < NT; n++) transpose4(w[n].q[0]);
#pragma unroll
            for (int t = 0; t < 4; t++) {
                floatx4_t c0[MT];
#pragma unroll
                for (int i = 0; i < MT; i++)
                    c0[i] = XDT == DT_BF16 ? mfma16<XDT>(x[i][t], splat(lowered<WF>(0xC308u)), zero) : zero;      // -136 sum x
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    const u32x4_t c = nibbles<XDT, 8>(w[n].q[0][t], mask);
                    const float d = scale(w[n], t);
#pragma unroll
                    for (int i = 0; i < MT; i++) {
                        const floatx4_t v = mfma16<XDT>(x[i][t], c, c0[i]);
#pragma unroll
                        for (int e = 0; e < 4; e++) acc[i][n][e] = fmaf(d, v[e], acc[i][n][e]);
                    }
                }
            }
        } else {
            if constexpr (WF == WF_AFFINE4) {
#pragma unroll
                for (int n = 0; n < NT; n++) transpose4(w[n].q[0]);
            }
            // 4 bits, bfloat16: the codes are 128 + q, so the sums of x enter as -128 sum x
            constexpr bool kOffset = WF == WF_AFFINE4 && XDT == DT_BF16;
            const uint32_t one = kOffset ? lowered<WF>(0xC300u) : XDT == DT_BF16 ? lowered<WF>(0x3F80u) : 0x3C003C00u;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                floatx4_t cs[MT];
#pragma unroll
                for (int i = 0; i < MT; i++)
                    cs[i] = mfma16<XDT>(x[i][2 * h + 1], splat(one), mfma16<XDT>(x[i][2 * h], splat(one), zero));
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    u32x4_t w0, w1;
                    if constexpr (WF == WF_AFFINE4) {
                        w0 = nibbles<XDT, 0>(w[n].q[0][2 * h], mask);
                        w1 = nibbles<XDT, 0>(w[n].q[0][2 * h + 1], mask);
                    } else {
                        w0 = bytes8<XDT>(w[n].q[h][0], w[n].q[h][1]);
                        w1 = bytes8<XDT>(w[n].q[h][2], w[n].q[h][3]);
                    }
                    const float s = scale(w[n], h), b = bias(w[n], h) * (kOffset ? -0.0078125f : 1.0f);
#pragma unroll
                    for (int i = 0; i < MT; i++) {
                        const floatx4_t v =
                            mfma16<XDT>(x[i][2 * h + 1], w1, mfma16<XDT>(x[i][2 * h], w0, kOffset ? cs[i] : zero));
#pragma unroll
                        for (int e = 0; e < 4; e++) acc[i][n][e] = fmaf(b, cs[i][e], fmaf(s, v[e], acc[i][n][e]));
                    }
                }
            }
        }
    };

    // A wave takes steps wave, wave + waves, ..
    constexpr int kChunks = kStep / 128;                     // of a step
    uint8_t* codes = lds + wave * NT * kStepB;
    uint8_t* scales = lds + kRing + wave * NT * kScaleB;
    // The step in flight (nothing later is) into registers: its scales change
    // places in LDS, its copies have landed.
    auto take = [&](Codes (&w)[kChunks][NT]) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < kSL; e++)
            if (e * 4 + g < NT) *reinterpret_cast<u32x4_t*>(scales + (e * 64 + lane) * 16) = sc[e];
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        Q4_WAIT_VMCNT(0);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
#pragma unroll
        for (int n = 0; n < NT; n++) {
            u32x4_t q[2];
#pragma unroll
            for (int h = 0; h < 2; h++)
                q[h] = *reinterpret_cast<const u32x4_t*>(codes + n * kStepB + j * 128 + (((4 * h + g) ^ (j & 7)) * 16));
            const u32x4_t s = *reinterpret_cast<const u32x4_t*>(scales + (n * 16 + j) * 16);
            if constexpr (WF == WF_AFFINE8) {
                w[0][n] = Codes{{q[0], q[1]}, {s[0], s[2]}};
            } else {
#pragma unroll
                for (int h = 0; h < kChunks; h++)
                    w[h][n] = WF == WF_Q4_0 ? Codes{{q[h]}, {s[2 * h], s[2 * h + 1]}} : Codes{{q[h]}, {s[h], s[2 + h]}};
            }
        }
        // the reads are in registers before the next copies overwrite them
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_s_waitcnt(0xC07F);                  // lgkmcnt(0)
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
    };
    if constexpr (DIAG) {
        // x is staged for `round` steps of every wave at a time, all of K as a
        // rule.  Its first pieces are requested before the codes (loads return in
        // order), so that x waits in LDS when the codes arrive.
        const int round = kX / (x_rows * 256 * kChunks) / waves;
        const int most = round * waves * kChunks, all = steps * kChunks;
        const int piece_shift = 4 + x_shift;                 // pieces of a chunk: 16 x_rows
        constexpr int kEarly = 4;
        u32x4_t early[kEarly];
        const int pieces0 = (all < most ? all : most) << piece_shift;
#pragma unroll
        for (int e = 0; e < kEarly; e++) {
            const int u = (int)(threadIdx.x + e * blockDim.x);
            early[e] = x_piece(u >> piece_shift, u);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (wave < steps) request(wave);         // a copy that nobody waits for would land in the sums
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = 0; e < kEarly; e++) {
            const int u = (int)(threadIdx.x + e * blockDim.x);
            if (u < pieces0) x_put(u, early[e]);
        }
        for (int r0 = 0; r0 * waves < steps; r0 += round) {
            if (r0 > 0) __syncthreads();
            const int first = r0 * waves * kChunks, left = all - first;
            const int pieces = (left < most ? left : most) << piece_shift;
            for (int u = (r0 == 0 ? kEarly * (int)blockDim.x : 0) + (int)threadIdx.x; u < pieces; u += blockDim.x)
                x_put(u, x_piece(first + (u >> piece_shift), u));
            __syncthreads();
            for (int r = r0; r < r0 + round; r++) {
                const int step = r * waves + wave;
                if (step >= steps) break;
                Codes w[kChunks][NT];
                take(w);
                if (step + waves < steps) request(step + waves);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int h = 0; h < kChunks; h++) compute(w[h], step * kChunks + h - first);
            }
        }
    } else {
        // x of kXC chunks of every wave at a time, requested into registers before
        // the codes of the step after, so that it does not wait behind them
        constexpr int kXC = MT == 1 ? kChunks : 1, kXP = kXC * MT * 4;       // pieces a thread
        static_assert(kMaxWaves * kXC * MT * 16 * 256 <= kX, "x of a round fits");
        u32x4_t xn[kXP];
        const int piece_shift = 4 + x_shift, pieces = (waves * kXC) << piece_shift;
        auto x_request = [&](int r, int h) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < kXP; e++) {
                const int u = (int)(threadIdx.x + e * blockDim.x), lc = u >> piece_shift;
                xn[e] = x_piece((r * waves + lc / kXC) * kChunks + h + lc % kXC, u);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        auto x_swap = [&]() __attribute__((always_inline)) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kXP; e++) {
                const int u = (int)(threadIdx.x + e * blockDim.x);
                if (u < pieces) x_put(u, xn[e]);
            }
            __syncthreads();
        };
        x_request(0, 0);
        if (wave < steps) request(wave);
        for (int r = 0; r * waves < steps; r++) {
            const int step = r * waves + wave;
            Codes w[kChunks][NT];
            x_swap();
            const bool live = step < steps;
            if (live) take(w);
            if (kXC == kChunks) {
                x_request(r + 1, 0);
                if (step + waves < steps) request(step + waves);
                __builtin_amdgcn_sched_barrier(0);
                if (live) {
#pragma unroll
                    for (int h = 0; h < kChunks; h++) compute(w[h], wave * kXC + h);
                }
            } else {
                x_request(r, 1);
                if (step + waves < steps) request(step + waves);
                __builtin_amdgcn_sched_barrier(0);
                if (live) compute(w[0], wave);
                x_swap();
                x_request(r + 1, 0);
                if (live) compute(w[kChunks - 1], wave);
            }
        }
    }
    __syncthreads();

    // lane: column j, rows 4 g + e of each 16 x 16 tile (DIAG: row g, its blocks)
#pragma unroll
    for (int n = 0; n < NT; n++) {
        if constexpr (kBlocks) {
            red[(wave * NT + n) * kTile + g * 16 + j] = (acc[0][n][0] + acc[0][n][1]) + (acc[0][n][2] + acc[0][n][3]);
            continue;
        }
        if constexpr (DIAG) {
            if (g == 0) {
#pragma unroll
                for (int e = 0; e < 4; e++) red[(wave * NT + n) * kTile + e * 16 + j] = acc[0][n][e];
            }
            continue;
        }
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                red[(wave * NT + n) * kTile + (i * 16 + 4 * g + e) * 16 + j] = acc[i][n][e];
    }
    __syncthreads();
    for (int o = threadIdx.x; o < M * kCols * 16; o += blockDim.x) {
        const int col = o & 15, p = (o >> 4) % kCols, m = (o >> 4) / kCols;
        const int n = n0 + p * 16 + col;
        if (n >= N) continue;
        auto sum = [&](int t) __attribute__((always_inline)) {
            float v = red[t * kTile + m * 16 + col];
            for (int w = 1; w < waves; w++) v += red[(w * NT + t) * kTile + m * 16 + col];
            if (v != v) {
                const int k0 = s0 * kStep, k1 = k0 + steps * kStep;
                v = spoilt_sum<WF>(a.w[GATED ? t & 1 : 0], static_cast<const uint16_t*>(a.x) + (int64_t)m * K, XDT, n, K, k0,
                                   k1 < K ? k1 : K, v);
            }
            return v;
        };
        const int64_t at = (int64_t)m * N + n;
        constexpr float kUp = (float)(1 << kDown<WF, XDT>);
        float z = sum(GATED ? 2 * p : p);
        if (split.part) {
            float* row = split.part + ((int64_t)blockIdx.y * split.rows + m) * split.np;
            row[GATED ? (n >> 5) * 64 + (n & 31) : n] = z;
            if constexpr (GATED) row[(n >> 5) * 64 + 32 + (n & 31)] = sum(2 * p + 1);
            continue;
        }
        z *= kUp;
        if (a.bias[0]) z += load_elem(a.bias[0], XDT, n);
        if (a.pre[0]) store_elem(a.pre[0], XDT, at, z);
        float zs[1] = {z}, none[1];
        activate_all<false>(a.act, zs, zs, none);
        float y = zs[0];
        if constexpr (GATED) {
            float u = sum(2 * p + 1) * kUp;
            if (a.bias[1]) u += load_elem(a.bias[1], XDT, n);
            if (a.pre[1]) store_elem(a.pre[1], XDT, at, u);
            y *= u;
        }
        if (a.residual) y += load_elem(a.residual, XDT, at);
        store_elem(a.y, XDT, at, y);
    }
}

// ---- host ------------------------------------------------------------------------

constexpr int kFewMaxM = 32;

// Column tiles (at q4_gated pairs) of a workgroup, its waves, the parts of a sum
// and the steps of a part.
struct FewPlan {
    int tiles, waves, parts, per;
};
FewPlan plan_few(int wf, int nmat, int64_t M, int64_t N, int64_t K);
// Rows at which three column tiles a workgroup are there (measured at plan_few).
constexpr bool few_three(int wf, int64_t M) { return wf != WF_AFFINE8 || (M > 4 && M <= 16); }
// What takes the factor off the sums of a split again.
inline float few_unit(int wf, int dtype) {
    return dtype != DT_BF16 ? 1.0f : (float)(1 << (wf == WF_AFFINE8 ? few::kDown<WF_AFFINE8, DT_BF16> : few::kDown<WF_Q4_0, DT_BF16>));
}

template <int WF, int XDT, int MT, int P, bool GATED, bool DIAG, int WAVES>
void few_launch(const LinearArgs& a, const FewPlan& plan, FewSplit split, hipStream_t s) {
    split.x_shift = 0;
    while ((1 << split.x_shift) < a.M) split.x_shift++;
    split.per = plan.per;
    const dim3 grid((unsigned)((a.N + 16 * P - 1) / (16 * P)), (unsigned)plan.parts);
    hipLaunchKernelGGL((k_linear_few<WF, XDT, MT, GATED ? 2 * P : P, GATED, DIAG, WAVES>), grid,
                       dim3(64 * (unsigned)(plan.per < WAVES ? plan.per : WAVES)), 0, s, a, split);
}
template <int WF, int XDT, int MT, int P, bool GATED, bool DIAG>
void few_waves(const LinearArgs& a, const FewPlan& p, const FewSplit& split, hipStream_t s) {
    if (DIAG || p.waves == 8) few_launch<WF, XDT, MT, P, GATED, DIAG, 8>(a, p, split, s);
    else few_launch<WF, XDT, MT, P, GATED, DIAG, DIAG ? 8 : 4>(a, p, split, s);
}
template <int WF, int XDT, int MT, bool DIAG>
void few_tiles(const LinearArgs& a, const FewPlan& p, const FewSplit& split, hipStream_t s) {
    if (a.nmat == 2) few_waves<WF, XDT, MT, 1, true, DIAG>(a, p, split, s);
    else if (p.tiles == 1) few_waves<WF, XDT, MT, 1, false, DIAG>(a, p, split, s);
    else if (p.tiles == 2) few_waves<WF, XDT, MT, 2, false, DIAG>(a, p, split, s);
    else if constexpr (few_three(WF, DIAG ? 1 : MT * 16)) few_launch<WF, XDT, MT, 3, false, DIAG, 8>(a, p, split, s);   // one workgroup a CU
}
template <int WF, int XDT>
void few_rows(const LinearArgs& a, const FewPlan& p, const FewSplit& split, hipStream_t s) {
    if (a.M <= 4) few_tiles<WF, XDT, 1, true>(a, p, split, s);
    else if (a.M <= 16) few_tiles<WF, XDT, 1, false>(a, p, split, s);
    else few_tiles<WF, XDT, 2, false>(a, p, split, s);
}
template <int WF>
hipError_t few_format(const LinearArgs& a, const FewPlan& p, const FewSplit& split, hipStream_t s) {
    if (a.dtype == DT_BF16) few_rows<WF, DT_BF16>(a, p, split, s);
    else few_rows<WF, DT_F16>(a, p, split, s);
    return hipGetLastError();
}

// One translation unit a format (linear_few_*.hip).
hipError_t launch_few_q4_0(const LinearArgs& a, const FewPlan& p, const FewSplit& split, hipStream_t s);
hipError_t launch_few_affine4(const LinearArgs& a, const FewPlan& p, const FewSplit& split, hipStream_t s);
hipError_t launch_few_affine8(const LinearArgs& a, const FewPlan& p, const FewSplit& split, hipStream_t s);

}  // namespace q4
