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
// of x against a constant that serves every column.  With binary16 x the codes
// are q - 8 and q themselves.  Products are exact, sums binary32: the result
// differs from the exact one by binary32 summation and the output's rounding.
//
// Layout.  A lane (j = lane & 15, g = lane >> 4) loads 16 bytes of row j of a
// column tile: 16 rows of 64 contiguous bytes an instruction, 128 weights of a
// row at 4 bits.  At 4 bits that is block 4 c + g whole, where the MFMA of block
// t wants dword g of block 4 c + t: a 4 x 4 transposition over the four g, four
// lane swaps (v_permlane32_swap, v_permlane16_swap).  At 8 bits the MFMA's k
// order follows the load instead (a group has one scale).  The x fragments
// follow the same order and come from L2: every workgroup reads all of x, so a
// workgroup takes NT column tiles.
//
// The waves of a workgroup split K by chunks of 128, two chunks in flight each,
// and add their sums through LDS in wave order (deterministic).  For q4_gated
// the tiles come in pairs, gate and up of the same 16 columns.
//
// Bound: memory at 1 to 16 rows (each weight byte is read once).
#pragma once

#include "block_common.hpp"

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

// Eight codes of a dword, in the pair order (byte 0, byte 2), (1, 3) of the low
// nibbles, then of the high ones: bfloat16 128 + q, binary16 q - SUB.
template <int XDT, int SUB>
__device__ __forceinline__ u32x4_t nibbles(uint32_t w, uint32_t mask) {
    const uint32_t base = XDT == DT_BF16 ? 0x43004300u : 0x64006400u;
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
// Eight 8-bit codes, exact in either type, in order.
template <int XDT>
__device__ __forceinline__ u32x4_t bytes8(uint32_t lo, uint32_t hi) {
    u32x4_t r;
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const uint32_t w = e < 2 ? lo : hi;
        const f32x2_t f = {(float)((w >> (16 * (e & 1))) & 0xFFu), (float)((w >> (16 * (e & 1) + 8)) & 0xFFu)};
        if constexpr (XDT == DT_BF16) r[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
        else r[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, half2_t));
    }
    return r;
}

// A chunk of 128 k of one column tile: codes and scales.
template <int WF>
struct ChunkW {
    u32x4_t q[WF == WF_AFFINE8 ? 2 : 1];
    u32x2_t s;      // Q4_0: d of the four blocks; affine: s and b of the two groups
};

}  // namespace few

constexpr int kFewMaxM = 64;

template <int WF, int XDT, int MT, int NT, bool GATED>
__global__ __launch_bounds__(NT * MT <= 3 ? 1024 : 512) void k_linear_few(const LinearArgs a) {
    using namespace few;
    constexpr int kMaxWaves = NT * MT <= 3 ? 16 : 8;
    constexpr int kTile = MT * 16 * 16;
    __shared__ float red[kMaxWaves * NT * kTile];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int j = lane & 15, g = lane >> 4;
    const int K = (int)a.K, N = (int)a.N, M = (int)a.M;
    const int nb = K / 32, chunks = (K + 127) / 128;
    constexpr int kCols = GATED ? NT / 2 : NT;              // column tiles of 16 outputs
    const int n0 = (int)blockIdx.x * kCols * 16;

    // each tile's first row (scalar) and this lane's row in it; rows past N
    // repeat the last one and are never stored
    const uint8_t* wq[NT];
    const uint16_t* ws[NT];
    const uint16_t* wb[NT];
    uint32_t row[NT];
    const int64_t row_q = WF == WF_AFFINE8 ? K : K / 2, row_s = WF == WF_Q4_0 ? nb : K / 64;
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const QuantW& w = a.w[GATED ? t & 1 : 0];
        int first = n0 + (GATED ? t >> 1 : t) * 16;
        first = first < N ? first : N - 1;
        const int in = N - 1 - first;
        row[t] = (uint32_t)(j < in ? j : in);
        wq[t] = w.q + first * row_q;
        ws[t] = w.s + first * row_s;
        wb[t] = WF == WF_Q4_0 ? nullptr : w.b + first * row_s;
    }
    const uint8_t* xr[MT];
    uint32_t xrow[MT];
#pragma unroll
    for (int i = 0; i < MT; i++) {
        int first = i * 16;
        first = first < M ? first : M - 1;
        const int in = M - 1 - first;
        xrow[i] = (uint32_t)(j < in ? j : in) * (uint32_t)K * 2u;
        xr[i] = static_cast<const uint8_t*>(a.x) + (int64_t)first * K * 2;
    }

    struct Stage {
        ChunkW<WF> w[NT];
        u32x4_t x[MT][4];       // fragments of the four MFMAs of the chunk
    };
    auto load = [&](int c, Stage& st) __attribute__((always_inline)) {
        const bool whole = (c + 1) * 4 <= nb;                // the last chunk may be short
#pragma unroll
        for (int t = 0; t < NT; t++) {
            if constexpr (WF == WF_AFFINE8) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    int grp = 2 * c + h;
                    grp = grp < K / 64 ? grp : K / 64 - 1;
                    st.w[t].q[h] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(
                        wq[t] + (row[t] * (uint32_t)K + (uint32_t)grp * 64u + (uint32_t)g * 16u)));
                }
            } else {
                int b = 4 * c + g;
                b = b < nb ? b : nb - 1;
                st.w[t].q[0] = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4_t*>(wq[t] + (row[t] * (uint32_t)(K / 2) + (uint32_t)b * 16u)));
            }
            if constexpr (WF == WF_Q4_0) {
                const uint16_t* p = ws[t] + row[t] * (uint32_t)nb;
                if (whole) {
                    st.w[t].s = *reinterpret_cast<const u32x2_u*>(p + 4 * c);
                } else {
                    uint32_t d[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) d[e] = p[4 * c + e < nb ? 4 * c + e : nb - 1];
                    st.w[t].s = u32x2_t{d[0] | d[1] << 16, d[2] | d[3] << 16};
                }
            } else {
                const uint32_t at = row[t] * (uint32_t)(K / 64) + 2 * c;
                if (whole) {
                    st.w[t].s = u32x2_t{*reinterpret_cast<const u32_u*>(ws[t] + at), *reinterpret_cast<const u32_u*>(wb[t] + at)};
                } else {
                    st.w[t].s = u32x2_t{ws[t][at], wb[t][at]};
                }
            }
        }
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int t = 0; t < 4; t++) {
                // a block past K is read at the row's last block and zeroed
                const int b = 4 * c + t, bc = b < nb ? b : nb - 1;
                const uint8_t* p = xr[i] + (xrow[i] + (uint32_t)(WF == WF_AFFINE8 ? (bc & ~1) : bc) * 64u);
                u32x4_t v;
                if constexpr (WF == WF_Q4_0) {
                    const u32x2_t lo = *reinterpret_cast<const u32x2_t*>(p + 8 * g);
                    const u32x2_t hi = *reinterpret_cast<const u32x2_t*>(p + 32 + 8 * g);
                    v = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
                } else if constexpr (WF == WF_AFFINE4) {
                    v = *reinterpret_cast<const u32x4_t*>(p + 16 * g);
                } else {
                    v = *reinterpret_cast<const u32x4_t*>(p + 32 * g + 16 * (bc & 1));
                }
                if (b >= nb) v = u32x4_t{0u, 0u, 0u, 0u};
                st.x[i][t] = v;
            }
    };

    floatx4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int t = 0; t < NT; t++) acc[i][t] = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f};
    uint32_t mask = 0x000F000Fu;
    asm volatile("" : "+v"(mask));           // in a register: one v_and_or_b32 a pair
    const floatx4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
    auto splat = [](uint32_t v) { return u32x4_t{v, v, v, v}; };

    auto compute = [&](Stage& st) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int t = 0; t < 4; t++) {
                const u32x4_t v = st.x[i][t];
                if constexpr (WF == WF_Q4_0) {
                    // lo: elements 4 g .. 4 g + 3, hi: 16 + 4 g ..; nibble pairs (0, 2), (1, 3)
                    st.x[i][t] = u32x4_t{__builtin_amdgcn_perm(v[1], v[0], 0x05040100u), __builtin_amdgcn_perm(v[1], v[0], 0x07060302u),
                                         __builtin_amdgcn_perm(v[3], v[2], 0x05040100u), __builtin_amdgcn_perm(v[3], v[2], 0x07060302u)};
                } else if constexpr (WF == WF_AFFINE4) {
                    // byte i holds elements 2 i and 2 i + 1: pairs (0, 4), (2, 6), (1, 5), (3, 7)
                    st.x[i][t] = u32x4_t{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x05040100u),
                                         __builtin_amdgcn_perm(v[2], v[0], 0x07060302u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
                }
            }
        if constexpr (WF == WF_Q4_0) {
#pragma unroll
            for (int n = 0; n < NT; n++) transpose4(st.w[n].q[0]);
#pragma unroll
            for (int t = 0; t < 4; t++) {
                floatx4_t c0[MT];
#pragma unroll
                for (int i = 0; i < MT; i++)
                    c0[i] = XDT == DT_BF16 ? mfma16<XDT>(st.x[i][t], splat(0xC308C308u), zero) : zero;      // -136 sum x
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    const u32x4_t w = nibbles<XDT, 8>(st.w[n].q[0][t], mask);
                    const float d = f16_to_f32((st.w[n].s[t >> 1] >> (16 * (t & 1))) & 0xFFFFu);
#pragma unroll
                    for (int i = 0; i < MT; i++) {
                        const floatx4_t v = mfma16<XDT>(st.x[i][t], w, c0[i]);
#pragma unroll
                        for (int e = 0; e < 4; e++) acc[i][n][e] = fmaf(d, v[e], acc[i][n][e]);
                    }
                }
            }
        } else {
            if constexpr (WF == WF_AFFINE4) {
#pragma unroll
                for (int n = 0; n < NT; n++) transpose4(st.w[n].q[0]);
            }
            // 4 bits, bfloat16: the codes are 128 + q, so the sums of x enter as -128 sum x
            constexpr bool kOffset = WF == WF_AFFINE4 && XDT == DT_BF16;
            const uint32_t one = kOffset ? 0xC300C300u : XDT == DT_BF16 ? 0x3F803F80u : 0x3C003C00u;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                floatx4_t cs[MT];
#pragma unroll
                for (int i = 0; i < MT; i++)
                    cs[i] = mfma16<XDT>(st.x[i][2 * h + 1], splat(one), mfma16<XDT>(st.x[i][2 * h], splat(one), zero));
#pragma unroll
                for (int n = 0; n < NT; n++) {
                    u32x4_t w0, w1;
                    if constexpr (WF == WF_AFFINE4) {
                        w0 = nibbles<XDT, 0>(st.w[n].q[0][2 * h], mask);
                        w1 = nibbles<XDT, 0>(st.w[n].q[0][2 * h + 1], mask);
                    } else {
                        w0 = bytes8<XDT>(st.w[n].q[h][0], st.w[n].q[h][1]);
                        w1 = bytes8<XDT>(st.w[n].q[h][2], st.w[n].q[h][3]);
                    }
                    const float s = bf16_to_f32((st.w[n].s[0] >> (16 * h)) & 0xFFFFu);
                    const float b = bf16_to_f32((st.w[n].s[1] >> (16 * h)) & 0xFFFFu) * (kOffset ? -0.0078125f : 1.0f);
#pragma unroll
                    for (int i = 0; i < MT; i++) {
                        const floatx4_t v =
                            mfma16<XDT>(st.x[i][2 * h + 1], w1, mfma16<XDT>(st.x[i][2 * h], w0, kOffset ? cs[i] : zero));
#pragma unroll
                        for (int e = 0; e < 4; e++) acc[i][n][e] = fmaf(b, cs[i][e], fmaf(s, v[e], acc[i][n][e]));
                    }
                }
            }
        }
    };

    // chunks wave, wave + waves, ..: the next one loads while this one multiplies
    if (wave < chunks) {
        Stage s0, s1;
        load(wave, s0);
        for (int c = wave;;) {
            const int c1 = c + waves;
            load(c1 < chunks ? c1 : c, s1);
            __builtin_amdgcn_sched_barrier(0);
            compute(s0);
            if (c1 >= chunks) break;
            const int c2 = c1 + waves;
            load(c2 < chunks ? c2 : c1, s0);
            __builtin_amdgcn_sched_barrier(0);
            compute(s1);
            if (c2 >= chunks) break;
            c = c2;
        }
    }

    // lane: column j, rows 4 g + e of each 16 x 16 tile
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                red[(wave * NT + n) * kTile + (i * 16 + 4 * g + e) * 16 + j] = acc[i][n][e];
    __syncthreads();
    for (int o = threadIdx.x; o < M * kCols * 16; o += blockDim.x) {
        const int col = o & 15, p = (o >> 4) % kCols, m = (o >> 4) / kCols;
        const int n = n0 + p * 16 + col;
        if (n >= N) continue;
        auto sum = [&](int t) __attribute__((always_inline)) {
            float v = red[t * kTile + m * 16 + col];
            for (int w = 1; w < waves; w++) v += red[(w * NT + t) * kTile + m * 16 + col];
            return v;
        };
        const int64_t at = (int64_t)m * N + n;
        float z = sum(GATED ? 2 * p : p);
        if (a.bias[0]) z += load_elem(a.bias[0], XDT, n);
        if (a.pre[0]) store_elem(a.pre[0], XDT, at, z);
        float y = activate(a.act, z);
        if constexpr (GATED) {
            float u = sum(2 * p + 1);
            if (a.bias[1]) u += load_elem(a.bias[1], XDT, n);
            if (a.pre[1]) store_elem(a.pre[1], XDT, at, u);
            y *= u;
        }
        if (a.residual) y += load_elem(a.residual, XDT, at);
        store_elem(a.y, XDT, at, y);
    }
}

// ---- host ------------------------------------------------------------------------

template <int WF, int XDT, int MT, int P, bool GATED>
void few_launch(const LinearArgs& a, hipStream_t s) {
    constexpr int NT = GATED ? 2 * P : P;
    constexpr int kMaxWaves = NT * MT <= 3 ? 16 : 8;
    const int64_t chunks = (a.K + 127) / 128;
    const int waves = (int)(chunks < kMaxWaves ? chunks : kMaxWaves);
    const unsigned grid = (unsigned)((a.N + 16 * P - 1) / (16 * P));
    hipLaunchKernelGGL((k_linear_few<WF, XDT, MT, NT, GATED>), dim3(grid), dim3(64 * waves), 0, s, a);
}
template <int WF, int XDT, int MT, bool GATED>
void few_tiles(const LinearArgs& a, hipStream_t s) {
    // as few column tiles a workgroup as fill the CUs: each workgroup reads all of x
    const int64_t tiles = (a.N + 15) / 16, cus = current_cu_count();
    if (tiles <= cus) few_launch<WF, XDT, MT, 1, GATED>(a, s);
    else if (tiles <= 2 * cus || (MT == 4 && GATED)) few_launch<WF, XDT, MT, 2, GATED>(a, s);
    else few_launch<WF, XDT, MT, (MT == 4 && GATED) ? 2 : 3, GATED>(a, s);
}
template <int WF, int XDT>
void few_rows(const LinearArgs& a, hipStream_t s) {
    if (a.nmat == 2) {
        if (a.M <= 16) few_tiles<WF, XDT, 1, true>(a, s);
        else if (a.M <= 32) few_tiles<WF, XDT, 2, true>(a, s);
        else few_tiles<WF, XDT, 4, true>(a, s);
    } else {
        if (a.M <= 16) few_tiles<WF, XDT, 1, false>(a, s);
        else if (a.M <= 32) few_tiles<WF, XDT, 2, false>(a, s);
        else few_tiles<WF, XDT, 4, false>(a, s);
    }
}
template <int WF>
hipError_t few_format(const LinearArgs& a, hipStream_t s) {
    if (a.dtype == DT_BF16) few_rows<WF, DT_BF16>(a, s);
    else few_rows<WF, DT_F16>(a, s);
    return hipGetLastError();
}

// One translation unit a format (linear_few_*.hip).
hipError_t launch_few_q4_0(const LinearArgs& a, hipStream_t s);
hipError_t launch_few_affine4(const LinearArgs& a, hipStream_t s);
hipError_t launch_few_affine8(const LinearArgs& a, hipStream_t s);

}  // namespace q4
