// mx_few.hip -- mx_linear and mx_gated at few rows (decode, small batches): the
// weights are streamed once, straight from their planes into the matrix
// instruction's registers.
//
// Mathematics.  With MX x a 16x16x128 scaled MFMA takes the codes and scales as
// they are.  With 16-bit x the codes are converted with their scale to bfloat16,
// which holds them exactly (2 bits and any scale up to 2^125; see bf16_scale), and
// multiplied by bfloat16 x in four 16x16x32 MFMAs; binary16 x is split into two
// bfloat16 parts, x = hi + lo exactly, and takes eight.  Products are exact, sums binary32.
//
// Layout.  Lane l of the MFMA holds one block of 32 of A's row j = l & 15, block
// slot g = l >> 4.  Taken as 16 rows of W, neighbouring lanes lie on different rows.
// Up to four rows of x (P = 4) A's row j is instead slice p = j & 3 of row j >> 2
// of W, and B's column the slice q = c & 3 of row c >> 2 of x: a load of W is four
// rows by 256 contiguous bytes, and of the 16 x 16 sums those with p = q count,
// four lanes' worth added up at the end.  Above four rows P is 1.
//
// A wave takes groups of four such chunks (64 blocks a row at P = 4, else 16) of R row
// tiles, all of a group's loads before its first product; the waves of a workgroup
// split the sum (KW of them) and the rows, and add their sums through LDS in wave
// order.  Of more than 64 rows a row of workgroups takes 64 each.  Scales: one 16-byte load a tile and group.  Above four rows x comes by
// direct copies to LDS, a wave's own part of it.
//
// Bounds.  One row: memory, and the round trip of a short launch: a pair of 12288 x 4096
// in 11.5 us (53.5 MB, 4.65 TB/s; a large copy reaches 5.2), one in 7.3, one 32768 x 4096 in
// 13.6 (5.2 TB/s), one 2048 x 8192 with bfloat16 x in 4.9.  5 to 64 rows: every workgroup
// reads all of x through LDS (12288 x 4096 with 8-bit x: 16 rows 8.5, 32 9.6, 64 13.0 us), and a
// wave waits for each stage of x with nothing else in flight, as it does for the weights of its
// next group; 16-bit x also the conversions beside the products (10.8 us at 32 rows with bfloat16,
// 16.2 with binary16, whose products are twice as many).
#include "gemm_common.hpp"
#include "mx_few.hpp"
#include "tile_image.hpp"

namespace q4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef u32x4_t u32x4_b __attribute__((aligned(1)));

// Dword r of lane row g's 16 bytes -> dword g of lane row r's.
__device__ __forceinline__ void transpose4(u32x4_t& q) {
    uint32_t a = q[0], b = q[1], c = q[2], d = q[3];
    auto swap32 = [](uint32_t& x, uint32_t& y) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
        x = r[0];
        y = r[1];
    };
    auto swap16 = [](uint32_t& x, uint32_t& y) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
        x = r[0];
        y = r[1];
    };
    swap32(a, c);
    swap32(b, d);
    swap16(a, b);
    swap16(c, d);
    q = u32x4_t{a, b, c, d};
}

// Sixteen scales of a row from block `first` on, zeros past the row's nb.
__device__ __forceinline__ u32x4_t scales16(const uint8_t* row, int first, int nb) {
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (first + 16 <= nb) return *reinterpret_cast<const u32x4_b*>(row + first);
#pragma unroll
    for (int e = 0; e < 16; e++)
        if (first + e < nb) v[e >> 2] |= (uint32_t)row[first + e] << (8 * (e & 3));
    return v;
}

// Four consecutive 16-bit values, `left` of them inside the tensor; vec: rows
// are multiples of four.
__device__ __forceinline__ void add4(const void* p, int dt, int64_t at, int left, bool vec, float (&z)[4]) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    if (vec) {
        const u32x2_t v = *reinterpret_cast<const u32x2_t*>(q);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const uint32_t h = (v[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
            z[e] += dt == DT_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; e++)
        if (e < left) z[e] += load_elem(p, dt, at + e);
}
__device__ __forceinline__ void put4(void* p, int dt, int64_t at, int left, bool vec, const float (&z)[4]) {
    if (vec) {
        *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(p) + at) = u32x2_t{pack2(dt, z[0], z[1]), pack2(dt, z[2], z[3])};
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; e++)
        if (e < left) store_elem(p, dt, at + e, z[e]);
}

}  // namespace

template <int XT, int P, int MT, int NM, int R>
__global__ __launch_bounds__(512, 1) void k_mx_few(const MxLinearArgs args, const MxFewPlan plan) {
    static_assert(P == 1 || MT == 1, "slices for few rows");
    constexpr bool kMx = XT == XT_MXFP4 || XT == XT_MXFP8;
    constexpr int kRows = 16 / P;                            // rows of W of a tile
    constexpr int kPitch = P == 4 ? 4 : 20;                  // sums of a tile: [x row][row of W], rows spread over the banks
    constexpr int kTile = (P == 4 ? 4 : 16 * MT) * kPitch;
    constexpr int kGroup = 16 * P;                           // blocks of a group of four chunks
    // x of a wave's stage of kStage chunks (P = 1): [chunk][tile of 16 rows][row][kRowB]
    constexpr int kRowB = XT == XT_MXFP8 ? 128 : XT == XT_MXFP4 ? 64 : 256;
    constexpr int kFit = 16384 / (kRowB * 16 * MT), kStage = P == 4 ? 0 : kFit < 4 ? kFit : 4;
    constexpr int kStageB = kStage * MT * 16 * kRowB, kRed = 8 * R * NM * kTile * 4;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[8 * kStageB > kRed ? 8 * kStageB : kRed];
    float* red = reinterpret_cast<float*>(lds);
    const LinearArgs& a = args.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kw = wave % plan.kw, rw = wave / plan.kw;
    const int j = lane & 15, g = lane >> 4, p = j & (P - 1);
    // above 64 rows a row of workgroups for each 64 of them
    const int64_t m_first = MT == 4 ? (int64_t)blockIdx.y * 64 : 0;
    const int K = (int)a.K, N = (int)a.N, nb = K / 32, M = (int)(MT == 4 && a.M - m_first > 64 ? 64 : a.M - m_first);
    const int n_first = ((int)blockIdx.x * plan.rw + rw) * R * kRows;

    const uint8_t* wq[R][NM];
    const uint8_t* wsc[R][NM];
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int t = 0; t < NM; t++) {
            int n = n_first + r * kRows + j / P;             // rows past N repeat the last one (never stored)
            n = n < N ? n : N - 1;
            wq[r][t] = a.w[t].q + (int64_t)n * (K / 2);
            wsc[r][t] = reinterpret_cast<const uint8_t*>(a.w[t].s) + (int64_t)n * nb;
        }
    int xm[MT];                                              // this lane's rows of x
#pragma unroll
    for (int i = 0; i < MT; i++) {
        xm[i] = i * 16 + j / P;
        xm[i] = xm[i] < M ? xm[i] : M - 1;
    }

    floatx4_t acc[R][NM][MT];
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int t = 0; t < NM; t++)
#pragma unroll
            for (int i = 0; i < MT; i++) acc[r][t][i] = floatx4_t{0.0f, 0.0f, 0.0f, 0.0f};

    // ---- P = 1: x by direct copies of whole lines, the pieces of 16 bytes of a row
    // placed by an XOR with the row, so that a wave's reads meet no bank twice ----
    constexpr int kPieces = kRowB / 16, kCopyRows = 64 / kPieces;       // of a row; rows of a copy
    auto swz = [](int r) { return kPieces == 4 ? ((r >> 1) & 3) ^ ((r >> 3) & 1) : kPieces == 8 ? (r & 7) ^ ((r >> 3) & 1) : r; };
    const uint32_t row_x = (uint32_t)(kMx ? (XT == XT_MXFP8 ? K : K / 2) : 2 * K), last_x = row_x / 16 - 1;
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds) +
                          (uint32_t)(wave * kStageB);
    auto stage_x = [&](int b0) __attribute__((always_inline)) {         // from block b0 on
#pragma unroll
        for (int i = 0; i < MT; i++) {
            const int first = i * 16 < M ? i * 16 : M - 1;
            const uint8_t* src = static_cast<const uint8_t*>(a.x) + (m_first + first) * row_x;
#pragma unroll
            for (int h = 0; h < 16 / kCopyRows; h++) {
                const int r = h * kCopyRows + lane / kPieces, in = M - 1 - first;
                const uint32_t at = (uint32_t)(r < in ? r : in) * row_x;
#pragma unroll
                for (int c = 0; c < kStage; c++) {
                    const uint32_t piece = (uint32_t)(b0 / 4 + c) * kPieces + (uint32_t)((lane % kPieces) ^ swz(r));
                    copy_unit(src, at + (piece < last_x ? piece : last_x) * 16,
                              lds0 + (uint32_t)(((c * MT + i) * 16 + h * kCopyRows) * kRowB));
                }
            }
        }
    };
    auto staged = [&](int c, int i, int piece) __attribute__((always_inline)) {
        return *reinterpret_cast<const u32x4_t*>(lds + wave * kStageB + ((c * MT + i) * 16 + j) * kRowB + ((piece ^ swz(j)) * 16));
    };

    const int groups = (nb + kGroup - 1) / kGroup;
    bool past = false;                                       // a scale was past bfloat16's range
    for (int kg = kw; kg < groups; kg += plan.kw) {
        const int b0 = kg * kGroup;
        // this lane's block of chunk c, kept inside the row
        auto block = [&](int c, int slot) __attribute__((always_inline)) {
            const int b = b0 + c * 4 * P + slot * P + p;
            return b < nb ? b : nb - 1;
        };
        u32x4_t w[R][NM][4], ws[R][NM];
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int t = 0; t < NM; t++) {
#pragma unroll
                for (int c = 0; c < 4; c++) w[r][t][c] = *reinterpret_cast<const u32x4_t*>(wq[r][t] + (int64_t)block(c, g) * 16);
                ws[r][t] = scales16(wsc[r][t], b0 + (P == 4 ? 16 * g : 0), nb);
            }
        // dword c: the scale of this lane's block of chunk c, in byte 0
        auto place = [&](u32x4_t& s) __attribute__((always_inline)) {
            if constexpr (P == 4) transpose4(s);
#pragma unroll
            for (int c = 0; c < 4; c++) s[c] >>= 8 * (P == 4 ? p : g);
        };
        u32x4_t xs[MT];
        if constexpr (kMx) {
#pragma unroll
            for (int i = 0; i < MT; i++) {
                xs[i] = scales16(args.x_s + (m_first + xm[i]) * nb, b0 + (P == 4 ? 16 * g : 0), nb);
                place(xs[i]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; r++)
#pragma unroll
            for (int t = 0; t < NM; t++) place(ws[r][t]);
#pragma unroll
        for (int c = 0; c < 4; c++) {
            if constexpr (P == 1) {
                if (c % kStage == 0) {
                    __atomic_signal_fence(__ATOMIC_SEQ_CST);
                    __builtin_amdgcn_s_waitcnt(0xC07F);      // lgkmcnt(0): the stage before is read
                    stage_x(b0 + 4 * c);
                    __atomic_signal_fence(__ATOMIC_SEQ_CST);
                    Q4_WAIT_VMCNT(0);
                    __atomic_signal_fence(__ATOMIC_SEQ_CST);
                }
            }
            if constexpr (kMx) {
                i32x8_t x[MT];
#pragma unroll
                for (int i = 0; i < MT; i++) {
                    const uint8_t* row = static_cast<const uint8_t*>(a.x) + (int64_t)xm[i] * (XT == XT_MXFP8 ? K : K / 2);
                    x[i] = i32x8_t{};
                    u32x4_t lo, hi = {0u, 0u, 0u, 0u};
                    if constexpr (P == 1) {
                        lo = staged(c % kStage, i, g);
                        if constexpr (XT == XT_MXFP8) hi = staged(c % kStage, i, 4 + g);
                    } else if constexpr (XT == XT_MXFP8) {
                        // the instruction's 8-bit order: half g & 1 of slots g >> 1 and 2 + (g >> 1)
                        lo = *reinterpret_cast<const u32x4_t*>(row + (int64_t)block(c, g >> 1) * 32 + 16 * (g & 1));
                        hi = *reinterpret_cast<const u32x4_t*>(row + (int64_t)block(c, 2 + (g >> 1)) * 32 + 16 * (g & 1));
                    } else {
                        lo = *reinterpret_cast<const u32x4_t*>(row + (int64_t)block(c, g) * 16);
                    }
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        x[i][e] = (int)lo[e];
                        if constexpr (XT == XT_MXFP8) x[i][4 + e] = (int)hi[e];
                    }
                }
#pragma unroll
                for (int r = 0; r < R; r++)
#pragma unroll
                    for (int t = 0; t < NM; t++) {
                        i32x8_t v = {};
#pragma unroll
                        for (int e = 0; e < 4; e++) v[e] = (int)w[r][t][c][e];
#pragma unroll
                        for (int i = 0; i < MT; i++)
                            acc[r][t][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                v, x[i], acc[r][t][i], 4, XT == XT_MXFP8 ? 0 : 4, 0, (int)ws[r][t][c], 0, (int)xs[i][c]);
                    }
            } else {
                const bool in = b0 + c * 4 * P + g * P + p < nb;
#pragma unroll
                for (int e = 0; e < 4; e++) {                // elements 8 e .. + 7 of every block
                    u32x4_t hi[MT], lo[MT];
#pragma unroll
                    for (int i = 0; i < MT; i++) {
                        const uint16_t* row = static_cast<const uint16_t*>(a.x) + (int64_t)xm[i] * K;
                        u32x4_t v;
                        if constexpr (P == 1) v = staged(c % kStage, i, 4 * g + e);
                        else v = *reinterpret_cast<const u32x4_t*>(row + (int64_t)block(c, g) * 32 + 8 * e);
                        if (!in) v = u32x4_t{0u, 0u, 0u, 0u};
                        if constexpr (XT == DT_BF16) {
                            hi[i] = v;
                        } else {
                            split_f16(v, hi[i], lo[i]);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < R; r++)
#pragma unroll
                        for (int t = 0; t < NM; t++) {
                            const float s = bf16_scale(ws[r][t][c] & 0xFFu, past);
                            const uint32_t d = w[r][t][c][e];
                            const u32x4_t q = {bf16_pair<0>(d, s), bf16_pair<1>(d, s), bf16_pair<2>(d, s), bf16_pair<3>(d, s)};
#pragma unroll
                            for (int i = 0; i < MT; i++) {
                                acc[r][t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    __builtin_bit_cast(bf16x8_t, q), __builtin_bit_cast(bf16x8_t, hi[i]), acc[r][t][i], 0, 0, 0);
                                if constexpr (XT == DT_F16)
                                    acc[r][t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                        __builtin_bit_cast(bf16x8_t, q), __builtin_bit_cast(bf16x8_t, lo[i]), acc[r][t][i], 0, 0, 0);
                            }
                        }
                }
            }
        }
    }

    // ---- 16-bit x: the blocks past bfloat16's range, as quarters of them four times ----
    if constexpr (!kMx) {
        if (__any(past)) {
#pragma unroll 1
            for (int slot = kw * 4; slot < groups * 4; slot = (slot & 3) == 3 ? slot + 4 * plan.kw - 3 : slot + 1) {
                const int b = slot * 4 * P + g * P + p, at = b < nb ? b : nb - 1;     // chunk of a group, its block of this lane
#pragma unroll 1
                for (int e = 0; e < 4; e++) {
                    u32x4_t hi[MT], lo[MT];
#pragma unroll
                    for (int i = 0; i < MT; i++) {
                        u32x4_t v = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.x) + (m_first + xm[i]) * K +
                                                                      (int64_t)at * 32 + 8 * e);
                        v = b < nb ? finite16<XT>(v) : u32x4_t{0u, 0u, 0u, 0u};
                        if constexpr (XT == DT_BF16) hi[i] = v;
                        else split_f16(v, hi[i], lo[i]);
                    }
#pragma unroll
                    for (int r = 0; r < R; r++)
#pragma unroll
                        for (int t = 0; t < NM; t++) {
                            const uint32_t s = wsc[r][t][at];
                            const uint32_t d = *reinterpret_cast<const uint32_t*>(wq[r][t] + (int64_t)at * 16 + 4 * e);
                            const u32x4_t q = bf16_quarters(past_bf16(s) ? d : 0u, mx_scale(past_bf16(s) ? s : 127u));
#pragma unroll
                            for (int i = 0; i < MT; i++)
#pragma unroll
                                for (int times = 0; times < 4; times++) {
                                    acc[r][t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                        __builtin_bit_cast(bf16x8_t, q), __builtin_bit_cast(bf16x8_t, hi[i]), acc[r][t][i], 0, 0, 0);
                                    if constexpr (XT == DT_F16)
                                        acc[r][t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                            __builtin_bit_cast(bf16x8_t, q), __builtin_bit_cast(bf16x8_t, lo[i]), acc[r][t][i], 0, 0, 0);
                                }
                        }
                }
            }
        }
    }

    // ---- the waves' sums, joined in order ----
    if constexpr (P == 1) __syncthreads();                   // they lie where x was
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int t = 0; t < NM; t++) {
            float* to = red + ((wave * R + r) * NM + t) * kTile;
            if constexpr (P == 4) {
                // lane (column c = 4 m + q, row g of W): its slice's sum, added over the four slices
                const floatx4_t v = acc[r][t][0];
                float s = p == 0 ? v[0] : p == 1 ? v[1] : p == 2 ? v[2] : v[3];
                s += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(s), 0xB1, 0xF, 0xF, false));
                s += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(s), 0x4E, 0xF, 0xF, false));
                if (p == 0) to[(j >> 2) * kPitch + g] = s;
            } else {
#pragma unroll
                for (int i = 0; i < MT; i++) *reinterpret_cast<floatx4_t*>(to + (i * 16 + j) * kPitch + 4 * g) = acc[r][t][i];
            }
        }
    __syncthreads();
    // four columns a thread
    auto finish = [&](auto type) __attribute__((always_inline)) {
        constexpr int kDt = decltype(type)::value;
        const int cols = plan.rw * R * kRows, quads = cols / 4, n0 = (int)blockIdx.x * cols;
        const bool vec = N % 4 == 0;
        for (int o = threadIdx.x; o < quads * M; o += blockDim.x) {
            const int m = o / quads, i = o % quads * 4, n = n0 + i, left = N - n;
            if (left <= 0) continue;
            const int tile = i / kRows, from = tile / R;          // row tile of the workgroup, its wave row
            auto sum = [&](int t, float (&z)[4]) __attribute__((always_inline)) {
                floatx4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int k = 0; k < plan.kw; k++)
                    v += *reinterpret_cast<const floatx4_t*>(red + (((from * plan.kw + k) * R + tile % R) * NM + t) * kTile +
                                                             m * kPitch + i % kRows);
#pragma unroll
                for (int e = 0; e < 4; e++) z[e] = v[e];
            };
            const int64_t at = (m_first + m) * N + n;
            float z[4], none[4];
            sum(0, z);
            if (a.bias[0]) add4(a.bias[0], kDt, n, left, vec, z);
            if (a.pre[0]) put4(a.pre[0], kDt, at, left, vec, z);
            activate_all<false>(a.act, z, z, none);
            if constexpr (NM == 2) {
                float u[4];
                sum(1, u);
                if (a.bias[1]) add4(a.bias[1], kDt, n, left, vec, u);
                if (a.pre[1]) put4(a.pre[1], kDt, at, left, vec, u);
#pragma unroll
                for (int e = 0; e < 4; e++) z[e] *= u[e];
            }
            if (a.residual) add4(a.residual, kDt, at, left, vec, z);
            put4(a.y, kDt, at, left, vec, z);
        }
    };
    if (XT == DT_BF16 || (XT != DT_F16 && a.dtype == DT_BF16)) finish(std::integral_constant<int, DT_BF16>{});
    else finish(std::integral_constant<int, DT_F16>{});
}

// ---- host ------------------------------------------------------------------------

namespace {

template <int XT, int P, int MT, int NM, int R>
void launch(const MxLinearArgs& a, const MxFewPlan& p, hipStream_t s) {
    hipLaunchKernelGGL((k_mx_few<XT, P, MT, NM, R>), dim3((unsigned)few_columns(p, a.a.M, a.a.N), (unsigned)few_chunks(a.a.M)),
                       dim3(few_threads(p)), 0, s, a, p);
}
template <int XT, int P, int MT, int NM>
void launch_r(const MxLinearArgs& a, const MxFewPlan& p, hipStream_t s) {
    if constexpr (MT * NM < 8) {
        if (p.r == 2) return launch<XT, P, MT, NM, 2>(a, p, s);
        if (p.r == 3) return launch<XT, P, MT, NM, 3>(a, p, s);
    }
    launch<XT, P, MT, NM, 1>(a, p, s);
}
template <int XT, int NM>
void launch_m(const MxLinearArgs& a, const MxFewPlan& p, hipStream_t s) {
    if (a.a.M <= 4) launch_r<XT, 4, 1, NM>(a, p, s);
    else if (a.a.M <= 16) launch_r<XT, 1, 1, NM>(a, p, s);
    else if (a.a.M <= 32) launch_r<XT, 1, 2, NM>(a, p, s);
    else launch_r<XT, 1, 4, NM>(a, p, s);
}
template <int XT>
void launch_x(const MxLinearArgs& a, const MxFewPlan& p, hipStream_t s) {
    if (a.a.nmat == 2) launch_m<XT, 2>(a, p, s);
    else launch_m<XT, 1>(a, p, s);
}

}  // namespace

bool mx_few_takes(int x_type, int nmat, int64_t M, int64_t N, int64_t K) {
    const bool mx = x_type == XT_MXFP8 || x_type == XT_MXFP4;
    return few_takes(mx ? FEW_MX : x_type == DT_BF16 ? FEW_BF16 : FEW_F16, nmat, M, N, K, current_cu_count());
}

hipError_t launch_mx_few(const MxLinearArgs& a, hipStream_t s) {
    const MxFewPlan p = plan_few(a.a.nmat, a.a.M, a.a.N, a.a.K, current_cu_count());
    if (!launchable(few_columns(p, a.a.M, a.a.N), few_threads(p))) return hipErrorInvalidValue;
    if (a.x_type == XT_MXFP8) launch_x<XT_MXFP8>(a, p, s);
    else if (a.x_type == XT_MXFP4) launch_x<XT_MXFP4>(a, p, s);
    else if (a.x_type == DT_BF16) launch_x<DT_BF16>(a, p, s);
    else launch_x<DT_F16>(a, p, s);
    return hipGetLastError();
}

}  // namespace q4
