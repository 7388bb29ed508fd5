// tile_pack.hip -- the packers of the dense product's operand images
// (tile_image.hpp): weights dequantised to binary16, by rows or transposed;
// activations and gradients scaled to binary16 row by row.  All are bound by
// memory (a quantised matrix read, two bytes a weight written).
#include "tile_image.hpp"

namespace q4 {

// ---- weights ---------------------------------------------------------------------
//
// Dequantised exactly in binary32 ((q - 8) d has 15 bits, q s + b one rounding)
// and rounded once to binary16.

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
template <int WF>
__device__ __forceinline__ RowScale<WF> row_scale(const QuantW& w, int64_t n, int64_t blk32, int64_t K) {
    if constexpr (WF == WF_Q4_0) {
        return {f16_to_f32(w.s[n * (K / 32) + blk32]), 0.0f};
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
// REST: the image has twice the slices, and the second half holds what the
// rounding to binary16 left of each weight (see launch_linear).
// Measured: two 12288 x 4096 Q4_0 matrices 44 us, 57 MB read and 201 MB written.
template <int WF, bool REST>
__global__ __launch_bounds__(256) void k_pack_weights(QuantW w0, QuantW w1, int mats, int N, int64_t K, int64_t slices,
                                                      int64_t kgroups, uint8_t* __restrict__ img) {
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
#pragma unroll
    for (int t = 0; t < kBlocks / 2; t++) {
        int64_t b = b0 + 2 * t + h;
        b = b < nb ? b : nb - 1;
        sc[t] = row_scale<WF>(w, n, b, K);
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
            if constexpr (REST) {
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
                                                        int64_t ktiles, int64_t ntiles, uint8_t* __restrict__ img) {
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
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const bool ok = in_k && n0 + i < N;
        const int64_t n = n0 + i < N ? n0 + i : N - 1, b = in_k ? blk : nb - 1;
        raw[i] = *reinterpret_cast<const uint32_t*>(w.q + (n * nb + b) * (128 / kPer) + wb * 4);
        sc[i] = row_scale<WF>(w, n, b, K);
        if (!ok) {
            sc[i].s = 0.0f;
            sc[i].b = 0.0f;
            raw[i] = 0u;
        }
    }
    uint8_t* base = lds + p * kPanelB + (o >> 1) * kUnit + (o & 1) * 512;
    auto put = [&](int j, auto code) __attribute__((always_inline)) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = sc[i](code(raw[i]));
        *reinterpret_cast<u32x4_t*>(base + j * 16) = pack8(DT_F16, f);
    };
    if constexpr (WF == WF_AFFINE8) {
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
static hipError_t pack_weights_t(int mats, const QuantW* w, int64_t N, int64_t K, bool transposed, bool rest, uint8_t* img,
                                 hipStream_t s) {
    if (!transposed) {
        constexpr int kGroupK = WF == WF_AFFINE8 ? 512 : 1024;
        const int64_t kgroups = (K + kGroupK - 1) / kGroupK, blocks = (N + 31) / 32 * mats * kgroups;
        if (!launchable(blocks, 256)) return hipErrorInvalidValue;
        hipLaunchKernelGGL((rest ? k_pack_weights<WF, true> : k_pack_weights<WF, false>), dim3((unsigned)blocks), dim3(256), 0,
                           s, w[0], w[mats - 1], mats, (int)N, K, image_slices(K) * (rest ? 2 : 1), kgroups, img);
    } else {
        constexpr int kTileK = WF == WF_AFFINE8 ? 128 : 256;
        const int64_t ktiles = (K + kTileK - 1) / kTileK, ntiles = (N + 63) / 64, blocks = ktiles * ntiles * mats;
        if (!launchable(blocks, 256)) return hipErrorInvalidValue;
        hipLaunchKernelGGL((k_pack_weights_t<WF>), dim3((unsigned)blocks), dim3(256), 0, s, w[0], w[mats - 1], (int)N, K,
                           image_slices(N) * mats, ktiles, ntiles, img);
    }
    return hipGetLastError();
}

hipError_t launch_pack_weights(int wf, int mats, const QuantW* w, int64_t N, int64_t K, bool transposed, bool rest,
                               uint8_t* img, hipStream_t s) {
    if (wf == WF_Q4_0) return pack_weights_t<WF_Q4_0>(mats, w, N, K, transposed, rest, img, s);
    if (wf == WF_AFFINE4) return pack_weights_t<WF_AFFINE4>(mats, w, N, K, transposed, rest, img, s);
    return pack_weights_t<WF_AFFINE8>(mats, w, N, K, transposed, rest, img, s);
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
constexpr int kPackThreads = 1024;

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

template <int ROWS>
__global__ __launch_bounds__(kPackThreads) void k_pack_rows(const void* __restrict__ x, int dtype, int64_t M, int64_t K,
                                                            int64_t slices, int twice, uint8_t* __restrict__ img,
                                                            int8_t* __restrict__ xexp) {
    __shared__ float red[kPackThreads / 64][8];
    const int lane = threadIdx.x & 63;
    constexpr int kStride = kPackThreads / ROWS;
    const int64_t m = (int64_t)blockIdx.x * ROWS + lane % ROWS, c0 = (threadIdx.x >> 6) * (64 / ROWS) + lane / ROWS;
    const int64_t row = (m < M ? m : M - 1) * K, chunks = K / 8;          // K % 32 == 0
    float v[8], mx = 0.0f;
    for (int64_t c = c0; c < chunks; c += kStride) {
        unpack8(dtype, load8_raw<true>(x, row + c * 8, 8), v);
        mx = max8(v, mx);
    }
    const int e = row_exponent(rows_max<ROWS>(mx, red));
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
                         hipStream_t s) {
    const int rows = pack_rows(M);
    const int64_t slices = image_slices(K) * (twice ? 2 : 1);
    for (int64_t m = 0; m < M; m += kLaunchRows) {
        const int64_t count = M - m < kLaunchRows ? M - m : kLaunchRows;
        hipLaunchKernelGGL(rows == 8 ? k_pack_rows<8> : k_pack_rows<4>, dim3((unsigned)((count + rows - 1) / rows)),
                           dim3(kPackThreads), 0, s, static_cast<const char*>(x) + m * K * 2, dtype, count, K, slices,
                           twice ? 1 : 0, img + m / 32 * slices * kUnit, xexp + m);
    }
    return hipGetLastError();
}

// dz of the projections: the same image (the projections' slices follow each
// other), the dz outputs rounded from the same binary32 values, and the sums of
// the workgroup's rows, joined by k_join_sums in a fixed order.
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
                                                          int8_t* __restrict__ xexp, float* __restrict__ sums) {
    __shared__ float red[kPackThreads / 64][8];
    const int lane = threadIdx.x & 63;
    constexpr int kStride = kPackThreads / ROWS;
    const int64_t m = (int64_t)blockIdx.x * ROWS + lane % ROWS, c0 = (threadIdx.x >> 6) * (64 / ROWS) + lane / ROWS;
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
                        if (col < left) sums[((int64_t)blockIdx.x * a.nmat + i) * a.N + c * 8 + col] = mine;
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

int64_t grad_sums_bytes(int nmat, int64_t M, int64_t N) { return (M + pack_rows(M) - 1) / pack_rows(M) * nmat * N * 4; }

hipError_t launch_pack_dz(const LinearGradArgs& a, uint8_t* img, int8_t* xexp, float* sums, hipStream_t s) {
    const int rows = pack_rows(a.M);
    const int64_t groups = (a.M + rows - 1) / rows, slices = image_slices(a.N);
    auto k = a.N % 8 == 0 ? (rows == 8 ? k_pack_dz<true, 8> : k_pack_dz<true, 4>)
                          : (rows == 8 ? k_pack_dz<false, 8> : k_pack_dz<false, 4>);
    for (int64_t m = 0; m < a.M; m += kLaunchRows) {
        LinearGradArgs t = a;
        auto from = [&](const void* p) { return p ? const_cast<char*>(static_cast<const char*>(p)) + m * a.N * 2 : nullptr; };
        t.M = a.M - m < kLaunchRows ? a.M - m : kLaunchRows;
        t.dy = from(a.dy);
        for (int i = 0; i < 2; i++) {
            t.pre[i] = from(a.pre[i]);
            t.dz[i] = from(a.dz[i]);
        }
        hipLaunchKernelGGL(k, dim3((unsigned)((t.M + rows - 1) / rows)), dim3(kPackThreads), 0, s, t, slices,
                           img + m / 32 * slices * a.nmat * kUnit, xexp + m, sums + m / rows * a.nmat * a.N);
    }
    if (a.dbias[0] || a.dbias[1])
        hipLaunchKernelGGL(k_join_sums, dim3((unsigned)((a.N + 63) / 64), a.nmat), dim3(1024), 0, s, sums, groups, a.nmat,
                           a.N, a.dbias[0], a.dbias[1]);
    return hipGetLastError();
}

}  // namespace q4
