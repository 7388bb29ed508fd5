// tile_gemm.hip -- the dense matrix-core product behind q4_linear, q4_gated
// and their gradients at many rows: Z[m][n] = sum_k X[m][k] W[n][k] over two
// binary16 images (tile_image.hpp), binary32 accumulation, with the operator's
// epilogue on the accumulators.
//
// A workgroup of four waves owns a tile of 2 NT x 2 MT panels (NT = MT = 4: 256
// columns x 256 rows); each wave owns NT x MT panels, that is NT MT accumulator
// tiles of 32 x 32 in the AGPRs: at 4 x 4 all 256 of them, one wave per SIMD.
// Per slice of 16 a wave reads NT + MT fragments for NT MT MFMAs, so at 4 x 4
// the CU reads 64 KiB and copies 32 KiB per 1024 MFMA cycles, 94 bytes a cycle
// of the about 110 that LDS moves; 8 waves of 4 x 2 would read 96 KiB.
//
// The sum runs in steps of two slices through a ring of four LDS slots that
// direct-to-LDS copies fill three to four steps ahead.  A step is T = 2 NT MT
// MFMAs with one barrier before MFMA 3 T / 4: by then this wave has read all of
// the step (its slot is free for the step after next but two) and waits until
// the next step has landed (two later ones stay in flight).  Reads stand at
// least six MFMAs before their use and copies are spread over the whole step:
// four waves in step that read one fragment per MFMA ask for all that LDS
// moves, and a burst of copies fills the address pipe; both held the matrix
// pipe (gated, M = 2048, N = 12288, K = 4096: 352 us with reads and copies
// bunched, 340 spread).  The order is written out and fenced: left alone, the
// compiler groups them again.
//
// What bounds it: power.  A loop of nothing but these MFMAs on random operands
// reaches 1.67 PFLOP/s (1.35 on 16x16x32 MFMAs), the clock then at 1.6 of 2.4
// GHz; this kernel 1.37 at K = 12288, M = 4096, N = 4096 (300 us, clock 1.67
// GHz, matrix pipe 0.77 busy).  Without the copies it takes 266 us, without the
// barriers 299.
//
// The epilogue passes the accumulators through LDS, 32 rows at a time, so that
// bias, residual and outputs move as whole rows of 16 bytes a lane.
#include "tile_image.hpp"

namespace q4 {

constexpr int kRing = 4;

template <int NT, int MT, int EPI>
__global__ __launch_bounds__(256, 1) void k_tile_gemm(const TileArgs a) {
    static_assert(EPI != EPI_GATED || NT % 2 == 0, "gate and up panels come in pairs");
    constexpr int kPanels = 2 * (NT + MT);                  // of a slot: weights first
    constexpr int kSlot = kPanels * 2 * kUnit;              // [panel][slice][unit]
    constexpr int kCopies = NT + MT;                        // of a wave and step
    constexpr int kRowF = NT * 32 + 4;                      // a row of the epilogue's LDS tile, floats
    constexpr int kLds = kRing * kSlot > 4 * 32 * kRowF * 4 ? kRing * kSlot : 4 * 32 * kRowF * 4;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = wave & 1, wm = wave >> 1;

    // ---- the tile ------------------------------------------------------------
    // Workgroup b runs on XCD b mod 8: consecutive tiles v go to one XCD, and
    // run down the rows first, in groups of eight row tiles, so that an XCD's
    // workgroups share a few row and column panels in its L2.
    const int64_t tiles_n = (a.w_panels + 2 * NT - 1) / (2 * NT), tiles_m = (a.x_panels + 2 * MT - 1) / (2 * MT);
    const int64_t G = gridDim.x, xcd = blockIdx.x % 8, each = G / 8, rest = G % 8;
    int64_t v = xcd * each + (xcd < rest ? xcd : rest) + blockIdx.x / 8;
    const int part = (int)(v / (tiles_n * tiles_m));
    v -= part * (tiles_n * tiles_m);
    const int64_t group = v / (8 * tiles_n), left_m = tiles_m - group * 8;
    const int64_t high = left_m < 8 ? left_m : 8;
    v -= group * 8 * tiles_n;
    const int64_t pn0 = v / high * (2 * NT), pm0 = (group * 8 + v % high) * (2 * MT);

    // ---- copies: unit t of this wave is slice (wave & 1) of panel (wave >> 1) + 2 t ----
    const int64_t steps_all = a.slices / 2;
    const int64_t s0 = steps_all * part / a.parts;
    const int S = (int)(steps_all * (part + 1) / a.parts - s0);
    const uint8_t* src[kCopies];
#pragma unroll
    for (int t = 0; t < kCopies; t++) {
        const int p = (wave >> 1) + 2 * t;
        const bool w = p < 2 * NT;
        // a panel past the image repeats its last one: those columns or rows are never stored
        const int64_t last = (w ? a.w_panels : a.x_panels) - 1, pp = w ? pn0 + p : pm0 + p - 2 * NT;
        src[t] = (w ? a.wimg : a.ximg) + ((pp < last ? pp : last) * a.slices + 2 * s0 + (wave & 1)) * kUnit;
    }
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds) +
                          (uint32_t)((wave >> 1) * 2 + (wave & 1)) * kUnit;
    // copy t of the next step to request, into slot; after the last step the
    // last one is copied again (and never read), so that a wait counts alike
    uint32_t voff = (uint32_t)lane * 16;                     // in the panel: below 2^32 for sums of at most 2^26 terms
    int ahead = 0;                                           // step it stands at
    auto copy = [&](int t, int slot) __attribute__((always_inline)) {
        copy_unit(src[t], voff, lds0 + (uint32_t)slot * kSlot + (uint32_t)t * 4 * kUnit);
    };
    auto advance = [&]() __attribute__((always_inline)) {
        ahead++;
        voff += ahead < S ? 2 * kUnit : 0;
    };

    floatx16_t acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; i++)
#pragma unroll
        for (int j = 0; j < MT; j++)
#pragma unroll
            for (int e = 0; e < 16; e++) acc[i][j][e] = 0.0f;

    // fragments of a slice: weights 0 .. NT-1, then x
    u32x4_t fa[NT + MT], fb[NT + MT];
    auto read = [&](int f, int slot, int slice, u32x4_t (&fr)[NT + MT]) __attribute__((always_inline)) {
        const int panel = f < NT ? wn * NT + f : 2 * NT + wm * MT + (f - NT);
        fr[f] = *reinterpret_cast<const u32x4_t*>(lds + slot * kSlot + (panel * 2 + slice) * kUnit + lane * 16);
    };
    auto mfma = [&](int q, const u32x4_t (&fr)[NT + MT]) __attribute__((always_inline)) {
        const int i = q / MT, j = q % MT;
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, fr[i]),
                                                           __builtin_bit_cast(half8_t, fr[NT + j]), acc[i][j], 0, 0, 0);
    };

    // ---- the schedule of a step: T MFMAs, the reads and copies between them ----
    // MFMA q of a slice uses weights fragment q / MT and x fragment q % MT, so a
    // slice's fragments are needed in the order W0, X0 .. , W1, W2 ..
    constexpr int kM = NT * MT, T = 2 * kM;
    constexpr int kFrags = NT + MT;
    constexpr int B = 3 * T / 4;                            // the barrier stands before MFMA B
    constexpr int kEarly = MT + 2;                          // W0, X*, W1 of slice 0: read after the step before's barrier
    constexpr int kLate = 2 * kFrags - kEarly;              // the rest, and slice 1: read before this step's barrier
    constexpr int kLead = T / 4 < 6 ? T / 4 : 6;            // MFMAs between the last of them and the barrier
    constexpr int kUnwrapped = (T - B - 1 + (T / kCopies) - 1) / (T / kCopies);   // copies from the barrier to the step's end
    static_assert(T >= kCopies, "at most one copy after an MFMA");
    auto frag_at = [](int r) constexpr { return r == 0 ? 0 : r <= MT ? NT + r - 1 : r - MT; };

    if (S > 0) {
        for (int p = 0; p < kRing - 1; p++) {
#pragma unroll
            for (int t = 0; t < kCopies; t++) copy(t, p);
            advance();
        }
#pragma unroll
        for (int t = 0; t < kUnwrapped; t++) copy(t, kRing - 1);
        step_barrier<2 * kCopies + kUnwrapped>();
#pragma unroll
        for (int r = 0; r < kEarly; r++) read(frag_at(r), 0, 0, fa);
    }
    for (int i = 0; i < S; i++) {
        const int slot = i & (kRing - 1), next = (i + 1) & (kRing - 1), before = (i + 3) & (kRing - 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < T; q++) {
            if (q == B) {
                advance();
                step_barrier<2 * kCopies>();
                __builtin_amdgcn_sched_barrier(0);
            }
            if (q < kM) mfma(q, fa);
            else mfma(q - kM, fb);
#pragma unroll
            for (int r = 0; r < kLate; r++)
                if (r * (B - kLead) / kLate == q) {
                    if (r < kFrags - kEarly) read(frag_at(r + kEarly), slot, 0, fa);
                    else read(frag_at(r - (kFrags - kEarly)), slot, 1, fb);
                }
#pragma unroll
            for (int r = 0; r < kEarly; r++)
                if (B + r * (T - B) / kEarly == q) read(frag_at(r), next, 0, fa);
#pragma unroll
            for (int t = 0; t < kCopies; t++) {
                const int at = B + 1 + t * (T / kCopies);
                if (at < T && at == q) copy(t, slot);
                if (at >= T && at - T == q) copy(t, before);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // ---- epilogue ----------------------------------------------------------------
    // every copy has landed and every wave has read its last fragments
    step_barrier<0>();
    float* tile = reinterpret_cast<float*>(lds) + wave * 32 * kRowF;
    constexpr int kCols = EPI == EPI_GATED ? NT * 16 : NT * 32;      // output columns of the wave
    constexpr int kChunks = kCols / 8;
    const int64_t N = a.epi.N, M = a.epi.M;
    const int64_t n0 = EPI == EPI_GATED ? (pn0 + wn * NT) * 16 : (pn0 + wn * NT) * 32;
    const bool vec = N % 8 == 0;
#pragma unroll
    for (int j = 0; j < MT; j++) {
        const int64_t m0 = (pm0 + wm * MT + j) * 32;
        const int64_t mine = m0 + (lane & 31);
        // (parts of a sum are joined first: alone they may leave the range)
        const float back = EPI == EPI_PARTIAL ? 1.0f : mine < M ? ldexpf(1.0f, -(int)a.xexp[mine]) : 0.0f;
        // lane: row lane & 31 of the panel, columns 8 (e / 4) + 4 (lane >> 5) + e % 4
#pragma unroll
        for (int i = 0; i < NT; i++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                floatx4_t t;
#pragma unroll
                for (int e = 0; e < 4; e++) t[e] = acc[i][j][4 * q + e] * back;
                *reinterpret_cast<floatx4_t*>(tile + (lane & 31) * kRowF + i * 32 + 8 * q + 4 * (lane >> 5)) = t;
            }
        for (int c0 = 0; c0 < 32 * kChunks; c0 += 64) {
            const int c = c0 + lane;
            const int row = c / kChunks, col = c % kChunks * 8;
            const int64_t m = m0 + row, n = n0 + col;
            float z[8], z2[8];
            auto fetch = [&](int at, float (&f)[8]) __attribute__((always_inline)) {
                const floatx4_t* p = reinterpret_cast<const floatx4_t*>(tile + row * kRowF + at);
                const floatx4_t lo = p[0], hi = p[1];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    f[e] = lo[e];
                    f[4 + e] = hi[e];
                }
            };
            if constexpr (EPI == EPI_GATED) {
                fetch(col / 32 * 64 + col % 32, z);
                fetch(col / 32 * 64 + 32 + col % 32, z2);
            } else {
                fetch(col, z);
            }
            if (m >= M) continue;
            if constexpr (EPI == EPI_PARTIAL) {
                const int64_t np = a.w_panels * 32;
                if (n < np) {
                    floatx4_t* p = reinterpret_cast<floatx4_t*>(a.part + ((int64_t)part * M + m) * np + n);
                    p[0] = floatx4_t{z[0], z[1], z[2], z[3]};
                    p[1] = floatx4_t{z[4], z[5], z[6], z[7]};
                }
            } else {
                if (n >= N) continue;
                if (vec) epilogue8<EPI, true>(a.epi, m, n, z, z2);
                else epilogue8<EPI, false>(a.epi, m, n, z, z2);
            }
        }
    }
}

// The parts of a split sum joined in order and scaled, then the epilogue: one
// thread for eight columns of a row.
template <int EPI>
__global__ __launch_bounds__(256) void k_tile_join(const TileArgs a) {
    const int64_t chunks = (a.epi.N + 7) / 8;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= a.epi.M * chunks) return;
    const int64_t m = id / chunks, n = id % chunks * 8, np = a.w_panels * 32;
    const int64_t at = EPI == EPI_GATED ? n / 32 * 64 + n % 32 : n;
    float z[8] = {0, 0, 0, 0, 0, 0, 0, 0}, z2[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int p = 0; p < a.parts; p++) {
        const float* row = a.part + ((int64_t)p * a.epi.M + m) * np + at;
        auto add = [&](const float* q, float (&f)[8]) __attribute__((always_inline)) {
            const floatx4_t lo = reinterpret_cast<const floatx4_t*>(q)[0], hi = reinterpret_cast<const floatx4_t*>(q)[1];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                f[e] += lo[e];
                f[4 + e] += hi[e];
            }
        };
        add(row, z);
        if constexpr (EPI == EPI_GATED) add(row + 32, z2);
    }
    const float back = a.xexp ? ldexpf(1.0f, -(int)a.xexp[m]) : a.unit;
#pragma unroll
    for (int e = 0; e < 8; e++) {
        z[e] *= back;
        z2[e] *= back;
    }
    if (a.epi.N % 8 == 0) epilogue8<EPI, true>(a.epi, m, n, z, z2);
    else epilogue8<EPI, false>(a.epi, m, n, z, z2);
}

// ---- host ------------------------------------------------------------------------

// Cost of a plan in cycles: rounds of workgroups over the CUs, each a start
// and, per step, the larger of the MFMAs' time and LDS's.
static double plan_cost(int nt, int mt, int parts, int64_t w_panels, int64_t x_panels, int64_t steps, int cus) {
    const int64_t tiles = ((w_panels + 2 * nt - 1) / (2 * nt)) * ((x_panels + 2 * mt - 1) / (2 * mt));
    const int64_t rounds = (tiles * parts + cus - 1) / cus;
    const double mfma = 64.0 * nt * mt, lds = 112.0 * (nt + mt);
    const double step = (mfma > lds ? mfma : lds) + 60.0;
    const double one = 5000.0 + step * (double)((steps + parts - 1) / parts);
    // the parts' sums travel to memory and back, and a join is a launch more
    const double join = parts > 1 ? 6000.0 + 8.0 * parts * (double)(x_panels * w_panels) * 1024.0 / 2000.0 : 0.0;
    return rounds * one + join;
}

TilePlan plan_tiles(int nmat, int64_t M, int64_t N, int64_t K) {
    const int64_t w_panels = (N + 31) / 32 * nmat, x_panels = (M + 31) / 32, steps = image_slices(K) / 2;
    const int cus = current_cu_count();
    TilePlan best{4, 4, 1};
    double least = -1.0;
    constexpr int kShapes[][2] = {{4, 4}, {4, 2}, {2, 4}, {2, 2}};
    for (const auto& sh : kShapes)
        for (int parts = 1; parts <= 16; parts *= 2) {
            if (parts > 1 && steps / parts < 8) break;
            const double c = plan_cost(sh[0], sh[1], parts, w_panels, x_panels, steps, cus);
            if (least < 0.0 || c < least) {
                least = c;
                best = TilePlan{sh[0], sh[1], parts};
            }
        }
    return best;
}

int64_t partial_bytes(const TilePlan& p, int64_t M, int64_t w_panels) {
    return p.parts > 1 ? (int64_t)p.parts * M * w_panels * 32 * 4 : 0;
}

template <int NT, int MT>
static void launch_shape(int epi, const TileArgs& a, unsigned grid, hipStream_t s) {
    if (epi == EPI_PARTIAL) hipLaunchKernelGGL((k_tile_gemm<NT, MT, EPI_PARTIAL>), dim3(grid), dim3(256), 0, s, a);
    else if (epi == EPI_GATED) hipLaunchKernelGGL((k_tile_gemm<NT, MT, EPI_GATED>), dim3(grid), dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_tile_gemm<NT, MT, EPI_LINEAR>), dim3(grid), dim3(256), 0, s, a);
}

hipError_t launch_tile_join(int nmat, const TileArgs& a, hipStream_t s) {
    const int64_t threads = a.epi.M * ((a.epi.N + 7) / 8);
    if (!launchable((threads + 255) / 256, 256)) return hipErrorInvalidValue;
    const dim3 grid((unsigned)((threads + 255) / 256));
    if (nmat == 2) hipLaunchKernelGGL((k_tile_join<EPI_GATED>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_tile_join<EPI_LINEAR>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_tile_gemm(const TilePlan& p, int nmat, const TileArgs& args, hipStream_t s) {
    TileArgs a = args;
    a.parts = p.parts;
    const int last = nmat == 2 ? EPI_GATED : EPI_LINEAR;
    const int epi = p.parts > 1 ? EPI_PARTIAL : last;
    const int64_t tiles =
        ((a.w_panels + 2 * p.nt - 1) / (2 * p.nt)) * ((a.x_panels + 2 * p.mt - 1) / (2 * p.mt)) * p.parts;
    if (!launchable(tiles, 256)) return hipErrorInvalidValue;
    if (p.nt == 4 && p.mt == 4) launch_shape<4, 4>(epi, a, (unsigned)tiles, s);
    else if (p.nt == 4) launch_shape<4, 2>(epi, a, (unsigned)tiles, s);
    else if (p.mt == 4) launch_shape<2, 4>(epi, a, (unsigned)tiles, s);
    else launch_shape<2, 2>(epi, a, (unsigned)tiles, s);
    if (p.parts > 1) return launch_tile_join(nmat, a, s);
    return hipGetLastError();
}

}  // namespace q4
