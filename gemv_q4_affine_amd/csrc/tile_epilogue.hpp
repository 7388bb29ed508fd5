// tile_epilogue.hpp -- what the tile products (tile_gemm.hip, mx_tile.hip) do with
// their accumulators: they pass through LDS, 32 rows at a time, so that bias,
// residual and outputs move as whole rows of 16 bytes a lane.
#pragma once

#include "tile_image.hpp"

namespace q4 {

// A row of a wave's LDS tile (32 of them), in floats.
template <int NT>
constexpr int tile_row_floats() { return NT * 32 + 4; }

// The wave's NT x MT accumulator tiles of 32 x 32 (columns n0 .., at EPI_GATED
// panels of gate and up in turn; rows first ..), times 2^back(m) -- not the parts
// of a split sum, which are joined first: alone they may leave the range.
template <int NT, int MT, int EPI, class Back>
__device__ __forceinline__ void tile_epilogue(const floatx16_t (&acc)[NT][MT], float* tile, const EpilogueArgs& epi,
                                              float* parts, int part, int64_t w_panels, int64_t n0, int64_t first,
                                              Back back_of) {
    constexpr int kRowF = tile_row_floats<NT>();
    constexpr int kCols = EPI == EPI_GATED ? NT * 16 : NT * 32;      // output columns of the wave
    constexpr int kChunks = kCols / 8;
    const int lane = threadIdx.x & 63;
    const int64_t N = epi.N, M = epi.M;
    const bool vec = N % 8 == 0;
    // Columns with powers of two of their own: a lane's are the same in every turn (kChunks
    // divides 64) and found once.
    const bool scaled = EPI != EPI_PARTIAL && epi.w_scale[0];
    constexpr int kFactors = EPI == EPI_GATED ? 2 : 1;
    u32x2_t scale[kFactors] = {};
    float factor[kFactors][8];
#pragma unroll
    for (int t = 0; t < kFactors; t++) {
        const int64_t n = n0 + lane % kChunks * 8;
        if (scaled && n < N) scale[t] = *reinterpret_cast<const u32x2_t*>(epi.w_scale[t] + n);
#pragma unroll
        for (int e = 0; e < 8; e++) factor[t][e] = 1.0f;
        unscale8(scale[t], 0, factor[t]);
    }
#pragma unroll
    for (int j = 0; j < MT; j++) {
        const int64_t m0 = first + j * 32;
        const int64_t mine = m0 + (lane & 31);
        const int by = EPI != EPI_PARTIAL && mine < M ? back_of(mine) : 0;
        // (sums lie between 2^-48 and 2^57: beyond 2^+-64 a row's power of two and a column's go
        // together, as halfway the value may leave the range; the row's waits behind the row)
        const bool far = scaled && __any(by < -64 || by > 64);
        const float back = far ? 1.0f : ldexpf(1.0f, by);
        if (far) tile[(lane & 31) * kRowF + NT * 32] = __int_as_float(by);
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
                const int64_t np = w_panels * 32;
                if (n < np) {
                    floatx4_t* p = reinterpret_cast<floatx4_t*>(parts + ((int64_t)part * M + m) * np + n);
                    p[0] = floatx4_t{z[0], z[1], z[2], z[3]};
                    p[1] = floatx4_t{z[4], z[5], z[6], z[7]};
                }
            } else {
                if (n >= N) continue;
                if (far) {
                    const int e = __float_as_int(tile[row * kRowF + NT * 32]);
                    unscale8(scale[0], e, z);
                    if constexpr (EPI == EPI_GATED) unscale8(scale[1], e, z2);
                } else if (scaled) {
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        z[e] *= factor[0][e];
                        if constexpr (EPI == EPI_GATED) z2[e] *= factor[1][e];
                    }
                }
                if (vec) epilogue8<EPI, true>(epi, m, n, z, z2);
                else epilogue8<EPI, false>(epi, m, n, z, z2);
            }
        }
    }
}

// The same with every load ahead of the first store: loads and stores return in one
// order, so that a load among the stores would wait for those before it.  A lane's
// eight columns are the same in all of its rows: its bias is read once; the residual
// of the whole tile waits in registers and passes through LDS beside the sums.
// VEC: rows are multiples of eight values (else the residual is read among the
// stores, value by value).  The type is known when compiling and four turns go
// through each step at once: with one wave a SIMD nothing else hides a latency or a
// branch.  (A 256 x 256 tile: 24000 cycles with the type asked for at every pair of
// values, 19000 with it known, 13000 so.)
template <int NT, int MT, int EPI>
struct RowEpilogue {
    static_assert(EPI != EPI_GATED, "gate_epilogue");
    static constexpr int kRowF = tile_row_floats<NT>();
    static constexpr int kChunks = NT * 4;                                // of eight columns, of a row
    static constexpr int kRows = 64 / kChunks, kTurns = 32 / kRows;       // rows of a turn
    static constexpr int kResB = EPI == EPI_LINEAR ? 32 * kChunks * 16 : 0;      // bytes of a row of tiles' residual
    static constexpr int kWaveB = 32 * kRowF * 4 + kResB;                 // LDS of a wave
};
template <int NT, int MT, int EPI, bool VEC, int DT>
__device__ __forceinline__ void row_epilogue(const floatx16_t (&acc)[NT][MT], uint8_t* lds, const EpilogueArgs& epi, float* parts,
                                             int part, int64_t w_panels, int64_t n0, int64_t first) {
    using E = RowEpilogue<NT, MT, EPI>;
    constexpr int U = E::kTurns < 4 ? E::kTurns : 4;         // turns at a time: one wave a SIMD hides no latency otherwise
    constexpr int kRowF = E::kRowF, kChunks = E::kChunks, kRows = E::kRows, kTurns = E::kTurns;
    float* tile = reinterpret_cast<float*>(lds);
    u32x4_t* kept = reinterpret_cast<u32x4_t*>(lds + 32 * kRowF * 4);
    const int lane = threadIdx.x & 63, row0 = lane / kChunks, col = lane % kChunks * 8;
    const int64_t N = epi.N, M = epi.M, n = n0 + col;
    const int left = (int)(N - n < 8 ? N - n : 8);
    auto load = [&](const void* p, int64_t at) __attribute__((always_inline)) {
        return left > 0 ? load8_raw<VEC>(p, at, left) : u32x4_t{0u, 0u, 0u, 0u};
    };
    const bool adds = EPI == EPI_LINEAR && epi.residual;
    constexpr bool kAhead = VEC && EPI == EPI_LINEAR;
    u32x4_t bias = {}, more[kAhead ? MT * kTurns : 1];
    if constexpr (EPI != EPI_PARTIAL) {
        if (epi.bias[0]) bias = load(epi.bias[0], n);
    }
    if constexpr (kAhead) {
        if (adds) {
#pragma unroll
            for (int t = 0; t < MT * kTurns; t++) {
                const int64_t m = first + t * kRows + row0;
                more[t] = m < M ? load(epi.residual, m * N + n) : u32x4_t{0u, 0u, 0u, 0u};
            }
        }
    }
    asm volatile("" : "+v"(bias));                           // here they are waited for
    // The accumulators are indexed by constants (a loop that is not unrolled would put
    // them into memory), but what follows is one body for all turns.
    auto put = [&](auto tile_j) __attribute__((always_inline)) {
        constexpr int j = decltype(tile_j)::value;
        // lane: row lane & 31 of the panel, columns 8 (e / 4) + 4 (lane >> 5) + e % 4
        if constexpr (j < MT) {
#pragma unroll
            for (int i = 0; i < NT; i++)
#pragma unroll
                for (int q = 0; q < 4; q++)
                    *reinterpret_cast<floatx4_t*>(tile + (lane & 31) * kRowF + i * 32 + 8 * q + 4 * (lane >> 5)) =
                        floatx4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            if constexpr (kAhead) {
                if (adds) {
#pragma unroll
                    for (int t = 0; t < kTurns; t++) kept[t * 64 + lane] = more[j * kTurns + t];
                }
            }
        }
    };
#pragma unroll 1
    for (int j = 0; j < MT; j++) {
        if (j == 0) put(std::integral_constant<int, 0>{});
        else if (j == 1) put(std::integral_constant<int, 1>{});
        else if (j == 2) put(std::integral_constant<int, 2>{});
        else put(std::integral_constant<int, 3>{});
        const int64_t m0 = first + j * 32 + row0;
        const float* row = tile + row0 * kRowF;
#pragma unroll 1
        for (int t = 0; t < kTurns; t += U, row += U * kRows * kRowF) {
            auto fetch = [&](int u, int at, float* f) __attribute__((always_inline)) {
                const floatx4_t* p = reinterpret_cast<const floatx4_t*>(row + u * kRows * kRowF + at);
                const floatx4_t lo = p[0], hi = p[1];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    f[e] = lo[e];
                    f[4 + e] = hi[e];
                }
            };
            float z[U * 8], none[U * 8];
            u32x4_t rest[kAhead ? U : 1];
            bool live[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
                fetch(u, col, z + u * 8);
                if constexpr (kAhead)
                    if (adds) rest[u] = kept[(t + u) * 64 + lane];
                live[u] = m0 + (t + u) * kRows < M && left > 0;
            }
            const int64_t at = (m0 + t * kRows) * N + n;
            if constexpr (EPI == EPI_PARTIAL) {
                const int64_t np = w_panels * 32;
#pragma unroll
                for (int u = 0; u < U; u++) {
                    const int64_t m = m0 + (t + u) * kRows;
                    if (m < M && n < np) {
                        floatx4_t* p = reinterpret_cast<floatx4_t*>(parts + ((int64_t)part * M + m) * np + n);
                        p[0] = floatx4_t{z[u * 8], z[u * 8 + 1], z[u * 8 + 2], z[u * 8 + 3]};
                        p[1] = floatx4_t{z[u * 8 + 4], z[u * 8 + 5], z[u * 8 + 6], z[u * 8 + 7]};
                    }
                }
                continue;
            }
            auto add = [&](const u32x4_t& v, float* f) __attribute__((always_inline)) {
                float s[8];
                unpack8(DT, v, s);
#pragma unroll
                for (int e = 0; e < 8; e++) f[e] += s[e];
            };
            auto put_out = [&](void* p, const float* f) __attribute__((always_inline)) {
#pragma unroll
                for (int u = 0; u < U; u++) {
                    u32x4_t r;
#pragma unroll
                    for (int e = 0; e < 4; e++) r[e] = pack2(DT, f[u * 8 + 2 * e], f[u * 8 + 2 * e + 1]);
                    if (live[u]) store8<VEC>(p, at + u * kRows * N, left, r);
                }
            };
            if (epi.bias[0]) {
#pragma unroll
                for (int u = 0; u < U; u++) add(bias, z + u * 8);
            }
            if (epi.pre[0]) put_out(epi.pre[0], z);
            if (epi.act != ACT_NONE) activate_all<false>(epi.act, z, z, none);
            if (adds) {
#pragma unroll
                for (int u = 0; u < U; u++) {
                    if constexpr (kAhead) add(rest[u], z + u * 8);
                    else if (live[u]) add(load(epi.residual, at + u * kRows * N), z + u * 8);
                }
            }
            put_out(epi.y, z);
        }
    }
}

// EPI_GATED (tiles of gate and up in turn) without LDS: lane swaps give a lane eight
// neighbouring columns of its row, 16 bytes of a tensor, two lanes 32 -- at half the
// columns faster than through LDS (11000 cycles a 256 x 256 tile against 17000; 17600
// against 19500 where both projections are stored too), at EPI_LINEAR slower (17000
// against 13000).
template <int NT, int MT, bool VEC, int DT>
__device__ __forceinline__ void gate_epilogue(const floatx16_t (&acc)[NT][MT], const EpilogueArgs& epi, int64_t n0, int64_t first) {
    constexpr int kPieces = NT;                              // of eight columns, of a lane's row
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int64_t N = epi.N, M = epi.M, n = n0 + 8 * h, m0 = first + (lane & 31);
    int left[kPieces];                                       // columns of a piece inside the output
#pragma unroll
    for (int u = 0; u < kPieces; u++) {
        const int64_t l = N - n - 16 * u;
        left[u] = l < 8 ? (int)(l < 0 ? 0 : l) : 8;
    }
    u32x4_t bias[2][kPieces];
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
        for (int u = 0; u < kPieces; u++) {
            bias[t][u] = u32x4_t{0u, 0u, 0u, 0u};
            if (epi.bias[t] && left[u] > 0) bias[t][u] = load8_raw<VEC>(epi.bias[t], n + 16 * u, left[u]);
        }
    // eight columns from 16 q + 8 h of a tile
    auto columns = [&](const floatx16_t& t, int q, float* z) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(t[8 * q + e]), __float_as_uint(t[8 * q + 4 + e]), false, false);
            z[e] = __uint_as_float(s[0]);
            z[4 + e] = __uint_as_float(s[1]);
        }
    };
    auto row_of_tiles = [&](auto tile) __attribute__((always_inline)) {
        constexpr int j = decltype(tile)::value;
        const int64_t m = m0 + j * 32;
        if (m >= M) return;
        const int64_t at = m * N + n;
        float z[8 * kPieces], z2[8 * kPieces], none[8 * kPieces];
#pragma unroll
        for (int u = 0; u < kPieces; u++) {
            columns(acc[u / 2 * 2][j], u & 1, z + 8 * u);
            columns(acc[u / 2 * 2 + 1][j], u & 1, z2 + 8 * u);
        }
        auto add = [&](const u32x4_t (&b)[kPieces], float* f) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < kPieces; u++) {
                float t[8];
                unpack8(DT, b[u], t);
#pragma unroll
                for (int e = 0; e < 8; e++) f[8 * u + e] += t[e];
            }
        };
        auto put = [&](void* p, const float* f) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < kPieces; u++) {
                u32x4_t r;
#pragma unroll
                for (int e = 0; e < 4; e++) r[e] = pack2(DT, f[8 * u + 2 * e], f[8 * u + 2 * e + 1]);
                if (left[u] > 0) store8<VEC>(p, at + 16 * u, left[u], r);
            }
        };
        if (epi.bias[0]) add(bias[0], z);
        if (epi.bias[1]) add(bias[1], z2);
        if (epi.pre[0]) put(epi.pre[0], z);
        if (epi.pre[1]) put(epi.pre[1], z2);
        if (epi.act != ACT_NONE) activate_all<false>(epi.act, z, z, none);
#pragma unroll
        for (int e = 0; e < 8 * kPieces; e++) z[e] *= z2[e];
        put(epi.y, z);
    };
    // (accumulators are indexed by constants only: a loop that is not unrolled would put them into memory)
    row_of_tiles(std::integral_constant<int, 0>{});
    row_of_tiles(std::integral_constant<int, 1>{});
    if constexpr (MT == 4) {
        row_of_tiles(std::integral_constant<int, 2>{});
        row_of_tiles(std::integral_constant<int, 3>{});
    }
}

}  // namespace q4
