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
// panels of gate and up in turn; rows first ..), scaled by back(m) -- not the parts
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
#pragma unroll
    for (int j = 0; j < MT; j++) {
        const int64_t m0 = first + j * 32;
        const int64_t mine = m0 + (lane & 31);
        const float back = EPI == EPI_PARTIAL ? 1.0f : mine < M ? back_of(mine) : 0.0f;
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
                if (vec) epilogue8<EPI, true>(epi, m, n, z, z2);
                else epilogue8<EPI, false>(epi, m, n, z, z2);
            }
        }
    }
}

}  // namespace q4
