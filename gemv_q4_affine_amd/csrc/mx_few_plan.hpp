// mx_few_plan.hpp -- which products the few-row kernel (mx_few.hip) takes, and how it is
// launched: arithmetic on sizes and the number of CUs, nothing of HIP.
#pragma once

#include <cstdint>

#include "launch_limits.hpp"

namespace q4 {

// Waves of a workgroup along the sum and along the rows of W, row tiles of a wave.
struct MxFewPlan {
    int kw, rw, r;
};
enum : int { FEW_MX = 0, FEW_BF16 = 1, FEW_F16 = 2 };       // kinds of x

inline int few_threads(const MxFewPlan& p) { return 64 * p.kw * p.rw; }
inline int64_t few_chunks(int64_t M) { return (M + 63) / 64; }           // of 64 rows of x: the grid's y
inline int64_t few_columns(const MxFewPlan& p, int64_t M, int64_t N) {   // workgroups along the columns: its x
    const int64_t cols = (int64_t)p.rw * p.r * (M <= 4 ? 4 : 16);
    return (N + cols - 1) / cols;
}

// Waves along the sum first, as many as it has groups.  (16 x 12288 x 4096 with 8-bit x: 8.5 us
// with eight of them, 11.1 with four and two along the rows; up to four rows no difference.)
// Then one to three row tiles a wave, so that the busiest CU has the fewest of them to do, and
// of equals the most: a wave then has more loads in flight, and a fragment of x serves more
// products.  us with one, two and three tiles, 8-bit x but where said:
//   1 x 4096 x 4096   3.5  4.0  4.3     1 x 12288 x 4096         7.8   7.1   7.3
//   1 x 8192 x 4096   6.3  5.4  6.4     1 x 12288 x 4096 gated   12.4  12.7  11.5
//   16 x 12288 x 4096 9.9  9.9  8.6     1 x 12288 x 4096 binary16 17.6 15.6  12.9
//   16 x 32768 x 4096 19.9 16.4 17.0    4 x 32768 x 4096 bfloat16 25.7 17.6  19.9
inline MxFewPlan plan_few(int nmat, int64_t M, int64_t N, int64_t K, int64_t cus) {
    const int P = M <= 4 ? 4 : 1;
    const int64_t groups = (K / 32 + 16 * P - 1) / (16 * P), tiles = (N + 16 / P - 1) / (16 / P);
    MxFewPlan p{};
    p.kw = (int)(groups < 8 ? groups : 8);
    p.rw = 8 / p.kw;
    int64_t least = 0;
    for (int r = nmat == 2 && M > 32 ? 1 : 3; r >= 1; r--) { // (the registers hold no more than one there)
        const int64_t workgroups = (tiles + p.rw * r - 1) / (p.rw * r), of_cu = (workgroups * few_chunks(M) + cus - 1) / cus * r;
        // (one tile a wave may be too many threads: 2^25 columns in workgroups of 512, four columns each)
        if (least == 0 || (of_cu < least && launchable(workgroups, few_threads(p)))) {
            least = of_cu;
            p.r = r;
        }
    }
    return p;
}

// Up to 64 rows (64 x 12288 x 4096 with 8-bit x: 13.0 us here, 18.9 as tiles; 64 x 4096 x 12288:
// 18.4 and 18.9).  Gated and above 32 rows a wave has one row tile, and where that makes more
// than one round of workgroups the tiles are faster (64 x 4096 x 4096: 11.4 here, 17.1 as tiles;
// 64 x 12288 x 4096: 28.3 and 22.5).
//
// Above 64 rows 64 at a time in one launch, by the turns (row tiles and groups) of the busiest CU's
// waves and its rounds of workgroups; us here and by the other route.
// bfloat16 x, whose other route makes images: to 128 rows (128 x 12288 x 4096 26.7 and 48.9, x 32768 x
// 1280 41.9, 44.0, x 512 x 512 9.4, 13.1, x 300 x 16384 28.3, 31.5; gated x 12288 x 1280 31.7, 36.2), and
// above where there are at most four turns, gated three (256 x 4096 x 4096, four turns, 22.1, 33.2; 512 x
// 4096 x 4096, eight, 43.8, 40.2; gated 256 x 4096 x 2048, two, 21.9, 33.0; 256 x 8192 x 2048, four, 42.0,
// 38.6), but short sums only in two rounds (256 x 16384 x 544, two, 21.5, 23.4; 384 x 8192 x 544, three,
// 24.2, 17.8).
// binary16 x takes twice the products: not (128 x 1024 x 1024 19.9 and 16.4, x 2048 x 8192 36.1, 33.2, x
// 300 x 16384 68, 35; but x 4096 x 4096 22.6, 31.2).
// MX x, whose other route reads the planes too: linear, at most two turns of long sums (128 x 4096 x 4096 9.1
// and 14.5, x 2048 x 2304 9.1, 10.1, x 4096 x 2048, 7.3, 9.8, x 2048 x 1536 5.9, 8.3, x 1024 x 1024 7.0, 7.1,
// 256 x 4096 x 2560, four turns, 12.3, 11.1); where a row's last group is not whole only of longer ones (128 x
// 4096 x 4128 13.8, 17.6, x 2048 x 1792 9.6, 8.9).  Gated 128 x 4096 x 4096 20.0 here, 19.4 as tiles.
inline bool few_takes(int x, int nmat, int64_t M, int64_t N, int64_t K, int64_t cus) {
    const bool mx = x == FEW_MX;
    if (M <= 64 && (nmat == 1 || M <= 32 || !mx)) return true;
    if (M > 64 && !(mx ? nmat == 1 && K >= (K % 512 == 0 ? 1536 : 4096) : x == FEW_BF16)) return false;
    const MxFewPlan p = plan_few(nmat, M, N, K, cus);
    const int64_t workgroups = few_columns(p, M, N) * few_chunks(M);
    if (M <= 64) return workgroups <= cus;
    const int64_t groups = (K / 32 + 15) / 16, rounds = (workgroups + cus - 1) / cus;
    const int64_t turns = rounds * p.r * ((groups + p.kw - 1) / p.kw);
    if (mx) return turns <= 2;
    if (M <= 128) return true;
    return nmat == 2 ? turns <= 3 : turns <= 4 && (K >= 1024 || rounds <= 2);
}

}  // namespace q4
