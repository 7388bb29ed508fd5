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
// Above 64 rows 64 at a time in one launch, by the turns (row tiles and groups) of the busiest CU's waves.
// bfloat16 x, whose other route makes images: to 128 rows, and where there are four turns at most
// (128 x 12288 x 4096 30.1 us here, 50.3 there; gated 65.0, 91.2; 256 x 4096 x 4096, four turns, 22.9, 33.4;
// 256 x 6176 x 1280, four, 23.4, 27.4; 512 x 4096 x 4096, eight, 42.4, 40.9; 512 x 6176 x 1280, eight,
// 51.6, 28.8).  binary16 x takes twice the products: never (128 x 2048 x 8192 36.8, 31.7).
// MX x: long sums of at most two turns (128 x 4096 x 4096 9.5, as tiles 15.8; 128 x 2048 x 8192 12.8, 17.0;
// but 128 x 6176 x 1280 11.8, 7.6, and gated 128 x 4096 x 4096 20.0, 19.4).
inline bool few_takes(int x, int nmat, int64_t M, int64_t N, int64_t K, int64_t cus) {
    const bool mx = x == FEW_MX;
    if (M <= 64 && (nmat == 1 || M <= 32 || !mx)) return true;
    if (M > 64 && !(mx ? nmat == 1 && K >= 4096 : x == FEW_BF16)) return false;
    const MxFewPlan p = plan_few(nmat, M, N, K, cus);
    const int64_t workgroups = few_columns(p, M, N) * few_chunks(M);
    if (M <= 64) return workgroups <= cus;
    const int64_t groups = (K / 32 + 15) / 16, turns = (workgroups + cus - 1) / cus * p.r * ((groups + p.kw - 1) / p.kw);
    return mx ? turns <= 2 : M <= 128 || turns <= 4;
}

}  // namespace q4
