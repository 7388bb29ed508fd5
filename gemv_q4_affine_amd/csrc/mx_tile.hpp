// mx_tile.hpp -- the records and launchers of the tile product on MX x
// (mx_tile.hip).
#pragma once

#include "mx_common.hpp"
#include "tile_image.hpp"

namespace q4 {

struct MxTileArgs {
    int nmat, parts;
    const uint8_t* wq[2];
    const uint8_t* ws[2];
    const uint8_t* xq;
    const uint8_t* xs;
    uint32_t* w_scales;        // images (k_mx_scales)
    uint32_t* x_scales;
    int64_t N, K;
    int64_t w_panels, w_pad, x_pad;      // panels of W (gate and up in turn), and of the scale images
    int64_t groups;            // of 256 k
    float* part;
    EpilogueArgs epi;
};

int64_t mx_tile_workspace_bytes(int x_type, int nmat, int64_t M, int64_t N, int64_t K);
hipError_t launch_mx_tile(const MxLinearArgs& p, const EpilogueArgs& epi, void* workspace, hipStream_t s);

}  // namespace q4
