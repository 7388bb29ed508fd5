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
    int64_t N, K;
    int64_t w_panels;          // of W: gate and up in turn
    int64_t groups;            // of 256 k
    uint8_t* scales;           // images of the scales, or null
    const uint8_t* w_scales[2];          // a row's eight bytes of group t: + row * scale_row + t * scale_group
    const uint8_t* x_scales;
    uint32_t scale_row;
    int64_t scale_group;
    float* part;
    EpilogueArgs epi;
};

int64_t mx_tile_workspace_bytes(int x_type, int nmat, int64_t M, int64_t N, int64_t K);
hipError_t launch_mx_tile(const MxLinearArgs& p, const EpilogueArgs& epi, void* workspace, hipStream_t s);

}  // namespace q4
