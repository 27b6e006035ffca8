// product_host.cuh -- host side of the tensor-core kernels of the products.
#pragma once

#include <algorithm>
#include <atomic>

#include "launch.h"
#include "product.h"
#include "product_tile.cuh"

namespace fp4q {

// Tensor map of a [rows][row_bytes] byte matrix, tiles of `box_rows` rows x 128
// bytes under the 128-byte swizzle; reads past the edges give zeros.
cudaError_t byte_tile_map(CUtensorMap* map, const void* base, int64_t rows, int64_t row_bytes, int box_rows);

// The kernel arguments that do not depend on the tile shape.
TileArgs tile_args(const Product& p, int step_cols, int scale_tile_cols);

// resident_blocks_per_sm without its lock once it is known for the device.
struct Residency {
    std::atomic<int> cached[64];
};
int product_blocks_per_sm(Residency& r, const void* kernel, int threads, size_t smem);

struct TileShape {
    int tokens;      // rows of x per tile, a multiple of 16 (of 32 above 128), at most 192
    int split;       // thread blocks that share a tile's K
};
// Sums longer than one accumulator may take: its steps, the tokens of a tile that
// has room for them, and whether blocks that share a tile have.
struct Runs {
    int steps, tokens;
    bool split;
};
// pair: thread blocks that share a tile of more than 128 tokens.
TileShape tile_shape(const Product& p, int k_steps, int pair, const Runs& runs);

// One launch over all tiles: as many clusters of thread blocks (`pair` or the
// shape's split) as are resident at once, or as there are tiles, if fewer, each
// striding over the tiles.  A grouped call knows only how many tiles there can
// be at most.
template <typename Kernel>
cudaError_t launch_tiles(Kernel kernel, const CUtensorMap& w_map, const CUtensorMap& x_map, const Product& p,
                         TileArgs& a, const TileShape& shape, int pair, int per_sm, int threads, size_t smem,
                         cudaStream_t s)
{
    a.tokens = shape.tokens;
    a.split = shape.split;
    a.n_tiles = (int)((p.n + 128 * pair - 1) / (128 * pair));
    int64_t token_tiles = (p.m + a.tokens - 1) / a.tokens;
    if (p.offsets) token_tiles = std::min<int64_t>(p.m, p.m / a.tokens + p.groups);
    const int blocks = pair * shape.split;
    const int64_t slots = std::max<int64_t>(1, (int64_t)sm_count() * per_sm / blocks);
    const int64_t clusters = std::min<int64_t>(token_tiles * a.n_tiles, slots);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(clusters * blocks));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, w_map, x_map, a);
}

}  // namespace fp4q
