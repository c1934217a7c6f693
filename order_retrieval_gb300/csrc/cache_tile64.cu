// cache_tile64.cu -- the tile kernel (cache_tile.cuh) for values up to 64 wide.
#include "cache_tile.cuh"

namespace zeta {

cudaError_t launch_cache_tile64(const Prob &p, const TileArgs &g, int wm, cudaStream_t st) {
    if (wm == 1) return dispatch_tile<64, 1, 8>(p, g, st);
    if (wm == 2) return dispatch_tile<64, 2, 8>(p, g, st);
    return dispatch_tile<64, 4, 8>(p, g, st);
}

}  // namespace zeta
