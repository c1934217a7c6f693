// cache_tile128.cu -- the tile kernel (cache_tile.cuh) for values up to 128 wide.
#include "cache_tile.cuh"

namespace zeta {

cudaError_t launch_cache_tile128(const Prob &p, const TileArgs &g, int wm, cudaStream_t st) {
    return wm == 1 ? dispatch_tile<128, 1, 4>(p, g, st) : dispatch_tile<128, 2, 4>(p, g, st);
}

}  // namespace zeta
