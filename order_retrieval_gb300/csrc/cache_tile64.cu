// cache_tile64.cu -- the tile kernel (cache_tile.cuh) for values up to 64 wide.
#include "cache_tile.cuh"

namespace zeta {

cudaError_t launch_cache_tile64(const Prob &p, const TileArgs &g, bool wide, cudaStream_t st) {
    return wide ? dispatch_tile<64, 8, 8>(p, g, st) : dispatch_tile<64, 1, 8>(p, g, st);
}

}  // namespace zeta
