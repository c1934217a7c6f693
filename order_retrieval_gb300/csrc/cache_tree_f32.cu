// cache_tree_f32.cu -- the tile kernel for drafted trees (cache_tree_tile.cuh), float32 values.
#include "cache_tree_tile.cuh"

namespace zeta {

cudaError_t launch_tree_tile_f32(const Prob &p, const TreeArgs &g, int ng, int cs, cudaStream_t st) {
    if (p.dV > 64) return dispatch_tree_tile<float, 128, 1, false>(p, g, cs, st);
    return ng == 2 ? dispatch_tree_tile<float, 64, 2, false>(p, g, cs, st) : dispatch_tree_tile<float, 64, 1, false>(p, g, cs, st);
}

}  // namespace zeta
