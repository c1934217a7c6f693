// cache_tree_bf16.cu -- the tile kernel for drafted trees (cache_tree_tile.cuh), bf16 values.
#include "cache_tree_tile.cuh"

namespace zeta {

cudaError_t launch_tree_tile_bf16(const Prob &p, const TreeArgs &g, int cs, cudaStream_t st) {
    return p.dV <= 64 ? dispatch_tree_tile<__nv_bfloat16, 64>(p, g, cs, st)
                      : dispatch_tree_tile<__nv_bfloat16, 128>(p, g, cs, st);
}

}  // namespace zeta
