// cache_tree_bf16.cu -- the tile kernel for drafted trees (cache_tree_tile.cuh), bf16 values.
#include "cache_tree_tile.cuh"

namespace zeta {

// 32 bytes of a value row a load where every row is 32-byte aligned.
cudaError_t launch_tree_tile_bf16(const Prob &p, const TreeArgs &g, int ng, int cs, cudaStream_t st) {
    using V = __nv_bfloat16;
    const bool wide = p.dV % 16 == 0 && ((reinterpret_cast<uintptr_t>(g.v) | reinterpret_cast<uintptr_t>(g.v_pages)) & 31) == 0;
    if (p.dV > 64) return wide ? dispatch_tree_tile<V, 128, 1, true>(p, g, cs, st) : dispatch_tree_tile<V, 128, 1, false>(p, g, cs, st);
    if (ng == 2) return wide ? dispatch_tree_tile<V, 64, 2, true>(p, g, cs, st) : dispatch_tree_tile<V, 64, 2, false>(p, g, cs, st);
    return wide ? dispatch_tree_tile<V, 64, 1, true>(p, g, cs, st) : dispatch_tree_tile<V, 64, 1, false>(p, g, cs, st);
}

}  // namespace zeta
