// cache_tree_bf16.cu -- the tile kernel for drafted trees (cache_tree_tile.cuh), bf16 values.
#include "cache_tree_tile.cuh"

namespace zeta {

// 32 bytes of a value row a load where every row is 32-byte aligned.
cudaError_t launch_tree_tile_bf16(const Prob &p, const TreeArgs &g, int cs, cudaStream_t st) {
    const bool wide = p.dV % 16 == 0 && ((reinterpret_cast<uintptr_t>(g.v) | reinterpret_cast<uintptr_t>(g.v_pages)) & 31) == 0;
    if (p.dV <= 64)
        return wide ? dispatch_tree_tile<__nv_bfloat16, 64, true>(p, g, cs, st)
                    : dispatch_tree_tile<__nv_bfloat16, 64, false>(p, g, cs, st);
    return wide ? dispatch_tree_tile<__nv_bfloat16, 128, true>(p, g, cs, st)
                : dispatch_tree_tile<__nv_bfloat16, 128, false>(p, g, cs, st);
}

}  // namespace zeta
