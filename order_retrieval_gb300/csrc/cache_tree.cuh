// cache_tree.cuh -- what the kernels on a tree of drafted tokens share.
//
// Node t of a sequence with `start` tokens hangs below node parent[t] < t or, with -1,
// below the sequence's last token.  Its position is start + depth; a line of nodes from
// the top to t is at most n long, and its node numbers rise.
#pragma once

#include "cache.cuh"

namespace zeta {

constexpr int kMaxDraft = 1024;       // nodes a sequence (a tree's parents are held in shared memory)

struct TreeArgs {
    Cache c;
    const int32_t *parent;            // [B, n]
    const float *q, *k, *gamma, *k_pages;
    const void *v, *v_pages, *order_codes;
    const int32_t *order_idx;
    void *out;
    float *rowsum;
    int32_t *idx, *status;
    int N, H, dK, dV, kw, C, bits, wk, code64;
};

// What sequence b drafts: as seq_of, but only the first drafted token needs room below N
// (what lies behind the chunk's end, and so behind N, has no result).
__device__ __forceinline__ Seq drafts_of(const Cache &c, int b, int N, int32_t *status) {
    Seq s{__ldg(c.start + b), __ldg(c.count + b)};
    if (s.start < 0 || s.count < 0 || s.count > c.n || s.start > N - (s.count > 0 ? 1 : 0)) {
        set_status(status, ZETA_ERR_BOUNDS);
        s.count = 0;
    }
    return s;
}

// Depth of node t, -1 where a parent on the way up is no earlier node; each node visited
// is handed to `visit` from t upwards.
template <typename Visit>
__device__ __forceinline__ int climb(const int *parent, int t, Visit visit) {
    int depth = -1;
    while (t >= 0) {
        visit(t);
        const int p = parent[t];
        ++depth;
        if (p < -1 || p >= t) return -1;
        t = p;
    }
    return depth;
}

// The same with the line as bits of `above`; run: bit t set where parent[t] == t - 1, t > 0,
// so that nodes that hang below one another by number (a chain) are one step of up to 32.
__device__ __forceinline__ int climb_bits(const int *parent, const uint32_t *run, int t,
                                          uint32_t *above) {
    int depth = -1;
    while (t >= 0) {
        const int w = t >> 5;
        const uint32_t upto = 0xffffffffu >> (31 - (t & 31));
        const uint32_t ends = ~run[w] & upto;        // nodes whose parent is not the one before
        const int s = ends ? 31 - __clz(ends) : 0;
        const uint32_t part = upto & (0xffffffffu << s);
        above[w] |= part;
        depth += __popc(part);
        const int top = w * 32 + s, p = ends ? parent[top] : top - 1;
        if (p < -1 || p >= top) return -1;
        t = p;
    }
    return depth;
}

// The bits of `run` for nodes 32 w .. 32 w + 31 (a warp).
__device__ __forceinline__ uint32_t run_bits(const int *parent, int w, int nodes) {
    const int u = w * 32 + (threadIdx.x & 31);
    return __ballot_sync(kFull, u < nodes && u > 0 && parent[u] == u - 1);
}

cudaError_t launch_cache_attend_tree(const Prob &p, const TreeArgs &g, cudaStream_t st);
cudaError_t launch_cache_accept(const Prob &p, const Cache &c, const int32_t *parent,
                                const int32_t *leaf, const int32_t *granted, const float *k,
                                const void *v, float *k_pages, void *v_pages, int32_t *accepted,
                                int32_t *path, int32_t *status, cudaStream_t st);
cudaError_t launch_cache_reserve(const Prob &p, const Cache &c, int32_t *table, int32_t *held,
                                 int32_t *free_list, int32_t *free_count, int32_t *granted,
                                 int32_t *slots, int32_t *status, cudaStream_t st);

}  // namespace zeta
