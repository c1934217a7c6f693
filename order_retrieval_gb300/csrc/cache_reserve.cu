// cache_reserve.cu -- page tables and row numbers from the requests' lengths.
//
// Sequence b shall hold w = ceil((start + count) / page) pages.  With r_b = held - w
// pages too many (or none) and m_b = w - held too few, free places F before the call:
//   back   the e-th page given back (b ascending, entry ascending) goes to place
//          F + R - 1 - e of the list, R = sum r_b, so that the first lies on top;
//   out    with F' = F + R and M_b = m_0 + .. + m_b, sequence b gets its pages if
//          M_b <= F': the e-th taken comes from place F' - 1 - e.
// The e-th page back is the e-th one out again: a shrink undoes a grow to the last
// place of the list.
//
// One cluster of eight blocks, a range of sequences each: sums of r and m, exchanged
// through distributed shared memory, give every block its offsets; the pages go back,
// and a cluster barrier stands between that and the pages that are taken.  A thread
// takes a sequence for the sums, a warp a sequence for its pages, the block all rows of
// its sequences for the row numbers.  No workspace, one launch.
#include <cooperative_groups.h>

#include "cache_tree.cuh"

namespace zeta {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32, kBlocks = 8;

struct Lists {
    int32_t *table, *held, *free_list, *free_count, *granted, *slots, *status;
    int B, N;
};

// Exclusive sum over the block's threads; *total gets the sum.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *sums, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, in, o);
        if (lane >= o) in += y;
    }
    __syncthreads();                                 // the array is free
    if (lane == 31) sums[warp] = in;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sums[w];
        all += sums[w];
    }
    *total = all;
    return before + in - x;
}

__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kThreads)
cache_reserve_kernel(Cache c, Lists l) {
    __shared__ int64_t sums[kWarps], mine[2], offs[kThreads];
    __shared__ int lo_sh[kThreads], hi_sh[kThreads], start_sh[kThreads], got_sh[kThreads];
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cl.block_rank();
    const int per = (l.B + kBlocks - 1) / kBlocks;
    const int b0 = min(rank * per, l.B), b1 = min(b0 + per, l.B);
    const int F0 = *l.free_count;

    // Sequence b: pages held and wanted; false where a length is out of range.
    auto sizes = [&](int b, int &start, int &count, int &held, int &want) {
        start = c.start[b];
        count = c.count[b];                          // may be the array granted goes to
        held = l.held[b];
        want = held;
        if (start < 0 || count < 0 || count > c.n || start > l.N - count || held < 0 ||
            held > c.tlen) {
            set_status(l.status, ZETA_ERR_BOUNDS);
            return false;
        }
        want = (int)(((int64_t)start + count + c.pmask) >> c.psh);
        return true;
    };

    // Sums of the block's range, and what the blocks before it and all have.
    int64_t back = 0, more = 0;
    for (int b = b0 + tid; b < b1; b += kThreads) {
        int start, count, held, want;
        sizes(b, start, count, held, want);
        back += max(held - want, 0);
        more += max(want - held, 0);
    }
    int64_t all_back, all_more;
    block_scan(back, sums, &all_back);
    block_scan(more, sums, &all_more);
    if (tid == 0) {
        mine[0] = all_back;
        mine[1] = all_more;
    }
    cl.sync();
    int64_t at_back = 0, at_more = 0, R = 0;
    for (int p = 0; p < kBlocks; ++p) {
        const int64_t *o = cl.map_shared_rank(mine, p);
        if (p < rank) {
            at_back += o[0];
            at_more += o[1];
        }
        R += o[0];
    }
    // A list that is not one: nothing moves.
    const bool sound = F0 >= 0 && F0 + R <= c.pages;
    if (!sound && tid == 0) set_status(l.status, ZETA_ERR_BOUNDS);
    const int64_t F = F0 + R;
    if (sound && rank == 0 && tid == 0) *l.free_count = (int)F;   // every block has read it

    for (int s0 = b0; s0 < b1 && sound; s0 += kThreads) {
        const int b = s0 + tid;
        int start = 0, count = 0, held = 0, want = 0;
        if (b < b1) sizes(b, start, count, held, want);
        int64_t total;
        offs[tid] = at_back + block_scan(max(held - want, 0), sums, &total);
        at_back += total;
        lo_sh[tid] = want;
        hi_sh[tid] = held;
        if (b < b1 && held > want) l.held[b] = want;
        __syncthreads();
        for (int s = warp; s < min(kThreads, b1 - s0); s += kWarps) {
            int32_t *tab = l.table + (int64_t)(s0 + s) * c.tlen;
            const int lo = lo_sh[s], hi = hi_sh[s];
            for (int e = lo + lane; e < hi; e += 32) {
                const int id = tab[e];
                if ((unsigned)id >= (unsigned)c.pages) set_status(l.status, ZETA_ERR_BOUNDS);
                l.free_list[F - 1 - (offs[s] + e - lo)] = id;
                tab[e] = -1;
            }
        }
        __syncthreads();
    }
    cl.sync();                                       // the list is whole; the sums have been read

    for (int s0 = b0; s0 < b1; s0 += kThreads) {
        const int b = s0 + tid, ns = min(kThreads, b1 - s0);
        int start = 0, count = 0, held = 0, want = 0;
        const bool fits = b < b1 && sizes(b, start, count, held, want);
        const int m = max(want - held, 0);
        int64_t total;
        const int64_t off = at_more + block_scan(m, sums, &total);
        at_more += total;
        const bool ok = fits && sound && (m == 0 || off + m <= F);
        offs[tid] = off;
        lo_sh[tid] = held;
        hi_sh[tid] = ok ? want : held;
        start_sh[tid] = start;
        got_sh[tid] = ok ? count : 0;
        if (b < b1) {
            l.granted[b] = ok ? count : 0;
            if (ok && m > 0) l.held[b] = want;
            // The last one that gets pages leaves the fewest places.
            if (ok && m > 0) atomicMin(l.free_count, (int)(F - off - m));
        }
        __syncthreads();
        for (int s = warp; s < ns; s += kWarps) {
            int32_t *tab = l.table + (int64_t)(s0 + s) * c.tlen;
            const int lo = lo_sh[s], hi = hi_sh[s];
            for (int e = lo + lane; e < hi; e += 32) {
                const int id = l.free_list[F - 1 - (offs[s] + e - lo)];
                if ((unsigned)id >= (unsigned)c.pages) set_status(l.status, ZETA_ERR_BOUNDS);
                tab[e] = id;
            }
        }
        __syncthreads();
        if (l.slots) {
            for (int64_t x = tid; x < (int64_t)ns * c.n; x += kThreads) {
                const int s = (int)(x / c.n), t = (int)(x - (int64_t)s * c.n);
                int slot = -1;
                if (t < got_sh[s]) {
                    const int i = start_sh[s] + t;
                    const int id = l.table[(int64_t)(s0 + s) * c.tlen + (i >> c.psh)];
                    if ((unsigned)id < (unsigned)c.pages) slot = (id << c.psh) | (i & c.pmask);
                    else set_status(l.status, ZETA_ERR_BOUNDS);
                }
                l.slots[(int64_t)s0 * c.n + x] = slot;
            }
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_cache_reserve(const Prob &p, const Cache &c, int32_t *table, int32_t *held,
                                 int32_t *free_list, int32_t *free_count, int32_t *granted,
                                 int32_t *slots, int32_t *status, cudaStream_t st) {
    const Lists l{table, held, free_list, free_count, granted, slots, status, p.B, p.N};
    cache_reserve_kernel<<<kBlocks, kThreads, 0, st>>>(c, l);
    return cudaGetLastError();
}

}  // namespace zeta
