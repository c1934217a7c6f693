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
// One cluster of eight blocks, a range of sequences each and of those some to a thread: one
// sum over r and m, its totals exchanged through distributed shared memory, gives every
// thread its offsets; the pages go back, and where there were any a cluster barrier stands
// between that and the pages that are taken.  A warp moves a sequence's pages (eight a lane
// under way), the block writes the row numbers of its sequences.  No workspace, one launch.
//
// 512 requests with a token each: 6 us, of which launch, three dependent loads and the two
// barriers are most; 256 requests of which half end or begin, up to 31 K pages moved, 262 K row numbers:
// 12 us for 0.8 MB (a page at a time a lane, and a 64-bit division a row number: 26).  Eight
// SMs write what there is to write.  A cluster of 16 (which a kernel has to ask for) and row numbers
// of sequences that move no pages, written before the barriers, were not tried.
#include <cooperative_groups.h>

#include "cache_tree.cuh"

namespace zeta {
namespace {

namespace cg = cooperative_groups;

constexpr int kBlocks = 8;
constexpr int kFlight = 8;             // pages a lane moves at a time

struct Lists {
    int32_t *table, *held, *free_list, *free_count, *granted, *slots, *status;
    int B, N;
};

// Exclusive sums of x and y over the block's threads; the totals.
struct Two {
    int64_t x, y;
};
template <int kWarps>
__device__ __forceinline__ Two block_scan(Two in, Two *sums, Two &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto scan = [&](Two v) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(kFull, v.x, o), y = __shfl_up_sync(kFull, v.y, o);
            if (lane >= o) {
                v.x += x;
                v.y += y;
            }
        }
        return v;
    };
    const Two mine = scan(in);
    __syncthreads();                                 // the array is free
    if (lane == 31) sums[warp] = mine;
    __syncthreads();
    const Two warps = scan(lane < kWarps ? sums[lane] : Two{0, 0});
    total = Two{__shfl_sync(kFull, warps.x, 31), __shfl_sync(kFull, warps.y, 31)};
    const int64_t bx = __shfl_sync(kFull, warps.x, warp - 1 & 31), by = __shfl_sync(kFull, warps.y, warp - 1 & 31);
    return Two{(warp ? bx : 0) + mine.x - in.x, (warp ? by : 0) + mine.y - in.y};
}

// A cluster barrier in two halves.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }

template <int kThreads>
__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kThreads)
cache_reserve_kernel(Cache c, Lists l) {
    constexpr int kWarps = kThreads / 32;
    __shared__ Two sums[kWarps], mine;
    __shared__ int64_t offs[kThreads];
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

    // The thread's sequences b(tid, 0), b(tid, 1), ..: what they need, what all before them do.
    const int each = (b1 - b0 + kThreads - 1) / kThreads;
    auto seq_of = [&](int s, int i) { return b0 + s * each + i; };
    Two need{0, 0}, all;                             // back and more
    for (int i = 0; i < each && seq_of(tid, i) < b1; ++i) {
        int start, count, held, want;
        sizes(seq_of(tid, i), start, count, held, want);
        need.x += max(held - want, 0);
        need.y += max(want - held, 0);
    }
    Two at = block_scan<kWarps>(need, sums, all);
    if (tid == 0) mine = all;
    cl.sync();
    int64_t R = 0;
#pragma unroll
    for (int p = 0; p < kBlocks; ++p) {
        const Two *o = cl.map_shared_rank(&mine, p);
        if (p < rank) {
            at.x += o->x;
            at.y += o->y;
        }
        R += o->x;
    }
    cluster_arrive();                                // the sums have been read
    // A list that is not one: nothing moves.
    const bool sound = F0 >= 0 && F0 + R <= c.pages;
    if (!sound && tid == 0) set_status(l.status, ZETA_ERR_BOUNDS);
    const int64_t F = F0 + R;

    // Pages [lo, hi) of a table, kFlight a lane at a time: get(e), then put(e, id).
    auto move = [&](int lo, int hi, auto get, auto put) {
        for (int e0 = lo + lane; e0 < hi; e0 += 32 * kFlight) {
            int id[kFlight];
#pragma unroll
            for (int u = 0; u < kFlight; ++u)
                if (e0 + 32 * u < hi) id[u] = get(e0 + 32 * u);
#pragma unroll
            for (int u = 0; u < kFlight; ++u)
                if (e0 + 32 * u < hi) {
                    if ((unsigned)id[u] >= (unsigned)c.pages) set_status(l.status, ZETA_ERR_BOUNDS);
                    put(e0 + 32 * u, id[u]);
                }
        }
    };
    if (sound && R > 0) {
        if (rank == 0 && tid == 0) *l.free_count = (int)F;     // every block has read it
        for (int i = 0; i < each && all.x > 0; ++i) {
            const int b = seq_of(tid, i);
            int start = 0, count = 0, held = 0, want = 0;
            if (b < b1) sizes(b, start, count, held, want);
            offs[tid] = at.x;
            at.x += max(held - want, 0);
            lo_sh[tid] = want;
            hi_sh[tid] = held;
            if (b < b1 && held > want) l.held[b] = want;
            __syncthreads();
            for (int s = warp; s < kThreads && seq_of(s, i) < b1; s += kWarps) {
                int32_t *tab = l.table + (int64_t)seq_of(s, i) * c.tlen;
                const int lo = lo_sh[s];
                const int64_t to = F - 1 - offs[s] + lo;
                move(lo, hi_sh[s], [&](int e) { return tab[e]; },
                     [&](int e, int id) {
                         l.free_list[to - e] = id;
                         tab[e] = -1;
                     });
            }
            __syncthreads();
        }
        cluster_wait();
        cl.sync();                                   // the list is whole
    }

    for (int i = 0; i < each; ++i) {
        const int b = seq_of(tid, i), ns = min(kThreads, (b1 - b0 - i + each - 1) / each);
        int start = 0, count = 0, held = 0, want = 0;
        const bool fits = b < b1 && sizes(b, start, count, held, want);
        const int m = max(want - held, 0);
        const int64_t off = at.y;
        at.y += m;
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
            int32_t *tab = l.table + (int64_t)seq_of(s, i) * c.tlen;
            const int lo = lo_sh[s];
            const int64_t from = F - 1 - offs[s] + lo;
            move(lo, hi_sh[s], [&](int e) { return l.free_list[from - e]; },
                 [&](int e, int id) { tab[e] = id; });
        }
        __syncthreads();
        if (l.slots) {
            // Four rows of a sequence a thread.
            const unsigned n = (unsigned)c.n, quads = (n + 3) / 4, cells = (unsigned)ns * quads;
            const bool whole = n % 4 == 0 && (reinterpret_cast<uintptr_t>(l.slots) & 15) == 0;
            for (unsigned x = tid; x < cells; x += kThreads) {
                const int s = (int)(x / quads), t0 = (int)(x - (unsigned)s * quads) * 4, got = got_sh[s];
                const int j0 = start_sh[s] + t0;
                const int32_t *tab = l.table + (int64_t)seq_of(s, i) * c.tlen;
                int slot[4], at = -1, id = -1;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    slot[u] = -1;
                    if (t0 + u >= got) continue;
                    const int j = j0 + u;
                    if (j >> c.psh != at) {
                        at = j >> c.psh;
                        id = tab[at];
                        if ((unsigned)id >= (unsigned)c.pages) {
                            set_status(l.status, ZETA_ERR_BOUNDS);
                            id = -1;
                        }
                    }
                    if (id >= 0) slot[u] = (id << c.psh) | (j & c.pmask);
                }
                int32_t *to = l.slots + (int64_t)seq_of(s, i) * c.n + t0;
                if (whole) {
                    *reinterpret_cast<int4 *>(to) = make_int4(slot[0], slot[1], slot[2], slot[3]);
                } else {
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (t0 + u < c.n) to[u] = slot[u];
                }
            }
        }
        __syncthreads();
    }
    if (!(sound && R > 0)) cluster_wait();           // no block ends before its sums have been read
}

}  // namespace

cudaError_t launch_cache_reserve(const Prob &p, const Cache &c, int32_t *table, int32_t *held,
                                 int32_t *free_list, int32_t *free_count, int32_t *granted,
                                 int32_t *slots, int32_t *status, cudaStream_t st) {
    const Lists l{table, held, free_list, free_count, granted, slots, status, p.B, p.N};
    // Blocks of 1024 threads take a call of many rows: 512 sequences of one row 5.8 us a call in
    // blocks of 512, 6.6 of 1024; 256 of 1024 rows, up to 31 K pages moved, 16 and 14 (before row numbers
    // were written four a thread).
    if ((int64_t)p.B * c.n < 16384) cache_reserve_kernel<512><<<kBlocks, 512, 0, st>>>(c, l);
    else cache_reserve_kernel<1024><<<kBlocks, 1024, 0, st>>>(c, l);
    return cudaGetLastError();
}

}  // namespace zeta
