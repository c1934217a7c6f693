// cache_order.cu -- the sorted prefix of every sequence that completes a chunk.
//
// Passage: OpenReview discussion of "ZETA: Leveraging Z-order Curves for
// Efficient Top-k Attention", reply A3 "Chunking ... & Where efficiency is
// coming from" (keys sorted by Z-order code within every causal prefix).
//
// Prefix c + 1 is prefix c (M = c C entries, already in order) merged with the C
// keys of chunk c.  Every key of the chunk is younger than every entry of the
// prefix, so with the chunk's run sorted by (code, token),
//   an old entry at position i with code z moves to i + #{run codes < z},
//   the run's entry j with code z goes to j + #{old codes <= z}.
// The call reads and writes the prefix once; nothing else moves with M.
//
// A block sorts the run of its (b, h) in shared memory, the token's place in the
// chunk packed below the code where both fit 64 bits: keys are dealt into buckets
// by the codes' top bits and ranked inside their bucket; where a bucket is crowded
// (equal or close codes) a bitonic sort takes over.  Its warps then stream the old
// prefix, each a span of its own, 128 entries at a time (four consecutive ones a
// lane) with the next ones on their way: the run entries that fall among them are
// found from where the last ones ended, counted into the old entries' places (one
// by one, or by binary search where there are many), and old and new go out
// through a ring in shared memory, so that the stores are whole 16-byte quads.  Several
// blocks share a slice when there are few slices; each sorts the run for itself,
// which costs less than a second launch and a round trip of the run through memory.
//
// 27 of 32 sequences completing a chunk of 1024 under prefixes of 7 K to 62 K entries, 36 K
// on average, 8 heads: 57 us for 128 MB, 2.2 TB/s; one sequence, 64 K entries, 8 heads:
// 10 us, the chain of sort, search and one or two steps.  Bound by how the work is dealt:
// with 256 slices in the call each prefix is one block's, and the 216 that have work lie
// two to an SM on some of the 152.  The longest sequence alone takes 38 us, the longest
// thirteen of the 27 take the whole 56, 27 equal prefixes of 35 K 47, of 61 K 65.  Within a
// block it is issue (58 % of the slots over the call, 101 instructions for an entry of
// each lane with the sorts; 64 registers, up to 40 bytes of spills).  Stores entry by entry
// took 67 us, a bitonic sort and a merge of the entries one by one 190 and 38 us.
#include "cache.cuh"

namespace zeta {
namespace {

constexpr int kThreads = 512;
constexpr int kStep = 128;              // old entries a warp takes at a time
constexpr int kFew = 16;                // run entries among them up to which they go one by one
                                        // (64 sequences under 32 K entries 65 us; 8: 68, 5: 74)
constexpr int kCrowd = 48;              // keys of a bucket above which the bitonic sort runs
constexpr int kLocBits = 13;            // a place in the chunk: C <= 8192

// The run in shared memory: keys ordered by (code, place).  Packed: one word
// (code << 13 | place); else the code and the place apart.
template <bool PACK>
struct Run {
    uint64_t *key;
    uint16_t *loc;
    // Compare-exchange of entries i < j, ascending if up.
    __device__ __forceinline__ void order2(int i, int j, bool up) {
        const uint64_t a = key[i], b = key[j];
        if constexpr (PACK) {
            if ((a > b) == up) {
                key[i] = b;
                key[j] = a;
            }
        } else {
            const uint16_t la = loc[i], lb = loc[j];
            if ((a > b || (a == b && la > lb)) == up) {
                key[i] = b;
                key[j] = a;
                loc[i] = lb;
                loc[j] = la;
            }
        }
    }
    // The steps of stride 16 .. 1 of stages [from, to] (sizes) on 32 entries, one a lane.
    __device__ __forceinline__ void order32(int base, int lane, int from, int to) {
        const int i = base + lane;
        uint64_t a = key[i];
        unsigned la = 0;
        if constexpr (!PACK) la = loc[i];
        for (int size = from; size <= to; size <<= 1) {
            for (int d = min(size >> 1, 16); d > 0; d >>= 1) {
                const uint64_t b = __shfl_xor_sync(kFull, a, d);
                const bool keep_min = ((i & size) == 0) == ((lane & d) == 0);
                if constexpr (PACK) {
                    if ((b < a) == keep_min) a = b;
                } else {
                    const unsigned lb = __shfl_xor_sync(kFull, la, d);
                    if ((b < a || (b == a && lb < la)) == keep_min) {
                        a = b;
                        la = lb;
                    }
                }
            }
        }
        key[i] = a;
        if constexpr (!PACK) loc[i] = (uint16_t)la;
    }
    __device__ __forceinline__ void set(int i, uint64_t code, int place) {
        if constexpr (PACK) key[i] = (code << kLocBits) | (unsigned)place;
        else { key[i] = code; loc[i] = (uint16_t)place; }
    }
    __device__ __forceinline__ void pad(int i) {
        key[i] = ~0ull;
        if constexpr (!PACK) loc[i] = 0xffff;
    }
    __device__ __forceinline__ uint64_t code(int i) const {
        return PACK ? key[i] >> kLocBits : key[i];
    }
    __device__ __forceinline__ int place(int i) const {
        return PACK ? (int)(key[i] & ((1u << kLocBits) - 1)) : loc[i];
    }
    // Entries with a code below z, known to be lo .. hi.
    __device__ __forceinline__ int below(uint64_t z, int lo, int hi) const {
        const uint64_t x = PACK ? z << kLocBits : z;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (key[mid] < x) lo = mid + 1; else hi = mid;
        }
        return lo;
    }
};

// Old entries in registers: four consecutive ones a lane.
template <typename K>
struct Old {
    K z[4];
    int token[4];
    bool lost;
};

// One warp's output stage: entry e of the new prefix at e % kRing.  At most kKeep
// entries stay when a step ends, so that the next one's kStep + kFew fit.
constexpr int kRing = 256;
constexpr int kKeep = kRing - kStep - kFew;
template <typename K>
struct Stage {
    K z[kRing];
    int token[kRing];
};

template <typename K, bool PACK>
__global__ void __launch_bounds__(kThreads, 2)
cache_order_kernel(Cache c, const float *__restrict__ k_pages, K *codes, int32_t *idx,
                   int32_t *status, int N, int H, int dK, int bits, int C, int C2, int NB) {
    extern __shared__ __align__(16) unsigned char raw[];
    __shared__ int warp_sum[kThreads / 32];
    const int s = blockIdx.y, b = s / H, h = s - b * H;
    const Seq q = seq_of(c, b, N, status);
    const int c1 = (q.start + q.count) / C;               // the prefix to make
    if (c1 <= q.start / C) return;
    const int M = (c1 - 1) * C;
    // The warps' spans of the old prefix; a block without any returns (the first
    // block stays for an empty prefix).
    constexpr int kWarps = kThreads / 32;
    const int warps = (int)gridDim.x * kWarps;
    const int span = ((M + warps - 1) / warps + kStep - 1) / kStep * kStep;
    if (blockIdx.x > 0 && (int64_t)blockIdx.x * kWarps * span >= M) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Run<PACK> run;
    run.key = reinterpret_cast<uint64_t *>(raw);
    uint64_t *tmp = run.key + C2;                          // dealt keys; later the stages
    int *cnt = reinterpret_cast<int *>(tmp + C2);          // buckets (NB + 1)
    run.loc = reinterpret_cast<uint16_t *>(tmp);           // !PACK: no buckets
    const int32_t *ptab = c.ptab + (int64_t)b * c.tlen, *otab = c.otab + (int64_t)b * c.tlen;

    const int64_t plane = (int64_t)c.opages * H << c.psh;
    const K *src_z = codes + ((c1 - 1) & 1) * plane;
    const int32_t *src_i = idx + ((c1 - 1) & 1) * plane;
    K *dst_z = codes + (c1 & 1) * plane;
    int32_t *dst_i = idx + (c1 & 1) * plane;
    auto order_row = [&](int id, int e) { return row_in(id, e, h, H, c.psh, c.pmask, c.opages); };

    // ------------------------------------------------------------ the run ---
    bool bad = false;
    const int sh = PACK ? max(0, dK * bits - (31 - __clz(NB))) + kLocBits : 0;
    if constexpr (PACK)
        for (int i = tid; i <= NB; i += kThreads) cnt[i] = 0;
    for (int j = tid; j < C2; j += kThreads) {
        if (j < C) {
            const int row = page_row(ptab, M + j, h, H, c.psh, c.pmask, c.pages);
            bad |= row < 0;
            float x[kMaxDK];
            load_point(x, k_pages + (int64_t)max(row, 0) * dK, dK);
            run.set(j, code_of(x, dK, bits), j);
        } else {
            run.pad(j);
        }
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) set_status(status, ZETA_ERR_BOUNDS);
        return;
    }
    bool crowded = true;
    if constexpr (PACK) {
        // Count, exclusive sums, deal; then each key's rank among its bucket's.
        for (int j = tid; j < C; j += kThreads) atomicAdd(&cnt[run.key[j] >> sh], 1);
        __syncthreads();
        const int per = NB / kThreads;                     // NB is a multiple
        int sum = 0, most = 0;
        for (int i = 0; i < per; ++i) {
            const int n = cnt[tid * per + i];
            most = max(most, n);
            sum += n;
        }
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) warp_sum[warp] = inc;
        crowded = __syncthreads_or(most > kCrowd);
        if (!crowded) {
            int base = inc - sum;
            for (int w = 0; w < warp; ++w) base += warp_sum[w];
            for (int i = 0; i < per; ++i) {
                const int n = cnt[tid * per + i];
                cnt[tid * per + i] = base;
                base += n;
            }
            __syncthreads();
            // Dealing moves every bucket's start to its end, the next one's start.
            for (int j = tid; j < C; j += kThreads) {
                const uint64_t x = run.key[j];
                tmp[atomicAdd(&cnt[x >> sh], 1)] = x;
            }
            __syncthreads();
            for (int j = tid; j < C; j += kThreads) {
                const uint64_t x = tmp[j];
                const int bk = (int)(x >> sh), first = bk > 0 ? cnt[bk - 1] : 0, end = cnt[bk];
                int r = first;
                for (int i = first; i < end; ++i) r += tmp[i] < x;
                run.key[r] = x;
            }
        }
    }
    if (crowded) {
        for (int g = warp * 32; g < C2; g += kThreads) run.order32(g, lane, 2, 32);
        for (int size = 64; size <= C2; size <<= 1) {
            for (int d = size >> 1; d >= 32; d >>= 1) {
                __syncthreads();
                for (int p = tid; p < C2 / 2; p += kThreads) {
                    const int i = 2 * p - (p & (d - 1));
                    run.order2(i, i + d, (i & size) == 0);
                }
            }
            __syncthreads();
            for (int g = warp * 32; g < C2; g += kThreads) run.order32(g, lane, size, size);
        }
    }
    __syncthreads();

    // ---------------------------------------------------------- the merge ---
    bool lost = false;
    auto put = [&](int id, int e, K z, int token) {        // entry e, id its page
        const int row = order_row(id, e);
        lost |= row < 0;
        if (row >= 0) {
            dst_z[row] = z;
            dst_i[row] = token;
        }
    };
    if (M == 0)
        for (int j = tid; j < C; j += kThreads)
            put(page_id(otab, j, c.psh), j, (K)run.code(j), run.place(j));
    const int i0 = (int)min((int64_t)(blockIdx.x * kWarps + warp) * span, (int64_t)M);
    const int i1 = min(i0 + span, M);
    Stage<K> &out = reinterpret_cast<Stage<K> *>(reinterpret_cast<unsigned char *>(tmp) +
                                                 (PACK ? 0 : (size_t)C2 * 2))[warp];
    // Pages of less than four entries are looked up entry by entry.
    const bool quad = c.pmask >= 3;
    struct Ids { int id[4]; };
    auto ask = [&](int i) {                                // pages of the lane's entries
        Ids a;
        const int e = i + 4 * lane;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k == 0 || !quad) a.id[k] = page_id(otab, min(e + k, M - 1), c.psh);
        return a;
    };
    auto fetch = [&](const Ids &a, int i) {                // the entries on those pages
        Old<K> o;
        o.lost = false;
        const int e = i + 4 * lane;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            o.z[k] = K(0);
            o.token[k] = 0;
        }
        if (quad && e + 3 < M) {
            const int row = order_row(a.id[0], e);
            o.lost = row < 0;
            if (row >= 0) {
                const int4 t = __ldg(reinterpret_cast<const int4 *>(src_i + row));
                o.token[0] = t.x; o.token[1] = t.y; o.token[2] = t.z; o.token[3] = t.w;
                if constexpr (sizeof(K) == 4) {
                    const uint4 z = __ldg(reinterpret_cast<const uint4 *>(src_z + row));
                    o.z[0] = z.x; o.z[1] = z.y; o.z[2] = z.z; o.z[3] = z.w;
                } else {
                    const ulonglong2 u = __ldg(reinterpret_cast<const ulonglong2 *>(src_z + row));
                    const ulonglong2 v = __ldg(reinterpret_cast<const ulonglong2 *>(src_z + row) + 1);
                    o.z[0] = u.x; o.z[1] = u.y; o.z[2] = v.x; o.z[3] = v.y;
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (e + k < M) {
                    const int row = order_row(quad ? a.id[0] : a.id[k], e + k);
                    o.lost |= row < 0;
                    if (row >= 0) {
                        o.z[k] = __ldg(src_z + row);
                        o.token[k] = __ldg(src_i + row);
                    }
                }
        }
        return o;
    };
    Old<K> one, two;
    Ids ids;
    if (i0 < i1) {
        const Ids first = ask(i0);
        ids = ask(i0 + kStep);
        one = fetch(first, i0);
    }
    // A step takes the run entries below its last code that no step before it took
    // (the prefix's last step all that are left): lo .. hi.
    int lo = 0;
    if (i0 > 0 && i0 < i1) {
        const int row = order_row(page_id(otab, i0 - 1, c.psh), i0 - 1);
        lo = row >= 0 ? run.below((uint64_t)__ldg(src_z + row), 0, C) : 0;
    }
    // Entries head .. tail - 1 of the new prefix wait in the stage.  They leave four a
    // lane, on 16-byte boundaries, until no more than kKeep are left (or none: `all`).
    int head = i0 + lo;
    auto flush = [&](int tail, bool all) {
        auto singly = [&](int to) {
            for (int e = head + lane; e < to; e += 32)
                put(page_id(otab, e, c.psh), e, out.z[e & (kRing - 1)], out.token[e & (kRing - 1)]);
            head = max(head, to);
        };
        if (all || !quad) {
            singly(tail);
        } else {
            singly(min((head + 3) & ~3, tail));
            while (tail - head > kKeep) {
                const int nq = min(32, (tail - head) >> 2);
                if (lane < nq) {
                    const int e = head + 4 * lane;
                    const int row = order_row(page_id(otab, e, c.psh), e);
                    lost |= row < 0;
                    if (row >= 0) {
                        const int at = e & (kRing - 1);
                        *reinterpret_cast<int4 *>(dst_i + row) = *reinterpret_cast<const int4 *>(out.token + at);
                        *reinterpret_cast<uint4 *>(dst_z + row) = *reinterpret_cast<const uint4 *>(out.z + at);
                        if constexpr (sizeof(K) == 8)
                            *reinterpret_cast<uint4 *>(dst_z + row + 2) = *reinterpret_cast<const uint4 *>(out.z + at + 2);
                    }
                }
                head += 4 * nq;
            }
        }
    };
    // Two sets of registers in turn: copying the next entries would wait for them.
    int i = i0;
    auto turn = [&](const Old<K> &cur, Old<K> &nxt) {
        nxt = fetch(ids, i + kStep);
        ids = ask(i + 2 * kStep);
        lost |= cur.lost;
        const int e = i + 4 * lane, cnt = min(kStep, M - i), mine = min(4, M - e);
        const bool last = i + kStep >= M;
        const K run_z = lo + lane < C ? (K)run.code(lo + lane) : K(0);
        const K zn = __shfl_sync(kFull, cur.z[3], 31);
        const unsigned in = __ballot_sync(kFull, lo + lane < C && (last || run_z < zn));
        const int few = __popc(in);
        int hi = lo + few;
        if (few <= kFew) {                                 // one at a time, through the stage
            int place[4] = {0, 0, 0, 0};
            const int token = M + run.place(min(lo + lane, C - 1));
            for (int j = 0; j < few; ++j) {
                const K z = __shfl_sync(kFull, run_z, j);
                int after = 0;                             // of the lane's entries
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool a = k < mine && cur.z[k] > z;
                    place[k] += a;
                    after += a;
                }
                const int le = cnt - (int)__reduce_add_sync(kFull, (unsigned)after);
                if (lane == j) {
                    out.z[(i + lo + j + le) & (kRing - 1)] = z;
                    out.token[(i + lo + j + le) & (kRing - 1)] = token;
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < mine) {
                    const int at = (e + k + lo + place[k]) & (kRing - 1);
                    out.z[at] = cur.z[k];
                    out.token[at] = cur.token[k];
                }
            __syncwarp();
            flush(i + lo + cnt + few, false);
            __syncwarp();
        } else {                                           // many: by binary search
            if (in == kFull) hi = last ? C : run.below(zn, lo, C);
            flush(i + lo, true);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < mine) {
                    const int at = e + k + run.below((uint64_t)cur.z[k], lo, hi);
                    put(page_id(otab, at, c.psh), at, cur.z[k], cur.token[k]);
                    out.z[4 * lane + k] = cur.z[k];
                }
            __syncwarp();
            for (int j = lo + lane; j < hi; j += 32) {
                const uint64_t z = run.code(j);
                int a = 0, n = cnt;                        // old entries of the step with code <= z
                while (a < n) {
                    const int mid = (a + n) >> 1;
                    if ((uint64_t)out.z[mid] <= z) a = mid + 1; else n = mid;
                }
                put(page_id(otab, i + j + a, c.psh), i + j + a, (K)z, M + run.place(j));
            }
            head = i + cnt + hi;
            __syncwarp();
        }
        lo = hi;
        i += kStep;
    };
    while (i < i1) {
        turn(one, two);
        if (i >= i1) break;
        turn(two, one);
    }
    if (i0 < i1) flush(min(i, M) + lo, true);
    if (lost) set_status(status, ZETA_ERR_BOUNDS);
}

template <typename K, bool PACK>
cudaError_t run_order(const Prob &p, const Cache &c, const float *k_pages, void *codes,
                      int32_t *idx, int32_t *status, cudaStream_t st) {
    static PerDeviceOnce once;
    // Keys; then the dealt keys and their buckets, or the places (!PACK), and in the
    // same space, after the sort, the warps' stages.
    int C2 = 32, NB = kThreads;
    while (C2 < p.C) C2 <<= 1;
    while (NB < C2 && NB < 4096) NB <<= 1;
    const size_t stages = sizeof(Stage<K>) * (kThreads / 32);
    auto bytes = [&](size_t n, size_t nb) {
        const size_t sort = PACK ? n * 8 + (nb + 1) * 4 : n * 2;
        return n * 8 + (PACK ? (sort > stages ? sort : stages) : sort + stages);
    };
    const size_t smem = bytes(C2, NB), most_smem = bytes(8192, 4096);
    cudaError_t e = once.run([&] {
        return cudaFuncSetAttribute(cache_order_kernel<K, PACK>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most_smem);
    });
    if (e != cudaSuccess) return e;
    // Blocks per slice: as many as fit at once, two on each of the 152 SMs; the kernel
    // leaves out those that its prefix has no entries for.  (Rounded up instead, 16
    // sequences under 64 K entries take 44 us instead of 36, 32 under 36 K 56 instead of 57.)
    int64_t g = 152 * 2 / p.S;
    const int64_t most = p.N / (kStep * kThreads / 32) + 1;
    g = g < most ? g : most;
    const dim3 grid((unsigned)(g < 1 ? 1 : g), (unsigned)p.S);
    cache_order_kernel<K, PACK><<<grid, kThreads, smem, st>>>(
        c, k_pages, static_cast<K *>(codes), idx, status, p.N, p.H, p.dK, p.bits, p.C, C2,
        NB);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_order(const Prob &p, const Cache &c, const float *k_pages,
                               void *order_codes, int32_t *order_idx, int32_t *status,
                               cudaStream_t st) {
    if (!p.code64)
        return run_order<uint32_t, true>(p, c, k_pages, order_codes, order_idx, status, st);
    if (p.dK * p.bits + kLocBits <= 64)
        return run_order<uint64_t, true>(p, c, k_pages, order_codes, order_idx, status, st);
    return run_order<uint64_t, false>(p, c, k_pages, order_codes, order_idx, status, st);
}

}  // namespace zeta
