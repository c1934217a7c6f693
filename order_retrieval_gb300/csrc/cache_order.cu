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
// A block sorts the run of its (b, h) in shared memory (bitonic, the token's
// place in the chunk packed below the code where both fit 64 bits), then takes
// tiles of the old prefix: the tile's codes in shared memory, each old entry
// placed by a binary search in the run, each run entry that falls into the tile
// by a binary search in the tile.  Several blocks share a slice when there are
// few slices; each sorts the run for itself, which costs less than a second
// launch and a round trip of the run through memory.
#include "cache.cuh"

namespace zeta {
namespace {

constexpr int kThreads = 512;
constexpr int kTile = 1024;             // old entries per tile
constexpr int kLocBits = 13;            // a place in the chunk: C <= 8192

// The run in shared memory: keys ordered by (code, place).  Packed: one word
// (code << 13 | place); else the code and the place apart.
template <bool PACK>
struct Run {
    uint64_t *key;
    uint16_t *loc;
    __device__ __forceinline__ bool after(int i, int j) const {   // entry i sorts after entry j
        if constexpr (PACK) return key[i] > key[j];
        else return key[i] > key[j] || (key[i] == key[j] && loc[i] > loc[j]);
    }
    __device__ __forceinline__ void swap(int i, int j) {
        const uint64_t a = key[i];
        key[i] = key[j];
        key[j] = a;
        if constexpr (!PACK) {
            const uint16_t l = loc[i];
            loc[i] = loc[j];
            loc[j] = l;
        }
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
    // Entries with a code below z.
    __device__ __forceinline__ int below(uint64_t z, int C) const {
        const uint64_t x = PACK ? z << kLocBits : z;
        int lo = 0, hi = C;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (key[mid] < x) lo = mid + 1; else hi = mid;
        }
        return lo;
    }
};

template <typename K, bool PACK>
__global__ void __launch_bounds__(kThreads)
cache_order_kernel(Cache c, const float *__restrict__ k_pages, K *codes, int32_t *idx,
                   int32_t *status, int N, int H, int dK, int bits, int C, int C2) {
    extern __shared__ __align__(16) unsigned char raw[];
    const int s = blockIdx.y, b = s / H, h = s - b * H;
    const Seq q = seq_of(c, b, N, status);
    const int c1 = (q.start + q.count) / C;               // the prefix to make
    if (c1 <= q.start / C) return;
    const int M = (c1 - 1) * C;
    Run<PACK> run;
    run.key = reinterpret_cast<uint64_t *>(raw);
    K *tile = reinterpret_cast<K *>(run.key + C2);
    run.loc = reinterpret_cast<uint16_t *>(tile + kTile + 1);
    const int32_t *ptab = c.ptab + (int64_t)b * c.tlen, *otab = c.otab + (int64_t)b * c.tlen;
    const int tid = threadIdx.x;

    // ------------------------------------------------------------ the run ---
    bool bad = false;
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
    for (int size = 2; size <= C2; size <<= 1) {
        for (int d = size >> 1; d > 0; d >>= 1) {
            for (int p = tid; p < C2 / 2; p += kThreads) {
                const int i = 2 * p - (p & (d - 1)), j = i + d;
                const bool up = (i & size) == 0;
                if (run.after(i, j) == up) run.swap(i, j);
            }
            __syncthreads();
        }
    }

    // ---------------------------------------------------------- the merge ---
    const int64_t plane = (int64_t)c.opages * H << c.psh;
    const K *src_z = codes + ((c1 - 1) & 1) * plane;
    const int32_t *src_i = idx + ((c1 - 1) & 1) * plane;
    K *dst_z = codes + (c1 & 1) * plane;
    int32_t *dst_i = idx + (c1 & 1) * plane;
    auto put = [&](int e, uint64_t z, int token) {
        const int row = page_row(otab, e, h, H, c.psh, c.pmask, c.opages);
        if (row < 0) {
            set_status(status, ZETA_ERR_BOUNDS);
            return;
        }
        dst_z[row] = (K)z;
        dst_i[row] = token;
    };
    if (M == 0) {
        for (int j = blockIdx.x * kThreads + tid; j < C; j += gridDim.x * kThreads)
            put(j, run.code(j), run.place(j));
        return;
    }
    const int tiles = (M + kTile - 1) / kTile;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int i0 = t * kTile, cnt = min(kTile, M - i0);
        int token[kTile / kThreads];
#pragma unroll
        for (int u = 0; u < kTile / kThreads; ++u) {
            const int l = u * kThreads + tid;
            token[u] = 0;
            if (l < cnt) {
                const int row = page_row(otab, i0 + l, h, H, c.psh, c.pmask, c.opages);
                if (row < 0) set_status(status, ZETA_ERR_BOUNDS);
                tile[l] = row < 0 ? K(0) : src_z[row];
                token[u] = row < 0 ? 0 : src_i[row];
            }
        }
        if (tid == 0 && i0 + cnt < M) {                    // the next tile's first code
            const int row = page_row(otab, i0 + cnt, h, H, c.psh, c.pmask, c.opages);
            tile[kTile] = row < 0 ? K(0) : src_z[row];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kTile / kThreads; ++u) {
            const int l = u * kThreads + tid;
            if (l < cnt) put(i0 + l + run.below(tile[l], C), tile[l], token[u]);
        }
        const int ja = t == 0 ? 0 : run.below(tile[0], C);
        const int jb = i0 + cnt < M ? run.below(tile[kTile], C) : C;
        for (int j = ja + tid; j < jb; j += kThreads) {
            const uint64_t z = run.code(j);
            int lo = 0, hi = cnt;                          // old entries of the tile with code <= z
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if ((uint64_t)tile[mid] <= z) lo = mid + 1; else hi = mid;
            }
            put(i0 + lo + j, z, M + run.place(j));
        }
        __syncthreads();
    }
}

template <typename K, bool PACK>
cudaError_t run_order(const Prob &p, const Cache &c, const float *k_pages, void *codes,
                      int32_t *idx, int32_t *status, cudaStream_t st) {
    static PerDeviceOnce once;
    constexpr size_t kMost = (size_t)8192 * 10 + (kTile + 1) * sizeof(K) + 16;
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(cache_order_kernel<K, PACK>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
    });
    if (e != cudaSuccess) return e;
    int C2 = 2;
    while (C2 < p.C) C2 <<= 1;
    const size_t smem = (size_t)C2 * (PACK ? 8 : 10) + (kTile + 1) * sizeof(K) + 16;
    // Blocks per slice: enough for four on each of the 152 SMs, at most one per tile.
    const int64_t tiles = (p.N + kTile - 1) / kTile;
    int64_t g = (152 * 4 + p.S - 1) / p.S;
    g = g < tiles ? g : tiles;
    const dim3 grid((unsigned)(g < 1 ? 1 : g), (unsigned)p.S);
    cache_order_kernel<K, PACK><<<grid, kThreads, smem, st>>>(
        c, k_pages, static_cast<K *>(codes), idx, status, p.N, p.H, p.dK, p.bits, p.C, C2);
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
