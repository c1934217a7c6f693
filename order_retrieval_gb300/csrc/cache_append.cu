// cache_append.cu -- keys and values of new tokens into their pages.
//
// A copy of count[b] rows of d_K floats and d_V values per (b, h): nothing is
// computed, the pages decide where a row goes.  A value row is cut into 16-byte
// pieces, one thread each (single values where the row is no multiple of 16
// bytes); the row's first threads also carry its d_K coordinates.  The rows of
// all slices are one list, so a batch of single tokens fills its blocks as well
// as a long piece does.  A block takes whole rows, so that the row a thread works
// for needs divisions of 32 bits only.
//
// 9,900 tokens in 16 sequences, 8 heads, 12 bytes a key and 128 a value: 7.7 us for
// 22 MB, 2.9 TB/s (8.0 us with the pieces of all rows as one list and a division of
// 64 bits).  What bounds it is finding the row: four pieces a thread, loads ahead of
// stores, took 10 us, for that arithmetic then has fewer warps to hide in.
#include "cache.cuh"

namespace zeta {
namespace {

constexpr int kThreads = 256;

template <typename Piece>
__global__ void __launch_bounds__(kThreads)
cache_append_kernel(const float *__restrict__ k, const Piece *__restrict__ v,
                    float *__restrict__ k_pages, Piece *__restrict__ v_pages, Cache c,
                    int32_t *status, unsigned rows, int N, int H, int dK, int ppr, int rpb) {
    const unsigned in = threadIdx.x / (unsigned)ppr;             // row of the block
    const int ch = (int)(threadIdx.x - in * (unsigned)ppr);
    const uint64_t r64 = (uint64_t)blockIdx.x * (unsigned)rpb + in;
    if (in >= (unsigned)rpb || r64 >= rows) return;
    const unsigned r = (unsigned)r64;
    const unsigned s = r / (unsigned)c.n;
    const int t = (int)(r - s * (unsigned)c.n);
    const int b = (int)(s / (unsigned)H), h = (int)(s - (unsigned)b * (unsigned)H);
    const Seq q = seq_of(c, b, N, status);
    if (t >= q.count) return;
    const int row = page_row(c.ptab + (int64_t)b * c.tlen, q.start + t, h, H, c.psh, c.pmask,
                             c.pages);
    if (row < 0) {
        set_status(status, ZETA_ERR_BOUNDS);
        return;
    }
    v_pages[(int64_t)row * ppr + ch] = v[(int64_t)r * ppr + ch];
    for (int d = ch; d < dK; d += ppr) k_pages[(int64_t)row * dK + d] = k[(int64_t)r * dK + d];
}

}  // namespace

cudaError_t launch_cache_append(const Prob &p, const Cache &c, const float *k, const void *v,
                                float *k_pages, void *v_pages, int32_t *status, cudaStream_t st) {
    const int esz = p.vdt == ZETA_BF16 ? 2 : 4;
    const int bytes = p.dV * esz;
    const unsigned rows = (unsigned)(p.S * c.n);
#define ZETA_APPEND(Piece)                                                                     \
    do {                                                                                       \
        const int ppr = bytes / (int)sizeof(Piece);                                            \
        const int rpb = kThreads / ppr;      /* at most 256 pieces a row: at least one */      \
        cache_append_kernel<Piece><<<(rows + rpb - 1) / rpb, kThreads, 0, st>>>(               \
            k, static_cast<const Piece *>(v), k_pages, static_cast<Piece *>(v_pages), c,       \
            status, rows, p.N, p.H, p.dK, ppr, rpb);                                           \
    } while (0)
    if (bytes % 16 == 0) ZETA_APPEND(uint4);
    else if (esz == 4) ZETA_APPEND(uint32_t);
    else ZETA_APPEND(uint16_t);
#undef ZETA_APPEND
    return cudaGetLastError();
}

}  // namespace zeta
