// cache_append.cu -- keys and values of new tokens into their pages.
//
// A copy of count[b] rows of d_K floats and d_V values per (b, h): nothing is
// computed, the pages decide where a row goes.  A value row is cut into 16-byte
// pieces, one thread each (single values where the row is no multiple of 16
// bytes); the row's first threads also carry its d_K coordinates.  The rows of
// all slices are one list, so a batch of single tokens fills its blocks as well
// as a long piece does.
#include "cache.cuh"

namespace zeta {
namespace {

constexpr int kThreads = 256;

template <typename Piece>
__global__ void __launch_bounds__(kThreads)
cache_append_kernel(const float *__restrict__ k, const Piece *__restrict__ v,
                    float *__restrict__ k_pages, Piece *__restrict__ v_pages, Cache c,
                    int32_t *status, unsigned rows, int N, int H, int dK, int ppr) {
    const uint64_t id = blockIdx.x * (uint64_t)kThreads + threadIdx.x;
    const uint64_t r64 = id / (unsigned)ppr;
    if (r64 >= rows) return;
    const unsigned r = (unsigned)r64;
    const int ch = (int)(id - r64 * (unsigned)ppr);
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
        const uint64_t blocks = ((uint64_t)rows * ppr + kThreads - 1) / kThreads;              \
        if (blocks > 0x7fffffffull) return cudaErrorInvalidConfiguration;                      \
        cache_append_kernel<Piece><<<(unsigned)blocks, kThreads, 0, st>>>(                     \
            k, static_cast<const Piece *>(v), k_pages, static_cast<Piece *>(v_pages), c,       \
            status, rows, p.N, p.H, p.dK, ppr);                                                \
    } while (0)
    if (bytes % 16 == 0) ZETA_APPEND(uint4);
    else if (esz == 4) ZETA_APPEND(uint32_t);
    else ZETA_APPEND(uint16_t);
#undef ZETA_APPEND
    return cudaGetLastError();
}

}  // namespace zeta
