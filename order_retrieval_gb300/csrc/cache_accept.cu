// cache_accept.cu -- the accepted branch of a draft into the pages.
//
// The line of nodes that ends in leaf[b], up to the end of the chunk that start lies in,
// becomes the sequence's next tokens: a copy of rows, as cache_append.cu, through the
// line.  A block per sequence and head finds the line in the parents in shared memory
// and copies its rows, a thread per 16-byte piece of a value row (a value where the row
// is no multiple of 16 bytes); the row's first threads also carry its coordinates.
#include "cache_tree.cuh"

namespace zeta {
namespace {

constexpr int kThreads = 256;

template <typename Piece>
__global__ void __launch_bounds__(kThreads)
cache_accept_kernel(const float *__restrict__ k, const Piece *__restrict__ v,
                    float *__restrict__ k_pages, Piece *__restrict__ v_pages, Cache c,
                    const int32_t *__restrict__ parents, const int32_t *__restrict__ leaves,
                    int32_t *__restrict__ accepted, int32_t *__restrict__ path, int32_t *status,
                    int N, int H, int C, int dK, int ppr) {
    __shared__ int parent[kMaxDraft], line[kMaxDraft];
    __shared__ int len_sh;
    const int tid = threadIdx.x, h = blockIdx.x, b = blockIdx.y;
    const Seq seq = drafts_of(c, b, N, status);
    int leaf = __ldg(leaves + b);
    if (leaf < -1 || leaf >= seq.count) {
        if (tid == 0 && seq.count > 0) set_status(status, ZETA_ERR_BOUNDS);
        leaf = -1;
    }
    for (int u = tid; u <= leaf; u += kThreads) parent[u] = __ldg(parents + (int64_t)b * c.n + u);
    __syncthreads();
    if (tid == 0) {
        int at = kMaxDraft;                          // the line, up against the array's end
        const int depth = climb(parent, leaf, [&](int u) { line[--at] = u; });
        if (leaf >= 0 && depth < 0) set_status(status, ZETA_ERR_BOUNDS);
        len_sh = depth + 1;
    }
    __syncthreads();
    const int *from = line + kMaxDraft - len_sh;
    const int len = min(len_sh, C - seq.start % C);  // no line: 0
    if (h == 0) {
        if (tid == 0) accepted[b] = len;
        if (path)
            for (int d = tid; d < c.n; d += kThreads) path[(int64_t)b * c.n + d] = d < len ? from[d] : -1;
    }
    const int32_t *ptab = c.ptab + (int64_t)b * c.tlen;
    const int64_t rows = ((int64_t)b * H + h) * c.n;
    const int in = tid / ppr, ch = tid - in * ppr, rpb = kThreads / ppr;
    if (in >= rpb) return;
    for (int d = in; d < len; d += rpb) {
        const int row = page_row(ptab, seq.start + d, h, H, c.psh, c.pmask, c.pages);
        if (row < 0) {
            set_status(status, ZETA_ERR_BOUNDS);
            continue;
        }
        const int64_t r = rows + from[d];
        v_pages[(int64_t)row * ppr + ch] = v[r * ppr + ch];
        for (int e = ch; e < dK; e += ppr) k_pages[(int64_t)row * dK + e] = k[r * dK + e];
    }
}

}  // namespace

cudaError_t launch_cache_accept(const Prob &p, const Cache &c, const int32_t *parent,
                                const int32_t *leaf, const float *k, const void *v, float *k_pages,
                                void *v_pages, int32_t *accepted, int32_t *path, int32_t *status,
                                cudaStream_t st) {
    const int esz = p.vdt == ZETA_BF16 ? 2 : 4;
    const int bytes = p.dV * esz;
#define ZETA_ACCEPT(Piece)                                                                     \
    cache_accept_kernel<Piece><<<dim3((unsigned)p.H, (unsigned)p.B), kThreads, 0, st>>>(       \
        k, static_cast<const Piece *>(v), k_pages, static_cast<Piece *>(v_pages), c, parent,   \
        leaf, accepted, path, status, p.N, p.H, p.C, p.dK, bytes / (int)sizeof(Piece))
    if (bytes % 16 == 0) ZETA_ACCEPT(uint4);
    else if (esz == 4) ZETA_ACCEPT(uint32_t);
    else ZETA_ACCEPT(uint16_t);
#undef ZETA_ACCEPT
    return cudaGetLastError();
}

}  // namespace zeta
