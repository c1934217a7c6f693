/*
 * zeta.h -- C ABI of the ZETA hot path on one GB300 (sm_103a).
 *
 * Method: "ZETA: Leveraging Z-order Curves for Efficient Top-k Attention"
 * (arXiv 2501.14577).  Queries and keys live in a low-dimensional space
 * (d_K = 3 by default), are quantised and bit-interleaved into one-dimensional
 * Z-order (Morton) codes, keys are sorted for every chunk-aligned causal prefix,
 * each query takes the k keys around its insertion rank in that order, and the
 * selected keys plus the query's own-chunk causal keys are combined with the
 * Adaptive Cauchy-softmax into a weighted sum of values.
 *
 * Conventions shared by every call
 *   - Every tensor is a contiguous row-major device array with the batch and
 *     head dimensions leading: [B, H, N, ...].  One (b, h) pair is a "slice";
 *     slices are independent except that the gamma gradient sums over b.
 *   - The caller owns and allocates every buffer, workspaces included (sizes
 *     come from the *_bytes / *_entries queries).  The library never allocates,
 *     never synchronises the stream and keeps no global state.
 *   - Work is enqueued on the given stream (0 = legacy default stream).  A
 *     returned ZETA_OK means the arguments were valid and the launches were
 *     enqueued; device-side findings are written to *dev_status when a status
 *     word is given (read it after synchronising).
 *   - Arguments are checked before anything is launched.  An empty problem
 *     (B*H*N == 0) is valid and launches nothing.
 *   - Code width: codes are uint32 when d_K*bits <= 32, else uint64.
 *   - Limits: 1 <= d_K <= 8, 1 <= bits <= 24, d_K*bits <= 64, C >= 1, C | N,
 *     1 <= k <= C, 1 <= d_V <= 256, N*k < 2^31, B*H <= 65535; zeta_sort_chunks
 *     also needs N / C <= 1024.
 */
#ifndef ZETA_H
#define ZETA_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ZETA_OK = 0,
    ZETA_ERR_INVALID_ARG = 1,     /* null pointer, bad size, C not dividing N, ...  */
    ZETA_ERR_UNSUPPORTED = 2,     /* valid request outside the implemented limits   */
    ZETA_ERR_WORKSPACE = 3,       /* workspace missing or smaller than required      */
    ZETA_ERR_CUDA = 4,            /* a launch failed (cudaGetLastError was not 0)    */
    ZETA_ERR_DEVICE_TIMEOUT = 5,  /* a bounded device wait gave up (status word)     */
    ZETA_ERR_BOUNDS = 6           /* an index outside its legal range (status word)  */
} zeta_status_t;

typedef enum { ZETA_F32 = 0, ZETA_BF16 = 1 } zeta_dtype_t;

/* Weight kernel of the attended set, in the low two bits of
 * zeta_problem_t.flags (d2 = |q_i - k_j|^2, a_ij = w_ij / s_i, s_i = sum_j w_ij):
 *   ZETA_W_CAUCHY      w = 1 / (1 + d2 / gamma^2): the method's Adaptive
 *                      Cauchy softmax (OpenReview reply A2 "Discussion on its
 *                      robustness").
 *   ZETA_W_SOFTMAX     w = exp(-(d2 - m_i) / gamma^2), m_i the smallest d2 of
 *                      query i's attended set: the usual softmax of
 *                      -d2 / gamma^2 ("negative Euclidean with traditional
 *                      softmax", reply A3 "Justification for Euclidean
 *                      Distance Claim"); rowsum_i is s_i with that shift.
 *   ZETA_W_INV_EUCLID  w = 1 / sqrt(d2 + 1e-12): inverse Euclidean distance
 *                      (same reply); gamma does not enter, dgamma is 0.
 * The squared distance inside the softmax and the 1e-12 guard are readings:
 * the pages name the kernels without formulas. */
typedef enum { ZETA_W_CAUCHY = 0, ZETA_W_SOFTMAX = 1, ZETA_W_INV_EUCLID = 2 } zeta_weight_t;

/* Problem statement: B batch, H heads, N tokens, d_K query/key width, d_V value
 * width, k window length, C chunk length, bits grid bits per coordinate,
 * v_dtype element type of v / out / dout / dv, flags: bits 0-1 the weight
 * kernel (zeta_weight_t), other bits reserved (pass 0).
 * These are the quantities the pages use to state the method: the 12-bit grid
 * and d_K = 3 (OpenReview reply A2 "Clarification of Binary Expansion and
 * Precision"), the chunk count and d_K = d_Q = 3 (reply A2 "Details about
 * experiments"), k and the trainable gamma (reply A2 "Discussion on its
 * robustness"). */
typedef struct {
    int32_t B, H, N, d_K, d_V, k, C, bits;
    int32_t v_dtype;
    uint32_t flags;
} zeta_problem_t;

/* Bytes per Z-order code (4 or 8); 0 when the problem is invalid. */
size_t zeta_code_bytes(const zeta_problem_t *p);

/* Entries T of the prefix table of one slice: C * n * (n - 1) / 2 with
 * n = N / C.  Prefix c (c = 1..n-1) occupies entries [C*c*(c-1)/2, +c*C).
 * Returns -1 when the problem is invalid. */
int64_t zeta_prefix_entries(const zeta_problem_t *p);

/* Workspace bytes needed by zeta_sort_chunks / zeta_attend_bwd (0 if invalid). */
size_t zeta_sort_workspace_bytes(const zeta_problem_t *p);
size_t zeta_bwd_workspace_bytes(const zeta_problem_t *p);

/* Human-readable name of a status code (static storage). */
const char *zeta_status_string(zeta_status_t s);

/*
 * zeta_encode -- Z-order code of every token.
 * Passage: OpenReview reply A2 "Clarification of Binary Expansion and
 * Precision" (normalise each coordinate to [0, 1], discretise to a grid of
 * 2^bits cells, interleave the bits of the d_K cell indices), and the reply on
 * dimension-ordering asymmetry (coordinate order K^1, K^2, K^3).
 * Reading: the normalisation is the fixed map [-1, 1) -> [0, 1); in float32,
 * t = (x + 1) * 2^(bits-1), u = min(max(floor(t), 0), 2^bits - 1) (NaN -> 0);
 * bit j of coordinate d goes to code bit j*d_K + (d_K - 1 - d).
 *   x      in : float  [B, H, N, d_K]
 *   codes  out: uint32 or uint64 (see zeta_code_bytes) [B, H, N]
 * Errors: ZETA_ERR_INVALID_ARG on null pointers or invalid sizes.
 */
zeta_status_t zeta_encode(const zeta_problem_t *p, const float *x, void *codes,
                          cudaStream_t stream);

/*
 * zeta_sort_chunks -- sorted key order of every chunk-aligned causal prefix.
 * Passage: OpenReview reply A3 "Chunking ... & Where efficiency is coming from"
 * (radix sort of the Z-order codes) and the atlas.scime.ai summary, "Approach"
 * (keys are sorted and split into chunks, so that all queries search their
 * causal past at the same time).
 * Prefix c holds the keys of chunks 0..c-1 ordered by (code, token index).
 *   key_codes     in : codes of the keys [B, H, N]
 *   prefix_codes  out: same code type [B, H, T]      (T = zeta_prefix_entries)
 *   prefix_idx    out: int32 token indices [B, H, T]
 *   workspace     scratch of at least zeta_sort_workspace_bytes, 256-B aligned
 * Errors: ZETA_ERR_INVALID_ARG, ZETA_ERR_UNSUPPORTED (N / C > 1024),
 *         ZETA_ERR_WORKSPACE (missing or too small).
 */
zeta_status_t zeta_sort_chunks(const zeta_problem_t *p, const void *key_codes,
                               void *prefix_codes, int32_t *prefix_idx,
                               void *workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * zeta_sort_chunks_noalloc -- zeta_sort_chunks without a workspace argument,
 * for callers that cannot allocate device memory when they need the sorted
 * prefixes (code running inside an allocator or memory-pool callback, plug-ins
 * whose host framework owns every device allocation, processes whose device
 * footprint must stay fixed after start-up).  The pages have no counterpart:
 * this is an interface convenience, not part of the method.
 * Scratch: one file-scope device array of 32 MiB, which every GPU that loads
 * this library holds until the process exits.
 * Checks, in order, before anything is launched: every check of
 * zeta_sort_chunks (the same errors; a problem with nothing to sort, empty or
 * with fewer than two chunks, returns ZETA_OK and touches no scratch), then
 * the scratch size: a problem whose zeta_sort_workspace_bytes exceeds 32 MiB
 * is rejected with ZETA_ERR_WORKSPACE.
 * Set-up: the first call on a device (with that device current) looks up the
 * array's device address with cudaGetSymbolAddress and caches it; make that
 * first call before any stream capture on that device.
 * Sharing: every call uses the same array, which keeps the previous call's
 * contents (nothing in it needs to start at zero).  Calls whose work overlaps
 * on the GPU (different streams, or different host threads on one device)
 * race on the array; order them on one stream.
 * Arguments and results are those of zeta_sort_chunks.
 * Allocates nothing: no cudaMalloc, cudaFree or allocating library routine.
 */
zeta_status_t zeta_sort_chunks_noalloc(const zeta_problem_t *p, const void *key_codes,
                                       void *prefix_codes, int32_t *prefix_idx,
                                       cudaStream_t stream);

/*
 * zeta_select_topk -- the k keys around each query's insertion rank.
 * Passage: OpenReview reply A3 (binary search of the insertion position) and
 * reply A2 "Clarification" (the window centred at the insertion position).
 * For query i in chunk c >= 1, with M = c*C: r = number of prefix-c keys whose
 * code is <= the query's code; start = min(max(r - ceil(k/2), 0), M - k); the
 * row is prefix_idx[prefix c][start .. start + k).  Chunk-0 rows are all -1.
 *   q_codes       in : codes of the queries [B, H, N]
 *   prefix_codes  in : from zeta_sort_chunks
 *   prefix_idx    in : from zeta_sort_chunks
 *   idx           out: int32 [B, H, N, k]
 * Errors: ZETA_ERR_INVALID_ARG.
 */
zeta_status_t zeta_select_topk(const zeta_problem_t *p, const void *q_codes,
                               const void *prefix_codes, const int32_t *prefix_idx,
                               int32_t *idx, cudaStream_t stream);

/*
 * zeta_encode_curves -- codes of every token along several Z-order curves.
 * Passage: OpenReview discussion, follow-up reply on interleaving the bits of
 * different dimensions (several curves)
 * (the key coordinates are interleaved in several orders: the three cyclic
 * shifts of (K^1, K^2, K^3), or all six orderings).
 * Curve m reads coordinate axes[m][s] into slot s, slot 0 being the most
 * significant bit of each level; with axes[m] = (0, 1, ..., d_K - 1) the code
 * is the one zeta_encode writes.  Quantisation as for zeta_encode.
 *   x       in : float [B, H, N, d_K]
 *   curves  in : 1..8
 *   axes    in : HOST int32 [curves][d_K], every row a permutation of 0..d_K-1
 *                (read during the call only)
 *   codes   out: code type of the problem [curves][B, H, N]
 * Errors: ZETA_ERR_INVALID_ARG (null pointers, curves out of range, a row of
 *         axes that is not a permutation).
 */
zeta_status_t zeta_encode_curves(const zeta_problem_t *p, const float *x, int32_t curves,
                                 const int32_t *axes, void *codes, cudaStream_t stream);

/*
 * zeta_select_topk_curves -- the union of one window per curve.
 * Passage: OpenReview discussion, follow-up reply on interleaving the bits of
 * different dimensions (several curves)
 * (every curve collects k // curves of the k tokens).
 * Reading of the union: with km = k // curves, curve m gives the km keys that
 * zeta_select_topk would give with km in place of k (its own prefix table);
 * the windows are listed in curve order, a key already listed is dropped, and
 * the row is padded to k with -1.  Chunk-0 rows are all -1.
 *   q_codes       in : [curves][B, H, N]  (zeta_encode_curves)
 *   prefix_codes  in : [curves][B, H, T]  (curve m's key codes sorted by
 *   prefix_idx    in : [curves][B, H, T]   zeta_sort_chunks; one call on the
 *                      problem with B replaced by curves*B sorts every curve,
 *                      as the two layouts coincide)
 *   idx           out: int32 [B, H, N, k], for zeta_attend_fwd / _bwd
 * Limits: 1 <= curves <= 8, k // curves >= 1, k <= 256.
 * Errors: ZETA_ERR_INVALID_ARG, ZETA_ERR_UNSUPPORTED (k > 256).
 */
zeta_status_t zeta_select_topk_curves(const zeta_problem_t *p, int32_t curves,
                                      const void *q_codes, const void *prefix_codes,
                                      const int32_t *prefix_idx, int32_t *idx,
                                      cudaStream_t stream);

/* Widths of the projection front end: D input features per token, F hidden
 * units per head. */
typedef struct {
    int32_t D, F;
} zeta_proj_t;

/*
 * zeta_project_encode -- queries and keys from token features, with their codes.
 * Passage: OpenReview reply A "LLMs impact the selection of d_K" (a two-layer
 * neural network projects the input into the keys) and reply A2
 * "Clarification of Binary Expansion and Precision" (the codes).
 * Reading: per head hd, and separately for queries (projection 0) and keys
 * (projection 1):
 *   h_f = max(0, W1[hd*F + f] . x_t + b1[hd*F + f]),  y_c = tanh(W2[hd][c] . h + b2[hd][c])
 * (tanh puts the coordinates in (-1, 1), the quantiser's range); y is written
 * out and encoded exactly as zeta_encode would encode it.
 *   x        in : bf16 [B, N, D]           (16-B aligned)
 *   w1       in : bf16 [2, H*F, D]         (16-B aligned; rows are hidden units)
 *   b1       in : float [2, H*F]
 *   w2       in : float [2, H, d_K, F]
 *   b2       in : float [2, H, d_K]
 *   q, k     out: float [B, H, N, d_K]
 *   q_codes, k_codes  out: code type of the problem [B, H, N]
 *   dev_status  optional int32 device word (ZETA_ERR_DEVICE_TIMEOUT if a
 *               bounded wait of the kernel gave up)
 * Limits: F = 64, D a multiple of 64, H = 4 or 8, d_K <= 4, B*N < 2^31.
 * The first layer runs on the tensor cores with bf16 inputs and float32
 * accumulation; the rest in float32.
 * Errors: ZETA_ERR_INVALID_ARG, ZETA_ERR_UNSUPPORTED (outside the limits).
 */
zeta_status_t zeta_project_encode(const zeta_problem_t *p, const zeta_proj_t *pj,
                                  const void *x, const void *w1, const float *b1,
                                  const float *w2, const float *b2, float *q, float *k,
                                  void *q_codes, void *k_codes, int32_t *dev_status,
                                  cudaStream_t stream);

/*
 * zeta_attend_fwd -- Adaptive Cauchy-softmax over the selected keys.
 * Passage: OpenReview reply A2 "Discussion on its robustness" (trainable gamma,
 * Cauchy softmax), reply A3 "Justification for Euclidean Distance Claim", and
 * the atlas.scime.ai summary, "Approach".
 * The attended set of query i in chunk c is its window (non-negative entries
 * of idx row i) plus every key j of its own chunk with cC <= j <= i.  With
 * w_ij = 1 / (1 + |q_i - k_j|^2 / gamma_h^2) (or the kernel that flags
 * selects, see zeta_weight_t) and s_i = sum_j w_ij:
 * out_i = sum_j w_ij v_j / s_i, rowsum_i = s_i.
 *   q, k    in : float [B, H, N, d_K]
 *   v       in : v_dtype [B, H, N, d_V]  (16-B aligned; the tensor-core kernel
 *                (bf16, d_V = 64, d_K <= 4) reads value rows 32 bytes at a time
 *                and runs only where v is 32-B aligned, the general kernel
 *                otherwise)
 *   gamma   in : float [H]
 *   idx     in : int32 [B, H, N, k]; entries must be -1 or in [0, cC)
 *   out     out: v_dtype [B, H, N, d_V]  (16-B aligned)
 *   rowsum  out: float [B, H, N]
 *   dev_status  optional int32 device word; an idx entry outside its range is
 *               skipped and ZETA_ERR_BOUNDS is recorded there.
 * Errors: ZETA_ERR_INVALID_ARG, ZETA_ERR_UNSUPPORTED.
 */
zeta_status_t zeta_attend_fwd(const zeta_problem_t *p, const float *q, const float *k,
                              const void *v, const float *gamma, const int32_t *idx,
                              void *out, float *rowsum, int32_t *dev_status,
                              cudaStream_t stream);

/*
 * zeta_select_attend_fwd -- zeta_select_topk and zeta_attend_fwd in one call.
 * Passage: as for those two calls (OpenReview reply A3 "Chunking ... & Where
 * efficiency is coming from": binary search of the insertion position; the
 * attended set and weights of zeta_attend_fwd).
 * On the tensor-core shapes (bf16 values, d_V = 64, d_K <= 4, v 32-B aligned)
 * one kernel finds each query's window by binary search in its sorted prefix,
 * reads the window as a contiguous run of prefix_idx, attends, and writes the
 * run to idx for zeta_attend_bwd; otherwise the two calls run one after the
 * other.
 * Results are those of zeta_select_topk followed by zeta_attend_fwd.
 *   q, k, v, gamma   in : as for zeta_attend_fwd
 *   q_codes          in : codes of the queries [B, H, N]
 *   prefix_codes, prefix_idx  in : from zeta_sort_chunks
 *   idx              out: int32 [B, H, N, k] (as zeta_select_topk writes it)
 *   out, rowsum      out: as for zeta_attend_fwd
 *   dev_status       optional int32 device word (as for zeta_attend_fwd)
 * Errors: ZETA_ERR_INVALID_ARG, ZETA_ERR_UNSUPPORTED.
 */
zeta_status_t zeta_select_attend_fwd(const zeta_problem_t *p, const float *q, const float *k,
                                     const void *v, const float *gamma, const void *q_codes,
                                     const void *prefix_codes, const int32_t *prefix_idx,
                                     int32_t *idx, void *out, float *rowsum,
                                     int32_t *dev_status, cudaStream_t stream);

/*
 * zeta_attend_bwd -- gradients through the weights, selection fixed.
 * Passage: the forward/backward timings of the OpenReview replies A3/A4 (the
 * method is trained end to end) and the forward definition above.
 * With a_ij = w_ij / s_i, g_ij = dO_i . v_j and gbar_i = sum_j a_ij g_ij
 * (= dO_i . out_i for the exact output):
 *   dL/dw_ij = (g_ij - gbar_i) / s_i
 *   dq_i     = sum_j dL/dw_ij * 2 (dw/dd2)_ij (q_i - k_j)
 *   dk_j     = -sum_i dL/dw_ij * 2 (dw/dd2)_ij (q_i - k_j)
 *   dv_j     = sum_i a_ij dO_i
 *   dgamma_h = sum_{b,i,j} dL/dw_ij * (dw/dgamma)_ij
 * with, per weight kernel, dw/dd2 = -w^2/gamma^2 and dw/dgamma =
 * 2 w (1 - w) / gamma (Cauchy); -w/gamma^2 and 2 w (d2 - m_i) / gamma^3
 * (softmax); -w^3/2 and 0 (inverse Euclidean).
 * s_i and gbar_i are recomputed from q, k, v and idx (one pass over each
 * query's set), so the forward's rounded output is not needed.
 *   q, k, v, gamma, idx  in : as for zeta_attend_fwd
 *   dout         in : v_dtype [B, H, N, d_V]  (16-B aligned)
 *   dq, dk       out: float [B, H, N, d_K]
 *   dv           out: v_dtype [B, H, N, d_V]  (16-B aligned)
 *   dgamma       out: float [H]
 *   workspace    scratch of at least zeta_bwd_workspace_bytes, 256-B aligned
 *   dev_status   optional int32 device word (ZETA_ERR_BOUNDS as for the forward;
 *                ZETA_ERR_DEVICE_TIMEOUT if a bounded wait of the tensor-core
 *                own-chunk kernel gave up)
 * Every output is overwritten.  Reductions run in a fixed order, so results
 * are bit-reproducible run to run.
 * Errors: ZETA_ERR_INVALID_ARG, ZETA_ERR_UNSUPPORTED, ZETA_ERR_WORKSPACE.
 */
zeta_status_t zeta_attend_bwd(const zeta_problem_t *p, const float *q, const float *k,
                              const void *v, const float *gamma, const int32_t *idx,
                              const void *dout, float *dq, float *dk, void *dv, float *dgamma,
                              void *workspace, size_t ws_bytes, int32_t *dev_status,
                              cudaStream_t stream);

/*
 * Paged cache: serving a trained model.
 *
 * The calls above take whole sequences.  The three calls below hold the keys and
 * values of many sequences in fixed-size pages and take, per call, a batch of up
 * to n <= C new tokens per sequence (n = 1: one token each).  A prompt read in
 * pieces and the tokens that follow it get the outputs that zeta_attend_fwd
 * computes for the whole sequence: the same codes, prefixes, windows and weights.
 * The cache holds the order along one curve, that of zeta_encode: selections over
 * several curves (zeta_encode_curves) have no cached form.
 *
 *   p     B sequences in this call, H, d_K, d_V, k, C, bits, v_dtype, flags as
 *         everywhere; N is the longest sequence the cache holds (C | N).
 *   cc    n: rows of new tokens per sequence in q, k, v, out (1 <= n <= C);
 *         page: tokens per page, a power of two up to 65536;
 *         pages, order_pages: pages in the pools (at least one each; append does
 *         not look at order_pages); table_len: row length of the page tables,
 *         table_len * page >= N.
 *   start, count   int32 [B] (device): tokens sequence b held before this call
 *         and tokens it brings (0 <= count <= n, start + count <= N).  Rows
 *         count[b] .. n-1 are padding: nothing depends on what they hold, and
 *         they are left as they were where they are outputs.  A sequence outside these ranges is skipped whole and
 *         ZETA_ERR_BOUNDS recorded.
 *   page_table     int32 [B, table_len]: token t of sequence b is row t % page of
 *         page page_table[b][t / page].  Only entries of tokens that exist are
 *         looked at; one outside [0, pages) skips its tokens (ZETA_ERR_BOUNDS).
 *   k_pages        float [pages, H, page, d_K]
 *   v_pages        v_dtype [pages, H, page, d_V]  (16-B aligned)
 *   order_codes    code type [2, order_pages, H, page]  (16-B aligned)
 *   order_idx      int32 [2, order_pages, H, page]  (16-B aligned)
 *   order_table    int32 [B, table_len]: entry e of prefix c of sequence b is row
 *         e % page of page order_table[b][e / page] in plane c % 2.  It may be
 *         page_table itself.  Sequences may share K/V pages (a common prompt), but
 *         a page of the order pools belongs to one sequence.
 *
 * One step: zeta_cache_append, zeta_cache_order (needed in the calls in which
 * some sequence completes a chunk, a no-op for the others), zeta_cache_attend,
 * on one stream, with the same n, start and count (another n would let one call
 * take a sequence that another one skips).  As n <= C a call completes at
 * most one chunk per sequence, and the two planes hold the prefixes of both
 * chunks that its tokens lie in.
 *
 * Limits beside those above: C <= 8192, pages * H * page < 2^31 (order_pages
 * likewise).  No call needs a workspace; calls on different
 * sequences may overlap on different streams.  The calls have no backward.
 */
typedef struct {
    int32_t n, page, pages, order_pages, table_len;
} zeta_cache_t;

/*
 * zeta_cache_append -- keys and values of new tokens into their pages.
 *   k         in : float [B, H, n, d_K]
 *   v         in : v_dtype [B, H, n, d_V]  (16-B aligned)
 *   k_pages, v_pages  in/out (written at the new tokens' rows only)
 *   dev_status  optional int32 device word (ZETA_ERR_BOUNDS as above)
 * Two new tokens of one call that map to the same row (a page given to two
 * sequences) leave one of them there, which one is not defined.
 * Errors: ZETA_ERR_INVALID_ARG, ZETA_ERR_UNSUPPORTED.
 */
zeta_status_t zeta_cache_append(const zeta_problem_t *p, const zeta_cache_t *cc, const float *k,
                                const void *v, const int32_t *start, const int32_t *count,
                                const int32_t *page_table, float *k_pages, void *v_pages,
                                int32_t *dev_status, cudaStream_t stream);

/*
 * zeta_cache_order -- the sorted prefix of every sequence that completes a chunk.
 * Passage: as for zeta_sort_chunks (OpenReview reply A3 "Chunking ... & Where
 * efficiency is coming from").
 * If floor((start + count) / C) > floor(start / C), with c the chunk completed,
 * prefix c + 1 (the (c + 1) C keys of chunks 0..c ordered by (code, token)) is
 * written to plane (c + 1) % 2 from prefix c in plane c % 2 and the keys of chunk
 * c, whose codes are those of zeta_encode.  Other sequences are left alone.
 *   k_pages   in : after zeta_cache_append
 *   order_codes, order_idx  in/out
 *   dev_status  optional int32 device word: a page out of range skips the
 *               sequence's head (nothing of its new prefix is defined then).
 * Errors: ZETA_ERR_INVALID_ARG, ZETA_ERR_UNSUPPORTED.
 */
zeta_status_t zeta_cache_order(const zeta_problem_t *p, const zeta_cache_t *cc,
                               const int32_t *start, const int32_t *count,
                               const int32_t *page_table, const float *k_pages,
                               const int32_t *order_table, void *order_codes, int32_t *order_idx,
                               int32_t *dev_status, cudaStream_t stream);

/*
 * zeta_cache_attend -- attention of the new tokens over the cache.
 * Passage: as for zeta_select_topk and zeta_attend_fwd.
 * The token at position i = start[b] + t, in chunk c = i / C, attends to the k
 * keys around its code's rank in prefix c (none for c = 0) and to the keys of
 * its own chunk up to itself; weights, out and rowsum as in zeta_attend_fwd.
 * Weights and sums are float32.  For bf16 values large calls run products on the
 * tensor cores, which take a weight as two bf16 parts, within 2^-16 of it; out is
 * rounded once.  The same token in calls of different sizes so has the same rowsum
 * to float32 roundings and the same out to one step of its type.
 *   q         in : float [B, H, n, d_K]
 *   gamma     in : float [H]
 *   k_pages, v_pages, order_codes, order_idx  in : after append and order
 *   out       out: v_dtype [B, H, n, d_V]  (16-B aligned)
 *   rowsum    out: float [B, H, n]
 *   idx       out: int32 [B, H, n, k], the window's tokens (-1 in chunk 0), or
 *             null
 *   dev_status  optional int32 device word; an order entry outside [0, cC) or a
 *             page out of range drops its key and records ZETA_ERR_BOUNDS (a row
 *             that loses all of them: rowsum 0, out NaN).
 * Errors: ZETA_ERR_INVALID_ARG, ZETA_ERR_UNSUPPORTED.
 */
zeta_status_t zeta_cache_attend(const zeta_problem_t *p, const zeta_cache_t *cc, const float *q,
                                const float *gamma, const int32_t *start, const int32_t *count,
                                const int32_t *page_table, const float *k_pages,
                                const void *v_pages, const int32_t *order_table,
                                const void *order_codes, const int32_t *order_idx, void *out,
                                float *rowsum, int32_t *idx, int32_t *dev_status,
                                cudaStream_t stream);

/*
 * Drafting: a tree of guessed tokens per sequence and step.
 *
 * Sequence b holds start[b] tokens and brings count[b] <= n drafted ones, the nodes of a
 * tree: node t hangs below node parent[b][t] < t, or below the sequence's last token
 * (parent -1); its depth is that of its parent plus one, 0 at the top, and its position
 * start[b] + depth.  Keys and values of the nodes stay in the step's own tensors.  One
 * step, on one stream:
 *   zeta_cache_reserve      with count = min(tokens of the longest line that may be
 *                           accepted, C - start % C): its pages;
 *   zeta_cache_attend_tree  every node over the cache and its own line (each layer's
 *                           cache; several nodes may be tried in one call);
 *   (the program decides which node's line is right)
 *   zeta_cache_accept_granted  that line becomes the sequence's next tokens (each layer's
 *                           cache), none where reserve had no pages for them;
 *   zeta_cache_order        with count = accepted, as after zeta_cache_append.
 * A line ends with the chunk that start lies in (C): attend_tree gives nodes behind that
 * end no result and accept cuts the line there, so that a step's nodes share one sorted
 * prefix.  A step that has a page can always accept a token: a chunk that is full begins
 * the next.
 *   parent   int32 [B, n] (device): entries count[b] .. n-1 are not looked at; an entry
 *            outside [-1, t) costs the lines through it (ZETA_ERR_BOUNDS).
 *   start, count  as for the cache calls, but 0 <= start <= N and, where count > 0,
 *            start < N: only the line's tokens need room.
 * Limit: n <= 1024.
 * No output of these calls may share memory with an input or another output, the pools aside
 * (ZETA_ERR_INVALID_ARG); zeta_cache_reserve's granted may be the array given as count.
 */

/*
 * zeta_cache_attend_tree -- attention of the nodes over the cache.
 * Passage: as for zeta_select_topk and zeta_attend_fwd.
 * Node t of sequence b, with position i < (c + 1) C, c = start[b] / C, attends to the k
 * keys around its code's rank in prefix c (none for c = 0), to the tokens cC .. start[b]-1
 * and to the nodes of its line, itself included; weights, out and rowsum as in
 * zeta_attend_fwd.  That is what zeta_cache_attend gives for the same tokens in a line.
 * Weights and sums are float32 in calls of every size (a weight on the tensor cores: three
 * bf16 parts that hold its 24 bits); out is rounded once.
 *   q, k      in : float [B, H, n, d_K]: the nodes' queries and keys
 *   v         in : v_dtype [B, H, n, d_V]  (16-B aligned)
 *   gamma     in : float [H]
 *   k_pages, v_pages, order_codes, order_idx  in : the cache before this step
 *   out       out: v_dtype [B, H, n, d_V]  (16-B aligned)
 *   rowsum    out: float [B, H, n]
 *   idx       out: int32 [B, H, n, k], the window's tokens (-1 in chunk 0), or null
 *   dev_status  optional int32 device word; an order entry outside [0, cC) or a page
 *             out of range drops its key and records ZETA_ERR_BOUNDS.
 * Rows of nodes behind the chunk's end, of nodes whose line has a bad parent and from
 * count[b] on are left as they were.
 * Errors: ZETA_ERR_INVALID_ARG, ZETA_ERR_UNSUPPORTED.
 */
zeta_status_t zeta_cache_attend_tree(const zeta_problem_t *p, const zeta_cache_t *cc,
                                     const float *q, const float *k, const void *v,
                                     const float *gamma, const int32_t *start,
                                     const int32_t *count, const int32_t *parent,
                                     const int32_t *page_table, const float *k_pages,
                                     const void *v_pages, const int32_t *order_table,
                                     const void *order_codes, const int32_t *order_idx, void *out,
                                     float *rowsum, int32_t *idx, int32_t *dev_status,
                                     cudaStream_t stream);

/*
 * zeta_cache_accept -- a line of nodes into the pages.
 * The pages have no counterpart: it is zeta_cache_append along a line.
 * Keys and values of the line that ends in node leaf[b], as far as it lies before the
 * chunk's end, become the tokens start[b] .. start[b] + accepted[b] - 1.
 *   k, v      in : the tensors given to zeta_cache_attend_tree (v 16-B aligned)
 *   leaf      in : int32 [B], -1: nothing is accepted; not looked at where count is 0
 *   k_pages, v_pages  in/out (written at the accepted tokens' rows only)
 *   accepted  out: int32 [B], tokens accepted: the count for zeta_cache_order.  Every token
 *             of the line counts, one without a page too: where pages may be missing call
 *             zeta_cache_accept_granted
 *   path      out: int32 [B, n], node of the j-th accepted token, -1 from accepted[b] on;
 *             or null
 *   dev_status  optional int32 device word (ZETA_ERR_BOUNDS: a leaf outside
 *             [-1, count), a line with a bad parent or a sequence out of range accepts
 *             nothing; a page out of range skips its token's row)
 * Two sequences whose accepted tokens map to the same row leave one of them there, as in
 * zeta_cache_append.
 * Errors: ZETA_ERR_INVALID_ARG, ZETA_ERR_UNSUPPORTED.
 */
zeta_status_t zeta_cache_accept(const zeta_problem_t *p, const zeta_cache_t *cc, const float *k,
                                const void *v, const int32_t *start, const int32_t *count,
                                const int32_t *parent, const int32_t *leaf,
                                const int32_t *page_table, float *k_pages, void *v_pages,
                                int32_t *accepted, int32_t *path, int32_t *dev_status,
                                cudaStream_t stream);

/*
 * zeta_cache_accept_granted -- zeta_cache_accept of no more tokens than were granted.
 * The pages have no counterpart: as for zeta_cache_accept.
 * The line ends after granted[b] tokens where it has more, so that with zeta_cache_reserve's
 * granted every token accepted has a page.
 *   granted   in : int32 [B] (negative as 0); all else as for zeta_cache_accept
 * Errors: ZETA_ERR_INVALID_ARG, ZETA_ERR_UNSUPPORTED.
 */
zeta_status_t zeta_cache_accept_granted(const zeta_problem_t *p, const zeta_cache_t *cc,
                                        const float *k, const void *v, const int32_t *start,
                                        const int32_t *count, const int32_t *parent,
                                        const int32_t *leaf, const int32_t *granted,
                                        const int32_t *page_table, float *k_pages, void *v_pages,
                                        int32_t *accepted, int32_t *path, int32_t *dev_status,
                                        cudaStream_t stream);

/*
 * zeta_cache_reserve -- page tables and row numbers from the requests' lengths.
 * The pages have no counterpart.
 * After the call sequence b holds ceil((start[b] + count[b]) / page) pages, entries
 * [0, held[b]) of its table.  First every sequence that holds more gives its last pages
 * back to the list (a request that has ended: start = count = 0), their entries become -1;
 * then the others take theirs in the order of b, from the list's end.  From the first
 * sequence on that the list is too short for, sequences that need pages get none and stay
 * as they were: granted[b] = 0.  All others: granted[b] = count[b].  Given granted as
 * their count, zeta_cache_append, _order and _attend take what has pages; of a draft, whose
 * count is one of nodes, zeta_cache_accept_granted does.
 *   p, cc     B, N, C as everywhere, n, page, pages, table_len of the cache (the heads and
 *             the order pools play no part); n bounds count: 0 where the call only gives back
 *   start, count  int32 [B], 0 <= count <= n, 0 <= start, start + count <= N (of a draft the
 *               tokens of its longest line up to the chunk's end: there is always room for them)
 *   page_table  in/out: int32 [B, table_len]
 *   held        in/out: int32 [B], pages that sequence b holds
 *   free_list   in/out: int32 [pages], places [0, *free_count) are the free pages
 *   free_count  in/out: int32 [1]
 *   granted     out: int32 [B]
 *   slots       out: int32 [B, n], row page_table[b][i / page] * page + i % page of the new
 *               token i = start[b] + t, for data that a program keeps in the same pages; -1
 *               from granted[b] on; or null
 *   dev_status  optional int32 device word (ZETA_ERR_BOUNDS: a length or held out of
 *               range, the sequence is skipped, granted 0; a list longer than the pools
 *               have pages, nothing changes; a page number out of range, it is passed on)
 * The result depends on the order of the sequences alone, and a call that takes pages is
 * undone by one that gives them back.  Calls on one list follow one another on a stream.
 * A page is in one table or in the list: a table whose entries below held were filled in
 * otherwise (shared prompts) gives them back as if they were its own.
 * Errors: ZETA_ERR_INVALID_ARG, ZETA_ERR_UNSUPPORTED.
 */
zeta_status_t zeta_cache_reserve(const zeta_problem_t *p, const zeta_cache_t *cc,
                                 const int32_t *start, const int32_t *count, int32_t *page_table,
                                 int32_t *held, int32_t *free_list, int32_t *free_count,
                                 int32_t *granted, int32_t *slots, int32_t *dev_status,
                                 cudaStream_t stream);

/*
 * zeta_check_bounded_wait -- diagnostic of the device-side failure detection.
 * The pages have no counterpart: every wait of the TMA-fed and tensor-core
 * kernels (zeta_project_encode, the own-chunk block of zeta_attend_bwd) on an
 * mbarrier polls a bounded number of times
 * and, when it gives up, records ZETA_ERR_DEVICE_TIMEOUT in the status word and
 * lets the kernel return.  This call runs that wait on one barrier, completed
 * beforehand when arrive != 0 and never completed otherwise, polling at most
 * `iterations` times.
 *   dev_status  int32 device word (required); ZETA_ERR_DEVICE_TIMEOUT is written
 *               there when the wait gave up, nothing otherwise.
 * Errors: ZETA_ERR_INVALID_ARG (null dev_status, zero iterations).
 */
zeta_status_t zeta_check_bounded_wait(uint32_t iterations, int32_t arrive, int32_t *dev_status,
                                      cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ZETA_H */
