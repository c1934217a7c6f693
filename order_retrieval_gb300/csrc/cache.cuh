// cache.cuh -- the paged key/value cache of the serving calls: the validated
// view of a call, page addressing and what the three kernels share.
//
// Token t of sequence b lives in row t % page of page table[b][t / page]; the
// pools are [pages, H, page, width], so one head's rows of a page are contiguous
// and a row number (page id * H + h) * page + t % page fits 31 bits (checked on
// the host).  Byte offsets are formed in 64 bits.
#pragma once

#include "zorder.cuh"

namespace zeta {

// One call on the cache: the problem plus the cache's sizes.
struct Cache {
    int n;             // rows of new tokens per sequence
    int psh, pmask;    // page = 1 << psh
    int pages, opages; // pages of the K/V pools and of the order pools
    int tlen;          // row length of the tables
    const int32_t *start, *count;   // [B]
    const int32_t *ptab, *otab;     // [B, tlen]
};

// What sequence b brings: tokens before, new tokens.  count = 0 (and a recorded
// status) when either is out of range.
struct Seq {
    int start, count;
};
__device__ __forceinline__ Seq seq_of(const Cache &c, int b, int N, int32_t *status) {
    Seq s{__ldg(c.start + b), __ldg(c.count + b)};
    if (s.start < 0 || s.count < 0 || s.count > c.n || s.start > N - s.count) {
        set_status(status, ZETA_ERR_BOUNDS);
        s.count = 0;
    }
    return s;
}

// Row of token t (0 <= t < N) in the pools, -1 when its page is out of range.
__device__ __forceinline__ int page_row(const int32_t *__restrict__ tab, int t, int h, int H,
                                        int psh, int pmask, int pages) {
    const int id = __ldg(tab + (t >> psh));
    return (unsigned)id < (unsigned)pages ? (((id * H + h) << psh) | (t & pmask)) : -1;
}

// The same in two halves, so that independent lookups are in flight together and
// nothing looks at a page number before it is needed (a warp issues in order: a
// check placed behind a load waits for that load).
__device__ __forceinline__ int page_id(const int32_t *__restrict__ tab, int t, int psh) {
    return __ldg(tab + (t >> psh));
}
__device__ __forceinline__ int row_in(int id, int t, int h, int H, int psh, int pmask, int pages) {
    return (unsigned)id < (unsigned)pages ? (((id * H + h) << psh) | (t & pmask)) : -1;
}

// Z-order code of one point in registers (zeta_encode's, see encode.cu).
__device__ __forceinline__ uint64_t code_of(const float (&x)[kMaxDK], int dK, int bits) {
    const float scale = __int_as_float((126 + bits) << 23);   // 2^(bits-1)
    const float umax = static_cast<float>((1u << bits) - 1u);
    if (dK == 3 && bits <= 10)
        return (dilate3_10(quantise(x[0], scale, umax)) << 2) |
               (dilate3_10(quantise(x[1], scale, umax)) << 1) |
               dilate3_10(quantise(x[2], scale, umax));
    if (dK == 3)
        return morton3(quantise(x[0], scale, umax), quantise(x[1], scale, umax),
                       quantise(x[2], scale, umax));
    if (dK == 2)
        return (dilate2(quantise(x[0], scale, umax)) << 1) | dilate2(quantise(x[1], scale, umax));
    if (dK == 1) return quantise(x[0], scale, umax);
    uint64_t code = 0;
#pragma unroll
    for (int d = 0; d < kMaxDK; ++d) {
        if (d < dK) {
            const uint32_t u = quantise(x[d], scale, umax);
            for (int j = 0; j < bits; ++j)
                code |= static_cast<uint64_t>((u >> j) & 1u) << (j * dK + dK - 1 - d);
        }
    }
    return code;
}

__device__ __forceinline__ void load_point(float (&x)[kMaxDK], const float *p, int dK) {
#pragma unroll
    for (int d = 0; d < kMaxDK; ++d) x[d] = d < dK ? p[d] : 0.f;
}

__device__ __forceinline__ float4 ld_key(const float *p, int dK) {
    return make_float4(p[0], dK > 1 ? p[1] : 0.f, dK > 2 ? p[2] : 0.f, dK > 3 ? p[3] : 0.f);
}

// 16 bytes through the read-only path, zeros where `ok` is false: one predicated
// load.  (Written as a branch, the loads of a row's pieces wait for one another:
// 7 us per gathered row instead of one memory latency.)
__device__ __forceinline__ uint4 ld16_if(const void *p, bool ok) {
    uint4 a = make_uint4(0u, 0u, 0u, 0u);
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %5, 0;\n"
        " @q ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];\n}\n"
        : "+r"(a.x), "+r"(a.y), "+r"(a.z), "+r"(a.w)
        : "l"(p), "r"((int)ok));
    return a;
}
__device__ __forceinline__ uint32_t ld4_if(const void *p, bool ok) {
    uint32_t a = 0u;
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n @q ld.global.nc.b32 %0, [%1];\n}\n"
                 : "+r"(a)
                 : "l"(p), "r"((int)ok));
    return a;
}
__device__ __forceinline__ uint32_t ld2_if(const void *p, bool ok) {
    unsigned short a = 0;
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n @q ld.global.nc.u16 %0, [%1];\n}\n"
                 : "+h"(a)
                 : "l"(p), "r"((int)ok));
    return a;
}

// The same for a word that is -1 where `ok` is false.
__device__ __forceinline__ int ldi_if(const int32_t *p, bool ok) {
    int a = -1;
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %2, 0;\n @q ld.global.nc.b32 %0, [%1];\n}\n"
                 : "+r"(a)
                 : "l"(p), "r"((int)ok));
    return a;
}

cudaError_t launch_cache_append(const Prob &p, const Cache &c, const float *k, const void *v,
                                float *k_pages, void *v_pages, int32_t *status, cudaStream_t st);
cudaError_t launch_cache_order(const Prob &p, const Cache &c, const float *k_pages,
                               void *order_codes, int32_t *order_idx, int32_t *status,
                               cudaStream_t st);
cudaError_t launch_cache_attend(const Prob &p, const Cache &c, const float *q, const float *gamma,
                                const float *k_pages, const void *v_pages,
                                const void *order_codes, const int32_t *order_idx, void *out,
                                float *rowsum, int32_t *idx, int32_t *status, cudaStream_t st);

}  // namespace zeta
