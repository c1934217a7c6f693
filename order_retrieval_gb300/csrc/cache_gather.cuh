// cache_gather.cuh -- the weighted sum of up to 64 gathered bf16 value rows by one
// warp on the tensor cores.
#pragma once

#include "cache.cuh"
#include "mma.cuh"

namespace zeta {

__device__ __forceinline__ float4 ld_key(const float *p, int dK) {
    return make_float4(p[0], dK > 1 ? p[1] : 0.f, dK > 2 ? p[2] : 0.f, dK > 3 ? p[3] : 0.f);
}

// Sums of w v over 64 CB columns: column 0 of 4 CB mma tiles.
template <int CB>
struct GatherSum {
    float c[CB][4][4];
    __device__ __forceinline__ void scale(float f) {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) c[cb][m][e] *= f;
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) c[cb][m][e] = 0.f;
    }
    // Column 0 lives in the lanes 4 g: mma rows g and g + 8 of tile m, which are the
    // dimensions 64 cb + 8 (g / 2) + 2 m + g % 2 and 32 more.
    template <typename Put>
    __device__ __forceinline__ void each(int lane, Put put) const {
        if ((lane & 3) == 0) {
            const int d0 = 8 * (lane >> 3) + ((lane >> 2) & 1);
#pragma unroll
            for (int cb = 0; cb < CB; ++cb)
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    put(64 * cb + d0 + 2 * m, c[cb][m][0]);
                    put(64 * cb + d0 + 2 * m + 32, c[cb][m][2]);
                }
        }
    }
};

// Lane L holds the pool rows of keys L and L + 32 of the pass (-1: none); nmt: 16-key
// groups in use.  The 16-byte pieces of 16 rows at a time are asked for by four
// lanes a row (pieces t and t + 4), transposed 8x8 in registers into A fragments of
// V^T, and multiplied with w (rounded to bf16) in column 0 of B.  between(), called
// once while the first 64 columns are on their way, gives the lane's two weights
// (and may rescale the sums).
template <int CB, typename Between>
__device__ __forceinline__ void gather64(GatherSum<CB> &a, const __nv_bfloat16 *v_pages, int dV,
                                         int ppr, const int (&prow)[2], int nmt, int lane,
                                         Between between) {
    const int g4 = lane >> 2, s4 = lane & 3;
    float2 w = make_float2(0.f, 0.f);
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        uint4 buf[4][4];                     // rows g4, g4 + 8 of group mt: pieces s4, s4 + 4
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const int pr = __shfl_sync(kFull, prow[mt >> 1], (16 * mt + 8 * hh + g4) & 31);
                const uint4 *vr = reinterpret_cast<const uint4 *>(v_pages + (int64_t)max(pr, 0) * dV);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int pc = cb * 8 + s4 + 4 * e;
                    buf[mt][2 * hh + e] = ld16_if(vr + pc, mt < nmt && pr >= 0 && pc < ppr);
                }
            }
        if (cb == 0) w = between();
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
            if (mt < nmt) {
                const float ww = mt < 2 ? w.x : w.y;
                const int sb = 16 * mt + 2 * s4;
                const float e0 = __shfl_sync(kFull, ww, sb & 31);
                const float e1 = __shfl_sync(kFull, ww, (sb + 1) & 31);
                const float e2 = __shfl_sync(kFull, ww, (sb + 8) & 31);
                const float e3 = __shfl_sync(kFull, ww, (sb + 9) & 31);
                const uint32_t ba = g4 == 0 ? pack_bf16(e0, e1) : 0u;
                const uint32_t bb = g4 == 0 ? pack_bf16(e2, e3) : 0u;
                const uint32_t a0[4] = {buf[mt][0].x, buf[mt][0].y, buf[mt][0].z, buf[mt][0].w};
                const uint32_t a1[4] = {buf[mt][1].x, buf[mt][1].y, buf[mt][1].z, buf[mt][1].w};
                const uint32_t b0[4] = {buf[mt][2].x, buf[mt][2].y, buf[mt][2].z, buf[mt][2].w};
                const uint32_t b1[4] = {buf[mt][3].x, buf[mt][3].y, buf[mt][3].z, buf[mt][3].w};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const uint32_t af[4] = {movmatrix_trans(a0[m]), movmatrix_trans(a1[m]),
                                            movmatrix_trans(b0[m]), movmatrix_trans(b1[m])};
                    mma16816(a.c[cb][m], af, ba, bb);
                }
            }
        }
    }
}

}  // namespace zeta
