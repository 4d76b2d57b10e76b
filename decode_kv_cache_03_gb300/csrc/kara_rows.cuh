// Arithmetic of a head row in the append kernels: a lane has eight neighbouring values
// of a row, as packed fp32 pairs (internal header).
#pragma once

#include "kara_sm100.cuh"

namespace kara {

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// (lo, hi) rounded to nearest-even bf16, lo in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float4 ldg4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }

// (a*b) on both halves, round-to-nearest.
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Eight bf16 as pairs of neighbours, in fp32; with `swap` each pair the other way round.
__device__ __forceinline__ void pairs4(const uint4 &u, uint64_t (&x)[4], bool swap)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float lo = bf_lo(w[e]), hi = bf_hi(w[e]);
        x[e] = swap ? ptx::pack2(hi, lo) : ptx::pack2(lo, hi);
    }
}

// The arithmetic of a lane's eight values, one for every kernel, so that a token's bits do not depend on the
// length of the call that brings it, nor its query's on the cache's type.  This lane's part of the row's sum of
// squares:
__device__ __forceinline__ float squares(const uint64_t (&x)[4])
{
    uint64_t s2 = mul2(x[0], x[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) s2 = ptx::fma2(x[e], x[e], s2);
    float lo, hi;
    ptx::unpack2(s2, lo, hi);
    return lo + hi;
}

// x wc + x' ws': a pair's cosines times weights, and its partners times theirs and signed sines.
__device__ __forceinline__ uint64_t turn2(uint64_t x, uint64_t wc, uint64_t xo, uint64_t ws)
{
    return ptx::fma2(x, wc, mul2(xo, ws));
}

__device__ __forceinline__ float inverse_norm(float sum, float per, float eps) { return rsqrtf(fmaf(sum, per, eps)); }

// z / the norm, rounded.
__device__ __forceinline__ uint4 finish(const uint64_t (&z)[4], float inv)
{
    const uint64_t i2 = ptx::pack2(inv, inv);
    uint32_t r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float lo, hi;
        ptx::unpack2(mul2(z[e], i2), lo, hi);
        r[e] = pack_bf16(lo, hi);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

}  // namespace kara
