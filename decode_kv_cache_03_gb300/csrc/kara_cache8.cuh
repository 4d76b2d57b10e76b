// The 8-bit form of the cache: codes, scales and the launchers of its entry points
// (internal header).
//
// A value is its e4m3 code times the scale of its block and head.  Scales are powers of
// two: a block that gets a larger one moves its codes' exponents and rounds only what
// falls among the subnormals, code times scale is exact in bf16, and e4m3, a floating
// type, would gain nothing from scales in between but the half of its top octave.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "kara_common.cuh"

namespace kara {

constexpr float kTop8 = 448.f;  // largest finite e4m3 value

// The smallest power of two s with amax <= 448 s, within 2^-63 .. 2^63; 0 for 0.  (448 is
// 1.75 * 2^8: the added bits carry into the exponent if the mantissa is above 1.75.)
__device__ __forceinline__ float scale_for(float amax)
{
    if (amax == 0.f) return 0.f;
    const int e = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - 127 - 8;
    return __uint_as_float((uint32_t)(min(max(e, -63), 63) + 127) << 23);
}

// 1 / s for a scale (a power of two: exact), 0 for 0.
__device__ __forceinline__ float inverse_scale(float s)
{
    return s == 0.f ? 0.f : __uint_as_float(0x7f000000u - __float_as_uint(s));
}

// Two values rounded to nearest-even e4m3 codes, lo in the low byte; above 448: 448, NaN: NaN.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// (lo, hi) rounded to nearest-even f16, lo in the low half.
__device__ __forceinline__ uint32_t f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// (lo, hi) rounded to nearest-even bf16, lo in the low half.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two codes as f16 values (exact), the low byte's in the low half.
__device__ __forceinline__ uint32_t f16_of_e4m3x2(uint32_t codes)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
    return r;
}

__device__ __forceinline__ void f32_of_f16x2(uint32_t h, float &lo, float &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
}

// Four codes as fp32 values.
__device__ __forceinline__ void values4(uint32_t codes, float (&x)[4])
{
    f32_of_f16x2(f16_of_e4m3x2(codes & 0xffffu), x[0], x[1]);
    f32_of_f16x2(f16_of_e4m3x2(codes >> 16), x[2], x[3]);
}

// Four codes of a block whose scale grows: times `ratio`, the old scale over the new.
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float ratio)
{
    float x[4];
    values4(codes, x);
    return e4m3x2(x[0] * ratio, x[1] * ratio) | e4m3x2(x[2] * ratio, x[3] * ratio) << 16;
}

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // defined beside the scoring kernel

// Tensor map over one pool of codes, (d, slot, kv head, block, layer) with the cache's strides; a box is
// a (block, head) slice, `swizzled` by its row size or as it lies in memory.
inline cudaError_t pool_map8(CUtensorMap *m, const void *pool, const kara_cache8 *c, bool swizzled)
{
    auto fn = tensor_map_encoder();
    if (!fn) return cudaErrorNotSupported;
    cuuint64_t dims[5] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->block_size, (cuuint64_t)c->num_kv_heads,
                          (cuuint64_t)c->num_blocks, (cuuint64_t)c->num_layers};
    cuuint64_t strides[4] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->head_stride, (cuuint64_t)c->block_stride,
                             (cuuint64_t)c->layer_stride};
    cuuint32_t box[5] = {(cuuint32_t)c->head_dim, (cuuint32_t)c->block_size, 1, 1, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const CUtensorMapSwizzle swizzle = !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE
                                       : c->head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(pool), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_append8(const kara_cache8 *c, int32_t layer, const kara_tokens *t, const kara_rope *r, const void *q,
                           int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                           void *q_out, void *ring, int32_t W, int32_t *err, cudaStream_t st);
int decode8_max_splits(const kara_cache8 *c, int32_t n, int32_t bt_stride);
size_t decode8_workspace_bytes(const kara_cache8 *c, int32_t n, int32_t bt_stride);
cudaError_t launch_decode8(const kara_cache8 *c, int32_t layer, int32_t n, const int32_t *len, const int32_t *bt,
                           int32_t bt_stride, const void *q, void *out, void *ws, int32_t *err, cudaStream_t st);
cudaError_t launch_chunk8(const kara_cache8 *c, int32_t layer, const kara_tokens *t, const int32_t *bt,
                          int32_t bt_stride, const void *q, void *out, void *ws, int32_t *err, cudaStream_t st);
cudaError_t launch_expand8(const kara_cache8 *c, const kara_cache *out, int32_t W, int32_t n, const int32_t *len,
                           const int32_t *bt, int32_t bt_stride, int32_t *out_table, int32_t *err, cudaStream_t st);
cudaError_t launch_compact8(const kara_cache8 *c, const Geo &g, SeqPlan *plan, int32_t *done, const int32_t *kept,
                            const int32_t *fresh, int64_t n_fresh, int32_t *freed, int32_t *new_len, int32_t *table,
                            int32_t *err, cudaStream_t st);

}  // namespace kara
