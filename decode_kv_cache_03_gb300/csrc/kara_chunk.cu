// Attention of a chunk of new tokens over the bf16 cache: the kernel of kara_chunk.cuh on it.
// (A source per cache: in one, what the kernels share out of line got the registers that suit
// the other, and the bf16 one ran 2 to 3 % slower.)
namespace kara {
namespace {

constexpr int kStages = 5;       // K and V tiles in flight
// V tiles issued and not cleaned yet, at most.  V tile i takes the stage of K tile i - (kStages - 1) / 2, and
// when both MMA warps have given that one back, every V tile two or more before it is clean: with two query
// tiles its logits are issued behind the weighted sum of the V tile before; with one, a warp passes the V
// tile two before it, clean, ahead of this K tile.
constexpr int kEdges = (kStages - 1) / 2 + 2;
static_assert(kEdges == 4 && kStages % 2 == 1, "Shared::edge tells four edge tiles apart, K and V take turns");

// In about 800 clocks: a key tile of two query tiles 3000 to 3400, of one 2500, an item's start and end about 6500;
// all at D = 128.  (Two to one for the tiles: the mixed batch of decodes and chunks takes 358 us, four to three
// 338, captured.)
constexpr int kPairCost = 4, kSingleCost = 3, kItemCost = 8;

}  // namespace
}  // namespace kara

#include "kara_chunk.cuh"

namespace kara {
namespace {

// Tensor map over one pool, (d, slot, kv head, block, layer) with the cache's
// strides; a box is one 64-dim half of a (block, head) slice, 128-byte swizzled.
cudaError_t pool_map(CUtensorMap *m, const void *pool, const kara_cache *c)
{
    auto fn = tensor_map_encoder();
    if (!fn) return cudaErrorNotSupported;
    cuuint64_t dims[5] = {(cuuint64_t)c->head_dim, (cuuint64_t)kBlk, (cuuint64_t)c->num_kv_heads,
                          (cuuint64_t)c->num_blocks, (cuuint64_t)c->num_layers};
    cuuint64_t strides[4] = {(cuuint64_t)c->head_dim * 2, (cuuint64_t)c->head_stride * 2,
                             (cuuint64_t)c->block_stride * 2, (cuuint64_t)c->layer_stride * 2};
    cuuint32_t box[5] = {64, (cuuint32_t)kBlk, 1, 1, 1};
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    if (fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(pool), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return cudaSuccess;
}

}  // namespace

size_t chunk_workspace_bytes(int32_t head_dim) { return layout(head_dim).total; }

cudaError_t launch_chunk(const kara_cache *c, int32_t layer, const kara_tokens *t, const int32_t *bt,
                         int32_t bt_stride, const void *q, void *out, void *ws, int32_t *err, cudaStream_t st)
{
    ChunkArgs a;
    CUtensorMap km, vm, qm;
    cudaError_t e = chunk_args(&a, &qm, c, layer, t, bt, bt_stride, q, out, ws, err);
    a.v = static_cast<const uint16_t *>(c->v) + (int64_t)layer * c->layer_stride;
    if (e == cudaSuccess) e = pool_map(&km, c->k, c);
    if (e == cudaSuccess) e = pool_map(&vm, c->v, c);
    if (e != cudaSuccess) return e;
    return c->head_dim == 128 ? launch_all<128, false>(km, vm, qm, a, st) : launch_all<64, false>(km, vm, qm, a, st);
}

}  // namespace kara
