// Attention of a chunk of new tokens over the 8-bit cache: the kernel of kara_chunk.cuh on it.
namespace kara {
namespace {

constexpr int kStages = 2;  // f16 tiles of V, beside which the tiles of codes in flight lie
constexpr int kEdges = 1;   // (no edge tiles of V: what converts a tile clears it)

// A key tile of two query tiles, of one, an item's start and end, in 490 clocks: 3900, 2440, and what serves best
// (its queries are split, its tiles of codes fetched and converted before the first product).  64 sequences of 1 to 128
// tokens, 48 of 1 to 200, 32 of 1 to 60, 64 of 1 to 8 over short caches: with the bf16 cache's costs 375, 294,
// 167 and 62.6 us, with these 364, 272, 158 and 62.3; 8 5 20 366 277 159 62.7, 8 5 40 364 269 158 62.2, 8 4 32 377 265 168 62.
constexpr int kPairCost = 8, kSingleCost = 5, kItemCost = 30;

}  // namespace
}  // namespace kara

#include "kara_chunk.cuh"

namespace kara {

cudaError_t launch_chunk8(const kara_cache8 *c, int32_t layer, const kara_tokens *t, const int32_t *bt,
                          int32_t bt_stride, const void *q, void *out, void *ws, int32_t *err, cudaStream_t st)
{
    ChunkArgs a;
    CUtensorMap km, vm, qm;
    cudaError_t e = chunk_args(&a, &qm, c, layer, t, bt, bt_stride, q, out, ws, err);
    const int64_t scales = (int64_t)layer * c->num_blocks * c->num_kv_heads;
    a.v8 = static_cast<const uint8_t *>(c->v) + (int64_t)layer * c->layer_stride;
    a.k_scale = c->k_scale + scales;
    a.v_scale = c->v_scale + scales;
    if (e == cudaSuccess) e = pool_map8(&km, c->k, c, true);
    if (e == cudaSuccess) e = pool_map8(&vm, c->v, c, false);
    if (e != cudaSuccess) return e;
    return c->head_dim == 128 ? launch_all<128, true>(km, vm, qm, a, st) : launch_all<64, true>(km, vm, qm, a, st);
}

}  // namespace kara
