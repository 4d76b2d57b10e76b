// Attention of a chunk of new tokens over the paged cache.
//
// Row t of q is the new token at position p of sequence s (its K and V are in
// the cache already); query head h belongs to KV head g = h / G:
//     out[t][h] = sum_{x <= p} softmax_x(<q[t][h], k_x> / sqrt(D)) v_x
// over the keys of the sequence, read through its block table.
//
// One warp per (row, query head): lanes take one key each for the logits, and
// D/32 dims each for the weighted sum, with the running maximum and sum of the
// softmax in fp32.
#include "kara_common.cuh"

namespace kara {
namespace {

constexpr int kWarps = 4;

struct ChunkArgs {
    const uint16_t *q;
    uint16_t *out;
    const uint16_t *k, *v;  // pools at the call's layer
    int64_t block_stride, head_stride;
    const int32_t *q_start, *len, *bt;
    int32_t *err;
    int32_t n, rows, bt_stride, num_blocks, bs, hq, G;
    float scale2;
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32) chunk_kernel(const ChunkArgs a)
{
    __shared__ float qs[kWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
    const int64_t t = unit / a.hq;
    const int h = (int)(unit % a.hq);
    if (blockIdx.x == 0)
        for (int s = threadIdx.x; s < a.n; s += kWarps * 32) {
            const int32_t r0 = a.q_start[s], r1 = a.q_start[s + 1];
            if (r0 < 0 || r1 < r0 || r1 > a.rows) set_err(a.err, KARA_EINVAL);
        }
    if (t >= a.rows || t >= a.q_start[a.n]) return;
    int lo = 0, hi = a.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q_start[mid] <= t) lo = mid; else hi = mid;
    }
    const int s = lo;
    const int32_t m = a.q_start[s + 1] - a.q_start[s], L = a.len[s];
    uint16_t *o = a.out + (t * a.hq + h) * D;
    if (m < 1 || L < m || t < a.q_start[s] || t >= a.q_start[s + 1] || ((int64_t)L + a.bs - 1) / a.bs > a.bt_stride) {
        if (lane == 0) set_err(a.err, KARA_EINVAL);
        for (int d = lane; d < D; d += 32) o[d] = 0;
        return;
    }
    const int32_t last = L - m + (int32_t)(t - a.q_start[s]);
    const uint16_t *qr = a.q + (t * a.hq + h) * D;
    for (int d = lane; d < D; d += 32) qs[warp][d] = __uint_as_float((uint32_t)qr[d] << 16) * a.scale2;
    __syncwarp();
    float mx = -INFINITY, z = 0.f, acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
    for (int32_t x0 = 0; x0 <= last; x0 += 32) {
        const int32_t x = x0 + lane;
        float l = -INFINITY;
        int64_t off = -1;
        if (x <= last) {
            const int32_t b = a.bt[(int64_t)s * a.bt_stride + x / a.bs];
            l = 0.f;
            if (b < 0 || b >= a.num_blocks) {
                set_err(a.err, KARA_EBADBLOCK);
            } else {
                off = b * a.block_stride + (int64_t)(h / a.G) * a.head_stride + (int64_t)(x % a.bs) * D;
                for (int d = 0; d < D; ++d) l = fmaf(qs[warp][d], __uint_as_float((uint32_t)a.k[off + d] << 16), l);
            }
        }
        float nm = l;
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, i));
        nm = fmaxf(nm, mx);
        const float c = exp2f(mx - nm), p = x <= last ? exp2f(l - nm) : 0.f;
        mx = nm;
        z = z * c + p;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] *= c;
        for (int j = 0; j < 32 && x0 + j <= last; ++j) {
            const float pj = __shfl_sync(0xffffffffu, p, j);
            const int64_t oj = __shfl_sync(0xffffffffu, off, j);
            if (oj >= 0)
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
                    acc[i] = fmaf(pj, __uint_as_float((uint32_t)a.v[oj + i * 32 + lane] << 16), acc[i]);
        }
    }
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) z += __shfl_xor_sync(0xffffffffu, z, i);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const float r = acc[i] / z;
        uint16_t b;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(r));
        o[i * 32 + lane] = b;
    }
}

}  // namespace

size_t chunk_workspace_bytes(const kara_cache *, int32_t, int32_t) { return 256; }

cudaError_t launch_chunk(const kara_cache *c, int32_t layer, const kara_tokens *t, const int32_t *bt,
                         int32_t bt_stride, const void *q, void *out, void *, int32_t *err, cudaStream_t st)
{
    ChunkArgs a;
    a.q = static_cast<const uint16_t *>(q);
    a.out = static_cast<uint16_t *>(out);
    a.k = static_cast<const uint16_t *>(c->k) + (int64_t)layer * c->layer_stride;
    a.v = static_cast<const uint16_t *>(c->v) + (int64_t)layer * c->layer_stride;
    a.block_stride = c->block_stride;
    a.head_stride = c->head_stride;
    a.q_start = t->q_start;
    a.len = t->len;
    a.bt = bt;
    a.err = err;
    a.n = t->n;
    a.rows = t->rows;
    a.bt_stride = bt_stride;
    a.num_blocks = c->num_blocks;
    a.bs = c->block_size;
    a.hq = c->num_q_heads;
    a.G = c->num_q_heads / c->num_kv_heads;
    a.scale2 = 1.4426950408889634f / sqrtf((float)c->head_dim);
    const int64_t grid = ((int64_t)t->rows * a.hq + kWarps - 1) / kWarps;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (c->head_dim == 128)
        chunk_kernel<128><<<(unsigned)grid, kWarps * 32, 0, st>>>(a);
    else
        chunk_kernel<64><<<(unsigned)grid, kWarps * 32, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace kara
