// New tokens into the cache: per-head norms of q and k, the position rotation,
// and the write of K and V into the pages in one pass.
//
// For a row x of a query or key head (D values), with the norm's weight w:
//     y = x / sqrt(mean(x^2) + eps) * w           (y = x without a weight)
//     (z_a, z_b) = (y_a c - y_b s, y_b c + y_a s)  for each rotated pair (a, b),
// c and s read from the caller's table at the token's rotary position; dims past
// rot_dim pass through.  All of it is fp32 with one rounding to bf16 at the end.
// V rows are copied.  Queries go to q_out, and those of a sequence's last W
// positions also to the window-query ring that the scorer reads.
//
// Nothing is reused but the table row, so the floor is one read of q, k, v and
// one write of them: HBM for long chunks, launch latency for a decode step.  D/8
// lanes hold a row, 16 bytes each, so a warp takes 32 / (D/8) rows at once; a
// row's sum of squares is a butterfly over its lanes, and the two halves of a
// rotated pair meet in a shuffle.
#include "kara_common.cuh"

namespace kara {
namespace {

constexpr int kAppThreads = 256;

struct AppArgs {
    const uint16_t *q, *k, *v;
    int64_t qs, ks, vs;  // token strides (elements)
    uint16_t *q_out, *kp, *vp, *ring;
    int64_t block_stride, head_stride;
    int64_t ring_seq, ring_head;  // strides of the ring (elements), at the call's layer
    const uint16_t *qw, *kw;
    const float *cos_sin;
    const int32_t *shift;
    const int64_t *slot;
    const int32_t *seq, *pos, *len;
    int32_t *err;
    float eps;
    int32_t n, rows, num_blocks, bs, hq, hkv, W, n_pos, rot, inter, parts;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8])
{
    x[0] = bf_lo(u.x), x[1] = bf_hi(u.x), x[2] = bf_lo(u.y), x[3] = bf_hi(u.y);
    x[4] = bf_lo(u.z), x[5] = bf_hi(u.z), x[6] = bf_lo(u.w), x[7] = bf_hi(u.w);
}

// (lo, hi) rounded to nearest-even bf16, lo in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A warp takes PASSES groups of 32 / (D/8) rows of one token.
template <int D, int PASSES>
__global__ void __launch_bounds__(kAppThreads) append_kernel(const AppArgs a)
{
    constexpr int LPR = D / 8;     // lanes per row
    constexpr int RPP = 32 / LPR;  // rows per pass
    const int64_t unit = ((int64_t)blockIdx.x * kAppThreads + threadIdx.x) >> 5;
    const int64_t t = unit / a.parts;
    if (t >= a.rows) return;
    const int part = (int)(unit % a.parts);
    const int lane = threadIdx.x & 31, l = lane % LPR;

    const int64_t slot = a.slot[t];
    if (slot == -1) return;  // padding
    const int32_t s = a.seq[t], x = a.pos[t];
    const bool known = s >= 0 && s < a.n;
    // without a rotation every rotary position will do
    const int64_t r = a.rot == 0 ? 0 : (int64_t)x + (known && a.shift ? a.shift[s] : 0);
    if (slot < 0 || slot >= (int64_t)a.num_blocks * a.bs) {
        if (part == 0 && lane == 0) set_err(a.err, KARA_EBADBLOCK);
        return;
    }
    if (!known || x < 0 || r < 0 || r >= a.n_pos) {
        if (part == 0 && lane == 0) set_err(a.err, KARA_EINVAL);
        return;
    }

    // this lane's cosines and signed sines, one per value it holds
    float c[8], sn[8];
    const int half = a.rot >> 1, d0 = l * 8;
    const bool turned = d0 < a.rot;
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = 1.f, sn[e] = 0.f;
    if (turned) {
        const float *row = a.cos_sin + r * a.rot;
        if (a.inter) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = d0 / 2 + e;
                c[2 * e] = c[2 * e + 1] = row[j];
                sn[2 * e + 1] = row[half + j];
                sn[2 * e] = -sn[2 * e + 1];
            }
        } else {
            const int j0 = d0 < half ? d0 : d0 - half;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                c[e] = row[j0 + e];
                sn[e] = d0 < half ? -row[half + j0 + e] : row[half + j0 + e];
            }
        }
    }
    // lane that holds the other half of this lane's pairs
    const int other = !turned || a.inter ? lane : d0 < half ? lane + half / 8 : lane - half / 8;

    const int nrow = a.hq + 2 * a.hkv;
    uint4 in[PASSES];
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int h = (part * PASSES + p) * RPP + lane / LPR;
        if (h >= nrow) continue;
        const uint16_t *src = h < a.hq            ? a.q + t * a.qs + h * D
                              : h < a.hq + a.hkv ? a.k + t * a.ks + (h - a.hq) * D
                                                 : a.v + t * a.vs + (h - a.hq - a.hkv) * D;
        in[p] = *reinterpret_cast<const uint4 *>(src + d0);
    }
    const int64_t page = (slot / a.bs) * a.block_stride + (slot % a.bs) * D + d0;
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
        const int h = (part * PASSES + p) * RPP + lane / LPR;
        const bool is_v = h >= a.hq + a.hkv, is_q = h < a.hq;
        uint4 out = in[p];
        float y[8];
        unpack8(in[p], y);
        const uint16_t *wp = is_q ? a.qw : a.kw;
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (wp) {
            float w[8];
            unpack8(__ldg(reinterpret_cast<const uint4 *>(wp + d0)), w);
            const float inv = 1.f / sqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = y[e] * inv * w[e];
        }
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float far = __shfl_sync(0xffffffffu, y[e], other);
            z[e] = fmaf(y[e], c[e], (a.inter ? y[e ^ 1] : far) * sn[e]);
        }
        if (h >= nrow) continue;
        if (!is_v) {
            out.x = pack_bf16(z[0], z[1]), out.y = pack_bf16(z[2], z[3]);
            out.z = pack_bf16(z[4], z[5]), out.w = pack_bf16(z[6], z[7]);
        }
        if (is_q) {
            *reinterpret_cast<uint4 *>(a.q_out + (t * a.hq + h) * D + d0) = out;
            if (a.ring) {
                const int32_t L = a.len[s];
                if (x < L && x >= (int64_t)L - a.W)
                    *reinterpret_cast<uint4 *>(a.ring + s * a.ring_seq + h * a.ring_head + (int64_t)(x % a.W) * D +
                                               d0) = out;
            }
        } else {
            uint16_t *pool = is_v ? a.vp : a.kp;
            const int g = is_v ? h - a.hq - a.hkv : h - a.hq;
            *reinterpret_cast<uint4 *>(pool + page + g * a.head_stride) = out;
        }
    }
}

template <int D, int PASSES>
cudaError_t launch(AppArgs a, cudaStream_t st)
{
    constexpr int RPP = 32 / (D / 8);
    a.parts = (a.hq + 2 * a.hkv + RPP * PASSES - 1) / (RPP * PASSES);
    const int64_t warps = (int64_t)a.rows * a.parts;
    const int64_t grid = (warps * 32 + kAppThreads - 1) / kAppThreads;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    append_kernel<D, PASSES><<<(unsigned)grid, kAppThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const kara_cache *c, int32_t layer, const kara_tokens *t, const kara_rope *r, const void *q,
                          int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                          void *q_out, void *ring, int32_t W, int32_t *err, cudaStream_t st)
{
    const int D = c->head_dim;
    AppArgs a;
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.qs = q_stride, a.ks = k_stride, a.vs = v_stride;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.kp = static_cast<uint16_t *>(c->k) + (int64_t)layer * c->layer_stride;
    a.vp = static_cast<uint16_t *>(c->v) + (int64_t)layer * c->layer_stride;
    a.block_stride = c->block_stride;
    a.head_stride = c->head_stride;
    a.W = ring ? W : 1;
    a.ring_head = (int64_t)W * D;
    a.ring_seq = (int64_t)c->num_layers * c->num_q_heads * a.ring_head;
    a.ring = ring ? static_cast<uint16_t *>(ring) + (int64_t)layer * c->num_q_heads * a.ring_head : nullptr;
    a.qw = static_cast<const uint16_t *>(r->q_weight);
    a.kw = static_cast<const uint16_t *>(r->k_weight);
    a.cos_sin = r->cos_sin;
    a.shift = r->pos_offset;
    a.slot = t->slot;
    a.seq = t->seq;
    a.pos = t->pos;
    a.len = t->len;
    a.err = err;
    a.eps = r->eps;
    a.n = t->n;
    a.rows = t->rows;
    a.num_blocks = c->num_blocks;
    a.bs = c->block_size;
    a.hq = c->num_q_heads;
    a.hkv = c->num_kv_heads;
    a.n_pos = r->rot_dim > 0 ? r->n_pos : 1;
    a.rot = r->rot_dim;
    a.inter = r->interleaved;
    return D == 128 ? launch<128, 1>(a, st) : launch<64, 1>(a, st);
}

}  // namespace kara
