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
// row's sum of squares is a butterfly over its lanes.  Two kernels, which give a
// token the same bits (one arithmetic, below): for short calls a warp per pass,
// everything in registers; for long ones tokens staged through shared memory by
// bulk copies, because what bounds a long call is the latency of its chain of
// loads (slot, offset, table row, rows): in registers it reached 4.0 TB/s with four
// passes a warp (8192 tokens, 40/8 heads of 128, with the ring: 70 us), staged
// 5.4 TB/s (52 us).  Pairs of neighbours take 50 us, a rotation of half the dims 56
// (54), the same at D = 64 with as many heads 32 us (4.3 TB/s).
#include "kara_rows.cuh"
#include "kara_sm100.cuh"
#include "kara_tokens.cuh"

namespace kara {
namespace {

constexpr int kAppThreads = 256;
constexpr int kBs = 16;  // tokens per cache block (the supported block size)

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
    int32_t stall;     // debug: the staged kernel issues no copies (see debug_stall)
    uint64_t wait_ns;  // limit of its waits
    int32_t n, rows, num_blocks, hq, hkv, W, n_pos, rot, inter;
};

// A warp takes 32 / (D/8) rows of one token: token blockIdx.x * 8 + warp, rows of part blockIdx.y.
// (Five blocks per SM, 48 registers: 4096 tokens of 320 and 2 x 80 heads take 346 us; as the compiler likes it,
// with 56, 407 us.)
template <int D, bool INTER>
__global__ void __launch_bounds__(kAppThreads, 5) append_kernel(const AppArgs a)
{
    constexpr int LPR = D / 8;     // lanes per row
    constexpr int RPP = 32 / LPR;  // rows per pass
    const int64_t t = (int64_t)blockIdx.x * (kAppThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.rows) return;
    const int lane = threadIdx.x & 31, l = lane % LPR, d0 = l * 8;
    const int h = blockIdx.y * RPP + lane / LPR;
    const int nrow = a.hq + 2 * a.hkv;

    const bool is_v = h >= a.hq + a.hkv, is_q = h < a.hq;

    // launched as a programmatic dependent of what precedes it on the stream
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // the row is on its way before the token's place is known (padding rows are read, not written)
    const int64_t slot = a.slot[t];
    const int32_t s = a.seq[t], x = a.pos[t];
    uint4 u = make_uint4(0, 0, 0, 0);
    if (h < nrow) {
        const uint16_t *src = is_q ? a.q + t * a.qs + h * D
                              : is_v ? a.v + t * a.vs + (h - a.hq - a.hkv) * D
                                     : a.k + t * a.ks + (h - a.hq) * D;
        u = *reinterpret_cast<const uint4 *>(src + d0);
    }
    if (slot == -1) return;  // padding
    const bool known = s >= 0 && s < a.n;
    // without a rotation every rotary position will do
    const int64_t r = a.rot == 0 ? 0 : (int64_t)x + (known && a.shift ? a.shift[s] : 0);
    if (slot < 0 || slot >= (int64_t)a.num_blocks * kBs || !known || x < 0 || r < 0 || r >= a.n_pos) {
        if (blockIdx.y == 0 && lane == 0)
            set_err(a.err, slot < 0 || slot >= (int64_t)a.num_blocks * kBs ? KARA_EBADBLOCK : KARA_EINVAL);
        return;
    }

    // this lane's cosines and signed sines, in pairs of neighbours
    uint64_t c[4], sn[4];
    const int half = a.rot >> 1;
    const bool turned = d0 < a.rot, low = d0 < half;
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = ptx::pack2(1.f, 1.f), sn[e] = ptx::pack2(0.f, 0.f);
    if (turned) {
        const float *row = a.cos_sin + r * a.rot;
        if (INTER) {
            const float4 cc = ldg4(row + d0 / 2), ss = ldg4(row + half + d0 / 2);
            c[0] = ptx::pack2(cc.x, cc.x), c[1] = ptx::pack2(cc.y, cc.y);
            c[2] = ptx::pack2(cc.z, cc.z), c[3] = ptx::pack2(cc.w, cc.w);
            sn[0] = ptx::pack2(-ss.x, ss.x), sn[1] = ptx::pack2(-ss.y, ss.y);
            sn[2] = ptx::pack2(-ss.z, ss.z), sn[3] = ptx::pack2(-ss.w, ss.w);
        } else {
            const int j0 = low ? d0 : d0 - half;
            const uint64_t sg = low ? ptx::pack2(-1.f, -1.f) : ptx::pack2(1.f, 1.f);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float4 cc = ldg4(row + j0 + 2 * e), ss = ldg4(row + half + j0 + 2 * e);
                c[e] = ptx::pack2(cc.x, cc.y), c[e + 1] = ptx::pack2(cc.z, cc.w);
                sn[e] = mul2(sg, ptx::pack2(ss.x, ss.y)), sn[e + 1] = mul2(sg, ptx::pack2(ss.z, ss.w));
            }
        }
    }
    // lane that holds the other half of this lane's pairs
    const int other = !turned || INTER ? lane : low ? lane + half / 8 : lane - half / 8;
    const int64_t page = (slot / kBs) * a.block_stride + (slot % kBs) * D + d0;
    uint16_t *ring = nullptr;  // this token's row of the ring, if it is of the last W
    if (a.ring) {
        const int32_t L = a.len[s];
        if (x < L && x >= (int64_t)L - a.W) ring = a.ring + s * a.ring_seq + (int64_t)(x % a.W) * D + d0;
    }
    // (a warp whose rows are all values has nothing to compute)
    if (__any_sync(0xffffffffu, !is_v)) {
        // z = (x w c + x' w' s) / sqrt(mean(x^2) + eps), x' and w' of the pair's other member
        const uint4 one = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
        const uint16_t *wp = is_q ? a.qw : a.kw;
        const uint4 uw = wp ? __ldg(reinterpret_cast<const uint4 *>(wp + d0)) : one;
        uint4 uo = u, uwo = uw;
        if (!INTER && a.rot > 0) {
            uo.x = __shfl_sync(0xffffffffu, u.x, other), uo.y = __shfl_sync(0xffffffffu, u.y, other);
            uo.z = __shfl_sync(0xffffffffu, u.z, other), uo.w = __shfl_sync(0xffffffffu, u.w, other);
            if (wp) uwo = __ldg(reinterpret_cast<const uint4 *>(wp + (turned ? low ? d0 + half : d0 - half : d0)));
        }
        uint64_t x[4], xo[4], w[4], wo[4], z[4];
        pairs4(u, x, false), pairs4(uo, xo, INTER);
        pairs4(uw, w, false), pairs4(uwo, wo, INTER);
        float inv = 1.f;
        if (a.qw || a.kw) {
            float ss = squares(x);
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (wp) inv = inverse_norm(ss, 1.f / D, a.eps);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = turn2(x[e], mul2(w[e], c[e]), xo[e], mul2(wo[e], sn[e]));
        if (!turned) {  // (0 times an infinity is no number)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = mul2(x[e], w[e]);
        }
        if (!is_v) u = finish(z, inv);
    }
    if (h >= nrow) return;
    if (is_q) {
        *reinterpret_cast<uint4 *>(a.q_out + (t * a.hq + h) * D + d0) = u;
        if (ring) *reinterpret_cast<uint4 *>(ring + h * a.ring_head) = u;
    } else {
        uint16_t *pool = is_v ? a.vp : a.kp;
        const int g = is_v ? h - a.hq - a.hkv : h - a.hq;
        *reinterpret_cast<uint4 *>(pool + page + g * a.head_stride) = u;
    }
}

// ---- long calls: tokens staged through shared memory ------------------------------
// One warp per CTA brings in tokens by bulk copies (a token's q, k and v rows and its
// row of the rotation table, four copies), as many tokens ahead as the stages hold; four
// warps take a token's rows from shared memory (eight: 5 % slower, two: 15 %).  The chain
// slot, sequence -> offset -> table row is looked up for 32 tokens at once.
constexpr int kTokWarps = 4;
constexpr int kTokThreads = 32 * (1 + kTokWarps);
constexpr int kTokMaxStages = 8;
constexpr int kTokMaxSmem = 110 * 1024;  // of a CTA, two of which share an SM
// Calls of up to this many head rows (tokens times heads) take the other kernel: all their
// loads are in flight at once and there is no pipeline to fill.  Measured with 56 heads of 128
// (staged / a warp per two rows, us): 128 tokens 4.6 / 2.6, 256 4.9 / 4.1, 384 5.4 / 4.9, 512 5.8 / 6.1,
// 1024 9.0 / 10.6.
constexpr int kSmallRows = 20480;
constexpr uint64_t kTokTimeoutNs = 1000000000ull;

struct TokMeta {
    int64_t page;    // offset of the token's row in a pool (of KV head 0); -1: no more tokens
    int64_t ring;    // offset of its row in the ring (of head 0), -1: none
    int32_t row;     // row of q, k, v
    int32_t pad[3];
};

struct TokShared {
    uint64_t full[kTokMaxStages], empty[kTokMaxStages];
    TokMeta meta[kTokMaxStages];
    int32_t abort;
};

// Bounded wait on phase `parity` of `bar`: gives up after limit_ns, or once another
// warp of the CTA gave up, recording KARA_ETIMEOUT.
__device__ __forceinline__ bool twait(uint32_t bar, uint32_t parity, TokShared *sh, const AppArgs &a)
{
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 63u) {
            if (*(volatile int32_t *)&sh->abort) return false;
            const uint64_t now = ptx::globaltimer();
            if (t0 == 0) {
                t0 = now;
            } else if (now - t0 > a.wait_ns) {
                set_err(a.err, KARA_ETIMEOUT);
                *(volatile int32_t *)&sh->abort = 1;
                return false;
            }
        }
    }
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

__host__ __device__ __forceinline__ int tok_stage_bytes(int hq, int hkv, int D, int rot)
{
    return (hq + 2 * hkv) * D * 2 + rot * 4;
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kTokThreads, 4) append_staged_kernel(const AppArgs a, int stages)
{
    constexpr int LPR = D / 8, RPP = 32 / LPR;
    extern __shared__ __align__(128) uint8_t tsm[];
    TokShared *sh = reinterpret_cast<TokShared *>(tsm);
    uint8_t *buf = tsm + (sizeof(TokShared) + 127) / 128 * 128;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nrow = a.hq + 2 * a.hkv, half = a.rot >> 1;
    const int row_bytes = nrow * D * 2, stage_bytes = row_bytes + a.rot * 4;
    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sh->full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->empty[i]), kTokWarps);
        }
        sh->abort = 0;
        ptx::fence_mbarrier_init();
    }
    __syncthreads();
    // launched as a programmatic dependent of what precedes it on the stream
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == kTokWarps) {
        uint32_t st = 0, ph = 1, issued = 0;
        bool ok = !a.stall;
        for (int64_t base = blockIdx.x; ok && base < a.rows; base += 32ll * gridDim.x) {
            // this lane's token
            const int64_t t = base + (int64_t)lane * gridDim.x;
            int64_t page = -1, ring = -1, r = 0;
            if (t < a.rows) {
                const int64_t slot = a.slot[t];
                const int32_t s = a.seq[t], x = a.pos[t];
                const bool known = s >= 0 && s < a.n, inside = slot >= 0 && slot < (int64_t)a.num_blocks * kBs;
                r = a.rot == 0 ? 0 : (int64_t)x + (known && a.shift ? a.shift[s] : 0);
                if (slot != -1) {
                    if (!inside || !known || x < 0 || r < 0 || r >= a.n_pos) {
                        set_err(a.err, inside ? KARA_EINVAL : KARA_EBADBLOCK);
                    } else {
                        page = (slot / kBs) * a.block_stride + (slot % kBs) * D;
                        if (a.ring) {
                            const int32_t L = a.len[s];
                            if (x < L && x >= (int64_t)L - a.W) ring = s * a.ring_seq + (int64_t)(x % a.W) * D;
                        }
                    }
                }
            }
            for (unsigned todo = __ballot_sync(0xffffffffu, page >= 0); ok && todo; todo &= todo - 1) {
                const int src = __ffs(todo) - 1;
                ok = twait(ptx::smem_u32(&sh->empty[st]), ph, sh, a);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == src) {
                    const uint32_t fb = ptx::smem_u32(&sh->full[st]);
                    const uint32_t d = ptx::smem_u32(buf + st * stage_bytes);
                    TokMeta &m = sh->meta[st];
                    m.page = page, m.ring = ring, m.row = (int32_t)t;
                    ptx::mbar_arrive_expect_tx(fb, (uint32_t)stage_bytes);
                    bulk_load(d, a.q + t * a.qs, a.hq * D * 2, fb);
                    bulk_load(d + a.hq * D * 2, a.k + t * a.ks, a.hkv * D * 2, fb);
                    bulk_load(d + (a.hq + a.hkv) * D * 2, a.v + t * a.vs, a.hkv * D * 2, fb);
                    if (a.rot) bulk_load(d + row_bytes, a.cos_sin + r * a.rot, a.rot * 4, fb);
                }
                __syncwarp();
                ++issued;
                if (++st == (uint32_t)stages) st = 0, ph ^= 1;
            }
        }
        if (ok) ok = __all_sync(0xffffffffu, twait(ptx::smem_u32(&sh->empty[st]), ph, sh, a));
        if (ok && lane == 0) {  // the end
            sh->meta[st].page = -1;
            ptx::mbar_arrive(ptx::smem_u32(&sh->full[st]));
        }
        // every copy has landed before the CTA's shared memory is released
        for (uint32_t i = issued > (uint32_t)stages ? issued - stages : 0; !ok && i < issued; ++i) {
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(ptx::smem_u32(&sh->full[i % stages]), (i / stages) & 1))
                if (ptx::globaltimer() - t0 > kTokTimeoutNs) break;
        }
        return;
    }

    const int l = lane % LPR, d0 = l * 8, sub = lane / LPR;
    const bool turned = d0 < a.rot, low = d0 < half;
    // the other half of this lane's pairs: 16 bytes further on or back (interleaved: in the lane itself)
    const int o0 = !turned || INTER ? d0 : low ? d0 + half : d0 - half;
    // weights of this lane's dims and of their partners (1 without a norm)
    const uint4 one = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    const uint4 wq = a.qw ? *reinterpret_cast<const uint4 *>(a.qw + d0) : one;
    const uint4 wqo = a.qw ? *reinterpret_cast<const uint4 *>(a.qw + o0) : one;
    const uint4 wk = a.kw ? *reinterpret_cast<const uint4 *>(a.kw + d0) : one;
    const uint4 wko = a.kw ? *reinterpret_cast<const uint4 *>(a.kw + o0) : one;
    uint32_t st = 0, ph = 0;
    for (;;) {
        bool ok = twait(ptx::smem_u32(&sh->full[st]), ph, sh, a);
        if (!__all_sync(0xffffffffu, ok)) return;
        const TokMeta m = sh->meta[st];
        if (m.page < 0) return;
        const uint16_t *rows = reinterpret_cast<const uint16_t *>(buf + st * stage_bytes);
        const float *tab = reinterpret_cast<const float *>(buf + st * stage_bytes + row_bytes);
        // cosines and signed sines of this lane's dims, in pairs of neighbours
        uint64_t c[4], sn[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = ptx::pack2(1.f, 1.f), sn[e] = ptx::pack2(0.f, 0.f);
        if (turned && INTER) {
            const float4 cc = *reinterpret_cast<const float4 *>(tab + d0 / 2);
            const float4 ss = *reinterpret_cast<const float4 *>(tab + half + d0 / 2);
            c[0] = ptx::pack2(cc.x, cc.x), c[1] = ptx::pack2(cc.y, cc.y);
            c[2] = ptx::pack2(cc.z, cc.z), c[3] = ptx::pack2(cc.w, cc.w);
            sn[0] = ptx::pack2(-ss.x, ss.x), sn[1] = ptx::pack2(-ss.y, ss.y);
            sn[2] = ptx::pack2(-ss.z, ss.z), sn[3] = ptx::pack2(-ss.w, ss.w);
        } else if (turned) {
            const int j0 = low ? d0 : d0 - half;
            const uint64_t sg = low ? ptx::pack2(-1.f, -1.f) : ptx::pack2(1.f, 1.f);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float4 cc = *reinterpret_cast<const float4 *>(tab + j0 + 2 * e);
                const float4 ss = *reinterpret_cast<const float4 *>(tab + half + j0 + 2 * e);
                c[e] = ptx::pack2(cc.x, cc.y), c[e + 1] = ptx::pack2(cc.z, cc.w);
                sn[e] = mul2(sg, ptx::pack2(ss.x, ss.y)), sn[e + 1] = mul2(sg, ptx::pack2(ss.z, ss.w));
            }
        }
        // a query row's factors: weight times cosine, and the partner's weight times sine
        uint64_t qa[4], qb[4];
        pairs4(wq, qa, false);
        pairs4(wqo, qb, INTER);
#pragma unroll
        for (int e = 0; e < 4; ++e) qa[e] = mul2(qa[e], c[e]), qb[e] = mul2(qb[e], sn[e]);
        uint16_t *qrow = a.q_out + (int64_t)m.row * a.hq * D + d0;
        for (int h = warp * RPP + sub; h - sub < nrow; h += kTokWarps * RPP) {
            const bool in = h < nrow, is_q = h < a.hq, is_v = h >= a.hq + a.hkv;
            uint4 u = make_uint4(0, 0, 0, 0), uo = u;
            if (in) {
                u = *reinterpret_cast<const uint4 *>(rows + h * D + d0);
                uo = *reinterpret_cast<const uint4 *>(rows + h * D + o0);
            }
            if (__any_sync(0xffffffffu, in && !is_v)) {
                // z = (x w c + x' w' s) / sqrt(mean(x^2) + eps), x' and w' of the pair's other member
                uint64_t x[4], xo[4], z[4];
                pairs4(u, x, false);
                pairs4(uo, xo, INTER);
                float inv = 1.f;
                if (a.qw || a.kw) {
                    float ss = squares(x);
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    if (is_q ? a.qw : a.kw) inv = inverse_norm(ss, 1.f / D, a.eps);
                }
                if (__all_sync(0xffffffffu, is_q)) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[e] = turn2(x[e], qa[e], xo[e], qb[e]);
                } else {
                    uint64_t w[4], wo[4];
                    pairs4(is_q ? wq : wk, w, false);
                    pairs4(is_q ? wqo : wko, wo, INTER);
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[e] = turn2(x[e], mul2(w[e], c[e]), xo[e], mul2(wo[e], sn[e]));
                }
                if (a.rot < D && !turned) {  // (0 times an infinity is no number)
                    uint64_t w[4];
                    pairs4(is_q ? wq : wk, w, false);
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[e] = mul2(x[e], w[e]);
                }
                if (!is_v) u = finish(z, inv);
            }
            if (!in) continue;
            if (is_q) {
                *reinterpret_cast<uint4 *>(qrow + h * D) = u;
                if (m.ring >= 0) *reinterpret_cast<uint4 *>(a.ring + m.ring + h * a.ring_head + d0) = u;
            } else {
                const int g = is_v ? h - a.hq - a.hkv : h - a.hq;
                *reinterpret_cast<uint4 *>((is_v ? a.vp : a.kp) + m.page + g * a.head_stride + d0) = u;
            }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh->empty[st]));
        if (++st == (uint32_t)stages) st = 0, ph ^= 1;
    }
}

template <int D>
cudaError_t launch(const AppArgs &a, cudaStream_t st)
{
    const size_t head = (sizeof(TokShared) + 127) / 128 * 128;
    const int sb = tok_stage_bytes(a.hq, a.hkv, D, a.rot);
    // As many CTAs per SM, up to four, as hold a token each: it is their warps that count, more than the tokens
    // staged.  Fewer than two (more than about 435 head rows of 128): the other kernel.  Measured, 4096 tokens,
    // at 4 / 3 / 2 / 1 CTAs with what then fits, and the other kernel (us): 64 and 2 x 64 heads of 128 (1, 1, 2
    // and 4 tokens) 88.3 / 102 / 119 / 209, 135; 192 and 2 x 24 - / 132 / 181 / 279, 177; 256 and 2 x 64
    // - / - / 270 / 429, 278; 320 and 2 x 80 - / - / - / 582, 346.
    int stages = 0, per_sm = 4;
    for (; per_sm > 1; --per_sm) {
        const size_t room = per_sm == 4 ? 54 * 1024 : per_sm == 3 ? 74 * 1024 : kTokMaxSmem;
        stages = (int)((room - head) / sb);
        if (stages > 0) break;
    }
    if ((int64_t)a.rows * (a.hq + 2 * a.hkv) <= kSmallRows || stages == 0) {
        constexpr int RPP = 32 / (D / 8), WPC = kAppThreads / 32;
        const int parts = (a.hq + 2 * a.hkv + RPP - 1) / RPP;
        if (parts > 65535) return cudaErrorInvalidConfiguration;
        const dim3 grid((unsigned)(((int64_t)a.rows + WPC - 1) / WPC), (unsigned)parts);
        const auto kern = a.inter ? append_kernel<D, true> : append_kernel<D, false>;
        return launch_dependent(kern, grid, kAppThreads, 0, st, a);
    }
    if (stages > kTokMaxStages) stages = kTokMaxStages;
    const size_t smem = head + (size_t)stages * sb;
    const auto kern = a.inter ? append_staged_kernel<D, true> : append_staged_kernel<D, false>;
    // (one limit for every shape: it is the kernel's, and another host thread may set it ahead of this launch)
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTokMaxSmem);
    int dev = 0, sms = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int grid = a.rows < sms * per_sm ? a.rows : sms * per_sm;
    return launch_dependent(kern, dim3((unsigned)grid), kTokThreads, smem, st, a, stages);
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
    const Stall dbg = debug_stall(kTokTimeoutNs);
    a.stall = dbg.on;
    a.wait_ns = dbg.wait_ns;
    a.n = t->n;
    a.rows = t->rows;
    a.num_blocks = c->num_blocks;
    a.hq = c->num_q_heads;
    a.hkv = c->num_kv_heads;
    a.n_pos = r->rot_dim > 0 ? r->n_pos : 1;
    a.rot = r->rot_dim;
    a.inter = r->interleaved;
    return D == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace kara
