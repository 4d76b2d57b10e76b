// Decode attention over the 8-bit cache: one query per sequence and head,
//     o_h = sum_x softmax_x(<q_h, k_x> / sqrt(D)) v_x,   k_x, v_x = code * |scale|.
//
// Bound by HBM, at half the bytes of the bf16 cache, so twice as many keys pass through
// an SM in the same time.  The frame is that of the bf16 kernel: one CTA per (sequence, KV
// head, split of 1024 keys or fewer); a producer warp streams the split's K, then its V, through a
// ring of 4 KB stages by TMA; four consumer warps turn 16 keys at a time into two small
// matrix products on the warp-level MMA,
//     S^T[16 keys][8 heads] = K[16][D] . Q^T[D][8],   O^T[D][8] += V^T[D][16] . P^T[16][8].
//
// What the 8 bits change:
//   * The operands are f16, in which every e4m3 code is exact: one conversion per two
//     codes, straight from what ldmatrix delivers.  A 16-bit element of ldmatrix is two
//     codes.  For K these are neighbouring dims of a key, and the order of the dims in
//     the product is free, so Q's fragments are loaded to match.  For V (transposed) they
//     are two dims of one key; one byte permutation pairs the keys, and the even dims
//     become the upper eight rows of the product and the odd ones the lower.
//   * Queries are scaled by a power of two for each head so that their largest element is
//     in [2^14, 2^15): bf16 values down to 2^-29 of it are exact in f16, and smaller ones
//     off by 2^-39 of it at most.
//   * K's scales multiply the logits, V's the weights, which then are brought to f16
//     with a power of two for each head that puts the largest of a split in
//     [2^14, 2^15): half of an f16 step, 2^-11 of a weight, for those within 2^-29 of the
//     largest (times its block's scale), 2^-39 of the largest for smaller ones.  So keys that
//     share little weight beside one that takes nearly all keep their digits; without the
//     factor, weights below 2^-14 would lose theirs.
// Softmax, sums and the merge of the splits are fp32; the output is rounded to bf16 once.
//
// 128 sequences of 2048 to 16384 keys, 40/8 heads of 128: 457 us, 5.9 TB/s (0.87 of the copy rate); without the
// products and the softmax the loads alone take 423.  ALU pipe 42 %, issue slots 44 %.  Not better: e4m3 operands
// with K = 32 (478, more registers), splits of 2048 keys, 12 stages, stages of 8 KB.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kara_cache8.cuh"
#include "kara_sm100.cuh"
#include "kara_tokens.cuh"

namespace kara {

namespace {

constexpr int kSplit = 1024;        // keys per CTA, at most
constexpr int kBlk = 16;            // tokens per cache block (the supported block size)
constexpr int kBlocks = kSplit / kBlk;
constexpr int kNC = 4;              // consumer warps
constexpr int kThreads = 32 * (1 + kNC);
constexpr int kStages = 8;          // ring of stages in flight
constexpr int kStageBytes = 4096;
constexpr int kLs = kSplit + 8;     // row stride of the logits (floats): the weight fragments load conflict-free
constexpr uint64_t kTimeoutNs = 1000000000ull;  // 1 s: a stage normally lands in microseconds
// Stages go to the consumer warps round-robin and waits are by phase parity, which tells
// only two neighbouring phases apart: a warp may wait for use j of a stage only after it
// has seen use j - kStages complete, so both uses must be its own.
static_assert(kStages % kNC == 0, "each stage is reused by the same consumer warp");

struct Decode8Args {
    int32_t layer, num_blocks, hkv, hq;
    const int32_t *len;
    const int32_t *bt;
    int32_t bt_stride, split, max_splits;
    const uint16_t *q;   // [n][hq][D]
    const float *k_scale, *v_scale;  // [num_blocks][hkv], at the call's layer
    float *part;         // [n][hq][max_splits][D]
    float2 *stat;        // [n][hq][max_splits]: (max, sum) in the log2 domain
    uint16_t *out;       // [n][hq][D]
    int32_t *err;
    float scale2;        // log2(e) / sqrt(D)
    int32_t stall;       // debug: the producer issues nothing (see debug_stall)
    uint64_t wait_ns;    // limit of the waits on progress
};

__device__ __forceinline__ bool length_ok(const Decode8Args &a, int32_t L)
{
    return L >= 0 && ((int64_t)L + kBlk - 1) / kBlk <= a.bt_stride;
}

// Barriers and per-split tables of one CTA (after the ring and the logits in
// dynamic shared memory).
struct Shared {
    uint64_t full[kStages], empty[kStages];
    int32_t blk[kBlocks];             // physical ids of the split's blocks; -1: outside the pool
    float ks[kBlocks], vs[kBlocks];   // their scales
    float most[kNC][8], sum[kNC][8], top[kNC][8];  // each warp's part: largest logit (in the log2 domain), sum
                                                   // of weights, largest weight times scale
    int32_t abort;
};

// The warps' parts of a head's value, joined in their order.
template <class F>
__device__ __forceinline__ float over_warps(const float (&x)[kNC][8], int h, F join)
{
    float v = x[0][h];
#pragma unroll
    for (int w = 1; w < kNC; ++w) v = join(v, x[w][h]);
    return v;
}

// Bounded wait on phase `parity` of `bar`.  Gives up after limit_ns, or when
// another warp of the CTA gave up, recording KARA_ETIMEOUT.
__device__ bool dwait(uint32_t bar, uint32_t parity, Shared *sh, int32_t *err, uint64_t limit_ns,
                      bool honour_abort = true)
{
    uint64_t t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if ((it & 255u) == 255u) {
            if (honour_abort && *(volatile int32_t *)&sh->abort) return false;
            const uint64_t now = ptx::globaltimer();
            if (t0 == 0) {
                t0 = now;
            } else if (now - t0 > limit_ns) {
                set_err(err, KARA_ETIMEOUT);
                *(volatile int32_t *)&sh->abort = 1;
                return false;
            }
        }
    }
}

// ---- warp-level tensor-core operands -------------------------------------------
// Four 8x8 tiles of 16-bit elements from shared memory; lanes 8i..8i+7 give the row
// addresses of tile i, which lands in r[i].
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// The same, each tile transposed on the way.
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// d += A[16x16] . B[16x8], f16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The power of two that brings a largest magnitude x into [2^14, 2^15), and its inverse
// (both normal: an x below 2^-112 stays below).
__device__ __forceinline__ void to_f16_range(float x, float &up, float &down)
{
    const int e = min(max(127 + 14 + 127 - (int)(__float_as_uint(x) >> 23), 1), 253);
    up = __uint_as_float((uint32_t)e << 23);
    down = __uint_as_float((uint32_t)(254 - e) << 23);
}

// Dynamic shared memory: 1 KB of alignment slack, ring[kStages] of stages (blocks of 16
// rows of D codes, swizzled by their row size), logit[G][kLs] fp32 (logits, then weights,
// then the consumers' partial outputs), Shared.
// Four CTAs per SM up to G = 5; wider groups' logits leave room for three.
template <int G>
constexpr int min_ctas() { return G >= 6 ? 3 : 4; }  // (few_ctas counts on it)

template <int G>
constexpr size_t smem_bytes()
{
    return 1024 + (size_t)kStages * kStageBytes + sizeof(float) * G * kLs + sizeof(Shared);
}

// The weighted sum of a block of V: chunks of 16 dims, even dims in the upper eight rows of the product, odd dims in
// the lower; MASKED: keys 2tq, 2tq + 1 and those eight further on under lo and hi.
template <int NC, bool MASKED>
__device__ __forceinline__ void weigh(float (&acc)[NC][4], uint32_t sb, uint32_t b0, uint32_t b1, uint32_t lo, uint32_t hi)
{
#pragma unroll
    for (int c = 0; c < NC; c += 2) {
        uint32_t r[4];
        ldsm_x4_t(sb ^ (c << 4), r);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // (two dims of a key, two dims of the next) -> (a dim of both keys, the other of both)
            const uint32_t u = __byte_perm(MASKED ? r[2 * e] & lo : r[2 * e], 0u, 0x3120);
            const uint32_t v = __byte_perm(MASKED ? r[2 * e + 1] & hi : r[2 * e + 1], 0u, 0x3120);
            mma_16816(acc[c + e], f16_of_e4m3x2(u), f16_of_e4m3x2(u >> 16), f16_of_e4m3x2(v),
                      f16_of_e4m3x2(v >> 16), b0, b1);
        }
    }
}

template <int D, int G>
__global__ void __launch_bounds__(kThreads, min_ctas<G>())
    decode8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const Decode8Args a)
{
    constexpr int BB = kBlk * D;             // bytes of one (block, head) slice
    constexpr int BPS = kStageBytes / BB;    // blocks of a stage
    constexpr int NC = D / 16;               // 16-dim chunks of a row
    static_assert(G <= 8, "heads per group: one n8 tile");
    static_assert(kNC * D <= kLs, "partial outputs fit in the logit area");
    extern __shared__ uint8_t dsm_raw[];
    // the swizzle pattern is taken from the address
    uint8_t *ring = dsm_raw + ((1024u - (ptx::smem_u32(dsm_raw) & 1023u)) & 1023u);
    float *logit = reinterpret_cast<float *>(ring + kStages * kStageBytes);  // [G][kLs]
    Shared *sh = reinterpret_cast<Shared *>(logit + G * kLs);

    // launched as a programmatic dependent of whatever precedes it on the stream:
    // nothing global is read before that grid has completed
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int sp = blockIdx.z, g = blockIdx.x, s = blockIdx.y;
    const int32_t L = a.len[s];
    const bool ok_len = length_ok(a, L);
    if (!ok_len || L == 0) {
        if (sp == 0) {
            if (!ok_len && g == 0 && threadIdx.x == 0) set_err(a.err, KARA_EINVAL);
            uint32_t *o = reinterpret_cast<uint32_t *>(a.out + ((int64_t)s * a.hq + g * G) * D);
            for (int i = threadIdx.x; i < G * D / 2; i += kThreads) o[i] = 0u;
        }
        return;
    }
    const int32_t k0 = sp * a.split;
    if (k0 >= L) return;
    const int nk = min(a.split, L - k0);
    const int nb = (nk + kBlk - 1) / kBlk, ns = (nb + BPS - 1) / BPS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    for (int i = threadIdx.x; i < nb; i += kThreads) {
        int32_t id = a.bt[(int64_t)s * a.bt_stride + k0 / kBlk + i];
        if (id < 0 || id >= a.num_blocks) {
            set_err(a.err, KARA_EBADBLOCK);
            id = -1;
        }
        sh->blk[i] = id;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(ptx::smem_u32(&sh->full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&sh->empty[i]), 1);
        }
        sh->abort = 0;
        ptx::fence_mbarrier_init();
    }
    __syncthreads();

    if (warp == 0) {
        // ---------------- producer: K stages 0..ns-1, then V stages --------------
        if (lane == 0) {
            int issued = 0;
            for (int j = 0; j < (a.stall ? 0 : 2 * ns); ++j) {
                const int st = j % kStages, b0 = (j < ns ? j : j - ns) * BPS;
                if (!dwait(ptx::smem_u32(&sh->empty[st]), ((j / kStages) & 1) ^ 1, sh, a.err, a.wait_ns)) break;
                const uint32_t fb = ptx::smem_u32(&sh->full[st]);
                const CUtensorMap *m = j < ns ? &kmap : &vmap;
                int32_t id[BPS];
                int live = 0;
#pragma unroll
                for (int b = 0; b < BPS; ++b) {
                    id[b] = b0 + b < nb ? sh->blk[b0 + b] : -1;
                    live += id[b] >= 0;
                }
                ptx::mbar_arrive_expect_tx(fb, live * BB);
#pragma unroll
                for (int b = 0; b < BPS; ++b)
                    if (id[b] >= 0)
                        ptx::tma_load_5d(ptx::smem_u32(ring + st * kStageBytes + b * BB), m, fb, 0, 0, g, id[b],
                                         a.layer);
                issued = j + 1;
            }
            // every copy issued has landed before the CTA's shared memory is released
            for (int j = max(0, issued - kStages); j < issued; ++j)
                dwait(ptx::smem_u32(&sh->full[j % kStages]), (j / kStages) & 1, sh, a.err, kTimeoutNs, false);
        }
        return;
    }

    // ---------------- consumers ----------------------------------------------------
    // MMA fragment coordinates: row group r8 = lane / 4, thread tq = lane % 4.
    const int cw = warp - 1, ctid = threadIdx.x - 32;
    const int r8 = lane >> 2, tq = lane & 3, h0 = 2 * tq;

    for (int i = ctid; i < 2 * nb; i += kNC * 32) {
        const int b = i < nb ? i : i - nb;
        const int32_t id = sh->blk[b];
        const float f = id < 0 ? 0.f : fabsf((i < nb ? a.k_scale : a.v_scale)[(int64_t)id * a.hkv + g]);
        (i < nb ? sh->ks : sh->vs)[b] = f;
    }
    // Logits' B operand Q^T[16 dims][8 heads]: of head r8 the dims that this thread's
    // codes of a 16-dim chunk have, 4tq..4tq+3; heads past G are zero.
    uint32_t qb[NC][2];
    float f0, f1;  // of heads h0 and h0 + 1: what their logits are to be multiplied by
    {
        const uint2 *qh = reinterpret_cast<const uint2 *>(a.q + ((int64_t)s * a.hq + g * G + min(r8, G - 1)) * D);
        float top = 0.f, up, down;
        uint2 w[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            w[c] = r8 < G ? __ldg(qh + c * 4 + tq) : make_uint2(0u, 0u);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t u = e & 2 ? w[c].y : w[c].x;
                const float x = fabsf(__uint_as_float(e & 1 ? u & 0xffff0000u : u << 16));
                if (finite(x)) top = fmaxf(top, x);
            }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        to_f16_range(top, up, down);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            qb[c][0] = f16x2(__uint_as_float(w[c].x << 16) * up, __uint_as_float(w[c].x & 0xffff0000u) * up);
            qb[c][1] = f16x2(__uint_as_float(w[c].y << 16) * up, __uint_as_float(w[c].y & 0xffff0000u) * up);
        }
        f0 = __shfl_sync(0xffffffffu, down, h0 * 4) * a.scale2;
        f1 = __shfl_sync(0xffffffffu, down, h0 * 4 + 4) * a.scale2;
    }
    ptx::named_barrier(1, kNC * 32);

    // this lane's row of the ldmatrix tiles: tiles 0 and 1 are rows 0-7 and 8-15 of a chunk, 2 and 3 of
    // the next; 16-byte chunk c of row t lies at chunk c ^ (t & 7) (D = 64: c ^ (t / 2 & 3))
    const int lt = lane & 15, lc = lane >> 4, lx = D == 128 ? lt & 7 : lt >> 1 & 3;
    const uint32_t lane_at = ptx::smem_u32(ring) + lt * D + ((lc ^ lx) << 4);  // chunk c + lc (c even): this ^ c << 4

    // ---- logits
    float m0 = -INFINITY, m1 = -INFINITY;  // the largest of heads h0 and h0 + 1 (passing over a NaN)
    for (int i = cw; i < ns; i += kNC) {
        const int st = i % kStages;
        if (!dwait(ptx::smem_u32(&sh->full[st]), (i / kStages) & 1, sh, a.err, a.wait_ns)) break;
        float acc[BPS][4];
#pragma unroll
        for (int b = 0; b < BPS; ++b) {
            const uint32_t sb = lane_at + st * kStageBytes + b * BB;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[b][e] = 0.f;
#pragma unroll
            for (int c = 0; c < NC; c += 2) {
                uint32_t r[4];
                ldsm_x4(sb ^ (c << 4), r);
                mma_16816(acc[b], f16_of_e4m3x2(r[0]), f16_of_e4m3x2(r[1]), f16_of_e4m3x2(r[0] >> 16),
                          f16_of_e4m3x2(r[1] >> 16), qb[c][0], qb[c][1]);
                mma_16816(acc[b], f16_of_e4m3x2(r[2]), f16_of_e4m3x2(r[3]), f16_of_e4m3x2(r[2] >> 16),
                          f16_of_e4m3x2(r[3] >> 16), qb[c + 1][0], qb[c + 1][1]);
            }
        }
        // the codes are in registers: hand the stage back
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh->empty[st]));
        // acc = S^T at (key r8, heads h0, h0 + 1) and (key r8 + 8, same heads)
#pragma unroll
        for (int b = 0; b < BPS; ++b) {
            const int blk = i * BPS + b, x = blk * kBlk + r8;
            if (x >= nk) continue;
            const bool in = sh->blk[blk] >= 0;  // a block outside the pool: zeros
            const float f = sh->ks[blk];
            const auto put = [&](int h, int y, float l, float &most) {
                logit[h * kLs + y] = l;
                most = fmaxf(most, l);
            };
            if (h0 < G) {
                put(h0, x, in ? acc[b][0] * f * f0 : 0.f, m0);
                if (x + 8 < nk) put(h0, x + 8, in ? acc[b][2] * f * f0 : 0.f, m0);
            }
            if (h0 + 1 < G) {
                put(h0 + 1, x, in ? acc[b][1] * f * f1 : 0.f, m1);
                if (x + 8 < nk) put(h0 + 1, x + 8, in ? acc[b][3] * f * f1 : 0.f, m1);
            }
        }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
    }
    if (lane < 4) sh->most[cw][h0] = m0, sh->most[cw][h0 + 1] = m1;
    ptx::named_barrier(1, kNC * 32);

    // ---- softmax: a quarter of the keys to a warp, all heads; what stays are the weights times V's scales.
    // (With a warp for a head three wait for the fifth head's, and the ring is full meanwhile.)
    {
        float z[G], top[G];
#pragma unroll
        for (int h = 0; h < G; ++h) {
            const float m = over_warps(sh->most, h, [](float x, float y) { return fmaxf(x, y); });
            const float ref = m == -INFINITY ? 0.f : m;
            float *lr = logit + h * kLs;
            z[h] = 0.f, top[h] = 0.f;
            for (int x = cw * (a.split / kNC) + lane; x < min(nk, (cw + 1) * (a.split / kNC)); x += 32) {
                const float p = ptx::ex2(lr[x] - ref), w = p * sh->vs[x / kBlk];
                lr[x] = w;
                z[h] += p;
                top[h] = fmaxf(top[h], w);
            }
            for (int x = nk + ctid; x < ns * BPS * kBlk; x += kNC * 32) lr[x] = 0.f;  // rows past the end weigh 0
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int h = 0; h < G; ++h) {
                z[h] += __shfl_xor_sync(0xffffffffu, z[h], o);
                top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], o));
            }
        if (lane == 0)
#pragma unroll
            for (int h = 0; h < G; ++h) sh->sum[cw][h] = z[h], sh->top[cw][h] = top[h];
    }
    ptx::named_barrier(1, kNC * 32);

    // ---- weighted sum: even dims of a chunk in the upper eight rows, odd dims in the lower
    float acc[NC][4];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[c][e] = 0.f;
    const auto most = [](float x, float y) { return fmaxf(x, y); };
    float up, unused;
    to_f16_range(over_warps(sh->top, min(r8, G - 1), most), up, unused);
    for (int i = cw; i < ns; i += kNC) {
        const int j = ns + i, st = j % kStages;
        if (!dwait(ptx::smem_u32(&sh->full[st]), (j / kStages) & 1, sh, a.err, a.wait_ns)) break;
#pragma unroll
        for (int b = 0; b < BPS; ++b) {
            const int blk = i * BPS + b;
            if (blk >= nb || sh->blk[blk] < 0) continue;
            // weights of head r8 for keys 2tq, 2tq+1 and 2tq+8, 2tq+9 of the block
            uint32_t b0 = 0u, b1 = 0u;
            if (r8 < G) {
                const float *w = logit + r8 * kLs + blk * kBlk + 2 * tq;
                const float2 x = *reinterpret_cast<const float2 *>(w), y = *reinterpret_cast<const float2 *>(w + 8);
                b0 = f16x2(x.x * up, x.y * up), b1 = f16x2(y.x * up, y.y * up);
            }
            // rows of the last block past the end hold whatever the block held (NaN
            // included): their halves of the fragments are zeroed
            const int tmax = nk - blk * kBlk;
            const uint32_t sb = lane_at + st * kStageBytes + b * BB;
            if (tmax >= kBlk) {
                weigh<NC, false>(acc, sb, b0, b1, 0u, 0u);
            } else {
                const uint32_t lo = (2 * tq < tmax ? 0x0000ffffu : 0u) | (2 * tq + 1 < tmax ? 0xffff0000u : 0u);
                const uint32_t hi = (2 * tq + 8 < tmax ? 0x0000ffffu : 0u) | (2 * tq + 9 < tmax ? 0xffff0000u : 0u);
                weigh<NC, true>(acc, sb, b0, b1, lo, hi);
            }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&sh->empty[st]));
    }
    // every consumer is done with the weights: the logit area takes the partial
    // outputs red[kNC][G][D], summed below over the warps in a fixed order
    ptx::named_barrier(1, kNC * 32);
    float *red = logit;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int d = c * 16 + 2 * r8;  // acc[c] = O^T at (dims d, d + 1; heads h0, h0 + 1)
        if (h0 < G) *reinterpret_cast<float2 *>(red + (cw * G + h0) * D + d) = make_float2(acc[c][0], acc[c][2]);
        if (h0 + 1 < G)
            *reinterpret_cast<float2 *>(red + (cw * G + h0 + 1) * D + d) = make_float2(acc[c][1], acc[c][3]);
    }
    ptx::named_barrier(1, kNC * 32);
    for (int x = 2 * ctid; x < G * D; x += 2 * kNC * 32) {
        const int h = x / D, d = x % D;
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kNC; ++w) {
            const float2 y = *reinterpret_cast<const float2 *>(red + (w * G + h) * D + d);
            v.x += y.x, v.y += y.y;
        }
        float up, f;
        to_f16_range(over_warps(sh->top, h, most), up, f);
        const int64_t row = (int64_t)s * a.hq + g * G + h, idx = row * a.max_splits + sp;
        const auto sum = [&] { return over_warps(sh->sum, h, [](float x, float y) { return x + y; }); };
        v.x *= f, v.y *= f;
        if (L <= a.split) {  // nothing to merge
            const float z = sum();
            *reinterpret_cast<uint32_t *>(a.out + row * D + d) = bf16x2(v.x / z, v.y / z);
            continue;
        }
        *reinterpret_cast<float2 *>(a.part + idx * D + d) = v;
        if (d == 0) a.stat[idx] = make_float2(over_warps(sh->most, h, most), sum());
    }
    // the merge kernel may be scheduled once every CTA of this grid got here
    // or exited; it still waits for this grid's completion before reading
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// out[s][h] = sum_sp part * 2^(m_sp - M) / sum_sp z_sp * 2^(m_sp - M), splits in order.  (Sequences of one split
// have written theirs, and tables that hold no more need no merge: a sequence of 256 keys takes 4.7 us captured, with it 6.4.)
template <int D>
__global__ void __launch_bounds__(D) decode8_merge_kernel(const Decode8Args a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int h = blockIdx.x, s = blockIdx.y, d = threadIdx.x;
    const int32_t L = a.len[s];
    if (!length_ok(a, L) || L <= a.split) return;  // written already
    const int nsp = (L + a.split - 1) / a.split;
    const int64_t row = (int64_t)s * a.hq + h, base = row * a.max_splits;
    float M = -INFINITY;
    for (int sp = 0; sp < nsp; ++sp) M = fmaxf(M, a.stat[base + sp].x);
    const float ref = M == -INFINITY ? 0.f : M;
    float den = 0.f, num = 0.f;
    for (int sp = 0; sp < nsp; ++sp) {
        const float2 st = a.stat[base + sp];
        const float w = exp2f(st.x - ref);
        den = fmaf(st.y, w, den);
        num = fmaf(a.part[(base + sp) * D + d], w, num);
    }
    const float o = num / den, next = __shfl_down_sync(0xffffffffu, o, 1);
    if ((d & 1) == 0) *reinterpret_cast<uint32_t *>(a.out + row * D + d) = bf16x2(o, next);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <int D, int G>
cudaError_t launch_g(const CUtensorMap &km, const CUtensorMap &vm, const Decode8Args &a, dim3 grid, cudaStream_t st)
{
    const auto kern = decode8_kernel<D, G>;
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<G>());
    return e != cudaSuccess ? e : launch_dependent(kern, grid, kThreads, smem_bytes<G>(), st, km, vm, a);
}

template <int D>
cudaError_t launch(const CUtensorMap &km, const CUtensorMap &vm, const Decode8Args &a, int32_t n, cudaStream_t st)
{
    // split-major: CTAs past a short sequence's end (they exit at once) come last,
    // where they take slots the grid's tail leaves idle anyway
    const dim3 grid((unsigned)a.hkv, (unsigned)n, (unsigned)a.max_splits);
    cudaError_t e = cudaErrorInvalidValue;
    switch (a.hq / a.hkv) {
        case 1: e = launch_g<D, 1>(km, vm, a, grid, st); break;
        case 2: e = launch_g<D, 2>(km, vm, a, grid, st); break;
        case 3: e = launch_g<D, 3>(km, vm, a, grid, st); break;
        case 4: e = launch_g<D, 4>(km, vm, a, grid, st); break;
        case 5: e = launch_g<D, 5>(km, vm, a, grid, st); break;
        case 6: e = launch_g<D, 6>(km, vm, a, grid, st); break;
        case 7: e = launch_g<D, 7>(km, vm, a, grid, st); break;
        case 8: e = launch_g<D, 8>(km, vm, a, grid, st); break;
    }
    if (e != cudaSuccess || a.max_splits == 1) return e;
    return launch_dependent(decode8_merge_kernel<D>, dim3((unsigned)a.hq, (unsigned)n), D, 0, st, a);
}

}  // namespace

// Keys per CTA: 1024, which serve full batches best, half or a quarter of it while the grid would leave half of the
// places for CTAs on the SMs empty, the merge has no more than 64 splits to go through, and a table holds more than
// 512 keys: a single split needs no merge (256 keys: 5.6 us with one, 4.7 without).  (us, captured, with splits of
// 256, 512 and 1024 keys, the choice in brackets; 40/8 heads of 128: one sequence of 1000 keys [8.8] 11.9 15.2, of
// 4000 [10.5] 12.5 18.6, of 16000 [16.9] 16.2 20.3, of 64000 63 44 [33]; 4 of 4000 [13.5] 13.8 18.9, 8 of 4000 19.7 [16.5]
// 20.2, 16 of 4000 38 32 [28]; 16/2 heads: one of 8000 [12.4] 14.5 20.1, of 64000 38 26.7 [26.0], 32 of 4000 28.8 24.7 [21.8].
// Splits of 128 keys bring one sequence of 1000 to 8.0, and one of 4000 to 11.4.)
constexpr int kLeast = 256, kMostSplits = 64;

static int64_t splits_of(int32_t bt_stride, int split) { return ((int64_t)bt_stride * kBlk + split - 1) / split; }

// CTAs that fill half of the places on the GB300's 152 SMs (a constant: the workspace's size, which follows from it, is
// asked for without a device too).
static int64_t few_ctas(const kara_cache8 *c) { return 152 * (c->num_q_heads / c->num_kv_heads >= 6 ? 3 : 4) / 2; }

static int split_of(const kara_cache8 *c, int32_t n, int32_t bt_stride)
{
    const int64_t rows = (int64_t)n * c->num_kv_heads;
    int split = kSplit;
    if (splits_of(bt_stride, 2 * kLeast) == 1) return split;
    while (split > kLeast && rows * splits_of(bt_stride, split) <= few_ctas(c) &&
           splits_of(bt_stride, split / 2) <= kMostSplits)
        split /= 2;
    return split;
}

int decode8_max_splits(const kara_cache8 *c, int32_t n, int32_t bt_stride)
{
    return (int)splits_of(bt_stride, split_of(c, n, bt_stride));
}

// Enough for this batch and every smaller one, whose splits may be more: halved splits are at most twice few_ctas.
size_t decode8_workspace_bytes(const kara_cache8 *c, int32_t n, int32_t bt_stride)
{
    const int64_t rows = (int64_t)n * c->num_kv_heads, least = rows * splits_of(bt_stride, kSplit);
    const int64_t most = rows * splits_of(bt_stride, kLeast), halved = most < 2 * few_ctas(c) ? most : 2 * few_ctas(c);
    const size_t npart = (size_t)(least > halved ? least : halved) * (c->num_q_heads / c->num_kv_heads);
    return align256(npart * c->head_dim * sizeof(float)) + align256(npart * sizeof(float2));
}

cudaError_t launch_decode8(const kara_cache8 *c, int32_t layer, int32_t n, const int32_t *len, const int32_t *bt,
                           int32_t bt_stride, const void *q, void *out, void *ws, int32_t *err, cudaStream_t st)
{
    CUtensorMap km, vm;
    cudaError_t e = pool_map8(&km, c->k, c, true);
    if (e == cudaSuccess) e = pool_map8(&vm, c->v, c, true);
    if (e != cudaSuccess) return e;
    const int64_t scales = (int64_t)layer * c->num_blocks * c->num_kv_heads;
    Decode8Args a;
    a.layer = layer;
    a.num_blocks = c->num_blocks;
    a.hkv = c->num_kv_heads;
    a.hq = c->num_q_heads;
    a.len = len;
    a.bt = bt;
    a.bt_stride = bt_stride;
    a.split = split_of(c, n, bt_stride);
    a.max_splits = decode8_max_splits(c, n, bt_stride);
    a.q = static_cast<const uint16_t *>(q);
    a.k_scale = c->k_scale + scales;
    a.v_scale = c->v_scale + scales;
    const size_t npart = (size_t)n * a.hq * a.max_splits;
    a.part = static_cast<float *>(ws);
    a.stat = reinterpret_cast<float2 *>(static_cast<char *>(ws) + align256(npart * c->head_dim * sizeof(float)));
    a.out = static_cast<uint16_t *>(out);
    a.err = err;
    a.scale2 = 1.4426950408889634f / sqrtf((float)c->head_dim);
    const Stall dbg = debug_stall(kTimeoutNs);
    a.stall = dbg.on;
    a.wait_ns = dbg.wait_ns;
    return c->head_dim == 128 ? launch<128>(km, vm, a, n, st) : launch<64>(km, vm, a, n, st);
}

}  // namespace kara
