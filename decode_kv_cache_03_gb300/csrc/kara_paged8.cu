// The compression step's copies on the 8-bit cache: the windows' keys back in bf16 for the
// scorer (expand), and the gather-compaction (compact).
//
// Follows the gist.science summary of Kara (arXiv 2607.01237), section "3. KvLLM Framework
// and Periodic Compression", as the bf16 compaction does: the plan, the checks of fresh ids
// and kept rows and the table commit are that one's.  What is new is that the 16 rows of a
// rebuilt block come from up to 16 blocks with scales of their own: with x = code * |scale|
// of the gathered rows,
//     s = the smallest power of two with max |x| <= 448 s,   code' = rn(x / s).
// Powers of two: x / s is exact unless it falls among e4m3's subnormals.
// Both are bound by HBM (a read and a write of every code, or of its bf16 value).  Expansion of 16 windows of
// 512 keys in 36 layers of 8 heads takes 140 us, the copy rate.  Compaction of 8 sequences (windows of
// 1024, 396 rows kept) in 40 layers takes 103.5 us: the copy about 84, at 0.9 of the copy rate, and the checks of kept rows and
// fresh ids, and the plan, ahead of it.
#include <cuda_fp16.h>

#include "kara_cache8.cuh"
#include "kara_plan.cuh"

namespace kara {
namespace {

constexpr int kBs = 16;  // tokens per cache block (the supported block size)
constexpr int kThreads = 256;
// Slices that an expanding thread has in flight (16 windows in 36 layers: 2, 4 and 8 take 145, 140 and 160 us).
constexpr int kSlices = 4;
// Warps of a compacting CTA, at most: its place is free again when the slowest is done (8 sequences in 40 layers:
// 16, 8, 4, 2 and 1 take 113, 108, 103.5, 103 and 103 us).
constexpr int kCopyWarps = 4;

struct Pool8 {
    const uint8_t *codes[2];
    const float *scale[2];
    int64_t layer_stride, block_stride, head_stride;
    int32_t num_blocks, hkv, heads;  // heads: layers * hkv

    // slice lh = layer * hkv + head of a block, and its scale
    __device__ __forceinline__ int64_t slice(int lh, int32_t blk) const
    {
        return lh / hkv * layer_stride + blk * block_stride + lh % hkv * head_stride;
    }
    __device__ __forceinline__ int64_t scale_at(int lh, int32_t blk) const
    {
        return ((int64_t)(lh / hkv) * num_blocks + blk) * hkv + lh % hkv;
    }
};

struct ExpandArgs {
    Pool8 in;
    uint16_t *out[2];
    int64_t layer_stride, block_stride, head_stride;  // of out, elements
    int32_t n, W, nw, bt_stride, pools;
    const int32_t *len, *bt;
    int32_t *out_table, *err;
};

// Block (x, y): block j of sequence s's window (x = s * nw + j), slices y * kSlices * SPB and on of all
// layers and heads (and of V after those of K).  A thread takes 16 codes of a slice.
template <int D>
__global__ void __launch_bounds__(kThreads) expand8_kernel(const ExpandArgs a)
{
    constexpr int SPB = kThreads / D;  // slices side by side (a slice: D threads)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s = blockIdx.x / a.nw, j = blockIdx.x % a.nw;
    const int32_t L = a.len[s];
    if (L < a.W || ((int64_t)L + kBs - 1) / kBs > a.bt_stride) {
        if (j == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_err(a.err, KARA_EINVAL);
        return;
    }
    const int32_t col = (L - a.W) / kBs + j;
    if (col >= (L + kBs - 1) / kBs) return;
    const int64_t entry = (int64_t)s * a.bt_stride + col;
    const int32_t id = a.bt[entry], to = blockIdx.x;
    const bool inside = id >= 0 && id < a.in.num_blocks;
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        if (!inside) set_err(a.err, KARA_EBADBLOCK);
        a.out_table[entry] = to;
    }
    const int part = threadIdx.x % D, row = part * 16 / D;
    const bool live = inside && (int64_t)col * kBs + row < L;
    const int first = blockIdx.y * kSlices * SPB + threadIdx.x / D, total = a.pools * a.in.heads;
    uint4 w[kSlices];
    float f[kSlices];
#pragma unroll
    for (int i = 0; i < kSlices; ++i) {
        const int lh = first + i * SPB, p = lh >= a.in.heads, h = p ? lh - a.in.heads : lh;
        w[i] = make_uint4(0, 0, 0, 0);
        f[i] = 0.f;
        if (live && lh < total) {
            w[i] = *reinterpret_cast<const uint4 *>(a.in.codes[p] + a.in.slice(h, id) + part * 16);
            f[i] = fabsf(a.in.scale[p][a.in.scale_at(h, id)]);
        }
    }
#pragma unroll
    for (int i = 0; i < kSlices; ++i) {
        const int lh = first + i * SPB, p = lh >= a.in.heads, h = p ? lh - a.in.heads : lh;
        if (lh >= total) break;
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        uint32_t r[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x[4];
            values4(u[e], x);
            r[2 * e] = bf16x2(x[0] * f[i], x[1] * f[i]);
            r[2 * e + 1] = bf16x2(x[2] * f[i], x[3] * f[i]);
        }
        uint4 *o = reinterpret_cast<uint4 *>(a.out[p] + h / a.in.hkv * a.layer_stride + to * a.block_stride +
                                             h % a.in.hkv * a.head_stride + part * 16);
        o[0] = make_uint4(r[0], r[1], r[2], r[3]);
        o[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}

struct CompactArgs {
    Pool8 in;
    uint8_t *codes[2];
    float *scale[2];
    const SeqPlan *plan;
    const int32_t *kept, *fresh, *bt;
    int64_t n_fresh;
    int32_t B, C, R, bt_stride;
    int32_t *err;
    // the last block to finish commits, if `done` counts them
    int32_t *done, *freed, *new_len, *table;
    Geo g;
};

// Largest magnitude among four codes, as 16-bit pairs of even and odd bytes: codes without their sign order
// like their values.
__device__ __forceinline__ uint32_t top_code(uint32_t top, uint32_t w)
{
    return __vmaxu2(top, __vmaxu2(w & 0x007f007fu, w >> 8 & 0x007f007fu));
}

// Codes times a power of two up to 2^15, or 0 (below 2^-24 it is): f16 holds every product exactly that does not
// round to code 0 anyway.
__device__ __forceinline__ uint32_t shift4(uint32_t w, __half2 f)
{
    const uint32_t lo = f16_of_e4m3x2(w & 0xffffu), hi = f16_of_e4m3x2(w >> 16);
    const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&lo), f);
    const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&hi), f);
    uint16_t a, b;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(a) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(b) : "r"(*reinterpret_cast<const uint32_t *>(&y)));
    return a | (uint32_t)b << 16;
}

// A warp rebuilds one block of one head, K and V (they come from the same rows): window blockIdx.x = (s * layers + l)
// * hkv + g, new block j.  The chain of loads plan, kept row, table entry, codes is long, and many warps hide it (one
// that took four blocks and looked up the next ones' rows ahead needed 111 registers: 162 us against 138).
// Conversions set the pace beside that (they run at 16 lanes a clock): the largest value is found on the
// codes, and rows whose scale stays are copied as they are.
template <int D>
__device__ __forceinline__ void rebuild(const CompactArgs &a)
{
    constexpr int LPR = D / 16, RPP = 32 / LPR, NP = kBs / RPP;  // lanes per row, rows per pass, passes
    const uint32_t window = blockIdx.x;
    const int lh = (int)(window % (uint32_t)a.in.heads), s = (int)(window / (uint32_t)a.in.heads);
    const int j = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int32_t failed = *(volatile const int32_t *)a.err;
    const SeqPlan p = a.plan[s];
    // nothing is written once an earlier kernel (plan, checks) recorded an error
    if (failed != 0 || p.p0 < 0 || j >= p.n_new || (int64_t)p.off_new + p.n_new > a.n_fresh) return;
    const int32_t dst = a.fresh[p.off_new + j];
    const int32_t *kept = a.kept + (int64_t)window * a.R, *bt = a.bt + (int64_t)s * a.bt_stride;
    const int c = lane % LPR, row = lane / LPR, x0 = (p.p0 + j) * kBs + row;
    int32_t id[NP], at[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int x = x0 + i * RPP;
        int old = x;
        if (x >= p.ws) old = x < p.ws + a.R ? p.ws + min(max(kept[x - p.ws], 0), a.C - 1) : p.L - a.B + (x - p.ws - a.R);
        at[i] = (old & (kBs - 1)) * D + c * 16;
        id[i] = x < p.Lnew ? max(bt[(uint32_t)old / kBs], -1) : -2;  // (-2: past the end)
    }
    if (dst < 0 || dst >= a.in.num_blocks) return;  // recorded by the check
    const int64_t head = a.in.slice(lh, 0), head_scale = a.in.scale_at(lh, 0);
    uint4 w[2][NP];
    float f[2][NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const bool in = id[i] >= 0 && id[i] < a.in.num_blocks;
        if (!in && id[i] != -2) set_err(a.err, KARA_EBADBLOCK);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            w[k][i] = make_uint4(0, 0, 0, 0);
            f[k][i] = 0.f;
            if (!in) continue;
            w[k][i] = *reinterpret_cast<const uint4 *>(a.in.codes[k] + head + id[i] * a.in.block_stride + at[i]);
            f[k][i] = a.in.scale[k][head_scale + (int64_t)id[i] * a.in.hkv];
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float top = 0.f;
        bool odd = false;  // a row of a block that may hold NaN codes
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            uint32_t t = top_code(top_code(top_code(top_code(0u, w[k][i].x), w[k][i].y), w[k][i].z), w[k][i].w);
            t = max(t & 0xffffu, t >> 16);
            float lo, hi;
            f32_of_f16x2(f16_of_e4m3x2(t), lo, hi);
            top = fmaxf(top, lo * f[k][i]);
            odd = odd || signbit(f[k][i]);
        }
        const bool marked = __any_sync(0xffffffffu, odd);
        if (__builtin_expect(marked, 0)) {  // again, value by value
            top = 0.f, odd = false;
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                float x[4];
                f[k][i] = fabsf(f[k][i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    values4(e == 0 ? w[k][i].x : e == 1 ? w[k][i].y : e == 2 ? w[k][i].z : w[k][i].w, x);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        odd = odd || x[v] != x[v];
                        top = fmaxf(top, fabsf(x[v]) * f[k][i]);  // (passes over a NaN)
                    }
                }
            }
            odd = __any_sync(0xffffffffu, odd);
        }
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
        const float sc = scale_for(top), inv = inverse_scale(sc);
        uint8_t *out = a.codes[k] + head + dst * a.in.block_stride + row * D + c * 16;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            // (2^17 at most for a row with a code that is not 0: 448 of the new scale against 2^-9 of the old one.  Rows of
            // zeros set no scale, and times an infinity they would be no numbers)
            const float ratio = fminf(f[k][i] * inv, 131072.f);
            if (ratio != 1.f) {
                const __half2 h = __float2half2_rn(fminf(ratio, 32768.f));
                w[k][i].x = shift4(w[k][i].x, h), w[k][i].y = shift4(w[k][i].y, h);
                w[k][i].z = shift4(w[k][i].z, h), w[k][i].w = shift4(w[k][i].w, h);
                if (ratio > 32768.f) {  // what is left of it
                    const __half2 g = __float2half2_rn(ratio * (1.f / 32768.f));
                    w[k][i].x = shift4(w[k][i].x, g), w[k][i].y = shift4(w[k][i].y, g);
                    w[k][i].z = shift4(w[k][i].z, g), w[k][i].w = shift4(w[k][i].w, g);
                }
            }
            if (id[i] != -2) *reinterpret_cast<uint4 *>(out + i * RPP * D) = w[k][i];
        }
        if (lane == 0) a.scale[k][head_scale + (int64_t)dst * a.in.hkv] = odd ? -sc : sc;
    }
}

template <int D>
__global__ void __launch_bounds__(32 * kCopyWarps, 8) compact8_kernel(const CompactArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    rebuild<D>(a);
    if (!a.done) return;
    __shared__ bool last;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(a.done, 1) == (int32_t)(gridDim.x * gridDim.y) - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    const int32_t error = *(volatile const int32_t *)a.err;
    for (int s = threadIdx.x >> 5; s < a.g.n; s += blockDim.x >> 5)
        commit_sequence(a.g, a.plan[s], error, a.fresh, a.freed, a.new_len, a.table, s, threadIdx.x & 31, 32);
}

Pool8 pool8(const kara_cache8 *c)
{
    Pool8 p;
    p.codes[0] = static_cast<const uint8_t *>(c->k), p.codes[1] = static_cast<const uint8_t *>(c->v);
    p.scale[0] = c->k_scale, p.scale[1] = c->v_scale;
    p.layer_stride = c->layer_stride, p.block_stride = c->block_stride, p.head_stride = c->head_stride;
    p.num_blocks = c->num_blocks, p.hkv = c->num_kv_heads;
    p.heads = c->num_layers * c->num_kv_heads;
    return p;
}

}  // namespace

cudaError_t launch_expand8(const kara_cache8 *c, const kara_cache *out, int32_t W, int32_t n, const int32_t *len,
                           const int32_t *bt, int32_t bt_stride, int32_t *out_table, int32_t *err, cudaStream_t st)
{
    ExpandArgs a;
    a.in = pool8(c);
    a.out[0] = static_cast<uint16_t *>(out->k), a.out[1] = static_cast<uint16_t *>(out->v);
    a.layer_stride = out->layer_stride, a.block_stride = out->block_stride, a.head_stride = out->head_stride;
    a.n = n, a.W = W, a.nw = W / kBs + 1, a.bt_stride = bt_stride;
    a.pools = out->v == out->k ? 1 : 2;
    a.len = len, a.bt = bt, a.out_table = out_table, a.err = err;
    const int per = kSlices * (kThreads / c->head_dim);
    const int64_t x = (int64_t)n * a.nw, y = ((int64_t)a.pools * a.in.heads + per - 1) / per;
    if (x > 0x7fffffffLL || y > 65535) return cudaErrorInvalidConfiguration;
    const auto kern = c->head_dim == 128 ? expand8_kernel<128> : expand8_kernel<64>;
    return launch_dependent(kern, dim3((unsigned)x, (unsigned)y), kThreads, 0, st, (const ExpandArgs)a);
}

// Comparisons of ids up to which one block plans and compares them in one launch, and kept entries up to which
// it checks those too and the copy's last block commits: two launches.  (Captured, with the copy of the table: one
// launch more for the checks against several blocks, 7280 comparisons 11.7 us and 12.3, 27 thousand 21.8 and 21.2,
// 118 thousand 15.7 and 13.1.  Two launches against three or four, 32 entries 10.2 us and 9.5, 2144 12.4 and 11.7,
// but at 32 the host has 4 us less to do, and the kernels wait for it.)
constexpr int64_t kSmallCompare = 1 << 14, kSmallKept = 1 << 10;

cudaError_t launch_compact8(const kara_cache8 *c, const Geo &g, SeqPlan *plan, int32_t *done, const int32_t *kept,
                            const int32_t *fresh, int64_t n_fresh, int32_t *freed, int32_t *new_len, int32_t *table,
                            int32_t *err, cudaStream_t st)
{
    CompactArgs a;
    a.in = pool8(c);
    a.codes[0] = static_cast<uint8_t *>(c->k), a.codes[1] = static_cast<uint8_t *>(c->v);
    a.scale[0] = c->k_scale, a.scale[1] = c->v_scale;
    a.plan = plan, a.kept = kept, a.fresh = fresh, a.bt = g.bt;
    a.n_fresh = n_fresh;
    a.B = g.B, a.C = g.C, a.R = g.R, a.bt_stride = g.bt_stride;
    const int max_new = (kBs - 1 + g.R + g.B + kBs - 1) / kBs;  // the window may start at any row of a block
    a.err = err;
    a.freed = freed, a.new_len = new_len, a.table = table;
    a.g = g;
    // up to kCopyWarps new blocks of a window to a CTA, evenly
    const int parts = (max_new + kCopyWarps - 1) / kCopyWarps, warps = (max_new + parts - 1) / parts;
    if (g.nwin * parts > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)g.nwin, (unsigned)parts);
    const int64_t most = (int64_t)g.n * max_new, used = most < n_fresh ? most : n_fresh;
    const bool one_block = (used + (int64_t)g.n * g.bt_stride) * used <= kSmallCompare;
    const bool small = one_block && g.nwin * g.R <= kSmallKept;
    a.done = small ? done : nullptr;
    cudaError_t e = cudaSuccess;
    if (one_block) {
        e = launch_prepare(g, small ? kept : nullptr, fresh, n_fresh, plan, done, err, st);
    } else {
        e = launch_plan(g, n_fresh, plan, err, st, true);
        if (e == cudaSuccess) e = launch_fresh_check(g, plan, fresh, n_fresh, err, st, true);
    }
    if (e == cudaSuccess && !small) e = launch_kept_check(g, kept, err, st, true);
    const auto kern = g.D == 128 ? compact8_kernel<128> : compact8_kernel<64>;
    if (e == cudaSuccess) e = launch_dependent(kern, grid, 32 * warps, 0, st, (const CompactArgs)a);
    if (e == cudaSuccess && !small) e = launch_commit(g, plan, fresh, freed, new_len, table, err, st, true);
    return e;
}

}  // namespace kara
