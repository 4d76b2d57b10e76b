// New tokens into the 8-bit cache: per-head norms of q and k, the position rotation, and
// the write of K and V, rounded to e4m3 with a scale for each block and head, in one pass.
//
// Rows are normed and turned as in the bf16 cache (kara_rows.cuh: a query gets the same
// bits there).  The new rows of a block and head, at most 16, are a run.  With z the fp32
// results (V: the inputs) and s0 the block's scale if the run continues it, else 0:
//     s = max(s0, the smallest power of two with max |z| <= 448 s)
//     code = rn(z / s),   and, if s > s0, code = rn(code s0 / s) for the rows ahead
// One rounding from fp32; nothing is rounded to bf16 on the way.  A run needs its largest
// value before its first code, so two warps hold a whole run of one head: all its loads are
// in flight at once, and the rows stay in registers between the maximum and the rounding.
// Queries go with them, a warp per token and a few heads.
//
// Runs follow from the slots alone: row t continues row t - 1 if its slot is the next one
// and not the first of a block.  A CTA looks at a window of `win` rows and takes the runs
// that begin there.
//
// Bound by HBM and issue slots: 8192 tokens, 40 and 2 x 8 heads of 128, with the ring, 60.5 us captured for 264 MB
// (4.4 TB/s).  On the way: a warp a run 102; two warps a run and the window's table rows in shared memory 76; five
// passes of query rows 72.5; a form for rotations of all dims 66; a key's factors formed once for a CTA 60.5.
// (Queries by the bf16 append's staged kernel, in a launch of their own: as fast at 76, and slower by that launch
// in shorter calls, 512 sequences of a token 26.5 against 23.2, 512 tokens 11.2 against 7.4.  Four CTAs to an SM
// instead of three, with spills: 57, but 512 tokens 7.1 for 6.5, 256 sequences of four 16.4 for 15.2; two heads to
// a pair of warps: 58, but 8.0 and 16.0.)  A token for each of up to 64 sequences takes 3.3 to 4.3 us captured, the chain
// of slot, table row, rows, largest value; 128 take 7.3, 256 11.7: runs of one row have two warps each all the same, and
// their CTAs come in rounds.
#include "kara_cache8.cuh"
#include "kara_rows.cuh"
#include "kara_tokens.cuh"

namespace kara {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBs = 16;      // tokens per cache block (the supported block size)
constexpr int kMaxWin = 16;  // rows that a CTA looks at for the beginnings of runs, at most

// Passes of query rows a warp has in flight (8192 tokens: 4, 5 and 10 take 64, 60.5 and 59.6 us, 256 sequences of four
// 15.3, 15.2 and 16.2; a decode step of 128 tokens 7.4, 7.5 and 7.75 with 2, 4 and 5).
__host__ __device__ constexpr int query_passes(bool many) { return many ? 5 : 4; }

struct Append8Args {
    const uint16_t *q, *k, *v;
    int64_t qs, ks, vs;  // token strides (elements)
    uint16_t *q_out, *ring;
    uint8_t *kp, *vp;          // codes, at the call's layer
    float *k_scale, *v_scale;  // [num_blocks][hkv], at the call's layer
    int64_t block_stride, head_stride;
    int64_t ring_seq, ring_head;  // strides of the ring (elements), at the call's layer
    const uint16_t *qw, *kw;
    const float *cos_sin;
    const int32_t *shift;
    const int64_t *slot;
    const int32_t *seq, *pos, *len;
    int32_t *err;
    float eps;
    int32_t n, rows, num_blocks, hq, hkv, W, n_pos, rot;
    int32_t win, kv_blocks;  // rows of a window; CTAs that take runs
};

// Where a token goes; ok: its row is to be written.
struct Place {
    int64_t slot, r;  // slot, row of the rotation table
    int32_t seq, pos;
    bool ok;
};

__device__ __forceinline__ Place place_of(const Append8Args &a, int64_t t, bool record)
{
    Place p;
    p.slot = a.slot[t];
    p.seq = a.seq[t];
    p.pos = a.pos[t];
    const bool known = p.seq >= 0 && p.seq < a.n, inside = p.slot >= 0 && p.slot < (int64_t)a.num_blocks * kBs;
    // without a rotation every rotary position will do
    p.r = a.rot == 0 ? 0 : (int64_t)p.pos + (known && a.shift ? a.shift[p.seq] : 0);
    p.ok = inside && known && p.pos >= 0 && p.r >= 0 && p.r < a.n_pos;
    if (record && !p.ok && p.slot != -1) set_err(a.err, inside ? KARA_EINVAL : KARA_EBADBLOCK);
    return p;
}

// What a lane does with its eight dims of every row: which of them turn, with which lane.
// (FULL: all D turn; INTER: pairs are neighbours.)
template <int D, bool INTER, bool FULL>
struct LaneDims {
    int d0, half, other;
    bool turned, low;
    __device__ LaneDims(const Append8Args &a, int lane)
    {
        d0 = lane % (D / 8) * 8;
        half = FULL ? D / 2 : a.rot >> 1;
        turned = FULL || d0 < a.rot, low = d0 < half;
        // lane that holds the other half of this lane's pairs
        other = !turned || INTER ? lane : low ? lane + half / 8 : lane - half / 8;
    }
    // cosines and signed sines, in pairs of neighbours
    __device__ __forceinline__ void factors(const float *row, uint64_t (&c)[4], uint64_t (&sn)[4]) const
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = ptx::pack2(1.f, 1.f), sn[e] = ptx::pack2(0.f, 0.f);
        if (!turned) return;
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
    // a norm's weights of this lane's dims and of their partners (1 without one)
    __device__ __forceinline__ void weights(const uint16_t *wp, uint4 &w, uint4 &wo) const
    {
        w = wo = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
        if (!wp) return;
        w = __ldg(reinterpret_cast<const uint4 *>(wp + d0));
        wo = INTER ? w : __ldg(reinterpret_cast<const uint4 *>(wp + (turned ? low ? d0 + half : d0 - half : d0)));
    }
    // z = (x w c + x' w' s), x' and w' of the pair's other member, and 1 / the norm; the whole warp.  wc, ws: the products
    __device__ __forceinline__ void turn(const Append8Args &a, const uint4 &u, bool norm, const uint64_t (&wc)[4],
                                         const uint64_t (&ws)[4], uint64_t (&z)[4], float &inv) const
    {
        uint4 uo = u;
        if (!INTER && (FULL || a.rot > 0)) {
            uo.x = __shfl_sync(0xffffffffu, u.x, other), uo.y = __shfl_sync(0xffffffffu, u.y, other);
            uo.z = __shfl_sync(0xffffffffu, u.z, other), uo.w = __shfl_sync(0xffffffffu, u.w, other);
        }
        uint64_t x[4], xo[4];
        pairs4(u, x, false), pairs4(uo, xo, INTER);
        inv = 1.f;
        if (norm) {
            float ss = squares(x);
#pragma unroll
            for (int o = D / 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            inv = inverse_norm(ss, 1.f / D, a.eps);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = turn2(x[e], wc[e], xo[e], ws[e]);
        if (!turned) {  // (0 times an infinity is no number)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = mul2(x[e], wc[e]);
        }
    }
    __device__ __forceinline__ void turn(const Append8Args &a, const uint4 &u, const uint16_t *wp, const uint4 &uw,
                                         const uint4 &uwo, const uint64_t (&c)[4], const uint64_t (&sn)[4],
                                         uint64_t (&z)[4], float &inv) const
    {
        uint64_t w[4], wo[4], wc[4], ws[4];
        pairs4(uw, w, false), pairs4(uwo, wo, INTER);
#pragma unroll
        for (int e = 0; e < 4; ++e) wc[e] = mul2(w[e], c[e]), ws[e] = mul2(wo[e], sn[e]);
        turn(a, u, wp != nullptr, wc, ws, z, inv);
    }
};

// What the two warps of a run tell each other: their largest magnitudes and whether they met a value that is
// not finite, in turn (one may be a run ahead).
struct Meet {
    float top[2][2];
    int32_t odd[2][2];
};

// Takes eight values into the running maximum; odd becomes NaN with the first one that is not finite.
__device__ __forceinline__ void take(const uint64_t (&z)[4], float &top, uint64_t &odd)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float lo, hi;
        ptx::unpack2(z[e], lo, hi);
        top = fmaxf(top, fmaxf(fabsf(lo), fabsf(hi)));
        odd = ptx::fma2(z[e], 0ull, odd);
    }
}

// The largest of eight that are finite.
__device__ __forceinline__ float finite_top(const uint64_t (&z)[4])
{
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float lo, hi;
        ptx::unpack2(z[e], lo, hi);
        if (finite(lo)) top = fmaxf(top, fabsf(lo));
        if (finite(hi)) top = fmaxf(top, fabsf(hi));
    }
    return top;
}

// Codes of eight values times f; `odd`: NaN for those that are not finite, as e4m3 has no infinity.
__device__ __forceinline__ uint2 codes8(const uint64_t (&z)[4], float f, bool odd)
{
    const uint64_t f2 = ptx::pack2(f, f);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float lo, hi;
        ptx::unpack2(mul2(z[e], f2), lo, hi);
        if (odd) {  // (0 times an infinity is NaN already)
            if (!finite(lo)) lo = __uint_as_float(0x7fffffffu);
            if (!finite(hi)) hi = __uint_as_float(0x7fffffffu);
        }
        w[e] = e4m3x2(lo, hi);
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// What a key is multiplied by: of a row of the rotation table, for all D dims, cosines times weights and then
// the signed sines times the partners' weights (the same products as a lane forms for itself), each as the first
// halves of the lanes' eight dims, then the second, so that 16-byte loads meet no bank twice.  A warp takes a row.
template <int D, bool INTER, bool FULL>
struct RowFactors {
    int d, half;
    bool turned, low;
    float w[4], wo[4];
    __device__ RowFactors(const Append8Args &a, int lane)
    {
        d = lane * 4 % D, half = FULL ? D / 2 : a.rot >> 1;
        turned = FULL || d < a.rot, low = d < half;
        const int other = !turned || INTER ? d : low ? d + half : d - half;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = a.kw ? __uint_as_float((uint32_t)__ldg(a.kw + d + e) << 16) : 1.f;
            wo[e] = a.kw ? __uint_as_float((uint32_t)__ldg(a.kw + other + (INTER ? e ^ 1 : e)) << 16) : 1.f;
        }
    }
    __device__ __forceinline__ void store(const float *row, float *to, int lane) const
    {
        float4 wc = make_float4(w[0], w[1], w[2], w[3]), ws = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane >= D / 4) return;
        if (turned && INTER) {
            const float2 c = __ldg(reinterpret_cast<const float2 *>(row + d / 2));
            const float2 s = __ldg(reinterpret_cast<const float2 *>(row + half + d / 2));
            wc = make_float4(w[0] * c.x, w[1] * c.x, w[2] * c.y, w[3] * c.y);
            ws = make_float4(wo[0] * -s.x, wo[1] * s.x, wo[2] * -s.y, wo[3] * s.y);
        } else if (turned) {
            const float *at = row + (low ? d : d - half);
            const float4 c = ldg4(at), s = ldg4(at + half);
            const float g = low ? -1.f : 1.f;
            wc = make_float4(w[0] * c.x, w[1] * c.y, w[2] * c.z, w[3] * c.w);
            ws = make_float4(wo[0] * (g * s.x), wo[1] * (g * s.y), wo[2] * (g * s.z), wo[3] * (g * s.w));
        }
        to += (d >> 3) * 4 + (d & 4 ? D / 2 : 0);
        *reinterpret_cast<float4 *>(to) = wc;
        *reinterpret_cast<float4 *>(to + D) = ws;
    }
};

// The runs that begin in a window, for four of the 2 hkv (K, then V) heads of a CTA; two warps share a run
// of a head, eight rows each: alone, with all rows in registers, so few fit on an SM that the chain of loads
// (slot, offset, table row) set the pace.  A CTA with keys brings in what the window's rows of the rotation table
// multiply them by, while the first run's rows are on their way.
// (LONG: windows of several rows.  With one each row's factors come straight from global memory.)
template <int D, bool INTER, bool FULL, bool LONG>
__device__ __forceinline__ void store_window(const Append8Args &a, const LaneDims<D, INTER, FULL> &dims, int64_t window,
                                             int h0, int pair, float *table, Meet *meet)
{
    constexpr int LPR = D / 8, RPP = 32 / LPR, NP = kBs / RPP / 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = warp & 1, h = h0 + pair;
    const bool mine = h < 2 * a.hkv, is_v = h >= a.hkv;
    const int g = is_v ? h - a.hkv : h, row0 = half * (kBs / 2) + lane / LPR;
    // lane i: row t0 - 1 + i.  Runs that begin in the window (lanes 1 .. win) end by lane win + 15.
    const int64_t t0 = window * a.win, t = t0 - 1 + lane;
    Place p{};
    p.slot = -1;
    if (t >= 0 && t < a.rows && lane < a.win + kBs) p = place_of(a, t, h == 0 && half == 0 && lane >= 1 && lane <= a.win);
    const int64_t ahead = __shfl_up_sync(0xffffffffu, p.ok ? p.slot : -2, 1);
    const bool follows = p.ok && lane > 0 && ahead + 1 == p.slot && p.slot % kBs != 0;
    const unsigned good = __ballot_sync(0xffffffffu, p.ok), cont = __ballot_sync(0xffffffffu, follows);
    unsigned heads = __ballot_sync(0xffffffffu, p.ok && !follows && lane >= 1 && lane <= a.win);
    const uint16_t *src = (is_v ? a.v : a.k) + g * D + dims.d0;
    const int64_t stride = is_v ? a.vs : a.ks;
    bool staged = false;
    for (int turn = 0; heads; heads &= heads - 1, turn ^= 1) {
        // m rows from lane `first` on go into the rows from `at` on of block blk
        const int first = __ffs(heads) - 1, m = __ffs(~(cont >> (first + 1)));
        const int64_t slot = __shfl_sync(0xffffffffu, p.slot, first), blk = slot / kBs;
        const int at = (int)(slot % kBs);
        uint4 u[NP];
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int i = k * RPP + row0;
            u[k] = mine && i < m ? *reinterpret_cast<const uint4 *>(src + (t0 - 1 + first + i) * stride)
                                 : make_uint4(0, 0, 0, 0);
        }
        float *sp = (is_v ? a.v_scale : a.k_scale) + blk * a.hkv + g;
        const float old = mine && at > 0 ? *sp : 0.f;
        if (LONG && !staged && h0 < a.hkv) {
            staged = true;
            const RowFactors<D, INTER, FULL> f(a, lane);
            for (int i = 1 + warp; i < a.win + kBs; i += kWarps) {
                const int64_t r = __shfl_sync(0xffffffffu, p.r, i);
                if (good >> i & 1u) f.store(a.cos_sin + r * a.rot, table + i * 2 * D, lane);
            }
            __syncthreads();
        }
        if (!mine) continue;
        // (rows past the run are zeros, and stay zeros)
        float top = 0.f, inv[NP];
        uint64_t z[NP][4], nan = 0ull;
        bool odd_here = false;
        if (is_v) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                pairs4(u[k], z[k], false);
                take(z[k], top, nan);
                inv[k] = 1.f;
            }
        } else {
            uint4 uw, uwo;
            if (!LONG) dims.weights(a.kw, uw, uwo);
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int i = k * RPP + row0, from = first + min(i, m - 1);
                if (LONG) {
                    const ulonglong2 *f = reinterpret_cast<const ulonglong2 *>(table + from * 2 * D + dims.d0 / 2);
                    const ulonglong2 c0 = f[0], c1 = f[D / 8], s0 = f[D / 4], s1 = f[D / 4 + D / 8];
                    dims.turn(a, u[k], a.kw != nullptr, {c0.x, c0.y, c1.x, c1.y}, {s0.x, s0.y, s1.x, s1.y}, z[k], inv[k]);
                } else {
                    uint64_t c[4], sn[4];
                    const int64_t r = __shfl_sync(0xffffffffu, p.r, from);
                    dims.factors(a.cos_sin + r * a.rot, c, sn);
                    dims.turn(a, u[k], a.kw, uw, uwo, c, sn, z[k], inv[k]);
                }
                float of_row = 0.f;
                take(z[k], of_row, nan);
                top = fmaxf(top, of_row * inv[k]);
                odd_here = odd_here || (i < m && !finite(inv[k]));
            }
        }
        float lo, hi;
        ptx::unpack2(nan, lo, hi);
        odd_here = __any_sync(0xffffffffu, odd_here || lo != lo || hi != hi);
        if (__builtin_expect(odd_here, 0)) {
            top = 0.f;
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const uint64_t i2 = ptx::pack2(inv[k], inv[k]);
#pragma unroll
                for (int e = 0; e < 4; ++e) z[k][e] = mul2(z[k][e], i2);
                inv[k] = 1.f;
                top = fmaxf(top, finite_top(z[k]));
            }
        }
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
        if (lane == 0) meet->top[turn][half] = top, meet->odd[turn][half] = odd_here;
        ptx::named_barrier(1 + (warp >> 1), 64);
        top = fmaxf(meet->top[turn][0], meet->top[turn][1]);
        const bool odd = meet->odd[turn][0] || meet->odd[turn][1];
        const float before = fabsf(old), s = fmaxf(before, scale_for(top)), f = inverse_scale(s);
        uint8_t *codes = (is_v ? a.vp : a.kp) + blk * a.block_stride + g * a.head_stride;
        if (s > before && at > 0) {
            const float ratio = before * f;
            for (int i = half * 32 + lane; i < at * D / 16; i += 64) {
                uint4 *q = reinterpret_cast<uint4 *>(codes) + i;
                uint4 w = *q;
                w.x = rescale4(w.x, ratio), w.y = rescale4(w.y, ratio);
                w.z = rescale4(w.z, ratio), w.w = rescale4(w.w, ratio);
                *q = w;
            }
        }
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int i = k * RPP + row0;
            if (i < m) *reinterpret_cast<uint2 *>(codes + (at + i) * D + dims.d0) = codes8(z[k], inv[k] * f, odd_here);
        }
        // the sign says that the block may hold a NaN
        if (half == 0 && lane == 0) *sp = odd || signbit(old) ? -s : s;
    }
}

template <int D, bool INTER, bool FULL, bool LONG>
__global__ void __launch_bounds__(kThreads, LONG ? 3 : 2) append8_kernel(const Append8Args a)
{
    constexpr int LPR = D / 8, RPP = 32 / LPR, NQ = query_passes(LONG), HPW = NQ * RPP;  // a warp's query heads
    const int lane = threadIdx.x & 31;
    const LaneDims<D, INTER, FULL> dims(a, lane);
    // launched as a programmatic dependent of what precedes it on the stream
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ Meet meet[kWarps / 2];
    __shared__ __align__(16) float table[LONG ? (kMaxWin + kBs) * 2 * D : 4];
    if (blockIdx.x < a.kv_blocks) {
        const int groups = (2 * a.hkv + kWarps / 2 - 1) / (kWarps / 2), pair = threadIdx.x >> 6;
        store_window<D, INTER, FULL, LONG>(a, dims, blockIdx.x / groups, blockIdx.x % groups * (kWarps / 2), pair, table,
                                           meet + pair);
        return;
    }
    const int parts = (a.hq + HPW - 1) / HPW;
    const int64_t task = (int64_t)(blockIdx.x - a.kv_blocks) * kWarps + (threadIdx.x >> 5), t = task / parts;
    if (t >= a.rows) return;
    const int h0 = (int)(task % parts) * HPW + lane / LPR;
    // the rows are on their way before the token's place is known (padding rows are read, not written)
    uint4 u[NQ];
#pragma unroll
    for (int p = 0; p < NQ; ++p) {
        const int h = h0 + p * RPP;
        u[p] = h < a.hq ? *reinterpret_cast<const uint4 *>(a.q + t * a.qs + h * D + dims.d0) : make_uint4(0, 0, 0, 0);
    }
    const Place pl = place_of(a, t, false);
    if (!pl.ok) return;
    uint64_t c[4], sn[4];
    dims.factors(a.cos_sin + pl.r * a.rot, c, sn);
    uint4 uw, uwo;
    dims.weights(a.qw, uw, uwo);
    uint16_t *ring = nullptr;  // this token's row of the ring, if it is of the last W
    if (a.ring) {
        const int32_t L = a.len[pl.seq];
        if (pl.pos < L && pl.pos >= (int64_t)L - a.W)
            ring = a.ring + pl.seq * a.ring_seq + (int64_t)(pl.pos % a.W) * D + dims.d0;
    }
#pragma unroll
    for (int p = 0; p < NQ; ++p) {
        const int h = h0 + p * RPP;
        if (h - lane / LPR >= a.hq) break;
        uint64_t z[4];
        float inv;
        dims.turn(a, u[p], a.qw, uw, uwo, c, sn, z, inv);
        const uint4 y = finish(z, inv);
        if (h >= a.hq) continue;
        *reinterpret_cast<uint4 *>(a.q_out + (t * a.hq + h) * D + dims.d0) = y;
        if (ring) *reinterpret_cast<uint4 *>(ring + h * a.ring_head) = y;
    }
}

template <int D, bool INTER>
cudaError_t launch(Append8Args &a, cudaStream_t st)
{
    const bool full = a.rot == D;
    // A CTA's runs go one after another, about 2 us each, and looking for them costs the same for a window of any
    // length: windows of several rows pay where the call has enough of them to hide that chain, 16 win (n / rows + 1/16)
    // runs.  (us with windows of 1, 4 and 16 rows, 40 and 2 x 8 heads of 128, the choice in brackets:
    // 256 sequences of 1 row [11.6] 12.2 32.8, 384 of 1 16.5 [14.2] 32.4, 1024 of 1 40 [27.5] 46, 4096 of 1 172 [112] 104;
    // 96 of 4 10.6 [7.9] 15.4, 256 of 4 25 [15.1] 18.8, 512 of 4 49 28.4 [24.3]; 64 of 12 16 [10.1] 11.9,
    // 64 of 20 24 13.2 [12.2]; 16 of 20 [7.5] 8.0 8.6; 1 of 192 [5.6] 5.1 4.8, 1 of 448 8.9 6.1 [5.9],
    // 4 of 2048 163 74 [60].)
    const double runs = a.n + a.rows / 16.0;
    a.win = (double)a.rows * a.rows >= 6144 * runs ? kMaxWin : a.rows > 320 ? 4 : 1;
    static_assert(kMaxWin + kBs <= 32, "a lane for each row of a window's runs");
    const int per = query_passes(a.win > 1) * (32 / (D / 8));
    const int64_t queries = (int64_t)a.rows * ((a.hq + per - 1) / per);
    const int64_t kv = ((int64_t)a.rows + a.win - 1) / a.win * ((2 * a.hkv + kWarps / 2 - 1) / (kWarps / 2));
    const int64_t blocks = kv + (queries + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    a.kv_blocks = (int32_t)kv;
    const auto kern = full ? (a.win > 1 ? append8_kernel<D, INTER, true, true> : append8_kernel<D, INTER, true, false>)
                           : (a.win > 1 ? append8_kernel<D, INTER, false, true> : append8_kernel<D, INTER, false, false>);
    return launch_dependent(kern, dim3((unsigned)blocks), kThreads, 0, st, (const Append8Args)a);
}

}  // namespace

cudaError_t launch_append8(const kara_cache8 *c, int32_t layer, const kara_tokens *t, const kara_rope *r, const void *q,
                           int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                           void *q_out, void *ring, int32_t W, int32_t *err, cudaStream_t st)
{
    const int D = c->head_dim;
    const int64_t scales = (int64_t)layer * c->num_blocks * c->num_kv_heads;
    Append8Args a;
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.v = static_cast<const uint16_t *>(v);
    a.qs = q_stride, a.ks = k_stride, a.vs = v_stride;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.kp = static_cast<uint8_t *>(c->k) + (int64_t)layer * c->layer_stride;
    a.vp = static_cast<uint8_t *>(c->v) + (int64_t)layer * c->layer_stride;
    a.k_scale = c->k_scale + scales;
    a.v_scale = c->v_scale + scales;
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
    a.hq = c->num_q_heads;
    a.hkv = c->num_kv_heads;
    a.n_pos = r->rot_dim > 0 ? r->n_pos : 1;
    a.rot = r->rot_dim;
    if (D == 128) return r->interleaved ? launch<128, true>(a, st) : launch<128, false>(a, st);
    return r->interleaved ? launch<64, true>(a, st) : launch<64, false>(a, st);
}

}  // namespace kara
