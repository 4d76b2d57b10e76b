// Extending the block tables by new tokens: the tables' new entries, and the
// indices (first row, slot, sequence, position) that the append and the
// attention of those tokens read.
//
// For each sequence s with a cached length len and m new tokens:
//     need   = ceil((len + m) / bs) - ceil(len / bs) blocks, taken from `fresh`
//              in sequence order (exclusive prefix sums of need),
//     q_start[s] = sum of m over the earlier sequences,
//     token q_start[s] + i: position len + i, slot = its block * bs + its row.
//
// The work is a few KB to a few MB and is bound by latency, so everything runs
// in one launch: one cluster of up to 8 CTAs.  Every CTA repeats the prefix sums
// over the lengths (n values, from L2), which costs less than handing them
// round; the checks, the table entries and the token rows are dealt out to the
// CTAs, and two cluster barriers make the call all-or-nothing: nothing is
// written before every check of every CTA has passed.  The check that no
// consumed id is used twice or still listed by a table keeps a bitmap of the
// consumed ids in shared memory (one bit per block of the pool, in windows of
// 2^20 blocks), so it reads each table entry once.
#include <cooperative_groups.h>

#include "kara_sm100.cuh"
#include "kara_tokens.cuh"

namespace cg = cooperative_groups;

namespace kara {
namespace {

constexpr int kExtThreads = 1024;
constexpr int kExtCtas = 8;             // portable cluster size
constexpr int kBitWindow = 1 << 20;     // ids per bitmap window: 128 KB of shared memory
constexpr int kStartCap = 16384;        // sequences whose q_start fits beside it (64 KB)
constexpr int kMaxSmem = kBitWindow / 8 + (int)sizeof(int32_t) * (kStartCap + 1);
constexpr int kScanItem = 512;          // table entries a warp checks per turn
// Up to this many entries to check and rows to write, one CTA does it all: the
// cluster's barriers then cost more than its width saves.
constexpr int64_t kOneCta = 4096;

// Calls of more rows leave them to a kernel over all SMs.  Measured (apart / in one kernel, us):
// 4096 rows 9.1 / 7.3, 8192 8.9 / 7.5, 16384 9.4 / 8.7, 131072 11.6 / 24.7.
constexpr int kRowsApart = 20480;

struct ExtArgs {
    int32_t n, rows, num_blocks, bt_stride, window;
    static constexpr int32_t bs = 16;  // tokens per cache block (the supported block size)
    int64_t n_fresh;
    const int32_t *len, *n_new, *fresh;
    int32_t *bt;
    int32_t *q_start, *new_len, *seq, *pos, *used, *err;
    int64_t *slot;
    int32_t start_in_smem;
    int32_t rows_apart;  // the token rows are another kernel's
};

enum : int { kBad = 1, kDup = 2, kEarlier = 4 };

// Inclusive scan of two 64-bit values over the block; tot gets the sums.
__device__ longlong2 block_scan2(longlong2 v, longlong2 *scratch /* 33 */, longlong2 &tot)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
        if (lane >= o) v.x += x, v.y += y;
    }
    if (lane == 31) scratch[warp] = v;
    __syncthreads();
    if (warp == 0) {
        longlong2 w = scratch[lane];
        const longlong2 own = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, w.x, o), y = __shfl_up_sync(0xffffffffu, w.y, o);
            if (lane >= o) w.x += x, w.y += y;
        }
        scratch[lane] = make_longlong2(w.x - own.x, w.y - own.y);
        if (lane == 31) scratch[32] = w;
    }
    __syncthreads();
    const longlong2 b = scratch[warp];
    tot = scratch[32];
    __syncthreads();
    return make_longlong2(b.x + v.x, b.y + v.y);
}

__device__ __forceinline__ int32_t blocks_of(const ExtArgs &a, int64_t x) { return (int32_t)((x + a.bs - 1) / a.bs); }

__device__ __forceinline__ bool seq_ok(const ExtArgs &a, int32_t len, int32_t m)
{
    return len >= 0 && m >= 0 && ((int64_t)len + m + a.bs - 1) / a.bs <= a.bt_stride;
}

// A barrier of all threads of the call (their writes to global memory are visible after it).
__device__ __forceinline__ void meet(int nc)
{
    if (nc == 1) {
        __syncthreads();
    } else {
        ptx::cluster_arrive();
        ptx::cluster_wait();
    }
}

__global__ void __launch_bounds__(kExtThreads, 1) extend_kernel(const ExtArgs a)
{
    extern __shared__ uint32_t ext_smem[];
    uint32_t *bits = ext_smem;                                               // window / 32 words
    int32_t *start = reinterpret_cast<int32_t *>(ext_smem + a.window / 32);  // [n + 1] when it fits
    __shared__ longlong2 scratch[33];
    __shared__ int flags;   // of the whole cluster, in CTA 0
    __shared__ int wrong;   // this CTA saw a bad length
    __shared__ int32_t taken[kExtThreads + 1];  // ids taken before each sequence of a pass
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), nc = (int)gridDim.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gw = warp * nc + rank, nw = nc * (kExtThreads / 32);  // warps of the call, dealt across CTAs

    for (int i = tid; i < a.window / 32; i += kExtThreads) bits[i] = 0;
    // launched as a programmatic dependent of what precedes it on the stream
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) {
        flags = rank == 0 && *(volatile int32_t *)a.err != 0 ? kEarlier : 0;
        wrong = 0;
    }
    __syncthreads();
    if (nc > 1) ptx::cluster_arrive();  // CTA 0's flags are set up (waited for before the first CTA adds to them)

    // ---- totals: tokens and blocks (every CTA, from the lengths); the entry of the block that a
    // growing sequence continues is looked at on the way, by one CTA
    int found = 0;
    longlong2 carry = make_longlong2(0, 0), in = carry;
    int32_t len = 0, m = 0, need = 0;  // of the last pass over the sequences
    for (int base = 0; base < a.n; base += kExtThreads) {
        const int s = base + tid;
        len = m = need = 0;
        int32_t open = 0;
        if (s < a.n) {
            len = a.len[s];
            m = a.n_new[s];
            if (!seq_ok(a, len, m)) {
                wrong = 1;
                m = 0;
            } else {
                need = blocks_of(a, (int64_t)len + m) - blocks_of(a, len);
                if (warp % nc == rank && m > 0 && len % a.bs) open = a.bt[(int64_t)s * a.bt_stride + len / a.bs];
            }
        }
        longlong2 tot;
        in = block_scan2(make_longlong2(m, need), scratch, tot);
        if (a.start_in_smem && s < a.n) start[s] = (int32_t)(carry.x + in.x - m);
        in.x += carry.x, in.y += carry.y;
        carry.x += tot.x, carry.y += tot.y;
        if (open < 0 || open >= a.num_blocks) found |= kBad;
    }
    if (a.start_in_smem && tid == 0) start[a.n] = (int32_t)carry.x;
    const int64_t total = carry.x, F = carry.y;
    const int plan = wrong || total > a.rows ? KARA_EINVAL : F > a.n_fresh ? KARA_ENOBLOCKS : KARA_OK;

    // ---- consumed ids: each once, and in no table of the batch (dealt over the cluster)
    const int per_row = (a.bt_stride + kScanItem - 1) / kScanItem;
    for (int64_t w0 = 0; plan == KARA_OK && F > 0 && w0 < a.num_blocks; w0 += a.window) {
        if (w0 > 0) {
            __syncthreads();
            for (int i = tid; i < a.window / 32; i += kExtThreads) bits[i] = 0;
            __syncthreads();
        }
        for (int64_t i = tid; i < F; i += kExtThreads) {
            const int32_t f = a.fresh[i];
            if (f < 0 || f >= a.num_blocks) found |= kBad;
            const uint32_t o = (uint32_t)f - (uint32_t)w0;
            if (o < (uint32_t)a.window && (atomicOr(&bits[o >> 5], 1u << (o & 31)) >> (o & 31) & 1u)) found |= kDup;
        }
        __syncthreads();
        for (int64_t it = gw; it < (int64_t)a.n * per_row; it += nw) {
            const int s = (int)(it / per_row), c0 = (int)(it % per_row) * kScanItem;
            const int32_t have = blocks_of(a, a.len[s]);
            const int32_t *row = a.bt + (int64_t)s * a.bt_stride;
            int32_t id[kScanItem / 32];
#pragma unroll
            for (int k = 0; k < kScanItem / 32; ++k) {
                const int c = c0 + k * 32 + lane;
                id[k] = c < have ? row[c] : -1;
            }
#pragma unroll
            for (int k = 0; k < kScanItem / 32; ++k) {
                const uint32_t o = (uint32_t)id[k] - (uint32_t)w0;
                if (id[k] >= 0 && o < (uint32_t)a.window && (bits[o >> 5] >> (o & 31) & 1u)) found |= kDup;
            }
        }
    }
    found = __reduce_or_sync(0xffffffffu, found);
    __syncwarp();
    if (nc > 1) ptx::cluster_wait();
    if (lane == 0 && found) atomicOr(cluster.map_shared_rank(&flags, 0), found);
    meet(nc);
    const int all = *cluster.map_shared_rank(&flags, 0);
    const bool ok = plan == KARA_OK && all == 0;

    // ---- commit: table entries, first rows, lengths (or the state of a call that did nothing)
    if (rank == 0 && tid == 0) {
        if (plan != KARA_OK) set_err(a.err, plan);
        else if (all & kDup) set_err(a.err, KARA_EDUPBLOCK);
        else if (all & kBad) set_err(a.err, KARA_EBADBLOCK);
        *a.used = ok ? (int32_t)F : 0;
        a.q_start[a.n] = ok ? (int32_t)total : 0;
    }
    const bool in_place = a.new_len == a.len;
    const bool one_pass = a.n <= kExtThreads;  // the sums of the pass above are still at hand
    carry = make_longlong2(0, 0);
    for (int base = 0; base < a.n; base += kExtThreads) {
        const int s = base + tid;
        if (!one_pass) {
            len = m = need = 0;
            if (s < a.n) {
                len = a.len[s];
                m = ok ? a.n_new[s] : 0;
                need = blocks_of(a, (int64_t)len + m) - blocks_of(a, len);
            }
            longlong2 tot = make_longlong2(0, 0);
            in = tot;
            if (ok) in = block_scan2(make_longlong2(m, need), scratch, tot);
            in.x += carry.x, in.y += carry.y;
            carry.x += tot.x, carry.y += tot.y;
        }
        if (warp % nc == rank && s < a.n) {
            a.q_start[s] = ok ? (int32_t)(in.x - m) : 0;
            if (!in_place) a.new_len[s] = ok ? len + m : len;
        }
        if (ok && F > 0) {
            // a warp per sequence fills its entries
            __syncthreads();
            taken[tid] = (int32_t)(in.y - need);
            if (tid == kExtThreads - 1) taken[kExtThreads] = (int32_t)in.y;
            __syncthreads();
            for (int i = gw; i < kExtThreads && base + i < a.n; i += nw) {
                const int32_t o = taken[i], cnt = taken[i + 1] - o;
                if (cnt == 0) continue;
                int32_t *row = a.bt + (int64_t)(base + i) * a.bt_stride + blocks_of(a, a.len[base + i]);
                for (int e = lane; e < cnt; e += 32) row[e] = a.fresh[o + e];
            }
        }
    }
    meet(nc);  // the new entries (and q_start, where it is searched in global memory) are visible

    if (a.rows_apart) {
        if (in_place && ok)
            for (int s = gw * 32 + lane; s < a.n; s += nw * 32) a.new_len[s] += a.n_new[s];
        return;
    }
    // ---- token rows: a warp takes 32 at a time, four times over so that the look-ups overlap; each
    // row's sequence by bisection of the first rows
    const int32_t *first = a.start_in_smem ? start : a.q_start;
    constexpr int kU = 4;
    for (int64_t t0 = (int64_t)gw * 32 + lane; t0 < a.rows; t0 += (int64_t)nw * 32 * kU) {
        int64_t slot[kU];
        int32_t s[kU], x[kU], b[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t t = t0 + (int64_t)u * nw * 32;
            s[u] = x[u] = -1;
            if (ok && t < total) {
                int lo = 0, hi = a.n;  // last sequence whose first row is <= t
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (first[mid] <= t) lo = mid; else hi = mid;
                }
                s[u] = lo;
                x[u] = a.len[lo] + (int32_t)(t - first[lo]);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
            b[u] = s[u] >= 0 ? __ldcg(a.bt + (int64_t)s[u] * a.bt_stride + x[u] / a.bs) : 0;
#pragma unroll
        for (int u = 0; u < kU; ++u) slot[u] = s[u] >= 0 ? (int64_t)b[u] * a.bs + x[u] % a.bs : -1;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t t = t0 + (int64_t)u * nw * 32;
            if (t >= a.rows) break;
            a.slot[t] = slot[u];
            a.seq[t] = s[u];
            a.pos[t] = x[u];
        }
    }
    if (in_place && ok) {
        meet(nc);  // every CTA has read the old lengths
        for (int s = gw * 32 + lane; s < a.n; s += nw * 32) a.new_len[s] += a.n_new[s];
    }
}

// The token rows of a long call, over all SMs: launched as a programmatic dependent of the
// kernel above, whose first rows, lengths and tables say everything (a call that did
// nothing left no tokens: every row is padding).
constexpr int kRowThreads = 256, kRowsPer = 4;  // threads, rows of each
constexpr int kRowCap = 8192;                   // sequences whose first rows a CTA keeps in shared memory

__global__ void __launch_bounds__(kRowThreads) token_rows_kernel(const ExtArgs a)
{
    __shared__ int32_t start[kRowCap];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t total = a.q_start[a.n];
    const bool in_smem = a.n <= kRowCap;
    if (in_smem)
        for (int i = threadIdx.x; i < a.n; i += kRowThreads) start[i] = a.q_start[i];
    __syncthreads();
    const int32_t *first = in_smem ? start : a.q_start;
    const int64_t t0 = (int64_t)blockIdx.x * (kRowThreads * kRowsPer) + threadIdx.x;
    int64_t slot[kRowsPer];
    int32_t s[kRowsPer], x[kRowsPer];
#pragma unroll
    for (int u = 0; u < kRowsPer; ++u) {
        const int64_t t = t0 + u * kRowThreads;
        s[u] = x[u] = -1;
        if (t < total) {
            int lo = 0, hi = a.n;  // last sequence whose first row is <= t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first[mid] <= t) lo = mid; else hi = mid;
            }
            s[u] = lo;
            x[u] = a.new_len[lo] - (int32_t)(a.q_start[lo + 1] - t);
        }
    }
#pragma unroll
    for (int u = 0; u < kRowsPer; ++u)
        slot[u] = s[u] < 0 ? -1
                           : (int64_t)a.bt[(int64_t)s[u] * a.bt_stride + x[u] / a.bs] * a.bs + x[u] % a.bs;
#pragma unroll
    for (int u = 0; u < kRowsPer; ++u) {
        const int64_t t = t0 + u * kRowThreads;
        if (t >= a.rows) break;
        a.slot[t] = slot[u];
        a.seq[t] = s[u];
        a.pos[t] = x[u];
    }
}

}  // namespace

cudaError_t launch_extend(int32_t num_blocks, const int32_t *len, const int32_t *n_new, int32_t *bt, int32_t bt_stride,
                          const int32_t *fresh, int64_t n_fresh, const kara_tokens *t,
                          int32_t *used, int32_t *err, cudaStream_t st)
{
    ExtArgs a;
    a.n = t->n;
    a.rows = t->rows;
    a.num_blocks = num_blocks;
    a.bt_stride = bt_stride;
    a.window = num_blocks < kBitWindow ? (num_blocks + 31) / 32 * 32 : kBitWindow;
    a.n_fresh = n_fresh;
    a.len = len;
    a.n_new = n_new;
    a.fresh = fresh;
    a.bt = bt;
    a.q_start = t->q_start;
    a.new_len = t->len;
    a.seq = t->seq;
    a.pos = t->pos;
    a.slot = t->slot;
    a.used = used;
    a.err = err;
    a.start_in_smem = t->n <= kStartCap;
    const size_t smem = (size_t)a.window / 8 + (a.start_in_smem ? sizeof(int32_t) * ((size_t)t->n + 1) : 0);
    if (smem > 40 * 1024) {
        // (one limit for every size: it is the kernel's, and another host thread may set it ahead of this launch)
        const cudaError_t e =
            cudaFuncSetAttribute(extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
    }
    a.rows_apart = t->rows > kRowsApart;
    const int nc = (int64_t)t->n * bt_stride + t->rows <= kOneCta ? 1 : kExtCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)nc);
    cfg.blockDim = dim3(kExtThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)nc;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, extend_kernel, a);
    if (e != cudaSuccess || !a.rows_apart) return e;
    constexpr int per = kRowThreads * kRowsPer;
    cudaLaunchConfig_t rows = {};
    rows.gridDim = dim3((unsigned)(((int64_t)t->rows + per - 1) / per));
    rows.blockDim = dim3(kRowThreads);
    rows.stream = st;
    cudaLaunchAttribute ra[1];
    ra[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    ra[0].val.programmaticStreamSerializationAllowed = 1;
    rows.attrs = ra;
    rows.numAttrs = 1;
    return cudaLaunchKernelEx(&rows, token_rows_kernel, a);
}

}  // namespace kara
