// Attention of a chunk of new tokens over the paged cache, bf16 or 8 bits.
//
// Row t of q is the new token at position p of sequence s (its K and V are in
// the cache already); query head h belongs to KV head g = h / G:
//     out[t][h] = sum_{x <= p} softmax_x(<q[t][h], k_x> / sqrt(D)) v_x
// over the keys of the sequence, read through its block table.
//
// Both contractions run on the 5th-generation tensor cores.  The G query heads
// of a KV head read the same keys, so a query tile is 128 rows of (token, head):
// TQ = 128 / G tokens.  A work item is up to two query tiles of one sequence and
// KV head and the keys that they see, in tiles of 128:
//     S[128 rows][128 keys] = Q . K^T       (both operands in shared memory)
//     O[128 rows][D]       += P . V         (P in TMEM over its S, V in shared memory)
// with the running maximum and sum of each row's softmax in the registers of
// the thread that owns it (warps 0-3: tile 0, warps 4-7: tile 1).  While one
// tile's logits are exponentiated the tensor cores work on the other's.  An item
// of at most TQ tokens (a decode or a short draft) has one query tile; its two
// halves then take the even and the odd key tiles and are joined at the end.
//
//   * The reference of a row's exponentials moves only when the row's maximum
//     has grown by more than 2^8 (kLazy): the weights stay below 2^8, where bf16
//     holds them as well as below 1, and O is rescaled in TMEM a few times per
//     row and not per tile.  The weights are rounded to bf16 for the second
//     product (2^-8 of each at most; the output's own rounding is as large);
//     logits, maxima, sums and O are fp32.  (A second bf16 term of the weights
//     would add half again to the tensor time of two query tiles.  With one, whose
//     time is HBM's, it took the error from 0.0023 to 0.00166 in the 2-norm; but its
//     terms are 0 or negative as well, and an infinite cached value became NaN.)
//   * K and V come by TMA, one (block, KV head) slice of 16 rows at a time,
//     128-byte swizzled, as 128-row tiles in a ring of 5 stages (160 KB in
//     flight per SM).  Blocks past a sequence's end, and ids outside the pool,
//     are copied from past the pool's end: the copy fills zeros.
//   * A weight of 0 times NaN or infinity is NaN, so what a row must not see is
//     cleared from V and not only masked in the logits: four warps zero the rows of
//     the last block past the sequence's end, whatever they hold, and clear the values
//     of the chunk's own tokens that are not finite (earlier tokens share their
//     tile).  The rows that do see such a value get it added at the end.
//   * Every CTA gets the same work (to within a key tile), whatever the lengths:
//     all items' key tiles, weighted by what they cost, are laid end to end and cut
//     evenly; in long calls whose items share keys, whole items go round the CTAs
//     first, so that L2 serves the keys again (share_out).  A cut inside an item
//     leaves partial (O, max, sum) in the workspace, joined by the merge kernel in
//     CTA order, so results do not depend on timing.
//
// What set the pace on the way (8192 tokens over 16384 keys, 40/8 heads, D 128; us, 20 calls
// in a captured graph): one thread issuing every MMA with the waits between them, 2008; its
// loop with ring positions and descriptors that only advance by additions, 1715; one issuing
// thread per query tile and one loading warp each for K and V (issuing a 2 KB copy takes about
// 90 clocks: one warp took 2900 clocks for the K and V tiles that two query tiles multiply
// in 2048), the two tiles taking turns, 1595; the turn taken before the weights are
// waited for, 1485; cuts by cost, 1455; waits that nap in the warps that have time, 1435;
// the instruction caches (one copy of the epilogue's code and of the MMAs', the control
// warps' waiting out of line, one warp that walks over the work and tells the others), 1390
// (512 tokens x 32 sequences at 4096 keys: 852 -> 750); the weighted sum begun on half the
// weights, 1330 to 1370 on several boxes; whole items dealt round, 1285 to 1340 (the 32
// sequences: 750 to 780 -> 675 to 715); logits that wait for the weighted sum whose weights
// they overwrite, 1335 to 1380 (705 to 730): 1.5 PFLOP/s, 0.8 of the measured cuBLAS burst.
// Uncaptured calls in a loop run longer and hotter and take 1440 and 768.
// Few rows over long caches (4 tokens x 128 sequences) read K and V at 6.9 to 7.0 TB/s.
// What is left: a step of two query tiles takes about 3050 clocks against 2048 of tensor time
// (logits, exponentials and weighted sum of a tile depend on each other, and TMEM holds
// one S per tile beside O), and the power limit: under back-to-back calls the clock falls
// to 1.5 - 1.8 GHz.  At D = 64 a step has half the tensor time and the same exponentials:
// 0.85 to 0.9 PFLOP/s, with 128 columns of TMEM unused.  Items of one to four key tiles are
// bound by their start and end: 256 sequences of 1 to 4 tokens over 64 to 512 keys take
// 102 us, 2.2 times their bytes.
//
// The 8-bit cache (E8; the comment ahead of load_queries has the arithmetic): tiles of K's codes are operands as
// they lie, tiles of V's codes pass through four warps that write them as f16, so the ring of 5 tiles is
// 2 (f16) + 3 + 2 (codes).  Four tokens x 128 sequences 610 us (bf16 745), 64 sequences of 1 to 128 tokens 367
// (358), 8192 tokens over 8192 keys 1630 (1405).  No unit is full (tensor 41 and 52 %, issue slots 32 and 48 %, HBM 53 %
// of the copy rate for few tokens): a step waits for logits, weights, and the conversion ahead of the weighted sum, whose
// tiles leave room for two.  (Few rows: a softmax a quarter as long, by rows loaded four times, one more tile of
// codes, or both kinds of codes a tile further ahead bring 0 to 1.5 %, and cost the others 1 to 5.)
//
// Two launches: the attention (persistent, one CTA per SM, each of which works out
// its own range) and the merge, programmatic dependents of what precedes them.
#pragma once

#include "kara_cache8.cuh"
#include "kara_sm100.cuh"
#include "kara_tokens.cuh"

namespace kara {

namespace {

using namespace ptx;

constexpr int kTile = 128;       // rows of a query tile, keys of a key tile
constexpr int kBlk = 16;         // tokens per cache block (the supported block size)
constexpr int kBlkPerTile = kTile / kBlk;
// (The including source has kStages, the tiles of K and V that the ring holds, or the f16 tiles of V alone,
// kEdges and the costs by which the work is cut.)
constexpr int kK8 = 3;           // of an 8-bit cache: tiles of K's codes in flight,
constexpr int kRaw8 = 2;         // and of V's
constexpr int kApart8 = 8;       // scales of a tile of V this many powers of two apart, at most: one exponent for the tile
constexpr int kLeast8 = -40;     // and that exponent not below this
constexpr float kFar8 = 0x1p126f;  // stands for it where there is none
constexpr int kScales8 = 8;      // K tiles whose scales are kept: the warps that read them are not this far behind
constexpr int kMaxCtas = 160;    // CTAs of the attention kernel, at most (workspace slots)
constexpr int kMaxRounds = 64;   // whole items that a CTA takes ahead of its range, at most
constexpr int kThreads = 512;    // two softmax warpgroups, two control warpgroups
constexpr int kWarpKv = 8, kWarpMma = 10, kWarpQ = 12;  // 8: K, 9: V; 10, 11: the MMAs of each query tile
// Registers per thread: at launch (65536 / 512), then after the warpgroups trade:
// 256 * kRegsSoft + 256 * kRegsCtl == 512 * kRegsLaunch.
constexpr int kRegsLaunch = 128;
template <bool E8>
struct Regs {
    static constexpr uint32_t kSoft = E8 ? 184 : 192, kCtl = E8 ? 72 : 64;
    static_assert(256 * kSoft + 256 * kCtl == kThreads * kRegsLaunch, "register trade must add up");
};
constexpr uint32_t kTmemCols = 512;  // S0 S1 (128 columns each), O0 O1 (128 each)
constexpr float kLazy = 8.f;         // see above: rescale when the maximum grew by more than 2^8
constexpr float kUp8 = 7.f;          // 8 bits: weights are up to 2^(kLazy + kUp8), which f16 holds,
constexpr int kUpV8 = 6;             // and values up to 448 * 2^kUpV8
constexpr uint64_t kTimeoutNs = 1000000000ull;

// One or two query tiles of a sequence (all KV heads have the same items).
struct Item {
    int32_t row0;   // first row of q
    int32_t ntok;   // tokens, <= 2 TQ
    int32_t pos0;   // position of the first token
    int32_t nt;     // key tiles that its last token sees
    int32_t len;    // cached length of the sequence
    int32_t m;      // new tokens of the sequence; 0: it has no items
};

// All items in order: head by head, sequence by sequence, 2 TQ tokens (a `pair` of query tiles)
// after another.  A CTA takes some whole items, and then a range.
//
// Where its range starts, and the one before it ends: key tile `off` of an item (off == nt: behind
// its last one; the end of everything: head hkv).
struct __align__(16) Start {
    int32_t head, seq, pair, off;
};

__device__ __forceinline__ bool same_item(const Start &a, const Start &b)
{
    return a.head == b.head && a.seq == b.seq && a.pair == b.pair;
}

struct ChunkArgs {
    const int32_t *q_start, *len, *bt;
    int32_t *err;
    int32_t n, rows, bt_stride, num_blocks, layer, hq, hkv, D, G, TQ, ctas;
    float scale2;     // log2(e) / sqrt(D)
    uint16_t *out;
    int32_t *used_ctas;  // CTAs that got work
    Start *start;        // [used_ctas + 1]
    Start *whole;        // [ctas][kMaxRounds]: each CTA's whole items
    float4 *part;        // [2 * ctas][D / 4][256]
    float2 *stat;        // [2 * ctas][256]: (max, sum) in the log2 domain
    const uint16_t *v;   // V pool at the call's layer
    const uint8_t *v8;   // of the 8-bit cache: V's codes,
    const float *k_scale, *v_scale;  // and K's and V's scales [num_blocks][hkv]
    int64_t block_stride, head_stride;
    int32_t wide;        // out is 32-byte aligned
    int32_t stall;
    uint64_t wait_ns;
};

__device__ __forceinline__ bool chunk_ok(const ChunkArgs &a, int32_t r0, int32_t r1, int32_t L)
{
    return r0 >= 0 && r1 >= r0 && r1 <= a.rows && L >= r1 - r0 && ((int64_t)L + kBlk - 1) / kBlk <= a.bt_stride;
}

// What a key tile costs a CTA (the including source's constants, with kItemCost, an item's start and end).
__device__ __forceinline__ int tile_cost(const ChunkArgs &a, int32_t ntok) { return ntok > a.TQ ? kPairCost : kSingleCost; }
constexpr int kTilesPerCta = 2;  // fewer, and CTAs stay without work: a split costs a merge
constexpr int kSharedTiles = 128;  // key tiles per CTA from which whole items are dealt round

// The item `pair` of sequence `seq`.
__device__ __forceinline__ Item make_item(const ChunkArgs &a, int seq, int pair)
{
    Item it;
    const int32_t r0 = a.q_start[seq], r1 = a.q_start[seq + 1], t0 = pair * 2 * a.TQ;
    it.len = a.len[seq];
    it.m = chunk_ok(a, r0, r1, it.len) ? r1 - r0 : 0;
    it.row0 = r0 + t0;
    it.ntok = min(2 * a.TQ, it.m - t0);
    it.pos0 = it.len - it.m + t0;
    it.nt = (it.pos0 + it.ntok - 1) / kTile + 1;
    return it;
}

// Query-tile pairs of a sequence.
__device__ __forceinline__ int32_t pairs_of(const ChunkArgs &a, int seq)
{
    const int32_t m = make_item(a, seq, 0).m, per = 2 * a.TQ;
    return m / per + (m % per != 0);
}

// ---- attention ------------------------------------------------------------------
constexpr int kPieces = 4;        // descriptions of pieces under way
constexpr int kPieceReaders = 15;  // warps that read them: softmax 8, V, MMAs 2, edge tiles 4
// The warps that clear V may be kPieces pieces ahead of a softmax warp that has yet to look whether it
// has values to add (it gave the description back when it read it), and no more: the description of
// piece n + kPieces + 1 goes where that of n + 1 is, which the softmax warp reads after it is done with n.
constexpr int kOddSlots = 2 * kPieces;
static_assert(kOddSlots > kPieces && (kOddSlots & (kOddSlots - 1)) == 0, "a slot is not written while it is read");

struct Shared {
    uint64_t full[kStages], empty[kStages];  // K / V tiles
    uint64_t q_full, q_empty;
    uint64_t s_full[2];   // logits of a query tile are in TMEM (and its earlier products are done)
    uint64_t p_half[2], p_full[2];  // the first half of its weights are in TMEM; all are
    uint64_t o_full[2];   // its last product is done
    uint64_t x_full, x_free;  // a single query tile's odd half is ready to be joined; is joined
    uint64_t edge[kEdges];  // an edge tile of V has landed (by their number); `full` then says that it is clean
    uint64_t turn[2];     // the tensor cores are free for a query tile's next products
    uint64_t pv[2];       // a query tile's last weighted sum is done: its weights may be overwritten
    uint64_t done[2];
    uint32_t tmem;
    int32_t abort;
    uint32_t loaded;      // K tiles issued so far
    int4 issued[2];       // K and V: tiles issued, edge tiles issued, which of the last tiles were (bit 0: the last)
    // quarters of an edge tile cleaned (by the tile's number: one warp may be a tile ahead), and
    // 1 + the last piece (by its number mod kOddSlots) whose V had values that are not finite
    int32_t fixed[kEdges], odd_values[kOddSlots];
    Start from, to;       // this CTA's range
    int32_t rounds;       // whole items ahead of it
    int64_t cut[2];       // its range of the costs of what is not taken whole
    int4 piece[kPieces][3];  // pieces of it, by their number mod kPieces
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    union {
        longlong2 scan[kThreads / 32 + 1];  // while the work is shared out
        float2 stat[kTile];   // (max, sum) of the odd key tiles, for joining a single query tile
    };
};

// The same of the 8-bit cache, beside it.
struct Shared8 {
    uint64_t kfull[kK8], kempty[kK8];      // tiles of K's codes
    uint64_t rfull[kRaw8], rempty[kRaw8];  // tiles of V's codes, which become f16 tiles of the ring
    uint64_t landed;                       // bf16 query tiles, which become codes
    uint32_t vfactor[kRaw8][kBlkPerTile];  // of V's blocks in their tile (f16, twice); the sign: a mark
    __align__(16) float kscale[kScales8][kBlkPerTile];
    float vexp[kScales8][kBlkPerTile];     // log2 of V's scales over 2^kUpV8
    // of V's tiles: log2 of the scale, its reciprocal and log2 again; blocks apart: kFar8, 0 and 0
    __align__(16) float vtile[kScales8][4];
    // of each row of the query tiles, by the piece's number mod 2: the next piece's are written as soon as this
    // one's last logits are there, and read for its first; those of the one after only behind the next one's logits
    float qscale[2][2][kTile];
};

static_assert(sizeof(Shared) % alignof(Shared8) == 0 && alignof(Shared) >= alignof(Shared8), "Shared8 follows Shared");

// Shared memory: query tiles, the ring, (8 bits: K's codes, V's codes,) barriers and tables.
template <int D, bool E8>
struct Cfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kHalfBytes = kTile * 128;            // 128 rows of 64 dims
    static constexpr int kTileBytes = kHalves * kHalfBytes;   // (8 bits: a query tile is two tiles of codes)
    static constexpr int kRawBytes = kTile * D;               // a tile of codes
    static constexpr int kRingBytes = kStages * kTileBytes + (E8 ? (kK8 + kRaw8) * kRawBytes : 0);
    static constexpr size_t kSmem = 1024 + 2 * kTileBytes + kRingBytes + sizeof(Shared) + (E8 ? sizeof(Shared8) : 0);
};

// Bounded wait on phase `parity` of `bar`: gives up after wait_ns, or once another
// warp of the CTA gave up, recording KARA_ETIMEOUT.  The waits that nap are those of warps with
// nothing to do for as long as an item takes (over 10^8 keys, a second): theirs begin anew
// while key tiles are being loaded.
template <int NAP = 0>
__device__ __forceinline__ bool cwait(uint32_t bar, uint32_t parity, Shared *sh, const ChunkArgs &a)
{
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = 0;
    uint32_t seen = 0;
    for (uint32_t it = 1;; ++it) {
        if (NAP) __nanosleep(NAP);
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (*(volatile int32_t *)&sh->abort) return false;
            const uint64_t now = globaltimer();
            const uint32_t loaded = NAP ? *(volatile uint32_t *)&sh->loaded : 0;
            if (t0 == 0 || loaded != seen) {
                t0 = now, seen = loaded;
            } else if (now - t0 > a.wait_ns) {
                set_err(a.err, KARA_ETIMEOUT);
                *(volatile int32_t *)&sh->abort = 1;
                return false;
            }
        }
    }
}

// The same for the control warps, whose code has to stay small beside the softmax's in the
// instruction caches: the waiting itself is out of line.
template <int NAP>
__device__ __noinline__ bool kwait_on(uint32_t bar, uint32_t parity, Shared *sh, const ChunkArgs &a)
{
    return cwait<NAP>(bar, parity, sh, a);
}

template <int NAP = 0>
__device__ __forceinline__ bool kwait(uint32_t bar, uint32_t parity, Shared *sh, const ChunkArgs &a)
{
    return mbar_try_wait(bar, parity) || kwait_on<NAP>(bar, parity, sh, a);
}

// Wait for work in flight that has to land whatever happened: by time alone.
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity)
{
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer() - t0 > kTimeoutNs) return;
}

// Every K (kv 0) or V (1) tile has landed before the CTA's shared memory is released, also when a wait ran
// out and nobody consumed it: the last issued of each stage (tile i is entry 2 i + kv of the ring; an entry
// kStages further on took the same stage, and took it only behind this one), and the last edge tiles.
__device__ __noinline__ void drain_tiles(Shared *sh, int kv)
{
    const uint32_t k = (uint32_t)sh->issued[kv].x, ne = (uint32_t)sh->issued[kv].y;
    const uint32_t edges = (uint32_t)sh->issued[kv].z, others = (uint32_t)sh->issued[1 - kv].x;
    for (uint32_t d = 1; d <= kEdges && d <= k; ++d) {
        const uint32_t e = 2 * (k - d) + kv;
        if ((e + kStages) / 2 >= others && !(edges >> (d - 1) & 1u))
            drain(smem_u32(&sh->full[e % kStages]), e / kStages & 1);
    }
    for (uint32_t i = ne > kEdges ? ne - kEdges : 0; i < ne; ++i)
        drain(smem_u32(&sh->edge[i % kEdges]), i / kEdges & 1);
}

// One thread of the warp (all of them call it).
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// D[tmem] (+)= A * B[smem], bf16 operands, fp32 accumulate; one thread issues.  A in shared
// memory (with B's upper descriptor word) or in TMEM; descriptors as 32-bit halves.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t alo, uint32_t hi, uint32_t blo, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %2};\n\t"
        "setp.ne.b32 p, %5, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(alo), "r"(hi), "r"(blo), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same with e4m3 operands.
__device__ __forceinline__ void mma_ss_e4m3(uint32_t d_tmem, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi,
                                            uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: kind::f8f6f4 with e4m3 A and B, fp32 D, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Instruction descriptor: kind::f16 with f16 A and B, fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N)
{
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Descriptor of a K-major operand of codes, rows of D bytes swizzled by their size (128 or 64 bytes), groups of
// eight rows one after another.
template <int D>
__device__ __forceinline__ uint64_t sdesc_codes(uint32_t saddr)
{
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)1 << 16;
    d |= (uint64_t)(8 * D >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)(D == 128 ? 2 : 4) << 61;
    return d;
}

__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t bhi, uint32_t idesc,
                                       uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of an operand whose rows (128 bytes, 128-byte swizzle) run along K:
// its M/N dim is contiguous in 64-element pieces `piece` bytes apart, K in groups
// of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_sw128_mn(uint32_t saddr, uint32_t piece)
{
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(piece >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// 32 lanes x 32 consecutive 32-bit columns into v[o..o+31].
template <int N>
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[N], const int o)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[o + 0]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]),
          "=r"(v[o + 6]), "=r"(v[o + 7]), "=r"(v[o + 8]), "=r"(v[o + 9]), "=r"(v[o + 10]), "=r"(v[o + 11]),
          "=r"(v[o + 12]), "=r"(v[o + 13]), "=r"(v[o + 14]), "=r"(v[o + 15]), "=r"(v[o + 16]), "=r"(v[o + 17]),
          "=r"(v[o + 18]), "=r"(v[o + 19]), "=r"(v[o + 20]), "=r"(v[o + 21]), "=r"(v[o + 22]), "=r"(v[o + 23]),
          "=r"(v[o + 24]), "=r"(v[o + 25]), "=r"(v[o + 26]), "=r"(v[o + 27]), "=r"(v[o + 28]), "=r"(v[o + 29]),
          "=r"(v[o + 30]), "=r"(v[o + 31])
        : "r"(taddr));
}

template <int N>
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[N], const int o)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[o + 0]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]),
        "r"(v[o + 7]), "r"(v[o + 8]), "r"(v[o + 9]), "r"(v[o + 10]), "r"(v[o + 11]), "r"(v[o + 12]), "r"(v[o + 13]),
        "r"(v[o + 14]), "r"(v[o + 15]), "r"(v[o + 16]), "r"(v[o + 17]), "r"(v[o + 18]), "r"(v[o + 19]),
        "r"(v[o + 20]), "r"(v[o + 21]), "r"(v[o + 22]), "r"(v[o + 23]), "r"(v[o + 24]), "r"(v[o + 25]),
        "r"(v[o + 26]), "r"(v[o + 27]), "r"(v[o + 28]), "r"(v[o + 29]), "r"(v[o + 30]), "r"(v[o + 31])
        : "memory");
}

// Waits for this thread's tcgen05.ld; ties the 32 registers so no use moves above it.
template <int N>
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&v)[N], const int o)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[o + 0]), "+r"(v[o + 1]), "+r"(v[o + 2]), "+r"(v[o + 3]), "+r"(v[o + 4]), "+r"(v[o + 5]),
                   "+r"(v[o + 6]), "+r"(v[o + 7]), "+r"(v[o + 8]), "+r"(v[o + 9]), "+r"(v[o + 10]), "+r"(v[o + 11]),
                   "+r"(v[o + 12]), "+r"(v[o + 13]), "+r"(v[o + 14]), "+r"(v[o + 15]), "+r"(v[o + 16]),
                   "+r"(v[o + 17]), "+r"(v[o + 18]), "+r"(v[o + 19]), "+r"(v[o + 20]), "+r"(v[o + 21]),
                   "+r"(v[o + 22]), "+r"(v[o + 23]), "+r"(v[o + 24]), "+r"(v[o + 25]), "+r"(v[o + 26]),
                   "+r"(v[o + 27]), "+r"(v[o + 28]), "+r"(v[o + 29])
                 :
                 : "memory");
    asm volatile("" : "+r"(v[o + 30]), "+r"(v[o + 31]) : : "memory");
}

__device__ __forceinline__ void ld_shared4(uint32_t addr, float (&x)[4])
{
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "r"(addr));
}

__device__ __forceinline__ float ld_shared(uint32_t addr)
{
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr));
    return x;
}

// 32 bytes (32-byte aligned) from v[o..o+7].
template <int N>
__device__ __forceinline__ void st_global_32b(void *p, const uint32_t (&v)[N], const int o)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[o + 0]), "r"(v[o + 1]),
                 "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])
                 : "memory");
}

// ---- the cut: every CTA works out its own range ---------------------------------------
// Inclusive scan of two values over the CTA; tot gets the sums.
__device__ longlong2 cta_scan2(longlong2 v, longlong2 *scratch, longlong2 &tot)
{
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
        if (lane >= o) v.x += x, v.y += y;
    }
    if (lane == 31) scratch[warp] = v;
    __syncthreads();
    if (warp == 0) {
        longlong2 w = lane < kWarps ? scratch[lane] : make_longlong2(0, 0);
        const longlong2 own = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, w.x, o), y = __shfl_up_sync(0xffffffffu, w.y, o);
            if (lane >= o) w.x += x, w.y += y;
        }
        if (lane < kWarps) scratch[lane] = make_longlong2(w.x - own.x, w.y - own.y);
        if (lane == kWarps - 1) scratch[kWarps] = w;
    }
    __syncthreads();
    const longlong2 b = scratch[warp];
    tot = scratch[kWarps];
    __syncthreads();
    return make_longlong2(b.x + v.x, b.y + v.y);
}

// Cost and key tiles of a sequence's items.
__device__ __forceinline__ longlong2 seq_cost(const ChunkArgs &a, int seq)
{
    longlong2 v = make_longlong2(0, 0);
    Item it = make_item(a, seq, 0);
    for (int t0 = 0; t0 < it.m; t0 += 2 * a.TQ) {
        const int32_t ntok = min(2 * a.TQ, it.m - t0), nt = (it.pos0 + t0 + ntok - 1) / kTile + 1;
        v.x += (int64_t)nt * tile_cost(a, ntok) + kItemCost;
        v.y += nt;
    }
    return v;
}

// The place at cost r of one head, inside the costs [before, before + its own) of sequence seq.
__device__ __forceinline__ Start place(const ChunkArgs &a, int head, int seq, int64_t before, int64_t r)
{
    Start p;
    p.head = head, p.seq = seq;
    for (p.pair = 0;; ++p.pair) {
        const Item it = make_item(a, seq, p.pair);
        const int w = tile_cost(a, it.ntok);
        const int64_t c = (int64_t)it.nt * w + kItemCost;
        if (r < before + c || (p.pair + 1) * 2 * a.TQ >= it.m) {
            p.off = (int32_t)min((int64_t)it.nt, (r - before) / w);
            return p;
        }
        before += c;
    }
}

// Item i of all, of which each head has per_head; `first` has those ahead of each sequence.
__device__ Start find_item(const ChunkArgs &a, const int32_t *first, int32_t per_head, int32_t i)
{
    const int32_t head = i / per_head, r = i % per_head;
    int lo = 0, hi = a.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= r) lo = mid; else hi = mid;
    }
    return Start{head, lo, r - first[lo], 0};
}

// Whole items go round the CTAs, as many rounds as leave no CTA above the average cost; the rest is
// cut so that all come to it.  False, with nothing done: no sequence has more than one pair of query
// tiles, or there are more sequences and items than fit in the scratch memory (about 40000, or 20000
// at D = 64; working their costs out again for each use would take a tenth of such a call).
__device__ __noinline__ bool whole_items(const ChunkArgs &a, Shared *sh, int ctas, int64_t units, int32_t *scratch,
                                         int scratch_words)
{
    const int tid = threadIdx.x, cta = blockIdx.x;
    bool shared = false;
    for (int s = tid; s < a.n; s += kThreads) shared = shared || make_item(a, s, 0).m > 2 * a.TQ;
    if (!__syncthreads_or(shared) || a.n >= scratch_words) return false;
    int32_t *first = scratch, *cost = scratch + a.n;
    longlong2 tot;
    int64_t per_head = 0;
    for (int base = 0; base < a.n; base += kThreads) {
        const int s = base + tid;
        const int64_t own = s < a.n ? pairs_of(a, s) : 0;
        const longlong2 in = cta_scan2(make_longlong2(own, 0), sh->scan, tot);
        if (s < a.n) first[s] = (int32_t)(per_head + in.x - own);
        per_head += tot.x;
    }
    fence_proxy_async_smem();  // the scratch is the ring of the copies that follow
    if (per_head * a.hkv > scratch_words - a.n) return false;
    const int32_t items = (int32_t)per_head * a.hkv;
    if (tid == 0) sh->rounds = kMaxRounds;
    __syncthreads();
    for (int32_t i = tid; i < items; i += kThreads) {
        const Start p = find_item(a, first, (int32_t)per_head, i);
        const Item it = make_item(a, p.seq, p.pair);
        cost[i] = it.nt * tile_cost(a, it.ntok) + kItemCost;
    }
    __syncthreads();
    const int64_t mean = units / ctas, more = units % ctas;
    int64_t mine = 0;
    if (tid < ctas) {
        int k = 0;
        for (; k < kMaxRounds && k * ctas + ctas <= items; ++k) {
            mine += cost[k * ctas + tid];
            if (mine > mean) break;
        }
        atomicMin(&sh->rounds, k);
    }
    __syncthreads();
    const int rounds = sh->rounds;
    mine = 0;
    if (tid < ctas)
        for (int k = 0; k < rounds; ++k) mine += cost[k * ctas + tid];
    const longlong2 lack = make_longlong2(tid < ctas ? mean - mine : 0, 0), in = cta_scan2(lack, sh->scan, tot);
    if (tid == cta) sh->cut[0] = in.x - lack.x + more * cta / ctas, sh->cut[1] = in.x + more * (cta + 1) / ctas;
    __syncthreads();
    int64_t before = 0;
    for (int32_t base = rounds * ctas; base < items; base += kThreads) {
        const int32_t i = base + tid;
        const int32_t own = i < items ? cost[i] : 0;
        const longlong2 x = cta_scan2(make_longlong2(own, 0), sh->scan, tot);
        const int64_t lo = before + x.x - own, hi = before + x.x;
        for (int e = 0; e < 2; ++e) {
            const int64_t u = sh->cut[e];
            if (lo <= u && u < hi) {
                Start p = find_item(a, first, (int32_t)per_head, i);
                const Item it = make_item(a, p.seq, p.pair);
                p.off = (int32_t)min((int64_t)it.nt, (u - lo) / tile_cost(a, it.ntok));
                if (e) sh->to = p; else sh->from = p;
            }
        }
        before += tot.x;
    }
    if (tid < rounds) a.whole[cta * kMaxRounds + tid] = find_item(a, first, (int32_t)per_head, tid * ctas + cta);
    fence_proxy_async_smem();
    return true;
}

// What this CTA does: sh->rounds whole items (listed in the workspace), then the range from sh->from
// to sh->to of what no CTA takes whole (equal: nothing; kept in the workspace too, for the merge).
// All items' key tiles of all heads, weighted by their cost and laid end to end, are cut into equal
// ranges: prefix sums over the sequences, a thread each (over 512 sequences: in passes, twice over).
// That alone has a CTA read the same keys again for each pair of query tiles, long after they have
// left L2 when there are many caches.  So where items share keys, whole items go round the CTAs
// first, those of the same keys at the same time: 512 tokens x 32 sequences at 4096 keys read 0.70 GB
// from HBM and not 4.24, and take 675 to 715 us captured and not 750 to 780.  It takes about 1.5 us more ahead
// of the first key tile, and gains nothing while a CTA has few: 82 to 86 against 80 us at 40 key tiles
// a CTA, 128 to 132 against 131.5 at 80, 130.6 against 129.7 at 110.  It starts at kSharedTiles = 128.
// Every CTA works all of this out for itself, from the lengths; a plan kernel ahead of this one
// took 3 us more.
__device__ void share_out(const ChunkArgs &a, Shared *sh, int32_t *scratch, int scratch_words)
{
    const int tid = threadIdx.x, cta = blockIdx.x;
    const bool one_pass = a.n <= kThreads;
    longlong2 sum = make_longlong2(0, 0), own = sum, in = sum;
    if (tid == 0) sh->from = sh->to = Start{a.hkv, 0, 0, 0}, sh->rounds = 0;
    for (int base = 0; base < a.n; base += kThreads) {
        const int s = base + tid;
        own = s < a.n ? seq_cost(a, s) : make_longlong2(0, 0);
        longlong2 tot;
        in = cta_scan2(own, sh->scan, tot);
        sum.x += tot.x, sum.y += tot.y;
    }
    const int64_t units = sum.x * a.hkv;
    const int ctas = sum.y == 0 ? 0 : (int)max(1ll, min((long long)a.ctas, sum.y * a.hkv / kTilesPerCta));
    const bool whole = sum.y * a.hkv >= (int64_t)kSharedTiles * a.ctas
                       && whole_items(a, sh, ctas, units, scratch, scratch_words);
    if (!whole && cta < ctas) {
        // (both ends: r = cost within the head; the last range ends with everything)
        const int64_t u0 = units * cta / ctas, u1 = units * (cta + 1) / ctas;
        const int64_t r0 = u0 % sum.x, r1 = u1 % sum.x;
        int64_t before = 0;
        for (int base = 0; base < a.n; base += kThreads) {
            const int s = base + tid;
            longlong2 tot = sum;
            if (!one_pass) {
                own = s < a.n ? seq_cost(a, s) : make_longlong2(0, 0);
                in = cta_scan2(own, sh->scan, tot);
            }
            const int64_t lo = before + in.x - own.x, hi = before + in.x;
            if (lo <= r0 && r0 < hi) sh->from = place(a, (int)(u0 / sum.x), s, lo, r0);
            if (lo <= r1 && r1 < hi && cta + 1 < ctas) sh->to = place(a, (int)(u1 / sum.x), s, lo, r1);
            before += tot.x;
        }
    }
    __syncthreads();
    if (tid == 0) {
        if (cta < ctas) a.start[cta] = sh->from;
        if (cta + 1 == ctas) a.start[ctas] = sh->to;
        if (cta == 0) *a.used_ctas = ctas;
    }
}

// A CTA's range of key tiles, piece by piece.  The warp that loads K, ahead of all others,
// walks over it and tells them (one copy of the walk's code, and few registers elsewhere).
struct Piece {
    Item it;
    int32_t seq, head, j0, j1;  // key tiles [j0, j1)
    bool whole;            // covers the item: the output is written, not a partial
};

// A CTA has at most two partials: one that starts inside an item, one that ends there.
__device__ __forceinline__ int64_t partial_slot(int cta, bool inside) { return 2 * (int64_t)cta + (inside ? 0 : 1); }

struct Walk {
    const ChunkArgs &a;
    const Start *whole;
    int rounds, round;
    Start at, end;
    Item it;  // at `at`
    __device__ Walk(const ChunkArgs &args, const Shared *sh) : a(args)
    {
        whole = a.whole + blockIdx.x * kMaxRounds, rounds = sh->rounds, round = 0;
        at = sh->from, end = sh->to;
        if (at.head < a.hkv) {
            it = make_item(a, at.seq, at.pair);
            if (at.off >= it.nt && !same_item(at, end)) advance();
        }
    }
    __device__ __forceinline__ void advance()
    {
        at.off = 0;
        ++at.pair;
        if (at.pair * 2 * a.TQ >= it.m) {
            at.pair = 0;
            do {
                if (++at.seq == a.n) at.seq = 0, ++at.head;
                it = make_item(a, at.seq, 0);
            } while (it.m == 0);
        } else {
            it = make_item(a, at.seq, at.pair);
        }
    }
    __device__ bool step(Piece &p)
    {
        if (round < rounds) {
            const Start w = whole[round++];
            p.it = make_item(a, w.seq, w.pair);
            p.seq = w.seq;
            p.head = w.head;
            p.j0 = 0;
            p.j1 = p.it.nt;
            p.whole = true;
            return true;
        }
        if (at.head >= a.hkv) return false;
        const bool last = same_item(at, end);
        p.it = it;
        p.seq = at.seq;
        p.head = at.head;
        p.j0 = at.off;
        p.j1 = last ? min(end.off, it.nt) : it.nt;
        if (p.j0 >= p.j1) return false;  // (only at the end)
        p.whole = p.j0 == 0 && p.j1 == it.nt;
        if (last) at.head = a.hkv; else advance();
        return true;
    }
};

// Piece number `n` as the walking warp told it; false: there is none, or a wait ran out.
// (WARP: a whole warp asks, not one thread.)
template <bool WARP, class Wait>
__device__ __forceinline__ bool next_piece(Piece &p, uint32_t n, Shared *sh, bool &ok, int lane, Wait wait)
{
    const int i = n % kPieces;
    ok = wait(smem_u32(&sh->piece_full[i]), n / kPieces & 1);
    if (!ok) return false;
    const int4 u = sh->piece[i][0], v = sh->piece[i][1], w = sh->piece[i][2];
    p.it.row0 = u.x, p.it.ntok = u.y, p.it.pos0 = u.z, p.it.nt = u.w;
    p.it.len = v.x, p.it.m = v.y, p.seq = v.z, p.head = v.w;
    p.j0 = w.x, p.j1 = w.y, p.whole = w.z;
    if (WARP) __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sh->piece_empty[i]));
    return p.j1 > 0;
}

// Key tiles of query tile x in a piece: `cnt` of them, from j, `by` apart.
struct Part {
    int32_t j, by, cnt;
};

__device__ __forceinline__ Part part_of(const Piece &p, int x, int TQ)
{
    Part r;
    if (p.it.ntok > TQ) {  // two query tiles: both take every key tile they see
        const int32_t seen = (p.it.pos0 + min(p.it.ntok, (x + 1) * TQ) - 1) / kTile + 1;
        r.j = p.j0, r.by = 1, r.cnt = max(0, min(p.j1, seen) - p.j0);
    } else {               // one query tile: the even and the odd key tiles of the piece
        r.j = p.j0 + x, r.by = 2, r.cnt = (p.j1 - p.j0 + 1 - x) / 2;
    }
    return r;
}

// Key tile j holds rows that not every row of the item sees: new tokens after the
// item's first, or the rest of the sequence's last block.
__device__ __forceinline__ bool edge_tile(const Item &it, int j)
{
    const int32_t end = it.len - j * kTile;
    return min(end, kTile) > it.pos0 + 1 - j * kTile || (end < kTile && end % kBlk != 0);
}

// A bf16 pair with its infinities and NaNs cleared.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w)
{
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
    return w;
}

// Values of new tokens that are not finite were cleared from V: adds those at positions
// [y0, y1] to a row of the output, or of a partial.
template <int D, bool E8>
__device__ __noinline__ void add_cleared(const ChunkArgs &a, int seq, int head, int y0, int y1, uint16_t *out,
                                         float4 *part)
{
    for (int y = y0; y <= y1; ++y) {
        const int32_t id = a.bt[(int64_t)seq * a.bt_stride + y / kBlk];
        if (id < 0 || id >= a.num_blocks) continue;
        const int64_t at = id * a.block_stride + head * a.head_stride + (int64_t)(y % kBlk) * D;
#pragma unroll 1
        for (int d = 0; d < D; ++d) {
            const uint32_t b = E8 ? ((a.v8[at + d] & 0x7fu) == 0x7fu ? 0x7fffu : 0u) : a.v[at + d];
            if ((b & 0x7f80u) != 0x7f80u) continue;
            const float f = __uint_as_float(b << 16);
            if (out) {
                out[d] = (uint16_t)bf16x2(__uint_as_float((uint32_t)out[d] << 16) + f, 0.f);
            } else {
                float *q = reinterpret_cast<float *>(part + d / 4 * 256) + d % 4;
                *q += f;
            }
        }
    }
}

// ---- the 8-bit cache ------------------------------------------------------------------
// K's codes are an operand of the tensor cores as they are, if the queries are codes too.  A bf16
// value has eight significant bits and a code four: with q' = q 2^k, the row's largest within (224, 448],
//     q' = hi + lo,   hi = rn(q'),  lo = rn(q' - hi)
// exactly while |q'| >= 1/4, and 2^-10 off at most below (2^-17 of the row's largest, or 2^-50).  The logits are then
// Q_hi K^T + Q_lo K^T, at twice the rate of bf16 operands, so in the same time; 2^-k and K's scales multiply them
// in the softmax, where the factor log2(e) / sqrt(D) is anyway.
// V's codes become f16 tiles of the ring, times their block's scale over 2^e, e of the tile's largest; 2^e goes into
// the weights, which are rounded to f16:
//     w_x = 2^(l_x + e - M + kUp8),   O = sum_x w_x (v_x 2^-e),   z = sum over tiles of 2^-e sum_x w_x,
// M the largest l_x + e so far (lazily, as above): weights within 2^-21 of it keep eleven bits, smaller ones are off by
// 2^-32 of it, and with the maximum's growth of 2^8 the largest stay within f16.  That is for tiles whose blocks'
// scales are no more than 2^kApart8 apart: f16 holds their values exactly, and M is at most that much above a row's largest
// weight times its own block's scale, whose 2^-24 bounds the error.  Further apart, a block that a row does not see, or
// gives no weight, would take the others' digits: then each block has an e of its own (logits_apart, out of line: the
// logits are written anew, V's tile holds the codes themselves, and z is summed from weights without e).  So have the
// blocks of tiles with an e below kLeast8, of zeros for one: with M from a tile at 2^57, the scaled weights of keys that
// count in z would leave fp32's range (w is 2^(kUp8 - 24 + kLeast8 - 57) = 2^-114 at least for those within 2^-24 of the
// largest weight).  K's and V's loading warps tell such tiles apart.  A row meets one where its largest logit seems to
// grow beyond all bounds (vtile), in the branch that it takes then anyway: a check of its own in every tile took the mixed
// batch from 368 to 398 us, this leaves it at 367, four tokens for each of 128 sequences at 610 (606), the prompt at
// 1625 to 1635 (1620).
// (As bf16, exact at any scale, two codes took four instructions instead of two, and weights kept eight bits: 64
// sequences of 1 to 128 tokens 387 us and 379, four tokens for each of 128 sequences 611 and 604, one prompt alike.
// With a scale for each block in the weights, and one instruction, the softmax took longer: 409 and 613.)

// The bf16 query tiles of a piece; one thread issues.
template <int D>
__device__ __forceinline__ void load_queries(const Piece &p, uint8_t *qbuf, const CUtensorMap *qmap, uint32_t bar, int qrows,
                                             const ChunkArgs &a)
{
    using C = Cfg<D, true>;
    const int tiles = p.it.ntok > a.TQ ? 2 : 1;
    mbar_arrive_expect_tx(bar, tiles * C::kHalves * qrows * 128);
    for (int x = 0; x < tiles; ++x)
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h)
            asm volatile(
                "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(qbuf + x * C::kTileBytes + h * C::kHalfBytes)),
                "l"(reinterpret_cast<uint64_t>(qmap)), "r"(h * 64), "r"(p.head * a.G), "r"(p.it.row0 + x * a.TQ),
                "r"(bar)
                : "memory");
}

// Rows [32 w, 32 w + 32) of each query tile as codes, in place, and their 2^-k.  D = 128: of a bf16 row's two
// 128-byte halves the first becomes hi and the second lo; D = 64: its 128 bytes are hi, then lo.  (Loaded into
// registers from global memory instead, two rows at a time, they kept the products waiting for 15 us an item.)
template <int D>
__device__ __forceinline__ void split_queries(int tiles, int w, uint8_t *qbuf, float (*qscale)[kTile])
{
    using C = Cfg<D, true>;
    constexpr int LPR = D / 8, RPP = 32 / LPR, kAhead = 4;
    const int lane = threadIdx.x & 31, l = lane % LPR;
#pragma unroll 1
    for (int r0 = 0; r0 < tiles * 32; r0 += kAhead * RPP) {
        const int x = r0 >> 5, rx = w * 32 + (r0 & 31) + lane / LPR;
        uint8_t *q = qbuf + x * C::kTileBytes;
        uint4 u[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = rx + i * RPP;
            u[i] = *reinterpret_cast<const uint4 *>(q + (l >> 3) * C::kHalfBytes + r * 128 + (((l & 7) ^ (r & 7)) << 4));
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = rx + i * RPP;
            const uint32_t v[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
            // the largest finite magnitude, as bits: of 16-bit patterns below 0x7f80
            uint32_t top = 0;
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t m0 = v[e] & 0x7fffu, m1 = v[e] >> 16 & 0x7fffu;
                if (m0 < 0x7f80u) top = max(top, m0); else odd = true;
                if (m1 < 0x7f80u) top = max(top, m1); else odd = true;
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            // the exponent of q' is 8 for mantissas up to 1.75 (448), 7 above; 2^-k at least 2^-40, so that
            // times the smallest scale it is no 0 (which a masked logit's infinity would turn to NaN)
            const int down = min(max((int)((top + 0x1fu) >> 7) - 8, 127 - 40), 253);
            const float f = __uint_as_float((uint32_t)(254 - down) << 23);
            if (l == 0) qscale[x][r] = __uint_as_float((uint32_t)down << 23);
            uint32_t h[2] = {0u, 0u}, g[2] = {0u, 0u};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float q0 = __uint_as_float(v[e] << 16) * f, q1 = __uint_as_float(v[e] & 0xffff0000u) * f;
                if (odd) {  // NaN for what is not finite: the row's logits are
                    if (!finite(q0)) q0 = __uint_as_float(0x7fffffffu);
                    if (!finite(q1)) q1 = __uint_as_float(0x7fffffffu);
                }
                const uint32_t c = e4m3x2(q0, q1);
                float c0, c1;
                f32_of_f16x2(f16_of_e4m3x2(c), c0, c1);
                h[e >> 1] |= c << (16 * (e & 1));
                g[e >> 1] |= e4m3x2(q0 - c0, q1 - c1) << (16 * (e & 1));
            }
            __syncwarp();  // (the whole row has been read)
            // eight codes, half of a 16-byte chunk, of hi and of lo
            uint8_t *o = q + r * 128 + (l & 1) * 8;
            const int c = l >> 1, d = D == 128 ? c : c + 4, sw = r & 7;
            *reinterpret_cast<uint2 *>(o + ((c ^ sw) << 4)) = make_uint2(h[0], h[1]);
            *reinterpret_cast<uint2 *>(o + (D == 128 ? C::kHalfBytes : 0) + ((d ^ sw) << 4)) = make_uint2(g[0], g[1]);
        }
    }
}

// A scale's log2, between -63 and 63 whatever it is (-63 for 0).
__device__ __forceinline__ int scale_log2(float s)
{
    return min(max((int)(__float_as_uint(s) >> 23 & 255u) - 127, -63), 63);
}

// 2^e as f16 in both halves, e <= 15: subnormal from 2^-15 on, 0 below 2^-24.
__device__ __forceinline__ uint32_t f16_power2(int e)
{
    const uint32_t h = e >= -14 ? (uint32_t)(e + 15) << 10 : e >= -24 ? 1u << (e + 24) : 0u;
    return h | h << 16;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Where a lane's 16-byte chunk of codes (of rows 32 / (D/16) apart) goes in an f16 tile of the 128-byte
// swizzled layout: two chunks of a 64-dim half.  Lanes of the upper half begin with the second, so that
// eight lanes write to all banks.
template <int D>
struct LaneChunk {
    static constexpr int CPR = D / 16, kRows = 32 / CPR;  // chunks of a row, rows of a pass
    int row, odd, src, dst, first, second;
    __device__ explicit LaneChunk(int lane)
    {
        const int c = lane % CPR, at = 2 * (c & 3);
        row = lane / CPR, odd = c >> 2;
        src = row * D + c * 16;
        dst = odd * kTile * 128 + row * 128;
        first = ((at + odd) ^ row) << 4, second = ((at + 1 - odd) ^ row) << 4;  // (D = 128: row < 4; 64: row < 8)
    }
    // both chunks of pass i, from words in the order of `swapped`
    __device__ __forceinline__ void store(uint8_t *tile, int i, const uint32_t (&r)[8]) const
    {
        uint8_t *o = tile + dst + i * kRows * 128;
        const int turn = i * kRows << 4 & 0x70;  // the rest of row mod 8
        *reinterpret_cast<uint4 *>(o + (first ^ turn)) = make_uint4(r[0], r[1], r[2], r[3]);
        *reinterpret_cast<uint4 *>(o + (second ^ turn)) = make_uint4(r[4], r[5], r[6], r[7]);
    }
    __device__ __forceinline__ void swapped(const uint4 &w, uint32_t (&u)[4]) const
    {
        u[0] = odd ? w.z : w.x, u[1] = odd ? w.w : w.y, u[2] = odd ? w.x : w.z, u[3] = odd ? w.y : w.w;
    }
};

// Sixteen codes times f, as f16.
__device__ __forceinline__ void convert16(const uint32_t (&u)[4], uint32_t f, uint32_t (&r)[8])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        r[2 * k] = mul_f16x2(f16_of_e4m3x2(u[k] & 0xffffu), f);
        r[2 * k + 1] = mul_f16x2(f16_of_e4m3x2(u[k] >> 16), f);
    }
}

// A block of codes as f16 rows.
template <int D>
__device__ __forceinline__ void convert_block(const uint8_t *raw, uint8_t *tile, uint32_t f, const LaneChunk<D> &lc)
{
    constexpr int NP = kBlk / LaneChunk<D>::kRows;
    uint4 w[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) w[i] = *reinterpret_cast<const uint4 *>(raw + lc.src + i * LaneChunk<D>::kRows * D);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        uint32_t u[4], r[8];
        lc.swapped(w[i], u);
        convert16(u, f, r);
        lc.store(tile, i, r);
    }
}

// The same of a block with something out of the ordinary: rows from `end` on, which become zeros; a mark, NaN
// codes: those of rows from `clear` on become 0 and are reported.
template <int D>
__device__ __noinline__ bool convert_odd_block(const uint8_t *raw, uint8_t *tile, int end, int clear, uint32_t f, int lane)
{
    const LaneChunk<D> lc(lane);
    bool found = false;
#pragma unroll 1
    for (int i = 0; i < kBlk / LaneChunk<D>::kRows; ++i) {
        const int row = i * LaneChunk<D>::kRows + lc.row;
        const uint4 w = row < end ? *reinterpret_cast<const uint4 *>(raw + lc.src + i * LaneChunk<D>::kRows * D)
                                  : make_uint4(0, 0, 0, 0);
        uint32_t u[4], r[8];
        lc.swapped(w, u);
        convert16(u, f & 0x7fff7fffu, r);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t t = k & 1 ? u[k / 2] >> 16 : u[k / 2];
            const bool lo = (t & 0x7fu) == 0x7fu, hi = (t & 0x7f00u) == 0x7f00u;
            if (row >= clear && (lo || hi)) {
                found = true;
                r[k] &= (lo ? 0u : 0xffffu) | (hi ? 0u : 0xffff0000u);
            }
        }
        lc.store(tile, i, r);
    }
    return found;
}

// Warps 12 to 15: a piece's queries (a quarter of their rows each), then its V tiles (two blocks each), with
// what rows must not see cleared on the way.
template <int D>
__device__ __forceinline__ void convert_tiles(int cw, uint8_t *qbuf, uint8_t *ring, const uint8_t *raw, Shared *sh,
                                              Shared8 *sh8, const CUtensorMap *qmap, int qrows, const ChunkArgs &a)
{
    using C = Cfg<D, true>;
    const int lane = threadIdx.x & 31;
    const LaneChunk<D> lc(lane);
    Piece p;
    uint32_t np = 0, nq = 0, k = 0;   // pieces, query tiles issued, V tiles
    uint32_t st = 0, ph = 1;  // the next stage of the ring and the phase that frees it
    bool ok = true;
    const auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, kwait<20>(bar, parity, sh, a)) != 0;
    };
    for (; ok && !a.stall && next_piece<true>(p, np, sh, ok, lane, wait); ++np) {
        if (cw == 0) {
            ok = wait(smem_u32(&sh->q_empty), (np & 1) ^ 1);
            if (!ok) break;
            if (lane == 0) load_queries<D>(p, qbuf, qmap, smem_u32(&sh8->landed), qrows, a);
            __syncwarp();
            ++nq;
        }
        ok = wait(smem_u32(&sh8->landed), np & 1);
        if (!ok) break;
        split_queries<D>(p.it.ntok > a.TQ ? 2 : 1, cw, qbuf, sh8->qscale[np & 1]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh->q_full));
        for (int j = p.j0; j < p.j1; ++j, ++k) {
            const uint32_t r = k % kRaw8;
            ok = wait(smem_u32(&sh8->rfull[r]), k / kRaw8 & 1) && wait(smem_u32(&sh->empty[st]), ph);
            if (!ok) break;
            // rows from `end` on: past the sequence; from `clear` on: not seen by every row of the item
            const int end = p.it.len - j * kTile, clear = p.it.pos0 + 1 - j * kTile;
            bool found = false;
#pragma unroll 1
            for (int b = 2 * cw; b < 2 * cw + 2; ++b) {
                const uint32_t f = sh8->vfactor[r][b];
                const uint8_t *src = raw + r * C::kRawBytes + b * kBlk * D;
                uint8_t *dst = ring + st * C::kTileBytes + b * kBlk * 128;
                if (__builtin_expect((int32_t)f >= 0 && end >= (b + 1) * kBlk, 1))
                    convert_block<D>(src, dst, f, lc);
                else
                    found = convert_odd_block<D>(src, dst, end - b * kBlk, clear - b * kBlk, f, lane) || found;
            }
            if (found) sh->odd_values[np % kOddSlots] = (int32_t)np + 1;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(smem_u32(&sh->full[st]));
                mbar_arrive(smem_u32(&sh8->rempty[r]));
            }
            if (++st == kStages) st = 0, ph ^= 1;
        }
    }
    // the last query tiles have landed too
    if (nq > 0) drain(smem_u32(&sh8->landed), (nq - 1) & 1);
}

// z times 2^x, x up to 0.  With the 8-bit cache's V scales in its reference a sum of weights may be far above 1, and count
// although 2^x itself is below fp32's range: half of x at a time.
template <bool E8>
__device__ __forceinline__ float scale_sum(float z, float x, float f)
{
    if (!E8) return z * f;
    const float h = ex2(0.5f * x);
    return z * h * h;
}

// The reference m of a row's exponentials becomes mt if that is much larger, and its sums z and O (in TMEM) follow.
template <int D, bool E8>
__device__ __forceinline__ void raise_reference(uint32_t to, float mt, float &m, float &z)
{
    const bool grew = mt > m + kLazy;
    const float f = grew ? ex2(m - mt) : 1.f;
    z = scale_sum<E8>(z, grew ? m - mt : 0.f, f);
    if (grew) m = mt;
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(to + c, o, 0);
        tmem_wait_ld32(o, 0);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
        tmem_st32(to + c, o, 0);
    }
    tmem_wait_st();
}

// A row's logits in a key tile whose blocks of V are apart: log2 of a block's scale, and not of the tile's, goes into its
// keys' logits (in TMEM; -infinity for those that the row does not see), and the weights without it into z.  Returns
// the row's m and z.  (Inside the loop that calls it this made the ordinary tiles 10 % slower; with all 128 logits in
// registers at once, 2 %.  If every tile is like that, four tokens for each of 128 sequences take 1130 us instead of 610, the
// mixed batch 500 instead of 367, a prompt of 8192 tokens 2000 instead of 1625; 32 logits at a time, each with factors
// of its own, 2870, 930 and 3410.)
template <int D>
__device__ __noinline__ float2 logits_apart(uint32_t ts, uint32_t to, const float *kscale, const float *vexp, float scale2,
                                            int lim, bool first, float2 mz)
{
    float mt = -INFINITY;
#pragma unroll 1
    for (int c0 = 0; c0 < kTile; c0 += 64) {
        uint32_t s[64];
#pragma unroll
        for (int c = 0; c < 64; c += 32) tmem_ld32(ts + c0 + c, s, c);
#pragma unroll
        for (int c = 0; c < 64; c += 32) tmem_wait_ld32(s, c);
#pragma unroll
        for (int b = 0; b < 64 / kBlk; ++b) {
            const float f = scale2 * kscale[c0 / kBlk + b], e = vexp[c0 / kBlk + b] / f;
            float most = -INFINITY;
#pragma unroll
            for (int c = b * kBlk; c < b * kBlk + kBlk; ++c) {
                const float l = c0 + c <= lim ? __uint_as_float(s[c]) + e : -INFINITY;
                most = fmaxf(most, l);
                s[c] = __float_as_uint(l);
            }
            mt = fmaxf(mt, most * f);
        }
#pragma unroll
        for (int c = 0; c < 64; c += 32) tmem_st32(ts + c0 + c, s, c);
    }
    tmem_wait_st();
    if (first)
        mz.x = mt;
    else if (__any_sync(0xffffffffu, mt > mz.x + kLazy))
        raise_reference<D, true>(to, mt, mz.x, mz.y);
    const float up = kUp8 - (mz.x == -INFINITY ? 0.f : mz.x);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int c0 = 0; c0 < kTile; c0 += 64) {
        uint32_t s[64];
#pragma unroll
        for (int c = 0; c < 64; c += 32) tmem_ld32(ts + c0 + c, s, c);
#pragma unroll
        for (int c = 0; c < 64; c += 32) tmem_wait_ld32(s, c);
#pragma unroll
        for (int b = 0; b < 64 / kBlk; ++b) {
            const float f = scale2 * kscale[c0 / kBlk + b], e = up - vexp[c0 / kBlk + b];
#pragma unroll
            for (int c = b * kBlk; c < b * kBlk + kBlk; ++c) sum[c & 3] += ex2(fmaf(__uint_as_float(s[c]), f, e));
        }
    }
    mz.y += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    return mz;
}

// Records the sequences whose rows or lengths are out of order and zeroes their rows.
__device__ __noinline__ void refuse_sequences(const ChunkArgs &a)
{
    for (int s = threadIdx.x; s < a.n; s += kThreads) {
        const int32_t r0 = a.q_start[s], r1 = a.q_start[s + 1];
        if (chunk_ok(a, r0, r1, a.len[s])) continue;
        set_err(a.err, KARA_EINVAL);
        const int64_t words = (int64_t)a.hq * a.D / 2, hi = min(r1, a.rows) * words;
        for (int64_t i = max(r0, 0) * words; i < hi; ++i) reinterpret_cast<uint32_t *>(a.out)[i] = 0u;
    }
}

// The MMAs of query tile x, issued by one thread: of this warp alone, as an issue takes
// a thread about 40 clocks and the tensor cores 64, so that one thread for both tiles
// would set the pace.  The warps of both tiles walk every K and V tile in ring order (one
// that the query tile skips is handed back at once), so each sees every phase of every
// stage.  With two query tiles they take turns: first one tile's weighted sum and next
// logits, then the other's, so that one tile is multiplied while the other is
// exponentiated.  A tile's next logits overwrite its weights in TMEM, so they wait until the
// weighted sum is done: PTX keeps two MMAs in order only if they have the same accumulator
// and shape.  (The wait takes the long prompt from 1330 to 1355 us, the mixed batch from 335
// to 341, and costs few rows nothing.  Passing the turn on ahead of it, so that the other
// tile's sum is multiplied meanwhile: 1420 and 357.  Polling: 1410 and 349.)
// Descriptors are 32-bit sums, and both tiles share one copy of the code: beside two busy
// softmax warps every instruction between two MMAs counts, and every line of the
// instruction caches.
template <int D, bool E8>
__device__ __forceinline__ void mma_warp(int x, uint32_t qbuf, uint32_t ring, Shared *sh, Shared8 *sh8, const ChunkArgs &a)
{
    using C = Cfg<D, E8>;
    if (elect_one()) {
        constexpr uint32_t id_qk = E8 ? idesc_e4m3(kTile, kTile) : idesc_bf16(kTile, kTile);
        // V: its dims are contiguous
        constexpr uint32_t id_pv = (E8 ? idesc_f16(kTile, D) : idesc_bf16(kTile, D)) | (1u << 16);
        constexpr uint32_t kTileDesc = C::kTileBytes >> 4, kHalfDesc = C::kHalfBytes >> 4;
        const uint32_t ts = x * kTile, to = 256 + x * 128;         // S (and P over it), O in TMEM
        const uint32_t kring = E8 ? ring + kStages * C::kTileBytes : ring;
        const uint64_t qd = sdesc_sw128(qbuf);
        const uint64_t kd = E8 ? sdesc_codes<D>(kring) : sdesc_sw128(kring), vd = sdesc_sw128_mn(ring, C::kHalfBytes);
        constexpr uint32_t kKeyDesc = E8 ? C::kRawBytes >> 4 : kTileDesc;
        const uint32_t full0 = smem_u32(&sh->full[0]), empty0 = smem_u32(&sh->empty[0]);
        // K's tiles share the ring with V's, or have one of their own
        const uint32_t kfull0 = E8 ? smem_u32(&sh8->kfull[0]) : full0, kempty0 = E8 ? smem_u32(&sh8->kempty[0]) : empty0;
        const uint32_t sf = smem_u32(&sh->s_full[x]), pf = smem_u32(&sh->p_full[x]), ph = smem_u32(&sh->p_half[x]);
        const uint32_t pv = smem_u32(&sh->pv[x]), mine = smem_u32(&sh->turn[x]), other = smem_u32(&sh->turn[1 - x]);
        Piece p;
        const auto wait = [&](uint32_t bar, uint32_t parity) { return kwait(bar, parity, sh, a); };
        uint32_t np = 0;
        uint32_t ks = 0, kp = 0, vs = E8 ? 0 : 1, vp = 0;  // next K and V tile: stage, phase
        uint32_t pp = 0, turn = 1 - x, iq = 0;    // phases of the next weights, turn, query tiles
        uint32_t sums = 0;                        // weighted sums issued
        bool ok = true;
        auto next = [](uint32_t &st, uint32_t &ph, int stages) {  // a tile further (K and V alternate)
            st += E8 ? 1 : 2;
            if (st >= stages) st -= stages, ph ^= 1;
        };
        auto next_k = [&]() { next(ks, kp, E8 ? kK8 : kStages); };
        auto next_v = [&]() { next(vs, vp, kStages); };
        auto skip_k = [&]() {
            ok = ok && kwait(kfull0 + ks * 8, kp, sh, a);
            if (ok) mbar_arrive(kempty0 + ks * 8);
            next_k();
        };
        auto skip_v = [&]() {
            ok = ok && kwait(full0 + vs * 8, vp, sh, a);
            if (ok) mbar_arrive(empty0 + vs * 8);
            next_v();
        };
        while (ok && next_piece<false>(p, np, sh, ok, 0, wait)) {
            ++np;
            const bool two = p.it.ntok > a.TQ;
            const int n = p.j1 - p.j0, cnt = part_of(p, x, a.TQ).cnt;
            const int by = two ? 1 : 2, first = two ? 0 : x, last = first + (cnt - 1) * by;
            const uint32_t ql = (uint32_t)qd + (two && x ? kTileDesc : 0);
            ok = kwait(smem_u32(&sh->q_full), iq & 1, sh, a);
            iq ^= 1;
            if (ok && cnt == 0) mbar_arrive(smem_u32(&sh->q_empty));
            for (int t = first - by; ok && t < n; t += by) {
                // weighted sum of tile t, then logits of tile t + by (a single query tile: its own
                // tiles, between the other warp's)
                const bool sum = t >= first && t <= last, logits = t + by <= last;
                if (!two && x == 1 && t >= 0) skip_v();
                if (t >= first && t < n) {
                    ok = ok && kwait(full0 + vs * 8, vp, sh, a);
                    if (two && ok && t + 1 < n) ok = kwait(kfull0 + ks * 8, kp, sh, a);
                    if (two && ok) ok = kwait(mine, turn, sh, a);
                    if (ok && sum) ok = kwait(ph, pp, sh, a);
                    if (!ok) break;
                    if (sum) {
                        tc_fence_after();
                        const uint32_t lo = (uint32_t)vd + vs * kTileDesc;
#pragma unroll
                        for (int e = 0; e < kTile / 32; ++e)
                            mma_ts(to, ts + e * 8, lo + e * 128, (uint32_t)(vd >> 32), id_pv, e > 0 || t != first);
                        ok = kwait(pf, pp, sh, a);
                        if (!ok) break;
                        pp ^= 1;
                        tc_fence_after();
#pragma unroll
                        for (int e = kTile / 32; e < kTile / 16; ++e)
                            mma_ts(to, ts + e * 8, lo + e * 128, (uint32_t)(vd >> 32), id_pv, 1);
                        mma_commit(pv);
                        ++sums;
                        if (!two) mma_commit(empty0 + vs * 8);
                        if (t == last) mma_commit(smem_u32(&sh->o_full[x]));
                    } else {
                        mbar_arrive(empty0 + vs * 8);
                    }
                }
                const uint32_t v_done = empty0 + vs * 8;
                if (t >= first && t < n) next_v();
                if (!two && x == 0 && t >= 0 && t + 1 < n) skip_v();
                if (!two && x == 1 && t + 1 < n) skip_k();
                if (t + by < n) {
                    if (!two || t < first) ok = ok && kwait(kfull0 + ks * 8, kp, sh, a);
                    if (!ok) break;
                    if (logits) {
                        // they go where the weights are: only once the sum of those is done
                        if (sums > 0) ok = kwait(pv, (sums - 1) & 1, sh, a);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t lo = (uint32_t)kd + ks * kKeyDesc;
                        if constexpr (E8) {
#pragma unroll
                            for (int e = 0; e < D / 16; ++e)  // 32 dims of the first term, then of the second
                                mma_ss_e4m3(ts, ql + ((e & 1) * (D == 128 ? kHalfDesc : 4) + (e >> 1) * 2), (uint32_t)(qd >> 32),
                                            lo + (e >> 1) * 2, (uint32_t)(kd >> 32), id_qk, e > 0);
                        } else {
#pragma unroll
                        for (int e = 0; e < D / 16; ++e)
                            mma_ss(ts, ql + ((e >> 2) * kHalfDesc + (e & 3) * 2), (uint32_t)(qd >> 32),
                                   lo + ((e >> 2) * kHalfDesc + (e & 3) * 2), id_qk, e > 0);
                        }
                    }
                }
                if (two && t >= first) {
                    turn ^= 1;
                    mbar_arrive(other);
                }
                if (t + by < n) {
                    if (logits) {
                        mma_commit(sf);
                        mma_commit(kempty0 + ks * 8);
                        if (t + by == last) mma_commit(smem_u32(&sh->q_empty));
                    } else {
                        mbar_arrive(kempty0 + ks * 8);
                    }
                    next_k();
                }
                if (two && sum) mma_commit(v_done);
                if (!two && x == 0 && t + by + 1 < n) skip_k();
            }
            if (!two && x == 1 && ok && n % 2) skip_v();
        }
        // the tensor cores are idle before TMEM and shared memory go
        mma_commit(smem_u32(&sh->done[x]));
        drain(smem_u32(&sh->done[x]), 0);
    }
    __syncwarp();
}

template <int D, bool E8>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ CUtensorMap qmap, const __grid_constant__ ChunkArgs a)
{
    using C = Cfg<D, E8>;
    extern __shared__ uint8_t csm_raw[];
    uint8_t *qbuf = csm_raw + ((1024u - (smem_u32(csm_raw) & 1023u)) & 1023u);  // two query tiles
    uint8_t *ring = qbuf + 2 * C::kTileBytes;
    Shared *sh = reinterpret_cast<Shared *>(ring + C::kRingBytes);
    Shared8 *sh8 = reinterpret_cast<Shared8 *>(sh + 1);  // (of the 8-bit cache)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&sh->full[i]), E8 ? 4 : 1);  // 4: the warps that convert it
            mbar_init(smem_u32(&sh->empty[i]), 2);
        }
        for (int i = 0; E8 && i < kK8; ++i) {
            mbar_init(smem_u32(&sh8->kfull[i]), 1);
            mbar_init(smem_u32(&sh8->kempty[i]), 2);
        }
        if (E8) mbar_init(smem_u32(&sh8->landed), 1);
        for (int i = 0; E8 && i < kRaw8; ++i) {
            mbar_init(smem_u32(&sh8->rfull[i]), 1);
            mbar_init(smem_u32(&sh8->rempty[i]), 4);
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(smem_u32(&sh->piece_full[i]), 1);
            mbar_init(smem_u32(&sh->piece_empty[i]), kPieceReaders);
        }
        mbar_init(smem_u32(&sh->q_full), E8 ? 4 : 1);
        mbar_init(smem_u32(&sh->q_empty), 2);
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&sh->s_full[x]), 1);
            mbar_init(smem_u32(&sh->p_half[x]), 4);
            mbar_init(smem_u32(&sh->p_full[x]), 4);
            mbar_init(smem_u32(&sh->o_full[x]), 1);
        }
        mbar_init(smem_u32(&sh->x_full), 4);
        mbar_init(smem_u32(&sh->x_free), 4);
        for (int i = 0; i < kEdges; ++i) mbar_init(smem_u32(&sh->edge[i]), 1);
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_u32(&sh->turn[x]), 1);
            mbar_init(smem_u32(&sh->pv[x]), 1);
            mbar_init(smem_u32(&sh->done[x]), 1);
        }
        sh->abort = 0;
        sh->loaded = 0;
        for (int i = 0; i < kEdges; ++i) sh->fixed[i] = 0;
        for (int i = 0; i < kOddSlots; ++i) sh->odd_values[i] = 0;
        fence_mbarrier_init();
    }
    // rows of the query tiles past G * TQ are never filled: zeros
    const int qrows = a.G * a.TQ;
    for (int i = tid; !E8 && i < (kTile - qrows) * 8 * 2 * C::kHalves; i += kThreads) {
        const int b = i / ((kTile - qrows) * 8), r = i % ((kTile - qrows) * 8);
        reinterpret_cast<uint4 *>(qbuf + b * C::kHalfBytes + qrows * 128)[r] = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(&sh->tmem), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;  // every column is this CTA's: the allocation starts at 0
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x == gridDim.x - 1) refuse_sequences(a);
    share_out(a, sh, reinterpret_cast<int32_t *>(ring), C::kRingBytes / 4);

    if (warp >= 8) {
        reg_dealloc<Regs<E8>::kCtl>();
        if (warp == kWarpKv || warp == kWarpKv + 1) {
            // ---------------- K tiles (warp 8) and V tiles (warp 9): a tile is 8 blocks x (D/64)
            // halves, a lane per copy.  Issuing a 2 KB copy takes about 90 clocks, so one warp for
            // both would take 2900 clocks for what two query tiles multiply in 2048.
            const int kv = warp - kWarpKv;
            const CUtensorMap *map = kv ? &vmap : &kmap;
            Walk w(a, sh);
            Piece p;
            const auto wait = [&](uint32_t bar, uint32_t parity) {
                return __all_sync(0xffffffffu, kwait(bar, parity, sh, a));
            };
            uint32_t np = 0;
            uint32_t st = E8 ? 0 : kv, ph = 1, k = 0;  // stage and the phase that frees it; tiles issued
            uint32_t ne = 0, were_edges = 0;  // edge tiles issued; which of the last tiles were
            const int b = lane % kBlkPerTile, h = lane / kBlkPerTile;
            const bool mine = E8 ? h == 0 : h < C::kHalves;
            bool ok = !a.stall;
            while (ok) {
                if (kv == 0) {
                    const bool more = w.step(p);
                    const int i = np % kPieces;
                    ok = wait(smem_u32(&sh->piece_empty[i]), (np / kPieces & 1) ^ 1);
                    if (!ok) break;
                    if (lane == 0) {
                        sh->piece[i][0] = make_int4(p.it.row0, p.it.ntok, p.it.pos0, p.it.nt);
                        sh->piece[i][1] = make_int4(p.it.len, p.it.m, p.seq, p.head);
                        sh->piece[i][2] = make_int4(p.j0, more ? p.j1 : 0, p.whole, 0);
                        mbar_arrive(smem_u32(&sh->piece_full[i]));
                    }
                    if (!more) break;
                } else if (!next_piece<true>(p, np, sh, ok, lane, wait)) {
                    break;
                }
                ++np;
                const int32_t *row = a.bt + (int64_t)p.seq * a.bt_stride;
                const int32_t nblk = (p.it.len + kBlk - 1) / kBlk;
                auto block_id = [&](int j) -> int32_t {
                    const int i = j * kBlkPerTile + b;
                    int32_t id = a.num_blocks;  // past the pool: zeros
                    if (i < nblk) {
                        id = row[i];
                        if (id < 0 || id >= a.num_blocks) {
                            set_err(a.err, KARA_EBADBLOCK);
                            id = a.num_blocks;
                        }
                    }
                    return id;
                };
                if constexpr (E8) {
                    // a tile of codes and its blocks' scales; ids are looked up two tiles ahead, scales one
                    const int stages = kv ? kRaw8 : kK8;
                    uint8_t *codes = ring + kStages * C::kTileBytes + kv * kK8 * C::kRawBytes;
                    const auto scale = [&](const float *scales, int32_t id) {
                        return id < a.num_blocks ? scales[(int64_t)id * a.hkv + p.head] : 0.f;
                    };
                    int32_t id = block_id(p.j0), next_id = p.j0 + 1 < p.j1 ? block_id(p.j0 + 1) : a.num_blocks;
                    float vs = scale(a.v_scale, id), ks = kv ? 0.f : scale(a.k_scale, id);
                    for (int j = p.j0; j < p.j1; ++j) {
                        const uint32_t fb = smem_u32((kv ? sh8->rfull : sh8->kfull) + st);
                        ok = __all_sync(0xffffffffu, kwait(smem_u32((kv ? sh8->rempty : sh8->kempty) + st), ph, sh, a));
                        if (!ok) break;
                        const bool live = mine && j * kBlkPerTile + b < nblk;
                        const int e = mine ? scale_log2(vs) : -63;
                        const int et = __reduce_max_sync(0xffffffffu, e) - kUpV8;
                        const bool apart = et < kLeast8 || __any_sync(0xffffffffu, live && e < et + kUpV8 - kApart8);
                        if (kv) {
                            if (mine)
                                sh8->vfactor[st][b] =
                                    f16_power2(apart ? kUpV8 : e - et) | (__float_as_uint(vs) & 0x80000000u);
                        } else {
                            // (codes of zeros alone are what they are at any scale, and 0 times a
                            // masked logit's infinity is none)
                            if (mine) sh8->kscale[k % kScales8][b] = ks == 0.f ? 1.f : fabsf(ks);
                            if (mine) sh8->vexp[k % kScales8][b] = (float)(e - kUpV8);
                            if (lane == 0)
                                *reinterpret_cast<float4 *>(sh8->vtile[k % kScales8]) =
                                    apart ? make_float4(kFar8, 0.f, 0.f, 0.f)
                                          : make_float4((float)et, __uint_as_float((uint32_t)(127 - et) << 23), (float)et, 0.f);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive_expect_tx(fb, C::kRawBytes);
                        __syncwarp();
                        if (mine)
                            tma_load_5d(smem_u32(codes + st * C::kRawBytes + b * kBlk * D), map, fb, 0, 0, p.head, id,
                                        a.layer);
                        ++k;
                        if (kv == 0 && lane == 0) *(volatile uint32_t *)&sh->loaded = k;
                        if (++st == stages) st = 0, ph ^= 1;
                        id = next_id;
                        vs = scale(a.v_scale, id);
                        if (kv == 0) ks = scale(a.k_scale, id);
                        if (j + 2 < p.j1) next_id = block_id(j + 2);
                    }
                    continue;
                }
                int32_t id = block_id(p.j0);
                for (int j = p.j0; j < p.j1; ++j) {
                    const int32_t cur = id;
                    if (j + 1 < p.j1) id = block_id(j + 1);
                    ok = __all_sync(0xffffffffu, kwait(smem_u32(&sh->empty[st]), ph, sh, a));
                    if (!ok) break;
                    const bool edge = kv && edge_tile(p.it, j);
                    const uint32_t fb = smem_u32(edge ? &sh->edge[ne % kEdges] : &sh->full[st]);
                    ne += edge;
                    were_edges = were_edges << 1 | (edge ? 1u : 0u);
                    if (lane == 0) mbar_arrive_expect_tx(fb, C::kTileBytes);
                    __syncwarp();
                    if (mine)
                        tma_load_5d(smem_u32(ring + st * C::kTileBytes + h * C::kHalfBytes + b * kBlk * 128), map, fb,
                                    h * 64, 0, p.head, cur, a.layer);
                    ++k;
                    if (kv == 0 && lane == 0) *(volatile uint32_t *)&sh->loaded = k;
                    st += 2;
                    if (st >= kStages) st -= kStages, ph ^= 1;
                }
            }
            if (lane == 0) sh->issued[kv] = make_int4((int)k, (int)ne, (int)were_edges, 0);
        } else if (warp == kWarpMma || warp == kWarpMma + 1) {
            mma_warp<D, E8>(warp - kWarpMma, smem_u32(qbuf), smem_u32(ring), sh, sh8, a);
        } else if constexpr (E8) {
            convert_tiles<D>(warp - kWarpQ, qbuf, ring, ring + kStages * C::kTileBytes + kK8 * C::kRawBytes, sh, sh8,
                             &qmap, qrows, a);
        } else {
            // ---------------- query tiles (warp 12), and the edge tiles of V (warps 12-15, a
            // quarter of the rows each: the products wait for them)
            Piece p;
            const auto wait = [&](uint32_t bar, uint32_t parity) {
                return __all_sync(0xffffffffu, kwait<200>(bar, parity, sh, a));
            };
            uint32_t k0 = 0, np = 0, ne = 0;
            bool ok = true;
            for (; ok && !a.stall && next_piece<true>(p, np, sh, ok, lane, wait); ++np) {
                if (warp == kWarpQ) {
                    ok = __all_sync(0xffffffffu, kwait<200>(smem_u32(&sh->q_empty), (np & 1) ^ 1, sh, a));
                    if (!ok) break;
                    if (lane == 0) {
                        const int tiles = p.it.ntok > a.TQ ? 2 : 1;
                        const uint32_t fb = smem_u32(&sh->q_full);
                        mbar_arrive_expect_tx(fb, tiles * C::kHalves * qrows * 128);
                        for (int x = 0; x < tiles; ++x)
#pragma unroll
                            for (int h = 0; h < C::kHalves; ++h)
                                asm volatile(
                                    "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
                                    "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                                        smem_u32(qbuf + x * C::kTileBytes + h * C::kHalfBytes)),
                                    "l"(reinterpret_cast<uint64_t>(&qmap)), "r"(h * 64), "r"(p.head * a.G),
                                    "r"(p.it.row0 + x * a.TQ), "r"(fb)
                                    : "memory");
                    }
                    __syncwarp();
                }
                for (int j = max(p.j0, (p.it.pos0 + 1) / kTile); ok && j < p.j1; ++j) {
                    if (!edge_tile(p.it, j)) continue;
                    const uint32_t st = (k0 + 2 * (j - p.j0) + 1) % kStages;
                    ok = __all_sync(0xffffffffu, kwait<200>(smem_u32(&sh->edge[ne % kEdges]), ne / kEdges & 1, sh, a));
                    if (!ok) break;
                    const int end = min(p.it.len - j * kTile, kTile);     // rows from here on: past the sequence
                    const int r0 = max(0, min(end, p.it.pos0 + 1 - j * kTile));  // rows from here on: new tokens
                    const int r1 = (end + kBlk - 1) / kBlk * kBlk;        // rows from here on are zeros already
                    const int part = (warp - kWarpQ) * 32 + lane;
                    uint32_t top = 0;  // largest magnitude, as integers: infinities and NaNs are 0x7f80 and up
#pragma unroll
                    for (int h = 0; h < C::kHalves; ++h) {
                        uint4 *t = reinterpret_cast<uint4 *>(ring + st * C::kTileBytes + h * C::kHalfBytes);
#pragma unroll 4
                        for (int e = r0 * 8 + part; e < end * 8; e += 128) {
                            const uint4 v = t[e];
                            top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                                         __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
                        }
                        for (int e = end * 8 + part; e < r1 * 8; e += 128) t[e] = make_uint4(0, 0, 0, 0);
                    }
                    if ((top & 0xffffu) >= 0x7f80u || top >= 0x7f800000u) {
                        for (int h = 0; h < C::kHalves; ++h) {
                            uint4 *t = reinterpret_cast<uint4 *>(ring + st * C::kTileBytes + h * C::kHalfBytes);
                            for (int e = r0 * 8 + part; e < end * 8; e += 128) {
                                const uint4 v = t[e];
                                t[e] = make_uint4(finite_pair(v.x), finite_pair(v.y), finite_pair(v.z),
                                                  finite_pair(v.w));
                            }
                        }
                        sh->odd_values[np % kOddSlots] = (int32_t)np + 1;
                    }
                    __threadfence_block();
                    fence_proxy_async_smem();
                    __syncwarp();
                    // the last of the four warps hands the tile over
                    if (lane == 0 && (atomicAdd(&sh->fixed[ne % kEdges], 1) & 3) == 3) {
                        __threadfence_block();
                        mbar_arrive(smem_u32(&sh->full[st]));
                    }
                    ++ne;
                }
                k0 += 2 * (p.j1 - p.j0);
            }
            // the last query tiles have landed too
            if (warp == kWarpQ && np > 0) drain(smem_u32(&sh->q_full), (np - 1) & 1);
        }
    } else {
        // ---------------- softmax: thread = one row of query tile x
        reg_alloc<Regs<E8>::kSoft>();
        const int x = warp >> 2, r = tid & 127;
        const int tok = r / a.G, hd = r - tok * a.G;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + x * kTile, to = tmem + lanes + 256 + x * 128;
        Piece p;
        const auto wait = [&](uint32_t bar, uint32_t parity) {
            return __all_sync(0xffffffffu, cwait(bar, parity, sh, a));
        };
        uint32_t ns = 0, no = 0, nj = 0, np = 0;
        uint32_t nk = 0;  // K tiles of the pieces before
        bool ok = true;
        for (; ok && next_piece<true>(p, np, sh, ok, lane, wait); ++np) {
            const bool two = p.it.ntok > a.TQ;
            const Part pt = part_of(p, x, a.TQ);
            const int t = (two ? x * a.TQ : 0) + tok;  // token of the item
            const bool live = r < qrows && t < p.it.ntok;
            const bool any = __any_sync(0xffffffffu, live);
            // a row without a token is computed like the others and dropped at the end
            const int32_t pos = live ? p.it.pos0 + t : 0x3fffffff;
            float m = -INFINITY, z = 0.f;
            float scale2 = a.scale2;
            for (int i = 0; i < pt.cnt; ++i) {
                const int j = pt.j + i * pt.by;
                ok = cwait(smem_u32(&sh->s_full[x]), ns & 1, sh, a);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ++ns;
                if (any) {
                    tc_fence_after();
                    uint32_t s[kTile];
                    const int lim = pos - j * kTile;  // last key of the tile that the row sees
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, s, c * 32);
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_wait_ld32(s, c * 32);
                    if (__builtin_expect(__any_sync(0xffffffffu, lim < kTile - 1), 0)) {
#pragma unroll
                        for (int c = 0; c < kTile; ++c)
                            if (c > lim) s[c] = 0xff800000u;
                    }
                    float mt;
                    const uint32_t ks = smem_u32(sh8->kscale[(nk + j - p.j0) % kScales8]);
                    const uint32_t vt = smem_u32(sh8->vtile[(nk + j - p.j0) % kScales8]);
                    if constexpr (E8) {
                        // a block's keys have a scale of their own (read where it is used: registers are short)
                        if (i == 0) scale2 = a.scale2 * sh8->qscale[np & 1][two ? x : 0][r];
                        mt = -INFINITY;
                        float kf[4];
#pragma unroll
                        for (int b = 0; b < kBlkPerTile; ++b) {
                            if (b % 4 == 0) ld_shared4(ks + b * 4, kf);
                            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                            for (int c = b * kBlk; c < b * kBlk + kBlk; c += 4)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(s[c + 2 * e]),
                                                               __uint_as_float(s[c + 2 * e + 1])));
                            mt = fmaxf(mt, fmaxf(mx[0], mx[1]) * kf[b % 4]);
                        }
                        mt = fmaf(mt, scale2, ld_shared(vt));
                    } else {
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int c = 0; c < kTile; c += 8)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(s[c + 2 * e]), __uint_as_float(s[c + 2 * e + 1])));
                        mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale2;
                    }
                    if constexpr (E8) {
                        if (__builtin_expect(i == 0 || __any_sync(0xffffffffu, mt > m + kLazy), 0)) {
                            // (a tile of blocks apart has logits this large)
                            if (__any_sync(0xffffffffu, mt >= kFar8 / 2) && ld_shared(vt + 4) == 0.f) {
                                const int slot = (nk + j - p.j0) % kScales8;
                                const float2 mz = logits_apart<D>(ts, to, sh8->kscale[slot], sh8->vexp[slot], scale2, lim,
                                                                  i == 0, make_float2(m, z));
                                m = mz.x, z = mz.y;
#pragma unroll
                                for (int c = 0; c < 4; ++c) tmem_ld32(ts + c * 32, s, c * 32);
#pragma unroll
                                for (int c = 0; c < 4; ++c) tmem_wait_ld32(s, c * 32);
                            } else if (i == 0) {
                                m = mt;
                            } else {
                                raise_reference<D, E8>(to, mt, m, z);
                            }
                        }
                    } else {
                        if (i == 0) {
                            m = mt;
                        } else if (__builtin_expect(__any_sync(0xffffffffu, mt > m + kLazy), 0)) {
                            raise_reference<D, E8>(to, mt, m, z);
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : m;  // a row that saw nothing yet: weights 2^-inf = 0
                    uint64_t sc = pack2(scale2, scale2);
                    const float mr1 = E8 ? ld_shared(vt + 8) + kUp8 - ref : -ref;
                    const uint64_t mr = pack2(mr1, mr1);
                    uint64_t sum[2] = {0ull, 0ull};
                    float kf[4];
#pragma unroll
                    for (int c = 0; c < kTile; c += 2) {
                        if (E8 && c % (4 * kBlk) == 0) ld_shared4(ks + c / kBlk * 4, kf);
                        if (E8 && c % kBlk == 0) {
                            const float f = scale2 * kf[c / kBlk % 4];
                            sc = pack2(f, f);
                        }
                        float lo, hi;
                        unpack2(fma2(pack2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc, mr), lo, hi);
                        lo = ex2(lo);
                        hi = ex2(hi);
                        sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pack2(lo, hi));
                        s[c >> 1] = E8 ? f16x2(lo, hi) : bf16x2(lo, hi);
                        if (c == 62) {
                            tmem_st32(ts, s, 0);
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(smem_u32(&sh->p_half[x]));
                        }
                    }
                    tmem_st32(ts + 32, s, 32);
                    float s0, s1;
                    unpack2(add2(sum[0], sum[1]), s0, s1);
                    z = E8 ? fmaf(s0 + s1, ld_shared(vt + 4), z) : z + (s0 + s1);
                    tmem_wait_st();
                    tc_fence_before();
                }
                __syncwarp();
                if (!any && lane == 0) mbar_arrive(smem_u32(&sh->p_half[x]));
                if (lane == 0) mbar_arrive(smem_u32(&sh->p_full[x]));
            }
            if (ok && pt.cnt > 0) {
                ok = cwait(smem_u32(&sh->o_full[x]), no & 1, sh, a);
                ++no;
            }
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            // ---- output: O / z, or the partial of a piece
            const bool joined = !two;
            float f0 = 1.f, f1 = 0.f;
            const bool odd = joined && p.j1 - p.j0 > 1;  // the odd key tiles have a partial too
            if (ok && joined && x == 1) {
                sh->stat[r] = make_float2(m, z);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh->x_full));
                // O1 is written again only after warps 0-3 have read it
                ok = cwait(smem_u32(&sh->x_free), nj & 1, sh, a);
            } else if (ok && joined) {
                ok = cwait(smem_u32(&sh->x_full), nj & 1, sh, a);
                tc_fence_after();
                if (ok && odd) {
                    const float2 o = sh->stat[r];
                    const float M = fmaxf(m, o.x), ref = M == -INFINITY ? 0.f : M;
                    f0 = ex2(m - ref);
                    f1 = ex2(o.x - ref);
                    z = E8 ? scale_sum<E8>(z, m - ref, f0) + scale_sum<E8>(o.y, o.x - ref, f1) : z * f0 + o.y * f1;
                    m = M;
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (ok && any && (x == 0 || two)) {
                const float inv = p.whole ? 1.f / z : 1.f;
                f0 *= inv, f1 *= inv;
                const int64_t row = p.it.row0 + t;
                const int rr = (two ? x * kTile : 0) + r;
                const bool add = *(volatile int32_t *)&sh->odd_values[np % kOddSlots] == (int32_t)np + 1;
                const int64_t slot = partial_slot(blockIdx.x, p.j0 > 0);
                float4 *pp = a.part + slot * (D / 4) * 256 + rr;  // dims d..d+3 at pp[d / 4 * 256]
                uint16_t *op = a.out + (row * a.hq + p.head * a.G + hd) * D;
#pragma unroll 1  // one copy: it runs once an item, out of a cold instruction cache
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_ld32(to + c, o, 0);
                    tmem_wait_ld32(o, 0);
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f0);
                    if (odd) {
                        uint32_t o1[32];
                        tmem_ld32(to + 128 + c, o1, 0);
                        tmem_wait_ld32(o1, 0);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), f1, __uint_as_float(o[e])));
                    }
                    if (live && p.whole) {
                        // a warp's store touches 32 rows: as few and as wide as the alignment allows
                        uint32_t b[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            b[e] = bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
                        if (a.wide) {
                            st_global_32b(op + c, b, 0);
                            st_global_32b(op + c + 16, b, 8);
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                *reinterpret_cast<uint4 *>(op + c + 2 * e) =
                                    make_uint4(b[e], b[e + 1], b[e + 2], b[e + 3]);
                        }
                    } else if (live) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            pp[(c + e) / 4 * 256] = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                                __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                    }
                    __syncwarp();  // all lanes load the next columns
                }
                if (add && live) add_cleared<D, E8>(a, p.seq, p.head, max(p.it.pos0 + 1, p.j0 * kTile),
                                                    min(pos, p.j1 * kTile - 1), p.whole ? op : nullptr, pp);
                if (live && !p.whole) a.stat[slot * 256 + rr] = make_float2(m, z);
            }
            nk += p.j1 - p.j0;
            // the next piece's products write O again only after these reads
            tc_fence_before();
            if (joined) {
                ++nj;
                __syncwarp();
                if (x == 0 && lane == 0) mbar_arrive(smem_u32(&sh->x_free));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) tmem_dealloc(sh->tmem, kTmemCols);
    if (warp == kWarpKv || warp == kWarpKv + 1) {
        if constexpr (E8) {
            const int kv = warp - kWarpKv;
            const uint32_t k = (uint32_t)sh->issued[kv].x, stages = kv ? kRaw8 : kK8;
            for (uint32_t i = k > stages ? k - stages : 0; i < k; ++i)
                drain(smem_u32((kv ? sh8->rfull : sh8->kfull) + i % stages), i / stages & 1);
        } else {
            drain_tiles(sh, warp - kWarpKv);
        }
    }
}

// ---- merge ----------------------------------------------------------------------
// Block (c, y): the item that the cut before CTA c falls into, if that is the item's
// first cut: out = sum_i O_i 2^(m_i - M) / sum_i z_i 2^(m_i - M), pieces in CTA order.
// A thread takes 8 dims of a row; lanes are rows, as the partials lie.
template <int D, bool E8>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkArgs a)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int ctas = *a.used_ctas, c = blockIdx.x + 1;
    if (c >= ctas) return;
    const Start s = a.start[c], b = a.start[c - 1];
    if (s.off == 0 || (same_item(s, b) && b.off > 0)) return;  // no cut, or an earlier one of the same item
    const Item it = make_item(a, s.seq, s.pair);
    if (s.off >= it.nt) return;  // behind the item
    const int rr = (blockIdx.y & 7) * 32 + (threadIdx.x & 31), d4 = ((blockIdx.y >> 3) * 8 + (threadIdx.x >> 5)) * 2;
    const bool two = it.ntok > a.TQ;
    const int x = rr / kTile, r = rr % kTile, t = x * a.TQ + r / a.G, hd = r % a.G;
    if (r >= a.G * a.TQ || t >= it.ntok || (x == 1 && !two)) return;
    // the piece that CTA c - 1 began the item with, then those of the CTAs that start inside it
    int end = c + 1;
    while (end < ctas && same_item(a.start[end], s) && a.start[end].off < it.nt) ++end;
    const auto empty = [&](int k) {  // CTA k got nothing of the item
        const Start p = a.start[k], q = a.start[k + 1];
        return same_item(p, q) && p.off >= q.off;
    };
    float M = -INFINITY;
    for (int k = c - 1; k < end; ++k)
        if (k < c || !empty(k)) M = fmaxf(M, a.stat[partial_slot(k, k >= c) * 256 + rr].x);
    float den = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int k = c - 1; k < end; ++k) {
        if (k >= c && empty(k)) continue;
        const int64_t slot = partial_slot(k, k >= c);
        const float2 st = a.stat[slot * 256 + rr];
        if (st.x == -INFINITY && st.y == 0.f) continue;  // nothing of this piece is seen by the row
        const float f = ex2(st.x - M);
        den = E8 ? den + scale_sum<E8>(st.y, st.x - M, f) : fmaf(st.y, f, den);
        const float4 u = a.part[(slot * (D / 4) + d4) * 256 + rr], v = a.part[(slot * (D / 4) + d4 + 1) * 256 + rr];
        acc[0] = fmaf(u.x, f, acc[0]), acc[1] = fmaf(u.y, f, acc[1]), acc[2] = fmaf(u.z, f, acc[2]);
        acc[3] = fmaf(u.w, f, acc[3]), acc[4] = fmaf(v.x, f, acc[4]), acc[5] = fmaf(v.y, f, acc[5]);
        acc[6] = fmaf(v.z, f, acc[6]), acc[7] = fmaf(v.w, f, acc[7]);
    }
    const float inv = 1.f / den;
    uint16_t *op = a.out + ((int64_t)(it.row0 + t) * a.hq + s.head * a.G + hd) * D + d4 * 4;
    *reinterpret_cast<uint4 *>(op) =
        make_uint4(bf16x2(acc[0] * inv, acc[1] * inv), bf16x2(acc[2] * inv, acc[3] * inv),
                   bf16x2(acc[4] * inv, acc[5] * inv), bf16x2(acc[6] * inv, acc[7] * inv));
}

// Tensor map over q, (d, head, row); a box is one 64-dim half of a query tile.
template <class Cache>
cudaError_t query_map(CUtensorMap *m, const void *q, const Cache *c, int32_t rows, int G, int TQ)
{
    auto fn = tensor_map_encoder();
    if (!fn) return cudaErrorNotSupported;
    cuuint64_t dims[3] = {(cuuint64_t)c->head_dim, (cuuint64_t)c->num_q_heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)c->head_dim * 2, (cuuint64_t)c->head_dim * c->num_q_heads * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)TQ};
    cuuint32_t estr[3] = {1, 1, 1};
    if (fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    return cudaSuccess;
}

// Workspace: [CTAs with work][starts][whole items][stats][partials].
struct Layout {
    size_t start, whole, stat, part, total;
};

Layout layout(int32_t D)
{
    Layout l;
    size_t o = 256;
    l.start = o, o += align256((kMaxCtas + 1) * sizeof(Start));
    l.whole = o, o += align256((size_t)kMaxCtas * kMaxRounds * sizeof(Start));
    l.stat = o, o += align256((size_t)2 * kMaxCtas * 256 * sizeof(float2));
    l.part = o, o += (size_t)2 * kMaxCtas * 256 * D * sizeof(float);
    l.total = o;
    return l;
}

template <int D, bool E8>
cudaError_t launch_all(const CUtensorMap &km, const CUtensorMap &vm, const CUtensorMap &qm, const ChunkArgs &a,
                       cudaStream_t st)
{
    constexpr size_t smem = Cfg<D, E8>::kSmem;
    static_assert(smem <= 227 * 1024, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(chunk_kernel<D, E8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_dependent(chunk_kernel<D, E8>, dim3((unsigned)a.ctas), kThreads, smem, st, km, vm, qm, a);
    if (e == cudaSuccess && a.ctas > 1)
        e = launch_dependent(chunk_merge_kernel<D, E8>, dim3((unsigned)a.ctas - 1, 8 * (D / 64)), 256, 0, st, a);
    return e;
}

// A call's arguments but for where the cache lies, and the map of its queries.
template <class Cache>
cudaError_t chunk_args(ChunkArgs *p, CUtensorMap *qm, const Cache *c, int32_t layer, const kara_tokens *t,
                       const int32_t *bt, int32_t bt_stride, const void *q, void *out, void *ws, int32_t *err)
{
    ChunkArgs &a = *p;
    a.q_start = t->q_start;
    a.len = t->len;
    a.bt = bt;
    a.err = err;
    a.n = t->n;
    a.rows = t->rows;
    a.bt_stride = bt_stride;
    a.num_blocks = c->num_blocks;
    a.layer = layer;
    a.hq = c->num_q_heads;
    a.hkv = c->num_kv_heads;
    a.D = c->head_dim;
    a.G = a.hq / a.hkv;
    a.TQ = kTile / a.G;
    a.scale2 = 1.4426950408889634f / sqrtf((float)c->head_dim);
    a.out = static_cast<uint16_t *>(out);
    a.v = nullptr;
    a.v8 = nullptr;
    a.k_scale = a.v_scale = nullptr;
    a.block_stride = c->block_stride;
    a.head_stride = c->head_stride;
    const Layout l = layout(c->head_dim);
    char *w = static_cast<char *>(ws);
    a.used_ctas = reinterpret_cast<int32_t *>(w);
    a.start = reinterpret_cast<Start *>(w + l.start);
    a.whole = reinterpret_cast<Start *>(w + l.whole);
    a.stat = reinterpret_cast<float2 *>(w + l.stat);
    a.part = reinterpret_cast<float4 *>(w + l.part);
    a.wide = ((uintptr_t)out & 31u) == 0;
    const Stall dbg = debug_stall(kTimeoutNs);
    a.stall = dbg.on;
    a.wait_ns = dbg.on ? dbg.wait_ns : debug_wait(kTimeoutNs);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    a.ctas = sms < kMaxCtas ? sms : kMaxCtas;
    return query_map(qm, q, c, t->rows, a.G, a.TQ);
}

}  // namespace
}  // namespace kara
