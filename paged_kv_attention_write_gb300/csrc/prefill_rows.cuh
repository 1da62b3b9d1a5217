// prefill_rows.cuh -- chunks of query rows over a paged cache, on the 5th-generation tensor
// cores: behind a sliding window with sinks (prefill_window.cu), or over the whole context with
// a range of keys per row (cross_chunk.cu).
//
// Row i of a chunk sits at position p = C - Lq + i and sees the keys j <= p with
// j > p - window or j < num_sinks.  A work item is 128 rows, (token, query head) pairs of one
// kv head (128/G tokens), of one sequence.
//
// What a row can see is bounded by window + num_sinks, so an item walks only the blocks that
// one of its rows sees: the sinks' blocks, then those from the first row's window to the last
// row, packed into one list of virtual blocks (a few sinks cost one block, not a key tile)
// and cut into tiles of 64 virtual keys.  Only tiles at a border are masked.
//
// Per key tile: S = Q K^T (tcgen05, fp32 in TMEM; kSBufs buffers: two at head dimension 128, three
// at 64), the softmax (online, log2 domain, the reference moves only when a score exceeds it by
// 2^8), P in the cache's type over the S columns, O += P V.  The row sums add the rounded weights, as the product does,
// so that a row that one key dominates loses nothing by the rounding.  The tensor core cuts off
// what falls below the last bits of O: of 65536 keys of 2^-20 of the first one's weight, 4 % of
// their share is lost (up to 2^-24 of a row's magnitude per key).
//
// Under a window items are short (a 1024-key window: nine 128-key tiles), and what costs is
// what does not overlap: an item's first loads, its last product, its output.  So two CTAs
// share an SM, each with half of TMEM (the 64-column S buffers and O) and of the shared
// memory, and one's tiles run under the other's beginning and end; every scheduler has four
// softmax warps.  The grid is one CTA per item, but a CTA whose loads near their end calls off
// one that has not started (cluster launch control) and goes on with its item: Q, keys and the
// first S of the next item are under way while the softmax warps finish this one, and the
// hardware still hands items out as places become free.  Warp 0 finds the items and passes them
// on through two slots in shared memory.  With fewer items than half the SMs a cluster of CTAs
// takes each, a run of its key tiles per CTA, and joins the (maximum, sum, output) of the rows
// through distributed shared memory.
//
// Measured (us; 8 chunks of 512 tokens, 64 q / 8 kv heads, window 4096, fp16 | 4 chunks of
// 512, 32 / 8, window 1024, bf16 | 9 ragged chunks, 16 / 16, D 64, window 301 | 16 fresh prompts
// of 100 to 1500, 32 / 8, window 1024): this 459 | 34.6 | 23.3 | 150 (1202, 630, 166 TFLOP/s);
// one item per CTA 460 | 37.6 | 23.3 | 188.  The loads of K and of V are one loop: as two copies
// the warps' loops together miss the instruction cache (476 | 38.0).  Steps tried on the way,
// each in its own build: CTAs that own every n-th item 507 | 45 | 28 (uneven, 9 to 68 key tiles
// per SM); one CTA per SM with 128-key tiles and three S buffers, as the causal kernel has, 545 |
// 47 | 42; two CTAs with 128-key tiles and one S buffer each 555 | 57 | 40, with S issued for two
// 64-key tiles at once 574 | 53 | 30; two row tiles per CTA taking turns, eight softmax warps
// each, 582 | 67 | 53.
// What bounds it: a tile takes its CTA 0.88 us behind windows up to 1024 keys and 0.97 (bf16) to
// 1.01 us (fp16) from 4096 on, where power holds the clocks down (1500 to 1700 clocks), nearly all
// in the softmax warps (TMEM load, maxima, exponentials, P store, hand-over), and an item about one
// tile more; the tensor core is busy 52 % of
// the time and its queue 76 % (an S product of 64 keys occupies it for 48 clocks, not 32: it
// reads 16 columns of all of Q, 4 KB, for 2 KB of K).  With no exponentials, no maxima and no P
// stores (a timing-only build of the 507 us step) 469 us were left; with no K and V loads at
// all, 427 of 500.
//
// Cross attention (CROSS): no order among the keys, each row sees [begin, end) of its own.  An item
// walks the blocks from the first to the last key that one of its rows sees; blocks that none
// reaches are not loaded, and only tiles that some row does not see whole are masked: a warp
// whose rows see nothing of a tile stores zero weights and is done with it.  The ranges of an item's
// rows wait in shared memory beside its slot.  Sequences with long contexts go first, and where
// ranges are given the last rows of all sequences, which see most of what stands before them.
// Measured (us): fp16, 8 x 512 rows of 64 q / 8 kv heads over 4096 to 12288 keys, D 128: 842 to
// 906 as power allows (1.23 to 1.32 PFLOP/s; in the sequences' order 904 beside 842); bf16, 4 x 512
// rows of 32 / 8 heads beside four images of 1601 keys: 94 (its longest items, 101 tiles, take 90); 23
// ragged chunks of 8 / 1 heads beside three images: 31 in clusters of two, 48 whole.  Half of each
// item's rows blind to all tiles but the first: 290 with scores masked one by one, 225 so, 187 when all
// rows see all.  A CTA per SM with the warps, rings and TMEM of two, both halves on one item, was tried for
// items of unequal length: the ragged chunks 33, 336 items of 500 to 8000 keys 134 -> 94, but the images 94 -> 96, 256 items of
// 6000 keys 92 -> 98 and the wide case 842 -> 912: nothing runs under an item's beginning and end.
//
// Warps: 0 items, TMA of Q and K, 2 of V (a lane per block), 1 issues S, 3 P.V (and clears the
// rows of V that no row of the item looks at, so that stale or NaN slots never meet a zero
// weight), 4-11 softmax and output, each a 16-row slab through the 16-lane TMEM shapes.
// Every mbarrier wait is bounded in time; if one gives up, loads and products under way still end before
// the CTA frees its TMEM and leaves (not run on a GPU: it would take a wait of two seconds).
#pragma once

#include <algorithm>
#include <type_traits>

#include "cluster.cuh"
#include "tcgen05.cuh"

namespace pa {
namespace {

constexpr int kThreads = 12 * 32;
constexpr int kBM = 128, kBN = 64;  // rows of an item, keys of a tile
constexpr float kGrowLog2 = 8.f;
// The softmax reference lies 2^kLiftLog2 below the score that set it, so that weights use fp16's upper
// range: it has no bits below 2^-24, and a weight is at most 2^(8 + 7), of 2^16.
template <class T>
constexpr float kLiftLog2 = std::is_same<T, F16>::value ? 7.f : 0.f;
constexpr int kMostRanked = 256;     // sequences whose items are ordered by length
constexpr int kPlanSeqs = 2047;      // sequences whose items are listed without gaps

struct Params {
    void *out;
    pa_dtype out_dtype;
    const int32_t *query_start_loc, *block_tables, *context_lens;
    int max_blocks_per_seq, max_context_len, num_tokens, num_seqs, num_heads, num_kv_heads, block_log2, num_blocks;
    int window, num_sinks;
    int group_log2;     // query heads per kv head
    int units_per_seq;  // items of one kv head in the longest chunk
    int listed;         // ragged chunks: items are numbered without gaps (else every sequence has units_per_seq)
    float qk_scale_log2;
    int32_t *status;
    const int32_t *key_ranges;  // cross attention: [num_tokens][2], or null
    int max_query_len;
    int by_length;  // cross attention: the sequences with long contexts first
};

// r += the two weights packed in w, each widened exactly inside the add (mixed-precision add).
template <class T>
__device__ __forceinline__ void add_pair(float2 &r, uint32_t w) {
    if constexpr (std::is_same<T, BF16>::value)
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "add.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;\n\t}"
            : "+f"(r.x), "+f"(r.y)
            : "r"(w));
    else
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "add.rn.f32.f16 %0, l, %0;\n\tadd.rn.f32.f16 %1, h, %1;\n\t}"
            : "+f"(r.x), "+f"(r.y)
            : "r"(w));
}

template <int D>
struct Shape {
    static constexpr int HALVES = D / 64;            // 128-byte swizzle atoms along D
    static constexpr int Q_BYTES = kBM * D * 2;      // [half][128 rows][128 B]
    static constexpr int KV_BYTES = kBN * D * 2;     // one K or V tile: [8-key group][half][8 keys][128 B]
    static constexpr int GSTR = HALVES * 1024;       // bytes between 8-key groups
    static constexpr int NK = D == 64 ? 4 : 2, NV = D == 64 ? 4 : 2;  // K and V stages
    static constexpr int SBUFS = D == 64 ? 3 : 2;   // S buffers in TMEM, beside O
    static constexpr int OFF_K = Q_BYTES;
    static constexpr int OFF_V = OFF_K + NK * KV_BYTES;
    static constexpr int OFF_BAR = OFF_V + NV * KV_BYTES;
    static constexpr int OFF_RANGES = OFF_BAR + 512 + 4 * (kPlanSeqs + 1);  // cross attention: two items' row ranges
    static constexpr int SMEM = 1024 + OFF_RANGES, SMEM_CROSS = SMEM + 2 * kBM * 8;
    static_assert(2 * (SMEM_CROSS + 1024) <= 228 * 1024, "two CTAs per SM");
    // split items: the CTA's output [128][PITCH] and its rows' maxima and sums, over Q and the rings
    static constexpr int PITCH = D + 8;              // floats (eight rows of a store on distinct banks)
    static constexpr int OFF_M = kBM * PITCH * 4, OFF_L = OFF_M + kBM * 4;
    static_assert(OFF_L + kBM * 4 <= OFF_BAR, "the output of a split item fits");
};

// The 16-lane TMEM shapes of 32 columns: four groups of 8 (16x256b), eight of 4 (16x128b).
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// mbar_wait (tma.cuh) that lets the hardware suspend the thread for up to a millisecond at a
// time, for the waits of a role that has run ahead.
__device__ __forceinline__ bool mbar_wait_idle(uint32_t bar, uint32_t parity, int32_t *status) {
    const unsigned long long t0 = global_ns();
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity), "r"(1000000u)
            : "memory");
        if (done) return true;
        if (global_ns() - t0 > kWaitLimitNs) {
            report(status, PA_DEVERR_TIMEOUT);
            return false;
        }
    }
}

// Query rows and (clamped) context of a sequence; false when it has nothing to compute
// (reported when `rep`).
__device__ __forceinline__ bool sequence(const Params &p, int q0, int q1, int C, bool rep, int &ctx) {
    const int cap = min(p.max_blocks_per_seq << p.block_log2, p.max_context_len);
    const int Lq = q1 - q0;
    ctx = C;
    if (q0 < 0 || q1 < q0 || q1 > p.num_tokens) {  // never index past the query
        if (rep) report(p.status, PA_DEVERR_QUERY);
        return false;
    }
    if (Lq == 0) return false;
    if (C > cap) {
        if (rep) report(p.status, PA_DEVERR_CONTEXT);
        ctx = cap;
    }
    if (Lq > ctx) {
        if (rep) report(p.status, PA_DEVERR_QUERY);
        return false;
    }
    return true;
}

// One work item and the keys its rows see.
struct Item {
    int s, g, q0, Lq;
    int tok;            // first chunk token
    int first, last;    // positions of the first and the last row
    int ns, lo;         // seen keys: [0, ns) and [lo, last]
    int sk, sh;         // virtual keys of the sinks' blocks; logical key of virtual v >= sk: v + sh
    int blocks, tiles;  // virtual blocks, key tiles
    int low, high;      // tiles < low hold sinks or keys behind some row's window, tiles >= high keys past some row

    // Virtual key of logical key j (of the next listed one, if its block is not listed).
    __device__ __forceinline__ int virt(int j) const { return j < sk ? j : max(sk, j - sh); }
};

// The work item of this CTA: unit and kv head of sequence s (unit: 128 rows of the chunk);
// false when it has no rows.
__device__ __forceinline__ bool make_item(const Params &p, int s, int unit, int g, bool rep, Item &it) {
    const int q0 = p.query_start_loc[s], q1 = p.query_start_loc[s + 1];
    int ctx;
    const bool ok = sequence(p, q0, q1, p.context_lens[s], rep, ctx);
    const int tt = kBM >> p.group_log2, bl = p.block_log2;
    it.s = s;
    it.g = g;
    it.q0 = q0;
    it.Lq = q1 - q0;
    it.tok = unit * tt;
    if (!ok || unit < 0 || it.tok >= it.Lq) return false;
    it.first = ctx - it.Lq + it.tok;
    it.last = ctx - it.Lq + min(it.Lq, it.tok + tt) - 1;
    it.lo = max(0, it.first - p.window + 1);
    it.ns = min(p.num_sinks, it.lo);
    const int sinks = it.ns > 0 ? ((it.ns - 1) >> bl) + 1 : 0;
    const int b = max(it.lo >> bl, sinks);
    it.sk = sinks << bl;
    it.sh = (b - sinks) << bl;
    it.blocks = sinks + (it.last >> bl) + 1 - b;
    const int per_tile = kBN >> bl;
    it.tiles = (it.blocks + per_tile - 1) / per_tile;
    const int behind = it.last - it.sh - p.window;  // last virtual key behind the last row's window
    it.low = max((it.sk + kBN - 1) / kBN, behind >= 0 ? behind / kBN + 1 : 0);
    it.high = max(0, it.first - it.sh + 1) / kBN;
    return true;
}

// Cross attention: query rows and (clamped) context of a sequence; false when it has no rows.
__device__ __forceinline__ bool cross_sequence(const Params &p, int q0, int q1, int C, bool rep, int &ctx) {
    const int cap = min(p.max_blocks_per_seq << p.block_log2, p.max_context_len);
    ctx = C;
    if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || q1 - q0 > p.max_query_len) {  // never index past the query
        if (rep) report(p.status, PA_DEVERR_QUERY);
        return false;
    }
    if (q1 == q0) return false;
    if (C < 0 || C > cap) {
        if (rep) report(p.status, PA_DEVERR_CONTEXT);
        ctx = C < 0 ? 0 : cap;
    }
    return true;
}

// One work item of the cross attention: the keys [lo, hi) hold all that its rows see.
struct CrossItem {
    int s, g, q0, Lq;
    int tok;            // first chunk token
    int ctx, lo, hi;
    int sh;             // logical key of virtual key v: v + sh (a whole number of blocks)
    int blocks, tiles;  // virtual blocks, key tiles (one, all masked, where no row sees anything)
    int low, high;      // every row sees all keys of the tiles low .. high - 1
    int holes;          // there may be keys of [lo, hi) that no row sees
};

// The keys [x, y) of the token at `tok + i` of an item's chunk (past the chunk's end: of its last token);
// (0, 0) where it sees none.
__device__ __forceinline__ int2 row_range(const Params &p, const CrossItem &it, int i) {
    if (!p.key_ranges) return make_int2(0, it.ctx);
    const int2 r = reinterpret_cast<const int2 *>(p.key_ranges)[it.q0 + min(it.tok + i, it.Lq - 1)];
    const int2 cut = make_int2(max(r.x, 0), min(r.y, it.ctx));
    return cut.x < cut.y ? cut : make_int2(0, 0);
}

// The work item of this CTA, found by a whole warp; false when it has no rows.
__device__ __forceinline__ bool make_item(const Params &p, int s, int unit, int g, bool rep, CrossItem &it) {
    const int q0 = p.query_start_loc[s], q1 = p.query_start_loc[s + 1];
    const bool ok = cross_sequence(p, q0, q1, p.context_lens[s], rep, it.ctx);
    const int tt = kBM >> p.group_log2, bl = p.block_log2, lane = threadIdx.x % 32;
    it.s = s;
    it.g = g;
    it.q0 = q0;
    it.Lq = q1 - q0;
    it.tok = unit * tt;
    if (!ok || unit < 0 || it.tok >= it.Lq) return false;
    int lo = INT32_MAX, hi = 0, lo_in = 0, hi_in = INT32_MAX, last = 0, first = INT32_MAX;
    for (int i = lane; i < tt; i += 32) {
        const int2 r = row_range(p, it, i);
        const bool none = r.x >= r.y;
        lo = min(lo, none ? INT32_MAX : r.x);
        hi = max(hi, none ? 0 : r.y);
        lo_in = max(lo_in, none ? INT32_MAX : r.x);
        hi_in = min(hi_in, none ? 0 : r.y);
        last = max(last, none ? 0 : r.x);
        first = min(first, none ? INT32_MAX : r.y);
    }
    // ranges that reach from before the last begin to past the first end leave nothing out
    it.holes = __reduce_max_sync(kFullMask, last) > __reduce_min_sync(kFullMask, first);
    hi = __reduce_max_sync(kFullMask, hi);
    lo = min(hi, __reduce_min_sync(kFullMask, lo));
    lo_in = __reduce_max_sync(kFullMask, lo_in);
    hi_in = __reduce_min_sync(kFullMask, hi_in);
    it.lo = lo;
    it.hi = hi;
    it.sh = lo >> bl << bl;
    it.blocks = hi > lo ? ((hi - 1) >> bl) + 1 - (lo >> bl) : 0;
    const int per_tile = kBN >> bl;
    it.tiles = max(1, (it.blocks + per_tile - 1) / per_tile);
    it.low = lo_in >= hi_in ? INT32_MAX : (int)(((unsigned)(lo_in - it.sh) + kBN - 1) / kBN);
    it.high = max(0, hi_in - it.sh) / kBN;
    return true;
}

// The keys of the tile at virtual key k0 that some row of the item sees, a bit each (a whole warp
// asks; `ranges` are the item's in shared memory).
__device__ __forceinline__ uint64_t seen_keys(const Params &p, const CrossItem &it, const int2 *ranges, int k0) {
    const int tt = kBM >> p.group_log2, lane = threadIdx.x % 32;
    auto below = [](int n) { return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1; };
    if (!it.holes) return below(it.hi - it.sh - k0) & ~below(it.lo - it.sh - k0);
    uint64_t seen = 0;
    for (int i = lane; i < tt; i += 32) {
        const int2 r = ranges[i];
        seen |= below(r.y - it.sh - k0) & ~below(r.x - it.sh - k0);
    }
    const uint32_t a = __reduce_or_sync(kFullMask, (uint32_t)seen), b = __reduce_or_sync(kFullMask, (uint32_t)(seen >> 32));
    return (uint64_t)b << 32 | a;
}

// Asks for the number of a CTA that has not started, which then never starts; the 16-byte answer
// lands at `answer` and on the barrier.
__device__ __forceinline__ void try_cancel(uint32_t answer, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     answer),
                 "r"(bar)
                 : "memory");
}
// false: every CTA has started
__device__ __forceinline__ bool canceled(uint32_t answer, unsigned &number) {
    uint32_t yes, x;
    asm volatile(
        "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\tld.shared.b128 a, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
        : "=r"(yes), "=r"(x)
        : "r"(answer)
        : "memory");
    if (yes) number = x;
    return yes != 0;
}

// SPLIT: a cluster of CTAs takes one item, each a run of its key tiles.  CROSS: whole contexts and
// ranges, not a window with sinks.
template <class T, int D, bool SPLIT, bool CROSS>
__global__ void __launch_bounds__(kThreads, 2)
prefill_rows_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const Params p) {
    using Sh = Shape<D>;
    using It = typename std::conditional<CROSS, CrossItem, Item>::type;
    constexpr int NK = Sh::NK, NV = Sh::NV, kSBufs = Sh::SBUFS;
    constexpr bool kBf16 = std::is_same<T, BF16>::value;
    constexpr uint32_t IDESC_S = mma_idesc(128, kBN, kBf16, false);
    constexpr uint32_t IDESC_PV = mma_idesc(128, D, kBf16, true);
    constexpr uint32_t kTmemCols = 256, kTmemO = kSBufs * kBN;  // S (and P) buffers, then O
    static_assert(kTmemO + D <= kTmemCols, "half of TMEM");

    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sQ = smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Sh::OFF_BAR);
    const uint32_t b0 = smem_u32(bars);
    auto bar = [&](int i) { return b0 + 8 * i; };
    constexpr int BQF = 0;            // Q landed
    constexpr int BSF = 1;            // S buffer written
    constexpr int BPF = BSF + kSBufs; // P written over it
    constexpr int BPV = BPF + kSBufs; // P.V of that P finished
    constexpr int BKF = BPV + kSBufs; // K stage landed
    constexpr int BKE = BKF + NK;     // S of that K finished
    constexpr int BVF = BKE + NK;     // V stage landed
    constexpr int BVE = BVF + NV;     // P.V of that V finished
    constexpr int BTM = BVE + NV;     // TMEM allocated
    constexpr int BQE = BTM + 1;      // S of an item finished: Q may be replaced
    constexpr int BOE = BQE + 1;      // O of an item read
    constexpr int BIF = BOE + 1;      // item slot written
    constexpr int BIE = BIF + 2;      // item slot read by warps 1-11
    constexpr int BCL = BIE + 2;      // answer to the request for another item
    constexpr int BDR = BCL + 1;      // products of warps 1 and 3 finished (only after a wait gave up)
    constexpr int NBAR = BDR + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + NBAR);
    int *abort_flag = reinterpret_cast<int *>(bars + NBAR) + 1;
    constexpr int OFF_ANSWER = 352, OFF_ITEMS = 368;
    It *items = reinterpret_cast<It *>(smem + Sh::OFF_BAR + OFF_ITEMS);  // [2]
    int *plan_mem = reinterpret_cast<int *>(smem + Sh::OFF_BAR + 512);
    int2 *row_ranges = reinterpret_cast<int2 *>(smem + Sh::OFF_RANGES);  // CROSS: [2][128 / G]
    static_assert((NBAR + 1) * 8 <= OFF_ANSWER && OFF_ITEMS + 2 * sizeof(It) <= 512, "barrier area");

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid == 0) {
        *abort_flag = 0;
        for (int i = 0; i < NBAR; ++i) {
            const bool softmax = (i >= BPF && i < BPF + kSBufs) || i == BOE;  // arrived on by those eight warps
            mbar_init(bar(i), softmax ? 8 : i == BIE || i == BIE + 1 ? 11 : 1);
        }
        fence_barrier_init();
        prefetch_tensormap(&qmap);
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    __syncthreads();  // barriers initialised
    pdl_wait_previous();
    pdl_launch_dependents();
    // CTAs are numbered sequence by sequence (the items of one share their keys in L2), from a
    // chunk's last rows to its first (the first rows of a fresh prompt see few keys), kv heads
    // side by side.
    int *order = plan_mem + 2 * kMostRanked;  // CROSS, by_length: the sequences from the shortest context to the longest
    if (CROSS && p.by_length) {
        // length and number in one key, so that a comparison ranks two sequences (lengths from 2^22 on
        // count as alike: the order is only a matter of time)
        int *keys = plan_mem + 3 * kMostRanked;
        for (int i = tid; i < kMostRanked; i += kThreads)
            keys[i] = i < p.num_seqs ? min(max(p.context_lens[i], 0), (1 << 22) - 1) << 8 | i : INT32_MAX;
        __syncthreads();
        for (int i = tid; i < p.num_seqs; i += kThreads) {
            const int key = keys[i];
            int rank = 0;
            for (int j = 0; j < p.num_seqs; j += 4) {
                const int4 x = *reinterpret_cast<const int4 *>(keys + j);
                rank += (x.x < key) + (x.y < key) + (x.z < key) + (x.w < key);
            }
            order[rank] = i;
        }
        __syncthreads();
    }
    if (p.listed) {  // prefix sums of the sequences' units
        for (int i = tid; i <= p.num_seqs; i += kThreads) {
            int units = 0, ctx;
            if (i < p.num_seqs) {
                const int s = CROSS && p.by_length ? order[i] : i;
                const int q0 = p.query_start_loc[s], q1 = p.query_start_loc[s + 1];
                if (CROSS ? cross_sequence(p, q0, q1, p.context_lens[s], true, ctx)
                          : sequence(p, q0, q1, p.context_lens[s], true, ctx))
                    units = min((q1 - q0 - 1) / (kBM >> p.group_log2) + 1, p.units_per_seq);
            }
            plan_mem[i] = units;
        }
        __syncthreads();
        if (warp == 0) {
            int carry = 0;
            for (int base = 0; base <= p.num_seqs; base += 32) {
                const int i = base + lane, n = i <= p.num_seqs ? plan_mem[i] : 0;
                int v = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int w = __shfl_up_sync(kFullMask, v, o);
                    if (lane >= o) v += w;
                }
                if (i <= p.num_seqs) plan_mem[i] = carry + v - n;
                carry += __shfl_sync(kFullMask, v, 31);
            }
        }
        __syncthreads();
    }
    // the item of a number; false when it has no rows
    auto find = [&](unsigned number, bool rep, It &it) {
        const int idx = (int)(number / (unsigned)p.num_kv_heads), g = (int)(number % (unsigned)p.num_kv_heads);
        int seq, unit;
        if (p.listed) {
            const int u = plan_mem[p.num_seqs] - 1 - idx;
            int lo = 0, hi = p.num_seqs;  // plan_mem[lo] <= u < plan_mem[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (plan_mem[mid] <= u) lo = mid; else hi = mid;
            }
            seq = lo;
            unit = u < 0 ? INT32_MAX >> 8 : u - plan_mem[lo];  // past the last item: no such rows
        } else {
            seq = idx / p.units_per_seq;
            unit = p.units_per_seq - 1 - idx % p.units_per_seq;
            if (CROSS && p.by_length) {
                if (p.key_ranges) {  // the last rows, which may see most, of all sequences first
                    unit = p.units_per_seq - 1 - idx / p.num_seqs;
                    seq = idx % p.num_seqs;
                }
                seq = p.num_seqs - 1 - seq;
            }
        }
        if (CROSS && p.by_length) seq = order[seq];
        return make_item(p, seq, unit, g, rep && !p.listed && unit == 0 && g == 0, it);
    };
    It it{};
    bool live = true;
    if constexpr (SPLIT) live = find(blockIdx.x / cluster_size(), tid == 0, it);
    // CROSS: the rows' ranges of an item, for the warps that mask tiles or clear rows of V
    auto keep_ranges = [&](int slot, int first, int step) {
        if constexpr (CROSS)
            for (int i = first; i < kBM >> p.group_log2; i += step) row_ranges[slot * kBM + i] = row_range(p, it, i);
    };
    if constexpr (SPLIT && CROSS) {
        if (live) keep_ranges(0, tid, kThreads);
        __syncthreads();
    }
    volatile int *abort_v = abort_flag;
    auto wait = [&](int b, uint32_t parity) {
        return mbar_try_wait(bar(b), parity & 1) || (!*abort_v && mbar_wait_idle(bar(b), parity & 1, p.status));
    };
    // The loads do not wait for TMEM: warp 1 allocates it while they are under way.
    uint32_t tmem = 0;
    auto wait_tmem = [&]() {
        const bool got = __all_sync(kFullMask, wait(BTM, 0));
        tc_fence_after();
        tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
        return got;
    };
    // this CTA's key tiles of the item: j0 + t, t < n; `done` tiles of the items before
    int j0 = 0, n = 0, done = 0;
    if constexpr (SPLIT) {
        const int cs = (int)cluster_size(), rank = (int)cluster_rank();
        j0 = (int)((int64_t)it.tiles * rank / cs);
        n = (int)((int64_t)it.tiles * (rank + 1) / cs) - j0;
    }
    // The k-th item of this CTA, for warps 1-11: false after the last.
    auto next_item = [&](int k) {
        if constexpr (SPLIT) return k == 0;
        done += n;
        if (!__all_sync(kFullMask, wait(BIF + (k & 1), k >> 1))) {
            *abort_v = 1;
            return false;
        }
        if (warp >= 4) {  // softmax warps look the item up when they need it, and let it go at its end
            n = items[k & 1].tiles;
            return n > 0;
        }
        it = items[k & 1];
        n = it.tiles;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BIE + (k & 1)));
        return n > 0;
    };
    bool ok = true;

    if (!live) {
        // no rows: every warp goes straight to the teardown
    } else if (warp == 0 || warp == 2) {
        // ============================================ TMA: Q and K, or V
        const bool is_k = warp == 0;
        const CUtensorMap *map = is_k ? &kmap : &vmap;
        const uint32_t ring = sQ + (is_k ? Sh::OFF_K : Sh::OFF_V);
        const int full = is_k ? BKF : BVF, empty = is_k ? BKE : BVE, NS = is_k ? NK : NV;
        // keys and values are read again by the next items of the sequence
        const uint64_t policy = policy_evict_normal();
        const int bl = p.block_log2, nb = kBN >> bl;  // blocks per key tile (2, 4 or 8)
        const uint32_t box_bytes = (uint32_t)(D * 2) << bl;
        // Warp 0 also finds the items.  The next one is asked of the hardware while this one's last
        // tiles run: a CTA that has not started yet is called off and its number taken.
        const uint32_t answer = sQ + Sh::OFF_BAR + OFF_ANSWER;
        unsigned number = blockIdx.x;
        int asked = 0, heard = 0;
        auto ask = [&] {
            if (lane == 0) {
                fence_async_smem();  // the last answer has been read
                mbar_arrive_expect_tx(bar(BCL), 16);
                try_cancel(answer, bar(BCL));
            }
            ++asked;
        };
        int k = 0, t = 0;  // queries and (beside `done`) key tiles whose loads have been issued
        for (; ok; ++k) {
            if (SPLIT && k > 0) break;
            t = 0;
            if (SPLIT || !is_k) {
                if (!next_item(k)) break;
            } else {
                bool more = true;  // the next item that has rows, if there is one
                done += n;
                n = 0;
                while (ok && more) {
                    if (asked > heard) {
                        ok = __all_sync(kFullMask, wait(BCL, heard++));
                        more = ok && canceled(answer, number);
                        __syncwarp();
                    }
                    if (more && find(number, lane == 0, it)) {
                        n = it.tiles;
                        break;
                    }
                    if (more) ask();
                }
                ok = ok && __all_sync(kFullMask, wait(BIE + (k & 1), (k >> 1) + 1));
                if (!ok) break;
                if (CROSS && n > 0) {
                    keep_ranges(k & 1, lane, 32);
                    __syncwarp();
                }
                if (lane == 0) {
                    it.tiles = n;
                    items[k & 1] = it;
                    mbar_arrive(bar(BIF + (k & 1)));
                }
                __syncwarp();
                if (n == 0) break;
            }
            const int32_t *bt = p.block_tables + (int64_t)it.s * p.max_blocks_per_seq;
            const int shift = it.sh >> bl;
            // CROSS: between the ranges of an item's rows there may be blocks that no row reaches
            auto reached = [&](int j) {
                if constexpr (CROSS) {
                    if (j >= n) return false;  // a look ahead, past this CTA's tiles
                    if (!it.holes || (j0 + j >= it.low && j0 + j < it.high)) return true;
                    const uint64_t seen = seen_keys(p, it, row_ranges + (k & 1) * kBM, (j0 + j) * kBN);
                    return lane < nb && (seen >> (lane << bl) & ((1ull << (1 << bl)) - 1)) != 0;
                }
                return true;
            };
            auto block_id = [&](int j) {
                const int v = (j0 + j) * nb + lane;
                if constexpr (CROSS) {
                    const bool in = reached(j) && lane < nb && v < it.blocks;
                    return in ? max(bt[v + shift], -1) : INT32_MIN;  // INT32_MIN: not looked up
                } else {
                    const int sink_blocks = it.sk >> bl;
                    return lane < nb && v < it.blocks ? bt[v < sink_blocks ? v : v + shift] : -1;
                }
            };
            int id0 = block_id(0), id1 = block_id(1);
            if (is_k) {
                int w_ok = 1;
                if (lane == 0) {
                    w_ok = SPLIT || wait(BQE, k + 1);
                    if (w_ok) {
                        mbar_arrive_expect_tx(bar(BQF), Sh::Q_BYTES);
                        for (int hf = 0; hf < Sh::HALVES; ++hf)
                            tma_load_3d(sQ + hf * (kBM * 128), &qmap, hf * 64, it.g << p.group_log2, it.q0 + it.tok,
                                        bar(BQF), policy);
                    }
                }
                ok = __shfl_sync(kFullMask, w_ok, 0);
                if (!ok) break;
            }
#pragma unroll 1
            for (; t < n; ++t) {
                const int id = id0;
                id0 = id1;
                id1 = block_id(t + 2);
                const bool in_range = CROSS ? id != INT32_MIN : lane < nb && (j0 + t) * nb + lane < it.blocks;
                const bool valid = id >= 0 && id < p.num_blocks;
                if (in_range && !valid) report(p.status, PA_DEVERR_BLOCK_ID);  // never dereferenced
                const uint32_t bytes = __popc(__ballot_sync(kFullMask, in_range)) * box_bytes;
                const int st = (done + t) % NS;
                int w_ok = 1;
                if (lane == 0) {
                    w_ok = wait(empty + st, (done + t) / NS + 1);
                    if (w_ok) mbar_arrive_expect_tx(bar(full + st), bytes);
                }
                ok = __shfl_sync(kFullMask, w_ok, 0);
                if (!ok) break;
                // A box past the pool's end is filled with zeros: a bad id's keys and values (not what the ring
                // held, another sequence's or NaN).  Masking such keys in the softmax instead took 3 to 8 % of
                // every call.
                if (in_range)
                    tma_load_5d(ring + st * Sh::KV_BYTES + lane * box_bytes, map, 0, 0, 0,
                                (valid ? id : p.num_blocks) << (bl - 3), it.g, bar(full + st), policy);
                __syncwarp();
                if (!SPLIT && is_k && t == n - 1) ask();
            }
        }
        // the last loads land before the warp leaves, also when a wait gave up
        bool landed = !is_k || k == 0 || mbar_wait(bar(BQF), (k - 1) & 1, p.status);
        for (int j = max(0, done + t - NS); j < done + t && landed; ++j)
            landed = mbar_wait(bar(full + j % NS), (j / NS) & 1, p.status);
        if (!SPLIT && asked > heard) mbar_wait(bar(BCL), heard & 1, p.status);  // no answer is left to land
        if (!ok) *abort_v = 1;
    } else if (warp == 1) {
        // ============================================ S_t = Q K_t^T
        // S_t overwrites the P of tile t - kSBufs: it waits until that P.V has finished.
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tmem = *reinterpret_cast<volatile uint32_t *>(tmem_slot);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BTM));
        for (int k = 0; ok && next_item(k); ++k) {
            if (lane == 0) {
                ok = wait(BQF, k);
                for (int t = 0; ok && t < n; ++t) {
                    const int st = (done + t) % NK, sb = (done + t) % kSBufs;
                    ok = wait(BKF + st, (done + t) / NK) && wait(BPV + sb, (done + t) / kSBufs + 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sK = sQ + Sh::OFF_K + st * Sh::KV_BYTES;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c)
                        mma_f16(tmem + sb * kBN, smem_desc(sQ + (c / 4) * (kBM * 128) + (c % 4) * 32, 16, 1024),
                                smem_desc(sK + (c / 4) * 1024 + (c % 4) * 32, 16, Sh::GSTR), IDESC_S, c > 0);
                    mma_commit(bar(BSF + sb));
                    mma_commit(bar(BKE + st));
                }
                if (!SPLIT && ok) mma_commit(bar(BQE));
            }
            ok = __shfl_sync(kFullMask, (int)ok, 0);
        }
        if (!ok) *abort_v = 1;
    } else if (warp == 3) {
        // ============================================ O += P_t V_t, P from TMEM
        ok = wait_tmem();
        for (int k = 0; ok && next_item(k); ++k) {
            for (int t = 0; ok && t < n; ++t) {
                const int st = (done + t) % NV, pb = (done + t) % kSBufs, k0 = (j0 + t) * kBN;
                const uint32_t sV = sQ + Sh::OFF_V + st * Sh::KV_BYTES;
                ok = __all_sync(kFullMask, wait(BVF + st, (done + t) / NV));
                if (ok && (j0 + t < it.low || j0 + t >= it.high)) {
                    // rows of V that no row of the item sees: [ns, lo) and past the last row (CROSS: outside
                    // every row's range)
                    int gap0 = 0, gap1 = 0, end = kBN;
                    uint64_t seen = 0;
                    if constexpr (CROSS) {
                        seen = seen_keys(p, it, row_ranges + (SPLIT ? 0 : (k & 1) * kBM), k0);
                    } else {
                        gap0 = it.ns - k0;
                        gap1 = it.virt(it.lo) - k0;
                        end = it.last + 1 - it.sh - k0;
                    }
                    constexpr int VEC = Sh::HALVES * 8;  // 16-byte pieces of a row
                    if (CROSS ? seen != ~0ull : gap1 > 0 || end < kBN)
                        for (int i = lane; i < kBN * VEC; i += 32) {
                            const int r = i / VEC, rest = i % VEC;
                            if (CROSS ? (seen >> r & 1) != 0 : r < end && (r < gap0 || r >= gap1)) continue;
                            sts128(sV + (r / 8) * Sh::GSTR + (rest / 8) * 1024 + (r % 8) * 128 + (rest % 8) * 16, 0u, 0u,
                                   0u, 0u);
                        }
                    if (!CROSS || seen != ~0ull) fence_async_smem();
                    __syncwarp();
                }
                if (lane == 0) {
                    ok = ok && (SPLIT || t > 0 || wait(BOE, k + 1)) && wait(BPF + pb, (done + t) / kSBufs);
                    if (ok) {
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < kBN / 16; ++c)
                            mma_f16_tmem_a(tmem + kTmemO, tmem + pb * kBN + c * 8,
                                           smem_desc(sV + c * 2 * Sh::GSTR, 1024, Sh::GSTR), IDESC_PV, t > 0 || c > 0);
                        mma_commit(bar(BPV + pb));
                        mma_commit(bar(BVE + st));
                    }
                }
                ok = __shfl_sync(kFullMask, (int)ok, 0);
            }
        }
        if (!ok) *abort_v = 1;
    } else {
        // ============================================ softmax and output
        // Warps 4-7 take rows 0-15 and warps 8-11 rows 16-31 of the TMEM lane quarter warp % 4:
        // a thread holds rows t/4 and t/4 + 8 of its slab, keys 8j + 2(t%4) and the next one of
        // each group of 8, so a row is spread over four lanes and a thread's pair of keys packs
        // into the P column 4j + t%4.
        const int quarter = warp & 3, slab = warp >= 8 ? 1 : 0;
        const int gi = lane >> 2, ga = lane & 3;
        const int lane0 = quarter * 32 + slab * 16;    // first TMEM lane (item row) of the slab
        const int row0 = lane0 + gi, row1 = row0 + 8;  // this thread's rows
        ok = wait_tmem();
        const uint32_t tL = tmem + ((uint32_t)lane0 << 16), tO = tL + kTmemO;
        const float sc = p.qk_scale_log2;
        constexpr float kGrow = kGrowLog2 + kLiftLog2<T>;
        for (int k = 0; ok && next_item(k); ++k) {
            const It &cur = SPLIT ? it : items[k & 1];
            const int low = cur.low, high = cur.high;
            float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // l: this lane's share
            for (int t = 0; ok && t < n; ++t) {
                const int sb = (done + t) % kSBufs;
                // CROSS: the keys of the tile that this thread's two rows see, and whether some row of the warp sees
                // a part of it
                int lo0 = 0, hi0 = kBN, lo1 = 0, hi1 = kBN;
                bool parts = false, blind = false;
                if constexpr (CROSS) {
                    if (j0 + t < low || j0 + t >= high) {
                        const int2 *ranges = row_ranges + (SPLIT ? 0 : (k & 1) * kBM);
                        const int k0 = cur.sh + (j0 + t) * kBN;
                        const int2 r0 = ranges[row0 >> p.group_log2], r1 = ranges[row1 >> p.group_log2];
                        lo0 = max(r0.x - k0, 0);
                        hi0 = min(r0.y - k0, kBN);
                        lo1 = max(r1.x - k0, 0);
                        hi1 = min(r1.y - k0, kBN);
                        const bool none0 = lo0 >= hi0, none1 = lo1 >= hi1;
                        blind = __all_sync(kFullMask, none0 && none1);
                        parts = __any_sync(kFullMask, (!none0 && (lo0 > 0 || hi0 < kBN)) || (!none1 && (lo1 > 0 || hi1 < kBN)));
                    }
                }
                ok = __all_sync(kFullMask, wait(BSF + sb, (done + t) / kSBufs));
                if (!ok) break;
                tc_fence_after();
                const uint32_t tS = tL + sb * kBN;
                // the tile is for other rows of the item (half of the rows of every item blind to all tiles but the
                // first: 290 us with their scores masked one by one, 225 so, 187 where all rows see all)
                if (CROSS && blind) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = 0u;
                    tmem_st_16x128b_x8(tS, w);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(BPF + sb));
                    continue;
                }
                uint32_t s[32];
                tmem_ld_16x256b<8>(tS, s);
                tmem_wait_ld();
                if (j0 + t < low || j0 + t >= high) {
                    if constexpr (CROSS) {
                        if (parts) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const int key = 8 * i + 2 * ga + e;
                                    if (key < lo0 || key >= hi0) s[4 * i + e] = __float_as_uint(-INFINITY);
                                    if (key < lo1 || key >= hi1) s[4 * i + 2 + e] = __float_as_uint(-INFINITY);
                                }
                        } else {  // rows that see all of the tile and rows that see nothing of it
                            const bool none0 = lo0 >= hi0, none1 = lo1 >= hi1;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                s[4 * i] = none0 ? __float_as_uint(-INFINITY) : s[4 * i];
                                s[4 * i + 1] = none0 ? __float_as_uint(-INFINITY) : s[4 * i + 1];
                                s[4 * i + 2] = none1 ? __float_as_uint(-INFINITY) : s[4 * i + 2];
                                s[4 * i + 3] = none1 ? __float_as_uint(-INFINITY) : s[4 * i + 3];
                            }
                        }
                    } else {
                        // in virtual keys a row sees v <= hi with v >= lo or v < ns; rows past the
                        // chunk (a ragged last item) as its last row: computed, never stored
                        const int k0 = (j0 + t) * kBN, ns = cur.virt(p.num_sinks) - k0;
                        const int p0 = min(cur.first + (row0 >> p.group_log2), cur.last);
                        const int p1 = min(cur.first + (row1 >> p.group_log2), cur.last);
                        const int hi0 = cur.virt(p0) - k0, lo0 = cur.virt(max(0, p0 - p.window + 1)) - k0;
                        const int hi1 = cur.virt(p1) - k0, lo1 = cur.virt(max(0, p1 - p.window + 1)) - k0;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int key = 8 * i + 2 * ga + e;
                                if (key > hi0 || (key < lo0 && key >= ns)) s[4 * i + e] = __float_as_uint(-INFINITY);
                                if (key > hi1 || (key < lo1 && key >= ns)) s[4 * i + 2 + e] = __float_as_uint(-INFINITY);
                            }
                    }
                }
                // maximum of the 16 scores per row in this lane
                float a0 = -INFINITY, a1 = -INFINITY, c0 = -INFINITY, c1 = -INFINITY;
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    a0 = fmax3(a0, __uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1]));
                    c0 = fmax3(c0, __uint_as_float(s[4 * i + 4]), __uint_as_float(s[4 * i + 5]));
                    a1 = fmax3(a1, __uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3]));
                    c1 = fmax3(c1, __uint_as_float(s[4 * i + 6]), __uint_as_float(s[4 * i + 7]));
                }
                float mx0 = fmaxf(a0, c0) * sc, mx1 = fmaxf(a1, c1) * sc;
                if (__any_sync(kFullMask, mx0 > m0 + kGrow || mx1 > m1 + kGrow)) {
                    // the row's maximum, the same in its four lanes
                    mx0 = fmaxf(mx0, __shfl_xor_sync(kFullMask, mx0, 1));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(kFullMask, mx1, 1));
                    mx0 = fmaxf(mx0, __shfl_xor_sync(kFullMask, mx0, 2));
                    mx1 = fmaxf(mx1, __shfl_xor_sync(kFullMask, mx1, 2));
                    const bool grow0 = mx0 > m0 + kGrow, grow1 = mx1 > m1 + kGrow;
                    const float n0 = grow0 ? mx0 - kLiftLog2<T> : m0, n1 = grow1 ? mx1 - kLiftLog2<T> : m1;
                    const float f0 = n0 == m0 ? 1.f : fast_exp2(m0 - n0);  // 0 from -inf
                    const float f1 = n1 == m1 ? 1.f : fast_exp2(m1 - n1);
                    l0 *= f0;
                    l1 *= f1;
                    m0 = n0;
                    m1 = n1;
                    if (t > 0) {  // O holds the tiles before: wait for the last P.V, scale the rows
                        ok = __all_sync(kFullMask, wait(BPV + (done + t - 1) % kSBufs, (done + t - 1) / kSBufs));
                        if (ok) {
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t o[16];
                                tmem_ld_16x256b_x4(tO + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    o[4 * i] = __float_as_uint(__uint_as_float(o[4 * i]) * f0);
                                    o[4 * i + 1] = __float_as_uint(__uint_as_float(o[4 * i + 1]) * f0);
                                    o[4 * i + 2] = __float_as_uint(__uint_as_float(o[4 * i + 2]) * f1);
                                    o[4 * i + 3] = __float_as_uint(__uint_as_float(o[4 * i + 3]) * f1);
                                }
                                tmem_st_16x256b_x4(tO + c, o);
                            }
                            tmem_wait_st();
                        }
                    }
                }
                {
                    const float b0_ = m0 == -INFINITY ? 0.f : m0, b1_ = m1 == -INFINITY ? 0.f : m1;
                    const float2 sc2 = make_float2(sc, sc), n0 = make_float2(-b0_, -b0_), n1 = make_float2(-b1_, -b1_);
                    float2 r0 = make_float2(0.f, 0.f), r1 = make_float2(0.f, 0.f);
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 x0 = __ffma2_rn(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])),
                                                     sc2, n0);
                        const float2 x1 = __ffma2_rn(
                            make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), sc2, n1);
                        w[2 * i] = pack2<T>(fast_exp2(x0.x), fast_exp2(x0.y));
                        w[2 * i + 1] = pack2<T>(fast_exp2(x1.x), fast_exp2(x1.y));
                        add_pair<T>(r0, w[2 * i]);
                        add_pair<T>(r1, w[2 * i + 1]);
                    }
                    if (ok) {
                        tmem_st_16x128b_x8(tS, w);
                        tmem_wait_st();
                    }
                    l0 += r0.x + r0.y;
                    l1 += r1.x + r1.y;
                }
                tc_fence_before();
                __syncwarp();
                if (!ok) break;
                if (lane == 0) mbar_arrive(bar(BPF + sb));
            }
            // ---- output
            ok = ok && (n == 0 || __all_sync(kFullMask, wait(BPV + (done + n - 1) % kSBufs, (done + n - 1) / kSBufs)));
            float L0 = l0 + __shfl_xor_sync(kFullMask, l0, 1), L1 = l1 + __shfl_xor_sync(kFullMask, l1, 1);
            L0 += __shfl_xor_sync(kFullMask, L0, 2);
            L1 += __shfl_xor_sync(kFullMask, L1, 2);
            if constexpr (SPLIT) {
                // into shared memory, over Q and the rings: every product that reads them is done
                if (ga == 0) {
                    float *ml = reinterpret_cast<float *>(smem + Sh::OFF_M);
                    ml[row0] = m0;
                    ml[row1] = m1;
                    ml[kBM + row0] = L0;
                    ml[kBM + row1] = L1;
                }
                if (ok && n > 0) {
                    tc_fence_after();
                    float *o = reinterpret_cast<float *>(smem);
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 64) {
                        uint32_t r[32];
                        tmem_ld_16x256b<8>(tO + c0, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            *reinterpret_cast<uint2 *>(o + row0 * Sh::PITCH + c0 + 8 * i + 2 * ga) =
                                make_uint2(r[4 * i], r[4 * i + 1]);
                            *reinterpret_cast<uint2 *>(o + row1 * Sh::PITCH + c0 + 8 * i + 2 * ga) =
                                make_uint2(r[4 * i + 2], r[4 * i + 3]);
                        }
                    }
                    tc_fence_before();
                }
            } else if (ok) {
                tc_fence_after();
                const float inv0 = L0 > 0.f ? 1.f / L0 : 0.f, inv1 = L1 > 0.f ? 1.f / L1 : 0.f;
                // one swap with the neighbouring lane gives each lane four consecutive columns, so
                // that a store instruction writes whole sectors of eight rows
                const bool odd = (ga & 1) != 0;
                auto write = [&](auto out_tag) {
                    using OT = decltype(out_tag);
                    OT *outp = static_cast<OT *>(p.out);
                    const int gl = p.group_log2;
                    const int tok0 = cur.tok + (row0 >> gl), tok1 = cur.tok + (row1 >> gl);
                    const int gm = (1 << gl) - 1, h = cur.g << gl;
                    const int64_t base0 = ((int64_t)(cur.q0 + tok0) * p.num_heads + h + (row0 & gm)) * D;
                    const int64_t base1 = ((int64_t)(cur.q0 + tok1) * p.num_heads + h + (row1 & gm)) * D;
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 64) {
                        uint32_t r[32];
                        tmem_ld_16x256b<8>(tO + c0, r);
                        tmem_wait_ld();
                        if (c0 + 64 == D) {  // the next item may write O
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar(BOE));
                        }
#pragma unroll
                        for (int rh = 0; rh < 2; ++rh) {
                            const float rinv = rh ? inv1 : inv0;
                            const int64_t base = (rh ? base1 : base0) + c0;
#pragma unroll
                            for (int i = 0; i < 8; i += 2) {
                                const int e0 = 4 * i + 2 * rh, e1 = 4 * (i + 1) + 2 * rh;
                                const float2 near = make_float2(__uint_as_float(r[e0]) * rinv, __uint_as_float(r[e0 + 1]) * rinv);
                                const float2 far = make_float2(__uint_as_float(r[e1]) * rinv, __uint_as_float(r[e1 + 1]) * rinv);
                                const int col = odd ? 8 * (i + 1) + 2 * (ga - 1) : 8 * i + 2 * ga;
                                const bool inside = (rh ? tok1 : tok0) < cur.Lq;
                                if constexpr (std::is_same<OT, float>::value) {
                                    const float2 keep = odd ? far : near, send = odd ? near : far;
                                    const float2 got = make_float2(__shfl_xor_sync(kFullMask, send.x, 1),
                                                                   __shfl_xor_sync(kFullMask, send.y, 1));
                                    const float2 a = odd ? got : keep, b = odd ? keep : got;
                                    if (inside) *reinterpret_cast<float4 *>(outp + base + col) = make_float4(a.x, a.y, b.x, b.y);
                                } else {
                                    using PT = typename std::conditional<std::is_same<OT, __half>::value, F16, BF16>::type;
                                    const uint32_t wn = pack2<PT>(near.x, near.y), wf = pack2<PT>(far.x, far.y);
                                    const uint32_t got = __shfl_xor_sync(kFullMask, odd ? wn : wf, 1);
                                    if (inside)
                                        *reinterpret_cast<uint2 *>(outp + base + col) =
                                            odd ? make_uint2(got, wf) : make_uint2(wn, got);
                                }
                            }
                        }
                    }
                };
                if (p.out_dtype == PA_F32)
                    write(float{});
                else if (p.out_dtype == PA_F16)
                    write(__half{});
                else
                    write(__nv_bfloat16{});
                tc_fence_before();
            }
            if constexpr (!SPLIT) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(BIE + (k & 1)));
            }
        }
        if (!ok) *abort_v = 1;
    }
    if (SPLIT && live) {
        // ---- the CTAs' outputs joined: each writes its share of the rows
        cluster_sync();
        const int cs = (int)cluster_size(), rows = kBM / cs, first = (int)cluster_rank() * rows;
        const uint32_t a_o = sQ, a_m = sQ + Sh::OFF_M, a_l = sQ + Sh::OFF_L;
        const int gl = p.group_log2;
        for (int i = tid; i < rows * (D / 4); i += kThreads) {
            const int row = first + i / (D / 4), d = i % (D / 4) * 4;
            const int tok = it.tok + (row >> gl);
            if (tok >= it.Lq) continue;
            float M = -INFINITY, L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r0 = 0; r0 < cs; r0 += 4) {  // four CTAs' loads in flight together
                float mr[4], lr[4];
                float4 xr[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int from = min(r0 + r, cs - 1);
                    mr[r] = ld_cluster(map_rank(a_m + 4 * row, from));
                    lr[r] = ld_cluster(map_rank(a_l + 4 * row, from));
                    xr[r] = ld_cluster4(map_rank(a_o + 4 * (row * Sh::PITCH + d), from));
                }
                float top = M;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if (r0 + r >= cs) mr[r] = -INFINITY;
                    top = fmaxf(top, mr[r]);
                }
                const float keep = M == -INFINITY ? 0.f : fast_exp2(M - top);
                M = top;
                L *= keep;
                acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // nothing seen (or no tile: no output there); NaN scores leave a NaN sum
                    if (lr[r] == 0.f || r0 + r >= cs) continue;
                    const float f = fast_exp2(mr[r] - M);
                    L = fmaf(lr[r], f, L);
                    acc.x = fmaf(xr[r].x, f, acc.x);
                    acc.y = fmaf(xr[r].y, f, acc.y);
                    acc.z = fmaf(xr[r].z, f, acc.z);
                    acc.w = fmaf(xr[r].w, f, acc.w);
                }
            }
            const float inv = L > 0.f ? 1.f / L : 0.f;
            const int64_t at =
                ((int64_t)(it.q0 + tok) * p.num_heads + (it.g << gl) + (row & ((1 << gl) - 1))) * D + d;
            if (p.out_dtype == PA_F32)
                *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) =
                    make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
            else if (p.out_dtype == PA_F16)
                *reinterpret_cast<uint2 *>(static_cast<__half *>(p.out) + at) =
                    make_uint2(pack2<F16>(acc.x * inv, acc.y * inv), pack2<F16>(acc.z * inv, acc.w * inv));
            else
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
                    make_uint2(pack2<BF16>(acc.x * inv, acc.y * inv), pack2<BF16>(acc.z * inv, acc.w * inv));
        }
        cluster_sync();  // nobody leaves while its shared memory is read
    }
    // ---- teardown: every TMEM access has completed before the columns are released
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (live && *abort_v) {  // a wait gave up: the products under way end before TMEM and shared memory go
        if (lane == 0 && (warp == 1 || warp == 3)) {
            mma_commit(bar(BDR + warp / 2));
            mbar_wait(bar(BDR + warp / 2), 0, p.status);
        }
        __syncthreads();
    }
    if (live && warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
}

// Both kernels are loaded by a device's first call, so that a captured call of other sizes
// than the eager ones before it loads nothing.
template <class T, int D, bool CROSS>
int load_typed() {
    constexpr int SMEM = CROSS ? Shape<D>::SMEM_CROSS : Shape<D>::SMEM;
    static std::atomic<int> loaded[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
    if (dev >= 0 && dev < kMaxDevices && loaded[dev].load(std::memory_order_acquire)) return PA_OK;
    for (auto kernel : {prefill_rows_kernel<T, D, false, CROSS>, prefill_rows_kernel<T, D, true, CROSS>})
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess)
            return PA_ERR_CUDA;
    if (dev >= 0 && dev < kMaxDevices) loaded[dev].store(1, std::memory_order_release);
    return PA_OK;
}

template <class T, int D, bool CROSS>
int launch_typed(const Params &p, int64_t items, int cluster, const CUtensorMap &qm, const CUtensorMap &km,
                 const CUtensorMap &vm, cudaStream_t st) {
    constexpr int SMEM = CROSS ? Shape<D>::SMEM_CROSS : Shape<D>::SMEM;
    static std::atomic<int> whole_ready[kMaxDevices], split_ready[kMaxDevices];  // shared-memory limit raised
    const int rc = load_typed<T, D, CROSS>();
    if (rc != PA_OK) return rc;
    const dim3 grid((unsigned)(items * cluster)), block(kThreads);
    const cudaError_t e = cluster > 1 ? launch_pdl_cluster(prefill_rows_kernel<T, D, true, CROSS>, split_ready, grid, block,
                                                           SMEM, SMEM, cluster, st, qm, km, vm, p)
                                      : launch_pdl_smem(prefill_rows_kernel<T, D, false, CROSS>, whole_ready, grid, block,
                                                        SMEM, st, qm, km, vm, p);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// The rows of `a`: CROSS with `key_ranges` (or null), or behind a.window and a.num_sinks.
template <bool CROSS>
int launch_rows(const PrefillArgs &a, const int32_t *key_ranges) {
    Params p{};
    p.key_ranges = key_ranges;
    p.max_query_len = a.max_query_len;
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.query_start_loc = a.query_start_loc;
    p.block_tables = a.block_tables;
    p.context_lens = a.context_lens;
    p.max_blocks_per_seq = a.max_blocks_per_seq;
    p.max_context_len = a.max_context_len;
    p.num_tokens = a.num_tokens;
    p.num_seqs = a.num_seqs;
    p.num_heads = a.num_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.block_log2 = a.block_size == 8 ? 3 : a.block_size == 16 ? 4 : 5;
    p.num_blocks = a.num_blocks;
    p.window = a.window;
    p.num_sinks = a.num_sinks;
    const int G = a.num_heads / a.num_kv_heads;
    p.group_log2 = G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3;
    const int longest = std::min(a.max_query_len, a.num_tokens);
    p.units_per_seq = (longest - 1) / (kBM / G) + 1;
    p.qk_scale_log2 = a.scale * kLog2e;
    p.status = a.status;
    // Chunks of one length fill num_seqs * units_per_seq items.  Ragged ones are numbered without
    // gaps, as long as the sequences fit the list: at most one item of each is not whole.
    const int64_t uniform = (int64_t)a.num_seqs * p.units_per_seq;
    const int64_t most = a.num_tokens / (kBM / G) + (int64_t)a.num_seqs;
    p.listed = a.num_seqs <= kPlanSeqs && most < uniform;
    const int64_t items = (p.listed ? most : uniform) * a.num_kv_heads;
    p.by_length = CROSS && a.num_seqs > 1 && a.num_seqs <= kMostRanked;
    // Few items: a cluster of CTAs takes each, up to one CTA per SM and at least four key tiles
    // per CTA (the join costs about one tile's time).  45 rows of 8 heads behind 4096 keys: 45.0
    // us whole, 13.9 in eights, 12.8 in sixteens; of 32 heads behind 512 keys: 11.7 whole, 9.6
    // in twos.
    const int64_t keys = CROSS ? a.max_context_len
                               : std::min<int64_t>(a.max_context_len, (int64_t)a.window + kBM / G + a.num_sinks);
    const int sms = device_sm_count();
    int cluster = 1;
    if constexpr (CROSS) {
        // A split item has no next one under its end, and pays about 8 us for that.  One sequence of 500,
        // 1500 and 6000 keys, whole | in twos | fours | eights (us): 32 items 12, 23, 74 | 14, 19, 46 |
        // 12, 15, 28 | 18, 20, 28; 72 items 12, 24, 73 | 15, 20, 45 | 15, 19, 35 | 32, 37, 53; 144 items
        // 14, 25, 75 | 19, 27, 57 | 28, 36, 66; 16 items of 6000 keys 28 in fours, 25 in eights.
        const int64_t slots = 2 * (int64_t)sms;
        // listed items: a sequence's last one is half full on average
        const int64_t likely = p.listed ? (a.num_tokens / (kBM / G) + (a.num_seqs + 1) / 2) * (int64_t)a.num_kv_heads : items;
        if (likely * 4 <= sms ? keys > 384 : likely * 4 <= slots * 63 / 64 && keys > 1024) cluster = 4;
        // Beyond that twos even out items of unequal length, at the cost of the joins.  Of the time of whole
        // items, chunks of one length and ragged ones alike, 154 to 202 items at head dimension 64 | 128:
        // contexts of 0 to 8000 keys 0.52 to 0.61 | 0.63 to 0.65, all of 6000 0.89 to 0.90 | 0.98 to 1.03, all of
        // 3000 1.01 to 1.02 | 1.12 to 1.18, all of 1500 1.17 to 1.20 | 1.26 to 1.33 (237 to 256 items of 3000
        // keys 1.20 to 1.21 | 1.26 to 1.35).  Ranges make the items of equal contexts unequal too: up to 243 items
        // beside one and four images, of 0 to 8000 keys 0.57 to 0.75 | 0.60 to 0.77, all of 6400 0.63 to 0.91 |
        // 0.67 to 1.01, all of 3200 0.74 to 1.07 | 0.83 to 1.17, all of 1600 0.92 to 1.35 | 1.00 to 1.54 (244 to
        // 296 items of 3200 keys 0.91 to 1.15 | 1.06 to 1.24).
        else if (likely * 2 <= slots ? keys > 2048
                                     : keys > 32 * (int64_t)a.head_dim &&
                                           (key_ranges ? likely * 5 <= slots * 4 : likely * 3 <= slots * 2))
            cluster = 2;
        while (cluster >= 4 && cluster < 16 && likely * cluster * 2 <= sms && keys > 512 * (int64_t)cluster) cluster *= 2;
    } else {
        while (cluster < 16 && items * cluster * 2 <= sms && keys > (int64_t)kBN * 4 * cluster) cluster *= 2;
    }
    const int64_t rows = (int64_t)a.num_blocks * a.block_size;
    if (rows <= 0 || rows > INT32_MAX || items > INT32_MAX) return PA_ERR_INVALID_ARG;
    // Q boxes are 64 elements (the swizzle span) wide and cover the G heads of one kv head for
    // 128/G tokens; a K/V box is one block of one kv head, all of D in 64-wide slices.
    CUtensorMap qm, km, vm;
    if (make_tensor_map_3d(&qm, a.query, a.kv_dtype, a.head_dim, a.num_heads, a.num_tokens, 64, G, kBM / G, true) !=
            PA_OK ||
        make_kv_block_map(&km, a.key_cache, a.kv_dtype, a.head_dim, a.num_kv_heads, rows, a.block_size) != PA_OK ||
        make_kv_block_map(&vm, a.value_cache, a.kv_dtype, a.head_dim, a.num_kv_heads, rows, a.block_size) != PA_OK)
        return PA_ERR_CUDA;
    switch (a.kv_dtype) {
        case PA_F16:
            return a.head_dim == 64 ? launch_typed<F16, 64, CROSS>(p, items, cluster, qm, km, vm, a.stream)
                                    : launch_typed<F16, 128, CROSS>(p, items, cluster, qm, km, vm, a.stream);
        case PA_BF16:
            return a.head_dim == 64 ? launch_typed<BF16, 64, CROSS>(p, items, cluster, qm, km, vm, a.stream)
                                    : launch_typed<BF16, 128, CROSS>(p, items, cluster, qm, km, vm, a.stream);
        default: return PA_ERR_UNSUPPORTED;
    }
}

}  // namespace
}  // namespace pa
