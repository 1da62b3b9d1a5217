// tables.cu -- block tables, row starts, positions and slots of a step, made on the GPU from
// the sequences' lengths, and blocks given back (include/pa.h: pa_tables_extend, pa_tables_trim).
//
// need_s = ceil((cached_s + new_s) / bs) - ceil(cached_s / bs); P = prefix sums of need; block i of
// the call is entry F - 1 - i of the free stack.  A sequence is served when its own blocks end
// within the F free ones (P is monotone, so those that need blocks are served in order until the
// stack is empty), and the blocks taken are the largest P of a served one.
//
// One cluster does it all, in one launch: a grid of independent CTAs would need a second launch
// (or a scratch array) between the prefix sums and what they address, and between reading
// cached_lens and num_free and writing them in place.  Every CTA sums all sequences, 2048 at
// a time, so that the CTAs exchange nothing but one barrier; then they share out the blocks and the
// tokens, one per thread, each found by a binary search in the prefix sums in shared memory.
// Sums saturate one past what they are compared with, so that no length overflows them.
#include <algorithm>

#include "cluster.cuh"
#include "tables.cuh"

namespace pa {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kPer = 2, kSlice = kThreads * kPer;  // sequences per thread and per pass

struct Pair {
    uint32_t rows, blocks;
};

// Inclusive sums over the block, both saturating at their caps.
__device__ __forceinline__ Pair block_scan(Pair v, Pair cap, Pair (&warp_sums)[kWarps]) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    auto scan = [&](Pair x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t r = __shfl_up_sync(kFullMask, x.rows, o), b = __shfl_up_sync(kFullMask, x.blocks, o);
            if (lane >= o) x = {min(x.rows + r, cap.rows), min(x.blocks + b, cap.blocks)};
        }
        return x;
    };
    v = scan(v);
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    if (warp == 0) warp_sums[lane] = scan(warp_sums[lane]);
    __syncthreads();
    if (warp > 0) {
        const Pair before = warp_sums[warp - 1];
        v = {min(v.rows + before.rows, cap.rows), min(v.blocks + before.blocks, cap.blocks)};
    }
    return v;
}

// Largest i < n with at[i] <= x (at[0] <= x).
__device__ __forceinline__ int last_not_past(const uint32_t *at, int n, uint32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int blocks_of(int tokens, int log2) { return (int)(((int64_t)tokens + (1 << log2) - 1) >> log2); }

// EXTEND: sequences grow by `lens` tokens.  Else they shrink to `lens` tokens.
template <bool EXTEND>
__global__ void __launch_bounds__(kThreads) tables_kernel(const TablesArgs p, int block_log2) {
    __shared__ uint32_t starts[kSlice + 1], firsts[kSlice + 1];  // row and block that a sequence begins with
    __shared__ int cached_of[kSlice];                            // its cached length; ~length: it is not served
    __shared__ Pair warp_sums[kWarps];
    __shared__ uint32_t taken;
    const int tid = threadIdx.x, rank = (int)cluster_rank(), ranks = (int)cluster_size();
    pdl_wait_previous();
    pdl_launch_dependents();

    int free0 = *p.num_free;
    int err = 0;
    if (free0 < 0 || free0 > p.free_capacity) {
        err |= PA_DEVERR_FREE_LIST;
        free0 = free0 < 0 ? 0 : p.free_capacity;
    }
    const uint32_t most_rows = EXTEND ? p.num_tokens : 0, most_blocks = EXTEND ? free0 : p.free_capacity - free0;
    const Pair cap{most_rows + 1, most_blocks + 1};
    const int64_t room = (int64_t)p.max_blocks_per_seq << block_log2;  // tokens of a table row
    if (tid == 0) taken = 0;
    Pair carry{0, 0};
    if (EXTEND && p.query_start_loc && rank == 0 && tid == 0) p.query_start_loc[0] = 0;

    for (int base = 0; base < p.num_seqs; base += kSlice) {
        const int n = min(kSlice, p.num_seqs - base);
        Pair mine[kPer];
        int cached[kPer], len[kPer];
        bool valid[kPer];
        Pair sum{0, 0};
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int i = tid * kPer + u;
            cached[u] = i < n ? p.cached_lens[base + i] : 0;
            len[u] = i < n ? p.lens[base + i] : 0;
        }
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int c = cached[u], m = len[u];
            if (EXTEND) {
                valid[u] = c >= 0 && m >= 0 && (int64_t)c + m <= room;
                if (m < 0) err |= PA_DEVERR_QUERY;
                if (c < 0 || (m >= 0 && (int64_t)c + m > room)) err |= PA_DEVERR_CONTEXT;
                len[u] = max(m, 0);
                mine[u].rows = min((uint32_t)len[u], cap.rows);
                mine[u].blocks = 0;  // set once it is known that its rows fit
            } else {
                valid[u] = c >= 0 && m >= 0 && m <= c && c <= room;
                if (!valid[u]) err |= PA_DEVERR_CONTEXT;
                mine[u].rows = 0;
                mine[u].blocks = valid[u] ? min((uint32_t)(blocks_of(c, block_log2) - blocks_of(m, block_log2)), cap.blocks) : 0;
            }
            cached[u] = max(c, 0);
        }
        uint32_t row_end[kPer];
        if (EXTEND) {  // rows first: a sequence whose rows do not fit takes no blocks
#pragma unroll
            for (int u = 0; u < kPer; ++u) sum.rows = min(sum.rows + mine[u].rows, cap.rows);
            const Pair incl = block_scan(sum, cap, warp_sums);
            // what lies before this thread's sequences: exact as long as it is not saturated
            uint32_t at = __shfl_up_sync(kFullMask, incl.rows, 1);
            if (tid % 32 == 0) at = tid == 0 ? 0 : warp_sums[tid / 32 - 1].rows;
            at = min(at + carry.rows, cap.rows);
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int i = tid * kPer + u;
                if (i < n) starts[i] = min(at, most_rows);
                at = min(at + mine[u].rows, cap.rows);
                row_end[u] = at;
                const bool fits = len[u] == 0 || at <= most_rows;
                if (!fits) err |= PA_DEVERR_QUERY;
                valid[u] = valid[u] && fits && len[u] > 0;
                if (valid[u])
                    mine[u].blocks = min((uint32_t)(blocks_of(cached[u] + len[u], block_log2) - blocks_of(cached[u], block_log2)), cap.blocks);
            }
            carry.rows = min(carry.rows + warp_sums[kWarps - 1].rows, cap.rows);
            __syncthreads();
        }
        sum = {0, 0};
#pragma unroll
        for (int u = 0; u < kPer; ++u) sum.blocks = min(sum.blocks + mine[u].blocks, cap.blocks);
        const Pair incl = block_scan(sum, cap, warp_sums);
        uint32_t at = __shfl_up_sync(kFullMask, incl.blocks, 1);
        if (tid % 32 == 0) at = tid == 0 ? 0 : warp_sums[tid / 32 - 1].blocks;
        at = min(at + carry.blocks, cap.blocks);
        uint32_t high = 0;
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int i = tid * kPer + u;
            bool served = valid[u];
            if (i < n) firsts[i] = at;
            at = min(at + mine[u].blocks, cap.blocks);
            if (served && mine[u].blocks > 0) {
                if (at <= most_blocks) {
                    high = at;
                } else {
                    err |= PA_DEVERR_FREE_LIST;
                    // trim: the blocks past the list's end are dropped, the length shrinks all the same
                    if (EXTEND) served = false;
                    else high = most_blocks;
                }
            }
            if (i < n) cached_of[i] = served ? cached[u] : ~cached[u];
            valid[u] = served;
        }
        if (high > 0) atomicMax(&taken, high);
        const uint32_t first_block = carry.blocks;
        const uint32_t rows_end = min(carry.rows, most_rows);  // of this slice
        carry.blocks = min(carry.blocks + warp_sums[kWarps - 1].blocks, cap.blocks);
        // Before anything is written in place, every CTA has read what it replaces.
        if (ranks > 1) cluster_sync();
        __syncthreads();
        if (rank == (base / kSlice) % ranks) {
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int i = tid * kPer + u;
                if (i >= n) continue;
                p.context_lens[base + i] = !valid[u] ? cached[u] : EXTEND ? cached[u] + len[u] : len[u];
                if (EXTEND && p.query_start_loc) p.query_start_loc[base + i + 1] = (int)min(row_end[u], most_rows);
            }
        }
        // ---- blocks: number i of the call
        for (uint32_t i = first_block + rank * kThreads + tid; i < min(taken, carry.blocks); i += ranks * kThreads) {
            const int s = last_not_past(firsts, n, i);
            const int c = cached_of[s] < 0 ? ~cached_of[s] : cached_of[s], have = blocks_of(c, block_log2);
            const int64_t row = (int64_t)(base + s) * p.max_blocks_per_seq;
            int id;
            if (EXTEND) {
                id = p.free_blocks[free0 - 1 - (int)i];
                p.block_tables[row + have + (int)(i - firsts[s])] = id;
            } else {
                id = p.block_tables[row + have - 1 - (int)(i - firsts[s])];
                p.free_blocks[free0 + (int)i] = id;
            }
            if (id < 0 || id >= p.num_blocks) err |= PA_DEVERR_BLOCK_ID;
        }
        // ---- tokens
        if (EXTEND) {
            const uint32_t begin = starts[0];
            for (uint32_t t = begin + rank * kThreads + tid; t < rows_end; t += ranks * kThreads) {
                const int s = last_not_past(starts, n, t);
                const int c = cached_of[s];
                int64_t slot = -1;
                int pos = 0;
                if (c >= 0) {
                    pos = c + (int)(t - starts[s]);
                    const int b = pos >> block_log2, have = blocks_of(c, block_log2);
                    const int id = b < have ? p.block_tables[(int64_t)(base + s) * p.max_blocks_per_seq + b]
                                            : p.free_blocks[free0 - 1 - (int)firsts[s] - (b - have)];
                    if (id >= 0 && id < p.num_blocks) slot = ((int64_t)id << block_log2) + (pos & ((1 << block_log2) - 1));
                    else err |= PA_DEVERR_BLOCK_ID;
                }
                if (p.positions) p.positions[t] = pos;
                p.slot_mapping[t] = slot;
            }
        }
        __syncthreads();  // the next slice writes the shared arrays
    }
    if (p.num_seqs == 0) {
        if (ranks > 1) cluster_sync();
        __syncthreads();
    }
    if (EXTEND) {  // rows behind the last sequence
        for (uint32_t t = min(carry.rows, most_rows) + rank * kThreads + tid; t < most_rows; t += ranks * kThreads) {
            if (p.positions) p.positions[t] = 0;
            p.slot_mapping[t] = -1;
        }
    }
    if (rank == 0 && tid == 0) *p.num_free_out = EXTEND ? free0 - (int)taken : free0 + (int)taken;
    if (err) report(p.status, err);
}

template <bool EXTEND>
int launch(const TablesArgs &a, int64_t work) {
    static std::atomic<int> ready[kMaxDevices];
    int cluster = 1;
    while (cluster < 8 && work > (int64_t)kThreads * cluster) cluster *= 2;
    const int log2 = a.block_size == 8 ? 3 : a.block_size == 16 ? 4 : 5;
    return launch_pdl_cluster(tables_kernel<EXTEND>, ready, dim3(cluster), dim3(kThreads), 0, cluster, a.stream, a, log2) ==
                   cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace

int launch_tables_extend(const TablesArgs &a) { return launch<true>(a, a.num_tokens); }
int launch_tables_trim(const TablesArgs &a) { return launch<false>(a, (int64_t)a.num_seqs * 8); }

}  // namespace pa
