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
// tokens, each found by a binary search in the prefix sums in shared memory, four of a thread's
// side by side.  Where every sequence has four at most (a decode step, rejected drafts), a
// thread sees to its own sequences and nothing is searched.  Sums saturate one past what they are
// compared with, so that no length overflows them.
//
// What bounds it is latency: the launch, the lengths, two barriers of the sums, a search (11 steps),
// an entry of the list or the table, the store.  Measured in a replayed graph (us): 64 sequences of
// one token each 3.9, 32 of 512 tokens 4.4 (11.2 in one CTA), 2048 of 0 to 60 tokens 7.4 (43.8 in one
// CTA); blocks given back by 256 sequences that lose up to 8 tokens 3.6, by 512 ended of 1024 (132000
// blocks) 7.6 (65.6 in one CTA).  One search at a time per thread took 8.8 and 17 us for the two large
// ones; searches for single tokens of 2000 sequences 7.2 us (bank conflicts), a thread per
// sequence 5.1.
#include <algorithm>
#include <type_traits>

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

// For each x: the largest i < n with at[i] <= x (at[0] <= x), F searches side by side.  What lies behind
// at[n - 1] is read but not used.
template <int F>
__device__ __forceinline__ void last_not_past(const uint32_t *at, int n, const uint32_t (&x)[F], int (&i)[F]) {
#pragma unroll
    for (int u = 0; u < F; ++u) i[u] = 0;
    auto steps = [&](auto first) {
#pragma unroll
        for (int step = decltype(first)::value; step; step >>= 1)
#pragma unroll
            for (int u = 0; u < F; ++u) {
                const int j = i[u] + step;
                const bool past = at[j] > x[u];
                if (j < n && !past) i[u] = j;
            }
    };
    if (n > 64) steps(std::integral_constant<int, kSlice / 2>{});
    else steps(std::integral_constant<int, 32>{});
}

__device__ __forceinline__ int blocks_of(int tokens, int log2) { return (int)(((int64_t)tokens + (1 << log2) - 1) >> log2); }

constexpr int kFlight = 4;  // blocks or tokens that a thread takes at once, so that their latencies overlap
constexpr int kDirect = 4;  // blocks or tokens per sequence up to which each thread sees to its own

// f(i, how many at once) over begin .. end - 1 by `stride` threads, this one the number `at`.
template <class Fn>
__device__ __forceinline__ void share_out(uint32_t begin, uint32_t end, uint32_t stride, uint32_t at, Fn f) {
    for (uint32_t i = begin; i < end;) {
        const bool rest = end - i <= stride;
        if (i + at < end) {
            if (rest) f(i + at, std::integral_constant<int, 1>{});
            else f(i + at, std::integral_constant<int, kFlight>{});
        }
        if (rest || end - i <= kFlight * stride) break;
        i += kFlight * stride;
    }
}

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
                valid[u] = valid[u] && len[u] > 0;
                mine[u].rows = min((uint32_t)len[u], cap.rows);
                mine[u].blocks = valid[u] ? min((uint32_t)(blocks_of(c + m, block_log2) - blocks_of(c, block_log2)), cap.blocks) : 0;
            } else {
                valid[u] = c >= 0 && m >= 0 && m <= c && c <= room;
                if (!valid[u]) err |= PA_DEVERR_CONTEXT;
                mine[u].rows = 0;
                mine[u].blocks = valid[u] ? min((uint32_t)(blocks_of(c, block_log2) - blocks_of(m, block_log2)), cap.blocks) : 0;
            }
            cached[u] = max(c, 0);
        }
        // Both sums at once, as if all rows fitted; only if they do not, the blocks are summed again
        // without the sequences whose rows end past num_tokens.
#pragma unroll
        for (int u = 0; u < kPer; ++u)
            sum = {min(sum.rows + mine[u].rows, cap.rows), min(sum.blocks + mine[u].blocks, cap.blocks)};
        const uint32_t before = carry.rows;
        Pair incl = block_scan(sum, cap, warp_sums);
        const uint32_t rows_end = min(before + warp_sums[kWarps - 1].rows, cap.rows);
        carry.rows = rows_end;
        uint32_t row_end[kPer];
        if (EXTEND) {
            uint32_t at = __shfl_up_sync(kFullMask, incl.rows, 1);  // rows before this thread's
            if (tid % 32 == 0) at = tid == 0 ? 0 : warp_sums[tid / 32 - 1].rows;
            at = min(at + before, cap.rows);
            sum.blocks = 0;
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int i = tid * kPer + u;
                if (i < n) starts[i] = min(at, most_rows);
                at = min(at + mine[u].rows, cap.rows);
                row_end[u] = at;
                if (at > most_rows && len[u] > 0) {
                    err |= PA_DEVERR_QUERY;
                    valid[u] = false;
                    mine[u].blocks = 0;
                }
                sum.blocks = min(sum.blocks + mine[u].blocks, cap.blocks);
            }
            if (rows_end > most_rows) {  // the same for every thread
                __syncthreads();
                incl = block_scan(sum, cap, warp_sums);
            }
        }
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
        carry.blocks = min(carry.blocks + warp_sums[kWarps - 1].blocks, cap.blocks);
        // Before anything is written in place, every CTA has read what it replaces.
        bool many = false;
#pragma unroll
        for (int u = 0; u < kPer; ++u) many = many || (EXTEND ? (uint32_t)len[u] : mine[u].blocks) > kDirect;
        if (ranks > 1) cluster_sync();
        const bool direct = !__syncthreads_or(many);
        if (rank == (base / kSlice) % ranks) {
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int i = tid * kPer + u;
                if (i >= n) continue;
                p.context_lens[base + i] = !valid[u] ? cached[u] : EXTEND ? cached[u] + len[u] : len[u];
                if (EXTEND && p.query_start_loc) p.query_start_loc[base + i + 1] = (int)min(row_end[u], most_rows);
            }
        }
        const uint32_t stride = ranks * kThreads;
        // ---- few of them per sequence: each thread sees to its own sequences, the warps shared out
        // over the CTAs (a search costs an access to a random bank per step)
        if (direct) {
            if (tid / 32 % ranks == rank) {
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    const int i = tid * kPer + u;
                    if (i >= n) continue;
                    const int have = blocks_of(cached[u], block_log2), first = (int)firsts[i];
                    int32_t *row = p.block_tables + (int64_t)(base + i) * p.max_blocks_per_seq;
                    if (EXTEND) {
                        const int rows = min((int)(min(row_end[u], most_rows) - starts[i]), kDirect);
                        for (int k = 0; k < rows; ++k) {
                            const int pos = valid[u] ? cached[u] + k : 0, b = pos >> block_log2;
                            int64_t slot = -1;
                            if (valid[u]) {
                                const int id = b < have ? row[b] : p.free_blocks[free0 - 1 - first - (b - have)];
                                // a new block's first token enters it into the table
                                if (b >= have && (k == 0 || (pos & ((1 << block_log2) - 1)) == 0)) row[b] = id;
                                if (id >= 0 && id < p.num_blocks) slot = ((int64_t)id << block_log2) + (pos & ((1 << block_log2) - 1));
                                else err |= PA_DEVERR_BLOCK_ID;
                            }
                            if (p.positions) p.positions[starts[i] + k] = pos;
                            p.slot_mapping[starts[i] + k] = slot;
                        }
                    } else if (valid[u]) {
                        for (int k = 0; k < (int)mine[u].blocks && first + k < (int)most_blocks; ++k) {
                            const int id = row[have - 1 - k];
                            p.free_blocks[free0 + first + k] = id;
                            if (id < 0 || id >= p.num_blocks) err |= PA_DEVERR_BLOCK_ID;
                        }
                    }
                }
            }
            __syncthreads();  // the next slice writes the shared arrays
            continue;
        }
        // ---- blocks: number i of the call
        const uint32_t blocks_end = min(taken, carry.blocks);
        auto blocks = [&](uint32_t i0, auto flight) {
            constexpr int F = decltype(flight)::value;
            uint32_t number[F];
            int s[F], id[F];
#pragma unroll
            for (int u = 0; u < F; ++u) number[u] = min(i0 + u * stride, blocks_end - 1);
            last_not_past<F>(firsts, n, number, s);
            int32_t *entry[F];
#pragma unroll
            for (int u = 0; u < F; ++u) {
                const int have = blocks_of(cached_of[s[u]], block_log2), k = (int)(number[u] - firsts[s[u]]);
                entry[u] = p.block_tables + (int64_t)(base + s[u]) * p.max_blocks_per_seq + (EXTEND ? have + k : have - 1 - k);
                id[u] = EXTEND ? p.free_blocks[free0 - 1 - (int)number[u]] : *entry[u];
            }
#pragma unroll
            for (int u = 0; u < F; ++u) {
                if (i0 + u * stride >= blocks_end) break;
                if (EXTEND) *entry[u] = id[u];
                else p.free_blocks[free0 + (int)number[u]] = id[u];
                if (id[u] < 0 || id[u] >= p.num_blocks) err |= PA_DEVERR_BLOCK_ID;
            }
        };
        share_out(first_block, blocks_end, stride, rank * kThreads + tid, blocks);
        // ---- tokens
        if (EXTEND) {
            const uint32_t end = min(rows_end, most_rows);
            auto tokens = [&](uint32_t t0, auto flight) {
                constexpr int F = decltype(flight)::value;
                uint32_t token[F];
                int s[F], pos[F], id[F];
                bool live[F];  // its sequence is served
#pragma unroll
                for (int u = 0; u < F; ++u) token[u] = min(t0 + u * stride, end - 1);
                last_not_past<F>(starts, n, token, s);
#pragma unroll
                for (int u = 0; u < F; ++u) {
                    const int c = cached_of[s[u]], first = (int)firsts[s[u]];
                    live[u] = c >= 0;
                    pos[u] = live[u] ? c + (int)(token[u] - starts[s[u]]) : 0;
                    const int b = pos[u] >> block_log2, have = blocks_of(max(c, 0), block_log2);
                    // its block: one that the sequence had, or one taken from the list
                    const int32_t *from = b < have ? p.block_tables + (int64_t)(base + s[u]) * p.max_blocks_per_seq + b
                                                   : p.free_blocks + (free0 - 1 - first - (b - have));
                    id[u] = -1;
                    if (live[u]) id[u] = *from;
                }
#pragma unroll
                for (int u = 0; u < F; ++u) {
                    const uint32_t t = t0 + u * stride;
                    if (t >= end) break;
                    const bool ok = id[u] >= 0 && id[u] < p.num_blocks;
                    if (live[u] && !ok) err |= PA_DEVERR_BLOCK_ID;
                    if (p.positions) p.positions[t] = pos[u];
                    p.slot_mapping[t] = ok ? ((int64_t)id[u] << block_log2) + (pos[u] & ((1 << block_log2) - 1)) : -1;
                }
            };
            share_out(min(before, most_rows), end, stride, rank * kThreads + tid, tokens);
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

// `work`: tokens, or table entries of which some go back.  More CTAs than the work needs cost next to nothing
// (one token of one sequence 4.1 us in one CTA, 4.3 in sixteen), fewer cost their share of it.
template <bool EXTEND>
int launch(const TablesArgs &a, int64_t work) {
    static std::atomic<int> ready[kMaxDevices];
    int cluster = 1;
    while (cluster < 16 && work > (int64_t)kThreads * cluster) cluster *= 2;
    const int log2 = a.block_size == 8 ? 3 : a.block_size == 16 ? 4 : 5;
    return launch_pdl_cluster(tables_kernel<EXTEND>, ready, dim3(cluster), dim3(kThreads), 0, 0, cluster, a.stream, a, log2) ==
                   cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // namespace

int launch_tables_extend(const TablesArgs &a) { return launch<true>(a, a.num_tokens); }
int launch_tables_trim(const TablesArgs &a) { return launch<false>(a, (int64_t)a.num_seqs * a.max_blocks_per_seq); }

}  // namespace pa
