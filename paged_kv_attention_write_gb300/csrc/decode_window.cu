// decode_window.cu -- decode attention over a sliding window with sinks, on GB300: one
// launch, TMA-fed, the pieces of a sequence merged through distributed shared memory.
//
// out[s][h] = sum_j softmax_j(scale q.k_j) v_j over the keys j < C with j >= C - window or
// j < num_sinks (C the context length).  The keys a row sees are bounded by window +
// num_sinks whatever C is, so the split needs no plan on the device: one cluster of CS CTAs
// takes one (sequence, kv head), each CTA an equal run of its visible keys, and the CTAs
// merge their (max, sum, output) through each other's shared memory before they exit.  No
// workspace, no second kernel, nothing shared between calls.
//
// Keys are walked in groups of 8 consecutive tokens (the finest piece that one block of any
// block size and one 128-byte-swizzled box holds), the groups of the sinks first, then
// those of the window: "virtual" group v is logical group v below the sink groups and v +
// shift above.  Only the groups at a border need a mask.  A TMA box brings one group, or a
// whole block where latency counts (both counts of groups then round to blocks).
//
// Per CTA one producer warp looks up block ids (one lane per group, a stage ahead) and
// issues the TMA boxes into a ring of stages; the consumer warps each take their own groups
// of a stage and keep their own running maximum, sum and output.
//   16-bit caches: tensor cores, mma.m16n8k16 with the keys (Q.K) or the head dimension
//     (P.V) as the 16 rows and the kv head's query heads, at most eight, as the 8 columns:
//     S = K Q^T, O^T = V^T P.  At one query token the products are far below the tensor
//     rate (the kernel is bound by HBM), but on the CUDA cores eight heads would bound it.
//     P enters as a rounded part plus its rounded remainder (two products), so that the
//     weights keep 2^-16 of themselves (bf16) or 2^-22 (fp16, but nothing below 2^-32 of the
//     largest), and the 16 keys of a step are summed apart from O.  Summed
//     into O, 65536 keys behind one that weighs e^14 of a light one came out 5.5e-4 off (now
//     7e-6); the sums cost 0.2 to 1 % (320 pairs of 260 keys, D 64, 13.5 -> 13.7 us; 1024 pairs
//     of 1028 keys, D 128, 87.5 -> 87.8).
//   fp32 caches: packed fp32 FMAs, eight lanes per key, eight keys per warp step, at most four
//     query heads per warp.
// Many (sequence, kv head) pairs of few keys each (16-bit caches; the rule is at the launch)
// take one warp, a CTA of its own, per pair instead: it issues its own boxes into its own ring
// and joins nothing.  In the clusters' kernel such pairs wait for the start and the end of a
// CTA of five warps, two of them at a time on an SM; here up to eight pairs are in flight.
// Measured (bf16 or fp16, D 128, GPU us): 128 sequences x 4112 keys, 64 q / 8 kv heads 314
// (6.83 TB/s, the measured copy rate is 6.68); 32 x 1028, 32 / 8 heads 23.1 (5.7 TB/s: 256 CTAs
// of 17 stages, the first loads and the last merges show); 1 x 516 5.5, 1 x 4100 7.7 (launch,
// a chain of context -> block table -> box -> scores -> joins).
// fp32 caches, 64 sequences x 2052 keys, 8 kv heads, D 128: 155 (1 query head per kv head, 6.9
// TB/s), 159 (4), 183 (8).  CTAs of eight consumer warps, one per SM, took 164, 171 and 210:
// nothing ran under their beginnings and ends.
// Every mbarrier wait is bounded in time; if one gives up, the boxes under way still land before the
// CTA leaves (not run on a GPU: it would take a wait of two seconds).
#include <algorithm>
#include <type_traits>

#include "cluster.cuh"
#include "tma.cuh"

namespace pa {
namespace {

constexpr float kGrowLog2 = 8.f;  // the softmax reference moves when a score exceeds it by 2^8
// Weights against the reference times 2^kLiftLog2: fp16 has no bits below 2^-24, so weights use its
// upper range (at most 2^(7 + 8), of 2^16).  The factor is in O and in the sum alike and cancels.
template <class T>
constexpr float kLiftLog2 = std::is_same<T, F16>::value ? 7.f : 0.f;

struct Params {
    void *out;
    pa_dtype out_dtype;
    const void *query;
    const int32_t *block_tables, *context_lens;
    int max_blocks_per_seq, max_context_len, num_heads, num_kv_heads, group, block_size, num_blocks;
    int window, num_sinks;
    int unit;  // groups of 8 keys that one TMA box brings: 1, or a block's
    float qk_scale_log2;
    int32_t *status;
};

template <class T, int D>
struct Shape {
    static constexpr bool kF32 = std::is_same<T, F32>::value;
    static constexpr int GROUP_BYTES = 8 * D * T::kBytes;        // 8 tokens of one kv head
    static constexpr int NGRP = 16384 / GROUP_BYTES;             // groups per stage (16 KB of K, 16 KB of V)
    static constexpr int KV_BYTES = NGRP * GROUP_BYTES;
    static constexpr int NSTAGE = 3;
    static constexpr int NW = 4;                     // consumer warps
    static constexpr int THREADS = (NW + 1) * 32;
    static constexpr int HW = kF32 ? 4 : 8;                      // query heads a warp holds
    static constexpr int PITCH = D + 4;                          // floats between the merge buffer's head rows
    static constexpr int OFF_O = NSTAGE * 2 * KV_BYTES;          // the CTA's merged output [8][D], then m, l [8]
    static constexpr int OFF_BAR = OFF_O + 8 * D * 4 + 64;
    static constexpr int SMEM = 1024 + OFF_BAR + 16 * NSTAGE + 4 * NSTAGE + 16;
    static_assert(NW * HW * (PITCH + 2) * 4 <= NSTAGE * 2 * KV_BYTES, "the warps' outputs fit the ring");
    static_assert(2 * NGRP <= 32, "one lane per box");
};

// The keys of one sequence's row, in groups of 8.
struct Keys {
    int ctx, lo, ns;         // visible: j < ctx and (j < ns or j >= lo)
    int sink_groups, shift;  // logical group of virtual group v: v, + shift from sink_groups on
    int groups;              // virtual groups
    __device__ __forceinline__ Keys(int ctx_, int window, int num_sinks, int unit) : ctx(ctx_) {
        const int rows = 8 * unit;
        lo = max(0, ctx - window);
        ns = min(num_sinks, lo);
        sink_groups = ns > 0 ? ((ns - 1) / rows + 1) * unit : 0;
        const int first = max(lo / rows * unit, sink_groups);
        shift = first - sink_groups;
        groups = ctx > 0 ? sink_groups + ((ctx - 1) / rows + 1) * unit - first : 0;
    }
    __device__ __forceinline__ int logical(int v) const { return v < sink_groups ? v : v + shift; }
    __device__ __forceinline__ bool sees(int j) const { return j < ctx && (j < ns || j >= lo); }
    __device__ __forceinline__ bool sees_group(int g) const {
        return 8 * g + 7 < ns || (8 * g >= lo && 8 * g + 7 < ctx);
    }
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <class T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, BF16>::value)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (a, b) rounded to a packed pair, and the remainders rounded to another.
__device__ __forceinline__ void split_pair(BF16, float a, float b, uint32_t &hi, uint32_t &lo) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    float x, y;
    widen_pair_bf16(hi, x, y);
    const __nv_bfloat162 l = __floats2bfloat162_rn(a - x, b - y);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}
__device__ __forceinline__ void split_pair(F16, float a, float b, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(a, b);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    float x, y;
    widen_pair_f16(hi, x, y);
    const __half2 l = __floats2half2_rn(a - x, b - y);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}
// (a, b) += (x, y) in one instruction
__device__ __forceinline__ void add_pair(float &a, float &b, float x, float y) {
    const float2 r = __fadd2_rn(make_float2(a, b), make_float2(x, y));
    a = r.x;
    b = r.y;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void sts_zero128(uint32_t addr) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
}

__device__ __forceinline__ void store_pair(void *out, pa_dtype dt, int64_t idx, float a, float b) {
    if (dt == PA_F32)
        store_out(static_cast<float *>(out) + idx, a, b);
    else if (dt == PA_F16)
        store_out(static_cast<__half *>(out) + idx, a, b);
    else
        store_out(static_cast<__nv_bfloat16 *>(out) + idx, a, b);
}

// What one consumer warp keeps of its keys, and how it takes a stage.  `first` is the
// stage's first virtual group, `valid` the bits of the stage's groups that were loaded.
// finish() leaves the warp's result in the merge buffer: red_o[HW][PITCH], red_m, red_l [HW]
// (unnormalised output, maximum in the log2 domain, sum).

template <class T, int D>
struct Consumer16 {
    using Sh = Shape<T, D>;
    uint32_t q[D / 16][2];  // Q^T as the 16 x 8 operand: head lane/4
    float o[D / 16][4];     // O^T: dims 16m + lane/4 (+8), heads 2(lane%4), +1
    float m[2], l[2];       // of those two heads (l: this lane's share)
    int warp, lane;

    __device__ __forceinline__ Consumer16(const Params &p, int warp_, int lane_, int s, int g)
        : warp(warp_), lane(lane_) {
        const int h = lane >> 2, d = (lane & 3) * 2;
        const typename T::storage *qp =
            static_cast<const typename T::storage *>(p.query) + ((int64_t)s * p.num_heads + g * p.group + h) * D + d;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            q[k][0] = h < p.group ? *reinterpret_cast<const uint32_t *>(qp + 16 * k) : 0u;
            q[k][1] = h < p.group ? *reinterpret_cast<const uint32_t *>(qp + 16 * k + 8) : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[k][i] = 0.f;
        }
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    // true when the stage was written by this warp
    __device__ __forceinline__ bool stage(const Params &p, const Keys &keys, uint32_t kbase, uint32_t vbase, int first,
                                          uint32_t valid) {
        bool wrote = false;
#pragma unroll
        for (int step = 0; step < Sh::NGRP / 8; ++step) {
            const int g0 = step * 8 + warp * 2;  // this warp's two groups of the stage
            if (!(valid >> g0 & 3u)) continue;
            wrote |= pair(p, keys, kbase + g0 * Sh::GROUP_BYTES, vbase + g0 * Sh::GROUP_BYTES, first + g0,
                          valid >> g0 & 3u);
        }
        return wrote;
    }

    __device__ __forceinline__ bool pair(const Params &p, const Keys &keys, uint32_t kb, uint32_t vb, int v,
                                         uint32_t valid) {
        const int mi = lane >> 3, r = lane & 7;
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t krow = kb + (mi & 1) * Sh::GROUP_BYTES + r * 128;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            const int c = 2 * k + (mi >> 1);
            uint32_t a[4];
            ldmatrix4(krow + (k / 4) * 1024 + (((c & 7) ^ r) << 4), a);
            mma16816<T>(k & 1 ? s1 : s, a, q[k][0], q[k][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] = (s[i] + s1[i]) * p.qk_scale_log2;
        const int l0 = keys.logical(v), l1 = keys.logical(v + 1);
        const bool whole = valid == 3u && keys.sees_group(l0) && keys.sees_group(l1);
        if (!whole) {
            const bool a = (valid & 1u) && keys.sees(8 * l0 + (lane >> 2));
            const bool b = (valid & 2u) && keys.sees(8 * l1 + (lane >> 2));
            s[0] = a ? s[0] : -INFINITY;
            s[1] = a ? s[1] : -INFINITY;
            s[2] = b ? s[2] : -INFINITY;
            s[3] = b ? s[3] : -INFINITY;
            // no NaN times zero: the rows of V that are not seen become zeros
            constexpr int VEC = D / 8;  // 16-byte pieces of a row
            for (int i = lane; i < 16 * VEC; i += 32) {
                const int row = i / VEC, c = i % VEC, gr = row >> 3;
                const bool seen = (valid >> gr & 1u) && keys.sees(8 * (gr ? l1 : l0) + (row & 7));
                if (!seen) sts_zero128(vb + gr * Sh::GROUP_BYTES + (c / 8) * 1024 + (row & 7) * 128 + (c % 8) * 16);
            }
            __syncwarp();
        }
        const bool grow = fmaxf(s[0], s[2]) > m[0] + kGrowLog2 || fmaxf(s[1], s[3]) > m[1] + kGrowLog2;
        if (__any_sync(kFullMask, grow)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float mx = fmaxf(s[i], s[i + 2]);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, off));
                const float mn = fmaxf(m[i], mx);
                const float a = m[i] == -INFINITY ? 0.f : fast_exp2(m[i] - mn);
                m[i] = mn;
                l[i] *= a;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    o[k][i] *= a;
                    o[k][i + 2] *= a;
                }
            }
        }
        const float m0 = (m[0] == -INFINITY ? 0.f : m[0]) - kLiftLog2<T>;
        const float m1 = (m[1] == -INFINITY ? 0.f : m[1]) - kLiftLog2<T>;
        const float p0 = fast_exp2(s[0] - m0), p1 = fast_exp2(s[1] - m1);
        const float p2 = fast_exp2(s[2] - m0), p3 = fast_exp2(s[3] - m1);
        l[0] += p0 + p2;
        l[1] += p1 + p3;
        uint32_t h0, h1, r0, r1;
        split_pair(T{}, p0, p1, h0, r0);
        split_pair(T{}, p2, p3, h1, r1);
        h0 = transpose8x8(h0);
        h1 = transpose8x8(h1);
        r0 = transpose8x8(r0);
        r1 = transpose8x8(r1);
        const uint32_t vrow = vb + (mi >> 1) * Sh::GROUP_BYTES + r * 128;
        // The tensor core cuts off, in every addition, what is below its accumulator's last bits: over
        // a long row behind one heavy key the light keys would fade.  So a step's products are
        // summed by themselves and added to O with rounding.
#pragma unroll
        for (int k = 0; k < D / 16; k += 2) {  // two at a time, so that one product hides the other's latency
            uint32_t a[2][4];
            float x[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = 2 * (k + u) + (mi & 1);
                ldmatrix4_trans(vrow + (k / 4) * 1024 + (((c & 7) ^ r) << 4), a[u]);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[u][i] = 0.f;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) mma16816<T>(x[u], a[u], h0, h1);
#pragma unroll
            for (int u = 0; u < 2; ++u) mma16816<T>(x[u], a[u], r0, r1);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                add_pair(o[k + u][0], o[k + u][1], x[u][0], x[u][1]);
                add_pair(o[k + u][2], o[k + u][3], x[u][2], x[u][3]);
            }
        }
        return !whole;
    }

    __device__ __forceinline__ void finish(float *red_o, float *red_m, float *red_l) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[i] += __shfl_xor_sync(kFullMask, l[i], off);
            const int h = 2 * (lane & 3) + i;
            if (lane < 4) {
                red_m[h] = m[i];
                red_l[h] = l[i];
            }
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                red_o[h * Sh::PITCH + 16 * k + (lane >> 2)] = o[k][i];
                red_o[h * Sh::PITCH + 16 * k + 8 + (lane >> 2)] = o[k][i + 2];
            }
        }
    }
};

// fp32: a warp takes a group of 8 keys at a time, lane = 8 * (key % 4) + part; a part owns the
// 16-byte pieces part, part + 8, .. of a row.  The partial scores of a lane (two keys, HW heads)
// are summed over the eight parts by halving: each exchange sends the half that the other lane
// keeps, so that a lane ends with one whole score, key u = part / 4 of head own, and takes one
// exponential (all lanes adding up all of their scores: 24 exchanges and 8 exponentials where
// this takes 7 and 1).
template <int D, int G>
struct Consumer32 {
    using Sh = Shape<F32, D>;
    static constexpr int HW = G < 4 ? G : 4;     // query heads of this warp
    static constexpr int QS = G / HW;            // warps that share a key, on different heads
    static constexpr int KW = Sh::NW / QS;       // warps over the groups of a stage
    static constexpr int NC = D / 32;            // 16-byte pieces per lane
    float2 q[HW][NC * 2], o[HW][NC * 2];
    float m, l;  // of head own (l: this lane's keys; lanes that differ in idle bits of part hold the same)
    int warp, lane;

    // part (below 4) whose lane holds head h
    static __device__ __forceinline__ int part_of(int h) { return HW == 4 ? h : HW == 2 ? 2 * h : 0; }

    __device__ __forceinline__ Consumer32(const Params &p, int warp_, int lane_, int s, int g)
        : m(-INFINITY), l(0.f), warp(warp_), lane(lane_) {
        const float *qp = static_cast<const float *>(p.query) +
                          ((int64_t)s * p.num_heads + g * G + (warp % QS) * HW) * D + (lane & 7) * 4;
#pragma unroll
        for (int h = 0; h < HW; ++h) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const float4 x = *reinterpret_cast<const float4 *>(qp + h * D + c * 32);
                q[h][2 * c] = make_float2(x.x * p.qk_scale_log2, x.y * p.qk_scale_log2);
                q[h][2 * c + 1] = make_float2(x.z * p.qk_scale_log2, x.w * p.qk_scale_log2);
                o[h][2 * c] = o[h][2 * c + 1] = make_float2(0.f, 0.f);
            }
        }
    }

    static __device__ __forceinline__ void row(uint32_t addr, float2 (&x)[NC * 2]) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const uint4 u = lds128(addr + c * 128);
            x[2 * c] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
            x[2 * c + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
        }
    }

    // v[0 .. N) summed over the lanes that differ in bit `off`; each keeps N / 2 of them, the
    // lanes with the bit set the upper ones (one value: both keep it).
    template <int N>
    __device__ __forceinline__ void halve(float (&v)[2 * HW], int off) {
        if constexpr (N == 1) {
            v[0] += __shfl_xor_sync(kFullMask, v[0], off);
        } else {
            const bool upper = (lane & off) != 0;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float send = upper ? v[i] : v[i + N / 2], keep = upper ? v[i + N / 2] : v[i];
                v[i] = keep + __shfl_xor_sync(kFullMask, send, off);
            }
        }
    }

    __device__ __forceinline__ bool stage(const Params &p, const Keys &keys, uint32_t kbase, uint32_t vbase, int first,
                                          uint32_t valid) {
#pragma unroll 1
        for (int gr = warp / QS; gr < Sh::NGRP; gr += KW) {
            if (!(valid >> gr & 1u)) continue;
            const int lg = keys.logical(first + gr), key = lane >> 3;  // keys `key` and `key` + 4 of the group
            const bool whole = keys.sees_group(lg);
            const uint32_t at = (gr * 8 + key) * D * 4 + (lane & 7) * 16;
            float v[2 * HW];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float2 x[NC * 2];
                row(kbase + at + u * 4 * D * 4, x);
#pragma unroll
                for (int h = 0; h < HW; ++h) {
                    float2 a = __fmul2_rn(q[h][0], x[0]);
#pragma unroll
                    for (int c = 1; c < NC * 2; ++c) a = __ffma2_rn(q[h][c], x[c], a);
                    v[u * HW + h] = a.x + a.y;
                }
            }
            halve<2 * HW>(v, 4);
            halve<HW>(v, 2);
            halve<(HW + 1) / 2>(v, 1);
            float s = v[0];
            if (!whole && !keys.sees(8 * lg + key + (lane & 4))) s = -INFINITY;
            if (__any_sync(kFullMask, s > m + kGrowLog2)) {
                float mx = s;
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, off));
                const float mn = fmaxf(m, mx);
                const float f = m == -INFINITY ? 0.f : fast_exp2(m - mn);
                m = mn;
                l *= f;
#pragma unroll
                for (int h = 0; h < HW; ++h) {
                    const float fh = __shfl_sync(kFullMask, f, part_of(h));
#pragma unroll
                    for (int c = 0; c < NC * 2; ++c) o[h][c] = __fmul2_rn(o[h][c], make_float2(fh, fh));
                }
            }
            // before the first seen key m is -inf: masked scores weigh nothing, NaN scores stay NaN
            const float w = fast_exp2(s - (m == -INFINITY ? 0.f : m));
            l += w;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float2 x[NC * 2];
                row(vbase + at + u * 4 * D * 4, x);
                if (!whole) {  // no NaN times zero
                    const bool seen = keys.sees(8 * lg + key + 4 * u);
#pragma unroll
                    for (int c = 0; c < NC * 2; ++c)
                        if (!seen) x[c] = make_float2(0.f, 0.f);
                }
#pragma unroll
                for (int h = 0; h < HW; ++h) {
                    const float wh = __shfl_sync(kFullMask, w, (lane & 24) + 4 * u + part_of(h));
#pragma unroll
                    for (int c = 0; c < NC * 2; ++c) o[h][c] = __ffma2_rn(make_float2(wh, wh), x[c], o[h][c]);
                }
            }
        }
        return false;
    }

    __device__ __forceinline__ void finish(float *red_o, float *red_m, float *red_l) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(kFullMask, l, off);
#pragma unroll
        for (int h = 0; h < HW; ++h) {
            if (lane == part_of(h)) {
                red_m[h] = m;
                red_l[h] = l;
            }
#pragma unroll
            for (int c = 0; c < NC * 2; ++c) {
                float2 v = o[h][c];
#pragma unroll
                for (int off = 8; off < 32; off <<= 1) {
                    v.x += __shfl_xor_sync(kFullMask, v.x, off);
                    v.y += __shfl_xor_sync(kFullMask, v.y, off);
                }
                if (lane < 8)
                    *reinterpret_cast<float2 *>(red_o + h * Sh::PITCH + (c / 2) * 32 + lane * 4 + (c % 2) * 2) = v;
            }
        }
    }
};

// grid = (cluster size, kv heads, sequences), cluster (cluster size, 1, 1).  G is the group
// size for fp32 caches; 0 (groups of 1, 2, 4 or 8) for 16-bit ones.
template <class T, int D, int G>
__global__ void __launch_bounds__(Shape<T, D>::THREADS, 2)
decode_window_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const Params p) {
    using Sh = Shape<T, D>;
    constexpr int NGRP = Sh::NGRP, NSTAGE = Sh::NSTAGE, KVB = Sh::KV_BYTES, NW = Sh::NW, HW = Sh::HW;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t ring = smem_u32(smem);
    float *sm_o = reinterpret_cast<float *>(smem + Sh::OFF_O);  // [8][D]
    float *sm_m = sm_o + 8 * D, *sm_l = sm_m + 8;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Sh::OFF_BAR);
    uint32_t *loaded = reinterpret_cast<uint32_t *>(bars + 2 * NSTAGE);  // per stage: bits of its valid groups
    int *abort_flag = reinterpret_cast<int *>(loaded + NSTAGE);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * NSTAGE;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < NSTAGE; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, NW);
        }
        fence_barrier_init();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    __syncthreads();
    pdl_wait_previous();
    pdl_launch_dependents();

    const int CS = (int)cluster_size(), rank = (int)cluster_rank();
    const int g = blockIdx.y, s = blockIdx.z;
    const int cap = min(p.max_blocks_per_seq * p.block_size, p.max_context_len);
    int ctx = p.context_lens[s];
    if (ctx < 0 || ctx > cap) {
        if (threadIdx.x == 0 && rank == 0 && g == 0) report(p.status, PA_DEVERR_CONTEXT);
        ctx = ctx < 0 ? 0 : cap;
    }
    const int unit = p.unit;
    const Keys keys(ctx, p.window, p.num_sinks, unit);
    const int64_t units = keys.groups / unit;
    const int v0 = (int)(units * rank / CS) * unit, v1 = (int)(units * (rank + 1) / CS) * unit;
    const int stages = (v1 - v0 + NGRP - 1) / NGRP;
    volatile int *abort_v = abort_flag;

    if (warp == NW) {
        // ============================================================ producer
        const int per_block = p.block_size / 8;
        const int32_t *bt = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
        const int per_stage = NGRP / unit;  // boxes of K, and of V
        const bool is_v = lane >= per_stage, mine = lane < 2 * per_stage;
        const int slot = (is_v ? lane - per_stage : lane) * unit;  // first group of the stage
        const uint32_t box_bytes = Sh::GROUP_BYTES * unit;
        const uint64_t policy = policy_evict_first();
        auto group_of = [&](int i) { return keys.logical(v0 + i * NGRP + slot); };
        auto block_id = [&](int i) {
            return mine && v0 + i * NGRP + slot < v1 ? bt[group_of(i) / per_block] : -1;
        };
        int next = block_id(0), i = 0;
        for (; i < stages; ++i) {
            const int id = next;
            next = block_id(i + 1);
            const int st = i % NSTAGE;
            int ok = 1;
            if (lane == 0) ok = !*abort_v && mbar_wait(empty0 + 8 * st, ((i / NSTAGE) & 1) ^ 1, p.status);
            if (!__shfl_sync(kFullMask, ok, 0)) {
                *abort_v = 1;
                break;
            }
            const bool in_range = mine && v0 + i * NGRP + slot < v1;
            const bool valid = in_range && id >= 0 && id < p.num_blocks;
            if (in_range && !valid) report(p.status, PA_DEVERR_BLOCK_ID);  // never dereferenced
            const unsigned boxes = __ballot_sync(kFullMask, valid);
            const uint32_t groups = __reduce_or_sync(kFullMask, valid && !is_v ? ((1u << unit) - 1u) << slot : 0u);
            if (lane == 0) {
                loaded[st] = groups;
                mbar_arrive_expect_tx(full0 + 8 * st, __popc(boxes) * box_bytes);
            }
            __syncwarp();
            if (valid) {
                const int at = id * per_block + group_of(i) % per_block;  // group of 8 rows of the pool
                const uint32_t dst = ring + st * 2 * KVB + (is_v ? KVB : 0) + slot * Sh::GROUP_BYTES;
                const CUtensorMap *map = is_v ? &vmap : &kmap;
                if constexpr (Sh::kF32)
                    tma_load_3d(dst, map, 0, g, at * 8, full0 + 8 * st, policy);
                else
                    tma_load_5d(dst, map, 0, 0, 0, at, g, full0 + 8 * st, policy);
            }
            __syncwarp();
        }
        // every box has landed before the warp leaves, whether or not a wait gave up
        bool landed = true;
        for (int j = max(0, i - NSTAGE); j < i && landed; ++j)
            landed = mbar_wait(full0 + 8 * (j % NSTAGE), (j / NSTAGE) & 1, p.status);
    } else {
        // ============================================================ consumers
        typename std::conditional<Sh::kF32, Consumer32<D, G ? G : 1>, Consumer16<T, D>>::type work(p, warp, lane, s, g);
        for (int i = 0; i < stages; ++i) {
            const int st = i % NSTAGE;
            const bool ok = !*abort_v && mbar_wait(full0 + 8 * st, (i / NSTAGE) & 1, p.status);
            if (!__all_sync(kFullMask, ok)) {
                *abort_v = 1;
                break;
            }
            const uint32_t kbase = ring + st * 2 * KVB;
            const bool wrote = work.stage(p, keys, kbase, kbase + KVB, v0 + i * NGRP, loaded[st]);
            // rows zeroed here are written by TMA (the async proxy) once the stage is free again
            if (wrote) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * st);
        }
        // ---- the warps' results into the ring (every box of it has landed and been read)
        __syncwarp();  // the barriers are of the aligned form
        named_barrier(1, NW * 32);
        float *red_m = reinterpret_cast<float *>(smem) + NW * HW * Sh::PITCH, *red_l = red_m + NW * HW;
        float *red_o = reinterpret_cast<float *>(smem);
        work.finish(red_o + warp * HW * Sh::PITCH, red_m + warp * HW, red_l + warp * HW);
        __syncwarp();
        named_barrier(1, NW * 32);
        // ---- joined over the warps: head h is row h % HW of the warps w with w % QS == h / HW
        const int heads = G ? G : p.group;
        const int qs = Sh::kF32 && heads > HW ? heads / HW : 1;
        for (int i = threadIdx.x; i < heads * (D / 2); i += NW * 32) {
            const int h = i / (D / 2), d = i % (D / 2) * 2;
            const int w0 = qs > 1 ? h / HW : 0, hr = qs > 1 ? h % HW : h;
            float M = -INFINITY, L = 0.f;
            for (int w = w0; w < NW; w += qs) M = fmaxf(M, red_m[w * HW + hr]);
            float2 acc = make_float2(0.f, 0.f);
            for (int w = w0; w < NW; w += qs) {
                const float mw = red_m[w * HW + hr];
                const float f = mw == -INFINITY ? 0.f : fast_exp2(mw - M);
                L = fmaf(red_l[w * HW + hr], f, L);
                const float2 x = *reinterpret_cast<const float2 *>(red_o + (w * HW + hr) * Sh::PITCH + d);
                acc.x = fmaf(x.x, f, acc.x);
                acc.y = fmaf(x.y, f, acc.y);
            }
            if (CS == 1) {
                const float inv = L > 0.f ? 1.f / L : 0.f;
                store_pair(p.out, p.out_dtype, ((int64_t)s * p.num_heads + g * heads + h) * D + d, acc.x * inv,
                           acc.y * inv);
            } else {
                *reinterpret_cast<float2 *>(sm_o + h * D + d) = acc;
                if (d == 0) {
                    sm_m[h] = M;
                    sm_l[h] = L;
                }
            }
        }
    }
    if (CS == 1) return;
    // ---- joined over the cluster: each CTA writes its share of the row
    cluster_sync();
    const int heads = G ? G : p.group;
    const int total = heads * (D / 2), i0 = total * rank / CS, i1 = total * (rank + 1) / CS;
    const uint32_t a_o = smem_u32(sm_o), a_m = smem_u32(sm_m), a_l = smem_u32(sm_l);
    for (int i = i0 + (int)threadIdx.x; i < i1; i += Sh::THREADS) {
        const int h = i / (D / 2), d = i % (D / 2) * 2;
        // eight CTAs' loads in flight together (a remote load takes a few hundred clocks)
        float M = -INFINITY, L = 0.f;
        float2 acc = make_float2(0.f, 0.f);
        for (int r0 = 0; r0 < CS; r0 += 8) {
            float mr[8], lr[8];
            float2 xr[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int from = min(r0 + r, CS - 1);
                mr[r] = ld_cluster(map_rank(a_m + 4 * h, from));
                lr[r] = ld_cluster(map_rank(a_l + 4 * h, from));
                xr[r] = ld_cluster2(map_rank(a_o + 4 * (h * D + d), from));
            }
            float top = M;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                if (r0 + r >= CS) mr[r] = -INFINITY;
                top = fmaxf(top, mr[r]);
            }
            const float keep = M == -INFINITY ? 0.f : fast_exp2(M - top);
            M = top;
            L *= keep;
            acc.x *= keep;
            acc.y *= keep;
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float f = mr[r] == -INFINITY ? 0.f : fast_exp2(mr[r] - M);
                L = fmaf(lr[r], f, L);
                acc.x = fmaf(xr[r].x, f, acc.x);
                acc.y = fmaf(xr[r].y, f, acc.y);
            }
        }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        store_pair(p.out, p.out_dtype, ((int64_t)s * p.num_heads + g * heads + h) * D + d, acc.x * inv, acc.y * inv);
    }
    cluster_sync();  // nobody leaves while its shared memory is read
}

// One warp per (sequence, kv head): block b takes pair b (sequence-major).  The ring's `depth`
// steps hold two groups of K and two of V each; the warp refills a step when it has read it.
template <class T, int D>
__global__ void __launch_bounds__(32)
decode_window_warp_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                          const Params p, int depth) {
    using Sh = Shape<T, D>;
    constexpr int GB = Sh::GROUP_BYTES, STEP = 4 * GB;
    static_assert(Sh::HW * (Sh::PITCH + 2) * 4 <= STEP, "the result fits one step");
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t ring = smem_u32(smem), full0 = ring + depth * STEP;
    const int lane = threadIdx.x;
    if (lane == 0) {
        for (int i = 0; i < depth; ++i) mbar_init(full0 + 8 * i, 1);
        fence_barrier_init();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    __syncwarp();
    pdl_wait_previous();
    pdl_launch_dependents();

    const int s = blockIdx.x / (unsigned)p.num_kv_heads, g = blockIdx.x % (unsigned)p.num_kv_heads;
    const int cap = min(p.max_blocks_per_seq * p.block_size, p.max_context_len);
    int ctx = p.context_lens[s];
    if (ctx < 0 || ctx > cap) {
        if (lane == 0 && g == 0) report(p.status, PA_DEVERR_CONTEXT);
        ctx = ctx < 0 ? 0 : cap;
    }
    const int unit = p.unit;  // 1 or 2
    const Keys keys(ctx, p.window, p.num_sinks, unit);
    const int steps = (keys.groups + 1) / 2, per_block = p.block_size / 8, k_boxes = 2 / unit;
    const int32_t *bt = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
    auto block_id = [&](int v) { return v < keys.groups ? bt[keys.logical(v) / per_block] : -1; };
    // block ids of 32 groups, one per lane, and of the next 32
    int ids = block_id(lane), ids_next = block_id(32 + lane);
    Consumer16<T, D> work(p, 0, lane, s, g);
    const uint64_t policy = policy_evict_first();
    uint32_t loaded = 0;  // two bits per step of the ring: its valid groups
    auto issue = [&](int t, int slot) {
        if (t > 0 && t % 16 == 0) {
            ids = ids_next;
            ids_next = block_id(2 * t + 32 + lane);
        }
        const int v = 2 * t + (unit == 1 ? lane & 1 : 0), id = __shfl_sync(kFullMask, ids, v & 31);
        const bool in_range = lane < 2 * k_boxes && v < keys.groups;
        const bool valid = in_range && id >= 0 && id < p.num_blocks;
        if (in_range && !valid) report(p.status, PA_DEVERR_BLOCK_ID);  // never dereferenced
        const unsigned boxes = __ballot_sync(kFullMask, valid);
        if (lane == 0) mbar_arrive_expect_tx(full0 + 8 * slot, __popc(boxes) * GB * unit);
        __syncwarp();
        if (valid) {
            const int at = id * per_block + (keys.logical(v) & (per_block - 1));  // group of 8 rows of the pool
            tma_load_5d(ring + slot * STEP + lane * GB * unit, lane < k_boxes ? &kmap : &vmap, 0, 0, 0, at, g,
                        full0 + 8 * slot, policy);
        }
        __syncwarp();
        loaded = (loaded & ~(3u << 2 * slot)) | (unit == 1 ? boxes & 3u : boxes & 1u ? 3u : 0u) << 2 * slot;
    };
    for (int t = 0; t < depth && t < steps; ++t) issue(t, t);
    int slot = 0, phase = 0, t = 0;
    auto advance = [&] {
        if (++slot == depth) {
            slot = 0;
            phase ^= 1;
        }
    };
    for (; t < steps; ++t, advance()) {
        if (!__all_sync(kFullMask, mbar_wait(full0 + 8 * slot, phase, p.status))) break;
        const uint32_t kb = ring + slot * STEP, valid = loaded >> 2 * slot & 3u;
        const bool wrote = valid && work.pair(p, keys, kb, kb + 2 * GB, 2 * t, valid);
        if (t + depth < steps) {
            // rows zeroed here are written by TMA (the async proxy) next
            if (wrote) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            issue(t + depth, slot);
        }
    }
    // if a wait gave up: the boxes under way land before the CTA leaves
    for (const int end = min(t + depth, steps); t < end; ++t, advance())
        if (!__all_sync(kFullMask, mbar_wait(full0 + 8 * slot, phase, p.status))) break;
    // the heads' rows through shared memory, so that the stores are contiguous
    __syncwarp();
    float *red_o = reinterpret_cast<float *>(smem), *red_m = red_o + Sh::HW * Sh::PITCH, *red_l = red_m + Sh::HW;
    work.finish(red_o, red_m, red_l);
    __syncwarp();
    for (int i = lane; i < p.group * (D / 2); i += 32) {
        const int h = i / (D / 2), d = i % (D / 2) * 2;
        const float L = red_l[h], inv = L > 0.f ? 1.f / L : 0.f;
        const float2 x = *reinterpret_cast<const float2 *>(red_o + h * Sh::PITCH + d);
        store_pair(p.out, p.out_dtype, ((int64_t)s * p.num_heads + g * p.group + h) * D + d, x.x * inv, x.y * inv);
    }
}

template <class T, int D, int G>
int launch_typed(const Params &p, int cluster, int num_seqs, const CUtensorMap &km, const CUtensorMap &vm,
                 cudaStream_t st) {
    using Sh = Shape<T, D>;
    static std::atomic<int> smem_ready[kMaxDevices];  // per device: shared-memory limit raised
    return launch_pdl_cluster(decode_window_kernel<T, D, G>, smem_ready, dim3(cluster, p.num_kv_heads, num_seqs),
                              dim3(Sh::THREADS), Sh::SMEM, cluster, st, km, vm, p) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

// 16-bit caches: clusters, or (`warps` > 0) a warp per pair, so many of them on an SM; at most 8,
// which leaves a ring three steps or more.
template <class T, int D>
int launch_16(const Params &p, int cluster, int num_seqs, int warps, const CUtensorMap &km, const CUtensorMap &vm,
              cudaStream_t st) {
    constexpr int STEP = 4 * Shape<T, D>::GROUP_BYTES, kMost = 16, kRest = 1024 + 8 * kMost;
    static_assert((228 * 1024 / 8 - 1024 - kRest) / STEP >= 3, "eight warps fit an SM");
    // A device's first call loads both kernels, with the shared memory that any call asks for: a
    // later one may be captured, whichever kernel it takes.
    static std::atomic<int> clusters_ready[kMaxDevices], warps_ready[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PA_ERR_CUDA;
    if (dev < 0 || dev >= kMaxDevices || !warps_ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(decode_window_kernel<T, D, 0>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Shape<T, D>::SMEM) != cudaSuccess ||
            cudaFuncSetAttribute(decode_window_warp_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kMost * STEP + kRest) != cudaSuccess)
            return PA_ERR_CUDA;
        if (dev >= 0 && dev < kMaxDevices) warps_ready[dev].store(1, std::memory_order_release);
    }
    cudaError_t e;
    if (warps > 0) {
        const int depth = std::min(kMost, (228 * 1024 / warps - 1024 - kRest) / STEP);  // 1 KB per CTA is the system's
        e = launch_pdl_cluster(decode_window_warp_kernel<T, D>, warps_ready, dim3(p.num_kv_heads * num_seqs), dim3(32),
                               depth * STEP + kRest, 1, st, km, vm, p, depth);
    } else {
        e = launch_pdl_cluster(decode_window_kernel<T, D, 0>, clusters_ready, dim3(cluster, p.num_kv_heads, num_seqs),
                               dim3(Shape<T, D>::THREADS), Shape<T, D>::SMEM, cluster, st, km, vm, p);
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int D>
int launch_f32(const Params &p, int cluster, int num_seqs, const CUtensorMap &km, const CUtensorMap &vm,
               cudaStream_t st) {
    switch (p.group) {
        case 1: return launch_typed<F32, D, 1>(p, cluster, num_seqs, km, vm, st);
        case 2: return launch_typed<F32, D, 2>(p, cluster, num_seqs, km, vm, st);
        case 4: return launch_typed<F32, D, 4>(p, cluster, num_seqs, km, vm, st);
        case 8: return launch_typed<F32, D, 8>(p, cluster, num_seqs, km, vm, st);
        default: return PA_ERR_UNSUPPORTED;
    }
}

}  // namespace

int launch_decode_window(const DecodeArgs &a) {
    Params p{};
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.query = a.query;
    p.block_tables = a.block_tables;
    p.context_lens = a.context_lens;
    p.max_blocks_per_seq = a.max_blocks_per_seq;
    p.max_context_len = a.max_context_len;
    p.num_heads = a.num_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.group = a.num_heads / a.num_kv_heads;
    p.block_size = a.block_size;
    p.num_blocks = a.num_blocks;
    p.window = a.window;
    p.num_sinks = a.num_sinks;
    p.qk_scale_log2 = a.scale * kLog2e;
    p.status = a.status;
    const int64_t rows = (int64_t)a.num_blocks * a.block_size;
    if (rows <= 0 || rows > INT32_MAX) return PA_ERR_INVALID_ARG;
    // The cluster size: the CTAs of one full wave, but none with less than one stage of keys
    // (two past eight CTAs).  A CTA past the first wave costs more than its shorter run of keys
    // gives back, and clusters start slowly: 256 (sequence, kv head) pairs of 1028 keys took 23,
    // 29, 40 and 61 us in clusters of 1, 2, 4 and 8; 61 pairs of 790 keys 11.8, 8.6, 7.0 and
    // 11.0 us; 8 pairs of 516 keys 11.1, 8.2, 6.5, 5.4 and (16) 5.7 us, of 4100 keys (8) 9.5 and
    // (16) 7.7 us (bf16).
    const int sms = std::max(1, device_sm_count());
    const int64_t slots = 2 * sms;  // resident CTAs
    const int64_t most = std::min<int64_t>(a.max_context_len, (int64_t)a.window + a.num_sinks);  // keys of a row
    const int64_t stage_keys = 16384 / (a.head_dim * (a.kv_dtype == PA_F32 ? 4 : 2));
    const int64_t pairs = (int64_t)a.num_seqs * a.num_kv_heads;
    // What is resident in clusters of a size, as the parts of the chip do not divide evenly: of
    // 304 CTAs 296 in fours, 288 in eights, 224 in sixteens.  One cluster more is a second wave
    // (76 pairs of 333 fp32 keys 6.0 us in twos, 9.1 in fours; 16 pairs of 2004 keys 7.4 in eights,
    // 11.6 in sixteens).
    auto fit = [&](int size) { return slots * (size <= 2 ? 64 : size == 4 ? 63 : size == 8 ? 61 : 48) / 64; };
    int cluster = 1;
    while (cluster < 16 && pairs * cluster * 2 <= fit(cluster * 2) &&
           most > stage_keys * cluster * (cluster < 8 ? 1 : 2))
        cluster *= 2;
    // A second wave that few pairs start takes as long as the first: two CTAs per pair halve it (312
    // to 384 pairs of 4096 keys 136 to 141 -> 122 to 128 us; 448 pairs are equal, of 2048 keys 77 ->
    // 82).
    if (pairs > slots && pairs <= slots * 4 / 3 && most >= 16 * stage_keys) cluster = 2;
    // A box of a whole block where one warp's issue of the boxes bounds a CTA (about 70 clocks
    // each: 8 pairs of 4100 keys 9.0 -> 7.7 us) or where the rows past the borders that it brings
    // along are few (1024 pairs of 4112 keys in blocks of 16, 333 -> 318 us; but 256 pairs of 1028
    // keys in blocks of 32, 23.3 -> 24.0 us).
    p.unit = cluster > 1 || most >= 64 * (int64_t)a.block_size ? a.block_size / 8 : 1;
    // A warp per pair where the clusters would be single CTAs in more than one wave, of rows of
    // about a thousand keys at most: 1024 pairs of 132, 516 and 1028 keys 29.8 -> 16.4, 59.7 -> 47.3
    // and 95.5 -> 87.7 us, 320 pairs of 516 keys 27.2 -> 24.6 us.  Of 2052 keys the two are equal,
    // of 4112 the clusters faster (318 and 332 us), and rows of unequal length leave the longest
    // to one warp: contexts of 10 to 1000 keys 52.6 -> 50.8, of 10 to 2000 90.8 -> 99 us.  Boxes of
    // 16 keys where the rows are long for the warps on an SM (320 pairs of 516 keys 26.3 -> 24.6,
    // but 1024 pairs of 132 keys 16.4 -> 17.9 us).
    // A step of 16 keys takes a warp 0.6 us at least, so at head dimension 64 (half the bytes) a few
    // warps per SM fall behind: 400 pairs of 260 keys 13.5 and 14.0 us (clusters), of 1004 keys 40.3
    // and 31.4; 800 pairs 44.3 and 47.1.
    const int per_sm = (int)std::min<int64_t>(8, (pairs + sms - 1) / sms);
    const bool by_warp = a.kv_dtype != PA_F32 && pairs > slots && pairs <= INT32_MAX &&
                         most <= (per_sm * a.head_dim >= 320 ? 1152 : 384);
    const int warps = by_warp ? per_sm : 0;
    if (by_warp) p.unit = a.block_size >= 16 && most >= a.head_dim * per_sm ? 2 : 1;
    CUtensorMap km, vm;
    for (int i = 0; i < 2; ++i) {
        CUtensorMap *m = i ? &vm : &km;
        const void *base = i ? a.value_cache : a.key_cache;
        const int rc = a.kv_dtype == PA_F32
                           ? make_kv_tensor_map(m, base, a.kv_dtype, a.head_dim, a.num_kv_heads, rows, 1, 8 * p.unit)
                           : make_kv_block_map(m, base, a.kv_dtype, a.head_dim, a.num_kv_heads, rows, 8 * p.unit);
        if (rc != PA_OK) return rc;
    }
    switch (a.kv_dtype) {
        case PA_F32:
            return a.head_dim == 64 ? launch_f32<64>(p, cluster, a.num_seqs, km, vm, a.stream)
                                    : launch_f32<128>(p, cluster, a.num_seqs, km, vm, a.stream);
        case PA_F16:
            return a.head_dim == 64 ? launch_16<F16, 64>(p, cluster, a.num_seqs, warps, km, vm, a.stream)
                                    : launch_16<F16, 128>(p, cluster, a.num_seqs, warps, km, vm, a.stream);
        case PA_BF16:
            return a.head_dim == 64 ? launch_16<BF16, 64>(p, cluster, a.num_seqs, warps, km, vm, a.stream)
                                    : launch_16<BF16, 128>(p, cluster, a.num_seqs, warps, km, vm, a.stream);
    }
    return PA_ERR_UNSUPPORTED;
}

}  // namespace pa
