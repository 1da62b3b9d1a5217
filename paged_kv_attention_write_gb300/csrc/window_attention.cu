// window_attention.cu -- sliding-window attention with sinks over the paged cache.
//
// out[row][h] = sum_j softmax_j(scale q.k_j) v_j over the keys j <= p with j > p - window or
// j < num_sinks, p the row's position.  One CTA per (query row, kv head): its warps take the
// visible keys in turn, every lane owns D/32 elements of the head dimension, and the warps'
// running maxima, sums and outputs are merged in shared memory (online softmax in the log2
// domain, fp32).
#include "common.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;

struct WindowParams {
    void *out;
    pa_dtype out_dtype;
    const void *query, *key_cache, *value_cache;
    const int32_t *query_start_loc;  // null: one row per sequence
    const int32_t *block_tables, *context_lens;
    int max_blocks_per_seq, max_context_len, num_seqs, num_tokens, num_heads, num_kv_heads, block_size, num_blocks;
    int window, num_sinks;
    float qk_scale_log2;
    int32_t *status;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ void store_one(void *out, pa_dtype dt, int64_t i, float v) {
    if (dt == PA_F32)
        static_cast<float *>(out)[i] = v;
    else if (dt == PA_F16)
        static_cast<__half *>(out)[i] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16_rn(v);
}

// grid = (query rows, kv heads)
template <class T, int D, int G>
__global__ void __launch_bounds__(kWarps * 32) window_row_kernel(const WindowParams p) {
    using ST = typename T::storage;
    constexpr int E = D / 32;
    __shared__ float red_o[kWarps][G][D], red_m[kWarps][G], red_l[kWarps][G];
    pdl_wait_previous();
    pdl_launch_dependents();
    const int row = blockIdx.x, g = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int cap = min(p.max_blocks_per_seq * p.block_size, p.max_context_len);
    const bool first = threadIdx.x == 0 && g == 0;
    int s = row, pos;
    if (!p.query_start_loc) {
        int C = p.context_lens[s];
        if (C < 0 || C > cap) {
            if (first) report(p.status, PA_DEVERR_CONTEXT);
            C = C < 0 ? 0 : cap;
        }
        pos = C - 1;
    } else {
        // the sequence whose rows hold this one (the starts may be invalid: every index is checked)
        for (s = 0; s < p.num_seqs; ++s)
            if (row >= p.query_start_loc[s] && row < p.query_start_loc[s + 1]) break;
        if (s == p.num_seqs) return;
        const int q0 = p.query_start_loc[s], Lq = p.query_start_loc[s + 1] - q0;
        int C = p.context_lens[s];
        if (q0 < 0 || (int64_t)q0 + Lq > p.num_tokens) {
            if (first) report(p.status, PA_DEVERR_QUERY);
            return;
        }
        if (C > cap) {
            if (first) report(p.status, PA_DEVERR_CONTEXT);
            C = cap;
        }
        if (Lq > C) {
            if (first) report(p.status, PA_DEVERR_QUERY);
            return;
        }
        pos = C - Lq + (row - q0);
    }
    const int lo = max(0, pos - p.window + 1);     // first key of the window
    const int ns = min(p.num_sinks, lo);           // sinks in front of it
    const int n = pos < 0 ? 0 : ns + (pos + 1 - lo);
    const ST *kc = static_cast<const ST *>(p.key_cache), *vc = static_cast<const ST *>(p.value_cache);
    const int32_t *bt = p.block_tables + (int64_t)s * p.max_blocks_per_seq;
    float q[G][E], acc[G][E], m[G], l[G];
    const int64_t q_base = ((int64_t)row * p.num_heads + g * G) * D + lane * E;
#pragma unroll
    for (int h = 0; h < G; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            q[h][e] = to_float(static_cast<const ST *>(p.query)[q_base + h * D + e]) * p.qk_scale_log2;
            acc[h][e] = 0.f;
        }
    }
    for (int i = warp; i < n; i += kWarps) {
        const int j = i < ns ? i : lo + (i - ns);
        const int id = bt[j / p.block_size];
        if (id < 0 || id >= p.num_blocks) {  // never dereferenced
            if (lane == 0) report(p.status, PA_DEVERR_BLOCK_ID);
            continue;
        }
        const int64_t at = (((int64_t)id * p.block_size + j % p.block_size) * p.num_kv_heads + g) * D + lane * E;
        float k[E], v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            k[e] = to_float(kc[at + e]);
            v[e] = to_float(vc[at + e]);
        }
#pragma unroll
        for (int h = 0; h < G; ++h) {
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) x = fmaf(q[h][e], k[e], x);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(kFullMask, x, o);
            const float mn = fmaxf(m[h], x), a = fast_exp2(m[h] - mn), w = fast_exp2(x - mn);
            m[h] = mn;
            l[h] = fmaf(l[h], a, w);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[h][e] = fmaf(w, v[e], acc[h][e] * a);
        }
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
        if (lane == 0) {
            red_m[warp][h] = m[h];
            red_l[warp][h] = l[h];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) red_o[warp][h][lane * E + e] = acc[h][e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * D; i += kWarps * 32) {
        const int h = i / D, d = i % D;
        float M = -INFINITY, L = 0.f, o = 0.f;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_m[w][h]);
        for (int w = 0; w < kWarps; ++w) {
            const float f = red_m[w][h] == -INFINITY ? 0.f : fast_exp2(red_m[w][h] - M);
            L = fmaf(red_l[w][h], f, L);
            o = fmaf(red_o[w][h][d], f, o);
        }
        store_one(p.out, p.out_dtype, ((int64_t)row * p.num_heads + g * G + h) * D + d, L > 0.f ? o / L : 0.f);
    }
}

template <class T, int D>
int dispatch_g(const WindowParams &p, cudaStream_t st) {
    const dim3 grid(p.num_tokens, p.num_kv_heads), block(kWarps * 32);
    cudaError_t e;
    switch (p.num_heads / p.num_kv_heads) {
        case 1: e = launch_pdl(window_row_kernel<T, D, 1>, grid, block, 0, st, p); break;
        case 2: e = launch_pdl(window_row_kernel<T, D, 2>, grid, block, 0, st, p); break;
        case 4: e = launch_pdl(window_row_kernel<T, D, 4>, grid, block, 0, st, p); break;
        case 8: e = launch_pdl(window_row_kernel<T, D, 8>, grid, block, 0, st, p); break;
        default: return PA_ERR_UNSUPPORTED;
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

int dispatch(const WindowParams &p, pa_dtype dt, int D, cudaStream_t st) {
    switch (dt) {
        case PA_F32: return D == 64 ? dispatch_g<F32, 64>(p, st) : dispatch_g<F32, 128>(p, st);
        case PA_F16: return D == 64 ? dispatch_g<F16, 64>(p, st) : dispatch_g<F16, 128>(p, st);
        case PA_BF16: return D == 64 ? dispatch_g<BF16, 64>(p, st) : dispatch_g<BF16, 128>(p, st);
    }
    return PA_ERR_UNSUPPORTED;
}

template <class A>
WindowParams params(const A &a) {
    WindowParams p{};
    p.out = a.out;
    p.out_dtype = a.out_dtype;
    p.query = a.query;
    p.key_cache = a.key_cache;
    p.value_cache = a.value_cache;
    p.block_tables = a.block_tables;
    p.context_lens = a.context_lens;
    p.max_blocks_per_seq = a.max_blocks_per_seq;
    p.max_context_len = a.max_context_len;
    p.num_seqs = a.num_seqs;
    p.num_heads = a.num_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.block_size = a.block_size;
    p.num_blocks = a.num_blocks;
    p.window = a.window;
    p.num_sinks = a.num_sinks;
    p.qk_scale_log2 = a.scale * kLog2e;
    p.status = a.status;
    return p;
}

}  // namespace

int launch_prefill_window(const PrefillArgs &a) {
    WindowParams p = params(a);
    p.num_tokens = a.num_tokens;
    p.query_start_loc = a.query_start_loc;
    return dispatch(p, a.kv_dtype, a.head_dim, a.stream);
}

}  // namespace pa
