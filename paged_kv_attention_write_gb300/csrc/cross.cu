// cross.cu -- attention of packed query rows over a sequence's whole paged context, each row
// within its own range of keys (include/pa.h: pa_cross_attention).
//
// A warp per (row, query head): each lane holds D/32 elements of the query and the output, the
// keys are taken one after another with a running maximum and sum.
#include "cross.cuh"

namespace pa {
namespace {

struct Params {
    PrefillArgs a;
    const int32_t *key_ranges;
};

template <class T>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    if constexpr (T::kBytes == 4) return static_cast<const float *>(p)[i];
    else return (float)static_cast<const typename T::storage *>(p)[i];
}

template <class T, int D>
__global__ void __launch_bounds__(128) cross_kernel(const Params c) {
    const PrefillArgs &p = c.a;
    pdl_wait_previous();
    pdl_launch_dependents();
    const int lane = threadIdx.x % 32;
    const int64_t item = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (item >= (int64_t)p.num_tokens * p.num_heads) return;
    const int row = (int)(item / p.num_heads), h = (int)(item % p.num_heads);
    int s = row;
    if (p.query_start_loc) {  // the sequence whose rows hold this one
        s = -1;
        for (int i = 0; i < p.num_seqs && s < 0; ++i) {
            const int q0 = p.query_start_loc[i], q1 = p.query_start_loc[i + 1];
            if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || q1 - q0 > p.max_query_len) {
                if (lane == 0) report(p.status, PA_DEVERR_QUERY);
            } else if (row >= q0 && row < q1) {
                s = i;
            }
        }
        if (s < 0) return;
    }
    const int cap = min(p.max_blocks_per_seq * p.block_size, p.max_context_len);
    int ctx = p.context_lens[s];
    if (ctx < 0 || ctx > cap) {
        if (lane == 0) report(p.status, PA_DEVERR_CONTEXT);
        ctx = ctx < 0 ? 0 : cap;
    }
    int begin = 0, end = ctx;
    if (c.key_ranges) {
        begin = max(0, c.key_ranges[2 * (int64_t)row]);
        end = min(ctx, c.key_ranges[2 * (int64_t)row + 1]);
    }
    constexpr int N = D / 32;
    float q[N], o[N], m = -INFINITY, l = 0.f;
    const int64_t at = ((int64_t)row * p.num_heads + h) * D + lane;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        q[i] = load1<T>(p.query, at + 32 * i) * p.scale;
        o[i] = 0.f;
    }
    const int g = h / (p.num_heads / p.num_kv_heads);
    for (int j = begin; j < end; ++j) {
        const int id = p.block_tables[(int64_t)s * p.max_blocks_per_seq + j / p.block_size];
        if (id < 0 || id >= p.num_blocks) {
            if (lane == 0) report(p.status, PA_DEVERR_BLOCK_ID);
            continue;
        }
        const int64_t kv = (((int64_t)id * p.block_size + j % p.block_size) * p.num_kv_heads + g) * D + lane;
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) x = fmaf(q[i], load1<T>(p.key_cache, kv + 32 * i), x);
#pragma unroll
        for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(kFullMask, x, off);
        if (x > m) {
            const float f = m == -INFINITY ? 0.f : fast_exp2((m - x) * kLog2e);
            m = x;
            l *= f;
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] *= f;
        }
        const float w = fast_exp2((x - (m == -INFINITY ? 0.f : m)) * kLog2e);
        l += w;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(w, load1<T>(p.value_cache, kv + 32 * i), o[i]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (p.out_dtype == PA_F32) static_cast<float *>(p.out)[at + 32 * i] = o[i] * inv;
        else if (p.out_dtype == PA_F16) static_cast<__half *>(p.out)[at + 32 * i] = __float2half(o[i] * inv);
        else static_cast<__nv_bfloat16 *>(p.out)[at + 32 * i] = __float2bfloat16(o[i] * inv);
    }
}

template <class T>
int launch_typed(const Params &p) {
    const int64_t ctas = ((int64_t)p.a.num_tokens * p.a.num_heads + 3) / 4;
    if (ctas > INT32_MAX) return PA_ERR_INVALID_ARG;
    const cudaError_t e = p.a.head_dim == 64
                              ? launch_pdl(cross_kernel<T, 64>, dim3((unsigned)ctas), dim3(128), 0, p.a.stream, p)
                              : launch_pdl(cross_kernel<T, 128>, dim3((unsigned)ctas), dim3(128), 0, p.a.stream, p);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

int launch_cross(const CrossArgs &c) {
    const int G = c.a.num_heads / c.a.num_kv_heads;
    if (c.a.kv_dtype != PA_F32 && c.a.query_start_loc && (int64_t)c.a.max_query_len * G > 8) return launch_cross_chunk(c);
    const Params p{c.a, c.key_ranges};
    switch (c.a.kv_dtype) {
        case PA_F32: return launch_typed<F32>(p);
        case PA_F16: return launch_typed<F16>(p);
        case PA_BF16: return launch_typed<BF16>(p);
    }
    return PA_ERR_UNSUPPORTED;
}

}  // namespace pa
