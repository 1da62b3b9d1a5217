// rope_axes.cu -- rotary positions with several axes, for a step's queries and keys, fused
// with the cache write.
//
// Pair i of token t turns by positions[pair_axis[i]][t] * freqs[i].  One CTA per token: the
// (cos, sin) of its pairs go to shared memory once and serve all of its heads; the threads
// then rotate the query and key elements pair by pair and copy the values.
#include "common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxPairs = 64;  // rope_dim <= head_dim <= 128

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float v, float &x) { x = v; }
__device__ __forceinline__ void from_float(float v, __half &x) { x = __float2half_rn(v); }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16 &x) { x = __float2bfloat16_rn(v); }

template <class ST>
__device__ void rotate_row(ST *dst, const ST *src, const float2 *cs, int heads, int D, int half, bool halves) {
    for (int i = threadIdx.x; i < heads * (D / 2); i += kThreads) {
        const int h = i / (D / 2), pair = i % (D / 2);
        int a, b;
        if (pair < half) {
            a = halves ? pair : 2 * pair;
            b = halves ? pair + half : 2 * pair + 1;
        } else {
            a = 2 * pair;
            b = 2 * pair + 1;
        }
        const ST xs = src[h * D + a], ys = src[h * D + b];
        if (pair < half) {
            const float2 c = cs[pair];
            const float x = to_float(xs), y = to_float(ys);
            from_float(x * c.x - y * c.y, dst[h * D + a]);
            from_float(x * c.y + y * c.x, dst[h * D + b]);
        } else {
            dst[h * D + a] = xs;
            dst[h * D + b] = ys;
        }
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) rope_axes_kernel(const RopeAxesArgs p) {
    using ST = typename T::storage;
    __shared__ float2 cs[kMaxPairs];
    pdl_wait_previous();
    pdl_launch_dependents();
    const int t = blockIdx.x, D = p.head_dim, half = p.rope.rope_dim / 2;
    for (int i = threadIdx.x; i < half; i += kThreads) {
        const int axis = p.rope.pair_axis[i];
        const bool ok = axis >= 0 && axis < p.rope.num_axes;
        if (!ok && t == 0) report(p.status, PA_DEVERR_AXIS);
        cs[i] = ok ? rope_cos_sin(p.positions[(int64_t)axis * p.num_tokens + t], p.rope.freqs[i]) : make_float2(1.f, 0.f);
    }
    __syncthreads();
    if (p.num_heads)
        rotate_row(static_cast<ST *>(p.query_out) + (int64_t)t * p.num_heads * D,
                   static_cast<const ST *>(p.query) + t * p.query_stride, cs, p.num_heads, D, half, p.rope.halves);
    const int64_t slot = p.slot_mapping[t];
    if (slot < 0) return;
    if (slot >= (int64_t)p.num_blocks * p.block_size) {
        if (threadIdx.x == 0) report(p.status, PA_DEVERR_SLOT);
        return;
    }
    const int64_t row = slot * p.num_kv_heads * D;
    rotate_row(static_cast<ST *>(p.key_cache) + row, static_cast<const ST *>(p.key) + t * p.key_stride, cs,
               p.num_kv_heads, D, half, p.rope.halves);
    for (int i = threadIdx.x; i < p.num_kv_heads * D; i += kThreads)
        static_cast<ST *>(p.value_cache)[row + i] = static_cast<const ST *>(p.value)[t * p.value_stride + i];
}

}  // namespace

int launch_reshape_and_cache_rope_axes(const RopeAxesArgs &a) {
    cudaError_t e;
    switch (a.kv_dtype) {
        case PA_F32: e = launch_pdl(rope_axes_kernel<F32>, dim3(a.num_tokens), dim3(kThreads), 0, a.stream, a); break;
        case PA_F16: e = launch_pdl(rope_axes_kernel<F16>, dim3(a.num_tokens), dim3(kThreads), 0, a.stream, a); break;
        case PA_BF16: e = launch_pdl(rope_axes_kernel<BF16>, dim3(a.num_tokens), dim3(kThreads), 0, a.stream, a); break;
        default: return PA_ERR_UNSUPPORTED;
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
