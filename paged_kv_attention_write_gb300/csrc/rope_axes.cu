// rope_axes.cu -- rotary positions with several axes, for a step's queries and keys, fused
// with the cache write.
//
// Pair i of token t turns by positions[pair_axis[i]][t] * freqs[i]:
// (x, y) -> (x cos - y sin, x sin + y cos).  Every element is read and written once, so the
// kernel is bound by HBM; what it must avoid is waiting.  One CTA per token: its threads have
// their first vectors in flight while the (cos, sin) of the token's pairs are computed into
// shared memory, at most one pair per thread; a thread then keeps the pairs of one place in
// the head in registers and applies them to the same place of every head it owns.
//
// Measured: 16384 tokens in fp32 (32 q / 8 kv heads, D 128, 805 MB) 117 us, 2048
// tokens in bf16 (50 MB) 10.2 us, 8 tokens 2.0 us.  CTAs of several tokens
// (their constants loaded once) took 122, 11.1 and 2.2 us in one wave, 121 and 12.9 us with four
// tokens each: the hardware's scheduling of many short CTAs hides the round trips better.
#include <cmath>
#include <type_traits>

#include "common.cuh"

namespace pa {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxPairs = 64;  // rope_dim <= head_dim <= 128
constexpr int kAhead = 3;      // heads of a thread whose loads are in flight together
constexpr int kPerSm = 6;      // resident CTAs per SM

// A 16-byte load that does not stay in L1 (queries may be rotated in place, so not through
// the read-only path).
__device__ __forceinline__ uint4 ld_once(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ void set_word(uint4 &v, int i, uint32_t w) {
    if (i == 0) v.x = w;
    if (i == 1) v.y = w;
    if (i == 2) v.z = w;
    if (i == 3) v.w = w;
}
__device__ __forceinline__ float2 unpack(F16, uint32_t w) {
    float2 f;
    widen_pair_f16(w, f.x, f.y);
    return f;
}
__device__ __forceinline__ float2 unpack(BF16, uint32_t w) {
    float2 f;
    widen_pair_bf16(w, f.x, f.y);
    return f;
}
__device__ __forceinline__ uint32_t pack(F16, float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack(BF16, float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 turn(float x, float y, float2 cs) {
    return make_float2(x * cs.x - y * cs.y, x * cs.y + y * cs.x);
}

// The elements of a against those of b (halves pairing), all rotated.
template <class T>
__device__ __forceinline__ void rotate_across(T t, uint4 &a, uint4 &b, const float2 *cs) {
    if constexpr (T::kPerVec == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 r = turn(__uint_as_float(word(a, i)), __uint_as_float(word(b, i)), cs[i]);
            set_word(a, i, __float_as_uint(r.x));
            set_word(b, i, __float_as_uint(r.y));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack(t, word(a, i)), y = unpack(t, word(b, i));
            const float2 r0 = turn(x.x, y.x, cs[2 * i]), r1 = turn(x.y, y.y, cs[2 * i + 1]);
            set_word(a, i, pack(t, r0.x, r1.x));
            set_word(b, i, pack(t, r0.y, r1.y));
        }
    }
}

// The first `n` adjacent pairs of a vector; the others keep their bits.
template <class T>
__device__ __forceinline__ void rotate_adjacent(T t, uint4 &a, const float2 *cs, int n) {
    if constexpr (T::kPerVec == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 r = turn(__uint_as_float(word(a, 2 * i)), __uint_as_float(word(a, 2 * i + 1)), cs[i]);
            if (i < n) {
                set_word(a, 2 * i, __float_as_uint(r.x));
                set_word(a, 2 * i + 1, __float_as_uint(r.y));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack(t, word(a, i)), r = turn(x.x, x.y, cs[i]);
            if (i < n) set_word(a, i, pack(t, r.x, r.y));
        }
    }
}

// The angle pos * f in turns.  Only its fraction matters, so it is formed as a 64-bit fraction, where
// whole turns fall off by themselves (Payne and Hanek's reduction, with one word of 1 / 2 pi):
// |f| / 2 pi to 2^-64, times pos.  (Subtracting a multiple of 2 pi in fp32 picks the wrong turn now
// and then from positions of 2^21 on.)
__device__ __forceinline__ uint64_t turns_per_position(float f) {
    constexpr uint64_t kPerTurn = 0xa2f9836e4e44152aull;  // 2^66 / 2 pi
    const uint32_t bits = __float_as_uint(f), exponent = bits >> 23 & 255u;
    const uint64_t m = (bits & 0x7fffffu) | (exponent ? 0x800000u : 0u);  // |f| = m 2^(exponent - 150)
    const int shift = 152 - (int)max(exponent, 1u);                       // |f| / 2 pi = m kPerTurn 2^-(64 + shift)
    const uint64_t lo = m * kPerTurn, hi = __umul64hi(m, kPerTurn);
    return shift <= 0 ? lo << min(-shift, 63) : shift < 64 ? hi << (64 - shift) | lo >> shift : hi >> min(shift - 64, 63);
}
// Its cosine and sine.  For every 32-bit position and frequencies below 4 the fraction, rounded to 32
// bits, is off by 1.9e-9 (as an angle) at most.  fp32 caches: rounding it to fp32 adds pi 2^-25,
// sincospif two units of the last place, 2.2e-7 in all.  16-bit caches round by 2^-11 at least, and
// there the hardware's sine and cosine (2^-21.2) of the fraction times pi do: under 1e-6 in all, and
// 2048 tokens take 10.1 us instead of 10.3.
template <class T>
__device__ __forceinline__ float2 cos_sin(int pos, uint64_t step, float f) {
    const uint64_t turn = step * (uint64_t)(int64_t)pos;
    const float x = (float)(int)((turn + 0x80000000ull) >> 32) * 0x1p-31f;  // in half turns, [-1, 1]
    float s, c;
    if constexpr (std::is_same<T, F32>::value)
        sincospif(x, &s, &c);
    else
        __sincosf(x * 3.14159265358979f, &s, &c);
    if (!(fabsf(f) < INFINITY)) c = s = NAN;
    return make_float2(c, f < 0.f ? -s : s);
}

// (cos, sin) of token t's pairs into cs, by all threads (a row has at most kMaxPairs pairs,
// one per thread).  The axis and frequency of a thread's pair and the token's positions on
// every axis are read together: one round trip, where following pair -> axis -> position
// would take two.
template <class T>
__device__ __forceinline__ void angles(const RopeAxesArgs &p, int t, float2 *cs) {
    __shared__ int32_t pos[PA_ROPE_MAX_AXES];
    const int i = threadIdx.x, half = p.rope.rope_dim / 2;
    const int axis = i < half ? p.rope.pair_axis[i] : 0;
    const float freq = i < half ? p.rope.freqs[i] : 0.f;
    if (i < p.rope.num_axes) pos[i] = p.positions[(int64_t)i * p.num_tokens + t];
    const uint64_t step = turns_per_position(freq);
    __syncthreads();
    if (i < half) {
        const bool ok = axis >= 0 && axis < p.rope.num_axes;
        if (!ok && t == 0) report(p.status, PA_DEVERR_AXIS);
        cs[i] = ok ? cos_sin<T>(pos[axis], step, freq) : make_float2(1.f, 0.f);  // not rotated
    }
    __syncthreads();
}

// One CTA per token; a thread owns vectors a and b (16 bytes each) of its heads.
template <class T, int D, bool HALVES>
__global__ void __launch_bounds__(kThreads, kPerSm) rope_axes_kernel(const RopeAxesArgs p) {
    using ST = typename T::storage;
    constexpr int EPV = T::kPerVec, PER_HEAD = D / EPV / 2;  // threads per head, two vectors each
    constexpr int STEP = kThreads / PER_HEAD;                // heads per pass of the CTA
    constexpr int HP = EPV / 2;                              // adjacent pairs of a vector
    __shared__ float2 cs[kMaxPairs];
    pdl_wait_previous();
    pdl_launch_dependents();
    const int half = p.rope.rope_dim / 2, j = threadIdx.x % PER_HEAD, h0 = threadIdx.x / PER_HEAD;
    const int Hq = p.num_heads, Hkv = p.num_kv_heads, heads = Hq + 2 * Hkv;
    // this thread's two vectors of a head, and what turns them
    int a, b, pa_ = 0, pb = 0, na = 0, nb = 0;
    bool rotated;
    if constexpr (HALVES) {
        const int hv = half / EPV;
        rotated = j < hv;
        a = rotated ? j : 2 * j;
        b = rotated ? j + hv : 2 * j + 1;
        pa_ = j * EPV;
    } else {
        a = j;
        b = j + PER_HEAD;
        pa_ = a * HP;
        pb = b * HP;
        na = max(0, min(HP, half - pa_));
        nb = max(0, min(HP, half - pb));
        rotated = na > 0;
    }
    a *= EPV;
    b *= EPV;
    const int t = blockIdx.x;
    const int64_t slot = p.slot_mapping[t];
    auto source = [&](int h) {
        return h < Hq ? static_cast<const ST *>(p.query) + t * p.query_stride + h * D
               : h < Hq + Hkv ? static_cast<const ST *>(p.key) + t * p.key_stride + (h - Hq) * D
                              : static_cast<const ST *>(p.value) + t * p.value_stride + (h - Hq - Hkv) * D;
    };
    auto target = [&](int h) {
        return h < Hq ? static_cast<ST *>(p.query_out) + ((int64_t)t * Hq + h) * D
               : h < Hq + Hkv ? static_cast<ST *>(p.key_cache) + (slot * Hkv + h - Hq) * D
                              : static_cast<ST *>(p.value_cache) + (slot * Hkv + h - Hq - Hkv) * D;
    };
    uint4 va[kAhead], vb[kAhead];
    auto load = [&](int first) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = first + u * STEP;
            if (h < heads) {  // whatever the slot: the loads do not wait for it
                const ST *src = source(h);
                va[u] = ld_once(src + a);
                vb[u] = ld_once(src + b);
            }
        }
    };
    load(h0);
    angles<T>(p, t, cs);
    const bool write = slot >= 0 && slot < (int64_t)p.num_blocks * p.block_size;
    if (slot >= 0 && !write && threadIdx.x == 0) report(p.status, PA_DEVERR_SLOT);
    const int todo = write ? heads : Hq;
    float2 c[EPV];
    if (rotated) {
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            if constexpr (HALVES)
                c[e] = cs[pa_ + e];
            else
                c[e] = e < HP ? (e < na ? cs[pa_ + e] : make_float2(1.f, 0.f))
                              : (e - HP < nb ? cs[pb + e - HP] : make_float2(1.f, 0.f));
        }
    }
    for (int first = h0; first < todo; first += kAhead * STEP) {
        if (first != h0) load(first);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int h = first + u * STEP;
            if (h < todo) {
                if (rotated && h < Hq + Hkv) {
                    if constexpr (HALVES) {
                        rotate_across(T{}, va[u], vb[u], c);
                    } else {
                        rotate_adjacent(T{}, va[u], c, na);
                        rotate_adjacent(T{}, vb[u], c + HP, nb);
                    }
                }
                ST *dst = target(h);
                *reinterpret_cast<uint4 *>(dst + a) = va[u];
                *reinterpret_cast<uint4 *>(dst + b) = vb[u];
            }
        }
    }
}

// The halves pairing of a width whose half is not a whole number of 16-byte vectors: element
// by element, one CTA per token.  A rare shape, twice the time of the kernel above: 2048 tokens
// of 32 q / 8 kv heads in bf16 22.5 us, 16384 133 (there 10.2 and 61.5).
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float v, float &x) { x = v; }
__device__ __forceinline__ void from_float(float v, __half &x) { x = __float2half_rn(v); }
__device__ __forceinline__ void from_float(float v, __nv_bfloat16 &x) { x = __float2bfloat16_rn(v); }

template <class ST>
__device__ void rotate_elements(ST *dst, const ST *src, const float2 *cs, int heads, int D, int half) {
    for (int i = threadIdx.x; i < heads * (D / 2); i += kThreads) {
        const int h = i / (D / 2), pair = i % (D / 2);
        const int a = h * D + (pair < half ? pair : 2 * pair), b = h * D + (pair < half ? pair + half : 2 * pair + 1);
        const ST xs = src[a], ys = src[b];
        if (pair < half) {
            const float2 r = turn(to_float(xs), to_float(ys), cs[pair]);
            from_float(r.x, dst[a]);
            from_float(r.y, dst[b]);
        } else {
            dst[a] = xs;
            dst[b] = ys;
        }
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) rope_axes_odd_halves_kernel(const RopeAxesArgs p) {
    using ST = typename T::storage;
    __shared__ float2 cs[kMaxPairs];
    pdl_wait_previous();
    pdl_launch_dependents();
    const int t = blockIdx.x, D = p.head_dim, half = p.rope.rope_dim / 2;
    angles<T>(p, t, cs);
    rotate_elements(static_cast<ST *>(p.query_out) + (int64_t)t * p.num_heads * D,
                    static_cast<const ST *>(p.query) + t * p.query_stride, cs, p.num_heads, D, half);
    const int64_t slot = p.slot_mapping[t];
    if (slot < 0) return;
    if (slot >= (int64_t)p.num_blocks * p.block_size) {
        if (threadIdx.x == 0) report(p.status, PA_DEVERR_SLOT);
        return;
    }
    const int64_t row = slot * p.num_kv_heads * D;
    rotate_elements(static_cast<ST *>(p.key_cache) + row, static_cast<const ST *>(p.key) + t * p.key_stride, cs,
                    p.num_kv_heads, D, half);
    for (int i = threadIdx.x; i < p.num_kv_heads * D; i += kThreads)
        static_cast<ST *>(p.value_cache)[row + i] = static_cast<const ST *>(p.value)[t * p.value_stride + i];
}

template <class T, int D>
cudaError_t launch_typed(const RopeAxesArgs &a) {
    if (a.rope.halves && (a.rope.rope_dim / 2) % T::kPerVec != 0)
        return launch_pdl(rope_axes_odd_halves_kernel<T>, dim3(a.num_tokens), dim3(kThreads), 0, a.stream, a);
    const dim3 grid(a.num_tokens);
    return a.rope.halves ? launch_pdl(rope_axes_kernel<T, D, true>, grid, dim3(kThreads), 0, a.stream, a)
                         : launch_pdl(rope_axes_kernel<T, D, false>, grid, dim3(kThreads), 0, a.stream, a);
}

template <class T>
cudaError_t launch_dim(const RopeAxesArgs &a) {
    return a.head_dim == 64 ? launch_typed<T, 64>(a) : launch_typed<T, 128>(a);
}

}  // namespace

int launch_reshape_and_cache_rope_axes(const RopeAxesArgs &a) {
    cudaError_t e;
    switch (a.kv_dtype) {
        case PA_F32: e = launch_dim<F32>(a); break;
        case PA_F16: e = launch_dim<F16>(a); break;
        case PA_BF16: e = launch_dim<BF16>(a); break;
        default: return PA_ERR_UNSUPPORTED;
    }
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
