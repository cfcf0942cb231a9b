// mla_append: RMSNorm of the latent, position rotation of the shared key part and of the
// queries' part, and the write into the paged cache, in one pass over the new tokens.
//
// One block per token: the block finds its sequence by a binary search over cu_seqlens,
// forms the token's d_rope/2 angles once (float64 product and reduction: a float32 product
// at position 10^6 is off by 0.03 rad) and shares them between the key part and all heads.
// Bound by memory: each input element is read once and each output written once.
#include <algorithm>

#include "mla_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxLatent = 512;
constexpr int kMaxRope = 64;

template <typename T> struct Io;
template <> struct Io<float> {
    static __device__ float get(const float *p) { return *p; }
    static __device__ void put(float *p, float x) { *p = x; }
};
template <> struct Io<__nv_bfloat16> {
    static __device__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    static __device__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
};

// V elements at p as floats (V * sizeof(T) is 16 bytes, or V = 1).
template <typename T, int V> __device__ __forceinline__ void load_vec(const T *p, float (&x)[V]) {
    if constexpr (V == 1) {
        x[0] = Io<T>::get(p);
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const T *e = reinterpret_cast<const T *>(&w);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = Io<T>::get(e + i);
    }
}
template <typename T, int V> __device__ __forceinline__ void store_vec(T *p, const float (&x)[V]) {
    if constexpr (V == 1) {
        Io<T>::put(p, x[0]);
    } else {
        uint4 w;
        T *e = reinterpret_cast<T *>(&w);
#pragma unroll
        for (int i = 0; i < V; ++i) Io<T>::put(e + i, x[i]);
        *reinterpret_cast<uint4 *>(p) = w;
    }
}

// One item of rotation work: V channels of the first half and their partners (half-split
// pairs), or 2V neighbouring channels (interleaved pairs).  dst and dst2 may be NULL.
template <typename T, int V>
__device__ __forceinline__ void rotate_item(const T *src, T *dst, T *dst2, int item, int half, bool interleaved,
                                            const float2 *cs, bool turn) {
    float a[V], b[V], x[V], y[V];
    const int o0 = interleaved ? 2 * V * item : V * item;
    const int o1 = interleaved ? o0 + V : o0 + half;
    load_vec<T, V>(src + o0, a);
    load_vec<T, V>(src + o1, b);
    if (!turn) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = a[i], y[i] = b[i];
    } else if (!interleaved) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 w = cs[V * item + i];
            x[i] = a[i] * w.x - b[i] * w.y;
            y[i] = a[i] * w.y + b[i] * w.x;
        }
    } else if constexpr (V == 1) {
        const float2 w = cs[item];
        x[0] = a[0] * w.x - b[0] * w.y;
        y[0] = a[0] * w.y + b[0] * w.x;
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 w = cs[V * item + i], u = cs[V * item + V / 2 + i];
            x[2 * i] = a[2 * i] * w.x - a[2 * i + 1] * w.y;
            x[2 * i + 1] = a[2 * i] * w.y + a[2 * i + 1] * w.x;
            y[2 * i] = b[2 * i] * u.x - b[2 * i + 1] * u.y;
            y[2 * i + 1] = b[2 * i] * u.y + b[2 * i + 1] * u.x;
        }
    }
    if (dst) store_vec<T, V>(dst + o0, x), store_vec<T, V>(dst + o1, y);
    if (dst2) store_vec<T, V>(dst2 + o0, x), store_vec<T, V>(dst2 + o1, y);
}

template <typename T, int V> __global__ void __launch_bounds__(kThreads) append_kernel(const MlaAppendArgs a) {
    __shared__ float2 cs[kMaxRope / 2];
    __shared__ float warp_sum[kThreads / 32];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x;
    // the sequence of row t: the last b with cu[b] <= t
    int lo = 0, hi = a.num_seqs;
    while (lo + 1 < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    if (t < a.cu[lo] || t >= a.cu[lo + 1]) return;  // behind the last sequence
    const int64_t pos = int64_t(a.past[lo]) + (t - a.cu[lo]);
    T *row = nullptr;
    if (pos >= 0 && pos / a.page_size < a.max_pages) {
        const int32_t page = a.page_table[int64_t(lo) * a.max_pages + pos / a.page_size];
        if (page >= 0 && page < a.num_pages)
            row = static_cast<T *>(a.cache) + (int64_t(page) * a.page_size + pos % a.page_size) * (a.dc + a.dr);
    }
    const int half = a.dr / 2;
    const bool turn = a.inv_freq != nullptr;
    if (turn && tid < half) {
        const double ang = double(pos) * double(a.inv_freq[tid]);
        const double two_pi = 6.283185307179586476925;
        float s, c;
        sincosf(float(ang - two_pi * rint(ang / two_pi)), &s, &c);
        cs[tid] = make_float2(c, s);
    }
    // latent: kept in registers between the sum of squares and the store
    constexpr int kChunks = (kMaxLatent + kThreads * V - 1) / (kThreads * V);
    float x[kChunks][V];
    const T *c_row = static_cast<const T *>(a.c) + t * a.c_stride;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int j = (i * kThreads + tid) * V;
        if (j < a.dc) {
            load_vec<T, V>(c_row + j, x[i]);
#pragma unroll
            for (int e = 0; e < V; ++e) ss = fmaf(x[i][e], x[i][e], ss);
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if ((tid & 31) == 0) warp_sum[tid >> 5] = ss;
    __syncthreads();
    ss = warp_sum[0] + warp_sum[1] + warp_sum[2] + warp_sum[3];
    if (a.norm_weight) {
        const float r = 1.f / sqrtf(ss / float(a.dc) + a.eps);
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int j = (i * kThreads + tid) * V + e;
                if (j < a.dc) x[i][e] *= r * a.norm_weight[j];
            }
    }
    T *c_out = a.c_out ? static_cast<T *>(a.c_out) + t * a.dc : nullptr;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int j = (i * kThreads + tid) * V;
        if (j < a.dc) {
            if (row) store_vec<T, V>(row + j, x[i]);
            if (c_out) store_vec<T, V>(c_out + j, x[i]);
        }
    }
    if (a.dr == 0) return;
    // rotation: the key part and the queries of every head, `items` pieces each
    const int items = half / V;
    const int heads = a.q_rope ? a.H : 0;
    for (int w = tid; w < items * (heads + 1); w += kThreads) {
        const int h = w / items - 1, item = w % items;
        if (h < 0) {
            const T *src = static_cast<const T *>(a.k_rope) + t * a.k_rope_stride;
            T *dst2 = a.k_rope_out ? static_cast<T *>(a.k_rope_out) + t * a.dr : nullptr;
            rotate_item<T, V>(src, row ? row + a.dc : nullptr, dst2, item, half, a.interleaved, cs, turn);
        } else {
            const T *src = static_cast<const T *>(a.q_rope) + t * a.q_st + h * a.q_sh;
            T *dst = static_cast<T *>(a.q_out) + t * a.qo_st + h * a.qo_sh;
            rotate_item<T, V>(src, dst, nullptr, item, half, a.interleaved, cs, turn);
        }
    }
}

// Whole 16-byte vectors everywhere: bases, strides, the latent's width and half a rotation.
template <typename T> bool vector_ok(const MlaAppendArgs &a) {
    constexpr int V = 16 / sizeof(T);
    auto p16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    const void *ptrs[] = {a.c, a.k_rope, a.cache, a.q_rope, a.q_out, a.c_out, a.k_rope_out};
    for (const void *p : ptrs)
        if (!p16(p)) return false;
    if (a.dc % V || (a.dr / 2) % V || a.c_stride % V) return false;
    if (a.dr && a.k_rope_stride % V) return false;
    return !a.q_rope || !(a.q_st % V || a.q_sh % V || a.qo_st % V || a.qo_sh % V);
}

template <typename T> cudaError_t launch(const MlaAppendArgs &a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (vector_ok<T>(a)) append_kernel<T, V><<<unsigned(a.total_tokens), kThreads, 0, st>>>(a);
    else append_kernel<T, 1><<<unsigned(a.total_tokens), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mla_append(const MlaAppendArgs &a, cudaStream_t st) {
    return a.dtype == KDA_DTYPE_F32 ? launch<float>(a, st) : launch<__nv_bfloat16>(a, st);
}

}  // namespace kda
