// mla_append: RMSNorm of the latent, position rotation of the shared key part and of the
// queries' part, and the write into the paged cache, in one pass over the new tokens.
//
// One block per token: the block finds its sequence from cu_seqlens, forms the token's d_rope/2 angles once (float64 product and reduction: a float32 product
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
// pairs), or 2V neighbouring channels (interleaved pairs).
template <typename T, int V> struct Item {
    float a[V], b[V];
    static __device__ __forceinline__ int first(int item, bool interleaved) { return interleaved ? 2 * V * item : V * item; }
    static __device__ __forceinline__ int second(int item, int half, bool interleaved) {
        return interleaved ? 2 * V * item + V : V * item + half;
    }
    __device__ __forceinline__ void load(const T *src, int item, int half, bool interleaved) {
        load_vec<T, V>(src + first(item, interleaved), a);
        load_vec<T, V>(src + second(item, half, interleaved), b);
    }
    __device__ __forceinline__ void turn(int item, bool interleaved, const float2 *cs) {
        if (!interleaved || V == 1) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float2 w = cs[V * item + i];
                const float x = a[i], y = b[i];
                a[i] = x * w.x - y * w.y;
                b[i] = x * w.y + y * w.x;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 w = cs[V * item + i], u = cs[V * item + V / 2 + i];
                float x = a[2 * i], y = a[2 * i + 1];
                a[2 * i] = x * w.x - y * w.y;
                a[2 * i + 1] = x * w.y + y * w.x;
                x = b[2 * i], y = b[2 * i + 1];
                b[2 * i] = x * u.x - y * u.y;
                b[2 * i + 1] = x * u.y + y * u.x;
            }
        }
    }
    __device__ __forceinline__ void store(T *dst, int item, int half, bool interleaved) const {
        store_vec<T, V>(dst + first(item, interleaved), a);
        store_vec<T, V>(dst + second(item, half, interleaved), b);
    }
};

// The last b with cu[b] <= t, by one warp: 32 offsets a step, the steps' loads independent.
__device__ __forceinline__ int find_sequence(const int32_t *cu, int num_seqs, int64_t t) {
    int lo = 0, hi = num_seqs;
    while (hi - lo > 256) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    int count = 0;
#pragma unroll 4
    for (int i = lo + 1 + int(threadIdx.x & 31); i - int(threadIdx.x & 31) < hi; i += 32)
        count += __popc(__ballot_sync(0xffffffffu, i < hi && cu[i] <= t));
    return lo + count;
}

// The inputs' loads come first: they need only t, and the way to the cache row (offsets, past,
// page) takes several dependent loads.
template <typename T, int V> __global__ void __launch_bounds__(kThreads) append_kernel(const MlaAppendArgs a) {
    __shared__ float2 cs[kMaxRope / 2];
    __shared__ float warp_sum[kThreads / 32];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, half = a.dr / 2, items = half / V;
    const int q_items = a.q_rope ? items * a.H : 0;
    // latent: kept in registers between the sum of squares and the store
    constexpr int kChunks = (kMaxLatent + kThreads * V - 1) / (kThreads * V);
    float x[kChunks][V];
    const T *c_row = static_cast<const T *>(a.c) + t * a.c_stride;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int j = (i * kThreads + tid) * V;
        if (j < a.dc) load_vec<T, V>(c_row + j, x[i]);
    }
    // the first queries' item of this thread; the last threads take the key part's
    Item<T, V> q, k;
    const T *q_row = static_cast<const T *>(a.q_rope) + t * a.q_st;
    T *q_to = static_cast<T *>(a.q_out) + t * a.qo_st;
    const int k_item = kThreads - 1 - tid;
    if (tid < q_items) q.load(q_row + tid / items * a.q_sh, tid % items, half, a.interleaved);
    if (k_item < items) k.load(static_cast<const T *>(a.k_rope) + t * a.k_rope_stride, k_item, half, a.interleaved);

    const int b = find_sequence(a.cu, a.num_seqs, t);
    if (t < a.cu[b] || t >= a.cu[b + 1]) return;  // behind the last sequence
    const int64_t pos = int64_t(a.past[b]) + (t - a.cu[b]);
    T *row = nullptr;
    if (pos >= 0 && pos / a.page_size < a.max_pages) {
        const int32_t page = a.page_table[int64_t(b) * a.max_pages + pos / a.page_size];
        if (page >= 0 && page < a.num_pages)
            row = static_cast<T *>(a.cache) + (int64_t(page) * a.page_size + pos % a.page_size) * (a.dc + a.dr);
    }
    const bool turn = a.inv_freq != nullptr;
    if (turn && tid < half) {
        const double ang = double(pos) * double(a.inv_freq[tid]);
        const double two_pi = 6.283185307179586476925;
        float s, c;
        sincosf(float(ang - two_pi * rint(ang / two_pi)), &s, &c);
        cs[tid] = make_float2(c, s);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e)
            if ((i * kThreads + tid) * V < a.dc) ss = fmaf(x[i][e], x[i][e], ss);
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
    if (k_item < items) {
        if (turn) k.turn(k_item, a.interleaved, cs);
        if (row) k.store(row + a.dc, k_item, half, a.interleaved);
        if (a.k_rope_out) k.store(static_cast<T *>(a.k_rope_out) + t * a.dr, k_item, half, a.interleaved);
    }
    for (int w = tid; w < q_items; w += kThreads) {
        const int h = w / items, item = w % items;
        if (w != tid) q.load(q_row + h * a.q_sh, item, half, a.interleaved);
        if (turn) q.turn(item, a.interleaved, cs);
        q.store(q_to + h * a.qo_sh, item, half, a.interleaved);
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
