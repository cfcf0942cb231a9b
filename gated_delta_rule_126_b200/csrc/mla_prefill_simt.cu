// mla_prefill and mla_backward on the CUDA cores, in float32: every type, head size and
// stride the calls take.  Tiles of scores with 64 streamed rows and 64 or 32 owned ones (the
// rows whose output a block makes), 256 threads with 4 x 4 or 4 x 2 scores each; the softmax
// is kept online (running maximum and sum), so scores never leave the SM.  The backward pass
// recomputes the scores from lse in two kernels, one per key tile (dk, dv) and one per query
// tile (dq), so that every sum has one owner and no atomics.  Bound by the float32 FMA pipes
// and shared memory; three float32 sequences of 700, 33 and 1025 tokens, 4 heads, d = 96 and
// 80, take 138 us forward, 182 us for dq and 252 us for dk and dv, the chain of the longest
// one's 17 tiles (146, 190 and 256 us with tiles loaded through registers, not asynchronously).
#include <cmath>

#include "mla_internal.h"
#include "mla_simt.cuh"

namespace kda {
namespace {

constexpr int kT = 64;  // streamed rows of a tile
constexpr int kThreads = 256;  // 16 x 16
constexpr int kLdP = kT + 4;
constexpr int kExact = 288;  // keys up to which a tile's delta is made from P and dP

struct Rows {  // one sequence's place
    int q0, lq, k0, lk;
};
__device__ __forceinline__ Rows rows_of(const MlaArgs &a, int s) {
    return Rows{a.cu_q[s], a.cu_q[s + 1] - a.cu_q[s], a.cu_k[s], a.cu_k[s + 1] - a.cu_k[s]};
}

template <typename T, int ROWS>
__device__ __forceinline__ void load_q(float *Q, int ld, const MlaArgs &a, const Rows &w, int h, int i0) {
    const int d = a.dn + a.dr, n = min(ROWS, w.lq - i0);
    load_tile<T, kThreads, ROWS>(Q, ld, 0, static_cast<const T *>(a.q) + (w.q0 + i0) * a.q_st + h * a.q_sh, a.q_st, d, n);
}
template <typename T, int ROWS>
__device__ __forceinline__ void load_k(float *K, int ld, const MlaArgs &a, const Rows &w, int h, int j0) {
    const int n = min(ROWS, w.lk - j0);
    load_tile<T, kThreads, ROWS>(K, ld, 0, static_cast<const T *>(a.k) + (w.k0 + j0) * a.k_st + h * a.k_sh, a.k_st, a.dn, n);
    if (a.dr)
        load_tile<T, kThreads, ROWS>(K, ld, a.dn, static_cast<const T *>(a.k_rope) + (w.k0 + j0) * a.kr_st, a.kr_st, a.dr, n);
}
template <typename T, int ROWS>
__device__ __forceinline__ void load_v(float *V, int ld, const MlaArgs &a, const Rows &w, int h, int j0) {
    const int n = min(ROWS, w.lk - j0);
    load_tile<T, kThreads, ROWS>(V, ld, 0, static_cast<const T *>(a.v) + (w.k0 + j0) * a.v_st + h * a.v_sh, a.v_st, a.dv, n);
}
template <typename T, int ROWS>
__device__ __forceinline__ void load_dO(float *D, int ld, const MlaArgs &a, const Rows &w, int h, int i0) {
    const int n = min(ROWS, w.lq - i0);
    load_tile<T, kThreads, ROWS>(D, ld, 0, static_cast<const T *>(a.dO) + (int64_t(w.q0 + i0) * a.H + h) * a.dv,
                               int64_t(a.H) * a.dv, a.dv, n);
}
// Keys that query i may see end here (bottom-right causal).
__device__ __forceinline__ int key_end(const MlaArgs &a, const Rows &w, int i) {
    return a.causal ? max(0, min(w.lk, i + 1 + w.lk - w.lq)) : w.lk;
}
__device__ __forceinline__ float half_warp_max(float x) {
#pragma unroll
    for (int d = 8; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
}
__device__ __forceinline__ float half_warp_sum(float x) {
#pragma unroll
    for (int d = 8; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// A block owns 16 I queries of a head.
template <typename T, int I> __global__ void __launch_bounds__(kThreads, I == 2 ? 2 : 1) prefill_kernel(const MlaArgs a) {
    extern __shared__ float sm[];
    __shared__ int64_t buf[kThreads / 32 + 2];
    constexpr int kOwn = 16 * I;
    const int d = a.dn + a.dr, d4 = (d + 3) & ~3, ldd = simt_row(d), ldv = simt_row(a.dv), h = blockIdx.y;
    float *Q = sm, *K = Q + kOwn * ldd, *V = K + kT * ldd, *P = V + kT * ldv;
    int seq, tile;
    if (!find_tile<kThreads>(a.cu_q, a.num_seqs, kOwn, gridDim.x - 1 - blockIdx.x, buf, &seq, &tile)) return;
    const Rows w = rows_of(a, seq);
    const int i0 = tile * kOwn, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    zero_columns<kThreads>(Q, ldd, d, d4, kOwn);
    zero_columns<kThreads>(K, ldd, d, d4, kT);
    zero_columns<kThreads>(V, ldv, a.dv, (a.dv + 3) & ~3, kT);
    load_q<T, kOwn>(Q, ldd, a, w, h, i0);
    float m[I], l[I], o[I][8] = {};
#pragma unroll
    for (int i = 0; i < I; ++i) m[i] = -INFINITY, l[i] = 0.f;
    const int last = key_end(a, w, min(i0 + kOwn, w.lq) - 1);
    for (int j0 = 0; j0 < last; j0 += kT) {
        __syncthreads();
        load_k<T, kT>(K, ldd, a, w, h, j0);
        load_v<T, kT>(V, ldv, a, w, h, j0);
        cp_async_wait();
        __syncthreads();
        float s[I][4] = {};
        tile_dot(s, Q, ldd, K, ldd, d4, ty, tx);
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int end = key_end(a, w, i0 + I * ty + i) - j0;
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = tx + 16 * j < end ? s[i][j] * a.scale : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
            top = fmaxf(m[i], half_warp_max(top));
            const float base = top == -INFINITY ? 0.f : top;  // nothing seen yet: exp(-inf) = 0 throughout
            const float keep = expf(m[i] - base);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = expf(s[i][j] - base);
                P[(I * ty + i) * kLdP + tx + 16 * j] = p;
                sum += p;
            }
            l[i] = l[i] * keep + half_warp_sum(sum);
            m[i] = top;
#pragma unroll
            for (int c = 0; c < 8; ++c) o[i][c] *= keep;
        }
        __syncwarp();  // a row of P is written and read by the same half warp
        tile_apply<I, 2>(o, P, kLdP, V, ldv, a.dv, ty, tx);
    }
    cp_async_wait();  // of a loop without turns
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int r = i0 + I * ty + i;
        if (r >= w.lq) continue;
        const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
        T *out = static_cast<T *>(a.o) + (int64_t(w.q0 + r) * a.H + h) * a.dv;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int col = (c >> 2) * 64 + 4 * tx + (c & 3);
            // a NaN among the seen scores makes l NaN: it reaches the output
            if (col < a.dv) out[col] = from_f32<T>(l[i] == 0.f ? 0.f : l[i] > 0.f ? o[i][c] * inv : l[i]);
        }
        if (a.lse && tx == 0) a.lse[int64_t(w.q0 + r) * a.H + h] = m[i] == -INFINITY && l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
    }
}

// Statistics of queries i0 + I ty + i (0 behind the sequence).
template <int I>
__device__ __forceinline__ void row_stats(const MlaArgs &a, const Rows &w, int h, int i0, int ty, float (&lse)[I], float (&delta)[I]) {
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int r = i0 + I * ty + i;
        lse[i] = r < w.lq ? a.lse[int64_t(w.q0 + r) * a.H + h] : 0.f;
        delta[i] = r < w.lq ? a.delta[int64_t(h) * a.Tq + w.q0 + r] : 0.f;
    }
}

// P and dP of one tile (queries I ty + i, keys tx + 16 j), from the recomputed scores: p = exp(s - lse); both 0 where
// the query does not see the key.
template <int I, int J>
__device__ __forceinline__ void tile_grads(const MlaArgs &a, const Rows &w, int i0, int j0, const float *Q, const float *K,
                                           const float *V, const float *D, int ldd, int ldv, int d4, int dv4, int ty, int tx,
                                           const float (&lse)[I], float (&p)[I][J], float (&dp)[I][J]) {
    float s[I][J] = {};
    tile_dot(s, Q, ldd, K, ldd, d4, ty, tx);
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) dp[i][j] = 0.f;
    tile_dot(dp, D, ldv, V, ldv, dv4, ty, tx);
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int r = i0 + I * ty + i, end = r < w.lq ? key_end(a, w, r) - j0 : 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool seen = tx + 16 * j < end;
            p[i][j] = seen ? expf(s[i][j] * a.scale - lse[i]) : 0.f;
            dp[i][j] = seen ? dp[i][j] : 0.f;
        }
    }
}

// A block owns 16 J keys of a head.
template <typename T, int J> __global__ void __launch_bounds__(kThreads, J == 2 ? 2 : 1) dkv_kernel(const MlaArgs a) {
    extern __shared__ float sm[];
    __shared__ int64_t buf[kThreads / 32 + 2];
    constexpr int kOwn = 16 * J;
    const int d = a.dn + a.dr, d4 = (d + 3) & ~3, dv4 = (a.dv + 3) & ~3, h = blockIdx.y;
    const int ldd = simt_row(d), ldv = simt_row(a.dv);
    float *Q = sm, *K = Q + kT * ldd, *V = K + kOwn * ldd, *D = V + kOwn * ldv, *Pt = D + kT * ldv, *St = Pt + kOwn * kLdP;
    int seq, tile;
    if (!find_tile<kThreads>(a.cu_k, a.num_seqs, kOwn, blockIdx.x, buf, &seq, &tile)) return;
    const Rows w = rows_of(a, seq);
    const int j0 = tile * kOwn, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    zero_columns<kThreads>(Q, ldd, d, d4, kT);
    zero_columns<kThreads>(K, ldd, d, d4, kOwn);
    zero_columns<kThreads>(V, ldv, a.dv, dv4, kOwn);
    zero_columns<kThreads>(D, ldv, a.dv, dv4, kT);
    load_k<T, kOwn>(K, ldd, a, w, h, j0);
    load_v<T, kOwn>(V, ldv, a, w, h, j0);
    float dk[J][12] = {}, dv[J][8] = {};
    // the first query that sees key j0
    const int first = a.causal ? max(0, j0 - (w.lk - w.lq)) / kT * kT : 0;
    for (int i0 = first; i0 < w.lq; i0 += kT) {
        __syncthreads();
        load_q<T, kT>(Q, ldd, a, w, h, i0);
        load_dO<T, kT>(D, ldv, a, w, h, i0);
        cp_async_wait();
        __syncthreads();
        float p[4][J], dp[4][J], lse[4], delta[4];
        row_stats(a, w, h, i0, ty, lse, delta);
        tile_grads(a, w, i0, j0, Q, K, V, D, ldd, ldv, d4, dv4, ty, tx, lse, p, dp);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                Pt[(tx + 16 * j) * kLdP + 4 * ty + i] = p[i][j];
                St[(tx + 16 * j) * kLdP + 4 * ty + i] = p[i][j] * (dp[i][j] - delta[i]) * a.scale;
            }
        __syncthreads();
        tile_apply<J, 2>(dv, Pt, kLdP, D, ldv, a.dv, ty, tx);
        tile_apply<J, 3>(dk, St, kLdP, Q, ldd, d, ty, tx);
    }
    cp_async_wait();  // of a loop without turns
#pragma unroll
    for (int i = 0; i < J; ++i) {
        const int r = j0 + J * ty + i;
        if (r >= w.lk) continue;
        const int64_t at = int64_t(w.k0 + r) * a.H + h;
#pragma unroll
        for (int c = 0; c < 12; ++c) {
            const int col = (c >> 2) * 64 + 4 * tx + (c & 3);
            if (col < a.dn) static_cast<T *>(a.dk)[at * a.dn + col] = from_f32<T>(dk[i][c]);
            else if (col < d) a.dkr_partial[(int64_t(h) * a.Tk + w.k0 + r) * a.dr + col - a.dn] = dk[i][c];
            if (c < 8 && col < a.dv) static_cast<T *>(a.dv_out)[at * a.dv + col] = from_f32<T>(dv[i][c & 7]);
        }
    }
}

// A block owns 16 I queries of a head.
template <typename T, int I> __global__ void __launch_bounds__(kThreads, I == 2 ? 2 : 1) dq_kernel(const MlaArgs a) {
    extern __shared__ float sm[];
    __shared__ int64_t buf[kThreads / 32 + 2];
    constexpr int kOwn = 16 * I;
    const int d = a.dn + a.dr, d4 = (d + 3) & ~3, dv4 = (a.dv + 3) & ~3, h = blockIdx.y;
    const int ldd = simt_row(d), ldv = simt_row(a.dv);
    float *Q = sm, *K = Q + kOwn * ldd, *V = K + kT * ldd, *D = V + kT * ldv, *S = D + kOwn * ldv;
    int seq, tile;
    if (!find_tile<kThreads>(a.cu_q, a.num_seqs, kOwn, gridDim.x - 1 - blockIdx.x, buf, &seq, &tile)) return;
    const Rows w = rows_of(a, seq);
    const int i0 = tile * kOwn, tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    zero_columns<kThreads>(Q, ldd, d, d4, kOwn);
    zero_columns<kThreads>(K, ldd, d, d4, kT);
    zero_columns<kThreads>(V, ldv, a.dv, dv4, kT);
    zero_columns<kThreads>(D, ldv, a.dv, dv4, kOwn);
    load_q<T, kOwn>(Q, ldd, a, w, h, i0);
    load_dO<T, kOwn>(D, ldv, a, w, h, i0);
    float dq[I][12] = {}, lse[I], delta[I];
    row_stats(a, w, h, i0, ty, lse, delta);
    const int last = key_end(a, w, min(i0 + kOwn, w.lq) - 1);
    // Rows that see few keys: delta = sum_j P dP first, for dk and dv too, in place of the one from the rounded o
    // (mla_backward_tc.cu says why); float32's o needs none of it.
    const bool exact = sizeof(T) == 2 && last <= kExact;
    float sum[I] = {};
    for (int pass = exact ? 0 : 1; pass < 2; ++pass) {
        for (int j0 = 0; j0 < last; j0 += kT) {
            __syncthreads();
            load_k<T, kT>(K, ldd, a, w, h, j0);
            load_v<T, kT>(V, ldv, a, w, h, j0);
            cp_async_wait();
            __syncthreads();
            float p[I][4], dp[I][4];
            tile_grads(a, w, i0, j0, Q, K, V, D, ldd, ldv, d4, dv4, ty, tx, lse, p, dp);
            if (pass == 0) {
#pragma unroll
                for (int i = 0; i < I; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum[i] = fmaf(p[i][j], dp[i][j], sum[i]);
                continue;
            }
#pragma unroll
            for (int i = 0; i < I; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) S[(I * ty + i) * kLdP + tx + 16 * j] = p[i][j] * (dp[i][j] - delta[i]) * a.scale;
            __syncwarp();
            tile_apply<I, 3>(dq, S, kLdP, K, ldd, d, ty, tx);
        }
        if (pass == 0) {
#pragma unroll
            for (int i = 0; i < I; ++i) {
                delta[i] = half_warp_sum(sum[i]);
                const int r = i0 + I * ty + i;
                if (tx == 0 && r < w.lq) a.delta[int64_t(h) * a.Tq + w.q0 + r] = delta[i];
            }
        }
    }
    cp_async_wait();  // of a loop without turns
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int r = i0 + I * ty + i;
        if (r >= w.lq) continue;
        T *out = static_cast<T *>(a.dq) + (int64_t(w.q0 + r) * a.H + h) * d;
#pragma unroll
        for (int c = 0; c < 12; ++c) {
            const int col = (c >> 2) * 64 + 4 * tx + (c & 3);
            if (col < d) out[col] = from_f32<T>(dq[i][c]);
        }
    }
}

// delta[h][t] = sum_c dO o and lse2[h][t] = lse log2(e) of the sequences' rows.  16 lanes a (token, head), eight
// channels a lane where a row's start and length allow 16-byte loads (V = 8 bf16 or 4 f32), else channel by
// channel; bound by memory (2 d_v elements a row).
template <typename T, int V> __global__ void delta_kernel(const MlaArgs a) {
    const int64_t row = int64_t(blockIdx.x) * (blockDim.x >> 4) + (threadIdx.x >> 4);
    if (row >= a.Tq * a.H) return;
    const T *x = static_cast<const T *>(a.dO) + row * a.dv, *y = static_cast<const T *>(a.o) + row * a.dv;
    float s = 0.f;
    for (int c = (threadIdx.x & 15) * V; c < a.dv; c += 16 * V) {
        if constexpr (V == 1) {
            s = fmaf(to_f32(x[c]), to_f32(y[c]), s);
        } else {
            const uint4 u = *reinterpret_cast<const uint4 *>(x + c), w = *reinterpret_cast<const uint4 *>(y + c);
            const T *p = reinterpret_cast<const T *>(&u), *q = reinterpret_cast<const T *>(&w);
#pragma unroll
            for (int e = 0; e < V; ++e) s = fmaf(to_f32(p[e]), to_f32(q[e]), s);
        }
    }
    const unsigned lanes = 0xffffu << (threadIdx.x & 16);  // a row's lanes, which all reach this
#pragma unroll
    for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(lanes, s, o);
    if ((threadIdx.x & 15) == 0) {
        const int64_t at = row % a.H * a.Tq + row / a.H;
        a.delta[at] = s;
        a.lse2[at] = a.lse[row] * 1.4426950408889634f;
    }
}

// dk_rope[t][c] = sum_h partial[h][t][c], in the order of the heads.
template <typename T> __global__ void dkr_kernel(const MlaArgs a) {
    const int64_t n = a.Tk * a.dr, i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= n) return;
    float s = 0.f;
    for (int h = 0; h < a.H; ++h) s += a.dkr_partial[h * n + i];
    static_cast<T *>(a.dk_rope)[i] = from_f32<T>(s);
}

// Shared memory of a kernel that owns `own` rows (floats): tiles of d and of d_v channels, own and streamed rows, and P.
size_t prefill_smem(const MlaArgs &a, int own) {
    return sizeof(float) * ((own + kT) * simt_row(a.dn + a.dr) + kT * simt_row(a.dv) + own * kLdP);
}
size_t grad_smem(const MlaArgs &a, int own, int tiles) {
    return sizeof(float) * ((own + kT) * (simt_row(a.dn + a.dr) + simt_row(a.dv)) + tiles * own * kLdP);
}

template <typename K> cudaError_t launch(K *kernel, int64_t tiles, size_t smem, const MlaArgs &a, cudaStream_t st) {
    if (tiles == 0) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    kernel<<<dim3(unsigned(tiles), unsigned(a.H)), kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

// 64 owned rows a block, or 32 where blocks of 64 would leave a third of the SMs idle: there the longest block's chain of
// tiles is the call's time, and smaller tiles shorten it.  One float32 sequence of 1024 tokens, d = 192 and 128, forward
// and backward: with 6 heads (96 blocks of 64) 163 and 521 us in tiles of 32, 185 and 627 in tiles of 64;
// with 8 heads (128 blocks) 213 and 681 against 214 and 626.
bool small_tiles(const int32_t *cu, const MlaArgs &a) { return 3 * count_tiles(cu, a.num_seqs, 64) * a.H < 2 * device_sm_count(); }

template <typename T> cudaError_t prefill(const MlaArgs &a, cudaStream_t st) {
    if (small_tiles(a.cu_q_host, a))
        return launch(prefill_kernel<T, 2>, count_tiles(a.cu_q_host, a.num_seqs, 32), prefill_smem(a, 32), a, st);
    return launch(prefill_kernel<T, 4>, count_tiles(a.cu_q_host, a.num_seqs, 64), prefill_smem(a, 64), a, st);
}

template <typename T> cudaError_t backward(const MlaArgs &a, cudaStream_t st) {
    cudaError_t e;  // dq first: it leaves the delta of the rows that see few keys
    if (small_tiles(a.cu_q_host, a))
        e = launch(dq_kernel<T, 2>, count_tiles(a.cu_q_host, a.num_seqs, 32), grad_smem(a, 32, 1), a, st);
    else
        e = launch(dq_kernel<T, 4>, count_tiles(a.cu_q_host, a.num_seqs, 64), grad_smem(a, 64, 1), a, st);
    if (e != cudaSuccess) return e;
    if (small_tiles(a.cu_k_host, a))
        return launch(dkv_kernel<T, 2>, count_tiles(a.cu_k_host, a.num_seqs, 32), grad_smem(a, 32, 2), a, st);
    return launch(dkv_kernel<T, 4>, count_tiles(a.cu_k_host, a.num_seqs, 64), grad_smem(a, 64, 2), a, st);
}

}  // namespace

cudaError_t launch_mla_prefill_simt(const MlaArgs &a, cudaStream_t st) {
    return a.dtype == KDA_DTYPE_F32 ? prefill<float>(a, st) : prefill<__nv_bfloat16>(a, st);
}

namespace {
template <typename T> cudaError_t delta(const MlaArgs &a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const int64_t blocks = (a.Tq * a.H + 15) / 16;
    if (blocks == 0) return cudaSuccess;
    const bool vec = a.dv % V == 0 && (reinterpret_cast<uintptr_t>(a.dO) & 15) == 0 && (reinterpret_cast<uintptr_t>(a.o) & 15) == 0;
    if (vec) delta_kernel<T, V><<<unsigned(blocks), 256, 0, st>>>(a);
    else delta_kernel<T, 1><<<unsigned(blocks), 256, 0, st>>>(a);
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_mla_delta(const MlaArgs &a, cudaStream_t st) {
    return a.dtype == KDA_DTYPE_F32 ? delta<float>(a, st) : delta<__nv_bfloat16>(a, st);
}

cudaError_t launch_mla_dkr_reduce(const MlaArgs &a, cudaStream_t st) {
    const int64_t blocks = (a.Tk * a.dr + 255) / 256;
    if (blocks == 0) return cudaSuccess;
    if (a.dtype == KDA_DTYPE_F32) dkr_kernel<float><<<unsigned(blocks), 256, 0, st>>>(a);
    else dkr_kernel<__nv_bfloat16><<<unsigned(blocks), 256, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_mla_backward_simt(const MlaArgs &a, cudaStream_t st) {
    return a.dtype == KDA_DTYPE_F32 ? backward<float>(a, st) : backward<__nv_bfloat16>(a, st);
}

}  // namespace kda
