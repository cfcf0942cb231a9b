// Building blocks of the latent-attention kernels that run on the CUDA cores in float32:
// tile loads with conversion, and register-tiled products over shared-memory tiles.
#pragma once

#include "mla_internal.h"

namespace kda {

template <typename T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Row length in floats of a shared tile of d channels: at least d, and 4 more than a
// multiple of 32, so that eight neighbouring rows' float4 loads touch all 32 banks.
__host__ __device__ constexpr int simt_row(int d) { return (d + 31) / 32 * 32 + 4; }

// The sequence and tile of block x when every sequence's rows are cut into tiles of `tile`
// rows, numbered in sequence order.  Called by all NT threads; `buf` holds NT / 32 + 2 int64.  False when x lies
// behind the last tile.
template <int NT>
__device__ bool find_tile(const int32_t *cu, int num_seqs, int tile, int64_t x, int64_t *buf, int *seq, int *index) {
    const int per = (num_seqs + NT - 1) / NT;
    const int s0 = threadIdx.x * per, s1 = min(num_seqs, s0 + per);
    int64_t own = 0;
    for (int s = s0; s < s1; ++s) own += (cu[s + 1] - cu[s] + tile - 1) / tile;
    int64_t scan = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, scan, d);
        if ((threadIdx.x & 31) >= d) scan += o;
    }
    if ((threadIdx.x & 31) == 31) buf[threadIdx.x >> 5] = scan;
    __syncthreads();
    int64_t total = 0;
    for (int w = 0; w < NT / 32; ++w) {
        if (w < int(threadIdx.x >> 5)) scan += buf[w];
        total += buf[w];
    }
    if (x >= total) return false;
    if (own > 0 && scan - own <= x && x < scan) {
        int64_t at = scan - own;
        int s = s0;
        for (; s < s1; ++s) {
            const int64_t nt = (cu[s + 1] - cu[s] + tile - 1) / tile;
            if (x < at + nt) break;
            at += nt;
        }
        buf[NT / 32] = s;
        buf[NT / 32 + 1] = x - at;
    }
    __syncthreads();
    *seq = int(buf[NT / 32]);
    *index = int(buf[NT / 32 + 1]);
    return true;
}

// The tile (the k-th of its sequence's n) and head of a block whose tile was found by its number x / H alone: within a
// sequence, blocks go through GROUP heads at a time, all tiles of those, so that what their tiles share stays in L2.
template <int GROUP> __device__ __forceinline__ void regroup(int64_t x, int H, int n, int *k, int *head) {
    const int local = int(x - (x / H - *k) * H);  // number of the block in its sequence
    const int g = local / (n * GROUP), in = local - g * n * GROUP, width = min(GROUP, H - g * GROUP);
    *k = in / width;
    *head = g * GROUP + in % width;
}

// Four elements at p (16 bytes of float32, 8 of bf16) as float32.
template <typename T> __device__ __forceinline__ float4 load4(const T *p);
template <> __device__ __forceinline__ float4 load4<float>(const float *p) { return *reinterpret_cast<const float4 *>(p); }
template <> __device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16 *p) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}
// Whether rows of this base, stride and width can be read four elements at a time.
template <typename T> __device__ __forceinline__ bool by4(const T *p, int64_t stride, int width) {
    return ((stride | width) & 3) == 0 && (reinterpret_cast<uintptr_t>(p) & (4 * sizeof(T) - 1)) == 0;
}

// Four float32 from p into shared memory without waiting (cp_async_wait before the barrier after which they are
// read), or four zeros.
__device__ __forceinline__ void copy4_async(float *dst, const float *p, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(p), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// dst[r][at + c] = src[r * stride + c] for r < ROWS, c < width, as float32; rows from `valid` on are zero.
// 16 threads a row.  float32 rows that can be read four elements at a time are copied asynchronously, so that all of a
// tile's loads, and those of several tiles, are under way together: cp_async_wait() before the barrier.
template <typename T, int NT, int ROWS>
__device__ __forceinline__ void load_tile(float *dst, int ld, int at, const T *src, int64_t stride, int width, int valid) {
    constexpr int kPer = ROWS / (NT / 16);
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    if (by4(src, stride, width) && (at & 3) == 0) {
        if constexpr (sizeof(T) == 4) {
            for (int c = 4 * tx; c < width; c += 64)
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int r = ty + NT / 16 * i;
                    copy4_async(dst + r * ld + at + c, src + (r < valid ? r * stride + c : 0), r < valid);
                }
            return;
        }
        for (int c = 4 * tx; c < width; c += 64) {
            float4 v[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int r = ty + NT / 16 * i;
                v[i] = r < valid ? load4(src + r * stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) *reinterpret_cast<float4 *>(dst + (ty + NT / 16 * i) * ld + at + c) = v[i];
        }
    } else {
        for (int c = tx; c < width; c += 16) {
            float v[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int r = ty + NT / 16 * i;
                v[i] = r < valid ? to_f32(src[r * stride + c]) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) dst[(ty + NT / 16 * i) * ld + at + c] = v[i];
        }
    }
}
// The blocks of a cluster, which share the work on one tile of owned rows.
struct Share {
    int rank, ranks;
    // Rows I ty + i of the owned tile whose sums this block makes and writes.
    __device__ __forceinline__ bool owns(int i) const { return i % ranks == rank; }
};
__device__ __forceinline__ Share cluster_share() {
    Share s;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(s.rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(s.ranks));
    return s;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// What block `rank` of the cluster holds where this one has p.
__device__ __forceinline__ uint32_t peer_smem(const float *p, int rank) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank));
    return at;
}
__device__ __forceinline__ float4 load4_peer(const float *p, int rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(peer_smem(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ float2 load2_peer(const float *p, int rank) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(peer_smem(p, rank)) : "memory");
    return v;
}
// Leaves this block's sums at `at` (I * C * NT floats, 16-byte aligned) for the cluster.
template <int NT, int I, int C> __device__ __forceinline__ void leave(float *at, const float (&acc)[I][C]) {
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
        for (int c = 0; c < C; c += 4)
            *reinterpret_cast<float4 *>(at + ((i * C + c) * NT + 4 * threadIdx.x)) = make_float4(acc[i][c], acc[i][c + 1], acc[i][c + 2], acc[i][c + 3]);
}
// After a cluster_sync: row i's sums over all blocks, in the order of their ranks, block r's times f[r] where given.
template <int NT, int C> __device__ __forceinline__ void gather(float (&row)[C], const float *at, int i, int ranks, const float *f = nullptr) {
#pragma unroll
    for (int c = 0; c < C; ++c) row[c] = 0.f;
    for (int r = 0; r < ranks; ++r) {
        const float w = f ? f[r] : 1.f;
#pragma unroll
        for (int c = 0; c < C; c += 4) {
            const float4 v = load4_peer(at + ((i * C + c) * NT + 4 * threadIdx.x), r);
            row[c] = fmaf(w, v.x, row[c]);
            row[c + 1] = fmaf(w, v.y, row[c + 1]);
            row[c + 2] = fmaf(w, v.z, row[c + 2]);
            row[c + 3] = fmaf(w, v.w, row[c + 3]);
        }
    }
}
// Zeroes columns [from, to) of every row.
template <int NT> __device__ __forceinline__ void zero_columns(float *dst, int ld, int from, int to, int rows) {
    const int w = to - from;
    for (int i = threadIdx.x; i < rows * w; i += NT) dst[(i / w) * ld + from + i % w] = 0.f;
}

// acc[i][j] += sum_c A[I ty + i][c] * B[tx + 16 j][c] over c < d4 (a multiple of 4).
template <int I, int J>
__device__ __forceinline__ void tile_dot(float (&acc)[I][J], const float *A, int lda, const float *B, int ldb, int d4,
                                         int ty, int tx) {
    float4 x[I], y[J];
#pragma unroll
    for (int i = 0; i < I; ++i) x[i] = *reinterpret_cast<const float4 *>(A + (I * ty + i) * lda);
#pragma unroll
    for (int j = 0; j < J; ++j) y[j] = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * ldb);
#pragma unroll 4
    for (int c = 4; c <= d4; c += 4) {  // the next four channels' loads run behind these products (the last ones read padding)
        float4 u[I], v[J];
#pragma unroll
        for (int i = 0; i < I; ++i) u[i] = *reinterpret_cast<const float4 *>(A + (I * ty + i) * lda + c);
#pragma unroll
        for (int j = 0; j < J; ++j) v[j] = *reinterpret_cast<const float4 *>(B + (tx + 16 * j) * ldb + c);
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
                acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
                acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
                acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
            }
#pragma unroll
        for (int i = 0; i < I; ++i) x[i] = u[i];
#pragma unroll
        for (int j = 0; j < J; ++j) y[j] = v[j];
    }
}

// Columns of a row of `width`: pieces of 64, four neighbours a thread (of 16), then one of 32 with two a thread where
// that covers the rest.  Column c of the sums of the thread at place tx; `width` itself when there is none.
__device__ __forceinline__ int full_pieces(int width) { return (width + 31) / 64; }
__device__ __forceinline__ int apply_column(int c, int width, int tx) {
    const int full = full_pieces(width);
    if (c < 4 * full) return (c >> 2) * 64 + 4 * tx + (c & 3);
    return c < 4 * full + 2 ? 64 * full + 2 * tx + (c & 1) : width;
}

// acc[i][c] += sum_r P[I ty + i][r] * B[r][column c] over r < 64, of N pieces of 64 columns and TAIL of 32.
template <int N, int TAIL, int I, int C>
__device__ __forceinline__ void tile_apply_n(float (&acc)[I][C], const float *P, int ldp, const float *B, int ldb, int ty, int tx) {
    constexpr int M = N + TAIL;
    float4 b[M], next[M];
    auto fetch = [&](float4 (&to)[M], int r) {
#pragma unroll
        for (int j = 0; j < N; ++j) to[j] = *reinterpret_cast<const float4 *>(B + r * ldb + 64 * j + 4 * tx);
        if constexpr (TAIL) {
            const float2 t = *reinterpret_cast<const float2 *>(B + r * ldb + 64 * N + 2 * tx);
            to[N].x = t.x, to[N].y = t.y;
        }
    };
    fetch(b, 0);
#pragma unroll 2
    for (int r = 0; r < 64; r += 4) {
        float4 p[I];
#pragma unroll
        for (int i = 0; i < I; ++i) p[i] = *reinterpret_cast<const float4 *>(P + (I * ty + i) * ldp + r);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            fetch(next, min(r + e + 1, 63));  // behind this row's products
#pragma unroll
            for (int j = 0; j < M; ++j)
#pragma unroll
                for (int i = 0; i < I; ++i) {
                    const float w = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
                    acc[i][4 * j] = fmaf(w, b[j].x, acc[i][4 * j]);
                    acc[i][4 * j + 1] = fmaf(w, b[j].y, acc[i][4 * j + 1]);
                    if (j == N) continue;
                    acc[i][4 * j + 2] = fmaf(w, b[j].z, acc[i][4 * j + 2]);
                    acc[i][4 * j + 3] = fmaf(w, b[j].w, acc[i][4 * j + 3]);
                }
#pragma unroll
            for (int j = 0; j < M; ++j) b[j] = next[j];
        }
    }
}

// The same for the columns below `width` (at most 16 C).  Threads whose columns lie behind `width` read what pads a
// row, or what follows it, and make sums that nobody stores: a test inside the loops keeps their loads from running
// ahead (16,500 cycles a 32 x 64 tile of 80 channels with one, 4,700 without, of 128 columns then).
template <int I, int C, int N = 0>
__device__ __forceinline__ void tile_apply(float (&acc)[I][C], const float *P, int ldp, const float *B, int ldb, int width, int ty, int tx) {
    if constexpr (4 * N < C) {
        if (width > 64 * N + 32) return tile_apply<I, C, N + 1>(acc, P, ldp, B, ldb, width, ty, tx);
        if (width > 64 * N) return tile_apply_n<N, 1>(acc, P, ldp, B, ldb, ty, tx);
    }
    if constexpr (N > 0) tile_apply_n<N, 0>(acc, P, ldp, B, ldb, ty, tx);
}

}  // namespace kda
