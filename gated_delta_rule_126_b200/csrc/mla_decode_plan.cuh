// How mla_decode cuts its work.  An item is (sequence b, tile of query rows); its keys are
// cut into tiles.  The tiles of all items, in the order (b, row tile, key tile), are dealt
// to the blocks in equal contiguous runs: block g of G takes tiles [g W / G, (g+1) W / G) of
// W, so every block has the same work however uneven the sequences are.  A run covers whole
// items except at its ends; a block writes the part of an item that it shares with other
// blocks (at most two: its first and its last) to the workspace as (running maximum, sum,
// unnormalised output), and a second kernel joins the parts.  Everything follows from
// seq_lens on the device, by a fixed rule.
#pragma once

#include "mla_internal.h"

namespace kda {

// What block g of the main kernel leaves for the join, at the front of the workspace.
struct MlaJoin {
    int32_t parts;  // blocks that share the item that begins inside block g's run and ends behind it; 0: none
    int32_t b;
    int32_t row_tile;
    int32_t first_slot;  // slot of block g's part; the following blocks' parts are in slot 2 (g + i)
};

__host__ __device__ inline size_t mla_meta_bytes(int grid) { return (size_t(grid) * sizeof(MlaJoin) + 255) & ~size_t(255); }
// Slot: row_tile rows of dc floats, then row_tile (maximum, sum) pairs.
__host__ __device__ inline size_t mla_slot_floats(int row_tile, int dc) { return size_t(row_tile) * (dc + 2); }

struct MlaRun {
    int64_t total, start, end;  // tiles of the whole call; this block's run
    int grid;                   // blocks that have work: min(grid, total)
    int b;                      // sequence of tile `start`
    int64_t before;             // tiles of the sequences before b
};

__device__ __forceinline__ int mla_len(const MlaDecodeArgs &a, int b) {
    const int64_t most = int64_t(a.max_pages) * a.page_size;
    const int L = a.seq_lens[b];
    return L < 0 ? 0 : (L > most ? int(most) : L);
}

// Called by every thread of a block of NT threads; `buf` is shared scratch of NT / 32 + 4 int64.
template <int NT>
__device__ MlaRun mla_find_run(const MlaDecodeArgs &a, int row_tiles, int key_tile, int64_t *buf) {
    const int per = (a.B + NT - 1) / NT;
    const int b0 = threadIdx.x * per, b1 = min(a.B, b0 + per);
    int64_t own = 0;
    for (int b = b0; b < b1; ++b) own += (mla_len(a, b) + key_tile - 1) / key_tile;
    own *= row_tiles;
    int64_t scan = own;  // inclusive over the warp, then over the block
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
    MlaRun r;
    r.total = total;
    r.grid = int(total < gridDim.x ? total : gridDim.x);
    r.start = r.end = 0;
    r.b = 0;
    r.before = 0;
    if (int(blockIdx.x) < r.grid) {
        r.start = int64_t(blockIdx.x) * total / r.grid;
        r.end = (int64_t(blockIdx.x) + 1) * total / r.grid;
        if (own > 0 && scan - own <= r.start && r.start < scan) {  // tile `start` is in this thread's sequences
            int64_t at = scan - own;
            int b = b0;
            for (; b < b1; ++b) {
                const int64_t nt = int64_t((mla_len(a, b) + key_tile - 1) / key_tile) * row_tiles;
                if (r.start < at + nt) break;
                at += nt;
            }
            buf[NT / 32] = b;
            buf[NT / 32 + 1] = at;
        }
    }
    __syncthreads();
    if (int(blockIdx.x) < r.grid) {
        r.b = int(buf[NT / 32]);
        r.before = buf[NT / 32 + 1];
    }
    return r;
}

// The block whose run holds tile x.
__device__ __forceinline__ int mla_block_of(int64_t x, int64_t total, int grid) {
    return int(((x + 1) * grid - 1) / total);
}

}  // namespace kda
