// mla_decode on the tensor cores (bf16, d_latent a multiple of 128, d_rope 0 or 64).
//
// A block holds RB = 32 or 64 query rows (token, head) and streams the cache in tiles of 64
// rows.  Both products read the same tile in shared memory:
//   S [64 x 64]          = Q [RB x W]  K^T        (K the tile, K-major, W = d_latent + d_rope)
//   O^T [d_latent x RB] += K[:, :d_latent]^T P^T   (the tile again, MN-major; P K-major)
// The output is kept transposed because RB rows of 512 float32 channels would fill all of TMEM
// as [RB x 512] with M = 128, while as d_latent / 128 blocks of [128 x RB] they take 4 RB columns.
// Bound by memory: a tile is 73,728 bytes and an SM's share of the bandwidth brings it in about
// 3,000 cycles; two tiles are in flight.
//
// Warps 0-3: softmax (row i of S lies in lane i % 16 of warp i / 16, the M = 64 layout), rescaling
// and output; warp 4: matrix instructions; warp 5: TMA loads through the page table.  S is double buffered, so the next tile's
// scores are formed while this one's softmax runs.
#include <cmath>

#include "mla_decode_plan.cuh"
#include "mla_tc.cuh"

namespace kda {
namespace {

constexpr int kThreads = 192;
constexpr int kKeys = 64;
constexpr int kMaxStages = 8;
constexpr uint32_t kTmemColumns = 512;
constexpr float kLog2e = 1.4426950408889634f;
// The running maximum that scales P and O is raised only when the true one has outgrown it by
// 2^8: sums stay exact in float32 (P <= 256), and rescaling O becomes rare.
constexpr float kLazy = 8.f;

struct Misc {
    uint64_t full[kMaxStages], empty[kMaxStages], s_full[2], p_full, pv_done, q_full, q_empty, drain;
    uint64_t mask[kMaxStages];  // which keys of the stage lie on a page of the pool
    float factor[64];
    uint32_t tmem, dead;
};
constexpr size_t kMiscBytes = 1024;
static_assert(sizeof(Misc) <= kMiscBytes, "misc");

struct Layout {
    int chunks, stages;  // 64-channel chunks of a row; tiles in flight
    uint32_t stage_bytes, q, p, misc, total;
};
__host__ __device__ inline Layout layout(int W, int rb) {
    Layout L;
    L.chunks = W / 64;
    L.stage_bytes = uint32_t(L.chunks) * 8192u;
    const uint32_t fixed = uint32_t(L.chunks) * rb * 128u + 8192u + uint32_t(kMiscBytes);  // Q, P (read to 64 rows), misc
    const uint32_t room = 232448u - 1024u - fixed;
    L.stages = int(room / L.stage_bytes);
    if (L.stages > kMaxStages) L.stages = kMaxStages;
    L.q = L.stages * L.stage_bytes;
    L.p = L.q + uint32_t(L.chunks) * rb * 128u;
    L.misc = L.p + 8192u;
    L.total = L.misc + uint32_t(kMiscBytes) + 1024u;
    return L;
}

struct Maps {
    CUtensorMap cache, q;
};

// Channel blocks of O^T for tile rows of RB: column of block i.
template <int RB> struct Tm {
    static constexpr uint32_t kS = 4 * RB;  // S buffers of 64 columns behind O
};

template <int RB>
__global__ void __launch_bounds__(kThreads, 1)
decode_tc_kernel(const __grid_constant__ Maps maps, const MlaDecodeArgs a, const MlaDecodeShape shape, const int box) {
    extern __shared__ uint8_t raw[];
    __shared__ int64_t buf[kThreads / 32 + 4];
    const uint32_t base = (ptx::smem_u32(raw) + 1023u) & ~1023u;
    uint8_t *sm = raw + (base - ptx::smem_u32(raw));
    const int W = a.dc + a.dr, R = a.n * a.H, blocks = a.dc / 128;
    const Layout L = layout(W, RB);
    Misc &mi = *reinterpret_cast<Misc *>(sm + L.misc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = blockIdx.x / shape.row_tiles, rt = blockIdx.x % shape.row_tiles, r0 = rt * RB, rows = min(RB, R - r0);

    if (tid == 0) {
        for (int i = 0; i < L.stages; ++i) ptx::mbar_init(&mi.full[i], 1), ptx::mbar_init(&mi.empty[i], 1);
        ptx::mbar_init(&mi.s_full[0], 1);
        ptx::mbar_init(&mi.s_full[1], 1);
        ptx::mbar_init(&mi.p_full, 128);
        ptx::mbar_init(&mi.pv_done, 1);
        ptx::mbar_init(&mi.q_full, 1);
        ptx::mbar_init(&mi.q_empty, 1);
        ptx::mbar_init(&mi.drain, 1);
        mi.dead = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 5 && lane == 0) ptx::prefetch_tmap(&maps.cache), ptx::prefetch_tmap(&maps.q);
    if (warp == 4) {
        ptx::tmem_alloc(&mi.tmem, kTmemColumns);
        ptx::tmem_relinquish();
    }
    const MlaRun run = mla_find_run<kThreads>(a, group, shape.groups, kKeys, buf);
    mla_empty_sequences<__nv_bfloat16, kThreads>(a, group, shape.groups, r0, rows);
    if (tid == 0) static_cast<MlaJoin *>(a.workspace)[blockIdx.x].parts = 0;
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = mi.tmem;
    volatile uint32_t *dead = &mi.dead;

    if (group < run.groups) {
        if (warp == 5) {
            // ---------------------------------------------------------------- loads
            const int boxes = kKeys / box;  // of one tile, each inside a page
            const int rows_total = a.num_pages * a.page_size;
            const uint64_t bits = box == 64 ? ~0ull : (1ull << box) - 1;
            int stage = 0, issued = 0;
            uint32_t round = 0, items = 0;
            bool ok = true;
            MlaWalk w(run);
            while (ok && w.next(a, kKeys, run)) {
                // the row of this lane's box of tile t, or one behind the pool (read as zeros)
                auto lookup = [&](int t) {
                    int row = rows_total;
                    const int key = t * kKeys + lane * box;
                    if (lane < boxes && t < w.t1 && key < w.len) {
                        const int page = a.page_table[int64_t(w.b) * a.max_pages + key / a.page_size];
                        if (page >= 0 && page < a.num_pages) row = page * a.page_size + key % a.page_size;
                    }
                    return row;
                };
                int row = lookup(w.t0);
                if (items) ok = tc::wait(&mi.q_empty, (items - 1) & 1, dead);
                if (!ok) break;
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(&mi.q_full, uint32_t(L.chunks) * RB * 128u);
                    for (int c = 0; c < L.chunks; ++c)
                        tc::tma_load_2d(base + L.q + c * RB * 128, &maps.q, &mi.q_full, 64 * c, w.b * R + r0);
                }
                ++items;
                for (int t = w.t0; t < w.t1; ++t) {
                    const int next = lookup(t + 1);
                    if (round && !(ok = tc::wait(&mi.empty[stage], (round - 1) & 1, dead))) break;
                    const uint32_t good = __ballot_sync(0xffffffffu, row != rows_total);
                    if (lane == 0) {
                        uint64_t m = 0;
                        for (int i = 0; i < boxes; ++i)
                            if (good >> i & 1) m |= bits << (i * box);
                        mi.mask[stage] = m;
                        ptx::mbar_arrive_expect_tx(&mi.full[stage], L.stage_bytes);
                    }
                    __syncwarp();
                    for (int i = lane; i < ((boxes * L.chunks + 31) & ~31); i += 32) {
                        const int at = __shfl_sync(0xffffffffu, row, i % boxes);
                        if (i < boxes * L.chunks)
                            tc::tma_load_2d(base + stage * L.stage_bytes + (i / boxes) * 8192 + (i % boxes) * box * 128,
                                            &maps.cache, &mi.full[stage], 64 * (i / boxes), at);
                    }
                    row = next;
                    ++issued;
                    if (++stage == L.stages) stage = 0, ++round;
                }
            }
            if (!ok && lane == 0) {  // an error: the copies in flight land before the block ends
                for (int i = max(0, issued - L.stages); i < issued; ++i)
                    ptx::mbar_wait_bounded(&mi.full[i % L.stages], (i / L.stages) & 1, tc::kWaitCycles);
                if (items) ptx::mbar_wait_bounded(&mi.q_full, (items - 1) & 1, tc::kWaitCycles);
            }
        } else if (warp == 4) {
            // ---------------------------------------------------------------- products
            constexpr uint32_t kIdS = tc::idesc(64, kKeys, false, false), kIdO = tc::idesc(128, RB, true, false);
            const uint64_t q_desc = ptx::sdesc_sw128(base + L.q), p_desc = ptx::sdesc_sw128(base + L.p),
                           k_desc = ptx::sdesc_sw128(base), v_desc = ptx::sdesc_sw128_mn(base, 8192, 1024);
            if (tc::elect()) {
                // Scores run up to two tiles ahead of O's products (two S buffers), as tiles arrive;
                // whichever of the two can go next goes, so neither waits for the other's input.
                MlaWalk ws(run), wp(run);
                bool more = ws.next(a, kKeys, run), ok = true;
                wp.next(a, kKeys, run);
                int s_tile = ws.t0, p_tile = wp.t0, s_stage = 0, p_stage = 0;
                uint32_t s_round = 0, s_item = 0, n_s = 0, n_pv = 0;
                const uint32_t n_all = uint32_t(run.end - run.start);
                long long since = clock64();
                while (n_pv < n_all) {
                    bool idle = true;
                    if (more && n_s - n_pv < 2 && (s_tile != ws.t0 || ptx::mbar_try_wait(&mi.q_full, s_item & 1)) &&
                        ptx::mbar_try_wait(&mi.full[s_stage], s_round & 1)) {
                        ptx::tc_fence_after();
                        uint64_t qd = q_desc, kd = tc::moved(k_desc, s_stage * L.stage_bytes);
                        const uint32_t to = tmem + Tm<RB>::kS + (n_s & 1) * 64;
                        ptx::mma_ss(to, qd, kd, kIdS, 0);
#pragma unroll
                        for (int k = 1; k < 4; ++k) ptx::mma_ss(to, tc::moved(qd, 32 * k), tc::moved(kd, 32 * k), kIdS, 1);
                        for (int c = 1; c < L.chunks; ++c) {
                            qd = tc::moved(qd, RB * 128);
                            kd = tc::moved(kd, 8192);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                ptx::mma_ss(to, tc::moved(qd, 32 * k), tc::moved(kd, 32 * k), kIdS, 1);
                        }
                        ptx::mma_commit(&mi.s_full[n_s & 1]);
                        ++n_s;
                        if (++s_stage == L.stages) s_stage = 0, ++s_round;
                        if (++s_tile == ws.t1) {
                            ptx::mma_commit(&mi.q_empty);
                            more = ws.next(a, kKeys, run);
                            s_tile = ws.t0;
                            ++s_item;
                        }
                        idle = false;
                    }
                    if (n_s > n_pv && ptx::mbar_try_wait(&mi.p_full, n_pv & 1)) {
                        ptx::tc_fence_after();
                        uint64_t vd = tc::moved(v_desc, p_stage * L.stage_bytes);
                        const uint32_t more_o = p_tile > wp.t0;
                        for (int i = 0; i < blocks; ++i, vd = tc::moved(vd, 16384)) {
                            ptx::mma_ss(tmem + i * RB, vd, p_desc, kIdO, more_o);
#pragma unroll
                            for (int k = 1; k < 4; ++k)
                                ptx::mma_ss(tmem + i * RB, tc::moved(vd, 2048 * k), tc::moved(p_desc, 32 * k), kIdO, 1);
                        }
                        ptx::mma_commit(&mi.empty[p_stage]);
                        ptx::mma_commit(&mi.pv_done);
                        ++n_pv;
                        if (++p_stage == L.stages) p_stage = 0;
                        if (++p_tile == wp.t1) {
                            wp.next(a, kKeys, run);
                            p_tile = wp.t0;
                        }
                        idle = false;
                    }
                    if (!idle) {
                        since = clock64();
                    } else if (*dead || clock64() - since > tc::kWaitCycles) {
                        if (!*dead) atomicExch(&mla_fault, 1u);
                        *dead = 1;
                        ok = false;
                        break;
                    }
                }
                if (!ok) {  // an error: the products in flight end before TMEM goes away
                    ptx::mma_commit(&mi.drain);
                    ptx::mbar_wait_bounded(&mi.drain, 0, tc::kWaitCycles);
                }
            }
            __syncwarp();
        } else {
            // ---------------------------------------------------------------- softmax, rescaling, output
            const uint32_t lanes = uint32_t(warp) << 21;  // TMEM lane 32 warp
            const int row = warp * 16 + lane;             // query row of this thread when lane < 16
            const bool mine = lane < 16 && row < rows;
            const int hidden = mine ? a.n - 1 - (r0 + row) / a.H : 0;  // last keys that this row's token does not see
            const float sl2 = a.scale * kLog2e;
            float *slots = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + mla_meta_bytes(gridDim.x));
            int stage = 0;
            uint32_t round = 0, n_s = 0, n_pv = 0;
            bool ok = true;
            MlaWalk w(run);
            while (ok && w.next(a, kKeys, run)) {
                float top = -INFINITY, sum = 0.f;  // the scale's maximum (raw scores) and the row's sum
                for (int t = w.t0; t < w.t1; ++t) {
                    // a wait that fails is voted on below: no warp leaves the others at a barrier
                    ok = tc::wait(&mi.s_full[n_s & 1], (n_s >> 1) & 1, dead) && ok;
                    ok = tc::wait(&mi.full[stage], round & 1, dead) && ok;  // complete: orders mask and rows
                    ptx::tc_fence_after();
                    uint32_t s0[32], s1[32];
                    const uint32_t sa = tmem + lanes + Tm<RB>::kS + (n_s & 1) * 64;
                    ptx::tmem_ld32(sa, s0);
                    ptx::tmem_ld32(sa + 32, s1);
                    const int left = w.len - t * kKeys, seen = mine ? left - hidden : 0;
                    uint64_t mask = mi.mask[stage];
                    mask &= seen >= 64 ? ~0ull : seen <= 0 ? 0ull : (1ull << seen) - 1;
                    if (left < kKeys) {
                        // rows behind the sequence may hold anything: as values they have to be zero
                        const int rows0 = max(left, 0), per = (kKeys - rows0) * 8;
                        for (int i = tid; i < per * (a.dc / 64); i += 128) {
                            const int c = i / per, at = rows0 * 8 + i % per;
                            tc::st_shared_v4(base + stage * L.stage_bytes + c * 8192 + at * 16, 0, 0, 0, 0);
                        }
                    }
                    ptx::tmem_wait_ld();
                    if (mask != ~0ull) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (!(mask >> i & 1)) s0[i] = 0xff800000u;
                            if (!(mask >> (i + 32) & 1)) s1[i] = 0xff800000u;
                        }
                    }
                    float m = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 32; ++i) m = fmaxf(m, fmaxf(__uint_as_float(s0[i]), __uint_as_float(s1[i])));
                    m = fmaxf(m, top);
                    bool raise = false;
                    float keep = 1.f;
                    if (top == -INFINITY) {
                        top = m;  // nothing summed yet
                    } else if ((m - top) * sl2 > kLazy) {
                        keep = ptx::ex2_approx((top - m) * sl2);
                        sum *= keep;
                        top = m;
                        raise = true;
                    }
                    const float off = top == -INFINITY ? 0.f : top * sl2;
                    uint32_t p[32];
                    float add = 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float x = ptx::ex2_approx(fmaf(__uint_as_float(s0[2 * i]), sl2, -off));
                        const float y = ptx::ex2_approx(fmaf(__uint_as_float(s0[2 * i + 1]), sl2, -off));
                        const float z = ptx::ex2_approx(fmaf(__uint_as_float(s1[2 * i]), sl2, -off));
                        const float u = ptx::ex2_approx(fmaf(__uint_as_float(s1[2 * i + 1]), sl2, -off));
                        p[i] = tc::pack_bf16(x, y);
                        p[i + 16] = tc::pack_bf16(z, u);
                        add += (x + y) + (z + u);
                    }
                    sum += add;
                    // the last product has read P and added to O
                    if (n_pv) ok = tc::wait(&mi.pv_done, (n_pv - 1) & 1, dead) && ok;
                    if (ptx::named_barrier_or(1, 128, raise || !ok)) {
                        if (lane < 16) mi.factor[row] = keep;
                        if (ptx::named_barrier_or(1, 128, !ok)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        for (int i = 0; i < blocks; ++i)
#pragma unroll
                            for (int c = 0; c < RB; c += 32) {
                                uint32_t v[32];
                                ptx::tmem_ld32(tmem + lanes + i * RB + c, v);
                                ptx::tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    v[e] = __float_as_uint(__uint_as_float(v[e]) * mi.factor[c + e]);
                                ptx::tmem_st32(tmem + lanes + i * RB + c, v);
                            }
                        ptx::tmem_wait_st();
                    }
                    if (lane < 16 && row < RB) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            tc::st_shared_v4(base + L.p + row * 128 + ((i ^ (row & 7)) << 4), p[4 * i], p[4 * i + 1],
                                             p[4 * i + 2], p[4 * i + 3]);
                    }
                    ptx::fence_proxy_async_smem();
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&mi.p_full);
                    ++n_s;
                    ++n_pv;
                    if (++stage == L.stages) stage = 0, ++round;
                }
                if (ok) ok = tc::wait(&mi.pv_done, (n_pv - 1) & 1, dead);
                if (ptx::named_barrier_or(1, 128, !ok)) break;  // and factor is free
                const bool whole = w.whole();
                float *slot = slots + mla_slot(w) * mla_slot_floats(RB, a.dc);
                if (lane < 16 && row < RB) {
                    mi.factor[row] = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
                    if (!whole) {
                        slot[RB * a.dc + 2 * row] = top == -INFINITY ? top : top * a.scale;
                        slot[RB * a.dc + 2 * row + 1] = sum;
                    } else if (a.lse && mine) {
                        a.lse[int64_t(w.b) * R + r0 + row] = sum == 0.f ? -INFINITY : top * a.scale + logf(sum);
                    }
                }
                if (tid == 0 && !whole && w.t0 == 0)
                    static_cast<MlaJoin *>(a.workspace)[blockIdx.x] = mla_join_entry(w, run, group);
                ptx::named_barrier(1, 128);
                ptx::tc_fence_after();
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.o) + (int64_t(w.b) * R + r0) * a.dc;
                for (int i = 0; i < blocks; ++i)
#pragma unroll
                    for (int c = 0; c < RB; c += 32) {
                        uint32_t v[32];
                        ptx::tmem_ld32(tmem + lanes + i * RB + c, v);
                        ptx::tmem_wait_ld();
                        const int ch = i * 128 + warp * 32 + lane;  // lane of TMEM: the channel
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float x = __uint_as_float(v[e]) * mi.factor[c + e];
                            if (!whole) slot[size_t(c + e) * a.dc + ch] = x;
                            else if (c + e < rows) out[size_t(c + e) * a.dc + ch] = __float2bfloat16_rn(x);
                        }
                    }
                ptx::tc_fence_before();
            }
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, kTmemColumns);
    }
}

// Rows of one TMA box: the largest power of two up to 64 that divides a page.
int box_rows(int page_size) {
    int b = 64;
    while (page_size % b) b /= 2;
    return b;
}

template <int RB>
cudaError_t launch(const Maps &maps, const MlaDecodeArgs &a, const MlaDecodeShape &s, int box, cudaStream_t st) {
    const Layout L = layout(a.dc + a.dr, RB);
    const cudaError_t e = cudaFuncSetAttribute(decode_tc_kernel<RB>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(L.total));
    if (e != cudaSuccess) return e;
    decode_tc_kernel<RB><<<s.grid(), kThreads, L.total, st>>>(maps, a, s, box);
    return cudaGetLastError();
}

}  // namespace

// Boxes of at least 8 rows keep the swizzle's phase, so pages have to be multiples of 8; the
// running maximum is taken before scaling, so the scale has to be positive; row numbers are 32-bit.
bool mla_decode_tc_supported(const MlaDecodeArgs &a) {
    return a.dtype == KDA_DTYPE_BF16 && a.dc % 128 == 0 && (a.dr == 0 || a.dr == 64) && a.page_size % 8 == 0 &&
           a.scale > 0.f && a.num_pages > 0 && int64_t(a.num_pages) * a.page_size < INT32_MAX &&
           int64_t(a.B) * a.n * a.H < INT32_MAX;
}

// 32 rows where the call has no more (one token of up to 32 heads), else 64; one block per SM.
MlaDecodeShape mla_decode_tc_shape(int n, int H) {
    const int R = n * H, rb = R <= 32 ? 32 : 64, tiles = R > 0 ? (R + rb - 1) / rb : 1, groups = device_sm_count() / tiles;
    return MlaDecodeShape{true, rb, tiles, groups > 1 ? groups : 1};
}

cudaError_t launch_mla_decode_tc(const MlaDecodeArgs &a, const MlaDecodeShape &s, cudaStream_t st) {
    const int64_t W = a.dc + a.dr;
    const int box = box_rows(a.page_size);
    Maps maps;
    const int64_t cache_dims[2] = {W, int64_t(a.num_pages) * a.page_size}, q_dims[2] = {W, int64_t(a.B) * a.n * a.H};
    const int cache_box[2] = {64, box}, q_box[2] = {64, s.row_tile};
    if (!tc::make_map(&maps.cache, a.cache, 2, cache_dims, &W, cache_box) ||
        !tc::make_map(&maps.q, a.q, 2, q_dims, &W, q_box))
        return cudaErrorInvalidValue;
    return s.row_tile == 32 ? launch<32>(maps, a, s, box, st) : launch<64>(maps, a, s, box, st);
}

cudaError_t mla_decode_fault(cudaStream_t st, unsigned int *out) { return mla_fault_read(st, out); }

}  // namespace kda
