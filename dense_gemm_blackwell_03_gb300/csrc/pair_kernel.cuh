// pair_kernel.cuh -- the large products of the gated feed-forward layer on 16-bit
// operands (bf16 or fp16) with fp32 sums:
//
//   kPairGated      G = X Wg^T, U = X Wu^T, H = act(G) * U     forward, in one pass
//   kPairBackward   dX = dG Wg + dU Wu                          input gradient, and
//                   dWg = dG^T X,  dWu = dU^T X                 weight gradients, in one launch
//
// One persistent, warp-specialised tcgen05 kernel, tiles of 256 x 256 on CTA pairs (or
// 128 x 128 on single CTAs for the gradients of small layers).  tcgen05 reads either
// major order, so no operand is transposed in memory: dX reads the weights as they are
// stored (columns of a row are outputs), dW both operands.
//
// Gated: the pair's MMA takes 256 rows of B, half of them from either CTA's shared
// memory.  The even CTA brings 128 rows of Wg, the odd one the same rows of Wu, so
// each accumulator row holds G in its first 128 columns and U in the last: every
// epilogue thread has both values of its outputs, and X's tile is read once for both.
//
// Backward: all tiles are one list of work, dX's first (its K is 2 N deep) and the weights'
// after them, so that no wave is left partly filled between the two.  dX sums both products
// in one accumulator (the K loop runs over dG, Wg, then over dU, Wu).  Few tiles and a deep
// K: slices of K, whose fp32 sums a second kernel adds in order.
//
// What bounds it: the MMAs, 1024 cycles per 128 of K of a 256 x 256 tile; the epilogue
// of a tile (other TMEM buffer) overlaps the next tile's.  Measured: gated 8192 x 28672 x 8192
// 4220 to 4470 us (1.72 to 1.82 PFLOP/s, the sustained rate under the power cap), tensor pipe 88 %
// active on 4096 x 8192 x 2048; gradients of 4096 x 28672 x 8192 4530 to 4820 us with the pass
// that makes dG and dU (1.60 to 1.70), tensor pipe 87 % active on 2048 x 4096 x 2048.  Each stage of
// the ring holds 128 of K of both operands (64 KiB per CTA), one 32 KiB copy each where the box lies
// in whole 64-element chunks, two of 16 KiB at a row's end (TMA fills zeros past it).
#pragma once

#include "activation.cuh"
#include "feed_forward.h"
#include "ortho_kernel.cuh"

namespace bwgemm {

struct PairTile {
    int which, r, c, result;  // of product `which`
    int k0, k1;
};

__device__ __forceinline__ PairTile pair_tile_at(const PairParams& p, int t)
{
    PairTile x;
    x.which = t >= p.prod[0].units ? 1 : 0;
    const PairProduct& d = p.prod[x.which];
    t -= x.which ? p.prod[0].units : 0;
    const int i = t / d.splits, slice = t - i * d.splits;
    x.k0 = 0;
    x.k1 = d.steps;
    if (d.splits > 1) {
        x.k0 = int(int64_t(slice) * d.steps / d.splits);
        x.k1 = int(int64_t(slice + 1) * d.steps / d.splits);
    }
    // groups of 8 tile rows (of all results), walked down before stepping along the columns
    const int rows = d.num_r * d.results;
    const int per_group = 8 * d.num_c;
    const int g = i / per_group;
    const int height = min(rows - 8 * g, 8);
    const int local = i - g * per_group;
    const int r = 8 * g + local % height;
    x.c = local / height;
    x.result = r / d.num_r;
    x.r = r - x.result * d.num_r;
    return x;
}

// The i-th unit of a worker, of `total`.  dX's units (the first product's) are dealt in turn; then those
// who got none in the last turn take `early` of the weights' tiles each, as one of dX's units
// is many times their length, and all take the rest in turn.
__device__ __forceinline__ int pair_unit(const PairParams& p, int worker, int workers, int i)
{
    const int first = p.prod[0].units, rest = first % workers;
    const int mine = first / workers + (worker < rest ? 1 : 0);
    if (i < mine)
        return worker + i * workers;
    i -= mine;
    if (worker >= rest) {
        if (i < p.early)
            return first + worker - rest + i * (workers - rest);
        i -= p.early;
    }
    return first + p.early * (workers - rest) + worker + i * workers;
}

// A worker's units one after the other.  The divisions that find a tile take as long as a step's
// MMAs: next() after a tile's first step, so that they overlap the rest.
struct PairWalk {
    PairTile x;
    int i = 0, t;
    __device__ __forceinline__ PairWalk(const PairParams& p, int worker, int workers, int total)
    {
        t = pair_unit(p, worker, workers, 0);
        if (t < total)
            x = pair_tile_at(p, t);
    }
    __device__ __forceinline__ void next(const PairParams& p, int worker, int workers, int total)
    {
        t = pair_unit(p, worker, workers, ++i);
        if (t < total)
            x = pair_tile_at(p, t);
    }
};

// A box of 128 rows x 128 elements of an operand: whole chunks in one copy, else chunk by
// chunk (zeros past the row's end, and past the last row).
template <int CG>
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* m, const CUtensorMap* m3, int chunks, uint32_t bar,
                                          int row, int col)
{
    if (col / 64 + 2 <= chunks) {
        if constexpr (CG == 2)
            ptx::tma_load_3d_pair(dst, m3, bar, 0, row, col / 64);
        else
            ptx::tma_load_3d(dst, m3, bar, 0, row, col / 64);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if constexpr (CG == 2)
                ptx::tma_load_2d_pair(dst + uint32_t(i * 16384), m, bar, col + 64 * i, row);
            else
                ptx::tma_load_2d(dst + uint32_t(i * 16384), m, bar, col + 64 * i, row);
    }
}

template <int CG, int FORM>
__global__ void __launch_bounds__(OrthoConfig<CG>::kThreads, 1)
    pair_kernel(const __grid_constant__ PairMaps maps, const PairParams p)
{
    using Cfg = OrthoConfig<CG>;
    static_assert(FORM != kPairGated || CG == 2, "gate and up rows come from the two CTAs");
    constexpr bool B_MN = FORM == kPairBackward;
    constexpr int STAGES = Cfg::kStages;
    constexpr int TILE = Cfg::kTile;
    constexpr int COLS = FORM == kPairGated ? TILE / 2 : TILE;  // result columns of a tile
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? ptx::cluster_ctarank() : 0u;
    const int worker = int(blockIdx.x) / CG;
    const int workers = int(gridDim.x) / CG;
    const int total = p.prod[0].units + (FORM == kPairBackward ? p.prod[1].units : 0);
    const uint32_t sA = base + Cfg::kOffA;
    const uint32_t sB = base + Cfg::kOffB;
    const uint32_t bar_full = base + Cfg::kOffBar;
    const uint32_t bar_empty = bar_full + 8 * STAGES;
    const uint32_t bar_acc_full = bar_empty + 8 * STAGES;
    const uint32_t bar_acc_empty = bar_acc_full + 16;
    const uint32_t bar_drain = bar_acc_empty + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffTmemSlot);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kOffAbort);

    if (threadIdx.x == 64) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(bar_acc_full + 8 * b, 1);
            ptx::mbar_init(bar_acc_empty + 8 * b, CG * Cfg::kEpiWarps);
        }
        ptx::mbar_init(bar_drain, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&maps.a[0]);
        ptx::prefetch_tensormap(&maps.a3[0]);
        ptx::prefetch_tensormap(&maps.b[0]);
        ptx::prefetch_tensormap(&maps.b3[0]);
        ptx::prefetch_tensormap(&maps.out[0]);
    }
    if (warp == 1) {
        ptx::tmem_alloc<CG>(ptx::smem_addr(tmem_slot), Cfg::kTmemCols);
        ptx::tmem_relinquish<CG>();
    }
    ptx::tc_fence_before_sync();
    if constexpr (CG == 2)
        ptx::cluster_sync();
    else
        __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    ptx::launch_dependents();
    uint32_t armed_mask = 0, armed_parity = 0;

    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        const uint32_t leader_full = CG == 2 ? ptx::map_to_cta(bar_full, 0) : bar_full;
        int s = 0, n = 0;
        uint32_t phase = 0;
        bool ok = true;
#pragma unroll 1
        for (PairWalk walk(p, worker, workers, total); ok && walk.t < total;) {
            const PairTile x = walk.x;
            const int a0 = x.r * TILE + int(rank) * 128;
            const int b0 = FORM == kPairGated ? x.c * COLS : x.c * TILE + int(rank) * 128;
#pragma unroll 1
            for (int i = x.k0; i < x.k1; ++i, ++n) {
                ok = warp_wait(bar_empty + 8 * s, phase ^ 1u, p, abort_flag, kStatusProducerTimeout);
                if (!ok)
                    break;
                const bool stall = p.stall_kblock >= 0 && blockIdx.x == 0 && p.stall_kblock == n;
                if (!stall && rank == 0) {
                    armed_mask |= 1u << s;
                    armed_parity = (armed_parity & ~(1u << s)) | (phase << s);
                }
                if (!stall && ptx::elect_one()) {
                    const bool of_w = FORM == kPairBackward && x.which == 1;  // a stored K x rows
                    const int term = FORM == kPairBackward && !of_w && i >= p.steps_k ? 1 : 0;
                    const int k = (i - term * p.steps_k) * kOrthoK;
                    const int za = of_w ? x.result : term;
                    const int zb = FORM == kPairGated ? int(rank) : of_w ? 2 : term;
                    const uint32_t fb = leader_full + 8 * s;
                    const uint32_t dA = sA + uint32_t(s * Cfg::kOperandBytes), dB = sB + uint32_t(s * Cfg::kOperandBytes);
                    if (rank == 0)
                        ptx::mbar_arrive_expect_tx(fb, uint32_t(CG * 2 * Cfg::kOperandBytes));
                    if (n == 0)  // all before it overlaps the kernel before
                        ptx::grid_dependency_wait();
                    pair_load<CG>(dA, &maps.a[za], &maps.a3[za], p.chunks_a, fb, of_w ? k : a0, of_w ? a0 : k);
                    pair_load<CG>(dB, &maps.b[zb], &maps.b3[zb], p.chunks_b, fb, B_MN ? k : b0, B_MN ? b0 : k);
                }
                __syncwarp();
                if (i == x.k0)
                    walk.next(p, worker, workers, total);
                if (++s == STAGES) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------------------------------------------------- MMA issue
        const uint64_t a_k0 = make_sdesc_sw128(sA), a_mn0 = make_sdesc_mn(sA);
        const uint64_t b_desc0 = B_MN ? make_sdesc_mn(sB) : make_sdesc_sw128(sB);
        const uint32_t idesc0 = make_idesc(p.dtype, 128 * CG, TILE) | (B_MN ? 1u << 16 : 0u);
        const uint32_t tmem0 = __shfl_sync(0xffffffffu, tmem_base, 0);
        int s = 0, b = 0;
        uint32_t phase = 0, bphase = 0;
        bool ok = true;
#pragma unroll 1
        for (PairWalk walk(p, worker, workers, total); ok && walk.t < total;) {
            const PairTile x = walk.x;
            ok = warp_wait(bar_acc_empty + 8 * b, bphase ^ 1u, p, abort_flag, kStatusMmaTimeout);
#pragma unroll 1
            for (int i = x.k0; ok && i < x.k1; ++i) {
                ok = warp_wait(bar_full + 8 * s, phase, p, abort_flag, kStatusMmaTimeout);
                if (!ok)
                    break;
                ptx::tc_fence_after_sync();
                if (ptx::elect_one()) {
                    const uint64_t bd = b_desc0 + uint64_t((s * Cfg::kOperandBytes) >> 4);
                    auto issue = [&](uint64_t ad, bool a_mn, uint32_t idesc) {
#pragma unroll
                        for (int kk = 0; kk < kOrthoK / 16; ++kk) {
                            // K-major: two chunks of 64 k, 32 bytes per MMA; MN-major: 128 k in rows of 128 bytes
                            const uint32_t k_major = uint32_t((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                            const uint32_t mn_major = uint32_t(kk * 2048) >> 4;
                            ptx::mma_f16<CG>(tmem0 + uint32_t(b * TILE), ad + (a_mn ? mn_major : k_major),
                                             bd + (B_MN ? mn_major : k_major), idesc, (i > x.k0 || kk > 0) ? 1u : 0u);
                        }
                    };
                    const uint64_t stage = uint64_t((s * Cfg::kOperandBytes) >> 4);
                    if (FORM == kPairBackward && x.which == 1)
                        issue(a_mn0 + stage, true, idesc0 | 1u << 15);
                    else
                        issue(a_k0 + stage, false, idesc0);
                    if constexpr (CG == 2) {
                        ptx::mma_commit_pair(bar_empty + 8 * s, 0x3);
                        if (i == x.k1 - 1)
                            ptx::mma_commit_pair(bar_acc_full + 8 * b, 0x3);
                    } else {
                        ptx::mma_commit(bar_empty + 8 * s);
                        if (i == x.k1 - 1)
                            ptx::mma_commit(bar_acc_full + 8 * b);
                    }
                }
                __syncwarp();
                if (i == x.k0)
                    walk.next(p, worker, workers, total);
                if (++s == STAGES) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (++b == 2) {
                b = 0;
                bphase ^= 1u;
            }
        }
    } else if (warp >= 2) {
        // ------------------------------------------------------------ epilogue
        ptx::grid_dependency_wait();
        const int e = warp - 2;
        const int q = warp & 3;
        const uint32_t sb = base + uint32_t(Cfg::kOffStore + e * Cfg::kStoreBytes);
        int b = 0;
        uint32_t bphase = 0;
        bool ok = true;
        // 64 columns of this lane's row, packed, to columns col.. of rows row0.. of result z
        auto put = [&](const uint32_t (&w)[32], const PairProduct& d, int z, int row0, int col) {
            if (row0 >= d.rows || col >= d.cols)
                return;
            if (lane == 0)
                ptx::bulk_wait_group_read<0>();  // the store before has read the staging block
            __syncwarp();
            ortho_stage(w, sb, lane);
            if ((d.cols & 7) != 0 && col + 64 > d.cols) {
                // a TMA store clips a row's end only in whole 16-byte pieces: eight lanes a row
                __syncwarp();
                const int c = col + 8 * (lane & 7), left = d.cols - c;
#pragma unroll 1
                for (int r = lane >> 3; r < 32 && row0 + r < d.rows; r += 4) {
                    uint4 v;
                    ptx::ld_shared_v4(sb + uint32_t(r * 128 + (((lane ^ r) & 7) << 4)), v.x, v.y, v.z, v.w);
                    uint16_t* dst = p.out[z] + int64_t(row0 + r) * p.ldo[z] + c;
                    if (left >= 8) {
                        *reinterpret_cast<uint4*>(dst) = v;
                    } else {
#pragma unroll
                        for (int i = 0; i < 7; ++i)
                            if (i < left)
                                dst[i] = uint16_t((&v.x)[i / 2] >> (16 * (i % 2)));
                    }
                }
                __syncwarp();
                return;
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                ptx::tma_store_2d(&maps.out[z], sb, col, row0);
                ptx::bulk_commit_group();
            }
        };
#pragma unroll 1
        for (int i = 0, t; ok && (t = pair_unit(p, worker, workers, i)) < total; ++i) {
            const PairTile x = pair_tile_at(p, t);
            const PairProduct& d = p.prod[x.which];
            const int row0 = x.r * TILE + int(rank) * 128 + 32 * q;
            ok = warp_wait(bar_acc_full + 8 * b, bphase, p, abort_flag, kStatusEpilogueTimeout);
            if (!ok)
                break;
            ptx::tc_fence_after_sync();
            const uint32_t taddr = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(b * TILE);
            if constexpr (FORM == kPairGated) {
                const int c0 = (e >> 2) * 64;  // this warp's 64 columns of the tile's 128
                uint32_t h[32], gw[32], uw[32];
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    uint32_t g[32], u[32];
                    ptx::tmem_ld_32x32b_x32(taddr + uint32_t(c0 + c), g);
                    ptx::tmem_ld_32x32b_x32(taddr + uint32_t(COLS + c0 + c), u);
                    ptx::tmem_ld_wait();
                    if (c == 32)
                        hand_back<CG>(bar_acc_empty + 8 * b, lane);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float v[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            v[k] = activate(__uint_as_float(g[2 * i + k]), p.activation) * __uint_as_float(u[2 * i + k]);
                        h[c / 2 + i] = pack2(__float_as_uint(v[0]), __float_as_uint(v[1]), p.dtype);
                        gw[c / 2 + i] = pack2(g[2 * i], g[2 * i + 1], p.dtype);
                        uw[c / 2 + i] = pack2(u[2 * i], u[2 * i + 1], p.dtype);
                    }
                }
                const int col = x.c * COLS + c0;
                put(h, d, 0, row0, col);
                if (p.out[1] != nullptr) {
                    put(gw, d, 1, row0, col);
                    put(uw, d, 2, row0, col);
                }
            } else {
                const int c0 = (e >> 2) * Cfg::kCols;
                if (d.splits == 1) {
#pragma unroll 1
                    for (int c = 0; c < Cfg::kCols; c += 64) {
                        uint32_t v[64], w[32];
                        ptx::tmem_ld_32x32b_x64(taddr + uint32_t(c0 + c), v);
                        ptx::tmem_ld_wait();
                        if (c + 64 >= Cfg::kCols)
                            hand_back<CG>(bar_acc_empty + 8 * b, lane);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            w[i] = pack2(v[2 * i], v[2 * i + 1], p.dtype);
                        put(w, d, x.which + x.result, row0, x.c * TILE + c0 + c);
                    }
                } else {
                    // a slice of K: its sums to global memory, where pair_join_kernel adds
                    // them; lanes next to each other, so a warp's store is 512 bytes
                    float* const part = p.partials + (size_t(t) * CG + rank) * (128 * TILE) + e * (32 * Cfg::kCols) + 4 * lane;
#pragma unroll 1
                    for (int c = 0; c < Cfg::kCols; c += 32) {
                        uint32_t v[32];
                        ptx::tmem_ld_32x32b_x32(taddr + uint32_t(c0 + c), v);
                        ptx::tmem_ld_wait();
                        if (c + 32 >= Cfg::kCols)
                            hand_back<CG>(bar_acc_empty + 8 * b, lane);
                        if (row0 < d.rows && x.c * TILE + c0 + c < d.cols) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                ptx::st_global_cg_v4(part + c * 32 + i * 128,
                                                     make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
                        }
                    }
                }
            }
            if (++b == 2) {
                b = 0;
                bphase ^= 1u;
            }
        }
        if (lane == 0)
            ptx::bulk_wait_group_all();
        __syncwarp();
    }

    // --------------------------------------------------------------- teardown
    // as in the other kernels: after an abort, drain MMAs and loads (bounded)
    // before TMEM and shared memory are released
    __syncwarp();
    __syncthreads();
    if (*abort_flag) {
        if (warp == 1 && rank == 0) {
            if (ptx::elect_one()) {
                if constexpr (CG == 2)
                    ptx::mma_commit_pair(bar_drain, 0x1);
                else
                    ptx::mma_commit(bar_drain);
            }
            __syncwarp();
            drain_wait(bar_drain, 0u, kDrainNs);
        }
        if (warp == 0) {
#pragma unroll 1
            for (int s = 0; s < STAGES; ++s)
                if ((armed_mask >> s) & 1u)
                    drain_wait(bar_full + 8 * s, (armed_parity >> s) & 1u, kDrainNs);
            if (lane == 0)
                settle(kSettleNs);
        }
        __syncwarp();
        __syncthreads();
    }
    ptx::tc_fence_before_sync();
    if constexpr (CG == 2)
        ptx::cluster_sync();
    if (warp == 1) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc<CG>(tmem_base, Cfg::kTmemCols);
    }
}

// Adds the slices of the tiles.  A warp takes 32 rows x 4 columns of a tile (512 bytes
// of a slice) and every join_share-th slice; the sums of that many warps meet in shared
// memory, in order.
template <int CG>
__global__ void __launch_bounds__(32 * kJoinWarps) pair_join_kernel(const PairParams p, int which)
{
    using Cfg = OrthoConfig<CG>;
    constexpr int TILE = Cfg::kTile, CHUNKS = Cfg::kCols / 32;
    __shared__ float4 sums[kJoinWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PairProduct& d = p.prod[which];
    const int share = d.join_share, first = warp % share;
    const int piece = int(blockIdx.x) * (kJoinWarps / share) + warp / share;
    const int i = piece % 8, c = piece / 8 % CHUNKS * 32, e = piece / (8 * CHUNKS) % 8, rank = piece / (64 * CHUNKS);
    const int t = (which ? p.prod[0].units : 0) + int(blockIdx.y) * d.splits;
    const PairTile x = pair_tile_at(p, t);
    const int row0 = x.r * TILE + rank * 128 + 32 * ((e + 2) & 3), row = row0 + lane;
    const int col = x.c * TILE + (e >> 2) * Cfg::kCols + c + 4 * i;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const float* at = p.partials + (size_t(t) * CG + rank) * (128 * TILE) + e * (32 * Cfg::kCols) + c * 32 + i * 128 + 4 * lane;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row0 < d.rows && col < d.cols) {
#pragma unroll 8
        for (int k = first; k < d.splits; k += share) {
            const uint4 v = ptx::ld_global_cg_v4(at + size_t(k) * (CG * 128 * TILE));
            f.x += __uint_as_float(v.x);
            f.y += __uint_as_float(v.y);
            f.z += __uint_as_float(v.z);
            f.w += __uint_as_float(v.w);
        }
    }
    sums[warp][lane] = f;
    __syncthreads();
    if (first != 0)
        return;
#pragma unroll 1
    for (int k = 1; k < share; ++k) {
        const float4 g = sums[warp + k][lane];
        f.x += g.x;
        f.y += g.y;
        f.z += g.z;
        f.w += g.w;
    }
    if (row >= d.rows || col >= d.cols)
        return;
    const uint32_t lo = pack2(__float_as_uint(f.x), __float_as_uint(f.y), p.dtype);
    const uint32_t hi = pack2(__float_as_uint(f.z), __float_as_uint(f.w), p.dtype);
    const int z = which + x.result;
    uint16_t* const out = p.out[z] + row * p.ldo[z] + col;
    if (col + 4 <= d.cols) {
        *reinterpret_cast<uint2*>(out) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (col + k < d.cols)
                out[k] = uint16_t((k < 2 ? lo : hi) >> (k & 1 ? 16 : 0));
    }
}

}  // namespace bwgemm
