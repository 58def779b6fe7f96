// scaled_kernel.cuh -- persistent, warp-specialised tcgen05 product of two
// 8-bit matrices with a scale per block of 128 along K:
//
//   C[m, n] = sum_kb sa[kb, m] * sb[kb, n] * sum_{k in kb} A[m, k] * B[n, k]
//
// The tensor cores know nothing of fp32 scales, so the inner sum of every K
// block is a fresh accumulator in TMEM (128 K elements: the first MMA
// overwrites) and the outer sum lives in the epilogue warps' registers: while
// the MMAs of the next block run into another TMEM buffer, eight warps read
// the finished block and add it, weighted, to their running sums with paired
// fp32 FMAs.  Per 128 x 256 block of a CTA that is 512 cycles of MMA beside
// 256 cycles of TMEM reads and 128 (a scale per 128 columns) or about 320 (one
// per column) issue slots per scheduler, so the tensor pipe stays the bound.
//
//   warp 0      TMA producer: a ring of stages of two K blocks (64 KiB for a
//               256 x 256 pair tile), one 3-D copy per operand and stage -- a
//               copy of two blocks moves about 1.7 times the bytes per second
//               and SM of single-block copies.
//   warp 1      TMEM allocator and (even CTA) MMA issuer: 4 tcgen05.mma of
//               K = 32 per block, kBufs accumulators in turn.
//   the others  epilogue: 8 warps, two per TMEM lane quarter with half the
//               columns each (tiles of 128 and 256 columns), else 4.
//
// The scales reach each epilogue warp through a small ring of its own in shared
// memory filled with 4-byte asynchronous copies a few blocks ahead (across tile
// boundaries too), so neither their latency nor a barrier between warps stands
// in the loop.
//
// Work: the last, partial wave of tiles is spread over all workers in K
// iterations (stream-K).  A worker's piece of a tile goes to an fp32 partial in
// global memory; the warp that completes the tile's K blocks adds the pieces in
// worker order -- the same sum whichever arrives last -- and stores.  Nobody
// waits for anybody.
//
// Swapped form (few rows of A): the weights fill the 128 lanes, A's rows are
// the MMA's N, C leaves through plain stores (a warp's 32 lanes are 32
// consecutive columns of C).
#pragma once

#include "gemm_kernel.cuh"
#include "operators.h"

namespace bwgemm {

template <int CG, int BN, bool SWAP, bool COLVEC>
struct ScaledConfig {
    static constexpr int kKps = kScaledKps;
    static constexpr int kEpiWarps = BN >= 128 ? 8 : 4;
    // 256 columns: 128 running sums per thread need more registers than an even
    // share of the file (168 at ten warps and more).  The launch then has three
    // warpgroups -- producer, MMA and two idle warps in the first -- and the
    // first gives registers to the two of the epilogue: 128 x 56 + 256 x 224 =
    // 64512, the 384 x 168 that the block is launched with (the launch code
    // checks the compiled count).
    static constexpr bool kSplitRegs = BN == 256;
    static constexpr int kFirstEpi = kSplitRegs ? 4 : 2;
    static constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
    static constexpr int kRegsFirst = 56, kRegsEpi = 224;
    static constexpr int kCols = BN >= 128 ? BN / 2 : BN;  // columns per epilogue warp
    static constexpr int kLBlock = kRowsPerCta * kBlock;   // one K block of the lane side: 16 KiB
    static constexpr int kCRows = BN / CG;                 // column-side rows this CTA copies
    static constexpr int kCBlock = kCRows * kBlock;
    static constexpr int kLBytes = kKps * kLBlock;
    static constexpr int kCBytes = kKps * kCBlock;
    static constexpr int kStages = (192 * 1024) / (kLBytes + kCBytes);
    static constexpr int kBufs = BN == 256 ? 2 : 4;        // accumulators in TMEM
    static constexpr int kTmemCols = kBufs * BN;
    static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM allocation");
    // per warp: scale slots of 32 lane scales and the column scales (or 32
    // copies of the one scale of its columns)
    static constexpr int kSlots = COLVEC && BN == 256 ? 3 : 4;
    static constexpr int kSlotBytes = 4 * (32 + (COLVEC ? kCols : 32));
    static constexpr int kStoreBytes = 2048;  // a 64-byte x 32-row output box
    static constexpr int kOffL = 0;
    static constexpr int kOffC = kStages * kLBytes;
    static constexpr int kOffStore = kOffC + kStages * kCBytes;
    static constexpr int kOffScale = kOffStore + (SWAP ? 0 : kEpiWarps * kStoreBytes);
    static constexpr int kOffBar = kOffScale + kEpiWarps * kSlots * kSlotBytes;
    static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 1;  // full, empty, acc_full, acc_empty, drain
    static constexpr int kOffTmemSlot = kOffBar + 8 * kNumBars;
    static constexpr int kOffAbort = kOffTmemSlot + 4;
    static constexpr int kSmemBytes = kOffAbort + 4 + 1024;  // + slack to align the base to 1 KiB
    static_assert(kLBlock % 1024 == 0 && kCBlock % 1024 == 0, "swizzle atoms need 1 KiB alignment");
    static_assert(kOffBar % 8 == 0 && kSlotBytes % 16 == 0, "alignment");
    static_assert(kSmemBytes <= 227 * 1024, "exceeds the 227 KiB shared memory of one CTA");
    static constexpr int kPartialFloats = kRowsPerCta * BN;  // one CTA's partial tile
};

struct ScaledSegment {
    int tile, kb0, kb1;
    int l_blk, c_blk;
    int slot;     // partial slot of the worker (0 or 1)
    bool whole;
};

// The pieces of work of one worker: its share of the stream-K iterations, then
// whole tiles.  Every role walks the same sequence.
struct ScaledIter {
    long long it, it_begin, it_end;
    int t, step;

    static __device__ __forceinline__ long long begin(const ScaledParams& p, int worker, int workers)
    {
        const long long prod = (long long)worker * p.sk_iters;
        return prod < (1ll << 32) ? (long long)(unsigned(prod) / unsigned(workers)) : prod / workers;
    }
    __device__ __forceinline__ void init(const ScaledParams& p, int worker, int workers)
    {
        it_begin = it = begin(p, worker, workers);
        it_end = begin(p, worker + 1, workers);
        t = worker;
        step = workers;
    }
    __device__ __forceinline__ bool next(const ScaledParams& p, ScaledSegment& s)
    {
        if (it < it_end) {
            const int tile = int(it / p.num_kb);
            s.kb0 = int(it - (long long)tile * p.num_kb);
            s.kb1 = int(min((long long)p.num_kb, s.kb0 + (it_end - it)));
            s.whole = s.kb0 == 0 && s.kb1 == p.num_kb;
            s.slot = it == it_begin ? 0 : 1;
            s.tile = p.dp_tiles + tile;
            it += s.kb1 - s.kb0;
        } else if (t < p.dp_tiles) {
            s.tile = t;
            s.kb0 = 0;
            s.kb1 = p.num_kb;
            s.whole = true;
            s.slot = 0;
            t += step;
        } else {
            return false;
        }
        const int per_group = p.raster_group * p.num_c;
        const int group = s.tile / per_group;
        const int first = group * p.raster_group;
        const int height = min(p.num_l - first, p.raster_group);
        const int local = s.tile - group * per_group;
        s.l_blk = first + local % height;
        s.c_blk = local / height;
        return true;
    }
};

__device__ __forceinline__ bool scaled_wait(uint32_t bar, uint32_t parity, const ScaledParams& p,
                                            volatile uint32_t* abort_flag, uint32_t code)
{
    if (ptx::mbar_try_wait(bar, parity))
        return true;
    WaitClock clock;
#pragma unroll 1
    while (true) {
        if (ptx::mbar_try_wait(bar, parity))
            return true;
        if (*abort_flag)
            return false;
        if (clock.expired(p.timeout_ns)) {
            atomicOr(p.status, code);
            *abort_flag = 1u;
            return false;
        }
    }
}

// Fills one epilogue warp's ring of scale slots, K block after K block of the
// warp's segments: slot i % SLOTS holds the i-th block's.
template <int CG, int BN, bool SWAP, bool COLVEC>
struct ScaleFeed {
    using Cfg = ScaledConfig<CG, BN, SWAP, COLVEC>;
    ScaledIter iter;
    ScaledSegment seg;
    int kb, n;
    bool live;

    __device__ __forceinline__ void init(const ScaledParams& p, int worker, int workers)
    {
        iter.init(p, worker, workers);
        live = iter.next(p, seg);
        kb = seg.kb0;
        n = 0;
    }
    // Start the copies of one block's scales (an empty group once all are read).
    __device__ __forceinline__ void issue(const ScaledParams& p, uint32_t ring, int rank, int q, int col, int lane)
    {
        if (live) {
            const uint32_t slot = ring + uint32_t((n % Cfg::kSlots) * Cfg::kSlotBytes);
            const int row = (seg.l_blk * CG + rank) * kRowsPerCta + 32 * q + lane;
            const bool in = row < p.lrows;
            ptx::cp_async_4(slot + 4 * lane, p.ls + (in ? int64_t(kb) * p.ls_ld + (row >> p.ls_shift) : 0), in ? 4 : 0);
            if constexpr (COLVEC) {
#pragma unroll
                for (int i = 0; i < (Cfg::kCols + 31) / 32; ++i) {
                    if (Cfg::kCols >= 32 || lane < Cfg::kCols) {
                        const int c = seg.c_blk * BN + col + 32 * i + lane;
                        const bool cin = c < p.crows;
                        ptx::cp_async_4(slot + 128 + 4 * (32 * i + lane),
                                        p.cs + (cin ? int64_t(kb) * p.cs_ld + (c >> p.cs_shift) : 0), cin ? 4 : 0);
                    }
                }
            } else {
                const int c = seg.c_blk * BN + col;  // the warp's columns share one block of 128
                const bool cin = c < p.crows;
                ptx::cp_async_4(slot + 128 + 4 * lane, p.cs + (cin ? int64_t(kb) * p.cs_ld + (c >> p.cs_shift) : 0),
                                cin ? 4 : 0);
            }
            if (++kb == seg.kb1) {
                live = iter.next(p, seg);
                kb = seg.kb0;
            }
            ++n;
        }
        ptx::cp_async_commit();
    }
};

__device__ __forceinline__ void scaled_store_one(const ScaledParams& p, int64_t row, int64_t col, float v)
{
    const int64_t at = row * p.ldc + col;
    if (p.out_type == BWGEMM_FP32) {
        float* c = static_cast<float*>(p.c) + at;
        *c = p.accumulate ? *c + v : v;
    } else if (p.out_type == BWGEMM_BF16) {
        static_cast<__nv_bfloat16*>(p.c)[at] = __float2bfloat16_rn(v);
    } else {
        static_cast<__half*>(p.c)[at] = __float2half_rn(v);
    }
}

// One thread's finished row piece (kCols sums of lane row `row`) to C.
template <int CG, int BN, bool SWAP, bool COLVEC>
__device__ __forceinline__ void scaled_store(const uint64_t (&acc)[ScaledConfig<CG, BN, SWAP, COLVEC>::kCols / 2],
                                             const ScaledParams& p, const CUtensorMap* tmap_out, uint32_t buf,
                                             int row0, int col0, int lane)
{
    using Cfg = ScaledConfig<CG, BN, SWAP, COLVEC>;
    if constexpr (SWAP) {
        const int n = row0 + lane;  // column of C
        if (n < p.lrows) {
#pragma unroll
            for (int j = 0; j < Cfg::kCols / 2; ++j) {
                float lo, hi;
                ptx::unpack_f32x2(acc[j], lo, hi);
                if (col0 + 2 * j < p.crows)
                    scaled_store_one(p, col0 + 2 * j, n, lo);
                if (col0 + 2 * j + 1 < p.crows)
                    scaled_store_one(p, col0 + 2 * j + 1, n, hi);
            }
        }
    } else {
        if (row0 >= p.lrows)
            return;
        const bool wide = p.out_type == BWGEMM_FP32;
        const int per_box = wide ? 16 : 32;           // columns of a 64-byte box row
        const bool ragged = (p.crows & (wide ? 3 : 7)) != 0;  // rows of C end off a 16-byte boundary
        const uint32_t row_addr = buf + uint32_t(lane * 64);
        const uint32_t swz = uint32_t((lane >> 1) & 3);
        auto flush = [&](int col) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (p.accumulate)
                    ptx::tma_add_2d(tmap_out, buf, col, row0);
                else
                    ptx::tma_store_2d(tmap_out, buf, col, row0);
                ptx::bulk_commit_group();
            }
        };
        auto claim = [&] {  // the previous box has been read
            if (lane == 0)
                ptx::bulk_wait_group_read<0>();
            __syncwarp();
        };
#pragma unroll
        for (int c = 0; c < Cfg::kCols; c += 16) {
            const int col = col0 + c;
            const int box = col & ~(per_box - 1);
            if (ragged && box < p.crows && box + per_box > p.crows) {
                // a TMA store clips a row end only in whole 16-byte pieces: the
                // box holding one off a boundary goes out element by element
                if (row0 + lane < p.lrows) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float lo, hi;
                        ptx::unpack_f32x2(acc[c / 2 + j], lo, hi);
                        if (col + 2 * j < p.crows)
                            scaled_store_one(p, row0 + lane, col + 2 * j, lo);
                        if (col + 2 * j + 1 < p.crows)
                            scaled_store_one(p, row0 + lane, col + 2 * j + 1, hi);
                    }
                }
            } else if (wide) {
                claim();
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    float a, b, d, e;
                    ptx::unpack_f32x2(acc[c / 2 + 2 * ch], a, b);
                    ptx::unpack_f32x2(acc[c / 2 + 2 * ch + 1], d, e);
                    ptx::st_shared_v4(row_addr + ((uint32_t(ch) ^ swz) << 4), __float_as_uint(a), __float_as_uint(b),
                                      __float_as_uint(d), __float_as_uint(e));
                }
                if (col < p.crows)
                    flush(col);
            } else {
                if ((c & 16) == 0)
                    claim();
                const int dt = p.out_type;
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float lo, hi;
                    ptx::unpack_f32x2(acc[c / 2 + j], lo, hi);
                    w[j] = pack2(__float_as_uint(lo), __float_as_uint(hi), dt);
                }
                const uint32_t ch = uint32_t((c & 16) >> 3);  // 16-byte piece of the box row
                ptx::st_shared_v4(row_addr + ((ch ^ swz) << 4), w[0], w[1], w[2], w[3]);
                ptx::st_shared_v4(row_addr + (((ch + 1) ^ swz) << 4), w[4], w[5], w[6], w[7]);
                if ((c & 16) != 0 && box < p.crows)
                    flush(box);
            }
        }
    }
}

template <int CG, int BN, bool SWAP, bool COLVEC>
__global__ void __launch_bounds__(ScaledConfig<CG, BN, SWAP, COLVEC>::kThreads, 1)
    scaled_kernel(const __grid_constant__ CUtensorMap tmap_l, const __grid_constant__ CUtensorMap tmap_c,
                  const __grid_constant__ CUtensorMap tmap_l3, const __grid_constant__ CUtensorMap tmap_c3,
                  const __grid_constant__ CUtensorMap tmap_out, const ScaledParams p)
{
    using Cfg = ScaledConfig<CG, BN, SWAP, COLVEC>;
    constexpr int STAGES = Cfg::kStages;
    constexpr int KPS = Cfg::kKps;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? ptx::cluster_ctarank() : 0u;
    const int worker = int(blockIdx.x) / CG;
    const int workers = int(gridDim.x) / CG;
    const uint32_t sL = base + Cfg::kOffL;
    const uint32_t sC = base + Cfg::kOffC;
    const uint32_t bar_full = base + Cfg::kOffBar;              // + 8 * stage
    const uint32_t bar_empty = bar_full + 8 * STAGES;           // + 8 * stage
    const uint32_t bar_acc_full = bar_empty + 8 * STAGES;       // + 8 * buffer
    const uint32_t bar_acc_empty = bar_acc_full + 8 * Cfg::kBufs;
    const uint32_t bar_drain = bar_acc_empty + 8 * Cfg::kBufs;  // after an abort: the issued MMAs completed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffTmemSlot);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kOffAbort);

    // K blocks of the stage that starts at block kb of a segment: two when both
    // are whole chunks of the 3-D views, else one (a ragged last block, or a
    // single one left over)
    auto blocks_at = [&](int kb, int kb1) { return kb + KPS <= min(p.chunks, kb1) ? KPS : 1; };

    if (threadIdx.x == 64) {
        for (int s = 0; s < STAGES; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);   // the even CTA's producer's arrive.expect_tx (+ bytes)
            ptx::mbar_init(bar_empty + 8 * s, 1);  // one tcgen05.commit
        }
        for (int b = 0; b < Cfg::kBufs; ++b) {
            ptx::mbar_init(bar_acc_full + 8 * b, 1);
            ptx::mbar_init(bar_acc_empty + 8 * b, CG * Cfg::kEpiWarps);
        }
        ptx::mbar_init(bar_drain, 1);
        *abort_flag = 0u;
        ptx::fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&tmap_l);
        ptx::prefetch_tensormap(&tmap_c);
        if (p.chunks >= KPS) {
            ptx::prefetch_tensormap(&tmap_l3);
            ptx::prefetch_tensormap(&tmap_c3);
        }
        if (!SWAP)
            ptx::prefetch_tensormap(&tmap_out);
    }
    if (warp == 1) {
        ptx::tmem_alloc<CG>(ptx::smem_addr(tmem_slot), Cfg::kTmemCols);
        ptx::tmem_relinquish<CG>();
    }
    ptx::tc_fence_before_sync();
    if constexpr (CG == 2)
        ptx::cluster_sync();  // both CTAs' barriers exist before either copies or commits to them
    else
        __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    ptx::launch_dependents();
    uint32_t armed_mask = 0, armed_parity = 0;

    if (warp < Cfg::kFirstEpi) {
        if constexpr (Cfg::kSplitRegs)
            ptx::setmaxnreg_dec<Cfg::kRegsFirst>();
        if (warp == 0) {
            // ------------------------------------------------------ TMA producer
            ptx::grid_dependency_wait();
            const uint32_t leader_full = CG == 2 ? ptx::map_to_cta(bar_full, 0) : bar_full;
            ScaledIter iter;
            ScaledSegment seg;
            iter.init(p, worker, workers);
            int s = 0, i = 0;
            uint32_t phase = 0;
            bool ok = true;
            while (ok && iter.next(p, seg)) {
                const int l_row = (seg.l_blk * CG + int(rank)) * kRowsPerCta;
                const int c_row = seg.c_blk * BN + int(rank) * Cfg::kCRows;
    #pragma unroll 1
                for (int kb = seg.kb0; kb < seg.kb1; ++i) {
                    const int nkb = blocks_at(kb, seg.kb1);
                    ok = __all_sync(0xffffffffu,
                                    scaled_wait(bar_empty + 8 * s, phase ^ 1u, p, abort_flag, kStatusProducerTimeout));
                    if (!ok)
                        break;
                    // test hook: the producer of CTA 0 never fills this stage of the launch
                    const bool stall = p.stall_kblock >= 0 && blockIdx.x == 0 && p.stall_kblock == i;
                    if (!stall && rank == 0) {
                        armed_mask |= 1u << s;
                        armed_parity = (armed_parity & ~(1u << s)) | (phase << s);
                    }
                    if (!stall && ptx::elect_one()) {
                        const uint32_t fb = leader_full + 8 * s;
                        const uint32_t dL = sL + uint32_t(s * Cfg::kLBytes), dC = sC + uint32_t(s * Cfg::kCBytes);
                        if (rank == 0)
                            ptx::mbar_arrive_expect_tx(fb, uint32_t(CG * nkb * (Cfg::kLBlock + Cfg::kCBlock)));
                        if constexpr (CG == 2) {
                            if (nkb == KPS) {
                                ptx::tma_load_3d_pair(dL, &tmap_l3, fb, 0, l_row, kb);
                                ptx::tma_load_3d_pair(dC, &tmap_c3, fb, 0, c_row, kb);
                            } else {
                                ptx::tma_load_2d_pair(dL, &tmap_l, fb, kb * kBlock, l_row);
                                ptx::tma_load_2d_pair(dC, &tmap_c, fb, kb * kBlock, c_row);
                            }
                        } else {
                            if (nkb == KPS) {
                                ptx::tma_load_3d(dL, &tmap_l3, fb, 0, l_row, kb);
                                ptx::tma_load_3d(dC, &tmap_c3, fb, 0, c_row, kb);
                            } else {
                                ptx::tma_load_2d(dL, &tmap_l, fb, kb * kBlock, l_row);
                                ptx::tma_load_2d(dC, &tmap_c, fb, kb * kBlock, c_row);
                            }
                        }
                    }
                    __syncwarp();
                    kb += nkb;
                    if (++s == STAGES) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
        } else if (warp == 1 && rank == 0) {
            // ---------------------------------------------------------- MMA issue
            const uint64_t l_desc0 = make_sdesc_sw128(sL);
            const uint64_t c_desc0 = make_sdesc_sw128(sC);
            const uint32_t tmem0 = __shfl_sync(0xffffffffu, tmem_base, 0);
            ScaledIter iter;
            ScaledSegment seg;
            iter.init(p, worker, workers);
            int s = 0, b = 0;
            uint32_t phase = 0, bphase = 0;
            bool ok = true;
            while (ok && iter.next(p, seg)) {
    #pragma unroll 1
                for (int kb = seg.kb0; ok && kb < seg.kb1;) {
                    const int nkb = blocks_at(kb, seg.kb1);
                    ok = __all_sync(0xffffffffu, scaled_wait(bar_full + 8 * s, phase, p, abort_flag, kStatusMmaTimeout));
    #pragma unroll 1
                    for (int c = 0; ok && c < nkb; ++c) {
                        ok = __all_sync(0xffffffffu, scaled_wait(bar_acc_empty + 8 * b, bphase ^ 1u, p, abort_flag,
                                                                 kStatusMmaTimeout));
                        if (!ok)
                            break;
                        ptx::tc_fence_after_sync();
                        if (ptx::elect_one()) {
                            const uint64_t ld = l_desc0 + uint64_t((s * Cfg::kLBytes + c * Cfg::kLBlock) >> 4);
                            const uint64_t cd = c_desc0 + uint64_t((s * Cfg::kCBytes + c * Cfg::kCBlock) >> 4);
    #pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                ptx::mma_f8<CG>(tmem0 + uint32_t(b * BN), ld + uint64_t(2 * kk), cd + uint64_t(2 * kk),
                                                p.idesc, kk > 0 ? 1u : 0u);
                            if constexpr (CG == 2) {
                                if (c == nkb - 1)
                                    ptx::mma_commit_pair(bar_empty + 8 * s, 0x3);
                                ptx::mma_commit_pair(bar_acc_full + 8 * b, 0x3);
                            } else {
                                if (c == nkb - 1)
                                    ptx::mma_commit(bar_empty + 8 * s);
                                ptx::mma_commit(bar_acc_full + 8 * b);
                            }
                        }
                        __syncwarp();
                        if (++b == Cfg::kBufs) {
                            b = 0;
                            bphase ^= 1u;
                        }
                    }
                    kb += nkb;
                    if (++s == STAGES) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        if constexpr (Cfg::kSplitRegs)
            ptx::setmaxnreg_inc<Cfg::kRegsEpi>();
        ptx::grid_dependency_wait();
        constexpr int COLS = Cfg::kCols;
        const int e = warp - Cfg::kFirstEpi;
        const int q = warp & 3;            // the TMEM lane quarter this warp may access
        const int col = (e >> 2) * COLS;   // its first column of the tile
        const uint32_t ring = base + uint32_t(Cfg::kOffScale + e * Cfg::kSlots * Cfg::kSlotBytes);
        const uint32_t store_buf = base + uint32_t(Cfg::kOffStore + e * Cfg::kStoreBytes);
        ScaleFeed<CG, BN, SWAP, COLVEC> feed;
        feed.init(p, worker, workers);
#pragma unroll 1
        for (int i = 0; i < Cfg::kSlots - 1; ++i)
            feed.issue(p, ring, int(rank), q, col, lane);
        ScaledIter iter;
        ScaledSegment seg;
        iter.init(p, worker, workers);
        int b = 0, slot = 0;
        uint32_t bphase = 0;
        bool ok = true;
        while (ok && iter.next(p, seg)) {
            uint64_t acc[COLS / 2];
#pragma unroll
            for (int j = 0; j < COLS / 2; ++j)
                acc[j] = 0ull;
#pragma unroll 1
            for (int kb = seg.kb0; kb < seg.kb1; ++kb) {
                ptx::cp_async_wait<Cfg::kSlots - 2>();
                __syncwarp();  // every lane's part of the slot has landed, and the slot before it has been read
                feed.issue(p, ring, int(rank), q, col, lane);
                const uint32_t sl = ring + uint32_t(slot * Cfg::kSlotBytes);
                float scale = ptx::ld_shared_f32(sl + 4 * lane);
                if constexpr (!COLVEC)
                    scale *= ptx::ld_shared_f32(sl + 128 + 4 * lane);
                const uint64_t scale2 = ptx::pack_f32x2(__float_as_uint(scale), __float_as_uint(scale));
                ok = __all_sync(0xffffffffu, scaled_wait(bar_acc_full + 8 * b, bphase, p, abort_flag,
                                                         kStatusEpilogueTimeout));
                if (!ok)
                    break;
                ptx::tc_fence_after_sync();
                const uint32_t taddr = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(b * BN + col);
                uint32_t r[2][16];
                ptx::tmem_ld_32x32b_x16(taddr, r[0]);
#pragma unroll
                for (int c = 0; c < COLS; c += 16) {
                    ptx::tmem_ld_wait();
                    if (c + 16 < COLS)
                        ptx::tmem_ld_32x32b_x16(taddr + uint32_t(c + 16), r[((c >> 4) + 1) & 1]);
                    else
                        release_accumulator<CG>(bar_acc_empty + 8 * b, lane, 0);
                    const uint32_t(&v)[16] = r[(c >> 4) & 1];
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        uint64_t x0 = ptx::pack_f32x2(v[2 * j], v[2 * j + 1]);
                        uint64_t x1 = ptx::pack_f32x2(v[2 * j + 2], v[2 * j + 3]);
                        if constexpr (COLVEC) {
                            uint64_t c0, c1;
                            ptx::ld_shared_v2_b64(sl + 128 + 4 * uint32_t(c + 2 * j), c0, c1);
                            x0 = ptx::mul_f32x2(x0, c0);
                            x1 = ptx::mul_f32x2(x1, c1);
                        }
                        acc[c / 2 + j] = ptx::fma_f32x2(x0, scale2, acc[c / 2 + j]);
                        acc[c / 2 + j + 1] = ptx::fma_f32x2(x1, scale2, acc[c / 2 + j + 1]);
                    }
                }
                if (++b == Cfg::kBufs) {
                    b = 0;
                    bphase ^= 1u;
                }
                if (++slot == Cfg::kSlots)
                    slot = 0;
            }
            if (!ok)
                break;
            const int row0 = (seg.l_blk * CG + int(rank)) * kRowsPerCta + 32 * q;
            bool done = seg.whole;
            if (!done) {
                // publish this piece; whoever brings the tile's last K block adds
                // all pieces in worker order
                const size_t stride = size_t(CG) * Cfg::kPartialFloats;
                const size_t mine = rank * size_t(Cfg::kPartialFloats) + size_t(e) * (32 * COLS) + 4 * lane;
                float* part = p.partials + (size_t(worker) * 2 + seg.slot) * stride + mine;
#pragma unroll
                for (int j = 0; j < COLS / 4; ++j) {
                    float a, b2, c, d;
                    ptx::unpack_f32x2(acc[2 * j], a, b2);
                    ptx::unpack_f32x2(acc[2 * j + 1], c, d);
                    ptx::st_global_cg_v4(part + size_t(j) * 128, make_uint4(__float_as_uint(a), __float_as_uint(b2),
                                                                            __float_as_uint(c), __float_as_uint(d)));
                }
                __threadfence();
                __syncwarp();
                const int st = seg.tile - p.dp_tiles;
                uint32_t* counter = p.counters + (size_t(st) * CG + rank) * Cfg::kEpiWarps + e;
                uint32_t before = 0;
                if (lane == 0)
                    before = ptx::atom_add_acq_rel_gpu(counter, uint32_t(seg.kb1 - seg.kb0));
                before = __shfl_sync(0xffffffffu, before, 0);
                done = before + uint32_t(seg.kb1 - seg.kb0) == uint32_t(p.num_kb);
                if (done) {
                    if (lane == 0)
                        *counter = 0u;  // ready for the next call
                    __threadfence();
                    const long long first = (long long)st * p.num_kb;
                    const int w0 = int(((first + 1) * workers - 1) / p.sk_iters);
                    const int w1 = int(((first + p.num_kb) * workers - 1) / p.sk_iters);
#pragma unroll
                    for (int j = 0; j < COLS / 2; ++j)
                        acc[j] = 0ull;
                    const uint64_t one2 = ptx::pack_f32x2(__float_as_uint(1.f), __float_as_uint(1.f));
#pragma unroll 1
                    for (int w = w0; w <= w1; ++w) {
                        const int wslot = ScaledIter::begin(p, w, workers) / p.num_kb == st ? 0 : 1;
                        const float* src = p.partials + (size_t(w) * 2 + wslot) * stride + mine;
#pragma unroll
                        for (int j = 0; j < COLS / 4; ++j) {
                            const uint4 v = ptx::ld_global_cg_v4(src + size_t(j) * 128);
                            acc[2 * j] = ptx::fma_f32x2(ptx::pack_f32x2(v.x, v.y), one2, acc[2 * j]);
                            acc[2 * j + 1] = ptx::fma_f32x2(ptx::pack_f32x2(v.z, v.w), one2, acc[2 * j + 1]);
                        }
                    }
                }
            }
            if (done)
                scaled_store<CG, BN, SWAP, COLVEC>(acc, p, &tmap_out, store_buf, row0, seg.c_blk * BN + col, lane);
        }
        ptx::cp_async_wait<0>();
        if (!SWAP && lane == 0)
            ptx::bulk_wait_group_all();
        __syncwarp();
    }

    // --------------------------------------------------------------- teardown
    // After an abort, drain the MMAs and the loads this CTA armed (bounded) and
    // settle before TMEM and shared memory are released; the even CTA's barriers
    // count both CTAs' loads and neither CTA leaves before the other.
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

}  // namespace bwgemm
