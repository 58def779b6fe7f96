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
// fp32 FMAs.
//
// What bounds it, on large products: per K block of a 128 x 256 tile the MMAs
// take 512 cycles, the FMAs 256 (512 with a scale per column, which is one more
// multiplication each), and the path of a block through the epilogue -- barrier,
// two TMEM loads, additions, hand-back, each waiting for the one before -- about
// 1050; the two TMEM buffers let that overlap only with the next block's MMAs.
// 8192 x 28672 x 8192 takes 1833 to 1875 us (2.1 PFLOP/s), with a scale per column
// 8192^3 696 (1.58).  Of its rate then, without the additions 1.14.  Tried and slower:
// CTA pairs (half the copies, but every hand-back crosses the pair; 0.95), 192 columns
// with twelve epilogue warps of 64 (0.86), 128 columns (0.77), TMEM loads of 32 columns.
// On few rows of A it is bound by HBM: see the swapped form.
//
//   warp 0      TMA producer: a ring of stages of several K blocks, one 3-D copy
//               per operand and stage (fewer, larger copies: a stage costs its
//               barrier round trip whatever its size).
//   warp 1      TMEM allocator and MMA issuer: 4 tcgen05.mma of K = 32 per block,
//               kBufs accumulators in turn.  Narrow tiles: warp 2 issues too.
//   warp 3      the scales.
//   warps 4..   epilogue: 8 warps, two per TMEM lane quarter with half the
//               columns each (tiles of 128 and 256 columns), else 4.
//
// The scales come through a ring of their own in shared memory, filled by a
// warp with 4-byte asynchronous copies as far ahead as it holds (across tile
// boundaries too): the epilogue neither computes an address nor waits for a
// load, and the scales need no alignment.
//
// Work: the last, partial wave of tiles is spread over all workers in K
// iterations (stream-K).  A worker's piece of a tile goes to an fp32 partial in
// global memory; the warp that completes the tile's K blocks adds the pieces in
// worker order -- the same sum whichever arrives last -- and stores.  Nobody
// waits for anybody.
//
// Swapped form (few rows of A): the weights fill the 128 lanes, A's rows are
// the MMA's N (16 to 64), C leaves through plain stores (a warp's 32 lanes are
// 32 consecutive columns of C).  Tiles may hold fewer than 128 weight rows, so
// that they fill the SMs without splitting K, and up to four K blocks share an
// accumulator hand-over.  64 rows on 28672 x 8192 take 53 us (35.7 at the copy rate
// of HBM), 16 rows 38; on 64 rows HBM is busy 48 % of the time, the rest is the
// way of a K block through barriers and epilogue.  A few rows on smaller weights are
// taken by scaled_few_sm103.cu.
#pragma once

#include "operators.h"
#include "pipeline.cuh"

namespace bwgemm {

template <int BN, bool SWAP, bool COLVEC>
struct ScaledConfig {
    static constexpr int kKps = scaled_kps(BN, SWAP);
    // Four warps of producer, MMA issue and scales, then the epilogue.  With eight
    // epilogue warps a thread has 64 or 128 running sums and 64 loaded values,
    // more registers than an even share of the file (168 at twelve warps), and
    // the first warpgroup gives some of its own: 128 x 56 + 256 x 224 = 64512, the
    // 384 x 168 that the block is launched with (the launch code checks the
    // compiled count).
    static constexpr int kCols = BN >= 128 ? BN / 2 : BN;   // columns per epilogue warp
    static constexpr int kEpiWarps = 4 * (BN / kCols);
    static constexpr int kFirstEpi = 4;
    static constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
    static constexpr bool kSplitRegs = BN >= 128;
    static constexpr int kRegsFirst = 56, kRegsEpi = 224;
    static constexpr int kLBlock = kRowsPerCta * kBlock;   // one K block of the lane side: 16 KiB
    static constexpr int kCBlock = BN * kBlock;
    // the ring: whole stages of the lane side, then of the column side; with
    // fewer lane rows (swapped form) more stages fit
    static constexpr int kCBytes = kKps * kCBlock;
    static constexpr int kMaxStages = SWAP ? kScaledMaxStages : scaled_stages(BN, SWAP, kRowsPerCta);
    // K blocks per handshake between the MMAs and the epilogue, each in columns
    // of its own: a handshake takes either about 0.3 us, more than a narrow
    // block's MMAs and additions (1 x 28672 x 8192: 53 us one by one, 46 joined)
    static constexpr int kJoin = !SWAP ? 1 : BN <= 32 ? 4 : BN == 64 ? 2 : 1;
    static constexpr int kIssuers = kJoin > 1 ? 2 : 1;     // MMA warps
    static constexpr int kBufCols = kJoin * BN;
    static constexpr int kBufs = kBufCols == 256 ? 2 : 4;  // such accumulators in TMEM
    static constexpr int kTmemCols = kBufs * kBufCols;
    static_assert(kTmemCols >= 32 && kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "TMEM allocation");
    // a scale slot holds four K blocks' scales: [lane][block], and [column group
    // of a warp][block] or, with a scale per column, [block][column]
    static constexpr int kGroup = 4;
    static constexpr int kColScaleOff = 4 * kGroup * kRowsPerCta;
    static constexpr int kSlotBytes = kColScaleOff + 4 * kGroup * (COLVEC ? BN : 4);
    static constexpr int kSlots = COLVEC && BN > 128 ? 2 : 3;
    static constexpr int kScaleThreads = 32;
    static constexpr int kStoreBytes = 2048;  // a 64-byte x 32-row output box
    static constexpr int kOffStore = kScaledRingBytes;
    static constexpr int kOffScale = kOffStore + (SWAP ? 0 : kEpiWarps * kStoreBytes);
    static constexpr int kOffBar = kOffScale + kSlots * kSlotBytes;
    // full, empty, acc_full, acc_empty, scale_full, scale_empty, drain
    static constexpr int kNumBars = 2 * (kMaxStages + kBufs + kSlots) + 1;
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
    int it, it_begin, it_end;
    int t, step;

    template <typename Params>
    static __device__ __forceinline__ int begin(const Params& p, int worker, int workers)
    {
        const long long prod = (long long)worker * p.sk_iters;
        return prod < (1ll << 32) ? int(unsigned(prod) / unsigned(workers)) : int(prod / workers);
    }
    template <typename Params>
    __device__ __forceinline__ void init(const Params& p, int worker, int workers)
    {
        it_begin = it = begin(p, worker, workers);
        it_end = begin(p, worker + 1, workers);
        t = worker;
        step = workers;
    }
    template <typename Params>
    __device__ __forceinline__ bool next(const Params& p, ScaledSegment& s)
    {
        if (it < it_end) {
            const int tile = it / p.num_kb;
            s.kb0 = it - tile * p.num_kb;
            s.kb1 = min(p.num_kb, s.kb0 + (it_end - it));
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

// A warp's finished sums (kCols of lane row row0 + lane, `rows` of them in the
// tile) to C.
template <int BN, bool SWAP, bool COLVEC>
__device__ __forceinline__ void scaled_store(const uint64_t (&acc)[ScaledConfig<BN, SWAP, COLVEC>::kCols / 2],
                                             const ScaledParams& p, const CUtensorMap* tmap_out, uint32_t buf,
                                             int row0, int rows, int col0, int lane)
{
    using Cfg = ScaledConfig<BN, SWAP, COLVEC>;
    if constexpr (SWAP) {
        const int n = row0 + lane;  // column of C
        if (lane < rows && n < p.lrows) {
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

template <int BN, bool SWAP, bool COLVEC>
__global__ void __launch_bounds__(ScaledConfig<BN, SWAP, COLVEC>::kThreads, 1)
    scaled_kernel(const __grid_constant__ CUtensorMap tmap_l, const __grid_constant__ CUtensorMap tmap_c,
                  const __grid_constant__ CUtensorMap tmap_l3, const __grid_constant__ CUtensorMap tmap_c3,
                  const __grid_constant__ CUtensorMap tmap_out, const ScaledParams p)
{
    using Cfg = ScaledConfig<BN, SWAP, COLVEC>;
    constexpr int KPS = Cfg::kKps;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int worker = int(blockIdx.x);
    const int workers = int(gridDim.x);
    // Lane rows of a tile, and the bytes of one K block of them: 128, or fewer
    // (swapped form) where that gives every CTA a tile of its own.  The MMAs then
    // read on into whatever lies behind the rows -- later stages, or the column
    // side, which is larger than the rows left out; the lanes that this fills are
    // not stored.
    const int l_rows = SWAP ? p.l_rows : kRowsPerCta;
    const int l_block = l_rows * kBlock;
    const int l_bytes = KPS * l_block;
    const int stages = SWAP ? p.stages : Cfg::kMaxStages;
    const uint32_t sL = base;
    const uint32_t sC = base + uint32_t(stages * l_bytes);
    const uint32_t bar_full = base + Cfg::kOffBar;              // + 8 * stage
    const uint32_t bar_empty = bar_full + 8 * Cfg::kMaxStages;           // + 8 * stage
    const uint32_t bar_acc_full = bar_empty + 8 * Cfg::kMaxStages;       // + 8 * buffer
    const uint32_t bar_acc_empty = bar_acc_full + 8 * Cfg::kBufs;
    const uint32_t bar_scale_full = bar_acc_empty + 8 * Cfg::kBufs;   // + 8 * slot
    const uint32_t bar_scale_empty = bar_scale_full + 8 * Cfg::kSlots;
    const uint32_t bar_drain = bar_scale_empty + 8 * Cfg::kSlots;  // after an abort: the issued MMAs completed
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffTmemSlot);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kOffAbort);

    // K blocks of the stage that starts at block kb of a segment: KPS when all are
    // whole chunks of the 3-D views, else one (a ragged last block, or single
    // ones left over)
    auto blocks_at = [&](int kb, int kb1) { return kb + KPS <= min(p.chunks, kb1) ? KPS : 1; };

    if (threadIdx.x == 64) {
        for (int s = 0; s < Cfg::kMaxStages; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);   // the producer's arrive.expect_tx (+ bytes)
            ptx::mbar_init(bar_empty + 8 * s, Cfg::kIssuers);  // a tcgen05.commit of each MMA warp
        }
        for (int b = 0; b < Cfg::kBufs; ++b) {
            ptx::mbar_init(bar_acc_full + 8 * b, Cfg::kIssuers);
            ptx::mbar_init(bar_acc_empty + 8 * b, Cfg::kEpiWarps);
        }
        for (int i = 0; i < Cfg::kSlots; ++i) {
            ptx::mbar_init(bar_scale_full + 8 * i, Cfg::kScaleThreads);
            ptx::mbar_init(bar_scale_empty + 8 * i, Cfg::kEpiWarps);
        }
        ptx::mbar_init(bar_drain, Cfg::kIssuers);
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
        ptx::tmem_alloc<1>(ptx::smem_addr(tmem_slot), Cfg::kTmemCols);
        ptx::tmem_relinquish<1>();
    }
    ptx::tc_fence_before_sync();
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
            ScaledIter iter;
            ScaledSegment seg;
            iter.init(p, worker, workers);
            int s = 0, i = 0;
            uint32_t phase = 0;
            bool ok = true;
            while (ok && iter.next(p, seg)) {
                const int l_row = seg.l_blk * l_rows;
                const int c_row = seg.c_blk * BN;
    #pragma unroll 1
                for (int kb = seg.kb0; kb < seg.kb1; ++i) {
                    const int nkb = blocks_at(kb, seg.kb1);
                    ok = __all_sync(0xffffffffu,
                                    pipe_wait(bar_empty + 8 * s, phase ^ 1u, p, abort_flag, kStatusProducerTimeout));
                    if (!ok)
                        break;
                    // test hook: the producer of CTA 0 never fills this stage of the launch
                    const bool stall = p.stall_kblock >= 0 && blockIdx.x == 0 && p.stall_kblock == i;
                    if (!stall) {
                        armed_mask |= 1u << s;
                        armed_parity = (armed_parity & ~(1u << s)) | (phase << s);
                    }
                    if (!stall && ptx::elect_one()) {
                        const uint32_t fb = bar_full + 8 * s;
                        const uint32_t dL = sL + uint32_t(s * l_bytes), dC = sC + uint32_t(s * Cfg::kCBytes);
                        ptx::mbar_arrive_expect_tx(fb, uint32_t(nkb * (l_block + Cfg::kCBlock)));
                        if (i == 0)  // all before it overlaps the kernel before
                            ptx::grid_dependency_wait();
                        if (nkb == KPS) {
                            ptx::tma_load_3d(dL, &tmap_l3, fb, 0, l_row, kb);
                            ptx::tma_load_3d(dC, &tmap_c3, fb, 0, c_row, kb);
                        } else {
                            ptx::tma_load_2d(dL, &tmap_l, fb, kb * kBlock, l_row);
                            ptx::tma_load_2d(dC, &tmap_c, fb, kb * kBlock, c_row);
                        }
                    }
                    __syncwarp();
                    kb += nkb;
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
        } else if (warp <= Cfg::kIssuers) {
            // ---------------------------------------------------------- MMA issue
            // With joint accumulators warps 1 and 2 take every other block of a
            // stage: one warp's serial path through waits, issue and
            // commits is some 600 cycles a block, more than a narrow block needs
            // otherwise.  Both wait for every stage and accumulator, and a stage is
            // free, an accumulator full, when both have committed.
            const int w = warp - 1;
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
                int sub = 0;  // block of the joint accumulator
#pragma unroll 1
                for (int kb = seg.kb0; ok && kb < seg.kb1;) {
                    const int nkb = blocks_at(kb, seg.kb1);
                    ok = __all_sync(0xffffffffu, pipe_wait(bar_full + 8 * s, phase, p, abort_flag, kStatusMmaTimeout));
                    // block c of the stage into column block d of the accumulator
                    auto issue = [&](int c, int d) {
                        const uint64_t ld = l_desc0 + uint64_t((s * l_bytes + c * l_block) >> 4);
                        const uint64_t cd = c_desc0 + uint64_t((s * Cfg::kCBytes + c * Cfg::kCBlock) >> 4);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            ptx::mma_f8(tmem0 + uint32_t(b * Cfg::kBufCols + d * BN), ld + uint64_t(2 * kk),
                                           cd + uint64_t(2 * kk), p.idesc, kk > 0 ? 1u : 0u);
                    };
                    if constexpr (Cfg::kIssuers == 2) {
                        static_assert(Cfg::kJoin % KPS == 0, "a stage lies in one accumulator");
                        if (ok && sub == 0)
                            ok = __all_sync(0xffffffffu, pipe_wait(bar_acc_empty + 8 * b, bphase ^ 1u, p, abort_flag,
                                                                   kStatusMmaTimeout));
                        if (!ok)
                            break;
                        ptx::tc_fence_after_sync();
                        const bool last = sub + nkb >= Cfg::kJoin || kb + nkb == seg.kb1;
                        if (ptx::elect_one()) {
                            for (int c = w; c < nkb; c += 2)
                                issue(c, sub + c);
                            ptx::mma_commit(bar_empty + 8 * s);
                            if (last)
                                ptx::mma_commit(bar_acc_full + 8 * b);
                        }
                        __syncwarp();
                        sub += nkb;
                        if (last) {
                            sub = 0;
                            b = (b + 1) & (Cfg::kBufs - 1);
                            bphase ^= b == 0 ? 1u : 0u;
                        }
                    } else {
#pragma unroll 1
                        for (int c = 0; ok && c < nkb; ++c) {
                            ok = __all_sync(0xffffffffu, pipe_wait(bar_acc_empty + 8 * b, bphase ^ 1u, p, abort_flag,
                                                                   kStatusMmaTimeout));
                            if (!ok)
                                break;
                            ptx::tc_fence_after_sync();
                            if (ptx::elect_one()) {
                                issue(c, 0);
                                if (c == nkb - 1)
                                    ptx::mma_commit(bar_empty + 8 * s);
                                ptx::mma_commit(bar_acc_full + 8 * b);
                            }
                            __syncwarp();
                            b = (b + 1) & (Cfg::kBufs - 1);
                            bphase ^= b == 0 ? 1u : 0u;
                        }
                    }
                    kb += nkb;
                    if (++s == stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
        } else if (warp == 3) {
            // -------------------------------------------------------- scales
            // Each thread's arrival on a slot comes when its copies have landed, so the
            // warp runs ahead of the epilogue as far as the slots allow.
            ScaledIter iter;
            ScaledSegment seg;
            iter.init(p, worker, workers);
            int slot = 0;
            uint32_t phase = 0;
            bool ok = true, first = true;
            while (ok && iter.next(p, seg)) {
                const int row0 = seg.l_blk * l_rows;
                const int col0 = seg.c_blk * BN;
#pragma unroll 1
                for (int kb = seg.kb0; kb < seg.kb1; kb += Cfg::kGroup) {
                    ok = __all_sync(0xffffffffu, pipe_wait(bar_scale_empty + 8 * slot, phase ^ 1u, p, abort_flag,
                                                           kStatusProducerTimeout));
                    if (!ok)
                        break;
                    if (first)
                        ptx::grid_dependency_wait();
                    first = false;
                    const int n = min(Cfg::kGroup, seg.kb1 - kb);
#pragma unroll 1
                    for (int g = 0; g < n; ++g) {
                        const uint32_t dst = base + uint32_t(Cfg::kOffScale + slot * Cfg::kSlotBytes);
                        const uint32_t dst_c = dst + Cfg::kColScaleOff;
                        const float* ls = p.ls + int64_t(kb + g) * p.ls_ld;
                        const float* cs = p.cs + int64_t(kb + g) * p.cs_ld;
#pragma unroll
                        for (int i = 0; i < kRowsPerCta / 32; ++i) {
                            const int row = row0 + 32 * i + lane;
                            ptx::cp_async_4(dst + 4 * (Cfg::kGroup * (32 * i + lane) + g),
                                            ls + (row < p.lrows ? row >> p.ls_shift : 0), row < p.lrows ? 4 : 0);
                        }
                        if constexpr (COLVEC) {
#pragma unroll
                            for (int i = 0; i < (BN + 31) / 32; ++i) {
                                const int col = col0 + 32 * i + lane;
                                if (BN >= 32 || lane < BN)
                                    ptx::cp_async_4(dst_c + 4 * (BN * g + 32 * i + lane),
                                                    cs + (col < p.crows ? col >> p.cs_shift : 0), col < p.crows ? 4 : 0);
                            }
                        } else if (lane < BN / Cfg::kCols) {
                            const int col = col0 + lane * Cfg::kCols;  // a warp's columns share one block of 128
                            ptx::cp_async_4(dst_c + 4 * (Cfg::kGroup * lane + g),
                                            cs + (col < p.crows ? col >> p.cs_shift : 0), col < p.crows ? 4 : 0);
                        }
                    }
                    ptx::cp_async_arrive(bar_scale_full + 8 * slot);
                    if (++slot == Cfg::kSlots) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
            ptx::cp_async_wait_all();
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
        const uint32_t store_buf = base + uint32_t(Cfg::kOffStore + e * Cfg::kStoreBytes);
        ScaledIter iter;
        ScaledSegment seg;
        iter.init(p, worker, workers);
        int b = 0, slot = 0;
        uint32_t bphase = 0, sphase = 0;
        bool ok = true;
        while (ok && iter.next(p, seg)) {
            uint64_t acc[COLS / 2];
#pragma unroll
            for (int j = 0; j < COLS / 2; ++j)
                acc[j] = 0ull;
#pragma unroll 1
            for (int kb = seg.kb0; ok && kb < seg.kb1; kb += Cfg::kGroup) {
                // the group's four scales of this lane, with its warp's column
                // scales where it has one per block
                ok = __all_sync(0xffffffffu, pipe_wait(bar_scale_full + 8 * slot, sphase, p, abort_flag,
                                                       kStatusEpilogueTimeout));
                const uint32_t sl = base + uint32_t(Cfg::kOffScale + slot * Cfg::kSlotBytes);
                const uint32_t scale_empty = bar_scale_empty + 8 * slot;
                float4 ls = ptx::ld_shared_f32x4(sl + 16 * (32 * q + lane));
                if constexpr (!COLVEC) {
                    const float4 cs = ptx::ld_shared_f32x4(sl + Cfg::kColScaleOff + 16 * (e >> 2));
                    ls = make_float4(ls.x * cs.x, ls.y * cs.y, ls.z * cs.z, ls.w * cs.w);
                }
                if (++slot == Cfg::kSlots) {
                    slot = 0;
                    sphase ^= 1u;
                }
                // unrolled, but with a scale per column: twice the code, which then
                // misses the instruction cache (8192^3: 722 us unrolled, 697 rolled;
                // 8192 x 28672 x 8192 with a scale per block: 1858 and 1962)
                constexpr int kUnroll = COLVEC && !SWAP ? 1 : Cfg::kGroup;
#pragma unroll kUnroll
                for (int g = 0; g < Cfg::kGroup; g += Cfg::kJoin) {
                    if (!ok || kb + g >= seg.kb1)
                        break;
                    const int blocks = min(Cfg::kJoin, seg.kb1 - kb - g);  // in this accumulator
                    ok = __all_sync(0xffffffffu, pipe_wait(bar_acc_full + 8 * b, bphase, p, abort_flag,
                                                           kStatusEpilogueTimeout));
                    if (!ok)
                        break;
                    ptx::tc_fence_after_sync();
                    const uint32_t taddr = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(b * Cfg::kBufCols + col);
                    const uint32_t empty = bar_acc_empty + 8 * b;
                    b = (b + 1) & (Cfg::kBufs - 1);
                    bphase ^= b == 0 ? 1u : 0u;
                    constexpr int LD = 64;  // columns per TMEM load: of one K block, or of several
                    constexpr int TOTAL = Cfg::kJoin * COLS;  // columns this warp reads
#pragma unroll
                    for (int i = 0; i < TOTAL; i += LD) {
                        uint32_t v[LD];
                        ptx::tmem_ld_32x32b_x64(taddr + uint32_t(i), v);
                        ptx::tmem_ld_wait();
                        if (i + LD == TOTAL)
                            hand_back<1>(empty, lane);
                        // the piece's columns, K block by K block
#pragma unroll
                        for (int part = 0; part < LD; part += COLS < LD ? COLS : LD) {
                            const int sub = (i + part) / COLS;
                            if (sub > 0 && sub >= blocks)
                                continue;
                            const int k = g + sub;
                            const float scale = k == 0 ? ls.x : k == 1 ? ls.y : k == 2 ? ls.z : ls.w;
                            const uint64_t scale2 = ptx::pack_f32x2(__float_as_uint(scale), __float_as_uint(scale));
                            const uint32_t sc = sl + Cfg::kColScaleOff + 4 * (BN * k + col);
                            const int c0 = (i + part) % COLS;  // first column
#pragma unroll
                            for (int j = 0; j < (COLS < LD ? COLS : LD); j += 4) {
                                uint64_t x0 = ptx::pack_f32x2(v[part + j], v[part + j + 1]);
                                uint64_t x1 = ptx::pack_f32x2(v[part + j + 2], v[part + j + 3]);
                                if constexpr (COLVEC) {
                                    uint64_t m0, m1;
                                    ptx::ld_shared_v2_b64(sc + 4 * uint32_t(c0 + j), m0, m1);
                                    x0 = ptx::mul_f32x2(x0, m0);
                                    x1 = ptx::mul_f32x2(x1, m1);
                                }
                                acc[(c0 + j) / 2] = ptx::fma_f32x2(x0, scale2, acc[(c0 + j) / 2]);
                                acc[(c0 + j) / 2 + 1] = ptx::fma_f32x2(x1, scale2, acc[(c0 + j) / 2 + 1]);
                            }
                        }
                    }
                }
                // released: every lane's reads of the slot come before the copies that
                // the scales' warp starts into it once it sees the arrivals
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive(scale_empty);
            }
            if (!ok)
                break;
            const int row0 = seg.l_blk * l_rows + 32 * q;
            bool done = seg.whole;
            if (!done) {
                // publish this piece; whoever brings the tile's last K block adds
                // all pieces in worker order
                const size_t stride = Cfg::kPartialFloats;
                const size_t mine = size_t(e) * (32 * COLS) + 4 * lane;
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
                uint32_t* counter = p.counters + size_t(st) * Cfg::kEpiWarps + e;
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
                scaled_store<BN, SWAP, COLVEC>(acc, p, &tmap_out, store_buf, row0, l_rows - 32 * q, seg.c_blk * BN + col, lane);
        }
        if (!SWAP && lane == 0)
            ptx::bulk_wait_group_all();
        __syncwarp();
    }

    // --------------------------------------------------------------- teardown
    // After an abort, drain the MMAs and the loads this CTA armed (bounded) and
    // settle before TMEM and shared memory are released.
    __syncwarp();
    __syncthreads();
    if (*abort_flag) {
        if (warp >= 1 && warp <= Cfg::kIssuers) {
            if (ptx::elect_one())
                ptx::mma_commit(bar_drain);
            __syncwarp();
            drain_wait(bar_drain, 0u, kDrainNs);
        }
        if (warp == 0) {
#pragma unroll 1
            for (int s = 0; s < stages; ++s)
                if ((armed_mask >> s) & 1u)
                    drain_wait(bar_full + 8 * s, (armed_parity >> s) & 1u, kDrainNs);
            if (lane == 0)
                settle(kSettleNs);
        }
        __syncwarp();
        __syncthreads();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc<1>(tmem_base, Cfg::kTmemCols);
    }
}

}  // namespace bwgemm
