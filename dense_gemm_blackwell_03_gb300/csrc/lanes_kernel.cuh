// lanes_kernel.cuh -- products whose weights fill the rows of the MMA: the gated layer
// on few rows of X, and the product of 8-bit integers at any size.
//
//   kLanesGated   H[m, n] = act(G) * U,  G = X Wg^T, U = X Wu^T      bf16 or fp16
//   kLanesInt8    C[m, n] = sx[m] * sw[n] * sum_k X[m, k] * W[n, k]  8-bit integers (turned: X
//                 in the lanes and W in its place, where there are fewer of W's rows)
//
// The accumulator holds the result transposed: a TMEM lane per weight row, a column per
// row of X (16 to 256), so that one to a few hundred tokens cost no more tensor time than
// they need, and a warp's lanes are consecutive columns of the result.
//
// Gated: tiles of 64 rows of each weight, two MMAs of M = 64 into columns of the same
// lanes -- a thread has both G and U of its outputs.
//
// 8-bit integers: the tensor cores of sm_103a have none, but an fp16 holds every 8-bit
// integer exactly, their products are exact in fp32 and so are sums up to 2^24.  (Past it the
// tensor cores cut off the last bits of what they add: 512 x 2048 x 131072, all 127, 5.1e-5 too
// small.)  So the weights travel as bytes -- HBM, L2 and shared memory --
// and become fp16 on the last stretch: four warps take a row each into registers, widen
// it (xor 0x80 makes u = x + 128, a byte permutation 0x6400 | u = 1024 + u, one
// subtraction 1024 + u - 1152 = x, all exact) and store it to TMEM, from where the MMA
// reads its A operand.  X goes through shared memory as fp16, widened once before
// (launch_widen) or, of up to 32 rows a tile (WIDENS), by a warp for every eight rows from one
// part of shared memory to another: no second launch (4 us of GPU and of host time each) and no
// workspace, but more work a step.  32 x 28672 x 8192 44.2 us, 43.1 when widened before; 48 x
// 8192 x 8192 22.2, 23.9 when widened before; 333 x 1000 x 5005 14.9 (18.2 with two warps).  At 16 rows four warps
// instead of two lose 5 %.
//
//   warp 0      TMA producer of the weights' ring (gated: of X's rows too)
//   warp 1      TMEM allocator and MMA issuer (in the even CTA of a pair)
//   warp 2      kLanesInt8: TMA producer of X's ring, or with warp 3 and the last two (of 32
//               rows a tile) what widens X into it
//   then        kLanesInt8: groups of four converting warps, a TMEM lane quarter each and a
//               group per 128 of K of a step
//   then        epilogue: four warps, eight from 128 columns on
//
// The integers' two rings: what bounds few rows of X is how many bytes of weights are on
// their way, so those get most of the shared memory, and a stage is free as soon as it is
// in registers.  They do not depend on launch_widen, which lets this kernel start only when
// all before it is done: where it ran, their copies do not wait for it.
//
// Measured (us, and what bounds it): gated 64 x 28672 x 8192 147 to 150 (HBM, 93 % of the copy
// rate); integers 64 x 28672 x 8192 46 (5.2 TB/s: 36 us of weights at HBM's rate, 4 to widen X before,
// the rest is the launch, the first bytes' way and the last tile's epilogue; without MMAs, widening and
// TMEM stores it takes as long.  A second set of converting warps that takes every other step: 50,
// tiles of 256 weight rows on CTA pairs 53, on one CTA 51),
// 8192 x 28672 x 8192, pairs, 1910 to 2070 (1.86 to 2.01 PFLOP/s, the fp16 rate under the power cap; 4096 x 8192
// x 8192 288, 304 with sums handed back after their stores).
//
// Work: whole tiles, and the last, partial wave spread over all workers in K steps; the
// warp that completes a tile's K adds the pieces in worker order (as in the block-scaled
// product).  Tiles may hold fewer weight rows than the MMA has, so that they fill the SMs.
#pragma once

#include "activation.cuh"
#include "feed_forward.h"
#include "int8_scales.cuh"
#include "scaled_kernel.cuh"

namespace bwgemm {

constexpr int kLanesK = 128;  // of K per stage

template <int MODE, int CG, int BN, bool WIDENS>
struct LanesConfig {
    static constexpr bool kGated = MODE == kLanesGated;
    static_assert(CG == 1 || (!kGated && BN == 256), "pairs: 8-bit integers, 256 rows of X");
    static constexpr int kLRows = kGated ? 64 : 128;          // weight rows per CTA and matrix
    static constexpr int kXRows = BN / CG;                    // rows of X this CTA copies
    static constexpr int kLBytes = kGated ? 2 * 64 * kLanesK * 2 : 128 * kLanesK;
    static constexpr int kXBytes = kXRows * kLanesK * 2;
    // The rings (gated: one, of both operands).  A step is what one barrier round trip covers:
    // kStep blocks of 128 of K, each widened by a group of converting warps into its part of a
    // TMEM slot, with X's part in shared memory.  A warp's way through a barrier, its copies or
    // MMAs and the arrivals is some 300 to 600 cycles, hence two blocks where tiles are narrow
    // (64 x 28672 x 8192: 49 us with two blocks a step, 55 with one).
    // kLanesInt8: 16-bit results of 32 weight rows x 32 rows of X, turned on their way out, per epilogue warp
    static constexpr int kTurnBytes = kGated ? 0 : 2048;
    static constexpr int kRingBytes = 222 * 1024 - lanes_epi_warps(BN) * kTurnBytes;
    static constexpr int kStep = !kGated && BN <= 64 ? 2 : 1;
    static constexpr int kXStep = kStep * kXBytes;
    static constexpr int kXStages = kGated ? kRingBytes / (kLBytes + kXBytes) : 3;
    static constexpr int kConvGroups = kGated ? 0 : kStep;
    // X's bytes of a step, copied with its weights, and the warps that widen them
    static constexpr bool kWidens = WIDENS;
    static_assert(!WIDENS || (!kGated && BN <= 32), "integers, few rows of X");
    static constexpr int kRawStep = kWidens ? BN * kStep * kLanesK : 0;
    static constexpr int kXWarps = kWidens ? BN / 8 : 0;
    static constexpr int kLStep = kStep * kLBytes;
    static constexpr int kFit = (kRingBytes - kXStages * kXStep) / (kLStep + kRawStep);
    static constexpr int kLStages = kGated ? kXStages : kFit > 10 / kStep ? 10 / kStep : kFit;
    static constexpr int kConvWarps = 4 * kConvGroups;
    static constexpr int kEpiWarps = lanes_epi_warps(BN);
    static constexpr int kFirstConv = 4;
    static constexpr int kFirstEpi = kFirstConv + kConvWarps;
    static constexpr int kLastX = kFirstEpi + kEpiWarps;  // what widens X beside warps 2 and 3
    static constexpr int kThreads = 32 * (kLastX + (kXWarps > 2 ? kXWarps - 2 : 0));
    static constexpr int kCols = BN / (kEpiWarps / 4);        // columns per epilogue warp
    static constexpr int kPiece = kCols < 32 ? kCols : 32;    // of which it reads this many at a time
    static constexpr int kAccCols = kGated ? 2 * BN : BN;
    static constexpr int kBufs = !kGated && BN == 256 ? 1 : 2;
    static constexpr int kACol0 = kBufs * kAccCols;           // widened weights in TMEM
    static constexpr int kACols = kLanesK / 2, kASlotCols = kStep * kACols;
    static constexpr int kTmemCols = kGated ? kBufs * kAccCols : 512;
    static_assert(kGated || kACol0 + kXStages * kASlotCols <= 512, "TMEM");
    static_assert(kTmemCols >= 32 && kTmemCols <= 512, "TMEM");
    static constexpr size_t kPartialFloats = lanes_partial_floats(MODE, BN);
    static constexpr int kOffL = 0;
    static constexpr int kOffX = kLStages * kLStep;
    static constexpr int kOffRaw = kOffX + kXStages * kXStep;
    static constexpr int kOffTurn = kOffRaw + kLStages * kRawStep;
    static constexpr int kScaleBytes = kGated ? 0 : 4 * kCols;
    static constexpr int kOffScale = kOffTurn + kEpiWarps * kTurnBytes;  // X's scales of a warp's columns
    static constexpr int kOffBar = kOffScale + kEpiWarps * kScaleBytes;
    // full, empty, wfull, wempty, acc_full, acc_empty, drain
    static constexpr int kNumBars = 2 * (kXStages + kLStages + kBufs) + 1;
    static constexpr int kOffTmemSlot = kOffBar + 8 * kNumBars;
    static constexpr int kOffAbort = kOffTmemSlot + 4;
    static constexpr int kSmemBytes = kOffAbort + 4 + 1024;
    static_assert(kLBytes % 1024 == 0 && kXBytes % 1024 == 0, "swizzle atoms need 1 KiB alignment");
    static_assert(kSmemBytes <= 227 * 1024, "exceeds the 227 KiB shared memory of one CTA");
};

// Four 8-bit integers as two pairs of fp16.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
}

__device__ __forceinline__ uint16_t round16(float v, int dtype)
{
    return dtype == BWGEMM_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

// TURNED: p.turned of the pairs, whose epilogue is the longer the more it has of both ways out
// (6978 x 3467 x 128 32 us, 37 with both in one kernel).
template <int MODE, int CG, int BN, bool WIDENS, bool TURNED = false>
__global__ void __launch_bounds__(LanesConfig<MODE, CG, BN, WIDENS>::kThreads, 1)
    lanes_kernel(const __grid_constant__ LanesMaps maps, const LanesParams p)
{
    using Cfg = LanesConfig<MODE, CG, BN, WIDENS>;
    constexpr bool GATED = Cfg::kGated;
    constexpr int XS = Cfg::kXStages, LS = Cfg::kLStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? ptx::cluster_ctarank() : 0u;
    const int worker = int(blockIdx.x) / CG;
    const int workers = int(gridDim.x) / CG;
    const int l_rows = p.l_rows;  // of this CTA
    const bool turned = CG == 2 ? TURNED : p.turned != 0;
    const uint32_t sL = base + Cfg::kOffL;
    const uint32_t sX = base + Cfg::kOffX;
    const uint32_t bar_full = base + Cfg::kOffBar;              // X has landed, the weights (widened) are there
    const uint32_t bar_empty = bar_full + 8 * XS;
    const uint32_t bar_wfull = bar_empty + 8 * XS;              // 8-bit weights (and X) have landed
    const uint32_t bar_wempty = bar_wfull + 8 * LS;
    const uint32_t bar_acc_full = bar_wempty + 8 * LS;
    const uint32_t bar_acc_empty = bar_acc_full + 8 * Cfg::kBufs;
    const uint32_t bar_drain = bar_acc_empty + 8 * Cfg::kBufs;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::kOffTmemSlot);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + Cfg::kOffAbort);

    if (threadIdx.x == 64) {
        for (int s = 0; s < XS; ++s) {
            ptx::mbar_init(bar_full + 8 * s, GATED ? 1 : (Cfg::kWidens ? Cfg::kXWarps : 1) + CG * Cfg::kConvWarps);
            ptx::mbar_init(bar_empty + 8 * s, 1);
        }
        for (int s = 0; !GATED && s < LS; ++s) {
            ptx::mbar_init(bar_wfull + 8 * s, 1);
            ptx::mbar_init(bar_wempty + 8 * s, Cfg::kConvWarps + Cfg::kXWarps);
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
        ptx::prefetch_tensormap(&maps.w);
        ptx::prefetch_tensormap(Cfg::kWidens ? &maps.x : &maps.x3);
        if (GATED) {
            ptx::prefetch_tensormap(&maps.w3);
            ptx::prefetch_tensormap(&maps.w23);
        }
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
    uint32_t armed_mask = 0, armed_parity = 0;  // of this warp's ring

    ScaledIter iter;
    ScaledSegment seg;
    iter.init(p, worker, workers);

    auto arm = [&](int s, uint32_t phase) {
        armed_mask |= 1u << s;
        armed_parity = (armed_parity & ~(1u << s)) | (phase << s);
    };
    // X's rows of a stage
    auto load_x = [&](uint32_t d, uint32_t bar, int row, int kb) {
        if (2 * kb + 2 <= p.c_chunks) {
            if constexpr (CG == 2)
                ptx::tma_load_3d_pair(d, &maps.x3, bar, 0, row, 2 * kb);
            else
                ptx::tma_load_3d(d, &maps.x3, bar, 0, row, 2 * kb);
        } else {
            ptx::tma_load_2d(d, &maps.x, bar, kb * kLanesK, row);
            ptx::tma_load_2d(d + uint32_t(Cfg::kXRows * 128), &maps.x, bar, kb * kLanesK + 64, row);
        }
    };

    if (warp == 0) {
        // -------------------------------------- TMA producer of the weights (gated: of all)
        int s = 0, n = 0;
        uint32_t phase = 0;
        bool ok = true;
        while (ok && iter.next(p, seg)) {
            const int l_row = (seg.l_blk * CG + int(rank)) * l_rows;
#pragma unroll 1
            for (int kb = seg.kb0; kb < seg.kb1; kb += Cfg::kStep, ++n) {
                ok = warp_wait((GATED ? bar_empty : bar_wempty) + 8 * s, phase ^ 1u, p, abort_flag, kStatusProducerTimeout);
                if (!ok)
                    break;
                // test hook: the producer of CTA 0 never fills this stage of the launch
                const bool stall = p.stall_kblock >= 0 && blockIdx.x == 0 && p.stall_kblock == n;
                if (!stall)
                    arm(s, phase);
                if (!stall && ptx::elect_one()) {
                    const uint32_t dL = sL + uint32_t(s * Cfg::kLStep);
                    const int k = kb * kLanesK;
                    if constexpr (GATED) {
                        const uint32_t fb = bar_full + 8 * s;
                        ptx::mbar_arrive_expect_tx(fb, uint32_t(Cfg::kXBytes + 4 * l_rows * 128));
                        if (n == 0)  // all before it overlaps the kernel before
                            ptx::grid_dependency_wait();
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t d = dL + uint32_t(i * 16384);
                            if (2 * kb + 2 <= p.l_chunks) {
                                ptx::tma_load_3d(d, i ? &maps.w23 : &maps.w3, fb, 0, l_row, 2 * kb);
                            } else {
                                ptx::tma_load_2d(d, i ? &maps.w2 : &maps.w, fb, k, l_row);
                                ptx::tma_load_2d(d + uint32_t(l_rows * 128), i ? &maps.w2 : &maps.w, fb, k + 64, l_row);
                            }
                        }
                        load_x(sX + uint32_t(s * Cfg::kXBytes), fb, seg.c_blk * BN, kb);
                    } else {
                        // a step's blocks in one copy where all lie in whole 128s of K
                        const uint32_t wb = bar_wfull + 8 * s, dR = base + uint32_t(Cfg::kOffRaw + s * Cfg::kRawStep);
                        const int count = min(Cfg::kStep, seg.kb1 - kb);
                        const int x_row = seg.c_blk * BN;
                        ptx::mbar_arrive_expect_tx(wb, uint32_t(count * kLanesK * (l_rows + (Cfg::kWidens ? BN : 0))));
                        if (Cfg::kWidens && n == 0)  // (launch_widen has waited for what was before it)
                            ptx::grid_dependency_wait();
                        if (Cfg::kStep == 2 && count == 2 && kb + 2 <= p.l_chunks) {
                            ptx::tma_load_3d(dL, &maps.w3, wb, 0, l_row, kb);
                            if (Cfg::kWidens)
                                ptx::tma_load_3d(dR, &maps.x3, wb, 0, x_row, kb);
                        } else {
                            for (int i = 0; i < count; ++i) {
                                ptx::tma_load_2d(dL + uint32_t(i * l_rows * kLanesK), &maps.w, wb, k + i * kLanesK, l_row);
                                if (Cfg::kWidens)
                                    ptx::tma_load_2d(dR + uint32_t(i * BN * kLanesK), &maps.x, wb, k + i * kLanesK, x_row);
                            }
                        }
                    }
                }
                __syncwarp();
                if (++s == LS) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (Cfg::kWidens && ((warp >= 2 && warp < Cfg::kFirstConv) || warp >= Cfg::kLastX)) {
        // --------------------------------- X's bytes to fp16, within shared memory
        // A row's step is 256 integers, 16 pieces; a warp takes two rows at a time.  Eight
        // lanes next to each other take four pieces of both, of different chunks: neither
        // their reads (rows of 128 bytes) nor their writes (pieces by row mod 8) share a bank.
        constexpr int PIECES = 4, APART = BN / 4;  // of 16 integers, for each lane and step; rows between them
        const int odd = (lane >> 2) & 1, block = lane >> 4, chunk = ((lane >> 3) & 1) ^ odd;
        const int r0 = 2 * (warp < Cfg::kFirstConv ? warp - 2 : warp - Cfg::kLastX + 2) + odd;  // this lane's rows: r0, r0 + APART, ...
        const uint32_t from0 = base + uint32_t(Cfg::kOffRaw + (block * BN + r0) * kLanesK + chunk * 64 + (lane & 3) * 16);
        // the piece's place: 16-byte pieces c0 and c0 + 1 of its rows in the block's chunk
        const uint32_t to0 = sX + uint32_t(block * Cfg::kXBytes + chunk * (Cfg::kXRows * 128) + r0 * 128);
        const uint32_t c0 = uint32_t(2 * (lane & 3));
        int s = 0, ws = 0;
        uint32_t phase = 0, wphase = 0;
        bool ok = true;
        while (ok && iter.next(p, seg)) {
#pragma unroll 1
            for (int kb = seg.kb0; kb < seg.kb1; kb += Cfg::kStep) {
                ok = warp_wait(bar_wfull + 8 * ws, wphase, p, abort_flag, kStatusMmaTimeout);
                if (!ok)
                    break;
                uint4 v[PIECES];
#pragma unroll
                for (int i = 0; i < PIECES; ++i)
                    ptx::ld_shared_v4(from0 + uint32_t(ws * Cfg::kRawStep + i * APART * kLanesK), v[i].x, v[i].y, v[i].z, v[i].w);
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive(bar_wempty + 8 * ws);
                ok = warp_wait(bar_empty + 8 * s, phase ^ 1u, p, abort_flag, kStatusMmaTimeout);
                if (!ok)
                    break;
                if (kb + block < seg.kb1) {
#pragma unroll
                    for (int i = 0; i < PIECES; ++i) {
                        uint4 a, b;
                        widen4(v[i].x, a.x, a.y);
                        widen4(v[i].y, a.z, a.w);
                        widen4(v[i].z, b.x, b.y);
                        widen4(v[i].w, b.z, b.w);
                        const uint32_t to = to0 + uint32_t(s * Cfg::kXStep + i * APART * 128);
                        const uint32_t swz = uint32_t((r0 + i * APART) & 7);
                        ptx::st_shared_v4(to + ((c0 ^ swz) << 4), a.x, a.y, a.z, a.w);
                        ptx::st_shared_v4(to + (((c0 + 1) ^ swz) << 4), b.x, b.y, b.z, b.w);
                    }
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    ptx::mbar_arrive(bar_full + 8 * s);
                if (++ws == LS) {
                    ws = 0;
                    wphase ^= 1u;
                }
                if (++s == XS) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (!GATED && !Cfg::kWidens && warp == 2) {
        // ------------------------------------------------------ TMA producer of X
        const uint32_t leader_full = CG == 2 ? ptx::map_to_cta(bar_full, 0) : bar_full;
        ptx::grid_dependency_wait();  // what X is widened by
        int s = 0;
        uint32_t phase = 0;
        bool ok = true;
        while (ok && iter.next(p, seg)) {
            const int x_row = seg.c_blk * BN + int(rank) * Cfg::kXRows;
#pragma unroll 1
            for (int kb = seg.kb0; kb < seg.kb1; kb += Cfg::kStep) {
                ok = warp_wait(bar_empty + 8 * s, phase ^ 1u, p, abort_flag, kStatusProducerTimeout);
                if (!ok)
                    break;
                if (rank == 0)
                    arm(s, phase);
                if (ptx::elect_one()) {
                    const int count = min(Cfg::kStep, seg.kb1 - kb);
                    if (rank == 0)
                        ptx::mbar_arrive_expect_tx(bar_full + 8 * s, uint32_t(CG * count * Cfg::kXBytes));
                    for (int i = 0; i < count; ++i)
                        load_x(sX + uint32_t(s * Cfg::kXStep + i * Cfg::kXBytes), leader_full + 8 * s, x_row, kb + i);
                }
                __syncwarp();
                if (++s == XS) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------------------------------------------------- MMA issue
        const uint64_t l_desc0 = make_sdesc_sw128(sL);
        const uint64_t x_desc0 = make_sdesc_sw128(sX);
        const uint32_t idesc = make_idesc(GATED ? p.dtype : int(BWGEMM_FP16), CG * Cfg::kLRows, BN);
        const uint32_t tmem0 = __shfl_sync(0xffffffffu, tmem_base, 0);
        int s = 0, b = 0;
        uint32_t phase = 0, bphase = 0;
        bool ok = true;
        while (ok && iter.next(p, seg)) {
            ok = warp_wait(bar_acc_empty + 8 * b, bphase ^ 1u, p, abort_flag, kStatusMmaTimeout);
#pragma unroll 1
            for (int kb = seg.kb0; ok && kb < seg.kb1; kb += Cfg::kStep) {
                ok = warp_wait(bar_full + 8 * s, phase, p, abort_flag, kStatusMmaTimeout);
                if (!ok)
                    break;
                ptx::tc_fence_after_sync();
                if (ptx::elect_one()) {
                    const uint64_t xd = x_desc0 + uint64_t((s * Cfg::kXStep) >> 4);
                    const uint32_t d = tmem0 + uint32_t(b * Cfg::kAccCols);
                    const uint32_t more = kb > seg.kb0 ? 1u : 0u;
#pragma unroll
                    for (int i = 0; i < Cfg::kStep; ++i) {
                        if (i > 0 && kb + i >= seg.kb1)
                            break;
#pragma unroll
                        for (int kk = 0; kk < kLanesK / 16; ++kk) {
                            const uint64_t xk =
                                xd + uint64_t((i * Cfg::kXBytes + (kk >> 2) * Cfg::kXRows * 128 + (kk & 3) * 32) >> 4);
                            const uint32_t on = i > 0 || kk > 0 ? 1u : more;
                            if constexpr (GATED) {
                                const uint64_t lk =
                                    l_desc0 + uint64_t((s * Cfg::kLBytes + (kk >> 2) * l_rows * 128 + (kk & 3) * 32) >> 4);
                                ptx::mma_f16<1>(d, lk, xk, idesc, on);
                                ptx::mma_f16<1>(d + BN, lk + uint64_t(16384 >> 4), xk, idesc, on);
                            } else {
                                const uint32_t at = uint32_t(Cfg::kACol0 + s * Cfg::kASlotCols + i * Cfg::kACols + 8 * kk);
                                ptx::mma_f16_tmem<CG>(d, tmem0 + at, xk, idesc, on);
                            }
                        }
                    }
                    if constexpr (CG == 2) {
                        ptx::mma_commit_pair(bar_empty + 8 * s, 0x3);
                        if (kb + Cfg::kStep >= seg.kb1)
                            ptx::mma_commit_pair(bar_acc_full + 8 * b, 0x3);
                    } else {
                        ptx::mma_commit(bar_empty + 8 * s);
                        if (kb + Cfg::kStep >= seg.kb1)
                            ptx::mma_commit(bar_acc_full + 8 * b);
                    }
                }
                __syncwarp();
                if (++s == XS) {
                    s = 0;
                    phase ^= 1u;
                }
            }
            if (++b == Cfg::kBufs) {
                b = 0;
                bphase ^= 1u;
            }
        }
    } else if (!GATED && warp >= Cfg::kFirstConv && warp < Cfg::kFirstEpi) {
        // ------------------------------------------------- 8-bit weights to fp16
        const int group = (warp - Cfg::kFirstConv) >> 2, q = warp & 3;
        const int row = 32 * q + lane;
        const uint32_t leader_full = CG == 2 ? ptx::map_to_cta(bar_full, 0) : bar_full;
        const uint32_t src0 = sL + uint32_t(group * l_rows * kLanesK + row * 128);
        const uint32_t dst0 = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(Cfg::kACol0);
        int s = 0, a = 0;
        uint32_t phase = 0, aphase = 0;
        bool ok = true;
        while (ok && iter.next(p, seg)) {
#pragma unroll 1
            for (int kb = seg.kb0; kb < seg.kb1; kb += Cfg::kStep) {
                ok = warp_wait(bar_wfull + 8 * s, phase, p, abort_flag, kStatusMmaTimeout);
                if (!ok)
                    break;
                const uint32_t src = src0 + uint32_t(s * Cfg::kLStep);
                // 16-byte pieces in registers: all eight of a row, or half of them where registers
                // are short (32 rows a tile 22.4 us on 48 x 8192 x 8192, 23.0 with all; from 128 on
                // all are 1 % faster)
                constexpr int HELD = BN <= 64 ? 4 : 8;
                uint32_t w[HELD][4];
                auto take = [&](int from) {
#pragma unroll
                    for (int c = 0; c < HELD; ++c)
                        ptx::ld_shared_v4(src + (uint32_t((from + c) ^ (row & 7)) << 4), w[c][0], w[c][1], w[c][2], w[c][3]);
                };
                take(0);
                ok = warp_wait(bar_empty + 8 * a, aphase ^ 1u, p, abort_flag, kStatusMmaTimeout);
                if (!ok)
                    break;
                ptx::tc_fence_after_sync();
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t r[32];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        widen4(w[(4 * half + i / 4) % HELD][i % 4], r[2 * i], r[2 * i + 1]);
                    if (HELD == 4 && half == 0)
                        take(4);
                    if (half == (HELD == 4 ? 1 : 0)) {  // the stage is in registers
                        __syncwarp();
                        if (lane == 0)
                            ptx::mbar_arrive(bar_wempty + 8 * s);
                    }
                    if (kb + group < seg.kb1)
                        ptx::tmem_st_32x32b_x32(dst0 + uint32_t(a * Cfg::kASlotCols + group * Cfg::kACols + 32 * half), r);
                }
                ptx::tmem_st_wait();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2)
                        ptx::mbar_arrive_cluster_relaxed(leader_full + 8 * a);
                    else
                        ptx::mbar_arrive(bar_full + 8 * a);
                }
                if (++s == LS) {
                    s = 0;
                    phase ^= 1u;
                }
                if (++a == XS) {
                    a = 0;
                    aphase ^= 1u;
                }
            }
        }
    } else if (warp >= Cfg::kFirstEpi && warp < Cfg::kLastX) {
        // ------------------------------------------------------------ epilogue
        ptx::grid_dependency_wait();
        constexpr int P = Cfg::kPiece;
        constexpr int MATS = GATED ? 2 : 1;
        const int e = warp - Cfg::kFirstEpi;
        const int q = warp & 3;
        const int col = (e >> 2) * Cfg::kCols;  // its first column of the tile
        // M = 64: row 16 q + i of the weights in lane i of quarter q, lanes 16 to 31 unused
        const int row = GATED ? 16 * q + lane : 32 * q + lane;
        const bool in_tile = row < l_rows && (!GATED || lane < 16);
        const uint32_t scale_buf = base + uint32_t(Cfg::kOffScale + e * Cfg::kScaleBytes);
        const uint32_t turn = base + uint32_t(Cfg::kOffTurn + e * Cfg::kTurnBytes);
        int b = 0;
        uint32_t bphase = 0;
        bool ok = true;
        while (ok && iter.next(p, seg)) {
            const int n = (seg.l_blk * CG + int(rank)) * l_rows + row;  // column of the result
            const int m0 = seg.c_blk * BN + col;                        // its row of column 0
            const bool live = in_tile && n < p.lrows;
            const float ls = !GATED && live ? p.ls[n] : 0.f;
            bool large = !GATED && turned && large_scale(ls);  // of the warp's tokens
            if constexpr (!GATED) {
                for (int c = lane; c < Cfg::kCols; c += 32) {
                    const float f = m0 + c < p.crows ? p.cs[m0 + c] : 0.f;
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(scale_buf + 4 * c), "f"(f) : "memory");
                    large = large || (!turned && large_scale(f));
                }
                large = __any_sync(0xffffffffu, large);
                __syncwarp();
            }
            // sums of P columns from c on, scaled
            auto scale = [&](const float(&v)[P], int c, float(&r)[P]) {
#pragma unroll
                for (int j = 0; j < P; j += 4) {
                    const float4 f = ptx::ld_shared_f32x4(scale_buf + 4 * (c + j));
                    if (!large) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            r[j + k] = turned ? v[j + k] * ls * (&f.x)[k] : v[j + k] * (&f.x)[k] * ls;
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            r[j + k] = scaled_sum(v[j + k], turned ? ls : (&f.x)[k], turned ? (&f.x)[k] : ls);
                    }
                }
            };
            // P rows of X from column c on, 32 columns of the result each, in this warp's `turn`: out in
            // 16-byte pieces (4096 x 4096 x 1024 39 us, 45 with a store of 64 bytes for each row and warp)
            auto turn_out = [&](int c) {
                __syncwarp();
                const int m = m0 + c, count = p.crows - m;
                const int piece = 8 * (lane & 3), n8 = n - lane + piece;  // of 8 columns
                const int left = row - lane + piece < l_rows ? p.lrows - n8 : 0;
                uint16_t* dst = static_cast<uint16_t*>(p.out[0]) + int64_t(m) * p.ldo[0] + n8;
#pragma unroll
                for (int j = lane >> 2; j < P; j += 8) {
                    uint4 w;
                    ptx::ld_shared_v4(turn + uint32_t(j * 64 + 2 * piece), w.x, w.y, w.z, w.w);
                    if (j >= count)
                        continue;
                    uint16_t* at = dst + j * p.ldo[0];
                    if (left >= 8) {
                        *reinterpret_cast<uint4*>(at) = w;
                    } else {
#pragma unroll
                        for (int k = 0; k < 7; ++k)
                            if (k < left)
                                at[k] = uint16_t((&w.x)[k / 2] >> (16 * (k % 2)));
                    }
                }
                __syncwarp();
            };
            auto turn_in = [&](int j, uint16_t h) {
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(turn + uint32_t(j * 64 + 2 * lane)), "h"(h) : "memory");
            };
            // Where p.turned, a lane is a row of the result: its columns c + 8 k .. to its place, or by
            // way of shared memory for eight rows of 64 bytes at a time (pairs: 4096 x 4000 x 1024 33.6 us,
            // 38.4 without; smaller tiles are 2 % slower so); and of 32 bits P columns
            auto row_in = [&](int k, uint4 w) {
                ptx::st_shared_v4(turn + uint32_t(lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)), w.x, w.y, w.z, w.w);
            };
            auto rows_out = [&](int c) {
                __syncwarp();
                const int piece = 8 * (lane & 3), left = p.crows - (m0 + c + piece);
#pragma unroll
                for (int r = lane >> 2; r < 32; r += 8) {
                    uint4 w;
                    ptx::ld_shared_v4(turn + uint32_t(r * 64 + (((lane ^ (r >> 1)) & 3) << 4)), w.x, w.y, w.z, w.w);
                    if (row - lane + r >= l_rows || n - lane + r >= p.lrows)
                        continue;
                    uint16_t* at = static_cast<uint16_t*>(p.out[0]) + int64_t(n - lane + r) * p.ldo[0] + m0 + c + piece;
                    if (left >= 8) {
                        *reinterpret_cast<uint4*>(at) = w;
                    } else {
#pragma unroll
                        for (int k = 0; k < 7; ++k)
                            if (k < left)
                                at[k] = uint16_t((&w.x)[k / 2] >> (16 * (k % 2)));
                    }
                }
                __syncwarp();
            };
            auto row_out = [&](int c, int k, uint4 w) {
                const int left = live ? p.crows - (m0 + c + 8 * k) : 0;
                uint16_t* at = static_cast<uint16_t*>(p.out[0]) + int64_t(n) * p.ldo[0] + m0 + c + 8 * k;
                if (left >= 8) {
                    *reinterpret_cast<uint4*>(at) = w;
                } else {
#pragma unroll
                    for (int i = 0; i < 7; ++i)
                        if (i < left)
                            at[i] = uint16_t((&w.x)[i / 2] >> (16 * (i % 2)));
                }
            };
            auto row_out32 = [&](int c, const float(&f)[P]) {
                const int left = live ? p.crows - (m0 + c) : 0;
                float* dst = static_cast<float*>(p.out[0]) + int64_t(n) * p.ldo[0] + m0 + c;
#pragma unroll
                for (int j = 0; j < P; j += 4) {
                    if (left >= j + 4) {
                        *reinterpret_cast<float4*>(dst + j) = make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 3; ++k)
                            if (j + k < left)
                                dst[j + k] = f[j + k];
                    }
                }
            };
            // P columns of finished sums (gated: of G, then of U) from column c of the warp's on
            auto finish = [&](int c, const float(&v)[MATS][P]) {
                const int m = m0 + c, count = p.crows - m;
                if constexpr (GATED) {
                    if (!live)
                        return;
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        if (j >= count)
                            break;
                        const float g = v[0][j], u = v[MATS - 1][j];
                        static_cast<uint16_t*>(p.out[0])[int64_t(m + j) * p.ldo[0] + n] =
                            round16(activate(g, p.activation) * u, p.dtype);
                        if (p.out[1] != nullptr) {
                            static_cast<uint16_t*>(p.out[1])[int64_t(m + j) * p.ldo[1] + n] = round16(g, p.dtype);
                            static_cast<uint16_t*>(p.out[2])[int64_t(m + j) * p.ldo[2] + n] = round16(u, p.dtype);
                        }
                    }
                } else {
                    if (count <= 0)
                        return;
                    float r[P];
                    scale(v[0], c, r);
                    if (turned) {
                        if (p.out_type == BWGEMM_FP32) {
                            row_out32(c, r);
                        } else {
                            uint32_t w[P / 2];
#pragma unroll
                            for (int j = 0; j < P / 2; ++j)
                                w[j] = pack2(__float_as_uint(r[2 * j]), __float_as_uint(r[2 * j + 1]), p.out_type);
#pragma unroll
                            for (int k = 0; k < P / 8; ++k)
                                row_out(c, k, make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
                        }
                    } else if (p.out_type == BWGEMM_FP32) {
                        if (!live)
                            return;
                        float* dst = static_cast<float*>(p.out[0]) + int64_t(m) * p.ldo[0] + n;
#pragma unroll
                        for (int j = 0; j < P; ++j)
                            if (j < count)
                                dst[j * p.ldo[0]] = r[j];
                    } else {
#pragma unroll
                        for (int j = 0; j < P; ++j)
                            turn_in(j, round16(r[j], p.out_type));
                        turn_out(c);
                    }
                }
            };
            ok = warp_wait(bar_acc_full + 8 * b, bphase, p, abort_flag, kStatusEpilogueTimeout);
            if (!ok)
                break;
            ptx::tc_fence_after_sync();
            const uint32_t taddr = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(b * Cfg::kAccCols + col);
            const uint32_t empty = bar_acc_empty + 8 * b;
            if (++b == Cfg::kBufs) {
                b = 0;
                bphase ^= 1u;
            }
            constexpr size_t kStride = Cfg::kPartialFloats;
            constexpr size_t kWarpFloats = size_t(MATS) * 32 * Cfg::kCols;
            const size_t mine = size_t(e) * kWarpFloats + 4 * lane;
            if constexpr (Cfg::kBufs == 1) {
                if (seg.whole && p.out_type != BWGEMM_FP32) {
                    // one buffer of sums: rounded and packed in registers, and handed back before they
                    // go out (4096 x 4096 x 1024 33 us; 39 with the buffer handed back after its stores)
                    uint32_t w[Cfg::kCols / 2];
#pragma unroll
                    for (int c = 0; c < Cfg::kCols; c += P) {
                        uint32_t v[P];
                        ptx::tmem_ld_32x32b_x32(taddr + uint32_t(c), v);
                        ptx::tmem_ld_wait();
                        if (c + P >= Cfg::kCols)
                            hand_back<CG>(empty, lane);
                        float f[P], r[P];
#pragma unroll
                        for (int j = 0; j < P; ++j)
                            f[j] = __uint_as_float(v[j]);
                        scale(f, c, r);
#pragma unroll
                        for (int j = 0; j < P / 2; ++j)
                            w[c / 2 + j] = pack2(__float_as_uint(r[2 * j]), __float_as_uint(r[2 * j + 1]), p.out_type);
                    }
#pragma unroll
                    for (int c = 0; c < Cfg::kCols; c += P) {
                        if (m0 + c >= p.crows)
                            break;
                        if (turned) {
#pragma unroll
                            for (int k = 0; k < P / 8; ++k) {
                                const int i = c / 2 + 4 * k;
                                row_in(k, make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]));
                            }
                            rows_out(c);
                        } else {
#pragma unroll
                            for (int j = 0; j < P; ++j)
                                turn_in(j, uint16_t(w[(c + j) / 2] >> (16 * (j % 2))));
                            turn_out(c);
                        }
                    }
                    continue;
                }
            }
            float* const part = p.partials + ((size_t(worker) * 2 + seg.slot) * CG + rank) * kStride + mine;
#pragma unroll 1
            for (int c = 0; c < Cfg::kCols; c += P) {
                uint32_t v[MATS][P];
#pragma unroll
                for (int i = 0; i < MATS; ++i) {
                    if constexpr (P == 16)
                        ptx::tmem_ld_32x32b_x16(taddr + uint32_t(i * BN + c), v[i]);
                    else
                        ptx::tmem_ld_32x32b_x32(taddr + uint32_t(i * BN + c), v[i]);
                }
                ptx::tmem_ld_wait();
                if (c + P >= Cfg::kCols)
                    hand_back<CG>(empty, lane);
                if (seg.whole) {
                    float f[MATS][P];
#pragma unroll
                    for (int i = 0; i < MATS; ++i)
#pragma unroll
                        for (int j = 0; j < P; ++j)
                            f[i][j] = __uint_as_float(v[i][j]);
                    finish(c, f);
                    __syncwarp();
                } else {
                    // a piece of a tile: its sums to global memory
#pragma unroll
                    for (int i = 0; i < MATS; ++i)
#pragma unroll
                        for (int j = 0; j < P; j += 4)
                            ptx::st_global_cg_v4(part + size_t(i) * 32 * Cfg::kCols + size_t(c + j) * 32,
                                                 make_uint4(v[i][j], v[i][j + 1], v[i][j + 2], v[i][j + 3]));
                }
            }
            if (seg.whole)
                continue;
            // whoever brings the tile's last K step adds all pieces in worker order
            __threadfence();
            __syncwarp();
            const int st = seg.tile - p.dp_tiles;
            uint32_t* counter = p.counters + (size_t(st) * CG + rank) * Cfg::kEpiWarps + e;
            uint32_t before = 0;
            if (lane == 0)
                before = ptx::atom_add_acq_rel_gpu(counter, uint32_t(seg.kb1 - seg.kb0));
            before = __shfl_sync(0xffffffffu, before, 0);
            if (before + uint32_t(seg.kb1 - seg.kb0) != uint32_t(p.num_kb))
                continue;
            if (lane == 0)
                *counter = 0u;  // ready for the next call
            __threadfence();
            const long long first = (long long)st * p.num_kb;
            const int w0 = int(((first + 1) * workers - 1) / p.sk_iters);
            const int w1 = int(((first + p.num_kb) * workers - 1) / p.sk_iters);
#pragma unroll 1
            for (int c = 0; c < Cfg::kCols; c += P) {
                float f[MATS][P];
#pragma unroll
                for (int i = 0; i < MATS; ++i)
#pragma unroll
                    for (int j = 0; j < P; ++j)
                        f[i][j] = 0.f;
                // pieces on their way at once, added in order (two of 32 columns take registers that
                // the integers' other warps lack: 48 x 8192 x 8192 23.9 us, 23.0 with one)
                constexpr int FLIGHT = 32 / P;
#pragma unroll 1
                for (int w = w0; w <= w1; w += FLIGHT) {
                    uint4 x[FLIGHT][MATS][P / 4];
#pragma unroll
                    for (int k = 0; k < FLIGHT; ++k) {
                        if (w + k > w1)
                            break;
                        const int wslot = ScaledIter::begin(p, w + k, workers) / p.num_kb == st ? 0 : 1;
                        const float* src = p.partials + ((size_t(w + k) * 2 + wslot) * CG + rank) * kStride + mine + size_t(c) * 32;
#pragma unroll
                        for (int i = 0; i < MATS; ++i)
#pragma unroll
                            for (int j = 0; j < P; j += 4)
                                x[k][i][j / 4] = ptx::ld_global_cg_v4(src + size_t(i) * 32 * Cfg::kCols + size_t(j) * 32);
                    }
#pragma unroll
                    for (int k = 0; k < FLIGHT; ++k) {
                        if (w + k > w1)
                            break;
#pragma unroll
                        for (int i = 0; i < MATS; ++i)
#pragma unroll
                            for (int j = 0; j < P; ++j)
                                f[i][j] += __uint_as_float((&x[k][i][j / 4].x)[j % 4]);
                    }
                }
                finish(c, f);
                __syncwarp();
            }
        }
    }

    // --------------------------------------------------------------- teardown
    // After an abort, drain the MMAs and the loads this CTA armed (bounded) and
    // settle before TMEM and shared memory are released.
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
        if (warp == 0 || (!GATED && !Cfg::kWidens && warp == 2)) {
            const uint32_t bar = GATED || warp == 2 ? bar_full : bar_wfull;
#pragma unroll 1
            for (int s = 0; s < (GATED || warp == 2 ? XS : LS); ++s)
                if ((armed_mask >> s) & 1u)
                    drain_wait(bar + 8 * s, (armed_parity >> s) & 1u, kDrainNs);
            if (lane == 0)
                settle(kSettleNs);
        }
        __syncwarp();
        __syncthreads();
    }
    ptx::tc_fence_before_sync();
    if constexpr (CG == 2)
        ptx::cluster_sync();
    else
        __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc<CG>(tmem_base, Cfg::kTmemCols);
    }
}

}  // namespace bwgemm
