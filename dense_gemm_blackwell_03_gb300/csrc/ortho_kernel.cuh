// ortho_kernel.cuh -- the products of the Newton-Schulz iteration
//
//   S = X X^T     B = a I + b S + c S S     X <- B X
//
// on fp16 operands with fp32 accumulation: one persistent, warp-specialised
// tcgen05 kernel for all three, over a stack of matrices.
//
// Symmetry: S and S S are computed on and below the diagonal of tiles only
// (m^2 n + m^3 instead of twice that); the epilogue stores an off-diagonal box
// a second time, transposed in shared memory.  The polynomial's b S and a I are
// added to the fp32 sums before their one rounding.
//
// Orientation: X is kept as it comes, its longer side along rows or columns.
// With more columns the first product contracts over columns (both operands
// K-major) and the last over rows of X (B K-major, X MN-major); with more rows
// the first contracts over rows (both MN-major) and the last is X B (both
// K-major).  tcgen05 reads either major order, so nothing is ever transposed
// in memory.
//
// Two terms: where `terms` is 2 the K loop runs twice, the second time with the
// operand's low part (what fp16 rounding lost) -- the sum of both products in
// one accumulator.
//
// The diagonal: where X's singular values are close together, B is close to a
// multiple of I, and fp16 rounds all of its diagonal the same way -- a relative
// error of the whole result.  In the first steps the diagonal tiles of B keep
// their low part too, and the product with X takes one more K step with it.
//
// Few tiles and a deep K (long, narrow matrices): the tiles of S are cut into
// slices of K whose fp32 sums go to global memory; a second kernel adds them in
// order, with as many CTAs as there is data.
//
// Each stage of the ring holds 128 of K of both operands (64 KiB), one 32 KiB
// copy each (box {64, 128 rows, 2 chunks}); the same box serves K-major (rows =
// output rows, chunks along K) and MN-major (rows = K, chunks along the
// output).  Roles, TMEM double buffering and bounded waits are as in the main
// GEMM kernel.
#pragma once

#include "operators.h"
#include "pipeline.cuh"

namespace bwgemm {

constexpr int kOrthoK = 128;  // of K per stage

template <int CG>
struct OrthoConfig {
    static constexpr int kTile = 128 * CG;                 // rows and columns of a tile
    static constexpr int kEpiWarps = 8;
    static constexpr int kThreads = 32 * (2 + kEpiWarps);
    static constexpr int kCols = kTile / 2;                // columns per epilogue warp
    static constexpr int kOperandBytes = 128 * kOrthoK * 2;  // 32 KiB: this CTA's 128 rows of A, or of B
    static constexpr int kStages = 3;
    static constexpr int kTmemCols = 2 * kTile;
    static constexpr int kStoreBytes = 4096;               // a warp's 32 x 64 16-bit values
    static constexpr int kIdleBytes = 2 * kStages * kOperandBytes / kEpiWarps;  // of the idle ring, per warp
    static_assert(kIdleBytes % 1024 == 0 && kIdleBytes >= kCols / 64 * 2 * kStoreBytes, "boxes of a tile");
    static constexpr int kOffA = 0;
    static constexpr int kOffB = kStages * kOperandBytes;
    static constexpr int kOffStore = 2 * kStages * kOperandBytes;
    static constexpr int kOffBar = kOffStore + kEpiWarps * kStoreBytes;
    static constexpr int kNumBars = 2 * kStages + 4 + 1;   // full, empty, acc_full[2], acc_empty[2], drain
    static constexpr int kOffTmemSlot = kOffBar + 8 * kNumBars;
    static constexpr int kOffAbort = kOffTmemSlot + 4;
    static constexpr int kSmemBytes = kOffAbort + 4 + 1024;
    static_assert(kSmemBytes <= 227 * 1024, "exceeds the 227 KiB shared memory of one CTA");
};

// Shared-memory descriptor of an MN-major operand block: 128-byte rows of 64
// output elements, one row per k, 128-byte swizzle (8 k per 1 KiB atom: stride
// byte offset); the next 64 output elements lie a whole chunk of kOrthoK rows
// further (leading byte offset).
__device__ __forceinline__ uint64_t make_sdesc_mn(uint32_t smem)
{
    uint64_t d = 0;
    d |= uint64_t((smem & 0x3FFFFu) >> 4);
    d |= uint64_t((kOrthoK * 128) >> 4) << 16;
    d |= uint64_t(1024 >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(2) << 61;
    return d;
}

struct OrthoTile {
    int r, c, matrix;
    int slice, k0, k1;  // slice of K: steps [k0, k1)
};

// K steps of a tile: the operands' terms, and the low part of its diagonal block.
template <int CG>
__device__ __forceinline__ int ortho_steps(const OrthoParams& p)
{
    return p.steps_k * p.terms + (p.low_side ? CG : 0);
}

template <int CG>
__device__ __forceinline__ OrthoTile ortho_tile_at(const OrthoParams& p, int t)
{
    OrthoTile x;
    const int whole = t / p.splits;
    const int steps = ortho_steps<CG>(p);
    x.slice = t - whole * p.splits;
    x.k0 = x.slice * steps / p.splits;
    x.k1 = (x.slice + 1) * steps / p.splits;
    x.matrix = whole / p.tiles;
    const int i = whole - x.matrix * p.tiles;
    if (p.symmetric) {
        // row r of the triangle holds tiles r (r + 1) / 2 .. + r
        int r = int((sqrtf(8.f * float(i) + 1.f) - 1.f) * 0.5f);
        while (r * (r + 1) / 2 > i)
            --r;
        while ((r + 1) * (r + 2) / 2 <= i)
            ++r;
        x.r = r;
        x.c = i - r * (r + 1) / 2;
    } else {
        // groups of 8 tile rows, walked down before stepping along the columns
        const int per_group = 8 * p.num_c;
        const int g = i / per_group;
        const int height = min(p.num_r - 8 * g, 8);
        const int local = i - g * per_group;
        x.r = 8 * g + local % height;
        x.c = local / height;
    }
    return x;
}

// Convert-and-store works on 64 columns of a warp's 32 rows at a time (lane = row,
// 32 packed words = its columns), staged in 4 KiB of the warp's shared memory:
// rows of 128 bytes with the 128-byte swizzle of the result maps (16-byte piece
// XOR row mod 8), or turned, 64 rows of 64 bytes with the 64-byte swizzle (piece
// XOR (row / 2) mod 4).
__device__ __forceinline__ void ortho_stage(const uint32_t (&w)[32], uint32_t sb, int lane)
{
    const uint32_t row = sb + uint32_t(lane * 128);
#pragma unroll
    for (int ch = 0; ch < 8; ++ch)
        ptx::st_shared_v4(row + ((uint32_t(ch) ^ uint32_t(lane & 7)) << 4), w[4 * ch], w[4 * ch + 1], w[4 * ch + 2],
                          w[4 * ch + 3]);
}

__device__ __forceinline__ void ortho_stage_turned(const uint32_t (&w)[32], uint32_t sb, int lane)
{
#pragma unroll
    for (int i = 0; i < 64; ++i)
        ptx::st_shared_u16(sb + uint32_t(i * 64) + ((uint32_t(lane >> 3) ^ uint32_t((i >> 1) & 3)) << 4) +
                               uint32_t((lane & 7) * 2),
                           uint16_t((i & 1) ? (w[i >> 1] >> 16) : (w[i >> 1] & 0xFFFFu)));
}

template <int CG, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(OrthoConfig<CG>::kThreads, 1)
    ortho_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                 const __grid_constant__ CUtensorMap tmap_a2, const __grid_constant__ CUtensorMap tmap_b2,
                 const __grid_constant__ CUtensorMap tmap_out, const __grid_constant__ CUtensorMap tmap_out2,
                 const OrthoParams p)
{
    using Cfg = OrthoConfig<CG>;
    constexpr int STAGES = Cfg::kStages;
    constexpr int TILE = Cfg::kTile;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? ptx::cluster_ctarank() : 0u;
    const int worker = int(blockIdx.x) / CG;
    const int workers = int(gridDim.x) / CG;
    const int total = p.tiles * p.batch * p.splits;  // a unit is a tile, or a slice of its K
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
        ptx::prefetch_tensormap(&tmap_a);
        ptx::prefetch_tensormap(&tmap_b);
        ptx::prefetch_tensormap(&tmap_out);
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
        for (int t = worker; ok && t < total; t += workers) {
            const OrthoTile x = ortho_tile_at<CG>(p, t);
            const int a0 = x.r * TILE + int(rank) * 128;  // this CTA's output rows, and columns of B
            const int b0 = x.c * TILE + int(rank) * 128;
#pragma unroll 1
            for (int i = x.k0; i < x.k1; ++i, ++n) {
                ok = __all_sync(0xffffffffu,
                                pipe_wait(bar_empty + 8 * s, phase ^ 1u, p, abort_flag, kStatusProducerTimeout));
                if (!ok)
                    break;
                const bool stall = p.stall_kblock >= 0 && blockIdx.x == 0 && p.stall_kblock == n;
                if (!stall && rank == 0) {
                    armed_mask |= 1u << s;
                    armed_parity = (armed_parity & ~(1u << s)) | (phase << s);
                }
                if (!stall && ptx::elect_one()) {
                    const bool low = i >= p.steps_k * p.terms;
                    const bool second = !low && i >= p.steps_k;
                    int k = (second ? i - p.steps_k : i) * kOrthoK, za = x.matrix, zb = x.matrix;
                    if (low) {
                        // the block of 128 of the diagonal that this CTA's rows (columns)
                        // lie in; past the last matrix the copy brings zeros
                        const int j = i - p.steps_k * p.terms;
                        const int z = j == int(rank) ? x.matrix + p.batch : 2 * p.batch;
                        k = (p.low_side == 1 ? x.r : x.c) * TILE + j * kOrthoK;
                        za = p.low_side == 1 ? z : za;
                        zb = p.low_side == 1 ? zb : z;
                    }
                    const CUtensorMap* ma = second ? &tmap_a2 : &tmap_a;
                    const CUtensorMap* mb = second ? &tmap_b2 : &tmap_b;
                    const uint32_t fb = leader_full + 8 * s;
                    const uint32_t dA = sA + uint32_t(s * Cfg::kOperandBytes), dB = sB + uint32_t(s * Cfg::kOperandBytes);
                    const int ra = A_MN ? k : a0, ca = (A_MN ? a0 : k) / 64;
                    const int rb = B_MN ? k : b0, cb = (B_MN ? b0 : k) / 64;
                    if (rank == 0)
                        ptx::mbar_arrive_expect_tx(fb, uint32_t(CG * 2 * Cfg::kOperandBytes));
                    // as late as can be: all before it, its instructions' way into the cache
                    // too (1200 to 2000 cycles), overlaps the product before
                    if (n == 0)
                        ptx::grid_dependency_wait();
                    if constexpr (CG == 2) {
                        ptx::tma_load_4d_pair(dA, ma, fb, 0, ra, ca, za);
                        ptx::tma_load_4d_pair(dB, mb, fb, 0, rb, cb, zb);
                    } else {
                        ptx::tma_load_4d(dA, ma, fb, 0, ra, ca, za);
                        ptx::tma_load_4d(dB, mb, fb, 0, rb, cb, zb);
                    }
                }
                __syncwarp();
                if (++s == STAGES) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---------------------------------------------------------- MMA issue
        // A K-major block holds two chunks of 64 k, 16 KiB apart, 32 bytes per
        // MMA; an MN-major one 128 k in rows of 128 bytes, 2 KiB per MMA.
        const uint64_t a_desc0 = A_MN ? make_sdesc_mn(sA) : make_sdesc_sw128(sA);
        const uint64_t b_desc0 = B_MN ? make_sdesc_mn(sB) : make_sdesc_sw128(sB);
        const uint32_t idesc = make_idesc(BWGEMM_FP16, 128 * CG, TILE) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
        const uint32_t tmem0 = __shfl_sync(0xffffffffu, tmem_base, 0);
        int s = 0, b = 0;
        uint32_t phase = 0, bphase = 0;
        bool ok = true;
#pragma unroll 1
        for (int t = worker; ok && t < total; t += workers) {
            const OrthoTile x = ortho_tile_at<CG>(p, t);
            ok = __all_sync(0xffffffffu,
                            pipe_wait(bar_acc_empty + 8 * b, bphase ^ 1u, p, abort_flag, kStatusMmaTimeout));
#pragma unroll 1
            for (int i = x.k0; ok && i < x.k1; ++i) {
                ok = __all_sync(0xffffffffu, pipe_wait(bar_full + 8 * s, phase, p, abort_flag, kStatusMmaTimeout));
                if (!ok)
                    break;
                ptx::tc_fence_after_sync();
                if (ptx::elect_one()) {
                    const uint64_t ad = a_desc0 + uint64_t((s * Cfg::kOperandBytes) >> 4);
                    const uint64_t bd = b_desc0 + uint64_t((s * Cfg::kOperandBytes) >> 4);
#pragma unroll
                    for (int kk = 0; kk < kOrthoK / 16; ++kk) {
                        const uint32_t k_major = uint32_t((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                        const uint32_t mn_major = uint32_t(kk * 2048) >> 4;
                        ptx::mma_f16<CG>(tmem0 + uint32_t(b * TILE), ad + (A_MN ? mn_major : k_major),
                                         bd + (B_MN ? mn_major : k_major), idesc, (i > x.k0 || kk > 0) ? 1u : 0u);
                    }
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
#pragma unroll 1
        for (int t = worker; ok && t < total; t += workers) {
            const OrthoTile x = ortho_tile_at<CG>(p, t);
            const int row0 = x.r * TILE + int(rank) * 128 + 32 * q;
            const int col0 = x.c * TILE + (e >> 2) * Cfg::kCols;
            const int row = row0 + lane;
            const float factor = p.alpha_dev ? ptx::ld_global_cg_f32(p.alpha_dev + x.matrix) : 1.f;  // on its way until the sums are there
            const bool mirror = p.symmetric && x.r != x.c;
            // The CTA's last tile: once its sums are there, the ring has been read and
            // takes the result's boxes, so that none waits for the one before it to leave.
            const bool idle = t + workers >= total;
            uint32_t box = idle ? base + uint32_t(e * Cfg::kIdleBytes) : sb;
            // The epilogue is bound by its own instructions (8 warps share four
            // schedulers with the issuing ones, and a 256-wide tile is 128 columns a
            // thread), so what only some products need is tested once per 64
            // columns, and fp32 values go in pairs.
            uint64_t alpha2 = 0;
            const uint64_t beta2 = ptx::pack_f32x2(__float_as_uint(p.beta), __float_as_uint(p.beta));
            // E's 64 columns, loaded before the sums are waited for, later ones a
            // piece ahead: four rows of 128 bytes at a time (eight lanes each), turned
            // to a row per lane through the staging block
            const uint16_t* const e_at = p.e + x.matrix * p.stride_e + (row0 + (lane >> 3)) * p.lde + col0 + 8 * (lane & 7);
            uint4 add[8];
            auto fetch = [&](int c) {
                if (p.e != nullptr && c < Cfg::kCols) {
                    const bool in = col0 + c + 8 * (lane & 7) < p.store_cols;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        add[i] = in && row0 + 4 * i + (lane >> 3) < p.rows
                                     ? ptx::ld_global_cg_v4(e_at + c + 4 * i * p.lde)
                                     : make_uint4(0u, 0u, 0u, 0u);
                }
            };
            fetch(0);
            // 64 columns of the finished sums (this lane's row) to D
            auto finish = [&](int c, const uint32_t(&v)[64]) {
                const int col = col0 + c;
                // the box itself, and its mirror image: columns of D from its rows, up
                // to the padded width (zeros there, which later products read)
                const bool direct = row0 < p.rows && col < p.store_cols;
                const bool mirrored = mirror && col < p.rows && row0 < p.store_cols;
                if (!direct && !mirrored)
                    return;
                auto claim = [&] {  // the store before has read the staging block
                    if (idle)
                        return;
                    if (lane == 0)
                        ptx::bulk_wait_group_read<0>();
                    __syncwarp();
                };
                uint64_t f[32];
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    f[i] = ptx::mul_f32x2(ptx::pack_f32x2(v[2 * i], v[2 * i + 1]), alpha2);
                if (p.e != nullptr) {
                    claim();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        ptx::st_shared_v4(box + uint32_t((4 * i + (lane >> 3)) * 128) +
                                              (uint32_t((lane & 7) ^ ((4 * i + (lane >> 3)) & 7)) << 4),
                                          add[i].x, add[i].y, add[i].z, add[i].w);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        uint32_t w[4];
                        ptx::ld_shared_v4(box + uint32_t(lane * 128) + (uint32_t((i >> 2) ^ (lane & 7)) << 4), w[0], w[1],
                                          w[2], w[3]);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                            f[i + k] = ptx::fma_f32x2(ptx::pack_f32x2(__float_as_uint(g.x), __float_as_uint(g.y)), beta2,
                                                      f[i + k]);
                        }
                    }
                    __syncwarp();
                }
                fetch(c + 64);
                if (p.diag != 0.f && row0 < col + 64 && col < row0 + 32) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float lo, hi;
                        ptx::unpack_f32x2(f[i], lo, hi);
                        lo += row == col + 2 * i ? p.diag : 0.f;
                        hi += row == col + 2 * i + 1 ? p.diag : 0.f;
                        f[i] = ptx::pack_f32x2(__float_as_uint(lo), __float_as_uint(hi));
                    }
                }
                uint32_t w[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    float lo, hi;
                    ptx::unpack_f32x2(f[i], lo, hi);
                    w[i] = pack2(__float_as_uint(lo), __float_as_uint(hi), p.out_bf16 ? 0 : 1);
                }
                auto put = [&](const CUtensorMap* map, int at_col, int at_row, int z) {
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::tma_store_3d(map, box, at_col, at_row, z);
                        ptx::bulk_commit_group();
                    }
                    if (idle)
                        box += Cfg::kStoreBytes;
                };
                if (p.plain_store) {
                    // the caller's rows are not on 16-byte boundaries: the block goes
                    // through shared memory and out a row at a time, two columns a lane
                    __syncwarp();
                    ortho_stage(w, sb, lane);
                    __syncwarp();
                    uint16_t* dst = p.out + x.matrix * p.stride_o + row0 * p.ldo + col;
                    const int n = min(32, p.rows - row0);
#pragma unroll 1
                    for (int i = 0; i < n; ++i)
#pragma unroll
                        for (int k = lane; k < 64; k += 32)
                            if (col + k < p.cols)
                                dst[i * p.ldo + k] = ptx::ld_shared_u16(
                                    sb + uint32_t(i * 128) + ((uint32_t(k >> 3) ^ uint32_t(i & 7)) << 4) +
                                    uint32_t((k & 7) * 2));
                    return;
                }
                if (direct) {
                    claim();
                    ortho_stage(w, box, lane);
                    put(&tmap_out, col, row0, x.matrix);
                }
                if (mirrored) {
                    claim();
                    ortho_stage_turned(w, box, lane);
                    put(&tmap_out2, row0, col, x.matrix);
                }
                if (p.low && direct && !mirror) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float lo, hi;
                        ptx::unpack_f32x2(f[i], lo, hi);
                        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                        w[i] = pack2(__float_as_uint(lo - h.x), __float_as_uint(hi - h.y), 1);
                    }
                    claim();
                    ortho_stage(w, box, lane);
                    if (p.symmetric)
                        put(&tmap_out, col, row0, x.matrix + p.batch);
                    else
                        put(&tmap_out2, col, row0, x.matrix);
                }
            };
            ok = __all_sync(0xffffffffu,
                            pipe_wait(bar_acc_full + 8 * b, bphase, p, abort_flag, kStatusEpilogueTimeout));
            if (!ok)
                break;
            ptx::tc_fence_after_sync();
            const float alpha = p.alpha * factor;
            alpha2 = ptx::pack_f32x2(__float_as_uint(alpha), __float_as_uint(alpha));
            const uint32_t taddr = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(b * TILE + (e >> 2) * Cfg::kCols);
            if (p.splits == 1) {
#pragma unroll 1
                for (int c = 0; c < Cfg::kCols; c += 64) {
                    uint32_t v[64];
                    ptx::tmem_ld_32x32b_x64(taddr + uint32_t(c), v);
                    ptx::tmem_ld_wait();
                    if (c + 64 >= Cfg::kCols)
                        hand_back<CG>(bar_acc_empty + 8 * b, lane);
                    finish(c, v);
                }
            } else {
                // a slice of K: its sums to global memory, where ortho_join_kernel adds
                // them; lanes next to each other, so a warp's store is 512 bytes
                float* const part = p.partials + (size_t(t) * CG + rank) * (128 * TILE) + e * (32 * Cfg::kCols) + 4 * lane;
#pragma unroll 1
                for (int c = 0; c < Cfg::kCols; c += 32) {
                    uint32_t v[32];
                    ptx::tmem_ld_32x32b_x32(taddr + uint32_t(c), v);
                    ptx::tmem_ld_wait();
                    if (c + 32 >= Cfg::kCols)
                        hand_back<CG>(bar_acc_empty + 8 * b, lane);
                    if (row0 < p.store_cols && col0 + c < p.store_cols) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            ptx::st_global_cg_v4(part + c * 32 + i * 128,
                                                 make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
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

// Adds the slices of a symmetric product's tiles: D = alpha times the sums, stored
// twice where the tile lies below the diagonal.  A warp takes 32 rows x 4 columns of
// a tile (512 bytes of a slice) and every join_share-th slice; the sums of that many
// warps meet in shared memory, in order.
constexpr int kJoinWarps = 8;

template <int CG>
__global__ void __launch_bounds__(32 * kJoinWarps) ortho_join_kernel(const OrthoParams p)
{
    using Cfg = OrthoConfig<CG>;
    constexpr int TILE = Cfg::kTile, CHUNKS = Cfg::kCols / 32;
    __shared__ float4 sums[kJoinWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int share = p.join_share, first = warp % share;
    const int piece = int(blockIdx.x) * (kJoinWarps / share) + warp / share;
    const int i = piece % 8, c = piece / 8 % CHUNKS * 32, e = piece / (8 * CHUNKS) % 8, rank = piece / (64 * CHUNKS);
    const int t = int(blockIdx.y) * p.splits;
    const OrthoTile x = ortho_tile_at<CG>(p, t);
    const int row0 = x.r * TILE + rank * 128 + 32 * ((e + 2) & 3), row = row0 + lane;
    const int col = x.c * TILE + (e >> 2) * Cfg::kCols + c + 4 * i;
    const bool mirror = x.r != x.c;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const float factor = p.alpha_dev ? ptx::ld_global_cg_f32(p.alpha_dev + x.matrix) : 1.f;
    const float* at = p.partials + (size_t(t) * CG + rank) * (128 * TILE) + e * (32 * Cfg::kCols) + c * 32 + i * 128 + 4 * lane;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if ((row0 < p.rows && col < p.store_cols) || (mirror && col < p.rows && row0 < p.store_cols)) {
#pragma unroll 8
        for (int k = first; k < p.splits; k += share) {
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
    const float alpha = p.alpha * factor;
    const uint32_t lo = pack2(__float_as_uint(f.x * alpha), __float_as_uint(f.y * alpha), 1);
    const uint32_t hi = pack2(__float_as_uint(f.z * alpha), __float_as_uint(f.w * alpha), 1);
    uint16_t* const out = p.out + x.matrix * p.stride_o;
    if (row < p.rows && col < p.store_cols)
        *reinterpret_cast<uint2*>(out + row * p.ldo + col) = make_uint2(lo, hi);
    if (mirror && row < p.store_cols) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (col + k < p.rows)
                out[(col + k) * p.ldo + row] = uint16_t((k < 2 ? lo : hi) >> (k & 1 ? 16 : 0));
    }
}

}  // namespace bwgemm
