// scaled_few_sm103.cu -- the block-scaled 8-bit product for one to sixteen rows
// of A (one generated token, a few beams): C = A B^T as in scaled_kernel.cuh.
//
// The weights' bytes are the time: N x K read once.  A tile of a few rows does
// not repay tcgen05's path (copies by TMA, barriers, an accumulator handed over per K
// block) until there are many of them, so here every lane copies the pieces that it
// needs itself and gives them to mma.sync from registers: 8 weight rows are the
// columns of m16n8k32, the rows of A its 16 rows.  The contraction does not care
// which K a position stands for as long as both operands agree, so every lane
// loads whole 16-byte pieces: lane (g, q) takes bytes 16 q and 64 + 16 q of weight
// row g's 128-byte block, and the same bytes of rows g and g + 8 of A; four MMAs
// consume a block.  The block's fresh accumulator is weighted with both scales and
// added to the running sums.
//
// Measured at one row, us with other weights in every call, so that they come from HBM
// (with the same weights, from L2): 1024 x 1024 1.5 (1.7; tiles 5.9), 4096 x 4096 6.3
// (4.9; tiles 10.6), 8192 x 8192 16.7 (12.2; tiles 19.0), 4 TB/s, 128 x 28672 16.5 (8.9;
// tiles 29.7).  Neither deeper rings nor more or fewer CTAs per SM help, and a persistent
// form that copies ahead into the next rows is slower (19.1) by the instructions it adds: a
// warp's own way through a block bounds it.  Larger products are left to the tiles.
//
// A CTA takes 8 weight rows -- many small CTAs, so that the last ones do not run
// alone (16 rows: 18.4 us) -- and its eight warps take the K blocks in turn, kRing
// blocks in flight each (asynchronous copies, which need no registers: with two
// blocks in registers 17.3 us, and 14.8 on 128 x 28672), the scales one block ahead,
// and add their sums through shared memory in warp order.
#include "operators.h"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace bwgemm {
namespace {

constexpr int kFewWarps = 8;
constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kFewRows = 8;  // weight rows per CTA
constexpr int kRing = 4;     // blocks of weights in flight per warp
constexpr int kFewSmem = kFewWarps * kRing * 1024;

// 16 bytes of a row at byte k, zeros from byte `len` on, where nothing is read
// (a row may end inside them).
__device__ __forceinline__ uint4 load_ragged(const uint8_t* row, int k, int len)
{
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (k + 16 <= len)
        return ptx::ld_global_cg_v4(row + k);
    uint32_t* w = &v.x;
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (k + i < len)
            w[i / 4] |= uint32_t(row[k + i]) << (8 * (i % 4));
    return v;
}

// D (16 rows of A x 8 weight rows) += A's piece times the weights' piece.
template <int F8X, int F8W>
__device__ __forceinline__ void mma_fp8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
#define BWGEMM_MMA(TA, TB)                                                                                      \
    asm volatile("mma.sync.aligned.m16n8k32.row.col.f32." TA "." TB ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, " \
                 "{%8, %9}, {%0, %1, %2, %3};"                                                                 \
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                              \
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
    if constexpr (F8X == 0 && F8W == 0)
        BWGEMM_MMA("e4m3", "e4m3");
    else if constexpr (F8X == 0)
        BWGEMM_MMA("e4m3", "e5m2");
    else if constexpr (F8W == 0)
        BWGEMM_MMA("e5m2", "e4m3");
    else
        BWGEMM_MMA("e5m2", "e5m2");
#undef BWGEMM_MMA
}

// NT: groups of 8 rows of A (1 or 2).
template <int NT, int F8W, int F8X>
__global__ void __launch_bounds__(kFewThreads, NT == 1 ? 4 : 3) scaled_few_kernel(const FewParams p)
{
    extern __shared__ __align__(16) uint8_t few_smem[];
    __shared__ float part[kFewWarps][8 * NT][kFewRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const int n0 = int(blockIdx.x) * kFewRows;
    // rows past the end repeat the last one: whatever they give is not stored
    const uint8_t* const w_at = p.w + int64_t(min(n0 + g, p.N - 1)) * p.ldw + 16 * q;
    const int ws_of[2] = {min(n0 + 2 * q, p.N - 1) >> p.ws_shift, min(n0 + 2 * q + 1, p.N - 1) >> p.ws_shift};
    int m_of[NT];
    const uint8_t* x_at[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        m_of[t] = min(8 * t + g, p.M - 1);
        x_at[t] = p.x + int64_t(m_of[t]) * p.ldx + 16 * q;
    }
    float sum[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        sum[t][0] = sum[t][1] = 0.f;

    struct Scales {
        float w0, w1, x[NT];
    };
    auto scales_of = [&](int kb) {
        Scales f;
        const float* ws = p.ws + int64_t(kb) * p.ws_ld;
        const float* xs = p.xs + int64_t(kb) * p.xs_ld;
        f.w0 = ptx::ld_global_ca_f32(ws + ws_of[0]);
        f.w1 = ptx::ld_global_ca_f32(ws + ws_of[1]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
            f.x[t] = ptx::ld_global_ca_f32(xs + (m_of[t] >> p.xs_shift));
        return f;
    };
    // the block's sums, weighted, onto the running ones; x(t, h) is A's part
    auto add = [&](const uint4& lo, const uint4& hi, const Scales& f, auto&& x) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 w = h ? hi : lo;
            const uint4 a = x(0, h);
            uint4 b = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (NT == 2)
                b = x(1, h);
            mma_fp8<F8X, F8W>(d, a.x, b.x, a.y, b.y, w.x, w.y);
            mma_fp8<F8X, F8W>(d, a.z, b.z, a.w, b.w, w.z, w.w);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            sum[t][0] = fmaf(d[2 * t], f.x[t] * f.w0, sum[t][0]);
            sum[t][1] = fmaf(d[2 * t + 1], f.x[t] * f.w1, sum[t][1]);
        }
    };

    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int whole = p.K / kBlock;
    // every lane copies and reads its own pieces only: nobody waits for anybody
    const uint32_t ring = ptx::smem_addr(few_smem) + uint32_t(warp * kRing * 1024 + 16 * lane);
    auto fetch = [&](int kb, int slot) {
        if (kb < whole) {
            ptx::cp_async_16(ring + uint32_t(slot * 1024), w_at + int64_t(kb) * kBlock);
            ptx::cp_async_16(ring + uint32_t(slot * 1024 + 512), w_at + int64_t(kb) * kBlock + 64);
        }
        ptx::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i)
        fetch(warp + i * kFewWarps, i);
    int slot = 0;
    Scales next = {};
    if (warp < whole)
        next = scales_of(warp);
#pragma unroll 1
    for (int kb = warp; kb < whole; kb += kFewWarps) {
        const Scales f = next;
        if (kb + kFewWarps < whole)
            next = scales_of(kb + kFewWarps);
        ptx::cp_async_wait_group<kRing - 1>();
        uint4 lo, hi;
        ptx::ld_shared_v4(ring + uint32_t(slot * 1024), lo.x, lo.y, lo.z, lo.w);
        ptx::ld_shared_v4(ring + uint32_t(slot * 1024 + 512), hi.x, hi.y, hi.z, hi.w);
        add(lo, hi, f, [&](int t, int h) { return ptx::ld_global_ca_v4(x_at[t] + int64_t(kb) * kBlock + 64 * h); });
        fetch(kb + kRing * kFewWarps, slot);
        slot = slot + 1 == kRing ? 0 : slot + 1;
    }
    if (whole < p.num_kb && warp == whole % kFewWarps) {  // the last block, cut off by the end of the rows
        const int k = whole * kBlock + 16 * q;
        add(load_ragged(w_at - 16 * q, k, p.K), load_ragged(w_at - 16 * q, k + 64, p.K), scales_of(whole),
            [&](int t, int h) { return load_ragged(x_at[t] - 16 * q, k + 64 * h, p.K); });
    }

#pragma unroll
    for (int t = 0; t < NT; ++t) {
        part[warp][8 * t + g][2 * q] = sum[t][0];
        part[warp][8 * t + g][2 * q + 1] = sum[t][1];
    }
    __syncthreads();
    const int m = int(threadIdx.x) / kFewRows, n = n0 + int(threadIdx.x) % kFewRows;
    if (m < p.M && m < 8 * NT && n < p.N) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kFewWarps; ++i)
            v += part[i][m][threadIdx.x % kFewRows];
        const int64_t at = int64_t(m) * p.ldc + n;
        if (p.out_type == BWGEMM_FP32) {
            float* c = static_cast<float*>(p.c) + at;
            *c = p.accumulate ? *c + v : v;
        } else if (p.out_type == BWGEMM_BF16) {
            static_cast<__nv_bfloat16*>(p.c)[at] = __float2bfloat16_rn(v);
        } else {
            static_cast<__half*>(p.c)[at] = __float2half_rn(v);
        }
    }
}

template <int NT, int F8W, int F8X>
cudaError_t launch_few(const FewParams& p, cudaStream_t stream, bool pdl)
{
    cudaLaunchConfig_t cfg = {};
    cfg.dynamicSmemBytes = kFewSmem;
    cfg.gridDim = dim3(unsigned((p.N + kFewRows - 1) / kFewRows), 1, 1);
    cfg.blockDim = dim3(kFewThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, scaled_few_kernel<NT, F8W, F8X>, p);
}

template <int NT>
cudaError_t launch_types(int w_type, int x_type, const FewParams& p, cudaStream_t stream, bool pdl)
{
    if (w_type == BWGEMM_E4M3)
        return x_type == BWGEMM_E4M3 ? launch_few<NT, 0, 0>(p, stream, pdl) : launch_few<NT, 0, 1>(p, stream, pdl);
    return x_type == BWGEMM_E4M3 ? launch_few<NT, 1, 0>(p, stream, pdl) : launch_few<NT, 1, 1>(p, stream, pdl);
}

}  // namespace

cudaError_t launch_scaled_few(int w_type, int x_type, const FewParams& p, cudaStream_t stream, bool pdl)
{
    return p.M <= 8 ? launch_types<1>(w_type, x_type, p, stream, pdl) : launch_types<2>(w_type, x_type, p, stream, pdl);
}

}  // namespace bwgemm
