// scaled_few_sm103.cu -- the block-scaled 8-bit product for one to sixteen rows
// of A (one generated token, a few beams): C = A B^T as in scaled_kernel.cuh.
//
// The weights' bytes are the time: N x K read once.  A tile of a few rows does
// not repay tcgen05's path (copies into shared memory, barriers, an accumulator
// handed over per K block) until there are many of them, so here the weights go
// from memory straight into the registers of mma.sync: 8 weight rows are the
// columns of m16n8k32, the rows of A its 16 rows.  The contraction does not care
// which K a position stands for as long as both operands agree, so every lane
// loads whole 16-byte pieces: lane (g, q) takes bytes 16 q and 64 + 16 q of weight
// row g's 128-byte block, and the same bytes of rows g and g + 8 of A; four MMAs
// consume a block.  The block's fresh accumulator is weighted with both scales and
// added to the running sums.
//
// Measured at one row: 1024 x 1024 1.7 us (tiles: 6.9), 4096 x 4096 4.8 (11.2),
// 8192 x 8192 17.3 (18.8), 3.9 TB/s: the loads in flight bound it, and what a
// block waits for besides them, its scales and A's piece out of L1 or L2.  Larger
// products are left to the tiles' copies, which keep more bytes in flight.
//
// A CTA takes 8 weight rows -- many small CTAs, so that the last ones do not run
// alone (16 rows: 18.4 us) -- and its eight warps take the K blocks in turn, kAhead
// blocks in flight each, and add their sums through shared memory in warp order.
// Two blocks ahead and four CTAs per SM were the best of 2, 4, 6 and 3 to 5: deeper
// needs the registers of a CTA (four ahead at the same bound spill: 20.2 us).
#include "operators.h"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace bwgemm {
namespace {

constexpr int kFewWarps = 8;
constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kFewRows = 8;  // weight rows per CTA
constexpr int kAhead = 2;    // blocks of weights in flight per warp

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

    // the block's sums, weighted, onto the running ones; x(t, h) is A's part
    auto add = [&](const uint4& lo, const uint4& hi, int kb, auto&& x) {
        const float* ws = p.ws + int64_t(kb) * p.ws_ld;
        const float* xs = p.xs + int64_t(kb) * p.xs_ld;
        const float w0 = ptx::ld_global_ca_f32(ws + ws_of[0]), w1 = ptx::ld_global_ca_f32(ws + ws_of[1]);
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
            const float s = ptx::ld_global_ca_f32(xs + (m_of[t] >> p.xs_shift));
            sum[t][0] = fmaf(d[2 * t], s * w0, sum[t][0]);
            sum[t][1] = fmaf(d[2 * t + 1], s * w1, sum[t][1]);
        }
    };

    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int whole = p.K / kBlock;
    uint4 w[kAhead][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int kb = warp + i * kFewWarps;
        if (kb < whole) {
            w[i][0] = ptx::ld_global_stream_v4(w_at + int64_t(kb) * kBlock);
            w[i][1] = ptx::ld_global_stream_v4(w_at + int64_t(kb) * kBlock + 64);
        }
    }
#pragma unroll 1
    for (int kb0 = warp; kb0 < whole; kb0 += kAhead * kFewWarps) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int kb = kb0 + i * kFewWarps;
            if (kb < whole) {
                add(w[i][0], w[i][1], kb,
                    [&](int t, int h) { return ptx::ld_global_ca_v4(x_at[t] + int64_t(kb) * kBlock + 64 * h); });
                const int next = kb + kAhead * kFewWarps;
                if (next < whole) {
                    w[i][0] = ptx::ld_global_stream_v4(w_at + int64_t(next) * kBlock);
                    w[i][1] = ptx::ld_global_stream_v4(w_at + int64_t(next) * kBlock + 64);
                }
            }
        }
    }
    if (whole < p.num_kb && warp == whole % kFewWarps) {  // the last block, cut off by the end of the rows
        const int k = whole * kBlock + 16 * q;
        add(load_ragged(w_at - 16 * q, k, p.K), load_ragged(w_at - 16 * q, k + 64, p.K), whole,
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
