// few_rows_sm103.cu -- one to sixteen rows of X (one generated token, a few beams) times
// weights of 8-bit integers, or times both weights of the gated layer.
//
// The weights' bytes are the time: each is read once.  16 weight rows are the rows of
// mma.sync's m16n8k32 (integers: exact 32-bit sums) or m16n8k16 (bf16, fp16), rows of X its
// 8 columns.  (The integer instruction is slow on this GPU: one row of X, 8192 x 8192, keeps
// the tensor pipe busy 56 % of the time; one and two rows take dot products instead.)  In the
// gated form rows 0 to 7 are Wg's and 8 to 15 the same rows of Wu: a lane's accumulator then
// holds G in its first half and U of the same outputs in its second.
// The contraction does not care which K a position stands for as long as both operands
// agree, so lane (g, q) takes whole 16-byte pieces: bytes 16 q and 64 + 16 q of rows g and
// g + 8 of a 128-byte block, and of rows g (and g + 8) of X; four MMAs consume it.
//
// A CTA takes 16 weight rows, its eight warps the blocks of their K in turn, kFewRing blocks
// in flight each (asynchronous copies that every lane makes and reads for itself: nobody
// waits for anybody), and their sums meet in shared memory in warp order.  Measured at one
// row: integers 8192 x 8192 12.5 to 12.9 us (5.3 TB/s), 28672 x 8192 36.9 (6.4 TB/s); gated 10240 x 8192
// 50 to 52 (6.6 TB/s, 95 to 98 % of the copy rate).  Rings of four blocks: 15.9 us on 8192 x 8192.
#include "activation.cuh"
#include "feed_forward.h"
#include "gemm_kernel.cuh"
#include "int8_scales.cuh"

namespace bwgemm {
namespace {

constexpr int kFewRing = 3;
constexpr int kFewBlock = 2048;  // 16 rows of 128 bytes

// 16 bytes of a row at byte k, zeros from byte `len` on, where nothing is read.
__device__ __forceinline__ uint4 load_ragged(const uint8_t* row, int64_t k, int64_t len)
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

// D (16 weight rows x 8 rows of X) += 16 bytes a row of either.
template <int KIND>
__device__ __forceinline__ void mma_piece(uint32_t (&d)[4], const uint4& lo, const uint4& hi, const uint4& x)
{
#define BWGEMM_MMA(OP, C, A0, A1, A2, A3, B0, B1)                                                                       \
    asm volatile("mma.sync.aligned." OP " {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"              \
                 : C(d[0]), C(d[1]), C(d[2]), C(d[3])                                                                   \
                 : "r"(A0), "r"(A1), "r"(A2), "r"(A3), "r"(B0), "r"(B1))
    if constexpr (KIND == kFewInt8) {
        BWGEMM_MMA("m16n8k32.row.col.s32.s8.s8.s32", "+r", lo.x, hi.x, lo.y, hi.y, x.x, x.y);
        BWGEMM_MMA("m16n8k32.row.col.s32.s8.s8.s32", "+r", lo.z, hi.z, lo.w, hi.w, x.z, x.w);
    } else if constexpr (KIND == kFewBf16) {
        BWGEMM_MMA("m16n8k16.row.col.f32.bf16.bf16.f32", "+r", lo.x, hi.x, lo.y, hi.y, x.x, x.y);
        BWGEMM_MMA("m16n8k16.row.col.f32.bf16.bf16.f32", "+r", lo.z, hi.z, lo.w, hi.w, x.z, x.w);
    } else {
        BWGEMM_MMA("m16n8k16.row.col.f32.f16.f16.f32", "+r", lo.x, hi.x, lo.y, hi.y, x.x, x.y);
        BWGEMM_MMA("m16n8k16.row.col.f32.f16.f16.f32", "+r", lo.z, hi.z, lo.w, hi.w, x.z, x.w);
    }
#undef BWGEMM_MMA
}

__device__ __forceinline__ uint16_t round_to(float v, int dtype)
{
    return dtype == BWGEMM_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

// One lane's part of 16 bytes of a weight row and of a row of X.
__device__ __forceinline__ void dot_piece(uint32_t& d, const uint4& w, const uint4& x)
{
    int v = int(d);
    v = __dp4a(int(w.x), int(x.x), v);
    v = __dp4a(int(w.y), int(x.y), v);
    v = __dp4a(int(w.z), int(x.z), v);
    v = __dp4a(int(w.w), int(x.w), v);
    d = uint32_t(v);
}

// NT: groups of 8 rows of X (1 or 2).  DOTS: no matrix instructions, but a dot product of four
// integers at a time for each of DOTS rows of X (0: none).
template <int KIND, int NT, int DOTS, int kFewWarps>
__global__ void __launch_bounds__(32 * kFewWarps, 32 / kFewWarps) few_rows_kernel(const FewRowsParams p)
{
    constexpr bool INT8 = KIND == kFewInt8;
    constexpr int ROWS = few_rows(KIND);
    extern __shared__ __align__(16) uint8_t few_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const int n0 = int(blockIdx.x) * ROWS;
    // rows past the end repeat the last one: whatever they give is not stored
    const uint8_t* const w0 = p.w[0] + int64_t(min(n0 + g, p.N - 1)) * p.ldw[0];
    const uint8_t* const w1 = INT8 ? p.w[0] + int64_t(min(n0 + 8 + g, p.N - 1)) * p.ldw[0]
                                   : p.w[1] + int64_t(min(n0 + g, p.N - 1)) * p.ldw[1];
    static_assert(DOTS == 0 || (INT8 && NT == 1 && DOTS <= 2), "integers, few rows");
    constexpr int XT = DOTS > 0 ? DOTS : NT;  // rows of X whose pieces a lane loads
    const uint8_t* x_at[XT];
#pragma unroll
    for (int t = 0; t < XT; ++t)
        x_at[t] = p.x + int64_t(min(DOTS > 0 ? t : 8 * t + g, p.M - 1)) * p.ldx;
    uint32_t sum[XT][4];  // (DOTS: of weight rows g and g + 8, in 0 and 1)
#pragma unroll
    for (int t = 0; t < XT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            sum[t][i] = 0u;

    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int whole = int(p.row_bytes / 128);
    const uint32_t ring = ptx::smem_addr(few_smem) + uint32_t(warp * kFewRing * kFewBlock + 16 * lane);
    auto fetch = [&](int kb, int slot) {
        if (kb < whole) {
            const int64_t at = int64_t(kb) * 128 + 16 * q;
            const uint32_t to = ring + uint32_t(slot * kFewBlock);
            ptx::cp_async_16(to, w0 + at);
            ptx::cp_async_16(to + 512, w0 + at + 64);
            ptx::cp_async_16(to + 1024, w1 + at);
            ptx::cp_async_16(to + 1536, w1 + at + 64);
        }
        ptx::cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kFewRing; ++i)
        fetch(warp + i * kFewWarps, i);
    int slot = 0;
#pragma unroll 1
    for (int kb = warp; kb < whole; kb += kFewWarps) {
        uint4 x[XT][2];
#pragma unroll
        for (int t = 0; t < XT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                x[t][h] = ptx::ld_global_ca_v4(x_at[t] + int64_t(kb) * 128 + 64 * h + 16 * q);
        ptx::cp_async_wait_group<kFewRing - 1>();
        uint4 lo[2], hi[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = ring + uint32_t(slot * kFewBlock + 512 * h);
            ptx::ld_shared_v4(at, lo[h].x, lo[h].y, lo[h].z, lo[h].w);
            ptx::ld_shared_v4(at + 1024, hi[h].x, hi[h].y, hi[h].z, hi[h].w);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < XT; ++t) {
                if constexpr (DOTS > 0) {
                    dot_piece(sum[t][0], lo[h], x[t][h]);
                    dot_piece(sum[t][1], hi[h], x[t][h]);
                } else {
                    mma_piece<KIND>(sum[t], lo[h], hi[h], x[t][h]);
                }
            }
        fetch(kb + kFewRing * kFewWarps, slot);
        slot = slot + 1 == kFewRing ? 0 : slot + 1;
    }
    if (int64_t(whole) * 128 < p.row_bytes && warp == whole % kFewWarps) {  // the last block, cut off by the end of the rows
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = int64_t(whole) * 128 + 64 * h + 16 * q;
            const uint4 lo = load_ragged(w0, k, p.row_bytes), hi = load_ragged(w1, k, p.row_bytes);
#pragma unroll
            for (int t = 0; t < XT; ++t) {
                const uint4 x = load_ragged(x_at[t], k, p.row_bytes);
                if constexpr (DOTS > 0) {
                    dot_piece(sum[t][0], lo, x);
                    dot_piece(sum[t][1], hi, x);
                } else {
                    mma_piece<KIND>(sum[t], lo, hi, x);
                }
            }
        }
    }

    // [warp][row of X][weight row], over the ring
    ptx::cp_async_wait_all();
    __syncthreads();
    uint32_t* const part = reinterpret_cast<uint32_t*>(few_smem);
    constexpr int kX = DOTS > 0 ? DOTS : 8 * NT;
    if constexpr (DOTS > 0) {
#pragma unroll
        for (int t = 0; t < DOTS; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                int v = int(sum[t][i]);
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                if (q == 0)
                    part[(warp * kX + t) * 16 + g + 8 * i] = uint32_t(v);
            }
    } else {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[(warp * kX + 8 * t + 2 * q + (i & 1)) * 16 + g + (i >> 1) * 8] = sum[t][i];
    }
    __syncthreads();
    const int r = int(threadIdx.x) % ROWS, m = int(threadIdx.x) / ROWS, n = n0 + r;
    if (m >= min(p.M, kX) || n >= p.N)
        return;
    auto total = [&](int row) {
        if constexpr (INT8) {
            int v = 0;
#pragma unroll
            for (int w = 0; w < kFewWarps; ++w)
                v += int(part[(w * kX + m) * 16 + row]);
            return float(v);
        } else {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kFewWarps; ++w)
                v += __uint_as_float(part[(w * kX + m) * 16 + row]);
            return v;
        }
    };
    if constexpr (INT8) {
        const float v = scaled_sum(total(r), p.cs[m], p.ls[n]);
        const int64_t at = int64_t(m) * p.ldo[0] + n;
        if (p.out_type == BWGEMM_FP32)
            static_cast<float*>(p.out[0])[at] = v;
        else
            static_cast<uint16_t*>(p.out[0])[at] = round_to(v, p.out_type);
    } else {
        const float gate = total(r), up = total(r + 8);
        static_cast<uint16_t*>(p.out[0])[int64_t(m) * p.ldo[0] + n] = round_to(activate(gate, p.activation) * up, p.out_type);
        if (p.out[1] != nullptr) {
            static_cast<uint16_t*>(p.out[1])[int64_t(m) * p.ldo[1] + n] = round_to(gate, p.out_type);
            static_cast<uint16_t*>(p.out[2])[int64_t(m) * p.ldo[2] + n] = round_to(up, p.out_type);
        }
    }
}

template <int KIND, int NT, int DOTS, int WARPS>
cudaError_t launch_one(const FewRowsParams& p, cudaStream_t stream, bool pdl)
{
    constexpr int kRows = few_rows(KIND), kSmem = WARPS * kFewRing * kFewBlock;
    auto kernel = few_rows_kernel<KIND, NT, DOTS, WARPS>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_smem(kernel, kSmem, allowed);
    if (err != cudaSuccess)
        return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((p.N + kRows - 1) / kRows), 1, 1);
    cfg.blockDim = dim3(32 * WARPS, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int KIND, int NT, int DOTS = 0>
cudaError_t launch_warps(int warps, const FewRowsParams& p, cudaStream_t stream, bool pdl)
{
    switch (warps) {
    case 8: return launch_one<KIND, NT, DOTS, 8>(p, stream, pdl);
    case 16: return launch_one<KIND, NT, DOTS, 16>(p, stream, pdl);
    case 32: return launch_one<KIND, NT, DOTS, 32>(p, stream, pdl);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_few_rows(int kind, int warps, const FewRowsParams& p, cudaStream_t stream, bool pdl)
{
    // (us, dot products against matrix instructions: 1 x 8192 x 8192 12.5 and 14.2, 2 rows 12.6 and
    // 14.2, 4 rows 14.2 and 14.2; 1 x 512 x 28672 8.3 and 10.9)
    if (kind == kFewInt8 && p.M <= 2)
        return p.M == 1 ? launch_warps<kFewInt8, 1, 1>(warps, p, stream, pdl)
                        : launch_warps<kFewInt8, 1, 2>(warps, p, stream, pdl);
    switch (2 * kind + (p.M > 8)) {
    case 2 * kFewInt8: return launch_warps<kFewInt8, 1>(warps, p, stream, pdl);
    case 2 * kFewInt8 + 1: return launch_warps<kFewInt8, 2>(warps, p, stream, pdl);
    case 2 * kFewBf16: return launch_warps<kFewBf16, 1>(warps, p, stream, pdl);
    case 2 * kFewBf16 + 1: return launch_warps<kFewBf16, 2>(warps, p, stream, pdl);
    case 2 * kFewFp16: return launch_warps<kFewFp16, 1>(warps, p, stream, pdl);
    case 2 * kFewFp16 + 1: return launch_warps<kFewFp16, 2>(warps, p, stream, pdl);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace bwgemm
