// quantize_sm103.cu -- a matrix to 8-bit floating point in blocks of 128 with
// one fp32 scale each, along the rows and, in the same pass, along the columns.
//
// For every block b (1 x 128 along a row; with `square` 128 x 128):
//
//   a_b = max(max_b |x|, 2^-100)      limit = 448 (e4m3) or 57344 (e5m2)
//   scale_b = a_b / limit             factor_b = limit / a_b
//   pow2:  scale_b = the next power of two >= a_b / limit, factor_b = 1 / scale_b
//   q = round_to_nearest_even_8bit(x * factor_b)
//
// all in fp32, so x ~ q * scale_b.  The transposed output quantises the
// columns: its blocks are 128 x 1 pieces of a column (the products of the
// backward pass contract over rows); with `square` it holds the same values
// and the transposed scales.
//
// One read of x serves both outputs: it is bound by HBM traffic.  Measured, of the
// 6690 GB/s of a plain copy: rows only 6100 (8192 x 8192 bf16, 33.3 us), both
// directions 5100 (53 us), square blocks in both 6200 (28672 x 8192, 152 us); from
// fp32, 8192 x 8192, rows only 6120 (55.1 us), both directions 5700 (71.4), square blocks
// in both 6270 (64.3); one row of 8192 takes 2.2 us.  (Loads marked evict-first: 56 and
// 159 us.)  A CTA takes a 128 x 128 tile, so that it holds whole blocks in both
// directions: a thread has 8 columns of 8 consecutive rows in registers (16 lanes cover a row of the
// tile: 16-byte loads, 8-byte stores, whole 128-byte lines), row maxima are
// reduced in half a warp, column maxima across the warps through shared memory,
// and the transposed tile goes through shared memory so that its rows leave as
// whole 128-byte lines too.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "operators.h"
#include "ptx.cuh"

namespace bwgemm {
namespace {

constexpr int kWarps = 8;
constexpr int kQuantThreads = 32 * kWarps;

// Eight consecutive elements of a row as loaded, and as fp32 values.
template <typename T>
struct Row8 {
    static constexpr int kWords = int(2 * sizeof(T));
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const T* src, int valid)
    {
        if (valid >= 8) {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 v = ptx::ld_global_cg_v4(reinterpret_cast<const uint4*>(src) + i / 4);
                w[i] = v.x;
                w[i + 1] = v.y;
                w[i + 2] = v.z;
                w[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                w[i] = 0u;
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < valid)
                        w[j] = reinterpret_cast<const uint32_t*>(src)[j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < valid)
                        w[j / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(src)[j]) << (16 * (j & 1));
            }
        }
    }
    __device__ __forceinline__ float get(int j) const
    {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(w[j]);
        } else {
            const uint32_t h = (j & 1) ? (w[j / 2] >> 16) : (w[j / 2] & 0xFFFFu);
            if constexpr (std::is_same<T, __nv_bfloat16>::value)
                return __uint_as_float(h << 16);
            else
                return __half2float(__ushort_as_half(uint16_t(h)));
        }
    }
};

// Magnitudes are compared as bit patterns: the same order for finite values,
// and a NaN, larger than infinity, reaches the scale of its block.  16-bit
// types two at a time.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

template <typename T>
struct Mag {
    static constexpr int kWords = Row8<T>::kWords;
    static constexpr bool kPairs = sizeof(T) == 2;
    static __device__ __forceinline__ uint32_t of(uint32_t w) { return w & (kPairs ? 0x7FFF7FFFu : 0x7FFFFFFFu); }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b)
    {
        if constexpr (kPairs)
            return max_u16x2(a, b);
        else
            return max(a, b);
    }
    // the larger of a word's values, and a value's fp32 bits
    static __device__ __forceinline__ uint32_t fold(uint32_t w) { return kPairs ? max(w & 0xFFFFu, w >> 16) : w; }
    static __device__ __forceinline__ uint32_t f32_bits(uint32_t m)
    {
        if constexpr (std::is_same<T, float>::value)
            return m;
        else if constexpr (std::is_same<T, __nv_bfloat16>::value)
            return m << 16;
        else
            return __float_as_uint(__half2float(__ushort_as_half(uint16_t(m))));
    }
};

template <int F8>
__device__ __forceinline__ uint32_t cvt2(float lo, float hi)
{
    return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, F8 == 0 ? __NV_E4M3 : __NV_E5M2));
}

struct Scale {
    float scale, factor;
};

template <int F8>
__device__ __forceinline__ Scale make_scale(uint32_t amax_bits, bool pow2)
{
    constexpr float limit = F8 == 0 ? 448.f : 57344.f;
    const float amax = __uint_as_float(max(amax_bits, __float_as_uint(kSmallestAmax)));
    Scale r;
    r.scale = amax / limit;
    r.factor = limit / amax;
    if (pow2 && amax_bits <= 0x7F800000u) {
        // any mantissa bit carries into the exponent
        r.scale = __uint_as_float((__float_as_uint(r.scale) + 0x7FFFFFu) & 0x7F800000u);
        r.factor = 1.f / r.scale;
    }
    return r;
}

// CTAs per SM: as many as registers allow without keeping the values unpacked
// (the compiler would otherwise take 182 for bf16 in both directions, one CTA per
// SM: 103 us on 8192 x 8192)
template <typename T, bool BOTH>
constexpr int kQuantCtas = sizeof(T) == 4 ? 2 : BOTH ? 3 : 4;

template <typename T, int F8, bool SQUARE, bool BOTH>
__global__ void __launch_bounds__(kQuantThreads, kQuantCtas<T, BOTH>) quantize_kernel(const QuantizeParams p, const int kblocks)
{
    __shared__ uint32_t s_max[BOTH && !SQUARE ? kWarps * kBlock : kWarps];
    __shared__ float s_factor[BOTH && !SQUARE ? kBlock : 1];
    __shared__ __align__(16) uint8_t s_tile[BOTH ? kBlock * kBlock : 16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane & 15, half = lane >> 4;
    const int kb = int(blockIdx.x) % kblocks;
    const int64_t rb = int(blockIdx.x) / kblocks;
    const int64_t col0 = int64_t(kb) * kBlock, row0 = rb * kBlock;
    const int r0 = 16 * warp + 8 * half;  // this thread's 8 rows of the tile
    const int c0 = 8 * g;                 // and its 8 columns
    const int valid = int(min(int64_t(8), p.cols - col0 - c0));
    const bool pow2 = p.pow2 != 0;

    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    Row8<T> x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = row0 + r0 + i;
        const bool in = row < p.rows && valid > 0;
        x[i].load(static_cast<const T*>(p.x) + (in ? row * p.ldx + col0 + c0 : 0), in ? valid : 0);
    }

    using M = Mag<T>;
    float factor[8];   // of the thread's rows
    uint32_t rmax[8];  // bits of the rows' largest magnitudes
    uint32_t cmax[M::kWords];
#pragma unroll
    for (int j = 0; j < M::kWords; ++j)
        cmax[j] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < M::kWords; ++j) {
            const uint32_t v = M::of(x[i].w[j]);
            m = M::larger(m, v);
            if constexpr (BOTH && !SQUARE)
                cmax[j] = M::larger(cmax[j], v);
        }
        rmax[i] = M::fold(m);
    }
    if constexpr (SQUARE) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max(m, rmax[i]);
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (lane == 0)
            s_max[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            m = max(m, s_max[w]);
        const Scale sc = make_scale<F8>(M::f32_bits(m), pow2);
        if (threadIdx.x == 0) {
            p.s[int64_t(kb) * p.lds + rb] = sc.scale;
            if (BOTH)
                p.st[rb * p.ldst + kb] = sc.scale;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            factor[i] = sc.factor;
    } else {
        // Eight row maxima over the 16 lanes of the row: each exchange halves the
        // rows a lane still holds, so that lane g ends with row g / 2 alone, one
        // division per lane makes its scale, and eight shuffles hand them out.
#pragma unroll
        for (int step = 8, keep = 4; step >= 2; step >>= 1, keep >>= 1) {
            const bool upper = (g & step) != 0;
#pragma unroll
            for (int i = 0; i < keep; ++i) {
                const uint32_t mine = upper ? rmax[i + keep] : rmax[i];
                const uint32_t other = upper ? rmax[i] : rmax[i + keep];
                rmax[i] = max(mine, __shfl_xor_sync(0xFFFFFFFFu, other, step));
            }
        }
        const uint32_t m = max(rmax[0], __shfl_xor_sync(0xFFFFFFFFu, rmax[0], 1));
        const Scale sc = make_scale<F8>(M::f32_bits(m), pow2);
        const int64_t row = row0 + r0 + (g >> 1);
        if ((g & 1) == 0 && row < p.rows)
            p.s[int64_t(kb) * p.lds + row] = sc.scale;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            factor[i] = __shfl_sync(0xFFFFFFFFu, sc.factor, 16 * half + 2 * i);
    }

#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = row0 + r0 + i;
        uint32_t w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            w[k] = cvt2<F8>(x[i].get(4 * k) * factor[i], x[i].get(4 * k + 1) * factor[i]) |
                   (cvt2<F8>(x[i].get(4 * k + 2) * factor[i], x[i].get(4 * k + 3) * factor[i]) << 16);
        if (row < p.rows && valid > 0) {
            uint8_t* dst = p.q + row * p.ldq + col0 + c0;
            if (valid == 8) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
            } else {
                for (int j = 0; j < valid; ++j)
                    dst[j] = uint8_t(w[j >> 2] >> (8 * (j & 3)));
            }
        }
    }

    if constexpr (BOTH) {
        if constexpr (!SQUARE) {
            constexpr int per = 8 / M::kWords;  // columns per word
#pragma unroll
            for (int j = 0; j < M::kWords; ++j) {
                const uint32_t m = M::larger(cmax[j], __shfl_xor_sync(0xFFFFFFFFu, cmax[j], 16));
                if (half == 0)
                    s_max[warp * (kBlock / per) + M::kWords * g + j] = m;
            }
            __syncthreads();
            if (threadIdx.x < kBlock) {
                uint32_t m = 0;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    m = M::larger(m, s_max[w * (kBlock / per) + threadIdx.x / per]);
                if constexpr (M::kPairs)
                    m = (threadIdx.x & 1) ? m >> 16 : m & 0xFFFFu;
                const Scale sc = make_scale<F8>(M::f32_bits(m), pow2);
                s_factor[threadIdx.x] = sc.factor;
                if (col0 + threadIdx.x < p.cols)
                    p.st[rb * p.ldst + col0 + threadIdx.x] = sc.scale;
            }
            __syncthreads();
        }
        // the thread's 8 rows of a column are 8 consecutive bytes of the
        // transposed tile; its 16-byte pieces are exchanged within a row by
        // (column / 8) mod 8, which spreads the 16 lanes over the banks
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float f[8];
            if constexpr (SQUARE) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    f[i] = factor[0];
            } else {
                const float fc = s_factor[c0 + j];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    f[i] = fc;
            }
            uint32_t w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                w[k] = cvt2<F8>(x[4 * k].get(j) * f[4 * k], x[4 * k + 1].get(j) * f[4 * k + 1]) |
                       (cvt2<F8>(x[4 * k + 2].get(j) * f[4 * k + 2], x[4 * k + 3].get(j) * f[4 * k + 3]) << 16);
            const int piece = (r0 >> 4) ^ (g & 7);
            *reinterpret_cast<uint2*>(s_tile + (c0 + j) * kBlock + 16 * piece + 8 * half) = make_uint2(w[0], w[1]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = 32 * i + int(threadIdx.x >> 3), piece = threadIdx.x & 7;
            const uint4 v = *reinterpret_cast<const uint4*>(s_tile + c * kBlock + 16 * (piece ^ ((c >> 3) & 7)));
            const int64_t row = row0 + 16 * piece;
            if (col0 + c < p.cols && row < p.rows) {
                uint8_t* dst = p.qt + (col0 + c) * p.ldqt + row;
                if (row + 16 <= p.rows) {
                    *reinterpret_cast<uint4*>(dst) = v;
                } else {
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    for (int b = 0; b < int(p.rows - row); ++b)
                        dst[b] = uint8_t(w[b >> 2] >> (8 * (b & 3)));
                }
            }
        }
    }
}

template <typename T, int F8, bool SQUARE, bool BOTH>
cudaError_t launch(const QuantizeParams& p, cudaStream_t stream, bool pdl)
{
    const int64_t kblocks = (p.cols + kBlock - 1) / kBlock, rblocks = (p.rows + kBlock - 1) / kBlock;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(kblocks * rblocks), 1, 1);
    cfg.blockDim = dim3(kQuantThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, quantize_kernel<T, F8, SQUARE, BOTH>, p, int(kblocks));
}

template <typename T, int F8>
cudaError_t launch_form(bool square, const QuantizeParams& p, cudaStream_t stream, bool pdl)
{
    if (square)
        return p.qt ? launch<T, F8, true, true>(p, stream, pdl) : launch<T, F8, true, false>(p, stream, pdl);
    return p.qt ? launch<T, F8, false, true>(p, stream, pdl) : launch<T, F8, false, false>(p, stream, pdl);
}

template <typename T>
cudaError_t launch_type(int fp8, bool square, const QuantizeParams& p, cudaStream_t stream, bool pdl)
{
    return fp8 == BWGEMM_E4M3 ? launch_form<T, 0>(square, p, stream, pdl) : launch_form<T, 1>(square, p, stream, pdl);
}

}  // namespace

cudaError_t launch_quantize(int dtype, int fp8, bool square, const QuantizeParams& p, cudaStream_t stream, bool pdl)
{
    switch (dtype) {
    case BWGEMM_BF16: return launch_type<__nv_bfloat16>(fp8, square, p, stream, pdl);
    case BWGEMM_FP16: return launch_type<__half>(fp8, square, p, stream, pdl);
    case BWGEMM_FP32: return launch_type<float>(fp8, square, p, stream, pdl);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace bwgemm
