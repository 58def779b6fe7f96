// int8_sm103.cu -- rows to 8-bit integers with a scale each, and 8-bit integers to the
// fp16 operand of their product.
//
// quantize_int8: a = max(max |x|, 2^-100) of the row, scale = a / 127, q = 127 x / a rounded
// to the nearest integer, ties to the even one, of the exact quotient.  x times fl(127 / a)
// is within 127 * 2^-24 < 2^-17 of it, so it is right but for values that close to the middle
// of two integers:
//
// * bf16: x = X 2^i and a = A 2^k with integers X, A < 2^8, so the quotient's distance from a
//   middle is a multiple of 2^d / A, d = i - k: 0, or more than 2^-16, as quotients of 1/2 and
//   more have d >= -8.  One fma that adds 384 rounds the quotient to a multiple of 2^-15: to the
//   middle itself from within 2^-17, never to it from beyond 2^-16; ties then go to the even
//   integer by themselves.
// * fp16: 127 x and r a are exact in fp32 and so is the rest e = 127 x - r a (a multiple of
//   x's last place, at most a / 2 or so: 20 bits); 2 |e| against a decides.
// * fp32: 254 |x| against (2 L + 1) a, both as the sum of two fp32 values.
//
// Bound by HBM: a row is read once, held in registers between the maximum and the
// rounding (up to 8 pieces of 16 bytes a thread; what a longer row has beyond that is
// read again, from L2), by a warp, 128, 256 or 512 threads according to its length.
// 8192 x 8192 bf16 30.7 us (96 % of the copy rate; 39.8 with the test of every value's rest that
// fp16 takes, before the fp32 pairs), fp16 33.2, fp32 52.7 (49.3 at the copy rate); 28672 x 1024
// 13.7 (22.6 with eight pieces a lane for rows of 128).
#include <type_traits>

#include "feed_forward.h"
#include "lanes_kernel.cuh"

namespace bwgemm {
namespace {

constexpr float kMagic = 12582912.f;  // 1.5 2^23: a sum with it holds the rounded integer in its low bits
constexpr float kSnap = 384.f;        // a sum with it is a multiple of 2^-15

template <typename T>
struct Piece {
    static constexpr int kN = 16 / sizeof(T);  // elements of 16 bytes
    uint4 w;

    __device__ __forceinline__ void load(const T* row, int64_t c, int64_t cols)
    {
        if (c + kN <= cols) {
            w = ptx::ld_global_cg_v4(row + c);
        } else {  // nothing is read past the row's end
            w = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < kN - 1; ++i)
                if (c + i < cols)
                    reinterpret_cast<T*>(&w)[i] = row[c + i];
        }
    }
    // the bits of the largest magnitude as fp32 (integers compare like magnitudes, NaN
    // above infinity)
    __device__ __forceinline__ uint32_t top() const
    {
        if constexpr (std::is_same<T, float>::value) {
            const uint32_t m = 0x7FFFFFFFu;
            return max(max(w.x & m, w.y & m), max(w.z & m, w.w & m));
        } else {
            // both halves of a word at once
            using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
            const T2* v = reinterpret_cast<const T2*>(&w);
            const T2 a = __hmax2_nan(__hmax2_nan(__habs2(v[0]), __habs2(v[1])), __hmax2_nan(__habs2(v[2]), __habs2(v[3])));
            return max(__float_as_uint(fabsf(__low2float(a))), __float_as_uint(fabsf(__high2float(a))));
        }
    }
    __device__ __forceinline__ float operator[](int i) const
    {
        const uint32_t h = (&w.x)[std::is_same<T, float>::value ? i : i / 2];
        if constexpr (std::is_same<T, float>::value)
            return __uint_as_float(h);
        else if constexpr (std::is_same<T, __nv_bfloat16>::value)
            return __uint_as_float(i & 1 ? h & 0xFFFF0000u : h << 16);
        else
            return __half2float(__ushort_as_half(uint16_t(i & 1 ? h >> 16 : h)));
    }
};

// 127 x / a rounded exactly, where fp32 leaves open on which side of the middle of two
// integers `near` lies (|x|, a below 2^118).
static __device__ __noinline__ int round_exactly(float x, float a, float near)
{
    const float y = fabsf(x), low = floorf(fabsf(near)), odd = 2.f * low + 1.f;
    const float p = 254.f * y, p2 = fmaf(254.f, y, -p);  // p + p2 = 254 |x|
    const float q = odd * a, q2 = fmaf(odd, a, -q);
    const float d = (p - q) + (p2 - q2);  // p and q are close: each difference is exact
    const int l = int(low);
    const int r = d > 0.f || (d == 0.f && (l & 1)) ? l + 1 : l;
    return x < 0.f ? -r : r;
}

__device__ __forceinline__ uint64_t twice(float v) { return ptx::pack_f32x2(__float_as_uint(v), __float_as_uint(v)); }

// One row by TR threads of the block, kHeld pieces each in registers; ROWS rows per block.
template <typename T, int TR, int ROWS, int kHeld>
__global__ void __launch_bounds__(TR* ROWS) quantize_rows_kernel(const RowsInt8Params p)
{
    using P = Piece<T>;
    __shared__ uint32_t tops[TR > 32 ? TR / 32 : 1];
    const int t = TR == 32 ? int(threadIdx.x & 31) : int(threadIdx.x);
    const int64_t row = int64_t(blockIdx.x) * ROWS + (TR == 32 ? threadIdx.x >> 5 : 0);
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    if (TR == 32 && row >= p.rows)
        return;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    P held[kHeld];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int64_t c = int64_t(i * TR + t) * P::kN;
        held[i].w = make_uint4(0u, 0u, 0u, 0u);
        if (c < p.cols)
            held[i].load(x, c, p.cols);
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        top = max(top, held[i].top());
#pragma unroll 4
    for (int64_t c = int64_t(kHeld * TR + t) * P::kN; c < p.cols; c += TR * P::kN) {
        P v;
        v.load(x, c, p.cols);
        top = max(top, v.top());
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (TR > 32) {
        if ((t & 31) == 0)
            tops[t >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TR / 32; ++i)
            top = max(top, tops[i]);
    }
    const bool finite = top < 0x7F800000u;
    const float a = fmaxf(__uint_as_float(top), kSmallestAmax);
    // x and a times a power of two, exact, that keeps 254 x in range
    const float down = a > 1.f ? 0.0009765625f : 1.f;
    const float as = a * down, half = 0.5f * as;
    const float inv = finite ? 1.f / as : 0.f, times = 127.f * down, up = finite ? 127.f / a : 0.f;
    const bool tie_exact = (__float_as_uint(a) & 0x7FFFFFu) == 0u;
    if (t == 0)
        p.scales[row] = finite ? a / 127.f : __uint_as_float(0x7FC00000u);
    int8_t* q = p.q + row * p.ldq;
    auto put = [&](const P& v, int64_t c) {
        uint32_t bits[P::kN];
        float worst = 0.f;
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
            for (int i = 0; i < P::kN; i += 2) {
                const uint64_t x2 = ptx::pack_f32x2(__float_as_uint(v[i]), __float_as_uint(v[i + 1]));
                float lo, hi;
                ptx::unpack_f32x2(ptx::fma_f32x2(ptx::fma_f32x2(x2, twice(up), twice(kSnap)), twice(1.f), twice(kMagic - kSnap)),
                                  lo, hi);
                bits[i] = __float_as_uint(lo);
                bits[i + 1] = __float_as_uint(hi);
            }
        } else if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
            for (int i = 0; i < P::kN; i += 2) {
                const uint64_t x2 = ptx::pack_f32x2(__float_as_uint(v[i]), __float_as_uint(v[i + 1]));
                const uint64_t y = ptx::mul_f32x2(x2, twice(times)), f = ptx::fma_f32x2(y, twice(inv), twice(kMagic));
                const uint64_t e = ptx::fma_f32x2(ptx::fma_f32x2(f, twice(-1.f), twice(kMagic)), twice(as), y);
                float lo, hi;
                ptx::unpack_f32x2(e, lo, hi);
                worst = fmaxf(worst, fmaxf(fabsf(lo), fabsf(hi)));
                ptx::unpack_f32x2(f, lo, hi);
                bits[i] = __float_as_uint(lo);
                bits[i + 1] = __float_as_uint(hi);
            }
            if (worst >= half && !tie_exact) {
#pragma unroll
                for (int i = 0; i < P::kN; ++i) {
                    const float e = fmaf(kMagic - __uint_as_float(bits[i]), as, v[i] * times);
                    if (fabsf(e) > half || (fabsf(e) == half && (bits[i] & 1u)))
                        bits[i] += e > 0.f ? 1u : 0xFFFFFFFFu;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < P::kN; i += 2) {
                const uint64_t x2 = ptx::pack_f32x2(__float_as_uint(v[i]), __float_as_uint(v[i + 1]));
                const uint64_t f = ptx::fma_f32x2(x2, twice(up), twice(kMagic));
                const uint64_t d = ptx::fma_f32x2(x2, twice(up), ptx::fma_f32x2(f, twice(-1.f), twice(kMagic)));
                float lo, hi;
                ptx::unpack_f32x2(d, lo, hi);
                worst = fmaxf(worst, fmaxf(fabsf(lo), fabsf(hi)));
                ptx::unpack_f32x2(f, lo, hi);
                bits[i] = __float_as_uint(lo);
                bits[i + 1] = __float_as_uint(hi);
            }
            if (worst > 0.4999f) {
#pragma unroll
                for (int i = 0; i < P::kN; ++i) {
                    const float near = v[i] * up;
                    if (fabsf(near - rintf(near)) > 0.4999f)
                        bits[i] = uint32_t(round_exactly(v[i] * down, as, near));
                }
            }
        }
        uint32_t w[P::kN / 4];
#pragma unroll
        for (int i = 0; i < P::kN / 4; ++i)
            w[i] = finite ? __byte_perm(__byte_perm(bits[4 * i], bits[4 * i + 1], 0x0040),
                                        __byte_perm(bits[4 * i + 2], bits[4 * i + 3], 0x0040), 0x5410)
                          : 0u;
        if (c + P::kN <= p.cols) {
            if constexpr (P::kN == 8)
                *reinterpret_cast<uint2*>(q + c) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint32_t*>(q + c) = w[0];
        } else {
#pragma unroll
            for (int i = 0; i < P::kN - 1; ++i)
                if (c + i < p.cols)
                    q[c + i] = int8_t(w[i / 4] >> (8 * (i % 4)));
        }
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int64_t c = int64_t(i * TR + t) * P::kN;
        if (c < p.cols)
            put(held[i], c);
    }
#pragma unroll 1
    for (int64_t c = int64_t(kHeld * TR + t) * P::kN; c < p.cols; c += TR * P::kN) {
        P v;
        v.load(x, c, p.cols);
        put(v, c);
    }
}

template <typename Kernel, typename Params>
cudaError_t launch_plain(Kernel kernel, unsigned grid, unsigned threads, const Params& p, cudaStream_t stream, bool pdl)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T>
cudaError_t launch_rows(const RowsInt8Params& p, cudaStream_t stream, bool pdl)
{
    const int64_t pieces = (p.cols + Piece<T>::kN - 1) / Piece<T>::kN;
    if (pieces <= 32 * 4)
        return launch_plain(quantize_rows_kernel<T, 32, 4, 4>, unsigned((p.rows + 3) / 4), 128, p, stream, pdl);
    if (pieces <= 128 * 8)
        return launch_plain(quantize_rows_kernel<T, 128, 1, 8>, unsigned(p.rows), 128, p, stream, pdl);
    if (pieces <= 256 * 8)
        return launch_plain(quantize_rows_kernel<T, 256, 1, 8>, unsigned(p.rows), 256, p, stream, pdl);
    return launch_plain(quantize_rows_kernel<T, 512, 1, 8>, unsigned(p.rows), 512, p, stream, pdl);
}

// Sixteen values a thread; the pad to whole stages of 128 is zeros.
constexpr int kWidenThreads = 256;

__global__ void __launch_bounds__(kWidenThreads) widen_kernel(const WidenParams p)
{
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int64_t per_row = p.ldy / 16, pieces = per_row * p.rows;
#pragma unroll 1
    for (int64_t i = int64_t(blockIdx.x) * kWidenThreads + threadIdx.x; i < pieces; i += int64_t(gridDim.x) * kWidenThreads) {
        const int64_t row = i / per_row;
        const int c = int(i - row * per_row) * 16;
        const int8_t* x = p.x + row * p.ldx + c;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (c + 16 <= p.cols) {
            v = ptx::ld_global_cg_v4(x);
        } else {
#pragma unroll
            for (int k = 0; k < 15; ++k)
                if (c + k < p.cols)
                    reinterpret_cast<int8_t*>(&v)[k] = x[k];
        }
        uint4 a, b;
        widen4(v.x, a.x, a.y);
        widen4(v.y, a.z, a.w);
        widen4(v.z, b.x, b.y);
        widen4(v.w, b.z, b.w);
        uint4* y = reinterpret_cast<uint4*>(p.y + row * p.ldy + c);
        y[0] = a;
        y[1] = b;
    }
}

}  // namespace

cudaError_t launch_quantize_int8(int dtype, const RowsInt8Params& p, cudaStream_t stream, bool pdl)
{
    switch (dtype) {
    case BWGEMM_BF16: return launch_rows<__nv_bfloat16>(p, stream, pdl);
    case BWGEMM_FP16: return launch_rows<__half>(p, stream, pdl);
    case BWGEMM_FP32: return launch_rows<float>(p, stream, pdl);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_widen(const WidenParams& p, cudaStream_t stream, bool pdl)
{
    const int64_t pieces = p.ldy / 16 * p.rows;
    const unsigned grid = unsigned(std::min<int64_t>((pieces + kWidenThreads - 1) / kWidenThreads, 1 << 20));
    return launch_plain(widen_kernel, grid, kWidenThreads, p, stream, pdl);
}

}  // namespace bwgemm
