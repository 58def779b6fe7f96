// ortho_sm103.cu -- the Newton-Schulz products' instances and launches
// (ortho_kernel.cuh), and the pass that brings the input into the workspace.
#include <type_traits>

#include "ortho_kernel.cuh"

namespace bwgemm {
namespace {

template <int CG, bool A_MN, bool B_MN>
cudaError_t launch_one(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& a2, const CUtensorMap& b2,
                       const CUtensorMap& out, const CUtensorMap& out2, const OrthoParams& p, int grid,
                       cudaStream_t stream, bool pdl)
{
    using Cfg = OrthoConfig<CG>;
    auto kernel = ortho_kernel<CG, A_MN, B_MN>;
    if (grid % CG != 0)
        return cudaErrorInvalidValue;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_smem(kernel, Cfg::kSmemBytes, allowed);
    if (err != cudaSuccess)
        return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid), 1, 1);
    cfg.blockDim = dim3(Cfg::kThreads, 1, 1);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (CG == 2) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = 2;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    err = cudaLaunchKernelEx(&cfg, kernel, a, b, a2, b2, out, out2, p);
    if (err != cudaSuccess || p.splits == 1)
        return err;
    cudaLaunchConfig_t join = {};
    join.gridDim = dim3(unsigned(CG * 8 * Cfg::kCols / 4 / kJoinWarps * p.join_share), unsigned(p.tiles * p.batch), 1);
    join.blockDim = dim3(32 * kJoinWarps, 1, 1);
    join.stream = stream;
    join.attrs = pdl ? attr + n - 1 : nullptr;  // the dependency's
    join.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&join, ortho_join_kernel<CG>, p);
}

// ------------------------------------------------------------ the input pass
// Both kernels are bound by HBM traffic: one read of G for the norm, one read
// of G and one write of X (from L2 where G fits it).  A thread takes 8 elements of
// X's padded rows at a time, neighbours next to each other whatever the shape, four
// such pieces in flight.  (A warp per row left most SMs without work on long or
// narrow matrices: both kernels 95 us on 300 x 28000 and 87 on 24000 x 17, of calls
// that now take 169 and 89.)
constexpr int kInThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f32(T v)
{
    if constexpr (std::is_same<T, float>::value)
        return v;
    else if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return __bfloat162float(v);
    else
        return __half2float(v);
}

__device__ __forceinline__ float block_sum(float v, float* shared)
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, d);
    if ((threadIdx.x & 31) == 0)
        shared[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kInThreads / 32; ++w)
        s += shared[w];
    __syncthreads();
    return s;
}

// Eight elements of a row of G from column c on, zeros past its end.
template <typename T>
struct Eight {
    uint4 w[sizeof(T) / 2];

    __device__ __forceinline__ void load(const OrthoInput& p, const T* g, int row, int c)
    {
        const T* at = g + int64_t(row) * p.ldg + c;
        if (p.vectors && c + 8 <= p.cols) {
#pragma unroll
            for (int i = 0; i < int(sizeof(T) / 2); ++i)
                w[i] = ptx::ld_global_cg_v4(reinterpret_cast<const uint4*>(at) + i);
        } else {
            T* t = reinterpret_cast<T*>(w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                t[i] = c + i < p.cols ? at[i] : T(0.f);
        }
    }

    __device__ __forceinline__ float operator[](int i) const { return to_f32(reinterpret_cast<const T*>(w)[i]); }
};

// This thread's pieces of a matrix, in the order of memory, all threads of the
// grid's row of blocks apart: calls f(piece, row, column) for each.
template <typename T, typename F>
__device__ __forceinline__ void each_piece(const OrthoInput& p, const T* g, F&& f)
{
    constexpr int kFlight = 4;
    const int per_row = int(p.ld / 8);
    const int threads = int(gridDim.x) * kInThreads, at = int(blockIdx.x) * kInThreads + int(threadIdx.x);
    const int rows = threads / per_row, pieces = threads % per_row;
    int row = at / per_row, piece = at % per_row;
    while (row < p.rows) {
        Eight<T> x[kFlight];
        int r[kFlight], c[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            r[i] = row;
            c[i] = 8 * piece;
            if (row < p.rows)
                x[i].load(p, g, row, c[i]);
            row += rows;
            piece += pieces;
            if (piece >= per_row) {
                piece -= per_row;
                ++row;
            }
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i)
            if (r[i] < p.rows)
                f(x[i], r[i], c[i]);
    }
}

template <typename T>
__global__ void __launch_bounds__(kInThreads) ortho_sums_kernel(const OrthoInput p)
{
    __shared__ float shared[kInThreads / 32];
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    float sum = 0.f;
    each_piece(p, static_cast<const T*>(p.g) + int64_t(blockIdx.y) * p.stride_g, [&](const Eight<T>& x, int, int) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum = fmaf(x[i], x[i], sum);
    });
    sum = block_sum(sum, shared);
    if (threadIdx.x == 0)
        p.sums[int64_t(blockIdx.y) * p.parts + blockIdx.x] = sum;
}

// X is stored as G times a power of two near 2^log2_scale / |G|: exact for bf16 and
// fp16 input (but for elements below fp16's range, 2^-24 and less of the largest),
// with elements around 2^log2_scale / sqrt(rows cols), clear of fp16's subnormals.
// The rest of the factor is applied to fp32 sums.
//
// Where |G| is far below eps, X is small and stays so for some steps: every step is then
// X <- a X, but for terms of X^3.  Stored times 2^log2_scale alone it would sink into
// fp16's subnormals (|G| = 1e-12, eps = 1e-7: 4 to 7 % off), so it is stored times a
// further 2^t: t0 = floor(log2((|G| + eps) / |G|)), and each step takes ceil(log2 |a|) off t
// until none is left, so that the stored X never grows by it.  t = 0 for |G| > eps.
template <typename T>
__global__ void __launch_bounds__(kInThreads) ortho_convert_kernel(const OrthoInput p)
{
    __shared__ float shared[kInThreads / 32];
    const int64_t mat = blockIdx.y;
    const T* g = static_cast<const T*>(p.g) + mat * p.stride_g;
    uint16_t* hi = p.hi + mat * p.stride;
    uint16_t* lo = p.lo ? p.lo + mat * p.stride : nullptr;
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    float sum = 0.f;
    for (int i = threadIdx.x; i < p.parts; i += kInThreads)
        sum += ptx::ld_global_cg_f32(p.sums + mat * p.parts + i);
    const float size = sqrtf(block_sum(sum, shared)), norm = size + p.eps;
    int e = 0, t = 0;
    if (size > 0.f && size <= 3.0e38f) {
        e = min(max(p.log2_scale - ilogbf(size), -120), 120);
        t = min(ilogbf(norm / size), 100);
    }
    const float up = ldexpf(1.f, e);
    if (blockIdx.x == 0 && int(threadIdx.x) < p.steps) {  // a thread per step
        const int step = threadIdx.x;
        auto less = [&](int i) { return t > 0 ? max(t - p.growth[i], 0) : 0; };
        for (int i = 0; i < step; ++i)
            t = less(i);
        const float f = norm == 0.f ? 0.f : ldexpf(1.f / norm, -e);  // zeros (eps = 0): not 0 / 0
        // the step's stored X to the true one, less 2^log2_scale after the first step
        const float down = step == 0 ? f : ldexpf(1.f, -t);
        float* const to = p.factors + int64_t(2 * step) * p.batch + mat;
        to[0] = down * down;
        to[p.batch] = step + 1 < p.steps ? ldexpf(down, less(step)) : down;
    }
    each_piece(p, g, [&](const Eight<T>& x, int row, int c) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = make_float2(x[2 * i] * up, x[2 * i + 1] * up);
            const __half2 a = __floats2half2_rn(v.x, v.y);
            const float2 b = __half22float2(a);
            const __half2 d = __floats2half2_rn(v.x - b.x, v.y - b.y);
            h[i] = *reinterpret_cast<const uint32_t*>(&a);
            l[i] = *reinterpret_cast<const uint32_t*>(&d);
        }
        *reinterpret_cast<uint4*>(hi + int64_t(row) * p.ld + c) = make_uint4(h[0], h[1], h[2], h[3]);
        if (lo)
            *reinterpret_cast<uint4*>(lo + int64_t(row) * p.ld + c) = make_uint4(l[0], l[1], l[2], l[3]);
    });
}

template <typename T>
cudaError_t launch_input(const OrthoInput& p, cudaStream_t stream, bool pdl)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(p.parts), unsigned(p.batch), 1);
    cfg.blockDim = dim3(kInThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, ortho_sums_kernel<T>, p);
    return err != cudaSuccess ? err : cudaLaunchKernelEx(&cfg, ortho_convert_kernel<T>, p);
}

}  // namespace

cudaError_t launch_ortho_input(const OrthoInput& p, cudaStream_t stream, bool pdl)
{
    switch (p.dtype) {
    case BWGEMM_BF16: return launch_input<__nv_bfloat16>(p, stream, pdl);
    case BWGEMM_FP16: return launch_input<__half>(p, stream, pdl);
    case BWGEMM_FP32: return launch_input<float>(p, stream, pdl);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_ortho(int form, int cg, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& a2,
                         const CUtensorMap& b2, const CUtensorMap& out, const CUtensorMap& out2, const OrthoParams& p,
                         int grid, cudaStream_t stream, bool pdl)
{
    switch (form * 2 + (cg - 1)) {
    case kOrthoNT * 2: return launch_one<1, false, false>(a, b, a2, b2, out, out2, p, grid, stream, pdl);
    case kOrthoNT * 2 + 1: return launch_one<2, false, false>(a, b, a2, b2, out, out2, p, grid, stream, pdl);
    case kOrthoNN * 2: return launch_one<1, false, true>(a, b, a2, b2, out, out2, p, grid, stream, pdl);
    case kOrthoNN * 2 + 1: return launch_one<2, false, true>(a, b, a2, b2, out, out2, p, grid, stream, pdl);
    case kOrthoTN * 2: return launch_one<1, true, true>(a, b, a2, b2, out, out2, p, grid, stream, pdl);
    case kOrthoTN * 2 + 1: return launch_one<2, true, true>(a, b, a2, b2, out, out2, p, grid, stream, pdl);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace bwgemm
