// gated_sm103.cu -- the gated feed-forward layer's large products (pair_kernel.cuh), and
// the gradients of its two projections.
#include <cfloat>

#include "pair_kernel.cuh"

namespace bwgemm {
namespace {

template <int CG, int FORM>
cudaError_t launch_form(const PairMaps& maps, const PairParams& p, int grid, cudaStream_t stream, bool pdl)
{
    using Cfg = OrthoConfig<CG>;
    auto kernel = pair_kernel<CG, FORM>;
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
    err = cudaLaunchKernelEx(&cfg, kernel, maps, p);
    for (int which = 0; which < 2 && err == cudaSuccess; ++which) {
        const PairProduct& d = p.prod[which];
        if (d.units == 0 || d.splits == 1)
            continue;
        cudaLaunchConfig_t join = {};
        join.gridDim = dim3(unsigned(CG * 8 * Cfg::kCols / 4 / kJoinWarps * d.join_share), unsigned(d.units / d.splits), 1);
        join.blockDim = dim3(32 * kJoinWarps, 1, 1);
        join.stream = stream;
        join.attrs = pdl ? attr + n - 1 : nullptr;  // the dependency's
        join.numAttrs = pdl ? 1 : 0;
        err = cudaLaunchKernelEx(&join, pair_join_kernel<CG>, p, which);
    }
    return err;
}

// dU = dH act(G), dG = dH U act'(G): three reads and two writes of rows x cols, eight
// values a thread, rounded to 16 bits as the operands that the products need.  Bound by HBM
// (2048 x 4096 18.5 us cold, of which 12 are its bytes; 20 with one piece a thread).
constexpr int kGradThreads = 256, kGradPieces = 2;  // a thread has two pieces on their way

__device__ __forceinline__ float2 unpack16(uint32_t w, int dtype)
{
    return dtype == BWGEMM_BF16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w))
                                : __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// dH U act'(G).  A slope can be tiny, so where dH U leaves fp32's range the larger of the two
// meets the slope first.
__device__ __forceinline__ float gate_grad(float dh, float u, float slope)
{
    const float p = dh * u;
    if (__builtin_expect(fabsf(p) <= FLT_MAX, 1))
        return p * slope;
    return fabsf(dh) > fabsf(u) ? dh * slope * u : u * slope * dh;
}

__global__ void __launch_bounds__(kGradThreads) gate_grad_kernel(const GateGradParams p)
{
    ptx::grid_dependency_wait();
    ptx::launch_dependents();
    const int64_t per_row = (p.cols + 7) / 8, pieces = per_row * p.rows;
    const int64_t step = int64_t(gridDim.x) * kGradThreads;
#pragma unroll 1
    for (int64_t i = int64_t(blockIdx.x) * kGradThreads + threadIdx.x; i < pieces; i += kGradPieces * step) {
        int64_t row[kGradPieces], col[kGradPieces];
        uint4 dh[kGradPieces], g[kGradPieces], u[kGradPieces];
#pragma unroll
        for (int n = 0; n < kGradPieces; ++n) {
            const int64_t at = i + n * step;
            row[n] = at / per_row;
            col[n] = (at - row[n] * per_row) * 8;
            if (at >= pieces)
                continue;
            if (col[n] + 8 <= p.cols) {
                dh[n] = ptx::ld_global_cg_v4(p.dh + row[n] * p.lddh + col[n]);
                g[n] = ptx::ld_global_cg_v4(p.g + row[n] * p.ldg + col[n]);
                u[n] = ptx::ld_global_cg_v4(p.u + row[n] * p.ldu + col[n]);
            } else {  // nothing is read past a row's end
                dh[n] = g[n] = u[n] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int k = 0; k < 7; ++k)
                    if (col[n] + k < p.cols) {
                        reinterpret_cast<uint16_t*>(&dh[n])[k] = p.dh[row[n] * p.lddh + col[n] + k];
                        reinterpret_cast<uint16_t*>(&g[n])[k] = p.g[row[n] * p.ldg + col[n] + k];
                        reinterpret_cast<uint16_t*>(&u[n])[k] = p.u[row[n] * p.ldu + col[n] + k];
                    }
            }
        }
#pragma unroll
        for (int n = 0; n < kGradPieces; ++n) {
            if (i + n * step >= pieces)
                break;
            uint4 dg, du;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 fh = unpack16((&dh[n].x)[k], p.dtype), fg = unpack16((&g[n].x)[k], p.dtype),
                             fu = unpack16((&u[n].x)[k], p.dtype);
                float2 value, slope;
                activate_slope(fg.x, p.activation, value.x, slope.x);
                activate_slope(fg.y, p.activation, value.y, slope.y);
                (&dg.x)[k] = pack2(__float_as_uint(gate_grad(fh.x, fu.x, slope.x)),
                                   __float_as_uint(gate_grad(fh.y, fu.y, slope.y)), p.dtype);
                (&du.x)[k] = pack2(__float_as_uint(fh.x * value.x), __float_as_uint(fh.y * value.y), p.dtype);
            }
            // the workspace's rows are whole pieces: what lies past the end is not read as a value
            *reinterpret_cast<uint4*>(p.dg + row[n] * p.ldd + col[n]) = dg;
            *reinterpret_cast<uint4*>(p.du + row[n] * p.ldd + col[n]) = du;
        }
    }
}

}  // namespace

cudaError_t launch_pair(int form, int cg, const PairMaps& maps, const PairParams& p, int grid, cudaStream_t stream, bool pdl)
{
    switch (form * 2 + (cg - 1)) {
    case kPairGated * 2 + 1: return launch_form<2, kPairGated>(maps, p, grid, stream, pdl);
    case kPairBackward * 2: return launch_form<1, kPairBackward>(maps, p, grid, stream, pdl);
    case kPairBackward * 2 + 1: return launch_form<2, kPairBackward>(maps, p, grid, stream, pdl);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_gate_grad(const GateGradParams& p, cudaStream_t stream, bool pdl)
{
    const int64_t pieces = (p.cols + 7) / 8 * p.rows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(std::min<int64_t>((pieces + kGradPieces * kGradThreads - 1) / (kGradPieces * kGradThreads), 1 << 20)), 1, 1);
    cfg.blockDim = dim3(kGradThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, gate_grad_kernel, p);
}

}  // namespace bwgemm
