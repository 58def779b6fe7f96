// lanes_sm103.cu -- instantiates and launches the products with the weights in the
// lanes (lanes_kernel.cuh).
#include "lanes_kernel.cuh"

namespace bwgemm {
namespace {

template <int MODE, int CG, int BN, bool WIDENS = false, bool TURNED = false>
cudaError_t launch_one(const LanesMaps& maps, const LanesParams& p, int grid, cudaStream_t stream, bool pdl)
{
    using Cfg = LanesConfig<MODE, CG, BN, WIDENS>;
    auto kernel = lanes_kernel<MODE, CG, BN, WIDENS, TURNED>;
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
    return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

}  // namespace

cudaError_t launch_lanes(int idx, const LanesMaps& maps, const LanesParams& p, int grid, cudaStream_t stream, bool pdl)
{
    static_assert(kNumLanesVariants == 10, "one case per variant below, in the order of kLanesVariants");
    switch (idx) {
    case 0: return launch_one<kLanesGated, 1, 16>(maps, p, grid, stream, pdl);
    case 1: return launch_one<kLanesGated, 1, 32>(maps, p, grid, stream, pdl);
    case 2: return launch_one<kLanesGated, 1, 64>(maps, p, grid, stream, pdl);
    case 3: return launch_one<kLanesGated, 1, 128>(maps, p, grid, stream, pdl);
    case 4: return launch_one<kLanesInt8, 1, 16, true>(maps, p, grid, stream, pdl);
    case 5: return launch_one<kLanesInt8, 1, 32, true>(maps, p, grid, stream, pdl);
    case 6: return launch_one<kLanesInt8, 1, 32>(maps, p, grid, stream, pdl);
    case 7: return launch_one<kLanesInt8, 1, 64>(maps, p, grid, stream, pdl);
    case 8: return launch_one<kLanesInt8, 1, 128>(maps, p, grid, stream, pdl);
    case 9:
        return p.turned ? launch_one<kLanesInt8, 2, 256, false, true>(maps, p, grid, stream, pdl)
                        : launch_one<kLanesInt8, 2, 256>(maps, p, grid, stream, pdl);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace bwgemm
