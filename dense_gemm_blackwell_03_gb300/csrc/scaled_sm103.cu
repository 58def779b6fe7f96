// scaled_sm103.cu -- instantiates and launches the block-scaled 8-bit product
// (scaled_kernel.cuh).
#include "scaled_kernel.cuh"

namespace bwgemm {
namespace {

template <int BN, bool SWAP, bool COLVEC>
cudaError_t launch_sc(const CUtensorMap& l, const CUtensorMap& c, const CUtensorMap& l3, const CUtensorMap& c3,
                      const CUtensorMap& out, const ScaledParams& p, int grid, cudaStream_t stream, bool pdl)
{
    using Cfg = ScaledConfig<BN, SWAP, COLVEC>;
    auto kernel = scaled_kernel<BN, SWAP, COLVEC>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_smem(kernel, Cfg::kSmemBytes, allowed);
    if (err != cudaSuccess)
        return err;
    if (Cfg::kSplitRegs) {
        // the warpgroups' shares must fit what the block is launched with: a
        // share that does not would wait for registers for ever
        static const int regs = [&] {
            cudaFuncAttributes a;
            return cudaFuncGetAttributes(&a, kernel) == cudaSuccess ? a.numRegs : 0;
        }();
        if (regs * Cfg::kThreads < 128 * Cfg::kRegsFirst + 32 * Cfg::kEpiWarps * Cfg::kRegsEpi ||
            regs < Cfg::kRegsFirst || regs > Cfg::kRegsEpi)
            return cudaErrorLaunchOutOfResources;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid), 1, 1);
    cfg.blockDim = dim3(Cfg::kThreads, 1, 1);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, l, c, l3, c3, out, p);
}

}  // namespace

cudaError_t launch_scaled(int idx, const CUtensorMap& l, const CUtensorMap& c, const CUtensorMap& l3,
                          const CUtensorMap& c3, const CUtensorMap& out, const ScaledParams& p, int grid,
                          cudaStream_t stream, bool pdl)
{
    static_assert(kNumScaledVariants == 7, "one case per variant below, in the order of kScaledVariants");
    switch (idx) {
    case 0: return launch_sc<256, false, false>(l, c, l3, c3, out, p, grid, stream, pdl);
    case 1: return launch_sc<256, false, true>(l, c, l3, c3, out, p, grid, stream, pdl);
    case 2: return launch_sc<128, false, false>(l, c, l3, c3, out, p, grid, stream, pdl);
    case 3: return launch_sc<128, false, true>(l, c, l3, c3, out, p, grid, stream, pdl);
    case 4: return launch_sc<64, true, true>(l, c, l3, c3, out, p, grid, stream, pdl);
    case 5: return launch_sc<32, true, true>(l, c, l3, c3, out, p, grid, stream, pdl);
    case 6: return launch_sc<16, true, true>(l, c, l3, c3, out, p, grid, stream, pdl);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace bwgemm
