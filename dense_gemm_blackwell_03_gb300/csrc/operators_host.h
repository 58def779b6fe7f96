// operators_host.h -- what the operators' host code shares: checks of arguments, tensor
// maps, and the options' limits.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "operators.h"
#include "plan.h"

namespace bwgemm {

// The workspace of a plan with these options (NULL = defaults).
inline uint64_t workspace_of(const bwgemm_plan_options_t* opts)
{
    return opts && opts->workspace_bytes ? opts->workspace_bytes : 64ull << 20;
}

// Of `workers` of `ctas` CTAs each, those that the options' cap on a persistent grid
// leaves (NULL = no cap).
inline int capped(int workers, int ctas, const bwgemm_plan_options_t* opts)
{
    return opts && opts->max_ctas > 0 ? std::min(workers, opts->max_ctas / ctas) : workers;
}

inline bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline int element_size(int dtype) { return dtype == BWGEMM_FP32 ? 4 : 2; }

inline int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// BWGEMM_OK when every pointer is device or managed memory of `device`.
inline bwgemm_status_t check_resident(std::initializer_list<const void*> ptrs, int device)
{
    for (const void* p : ptrs) {
        if (!p)
            continue;
        cudaPointerAttributes a;
        if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
            cudaGetLastError();  // an address the driver does not know: not this GPU's memory
            return BWGEMM_ERR_INVALID_ARG;
        }
        if ((a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged) || a.device != device)
            return BWGEMM_ERR_INVALID_ARG;
    }
    return BWGEMM_OK;
}

// Whether sizes and strides fit the kernels: rows, columns and K within a tile, at most
// 256 past its first, are counted in 32 bits; products with strides stay far inside 64.
inline bool extent_ok(int64_t rows, int64_t cols, int64_t ld)
{
    constexpr int64_t kMost = (1ll << 31) - 256;
    return rows <= kMost && cols <= kMost && ld < (1ll << 40);
}

inline bwgemm_status_t encode(CUtensorMap* map, CUtensorMapDataType type, uint32_t rank, const void* ptr, const cuuint64_t* dims,
                       const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle,
                       CUtensorMapL2promotion promotion)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc)
        return BWGEMM_ERR_NO_DEVICE;
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, type, rank, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? BWGEMM_OK
               : BWGEMM_ERR_CUDA;
}

}  // namespace bwgemm
