// plan.h -- the plan behind bwgemm_plan_t, shared by the host-side translation
// units that launch on its behalf.
#pragma once

#include <vector>

#include "internal.h"

namespace bwgemm {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, looked up once; NULL without a driver.
EncodeTiledFn encode_fn();

struct TmapSlot {
    const void* ptr = nullptr;
    int64_t inner = 0, outer = 0, ld = 0;
    int64_t chunks = 0;  // 3-D K-chunk views: number of whole 64-element chunks (0: 2-D map)
    int dtype = -1;
    uint32_t box_inner = 0, box_outer = 0, box_depth = 0;
    int swizzle = -1;
    bool valid = false;
    CUtensorMap map;
};

// Makes the plan's device current for the lifetime of the guard.
struct DeviceGuard {
    int prev = -1;
    bool ok = false;
    explicit DeviceGuard(int dev)
    {
        if (cudaGetDevice(&prev) != cudaSuccess)
            prev = -1;
        ok = (prev == dev) || (cudaSetDevice(dev) == cudaSuccess);
    }
    ~DeviceGuard()
    {
        if (ok && prev >= 0)
            cudaSetDevice(prev);
    }
};

}  // namespace bwgemm

struct bwgemm_plan_s {
    int device = 0;
    int num_sms = 0;
    int max_active[bwgemm::kNumVariants] = {};
    bwgemm_plan_options_t opts;
    uint32_t* d_status = nullptr;
    uint8_t* d_workspace = nullptr;
    uint64_t workspace_bytes = 0;
    bwgemm::TmapSlot tmaps[6];  // A, B, C, the 3-D two-K-block views of A and B, C for paired stores
    bwgemm_config_t last;
    uint64_t launches = 0;
    uint32_t last_status_bits = 0;
    // device staging buffers of bwgemm_run_host
    void* h2d[3] = {nullptr, nullptr, nullptr};
    size_t h2d_cap[3] = {0, 0, 0};
    // bwgemm_run_host's pipeline over row blocks: copy-in, GEMM and copy-out
    // streams and their events (created on first use)
    cudaStream_t side[3] = {nullptr, nullptr, nullptr};
    cudaEvent_t events[bwgemm::kHostEvents] = {};
    bool side_ready = false;
    // optional timeline (opts.trace): kTraceSlots stamps per CTA of the last launch
    uint64_t* d_trace = nullptr;
    int trace_ctas = 0;
    int last_grid = 0;
    // options chosen by bwgemm_tune, per shape; bwgemm_run uses them for that shape
    struct Tuned {
        int64_t M, N, K;
        int dtype;
        bwgemm_plan_options_t opts;
    };
    std::vector<Tuned> tuned;
};
