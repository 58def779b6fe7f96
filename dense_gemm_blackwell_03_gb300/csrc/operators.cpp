// operators.cpp -- argument checks, tensor maps and work division of the
// operators beside the 16-bit GEMM (quantise, block-scaled product).
#include <algorithm>

#include "operators.h"
#include "plan.h"

using namespace bwgemm;

namespace {

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

int element_size(int dtype) { return dtype == BWGEMM_FP32 ? 4 : 2; }

int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

// BWGEMM_OK when every pointer is device or managed memory of `device`.
bwgemm_status_t check_resident(std::initializer_list<const void*> ptrs, int device)
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

// Elements between the first and one past the last of `rows` rows of `cols`.
bool extent_ok(int64_t rows, int64_t cols, int64_t ld)
{
    // products of sizes and strides stay far inside 64 bits
    return rows < (1ll << 31) && cols < (1ll << 31) && ld < (1ll << 40);
}

bwgemm_status_t encode(CUtensorMap* map, CUtensorMapDataType type, uint32_t rank, const void* ptr, const cuuint64_t* dims,
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

// An 8-bit operand in boxes of 128 bytes x box_rows, and its 3-D view in boxes
// of kScaledKps whole K blocks (dimension 2: K blocks, 128 bytes apart).
bwgemm_status_t encode_operand(CUtensorMap* map, CUtensorMap* map3, const bwgemm_scaled_t& x, int64_t rows, int64_t K,
                               uint32_t box_rows)
{
    const cuuint64_t dims[2] = {cuuint64_t(K), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(x.ld)};
    const cuuint32_t box[2] = {uint32_t(kBlock), box_rows};
    bwgemm_status_t st = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, x.values, dims, strides, box,
                                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    if (st != BWGEMM_OK)
        return st;
    *map3 = *map;
    const int64_t chunks = K / kBlock;
    if (chunks < kScaledKps)
        return BWGEMM_OK;
    const cuuint64_t dims3[3] = {cuuint64_t(kBlock), cuuint64_t(rows), cuuint64_t(chunks)};
    const cuuint64_t strides3[2] = {cuuint64_t(x.ld), cuuint64_t(kBlock)};
    const cuuint32_t box3[3] = {uint32_t(kBlock), box_rows, uint32_t(kScaledKps)};
    return encode(map3, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, x.values, dims3, strides3, box3, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

bwgemm_status_t check_operand(const bwgemm_scaled_t* x, int64_t rows, int64_t K)
{
    if (!x || (x->type != BWGEMM_E4M3 && x->type != BWGEMM_E5M2) ||
        (x->block != BWGEMM_BLOCK_ROW && x->block != BWGEMM_BLOCK_SQUARE))
        return BWGEMM_ERR_INVALID_ARG;
    if (rows == 0 || K == 0)
        return BWGEMM_OK;  // neither read
    if (!x->values || !x->scales || x->ld < K ||
        x->ld_scales < (x->block == BWGEMM_BLOCK_ROW ? rows : blocks_of(rows)))
        return BWGEMM_ERR_INVALID_ARG;
    if (!extent_ok(rows, K, x->ld) || x->ld_scales >= (1ll << 40))
        return BWGEMM_ERR_UNSUPPORTED;
    if (!aligned(x->values, 16) || x->ld % 16 != 0 || !aligned(x->scales, 4))
        return BWGEMM_ERR_ALIGNMENT;
    return BWGEMM_OK;
}

// The compiled form and the division of the work for one product.
struct ScaledPlan {
    int variant;
    int workers, grid;
    int num_l, num_c, dp_tiles, sk_tiles;
    int64_t sk_iters;
    int raster;
};

// Microseconds of one K block of a tile on its CTA (or pair): the larger of the
// MMAs and of the bytes' way from L2 into shared memory.
double block_us(const ScaledVariant& v)
{
    const double mma = 2.0 * 128 * v.bn * 128 / (v.bn >= 64 ? 16384.0 : 8192.0) / 1.9e3;
    const double bytes = (128.0 + double(v.bn) / v.cg) * 128;
    return std::max(mma, bytes / 150e3);
}

ScaledPlan plan_scaled(int num_sms, int max_pairs, int64_t M, int64_t N, int64_t K, bool b_square,
                       uint64_t workspace_bytes)
{
    const int64_t kb = blocks_of(K);
    ScaledPlan best = {};
    double best_us = 0;
    for (int i = 0; i < kNumScaledVariants; ++i) {
        const ScaledVariant& v = kScaledVariants[i];
        if (!v.swap && v.colvec == b_square)
            continue;  // the other form of the same tile
        ScaledPlan s = {};
        s.variant = i;
        const int64_t lrows = v.swap ? N : M, crows = v.swap ? M : N;
        const int64_t nl = (lrows + v.cg * 128 - 1) / (v.cg * 128), nc = (crows + v.bn - 1) / v.bn;
        const int64_t tiles = nl * nc;
        if (tiles > (1ll << 30))
            continue;
        const int W = v.cg == 2 ? max_pairs : num_sms;
        s.num_l = int(nl);
        s.num_c = int(nc);
        // whole tiles for the full waves; the rest in K iterations over all
        // workers unless it nearly fills a wave itself, at least four K blocks
        // a piece (a shorter piece costs more in partial sums than it saves)
        const int64_t full = tiles / W * W, rest = tiles - full;
        const uint64_t slot_bytes = uint64_t(v.cg) * 128 * v.bn * 4;
        const bool room = kCounterRegionBytes + uint64_t(W) * 2 * slot_bytes <= workspace_bytes &&
                          uint64_t(rest) * uint64_t(v.cg) * 8 * 4 <= kCounterRegionBytes;
        const bool spread = rest > 0 && rest * 100 < int64_t(W) * 90 && room && (full > 0 || rest * kb / 4 > rest);
        s.workers = W;
        if (spread) {
            s.dp_tiles = int(full);
            s.sk_tiles = int(rest);
            s.sk_iters = rest * kb;
            if (full == 0)
                s.workers = int(std::max<int64_t>(std::min<int64_t>(W, s.sk_iters / 4), 1));
        } else {
            s.dp_tiles = int(tiles);
            s.workers = int(std::min<int64_t>(tiles, W));
        }
        s.grid = s.workers * v.cg;
        const double us = block_us(v);
        const double waves = double((s.dp_tiles + s.workers - 1) / s.workers);
        double t = waves * double(kb) * us;
        if (spread) {
            const double pieces = double(s.workers) / double(rest);
            t += double((s.sk_iters + s.workers - 1) / s.workers) * us;
            // a piece's partial tile out, and the pieces of a tile in again by one CTA
            if (pieces > 1.0)
                t += (1.0 + pieces) * 128.0 * v.bn * 4 / 200e3 + 1.0;
        }
        if (best_us == 0 || t < best_us) {
            best_us = t;
            best = s;
        }
    }
    const ScaledVariant& v = kScaledVariants[best.variant];
    best.raster = v.swap ? best.num_l : 8;
    best.raster = std::max(1, std::min(best.raster, best.num_l));
    return best;
}

}  // namespace

extern "C" {

bwgemm_status_t bwgemm_quantize(bwgemm_plan_t plan, const void* X, bwgemm_dtype_t dtype, int64_t rows,
                                int64_t cols, int64_t ldx, bwgemm_block_t block, bwgemm_fp8_t type,
                                int32_t pow2, void* q, int64_t ldq, float* scales, int64_t ld_scales,
                                void* qt, int64_t ldqt, float* scales_t, int64_t ld_scales_t, void* stream)
{
    if (!plan || (dtype != BWGEMM_BF16 && dtype != BWGEMM_FP16 && dtype != BWGEMM_FP32) ||
        (block != BWGEMM_BLOCK_ROW && block != BWGEMM_BLOCK_SQUARE) || (type != BWGEMM_E4M3 && type != BWGEMM_E5M2) ||
        rows < 0 || cols < 0)
        return BWGEMM_ERR_INVALID_ARG;
    if ((qt == nullptr) != (scales_t == nullptr))
        return BWGEMM_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0)
        return BWGEMM_OK;
    const bool square = block == BWGEMM_BLOCK_SQUARE;
    const int64_t kblocks = blocks_of(cols), rblocks = blocks_of(rows);
    if (!X || !q || !scales || ldx < cols || ldq < cols || ld_scales < (square ? rblocks : rows))
        return BWGEMM_ERR_INVALID_ARG;
    if (qt && (ldqt < rows || ld_scales_t < (square ? kblocks : cols)))
        return BWGEMM_ERR_INVALID_ARG;
    if (!extent_ok(rows, cols, ldx) || !extent_ok(rows, cols, ldq) || !extent_ok(rows, cols, ldqt) ||
        kblocks * rblocks >= (1ll << 31))
        return BWGEMM_ERR_UNSUPPORTED;
    if (!aligned(X, 16) || ldx * element_size(dtype) % 16 != 0 || !aligned(q, 16) || ldq % 16 != 0 ||
        !aligned(scales, 4) || !aligned(qt, 16) || (qt && ldqt % 16 != 0) || !aligned(scales_t, 4))
        return BWGEMM_ERR_ALIGNMENT;
    DeviceGuard guard(plan->device);
    if (!guard.ok)
        return BWGEMM_ERR_CUDA;
    const bwgemm_status_t st = check_resident({X, q, scales, qt, scales_t}, plan->device);
    if (st != BWGEMM_OK)
        return st;
    QuantizeParams p = {};
    p.x = X;
    p.ldx = ldx;
    p.rows = rows;
    p.cols = cols;
    p.q = static_cast<uint8_t*>(q);
    p.ldq = ldq;
    p.s = scales;
    p.lds = ld_scales;
    p.qt = static_cast<uint8_t*>(qt);
    p.ldqt = ldqt;
    p.st = scales_t;
    p.ldst = ld_scales_t;
    p.pow2 = pow2 != 0;
    if (launch_quantize(dtype, type, square, p, static_cast<cudaStream_t>(stream), plan->opts.pdl_off == 0) !=
        cudaSuccess)
        return BWGEMM_ERR_CUDA;
    plan->launches += 1;
    return BWGEMM_OK;
}

bwgemm_status_t bwgemm_run_scaled(bwgemm_plan_t plan, const bwgemm_scaled_t* A, const bwgemm_scaled_t* B,
                                  void* C, int64_t M, int64_t N, int64_t K, int64_t ldc, bwgemm_dtype_t out,
                                  int32_t accumulate, void* stream)
{
    if (!plan || M < 0 || N < 0 || K < 0 || (out != BWGEMM_BF16 && out != BWGEMM_FP16 && out != BWGEMM_FP32) ||
        (accumulate && out != BWGEMM_FP32))
        return BWGEMM_ERR_INVALID_ARG;
    bwgemm_status_t st;
    if ((st = check_operand(A, M, K)) != BWGEMM_OK || (st = check_operand(B, N, K)) != BWGEMM_OK)
        return st;
    if (M == 0 || N == 0)
        return BWGEMM_OK;
    const int es = element_size(out);
    if (!C || ldc < N)
        return BWGEMM_ERR_INVALID_ARG;
    if (!extent_ok(M, N, ldc))
        return BWGEMM_ERR_UNSUPPORTED;
    if (!aligned(C, 16) || ldc * es % 16 != 0)
        return BWGEMM_ERR_ALIGNMENT;
    DeviceGuard guard(plan->device);
    if (!guard.ok)
        return BWGEMM_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) {  // empty sum
        if ((st = check_resident({C}, plan->device)) != BWGEMM_OK || accumulate)
            return st;
        return cudaMemset2DAsync(C, size_t(ldc) * es, 0, size_t(N) * es, size_t(M), s) == cudaSuccess ? BWGEMM_OK
                                                                                                     : BWGEMM_ERR_CUDA;
    }
    if ((st = check_resident({A->values, A->scales, B->values, B->scales, C}, plan->device)) != BWGEMM_OK)
        return st;

    const ScaledPlan sel =
        plan_scaled(plan->num_sms, plan->max_active[find_variant(2, 256, false, 1)], M, N, K,
                    B->block == BWGEMM_BLOCK_SQUARE, plan->workspace_bytes);
    const ScaledVariant& v = kScaledVariants[sel.variant];
    const bwgemm_scaled_t& L = v.swap ? *B : *A;
    const bwgemm_scaled_t& R = v.swap ? *A : *B;
    ScaledParams p = {};
    p.lrows = int32_t(v.swap ? N : M);
    p.crows = int32_t(v.swap ? M : N);
    p.K = int32_t(K);
    p.num_kb = int32_t(blocks_of(K));
    p.chunks = K / kBlock >= kScaledKps ? int32_t(K / kBlock) : 0;
    p.num_l = sel.num_l;
    p.num_c = sel.num_c;
    p.raster_group = sel.raster;
    p.dp_tiles = sel.dp_tiles;
    p.sk_tiles = sel.sk_tiles;
    p.sk_iters = sel.sk_iters;
    p.ls = L.scales;
    p.ls_ld = L.ld_scales;
    p.ls_shift = L.block == BWGEMM_BLOCK_SQUARE ? 7 : 0;
    p.cs = R.scales;
    p.cs_ld = R.ld_scales;
    p.cs_shift = R.block == BWGEMM_BLOCK_SQUARE ? 7 : 0;
    p.c = C;
    p.ldc = ldc;
    p.out_type = out;
    p.accumulate = accumulate ? 1 : 0;
    // the instruction descriptor of the 16-bit products with the operand types
    // of kind::f8f6f4 (e4m3 = 0, e5m2 = 1) in the same fields
    p.idesc = (make_idesc(BWGEMM_FP16, 128 * v.cg, v.bn) & ~((7u << 7) | (7u << 10))) | (uint32_t(L.type) << 7) |
              (uint32_t(R.type) << 10);
    p.timeout_ns = plan->opts.timeout_ns ? plan->opts.timeout_ns : 4000000000ull;
    p.status = plan->d_status;
    p.counters = reinterpret_cast<uint32_t*>(plan->d_workspace);
    p.partials = reinterpret_cast<float*>(plan->d_workspace + kCounterRegionBytes);
    p.stall_kblock = plan->opts.stall_kblock;

    CUtensorMap ml, ml3, mc, mc3, mo;
    if ((st = encode_operand(&ml, &ml3, L, p.lrows, K, uint32_t(kRowsPerCta))) != BWGEMM_OK ||
        (st = encode_operand(&mc, &mc3, R, p.crows, K, uint32_t(v.bn / v.cg))) != BWGEMM_OK)
        return st;
    mo = ml;
    if (!v.swap) {
        const cuuint64_t dims[2] = {cuuint64_t(N), cuuint64_t(M)};
        const cuuint64_t strides[1] = {cuuint64_t(ldc) * es};
        const cuuint32_t box[2] = {uint32_t(64 / es), 32};
        const CUtensorMapDataType type = out == BWGEMM_FP32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                         : out == BWGEMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        if ((st = encode(&mo, type, 2, C, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_NONE)) != BWGEMM_OK)
            return st;
    }
    if (launch_scaled(sel.variant, ml, mc, ml3, mc3, mo, p, sel.grid, s, plan->opts.pdl_off == 0) != cudaSuccess)
        return BWGEMM_ERR_CUDA;
    plan->launches += 1;
    return BWGEMM_OK;
}

}  // extern "C"
