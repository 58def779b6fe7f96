// operators.cpp -- argument checks, tensor maps and work division of the
// operators beside the 16-bit GEMM (quantise, block-scaled product,
// orthogonalisation).
#include <algorithm>
#include <cmath>

#include "operators.h"
#include "operators_host.h"

using namespace bwgemm;

namespace {

// An 8-bit operand in boxes of 128 bytes x box_rows, and its 3-D view in boxes
// of `kps` whole K blocks (dimension 2: K blocks, 128 bytes apart).
bwgemm_status_t encode_operand(CUtensorMap* map, CUtensorMap* map3, const bwgemm_scaled_t& x, int64_t rows, int64_t K,
                               uint32_t box_rows, int kps)
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
    if (chunks < kps)
        return BWGEMM_OK;
    const cuuint64_t dims3[3] = {cuuint64_t(kBlock), cuuint64_t(rows), cuuint64_t(chunks)};
    const cuuint64_t strides3[2] = {cuuint64_t(x.ld), cuuint64_t(kBlock)};
    const cuuint32_t box3[3] = {uint32_t(kBlock), box_rows, uint32_t(kps)};
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

// The compiled form and the division of the work for one product; no workers where
// every form has more tiles than are counted.
struct ScaledPlan {
    int variant;
    int workers;
    int l_rows, num_l, num_c, dp_tiles, sk_tiles;
    int32_t sk_iters;
    int raster;
};

// Microseconds of one K block of a tile on its CTA: the bytes' way from L2 into
// shared memory (150 GB/s and SM), or the handshake with the epilogue and its
// additions (measured per form), whichever is longer.
double block_us(const ScaledVariant& v, int l_rows)
{
    const double step = v.bn == 256 ? 0.56 : v.bn == 128 ? 0.32 : v.bn == 64 ? 0.17 : 0.1;
    return std::max(step, (l_rows + v.bn) * 128.0 / 150e3);
}

// Whether the kernel for few rows of A takes the product, by both kernels' time:
// fitted in microseconds to M = 1, 8, 9 and 16 on 18 shapes.  Few rows: the bytes,
// the K blocks that a warp takes one after another, and the CTAs; tiles: the K
// blocks of a tile, split over CTAs where they are many, or the bytes.  Measured,
// few rows against tiles, weights from HBM: 1 x 1024 x 1024 1.5 and 5.9, 1 x 4096 x 4096
// 6.3 and 10.6, 1 x 8192 x 8192 16.7 and 19.0, 8 x 8192 x 8192 18.9 and 17.7 (from L2 12.9
// and 16.4), 1 x 16384 x 8192 30.2 and 23.3, 1 x 128 x 28672 16.5 and 29.7, 1 x 28672 x
// 1024 11.3 and 9.0; 16 x 4096 x 4096 10.3 and 10.7, 16 x 4096 x 8192 16.6 and 20.1,
// 16 x 8192 x 4096 14.5 and 12.1.
bool takes_few_rows(int64_t M, int64_t N, int64_t K)
{
    if (M > kScaledFewRows)
        return false;
    const double bytes = double(N) * double(K), kb = double(blocks_of(K));
    const double few = 1.5 + bytes / (M <= 8 ? 5.2e6 : 3.3e6) + 0.25 * kb / 8 + 75e-6 * double(N);
    const double tiles = 4.5 + std::max(std::min(0.2 * kb, 15.0), bytes / 6.5e6);
    return few <= tiles;
}

ScaledPlan plan_scaled(int num_sms, int64_t M, int64_t N, int64_t K, bool b_square, uint64_t workspace_bytes)
{
    const int64_t kb = blocks_of(K);
    const int W = num_sms;
    const double hbm_us = double(M + N) * double(K) / 6.5e6;  // both operands once
    ScaledPlan best = {};
    double best_us = 0;
    for (int i = 0; i < kNumScaledVariants; ++i) {
        const ScaledVariant& v = kScaledVariants[i];
        if (!v.swap && v.colvec == b_square)
            continue;  // the other form of the same tile
        const int64_t lrows = v.swap ? N : M, crows = v.swap ? M : N;
        const int64_t nc = (crows + v.bn - 1) / v.bn;
        // tiles of 128 lane rows; in the swapped form also lower ones, as high as
        // makes the tiles fill whole waves
        for (int low = 0; low <= (v.swap ? 1 : 0); ++low) {
            ScaledPlan s = {};
            s.variant = i;
            s.l_rows = 128;
            if (low) {
                const int64_t waves = ((lrows + 127) / 128 * nc + W - 1) / W;
                const int64_t blocks = std::max<int64_t>(waves * W / nc, 1);
                s.l_rows = int(std::min<int64_t>(128, ((lrows + blocks - 1) / blocks + 7) / 8 * 8));
            }
            const int64_t nl = (lrows + s.l_rows - 1) / s.l_rows, tiles = nl * nc;
            if (tiles > (1ll << 30))
                continue;
            s.num_l = int(nl);
            s.num_c = int(nc);
            // whole tiles, or whole tiles for the full waves and the rest in K iterations
            // over all workers; without a full wave over as many as have four K blocks each
            const int64_t full = tiles / W * W, rest = tiles - full;
            const uint64_t slot_bytes = uint64_t(128) * v.bn * 4;
            const bool room = kCounterRegionBytes + uint64_t(W) * 2 * slot_bytes <= workspace_bytes &&
                              uint64_t(rest) * 8 * 4 <= kCounterRegionBytes;
            for (int spread = 0; spread <= (rest > 0 && room && rest * kb < (1ll << 30) ? 1 : 0); ++spread) {
                s.workers = int(std::min<int64_t>(tiles, W));
                s.dp_tiles = int(tiles);
                s.sk_tiles = 0;
                s.sk_iters = 0;
                if (spread) {
                    s.dp_tiles = int(full);
                    s.sk_tiles = int(rest);
                    s.sk_iters = int32_t(rest * kb);
                    s.workers = full == 0 ? std::max(std::min(W, s.sk_iters / 4), 1) : W;
                    // the kernel adds the pieces of all workers from a tile's first to its last: each has one
                    if (s.sk_iters < s.workers)
                        continue;
                }
                const double us = block_us(v, s.l_rows);
                double t = double((s.dp_tiles + s.workers - 1) / s.workers) * double(kb) * us;
                if (spread) {
                    // a piece's partial tile out, the fence and the counter, and the
                    // pieces of a tile in again by one CTA
                    const double pieces = double(s.workers) / double(rest);
                    t += double((s.sk_iters + s.workers - 1) / s.workers) * us;
                    t += 4.0 + (1.0 + pieces) * 128.0 * v.bn * 4 / 200e3;
                }
                // bound by HBM, the form with the least work of its own is taken
                t = std::max(t, hbm_us) + 0.1 * t;
                if (best_us == 0 || t < best_us) {
                    best_us = t;
                    best = s;
                }
            }
        }
    }
    const ScaledVariant& v = kScaledVariants[best.variant];
    best.raster = v.swap ? best.num_l : 16;
    best.raster = std::max(1, std::min(best.raster, best.num_l));
    return best;
}

// ---------------------------------------------------------- orthogonalisation
constexpr int kOrthoMaxSteps = 64;
// The first products of the iteration take X in two fp16 terms: those of the
// second and third step (and the first, for fp32 input; 16-bit input is one
// term exactly).
//
// Why: rounding X to fp16 puts an error of 2^-12 of its large singular
// directions into its small ones, and the iteration multiplies small ones by up
// to 3.44 a step until all are near one; the earlier the rounding, the more it
// is amplified.  Rounding S and B matters less: S enters B beside a I.  Error
// of the result against 64 bits (512 x 512, 5 steps), with X in one term
// throughout / two terms in step 2 / in steps 2 and 3 / in steps 2 to 4:
// N(0, 1) 1.2e-3 / 1.1e-3 / 1.1e-3 / 1.1e-3; eight directions 30 times the
// rest 1.3e-2 / 2.9e-3 / 1.4e-3 / 1.3e-3; singular values 1 / i 1.8e-3 /
// 1.1e-3 / 7e-4 / 7e-4.  (Rounding the result to bf16 alone is 1.7e-3.)
// Rounding B in the same steps matters where all singular values are close (long
// matrices, or nearly orthogonal ones): its diagonal is then one value that rounds
// one way, an error of the whole result.  The diagonal blocks of 128 of B keep
// their low part: largest error over 60 matrices of 16 to 128 rows, up to 4096
// columns, N(0, 1), as a multiple of the bf16 rounding of the result: 2.34
// without, 1.42 with it (1.48 in steps 2 and 3 alone); 512 x 16384 1.82 and 1.28.
// It costs a K step per 128 rows of the tile, 16 x 512 x 1344 212 -> 226 us.
constexpr int kTwoTermSteps = 3;

struct OrthoLayout {
    bool wide;                    // columns >= rows: X X^T contracts over columns
    int64_t m, n;                 // the shorter and longer side
    int64_t ldx, lds;             // fp16 elements between rows of X, and of S and B
    int64_t x_stride, s_stride;   // per matrix
    int parts;                    // blocks per matrix of the input pass
    uint64_t hi[2], lo[2], s, b, sums, factors, total;  // byte offsets
};

OrthoLayout ortho_layout(int64_t batch, int64_t rows, int64_t cols)
{
    auto pad = [](int64_t v) { return (v + 63) / 64 * 64; };  // whole 64-column chunks
    OrthoLayout l;
    l.wide = rows <= cols;
    l.m = std::min(rows, cols);
    l.n = std::max(rows, cols);
    l.ldx = pad(cols);
    l.lds = pad(l.m);
    l.x_stride = rows * l.ldx;
    l.s_stride = l.m * l.lds;
    // 8K elements per block (a thread's pieces in flight), and all matrices
    // together a few blocks per SM
    const int64_t want = (rows * l.ldx + 8191) / 8192;
    l.parts = int(std::max<int64_t>(1, std::min<int64_t>(want, 1216 / batch)));
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    for (int i = 0; i < 2; ++i) {
        l.hi[i] = take(uint64_t(batch) * l.x_stride * 2);
        l.lo[i] = take(uint64_t(batch) * l.x_stride * 2);
    }
    l.s = take(uint64_t(batch) * l.s_stride * 2);
    l.b = take(uint64_t(batch) * l.s_stride * 2 * 2);  // B and its low part
    l.sums = take(uint64_t(batch) * l.parts * 4);
    l.factors = take(uint64_t(batch) * 2 * 4 * kOrthoMaxSteps);
    l.total = at;
    return l;
}

// A stack of fp16 matrices as operand: boxes of two 64-column chunks of 128 rows.
bwgemm_status_t encode_stack(CUtensorMap* map, const void* ptr, int64_t rows, int64_t ld, int64_t stride, int64_t batch)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc)
        return BWGEMM_ERR_NO_DEVICE;
    const cuuint64_t dims[4] = {64, cuuint64_t(rows), cuuint64_t(ld / 64), cuuint64_t(batch)};
    const cuuint64_t strides[3] = {cuuint64_t(ld) * 2, 128, cuuint64_t(stride) * 2};
    const cuuint32_t box[4] = {64, 128, 2, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? BWGEMM_OK
               : BWGEMM_ERR_CUDA;
}

// A stack of 16-bit matrices as result: boxes of 64 columns x 32 rows, or turned
// ones of 32 columns x 64 rows.
bwgemm_status_t encode_result(CUtensorMap* map, int dtype, void* ptr, int64_t rows, int64_t cols, int64_t ld,
                              int64_t stride, int64_t batch, bool turned = false)
{
    const cuuint64_t dims[3] = {cuuint64_t(cols), cuuint64_t(rows), cuuint64_t(batch)};
    const cuuint64_t strides[2] = {cuuint64_t(ld) * 2, cuuint64_t(stride) * 2};
    const cuuint32_t box[3] = {turned ? 32u : 64u, turned ? 64u : 32u, 1};
    return encode(map, dtype == BWGEMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, ptr,
                  dims, strides, box, turned ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

// A step's three products.
enum : int { kOrthoS = 0, kOrthoB = 1, kOrthoX = 2 };

int ortho_first_terms(int dtype) { return dtype == BWGEMM_FP32 ? 2 : 1; }

// The sizes of one of them: S = X X^T, B = a I + b S + c S S, X <- B X (X B upright).
OrthoParams ortho_shape(int which, const OrthoLayout& l, int64_t batch, int64_t rows, int64_t cols, int step,
                        int first_terms)
{
    OrthoParams p = {};
    p.batch = int32_t(batch);
    p.symmetric = which != kOrthoX;
    p.rows = int32_t(p.symmetric ? l.m : rows);
    p.cols = int32_t(p.symmetric ? l.m : cols);
    p.steps_k = int32_t(blocks_of(which == kOrthoS ? l.n : l.m));
    p.terms = 1;
    if (which == kOrthoX) {
        p.terms = step == 0 ? first_terms : (step < kTwoTermSteps ? 2 : 1);
        p.low_side = step >= kTwoTermSteps ? 0 : l.wide ? 1 : 2;
    }
    return p;
}

struct OrthoPlan {
    int cg;           // CTAs per tile: tiles of 128 on one, of 256 on a pair
    int64_t tiles;    // of all matrices
    int64_t workers;  // CTAs or pairs
};

// One product: square tiles of 256 on CTA pairs (1024 SM cycles per 128 of
// K, bound by the MMAs) or of 128 on single CTAs (about 740, bound by the
// copies of both operands), whichever takes fewer cycles in its waves; a
// deep K of few tiles in slices (`sliceable`: S), whose join costs a kernel more and the
// way of its bytes (us for the whole call, whole and in slices: 128 x 20000 335 and 93,
// 1024 x 4096 185 and 163, 300 x 1000 88 and 85; 2048 x 8192, whole, 538 and 546).
// Fills in p's division of the work; false where that would pass 32 bits.
bool plan_ortho_product(OrthoParams* p, bool sliceable, int singles, int pairs, uint64_t workspace_bytes, OrthoPlan* out)
{
    int64_t tiles[3] = {}, best = 0;
    int cg = 0;
    for (int g = 1; g <= (pairs > 0 ? 2 : 1); ++g) {
        const int64_t r = (p->rows + 128 * g - 1) / (128 * g), c = (p->cols + 128 * g - 1) / (128 * g);
        tiles[g] = (p->symmetric ? r * (r + 1) / 2 : r * c) * p->batch;
        const int64_t steps_all = int64_t(p->steps_k) * p->terms + (p->low_side ? g : 0);
        const int64_t workers = g == 2 ? pairs : singles;
        int64_t most = 1;
        if (sliceable) {
            const int64_t room = (int64_t(workspace_bytes) - int64_t(kCounterRegionBytes)) / (g * g * 128 * 128 * 4);
            most = std::max<int64_t>(1, std::min(std::min(workers, room) / tiles[g], steps_all / 2));
        }
        for (int64_t splits = 1; splits <= most; ++splits) {
            const int64_t cost = (tiles[g] * splits + workers - 1) / workers * ((steps_all + splits - 1) / splits) *
                                     (g == 2 ? 1024 : 740) +
                                 (splits > 1 ? 3000 + tiles[g] * splits * g * g * 65536 / 1250 : 0);
            if (cg == 0 || cost < best) {
                best = cost;
                cg = g;
                p->splits = int32_t(splits);
            }
        }
    }
    // of the join's CTAs some 2000 at most (24 tiles of 256 in three slices with
    // eight warps a piece, five of them idle: 13 us a product more than with one)
    for (p->join_share = 8;
         p->join_share > 1 && (p->join_share > p->splits || tiles[cg] * cg * cg * 16 * p->join_share > 2048);)
        p->join_share /= 2;
    if (tiles[cg] * p->splits >= (1ll << 31))
        return false;
    p->num_r = int32_t((p->rows + 128 * cg - 1) / (128 * cg));
    p->num_c = int32_t((p->cols + 128 * cg - 1) / (128 * cg));
    p->tiles = int32_t(tiles[cg] / p->batch);
    out->cg = cg;
    out->tiles = tiles[cg];
    out->workers = std::min<int64_t>(tiles[cg] * p->splits, cg == 2 ? pairs : singles);
    return true;
}

bwgemm_status_t check_ortho(int64_t batch, int64_t rows, int64_t cols)
{
    if (batch < 0 || rows < 0 || cols < 0)
        return BWGEMM_ERR_INVALID_ARG;
    if (batch > 65535 || rows > (1 << 24) || cols > (1 << 24) || std::min(rows, cols) > (1 << 17))
        return BWGEMM_ERR_UNSUPPORTED;
    return BWGEMM_OK;
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

    if (takes_few_rows(M, N, K)) {
        FewParams f = {};
        f.w = static_cast<const uint8_t*>(B->values);
        f.x = static_cast<const uint8_t*>(A->values);
        f.ldw = B->ld;
        f.ldx = A->ld;
        f.ws = B->scales;
        f.xs = A->scales;
        f.ws_ld = B->ld_scales;
        f.xs_ld = A->ld_scales;
        f.ws_shift = B->block == BWGEMM_BLOCK_SQUARE ? 7 : 0;
        f.xs_shift = A->block == BWGEMM_BLOCK_SQUARE ? 7 : 0;
        f.M = int32_t(M);
        f.N = int32_t(N);
        f.K = int32_t(K);
        f.num_kb = int32_t(blocks_of(K));
        f.c = C;
        f.ldc = ldc;
        f.out_type = out;
        f.accumulate = accumulate ? 1 : 0;
        if (launch_scaled_few(B->type, A->type, f, s, plan->opts.pdl_off == 0) != cudaSuccess)
            return BWGEMM_ERR_CUDA;
        plan->launches += 1;
        return BWGEMM_OK;
    }

    const ScaledPlan sel =
        plan_scaled(capped(plan->num_sms, 1, &plan->opts), M, N, K, B->block == BWGEMM_BLOCK_SQUARE, plan->workspace_bytes);
    if (sel.workers == 0)
        return BWGEMM_ERR_UNSUPPORTED;
    const ScaledVariant& v = kScaledVariants[sel.variant];
    const bwgemm_scaled_t& L = v.swap ? *B : *A;
    const bwgemm_scaled_t& R = v.swap ? *A : *B;
    ScaledParams p = {};
    p.lrows = int32_t(v.swap ? N : M);
    p.crows = int32_t(v.swap ? M : N);
    p.K = int32_t(K);
    p.num_kb = int32_t(blocks_of(K));
    const int kps = scaled_kps(v.bn, v.swap);
    p.chunks = K / kBlock >= kps ? int32_t(K / kBlock) : 0;
    p.stages = scaled_stages(v.bn, v.swap, sel.l_rows);
    p.l_rows = sel.l_rows;
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
    p.idesc = (make_idesc(BWGEMM_FP16, 128, v.bn) & ~((7u << 7) | (7u << 10))) | (uint32_t(L.type) << 7) |
              (uint32_t(R.type) << 10);
    p.timeout_ns = plan->opts.timeout_ns ? plan->opts.timeout_ns : 4000000000ull;
    p.status = plan->d_status;
    p.counters = reinterpret_cast<uint32_t*>(plan->d_workspace);
    p.partials = reinterpret_cast<float*>(plan->d_workspace + kCounterRegionBytes);
    p.stall_kblock = plan->opts.stall_kblock;

    CUtensorMap ml, ml3, mc, mc3, mo;
    if ((st = encode_operand(&ml, &ml3, L, p.lrows, K, uint32_t(sel.l_rows), kps)) != BWGEMM_OK ||
        (st = encode_operand(&mc, &mc3, R, p.crows, K, uint32_t(v.bn), kps)) != BWGEMM_OK)
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
    if (launch_scaled(sel.variant, ml, mc, ml3, mc3, mo, p, sel.workers, s, plan->opts.pdl_off == 0) != cudaSuccess)
        return BWGEMM_ERR_CUDA;
    plan->launches += 1;
    return BWGEMM_OK;
}

bwgemm_status_t bwgemm_select_scaled(int32_t num_sms, int64_t M, int64_t N, int64_t K, bwgemm_block_t b_block,
                                     const bwgemm_plan_options_t* opts, bwgemm_scaled_config_t* out)
{
    if (!out || num_sms < 1 || M < 1 || N < 1 || K < 1 || (b_block != BWGEMM_BLOCK_ROW && b_block != BWGEMM_BLOCK_SQUARE))
        return BWGEMM_ERR_INVALID_ARG;
    if (!extent_ok(M, K, K) || !extent_ok(N, K, K))
        return BWGEMM_ERR_UNSUPPORTED;
    *out = {};
    if (takes_few_rows(M, N, K)) {
        out->few_rows = 1;
        return BWGEMM_OK;
    }
    const ScaledPlan s =
        plan_scaled(capped(num_sms, 1, opts), M, N, K, b_block == BWGEMM_BLOCK_SQUARE, workspace_of(opts));
    if (s.workers == 0)
        return BWGEMM_ERR_UNSUPPORTED;
    const ScaledVariant& v = kScaledVariants[s.variant];
    out->swap_ab = v.swap;
    out->tile_l = s.l_rows;
    out->tile_c = v.bn;
    out->column_scales = v.colvec;
    out->dp_tiles = s.dp_tiles;
    out->sk_tiles = s.sk_tiles;
    out->workers = s.workers;
    return BWGEMM_OK;
}

bwgemm_status_t bwgemm_select_orthogonalize(int32_t num_sms, int32_t max_pairs, int64_t batch, int64_t rows, int64_t cols,
                                            bwgemm_dtype_t dtype, int32_t step, const bwgemm_plan_options_t* opts,
                                            bwgemm_ortho_config_t out[3])
{
    if (!out || num_sms < 1 || max_pairs < 0 || batch < 1 || rows < 1 || cols < 1 || step < 0 || step >= kOrthoMaxSteps ||
        (dtype != BWGEMM_BF16 && dtype != BWGEMM_FP16 && dtype != BWGEMM_FP32))
        return BWGEMM_ERR_INVALID_ARG;
    const bwgemm_status_t st = check_ortho(batch, rows, cols);
    if (st != BWGEMM_OK)
        return st;
    const OrthoLayout l = ortho_layout(batch, rows, cols);
    for (int which = kOrthoS; which <= kOrthoX; ++which) {
        OrthoParams p = ortho_shape(which, l, batch, rows, cols, step, ortho_first_terms(dtype));
        OrthoPlan s;
        if (!plan_ortho_product(&p, which == kOrthoS, capped(num_sms, 1, opts),
                                capped(max_pairs ? max_pairs : num_sms / 2, 2, opts), workspace_of(opts), &s))
            return BWGEMM_ERR_UNSUPPORTED;
        out[which] = {ortho_tile(s.cg), p.splits, s.tiles, int32_t(s.workers)};
    }
    return BWGEMM_OK;
}

bwgemm_status_t bwgemm_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols, uint64_t* bytes)
{
    if (!bytes)
        return BWGEMM_ERR_INVALID_ARG;
    *bytes = 0;
    const bwgemm_status_t st = check_ortho(batch, rows, cols);
    if (st != BWGEMM_OK || batch == 0 || rows == 0 || cols == 0)
        return st;
    *bytes = ortho_layout(batch, rows, cols).total;
    return BWGEMM_OK;
}

bwgemm_status_t bwgemm_orthogonalize(bwgemm_plan_t plan, const void* G, bwgemm_dtype_t dtype, void* X,
                                     bwgemm_dtype_t out, int64_t batch, int64_t rows, int64_t cols, int64_t ldg,
                                     int64_t stride_g, int64_t ldx, int64_t stride_x, int32_t steps,
                                     const float* coefficients, float eps, float scale, void* workspace,
                                     uint64_t workspace_bytes, void* stream)
{
    if (!plan || (dtype != BWGEMM_BF16 && dtype != BWGEMM_FP16 && dtype != BWGEMM_FP32) ||
        (out != BWGEMM_BF16 && out != BWGEMM_FP16) || steps < 1 || steps > kOrthoMaxSteps || !(eps >= 0.f))
        return BWGEMM_ERR_INVALID_ARG;
    bwgemm_status_t st = check_ortho(batch, rows, cols);
    if (st != BWGEMM_OK)
        return st;
    if (batch == 0 || rows == 0 || cols == 0)
        return BWGEMM_OK;
    if (!G || !X || !workspace || ldg < cols || ldx < cols ||
        (batch > 1 && (stride_g < (rows - 1) * ldg + cols || stride_x < (rows - 1) * ldx + cols)))
        return BWGEMM_ERR_INVALID_ARG;
    if (ldg >= (1ll << 31) || ldx >= (1ll << 31) || stride_g >= (1ll << 38) || stride_x >= (1ll << 38))
        return BWGEMM_ERR_UNSUPPORTED;
    if (!aligned(G, element_size(dtype)) || !aligned(X, 2) || !aligned(workspace, 256))
        return BWGEMM_ERR_ALIGNMENT;
    const OrthoLayout l = ortho_layout(batch, rows, cols);
    if (workspace_bytes < l.total)
        return BWGEMM_ERR_WORKSPACE;
    DeviceGuard guard(plan->device);
    if (!guard.ok)
        return BWGEMM_ERR_CUDA;
    if ((st = check_resident({G, X, workspace}, plan->device)) != BWGEMM_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool pdl = plan->opts.pdl_off == 0;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const int log2_scale = std::min(8, int(std::lround(0.5 * std::log2(double(l.m)))));
    const int first_terms = ortho_first_terms(dtype);

    OrthoInput in = {};
    in.g = G;
    in.ldg = ldg;
    in.stride_g = batch > 1 ? stride_g : 0;
    in.dtype = dtype;
    in.rows = int32_t(rows);
    in.cols = int32_t(cols);
    in.batch = int32_t(batch);
    const int64_t per_vector = 16 / element_size(dtype);
    in.vectors = aligned(G, 16) && ldg % per_vector == 0 && in.stride_g % per_vector == 0;
    in.eps = eps;
    in.log2_scale = log2_scale;
    in.steps = steps;
    for (int i = 0; i < steps; ++i) {
        const float a = std::fabs(coefficients ? coefficients[3 * i] : 3.4445f);
        in.growth[i] = a > 0.f && a < 1e30f ? int8_t(std::max(std::ceil(std::log2(a)), -100.f)) : 0;
    }
    in.sums = reinterpret_cast<float*>(ws + l.sums);
    in.parts = l.parts;
    in.hi = reinterpret_cast<uint16_t*>(ws + l.hi[0]);
    in.lo = first_terms == 2 ? reinterpret_cast<uint16_t*>(ws + l.lo[0]) : nullptr;
    in.ld = l.ldx;
    in.stride = l.x_stride;
    in.factors = reinterpret_cast<float*>(ws + l.factors);
    if (launch_ortho_input(in, s, pdl) != cudaSuccess)
        return BWGEMM_ERR_CUDA;
    plan->launches += 2;

    // operand maps of X (two buffers, two terms), S and B, and their result maps
    CUtensorMap x_op[2][2], x_res[2][2], s_op, s_res, s_turned, b_op, b_res, b_turned, final_res;
    for (int i = 0; i < 2; ++i)
        for (int t = 0; t < 2; ++t) {
            void* at = ws + (t ? l.lo[i] : l.hi[i]);
            if ((st = encode_stack(&x_op[i][t], at, rows, l.ldx, l.x_stride, batch)) != BWGEMM_OK ||
                (st = encode_result(&x_res[i][t], BWGEMM_FP16, at, rows, l.ldx, l.ldx, l.x_stride, batch)) != BWGEMM_OK)
                return st;
        }
    if ((st = encode_stack(&s_op, ws + l.s, l.m, l.lds, l.s_stride, batch)) != BWGEMM_OK ||
        (st = encode_result(&s_res, BWGEMM_FP16, ws + l.s, l.m, l.lds, l.lds, l.s_stride, batch)) != BWGEMM_OK ||
        (st = encode_result(&s_turned, BWGEMM_FP16, ws + l.s, l.m, l.lds, l.lds, l.s_stride, batch, true)) != BWGEMM_OK ||
        (st = encode_result(&b_turned, BWGEMM_FP16, ws + l.b, l.m, l.lds, l.lds, l.s_stride, 2 * batch, true)) != BWGEMM_OK ||
        (st = encode_stack(&b_op, ws + l.b, l.m, l.lds, l.s_stride, 2 * batch)) != BWGEMM_OK ||
        (st = encode_result(&b_res, BWGEMM_FP16, ws + l.b, l.m, l.lds, l.lds, l.s_stride, 2 * batch)) != BWGEMM_OK)
        return st;
    // a TMA store needs 16-byte rows, and clips a row's end only in whole
    // 16-byte pieces
    const bool plain = !aligned(X, 16) || ldx % 8 != 0 || cols % 8 != 0 || (batch > 1 && stride_x % 8 != 0);
    final_res = x_res[0][0];
    if (!plain && (st = encode_result(&final_res, out, X, rows, cols, ldx, batch > 1 ? stride_x : rows * ldx, batch)) !=
                      BWGEMM_OK)
        return st;

    const int singles = capped(plan->num_sms, 1, &plan->opts);
    const int pairs = capped(plan->max_active[find_variant(2, 256, false, 1)], 2, &plan->opts);
    auto product = [&](int form, OrthoParams p, bool sliceable, const CUtensorMap& a, const CUtensorMap& b,
                       const CUtensorMap& a2, const CUtensorMap& b2, const CUtensorMap& res, const CUtensorMap& res2) {
        p.timeout_ns = plan->opts.timeout_ns ? plan->opts.timeout_ns : 4000000000ull;
        p.status = plan->d_status;
        p.stall_kblock = plan->opts.stall_kblock;
        p.partials = reinterpret_cast<float*>(plan->d_workspace + kCounterRegionBytes);
        OrthoPlan sel;
        if (!plan_ortho_product(&p, sliceable, singles, pairs, plan->workspace_bytes, &sel))
            return BWGEMM_ERR_UNSUPPORTED;
        if (launch_ortho(form, sel.cg, a, b, a2, b2, res, res2, p, int(sel.workers * sel.cg), s, pdl) != cudaSuccess)
            return BWGEMM_ERR_CUDA;
        plan->launches += p.splits > 1 ? 2 : 1;
        return BWGEMM_OK;
    };

    const float down = std::ldexp(1.f, -log2_scale);
    int cur = 0;
    for (int i = 0; i < steps; ++i) {
        const float a = coefficients ? coefficients[3 * i] : 3.4445f;
        const float b = coefficients ? coefficients[3 * i + 1] : -4.7750f;
        const float c = coefficients ? coefficients[3 * i + 2] : 2.0315f;
        const CUtensorMap& x = x_op[cur][0];
        // S = X X^T over the longer side
        OrthoParams p = ortho_shape(kOrthoS, l, batch, rows, cols, i, first_terms);
        p.alpha = i == 0 ? 1.f : down * down;
        p.alpha_dev = in.factors + 2 * i * batch;
        p.store_cols = int32_t(l.lds);
        p.out = reinterpret_cast<uint16_t*>(ws + l.s);
        p.ldo = l.lds;
        p.stride_o = l.s_stride;
        if ((st = product(l.wide ? kOrthoNT : kOrthoTN, p, true, x, x, x, x, s_res, s_turned)) != BWGEMM_OK)
            return st;
        // B = a I + b S + c S S
        p = ortho_shape(kOrthoB, l, batch, rows, cols, i, first_terms);
        p.alpha = c;
        p.store_cols = int32_t(l.lds);
        p.beta = b;
        p.diag = a;
        p.low = i < kTwoTermSteps;
        p.e = reinterpret_cast<const uint16_t*>(ws + l.s);
        p.lde = l.lds;
        p.stride_e = l.s_stride;
        if ((st = product(kOrthoNT, p, false, s_op, s_op, s_op, s_op, b_res, b_turned)) != BWGEMM_OK)
            return st;
        // X <- B X, or X B with X stored upright
        const bool last = i == steps - 1;
        p = ortho_shape(kOrthoX, l, batch, rows, cols, i, first_terms);
        p.alpha = last ? scale * (i == 0 ? 1.f : down) : (i == 0 ? 1.f / down : 1.f);
        p.alpha_dev = in.factors + (2 * i + 1) * batch;
        p.store_cols = int32_t(last ? cols : l.ldx);
        p.low = !last && i + 1 < kTwoTermSteps;
        p.out_bf16 = last && out == BWGEMM_BF16;
        p.plain_store = last && plain;
        p.out = static_cast<uint16_t*>(X);
        p.ldo = ldx;
        p.stride_o = batch > 1 ? stride_x : 0;
        const CUtensorMap &x2 = p.terms == 2 ? x_op[cur][1] : x, &res = last ? final_res : x_res[cur ^ 1][0],
                          &res2 = x_res[cur ^ 1][1];
        st = l.wide ? product(kOrthoNN, p, false, b_op, x, b_op, x2, res, res2)
                    : product(kOrthoNT, p, false, x, b_op, x2, b_op, res, res2);
        if (st != BWGEMM_OK)
            return st;
        cur ^= 1;
    }
    return BWGEMM_OK;
}

}  // extern "C"
