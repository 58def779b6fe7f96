// feed_forward.cpp -- argument checks, tensor maps and work division of the gated
// feed-forward layer and of the 8-bit integer product.
#include <cmath>

#include "feed_forward.h"
#include "operators_host.h"

using namespace bwgemm;

namespace {

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

uint64_t limit_ns(bwgemm_plan_t plan) { return plan->opts.timeout_ns ? plan->opts.timeout_ns : 4000000000ull; }

// Whether the pointer is there (an absent matrix, or one without data, is none).
bool present(const bwgemm_matrix_t* x) { return x && x->data; }

bwgemm_status_t check_matrix(const bwgemm_matrix_t* x, int64_t rows, int64_t cols)
{
    if (!present(x) || x->ld < cols)
        return BWGEMM_ERR_INVALID_ARG;
    if (!extent_ok(rows, cols, x->ld))
        return BWGEMM_ERR_UNSUPPORTED;
    if (!aligned(x->data, 16) || x->ld % 8 != 0)
        return BWGEMM_ERR_ALIGNMENT;
    return BWGEMM_OK;
}

CUtensorMapDataType type16(int dtype)
{
    return dtype == BWGEMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// A 16-bit operand in boxes of two whole 64-element chunks x box_rows (map3), and of one
// (map), which is read at and past the end of rows that are no multiple of `step`, the columns
// that its tiles advance by.  A map that no copy uses is a copy of the other.
bwgemm_status_t encode_operand16(CUtensorMap* map, CUtensorMap* map3, const void* data, int64_t ld, int dtype, int64_t rows,
                                 int64_t cols, uint32_t box_rows, int64_t step = 128)
{
    const int64_t chunks = cols / 64;
    if (chunks >= 2) {
        const cuuint64_t dims3[3] = {64, cuuint64_t(rows), cuuint64_t(chunks)};
        const cuuint64_t strides3[2] = {cuuint64_t(ld) * 2, 128};
        const cuuint32_t box3[3] = {64, box_rows, 2};
        const bwgemm_status_t st = encode(map3, type16(dtype), 3, data, dims3, strides3, box3, CU_TENSOR_MAP_SWIZZLE_128B,
                                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
        if (st != BWGEMM_OK)
            return st;
        *map = *map3;
        if (cols % step == 0)
            return BWGEMM_OK;
    }
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
    const cuuint32_t box[2] = {64, box_rows};
    const bwgemm_status_t st = encode(map, type16(dtype), 2, data, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    if (chunks < 2)
        *map3 = *map;
    return st;
}

// 8-bit integers in boxes of 128 x box_rows (map), and of two whole 128s of K (map3); as above.
bwgemm_status_t encode_bytes(CUtensorMap* map, CUtensorMap* map3, const void* data, int64_t ld, int64_t rows, int64_t K,
                             uint32_t box_rows, CUtensorMapSwizzle swizzle)
{
    if (K >= 256) {
        const cuuint64_t dims3[3] = {128, cuuint64_t(rows), cuuint64_t(K / 128)};
        const cuuint64_t strides3[2] = {cuuint64_t(ld), 128};
        const cuuint32_t box3[3] = {128, box_rows, 2};
        const bwgemm_status_t st = encode(map3, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, data, dims3, strides3, box3, swizzle,
                                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
        if (st != BWGEMM_OK)
            return st;
    }
    const cuuint64_t dims[2] = {cuuint64_t(K), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld)};
    const cuuint32_t box[2] = {128, box_rows};
    const bwgemm_status_t st = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, data, dims, strides, box, swizzle,
                                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    if (K < 256)
        *map3 = *map;
    return st;
}

bwgemm_status_t encode_result16(CUtensorMap* map, const bwgemm_matrix_t& x, int dtype, int64_t rows, int64_t cols)
{
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(x.ld) * 2};
    const cuuint32_t box[2] = {64, 32};
    return encode(map, type16(dtype), 2, x.data, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

// ------------------------------------------------ work with the weights in the lanes
struct LanesPlan {
    int variant;      // of kLanesVariants
    int workers;      // CTAs or pairs; 0: none
    int l_rows, num_l, num_c, dp_tiles, sk_tiles, sk_iters, raster;
    double us;
};

// What a launch takes in microseconds, fitted to 20 to 400 rows on eight shapes (1024 x 8192 to
// 14336 x 4096): a call without its K steps; 128 of K of a tile on its CTA or pair, weights at
// hand (the way through its barriers, the MMAs, and the widening); and, where tiles are cut into
// pieces, a piece's way out and the others' in again by the warps that come last.
double lanes_base_us(const LanesVariant& v)
{
    return v.mode == kLanesGated ? 6.0 : v.widens ? 5.0 : 9.0;  // (9: launch_widen before it)
}

double lanes_step_us(const LanesVariant& v)
{
    if (v.mode == kLanesGated)
        return v.bn == 128 ? 0.78 : v.bn == 64 ? 0.51 : v.bn == 32 ? 0.41 : 0.36;
    return v.cg == 2 ? 0.58 : v.bn == 128 ? 0.375 : v.bn >= 32 ? 0.27 : 0.24;
}

double lanes_join_us(const LanesVariant& v, int pieces)
{
    const int groups = std::max(v.bn / (lanes_epi_warps(v.bn) / 4) / 32, 1);  // of columns that a warp adds one after the other
    if (v.mode == kLanesGated)
        return (v.bn == 128 ? 20.0 : v.bn == 64 ? 15.0 : v.bn == 32 ? 7.5 : 4.0) + groups * std::max(pieces - 4, 0);
    return 2.5 + 0.55 * groups * pieces;
}

// Weights from which on tiles of 32 rows of X take it widened before: their bytes come faster
// than a step of 32 rows is widened (see lanes_kernel.cuh).
constexpr double kWidenedBefore = 100e6;

// Whether a product of 8-bit integers takes X as it is at every division of its work: there
// is no workspace for its fp16 then.
bool widens_always(int64_t M, int64_t N, int64_t K)
{
    return M <= 16 || (M <= 32 && double(N) * double(K) <= kWidenedBefore);
}

// Whether the integers' product is computed with A's rows in the lanes: where B has fewer rows
// it is B that is widened then, and read again by every tile.  That saves the way of 3 bytes for
// each element that A has more, and costs a little for each of the result (us, so and with B's
// rows in the lanes: 8192 x 1024 x 8192 81 and 114, 7791 x 260 x 23859 99 and 216, 4416 x 256 x 2790
// 12.6 and 19.0, 4096 x 3000 x 4096 71.2 and 71.5; 6978 x 3467 x 128 37 and 32, 4096 x 4000 x 1024 33.6 and 31.8).
bool takes_turned(int64_t M, int64_t N, int64_t K)
{
    return M > N && N > 32 && 3.0 * double(M - N) * double(K) > double(M) * double(N);
}

LanesPlan plan_lanes(int mode, int num_sms, int max_pairs, int64_t M, int64_t N, int64_t K,
                     const bwgemm_plan_options_t* opts, uint64_t workspace_bytes)
{
    const int64_t kb = blocks_of(K);
    const double weights = double(N) * double(K) * (mode == kLanesGated ? 4 : 1);
    LanesPlan best = {};
    for (int i = 0; i < kNumLanesVariants; ++i) {
        const LanesVariant& v = kLanesVariants[i];
        if (v.mode != mode)
            continue;
        if (mode == kLanesInt8 && (widens_always(M, N, K) ? !v.widens : v.widens && double(N) * double(K) > kWidenedBefore))
            continue;
        const int W = v.cg == 2 ? capped(max_pairs, 2, opts) : capped(num_sms, 1, opts);
        if (W < 1)
            continue;
        const int most = v.mode == kLanesGated ? 64 : 128 * v.cg;  // weight rows per tile
        const int64_t nc = (M + v.bn - 1) / v.bn;
        for (int low = v.cg == 1 ? 1 : 0; low >= 0; --low) {
            LanesPlan s = {};
            s.variant = i;
            s.l_rows = most;
            if (low) {  // tiles as high as makes them fill whole waves
                const int64_t waves = ((N + most - 1) / most * nc + W - 1) / W;
                const int64_t blocks = std::max<int64_t>(waves * W / nc, 1);
                s.l_rows = int(std::min<int64_t>(most, round_up((N + blocks - 1) / blocks, 8)));
            }
            const int64_t nl = (N + s.l_rows - 1) / s.l_rows, tiles = nl * nc;
            if (tiles > (1ll << 30))
                continue;
            s.num_l = int(nl);
            s.num_c = int(nc);
            // whole tiles, or whole tiles for the full waves and the rest in K steps over all workers
            const int64_t full = tiles / W * W, rest = tiles - full;
            const uint64_t slot_bytes = uint64_t(lanes_partial_floats(mode, v.bn)) * 4 * v.cg;
            const bool room = kCounterRegionBytes + uint64_t(W) * 2 * slot_bytes <= workspace_bytes &&
                              uint64_t(rest) * v.cg * lanes_epi_warps(v.bn) * 4 <= kCounterRegionBytes;
            // (spread: over all workers, or, where there is no full wave, over all that have four
            // steps each, over as many a tile as there are for each, or half as many: a worker
            // then has one piece, not two)
            for (int spread = 0; spread <= (rest > 0 && room && rest * kb < (1ll << 30) ? (full == 0 ? 3 : 1) : 0); ++spread) {
                s.workers = int(std::min<int64_t>(tiles, W));
                s.dp_tiles = int(tiles);
                s.sk_tiles = s.sk_iters = 0;
                if (spread) {
                    s.dp_tiles = int(full);
                    s.sk_tiles = int(rest);
                    s.sk_iters = int(rest * kb);
                    s.workers = full == 0 ? std::max(std::min(W, s.sk_iters / 4), 1) : W;
                    if (spread > 1)
                        s.workers = int(std::max<int64_t>(s.workers / rest / (spread - 1), 1) * rest);
                    // the kernel adds the pieces of all workers from a tile's first to its last: each has one
                    if (s.workers > W || s.sk_iters < s.workers)
                        continue;
                }
                const double us = lanes_step_us(v), whole = double((s.dp_tiles + s.workers - 1) / s.workers) * double(kb) * us;
                const double steps = whole + (spread ? double((s.sk_iters + s.workers - 1) / s.workers) * us : 0.0);
                // the weights once from HBM; bound by that, the form with the least work of its own
                double t = lanes_base_us(v) + std::max(steps, weights / 6.5e6 + 0.1 * steps);
                if (spread) {
                    // two pieces a worker: what the second's steps do not cover of the first's; whole
                    // tiles, which come after them, cover them but for what delays their own, and no
                    // more of them than TMEM has buffers for
                    const bool one = s.workers % rest == 0;
                    const double join = lanes_join_us(v, int((s.workers + rest - 1) / rest) + (one ? 0 : 1));
                    if (full > 0)
                        t += std::max((mode == kLanesGated ? 1.0 : 0.5) * join,
                                      2.0 * join - std::min(whole, (v.bn == 256 ? 1 : 2) * double(kb) * us));
                    else
                        t += join + (one ? 0.0 : std::max(0.0, join - steps / 2));
                }
                if (best.workers == 0 || t < best.us) {
                    s.us = t;
                    best = s;
                }
            }
        }
    }
    // groups of eight tile rows, all columns of one before the next: weights are read again from L2
    best.raster = std::max(std::min(8, best.num_l), 1);
    return best;
}

// ------------------------------------------------------------- tiles of products
// The gradients' products.  No workers where there is no division.
struct PairPlan {
    PairProduct prod[2];
    int early;
    int cg;
    int workers;  // CTAs or pairs
};

// The longest worker's cycles when `workers` share the units of both products as pair_unit has
// it, and the count of early ones that makes them fewest.
int64_t pair_cycles(const PairProduct (&d)[2], int64_t workers, int64_t step, int* early)
{
    int64_t unit[2], best = -1;
    for (int i = 0; i < 2; ++i)
        unit[i] = (d[i].steps + d[i].splits - 1) / d[i].splits * step + 500;
    const int64_t turns = d[0].units / workers, rest = d[0].units % workers, others = workers - rest;
    const int64_t even = rest > 0 ? unit[0] / unit[1] : 0, most = (d[1].units + others - 1) / others;
    for (int64_t e : {int64_t(0), even, even + 1}) {
        if (e > 0 && (rest == 0 || d[1].units == 0))
            continue;
        e = std::min(e, most);
        const int64_t left = std::max<int64_t>(d[1].units - e * others, 0);
        // of those with one more of the first product's, and of the others
        const int64_t with = (turns + 1) * unit[0] + (left + workers - 1) / workers * unit[1];
        const int64_t without = turns * unit[0] + (e + (left + workers - 1 - rest) / workers) * unit[1];
        const int64_t cycles = rest > 0 ? std::max(with, without) : without;
        if (best < 0 || cycles < best) {
            best = cycles;
            *early = int(e);
        }
    }
    return best;
}

// Tiles of 256 on CTA pairs (1024 SM cycles per 128 of K, bound by the MMAs) or of 128 on
// single CTAs (about 740, bound by the copies of both operands), whichever take fewer
// cycles; few tiles and a deep K in slices, whose join costs a kernel more and the way of
// its bytes.
PairPlan plan_backward(int64_t M, int64_t N, int64_t K, bool of_x, bool of_w, int singles, int pairs,
                       uint64_t workspace_bytes)
{
    PairPlan best = {};
    int64_t best_cycles = 0;
    for (int g = 1; g <= 2; ++g) {
        const int64_t workers = g == 2 ? pairs : singles, tile = 128 * g;
        if (workers < 1)
            continue;
        PairPlan s = {};
        s.cg = g;
        PairProduct &x = s.prod[0], &w = s.prod[1];
        x = {int32_t(M), int32_t(K), int32_t(2 * blocks_of(N)), 1, int32_t((M + tile - 1) / tile), int32_t((K + tile - 1) / tile),
             1, 0, 1};
        w = {int32_t(N), int32_t(K), int32_t(blocks_of(M)), 2, int32_t((N + tile - 1) / tile), x.num_c, 1, 0, 1};
        const int64_t tiles[2] = {of_x ? int64_t(x.num_r) * x.num_c : 0, of_w ? 2 * int64_t(w.num_r) * w.num_c : 0};
        if (tiles[0] + tiles[1] >= (1ll << 31))
            continue;
        const int64_t room = (int64_t(workspace_bytes) - int64_t(kCounterRegionBytes)) / (tile * tile * 4);
        auto slices = [&](int i, int64_t splits) {  // whether product i may be cut so
            return splits == 1 || (tiles[i] * splits <= std::min(2 * workers, room) && s.prod[i].steps >= 2 * splits);
        };
        for (int64_t sx = 1; slices(0, sx); sx = sx < 4 ? sx + 1 : sx * 3 / 2)
            for (int64_t sw = 1; slices(1, sw); sw = sw < 4 ? sw + 1 : sw * 3 / 2) {
                x.splits = int32_t(sx);
                w.splits = int32_t(sw);
                x.units = int32_t(tiles[0] * sx);
                w.units = int32_t(tiles[1] * sw);
                // partial sums lie by unit, of both products where either has slices
                if ((sx > 1 || sw > 1) && int64_t(sw > 1 ? x.units + w.units : x.units) > room)
                    continue;
                s.workers = int(std::min<int64_t>(x.units + w.units, workers));
                int64_t cycles = pair_cycles(s.prod, s.workers, g == 2 ? 1024 : 740, &s.early);
                for (int i = 0; i < 2; ++i)
                    if (s.prod[i].splits > 1)
                        cycles += 3000 + s.prod[i].units * tile * tile * 4 / 1250;
                if (best.workers == 0 || cycles < best_cycles) {
                    best_cycles = cycles;
                    best = s;
                }
                if (tiles[1] == 0)
                    break;
            }
    }
    for (PairProduct& d : best.prod)
        if (d.units > 0)
            for (d.join_share = 8; d.join_share > 1 && (d.join_share > d.splits ||
                                                        d.units / d.splits * best.cg * best.cg * 16 * d.join_share > 2048);)
                d.join_share /= 2;
    return best;
}

// The gated layer's forward product in tiles of 256 rows of X x 128 of each weight on
// CTA pairs.
struct GatedPlan {
    bool lanes;
    LanesPlan l;
    int64_t num_r, num_c;
    int workers;
};

GatedPlan plan_gated(int num_sms, int max_pairs, int64_t M, int64_t N, int64_t K, const bwgemm_plan_options_t* opts,
                     uint64_t workspace_bytes)
{
    GatedPlan g = {};
    g.l = plan_lanes(kLanesGated, num_sms, max_pairs, M, N, K, opts, workspace_bytes);
    g.num_r = (M + 255) / 256;
    g.num_c = (N + 127) / 128;
    const int pairs = capped(max_pairs, 2, opts);
    g.lanes = true;
    if (pairs < 1 || g.num_r * g.num_c >= (1ll << 31))
        return g;
    g.workers = int(std::min<int64_t>(g.num_r * g.num_c, pairs));
    // measured, lanes against pairs: 64 x 28672 x 8192 147 and 158 us, 128 x 28672 x 8192 165 and 159,
    // 64 x 10240 x 8192 72 and 93, 100 x 10240 x 8192 98 and 94, 100 x 4096 x 4096 25.1 and 24.5, 200 x
    // 4096 x 4096 32 and 24, 200 x 2048 x 8192 38 and 42, 333 x 1000 x 5005 27 and 29
    const double waves = double((g.num_r * g.num_c + pairs - 1) / pairs), t = waves * double(blocks_of(K)) * 0.6;
    const double us = 5.0 + std::max(t, double(N) * double(K) * 4 / 6.5e6) + 0.1 * t;
    g.lanes = g.l.workers > 0 && g.l.us < us;
    return g;
}

// Whether the kernel for few rows takes the product.  Measured in us, it against tiles: integers
// 8 x 8192 x 8192 15.3 and 16.6, 8 x 28672 x 8192 44 and 40, 3 x 28672 x 8192 39.5 and 38.8, 16 x 4096 x
// 4096 8.8 and 10.5, 16 x 5120 x 5120 14.7 and 11.5; gated 2 x 28672 x 8192 135.7 and 140.8, 2 x 8192 x
// 8192 43.0 and 42.5, 16 x 4096 x 4096 15.2 and 16.6, 4 x 5120 x 5120 24.9 and 20.0.
bool takes_few_rows(int mode, int64_t M, int64_t N, int64_t K)
{
    if (M > kFewMost)
        return false;
    const double weights = double(N) * double(K);
    if (mode == kLanesInt8)
        return K <= kFewIntegerK && (M <= 2 || weights <= (M <= 8 ? 100e6 : 20e6));
    return M <= 2 || weights <= 20e6;
}

// Its warps per CTA: eight, so that many CTAs share an SM; more where there are too few of
// them and K is deep (us with 8, 16 and 32 warps, one row: integers 512 x 28672 23.5, 14.3, 10.8,
// 2048 x 4096 5.2, 4.4, 4.5, 1024 x 1024 1.8, 2.0, 2.3, 8192 x 8192 14.4, 16.8, 20.5; gated
// 512 x 8192 12.3, 7.5, 6.3, 4096 x 4096 12.7, 14.2, 17.5).
int few_warps(int kind, int64_t N, int64_t row_bytes)
{
    const int64_t ctas = (N + few_rows(kind) - 1) / few_rows(kind), blocks = row_bytes / 128;
    return ctas <= 64 && blocks >= 64 ? 32 : ctas <= 256 && blocks >= 32 ? 16 : 8;
}

int pairs_of(bwgemm_plan_t plan) { return plan->max_active[find_variant(2, 256, false, 1)]; }

bool dtype16(bwgemm_dtype_t dtype) { return dtype == BWGEMM_BF16 || dtype == BWGEMM_FP16; }

bool known(bwgemm_activation_t a) { return a == BWGEMM_SILU || a == BWGEMM_GELU || a == BWGEMM_GELU_TANH; }

bool fits(int64_t n) { return n <= (1ll << 31) - 256; }

constexpr int64_t kMostElements = 1ll << 56;  // of a workspace's matrix: its bytes stay far inside 64 bits

void take_lanes(LanesParams* p, const LanesPlan& s, bwgemm_plan_t plan, int64_t M, int64_t N, int64_t K)
{
    p->lrows = int32_t(N);
    p->crows = int32_t(M);
    p->K = int32_t(K);
    p->num_kb = int32_t(blocks_of(K));
    p->l_rows = s.l_rows / kLanesVariants[s.variant].cg;
    p->num_l = s.num_l;
    p->num_c = s.num_c;
    p->raster_group = std::max(1, std::min(s.raster, s.num_l));
    p->dp_tiles = s.dp_tiles;
    p->sk_tiles = s.sk_tiles;
    p->sk_iters = s.sk_iters;
    p->timeout_ns = limit_ns(plan);
    p->status = plan->d_status;
    p->counters = reinterpret_cast<uint32_t*>(plan->d_workspace);
    p->partials = reinterpret_cast<float*>(plan->d_workspace + kCounterRegionBytes);
    p->stall_kblock = plan->opts.stall_kblock;
}

bwgemm_status_t zero(void* data, int64_t ld, int64_t rows, int64_t cols, int size, cudaStream_t s)
{
    if (rows == 0 || cols == 0)
        return BWGEMM_OK;
    return cudaMemset2DAsync(data, size_t(ld) * size, 0, size_t(cols) * size, size_t(rows), s) == cudaSuccess
               ? BWGEMM_OK
               : BWGEMM_ERR_CUDA;
}

}  // namespace

extern "C" {

bwgemm_status_t bwgemm_gated(bwgemm_plan_t plan, const bwgemm_matrix_t* X, const bwgemm_matrix_t* Wg,
                             const bwgemm_matrix_t* Wu, const bwgemm_matrix_t* H, const bwgemm_matrix_t* G,
                             const bwgemm_matrix_t* U, int64_t M, int64_t N, int64_t K, bwgemm_dtype_t dtype,
                             bwgemm_activation_t activation, void* stream)
{
    if (!plan || M < 0 || N < 0 || K < 0 || !dtype16(dtype) || !known(activation) || present(G) != present(U))
        return BWGEMM_ERR_INVALID_ARG;
    if (!fits(M) || !fits(N) || !fits(K))
        return BWGEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0)
        return BWGEMM_OK;
    bwgemm_status_t st;
    const bool keep = present(G);
    const bwgemm_matrix_t* out[3] = {H, keep ? G : nullptr, keep ? U : nullptr};
    for (int i = 0; i < (keep ? 3 : 1); ++i)
        if ((st = check_matrix(out[i], M, N)) != BWGEMM_OK)
            return st;
    if (K > 0 && ((st = check_matrix(X, M, K)) != BWGEMM_OK || (st = check_matrix(Wg, N, K)) != BWGEMM_OK ||
                  (st = check_matrix(Wu, N, K)) != BWGEMM_OK))
        return st;
    DeviceGuard guard(plan->device);
    if (!guard.ok)
        return BWGEMM_ERR_CUDA;
    if ((st = check_resident({H->data, keep ? G->data : nullptr, keep ? U->data : nullptr, K ? X->data : nullptr,
                              K ? Wg->data : nullptr, K ? Wu->data : nullptr}, plan->device)) != BWGEMM_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) {  // empty sums: act(0) * 0
        for (int i = 0; i < (keep ? 3 : 1); ++i)
            if ((st = zero(out[i]->data, out[i]->ld, M, N, 2, s)) != BWGEMM_OK)
                return st;
        return BWGEMM_OK;
    }
    const bool pdl = plan->opts.pdl_off == 0;
    if (takes_few_rows(kLanesGated, M, N, K)) {
        FewRowsParams p = {};
        p.w[0] = static_cast<const uint8_t*>(Wg->data);
        p.w[1] = static_cast<const uint8_t*>(Wu->data);
        p.ldw[0] = 2 * Wg->ld;
        p.ldw[1] = 2 * Wu->ld;
        p.x = static_cast<const uint8_t*>(X->data);
        p.ldx = 2 * X->ld;
        p.row_bytes = 2 * K;
        p.M = int32_t(M);
        p.N = int32_t(N);
        p.out_type = dtype;
        p.activation = activation;
        for (int i = 0; i < (keep ? 3 : 1); ++i) {
            p.out[i] = out[i]->data;
            p.ldo[i] = out[i]->ld;
        }
        if (launch_few_rows(dtype == BWGEMM_BF16 ? kFewBf16 : kFewFp16, few_warps(kFewBf16, N, p.row_bytes), p, s, pdl) != cudaSuccess)
            return BWGEMM_ERR_CUDA;
        plan->launches += 1;
        return BWGEMM_OK;
    }
    const GatedPlan sel = plan_gated(plan->num_sms, pairs_of(plan), M, N, K, &plan->opts, plan->workspace_bytes);
    if (sel.lanes) {
        if (sel.l.workers == 0)
            return BWGEMM_ERR_UNSUPPORTED;
        const LanesVariant& v = kLanesVariants[sel.l.variant];
        LanesParams p = {};
        take_lanes(&p, sel.l, plan, M, N, K);
        p.l_chunks = p.c_chunks = int32_t(K / 64);
        p.dtype = p.out_type = dtype;
        p.activation = activation;
        for (int i = 0; i < (keep ? 3 : 1); ++i) {
            p.out[i] = out[i]->data;
            p.ldo[i] = out[i]->ld;
        }
        LanesMaps maps;
        if ((st = encode_operand16(&maps.w, &maps.w3, Wg->data, Wg->ld, dtype, N, K, uint32_t(p.l_rows))) != BWGEMM_OK ||
            (st = encode_operand16(&maps.w2, &maps.w23, Wu->data, Wu->ld, dtype, N, K, uint32_t(p.l_rows))) != BWGEMM_OK ||
            (st = encode_operand16(&maps.x, &maps.x3, X->data, X->ld, dtype, M, K, uint32_t(v.bn))) != BWGEMM_OK)
            return st;
        if (launch_lanes(sel.l.variant, maps, p, sel.l.workers, s, pdl) != cudaSuccess)
            return BWGEMM_ERR_CUDA;
        plan->launches += 1;
        return BWGEMM_OK;
    }
    PairParams p = {};
    p.prod[0] = {int32_t(M), int32_t(N), int32_t(blocks_of(K)), 1, int32_t(sel.num_r), int32_t(sel.num_c), 1,
                 int32_t(sel.num_r * sel.num_c), 1};
    p.steps_k = p.prod[0].steps;
    p.chunks_a = p.chunks_b = int32_t(K / 64);
    p.dtype = dtype;
    p.activation = activation;
    p.timeout_ns = limit_ns(plan);
    p.status = plan->d_status;
    p.stall_kblock = plan->opts.stall_kblock;
    PairMaps maps;
    if ((st = encode_operand16(&maps.a[0], &maps.a3[0], X->data, X->ld, dtype, M, K, 128)) != BWGEMM_OK ||
        (st = encode_operand16(&maps.b[0], &maps.b3[0], Wg->data, Wg->ld, dtype, N, K, 128)) != BWGEMM_OK ||
        (st = encode_operand16(&maps.b[1], &maps.b3[1], Wu->data, Wu->ld, dtype, N, K, 128)) != BWGEMM_OK)
        return st;
    maps.a[1] = maps.a[0];
    maps.a3[1] = maps.a3[0];
    maps.b[2] = maps.b[1];
    maps.b3[2] = maps.b3[1];
    for (int i = 0; i < 3; ++i) {
        if (!out[i]) {
            maps.out[i] = maps.out[0];
            continue;
        }
        if ((st = encode_result16(&maps.out[i], *out[i], dtype, M, N)) != BWGEMM_OK)
            return st;
        p.out[i] = static_cast<uint16_t*>(out[i]->data);
        p.ldo[i] = out[i]->ld;
    }
    if (launch_pair(kPairGated, 2, maps, p, 2 * sel.workers, s, pdl) != cudaSuccess)
        return BWGEMM_ERR_CUDA;
    plan->launches += 1;
    return BWGEMM_OK;
}

bwgemm_status_t bwgemm_gated_backward_workspace(int64_t M, int64_t N, uint64_t* bytes)
{
    if (!bytes)
        return BWGEMM_ERR_INVALID_ARG;
    *bytes = 0;
    if (M < 0 || N < 0)
        return BWGEMM_ERR_INVALID_ARG;
    if (!fits(M) || !fits(N) || M > kMostElements / round_up(std::max<int64_t>(N, 1), 8))
        return BWGEMM_ERR_UNSUPPORTED;
    *bytes = 2 * uint64_t(round_up(M * round_up(N, 8) * 2, 256));
    return BWGEMM_OK;
}

bwgemm_status_t bwgemm_gated_backward(bwgemm_plan_t plan, const bwgemm_matrix_t* dH, const bwgemm_matrix_t* G,
                                      const bwgemm_matrix_t* U, const bwgemm_matrix_t* X, const bwgemm_matrix_t* Wg,
                                      const bwgemm_matrix_t* Wu, const bwgemm_matrix_t* dX, const bwgemm_matrix_t* dWg,
                                      const bwgemm_matrix_t* dWu, int64_t M, int64_t N, int64_t K, bwgemm_dtype_t dtype,
                                      bwgemm_activation_t activation, void* workspace, uint64_t workspace_bytes,
                                      void* stream)
{
    if (!plan || M < 0 || N < 0 || K < 0 || !dtype16(dtype) || !known(activation))
        return BWGEMM_ERR_INVALID_ARG;
    if (!fits(M) || !fits(N) || !fits(K))
        return BWGEMM_ERR_UNSUPPORTED;
    // results without elements need no memory
    const bool of_x = present(dX) && M > 0 && K > 0, of_w = (present(dWg) || present(dWu)) && N > 0 && K > 0;
    if (!of_x && !of_w)
        return BWGEMM_OK;
    bwgemm_status_t st;
    if (of_x && (st = check_matrix(dX, M, K)) != BWGEMM_OK)
        return st;
    if (of_w && ((st = check_matrix(dWg, N, K)) != BWGEMM_OK || (st = check_matrix(dWu, N, K)) != BWGEMM_OK))
        return st;
    const bool sums = M > 0 && N > 0;  // else empty ones
    uint64_t need = 0;
    if (sums) {
        for (const bwgemm_matrix_t* x : {dH, G, U})
            if ((st = check_matrix(x, M, N)) != BWGEMM_OK)
                return st;
        if (of_x && ((st = check_matrix(Wg, N, K)) != BWGEMM_OK || (st = check_matrix(Wu, N, K)) != BWGEMM_OK))
            return st;
        if (of_w && (st = check_matrix(X, M, K)) != BWGEMM_OK)
            return st;
        if ((st = bwgemm_gated_backward_workspace(M, N, &need)) != BWGEMM_OK)
            return st;
        if (workspace_bytes < need || !workspace)
            return BWGEMM_ERR_WORKSPACE;
        if (!aligned(workspace, 256))
            return BWGEMM_ERR_ALIGNMENT;
    }
    DeviceGuard guard(plan->device);
    if (!guard.ok)
        return BWGEMM_ERR_CUDA;
    auto at = [](bool read, const bwgemm_matrix_t* x) { return read ? x->data : nullptr; };
    if ((st = check_resident({at(of_x, dX), at(of_w, dWg), at(of_w, dWu), at(sums, dH), at(sums, G), at(sums, U),
                              at(sums && of_w, X), at(sums && of_x, Wg), at(sums && of_x, Wu), sums ? workspace : nullptr},
                             plan->device)) != BWGEMM_OK)
        return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!sums) {
        if (of_x && (st = zero(dX->data, dX->ld, M, K, 2, s)) != BWGEMM_OK)
            return st;
        if (of_w && ((st = zero(dWg->data, dWg->ld, N, K, 2, s)) != BWGEMM_OK ||
                     (st = zero(dWu->data, dWu->ld, N, K, 2, s)) != BWGEMM_OK))
            return st;
        return BWGEMM_OK;
    }
    const bool pdl = plan->opts.pdl_off == 0;
    const int64_t ldd = round_up(N, 8);
    uint16_t* const d[2] = {static_cast<uint16_t*>(workspace),
                            reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + need / 2)};
    // the division before the first launch: a size without one launches nothing
    const PairPlan sel = plan_backward(M, N, K, of_x, of_w, capped(plan->num_sms, 1, &plan->opts),
                                       capped(pairs_of(plan), 2, &plan->opts), plan->workspace_bytes);
    if (sel.workers == 0)
        return BWGEMM_ERR_UNSUPPORTED;

    GateGradParams gg = {};
    gg.dh = static_cast<const uint16_t*>(dH->data);
    gg.g = static_cast<const uint16_t*>(G->data);
    gg.u = static_cast<const uint16_t*>(U->data);
    gg.lddh = dH->ld;
    gg.ldg = G->ld;
    gg.ldu = U->ld;
    gg.dg = d[0];
    gg.du = d[1];
    gg.ldd = ldd;
    gg.rows = M;
    gg.cols = N;
    gg.dtype = dtype;
    gg.activation = activation;
    PairParams p = {};
    p.prod[0] = sel.prod[0];
    p.prod[1] = sel.prod[1];
    p.early = sel.early;
    p.steps_k = int32_t(blocks_of(N));
    p.chunks_a = int32_t(N / 64);
    p.chunks_b = int32_t(K / 64);
    p.dtype = dtype;
    p.partials = reinterpret_cast<float*>(plan->d_workspace + kCounterRegionBytes);
    p.timeout_ns = limit_ns(plan);
    p.status = plan->d_status;
    p.stall_kblock = plan->opts.stall_kblock;
    // dG and dU: rows of tokens, K-major for dX, stored K x rows for the weights.  A pair's second
    // CTA reads past rows that end in the first one's half of a tile.
    PairMaps maps;
    for (int i = 0; i < 2; ++i)
        if ((st = encode_operand16(&maps.a[i], &maps.a3[i], d[i], ldd, dtype, M, N, 128, pair_tile(sel.cg))) != BWGEMM_OK)
            return st;
    const bwgemm_matrix_t* const b[3] = {of_x ? Wg : nullptr, of_x ? Wu : nullptr, of_w ? X : nullptr};
    const bwgemm_matrix_t* const out[3] = {of_x ? dX : nullptr, of_w ? dWg : nullptr, of_w ? dWu : nullptr};
    for (int i = 0; i < 3; ++i) {
        maps.b[i] = maps.b3[i] = maps.out[i] = maps.a[0];  // where there is none, none is read
        if (b[i] && (st = encode_operand16(&maps.b[i], &maps.b3[i], b[i]->data, b[i]->ld, dtype, i < 2 ? N : M, K, 128,
                                           pair_tile(sel.cg))) != BWGEMM_OK)
            return st;
        if (!out[i])
            continue;
        if ((st = encode_result16(&maps.out[i], *out[i], dtype, i ? N : M, K)) != BWGEMM_OK)
            return st;
        p.out[i] = static_cast<uint16_t*>(out[i]->data);
        p.ldo[i] = out[i]->ld;
    }
    if (launch_gate_grad(gg, s, pdl) != cudaSuccess)
        return BWGEMM_ERR_CUDA;
    plan->launches += 1;
    if (launch_pair(kPairBackward, sel.cg, maps, p, sel.workers * sel.cg, s, pdl) != cudaSuccess)
        return BWGEMM_ERR_CUDA;
    plan->launches += 1;
    for (const PairProduct& q : sel.prod)
        plan->launches += q.units > 0 && q.splits > 1 ? 1 : 0;
    return BWGEMM_OK;
}

bwgemm_status_t bwgemm_quantize_integer(bwgemm_plan_t plan, const void* X, bwgemm_dtype_t dtype, int64_t rows,
                                     int64_t cols, int64_t ldx, int8_t* q, int64_t ldq, float* scales, void* stream)
{
    if (!plan || (!dtype16(dtype) && dtype != BWGEMM_FP32) || rows < 0 || cols < 0)
        return BWGEMM_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0)
        return BWGEMM_OK;
    if (!X || !q || !scales || ldx < cols || ldq < cols)
        return BWGEMM_ERR_INVALID_ARG;
    if (!extent_ok(rows, cols, ldx) || !extent_ok(rows, cols, ldq))
        return BWGEMM_ERR_UNSUPPORTED;
    if (!aligned(X, 16) || ldx * element_size(dtype) % 16 != 0 || !aligned(q, 16) || ldq % 16 != 0 || !aligned(scales, 4))
        return BWGEMM_ERR_ALIGNMENT;
    DeviceGuard guard(plan->device);
    if (!guard.ok)
        return BWGEMM_ERR_CUDA;
    const bwgemm_status_t st = check_resident({X, q, scales}, plan->device);
    if (st != BWGEMM_OK)
        return st;
    const RowsInt8Params p = {X, ldx, rows, cols, q, ldq, scales};
    if (launch_quantize_int8(dtype, p, static_cast<cudaStream_t>(stream), plan->opts.pdl_off == 0) != cudaSuccess)
        return BWGEMM_ERR_CUDA;
    plan->launches += 1;
    return BWGEMM_OK;
}

bwgemm_status_t bwgemm_run_integer_workspace(int64_t M, int64_t N, int64_t K, uint64_t* bytes)
{
    if (!bytes)
        return BWGEMM_ERR_INVALID_ARG;
    *bytes = 0;
    if (M < 0 || N < 0 || K < 0)
        return BWGEMM_ERR_INVALID_ARG;
    if (!fits(M) || !fits(N) || !fits(K) || M > kMostElements / round_up(std::max<int64_t>(K, 1), 128))
        return BWGEMM_ERR_UNSUPPORTED;
    // A as fp16, or B
    if (M > 0 && N > 0 && K > 0 && !takes_few_rows(kLanesInt8, M, N, K) && !widens_always(M, N, K))
        *bytes = uint64_t(round_up((takes_turned(M, N, K) ? N : M) * round_up(K, 128) * 2, 256));
    return BWGEMM_OK;
}

bwgemm_status_t bwgemm_run_integer(bwgemm_plan_t plan, const int8_t* A, const float* scale_a, const int8_t* B,
                                const float* scale_b, void* C, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb,
                                int64_t ldc, bwgemm_dtype_t out, void* workspace, uint64_t workspace_bytes, void* stream)
{
    if (!plan || M < 0 || N < 0 || K < 0 || (!dtype16(out) && out != BWGEMM_FP32))
        return BWGEMM_ERR_INVALID_ARG;
    uint64_t need = 0;
    bwgemm_status_t st = bwgemm_run_integer_workspace(M, N, K, &need);
    if (st != BWGEMM_OK || M == 0 || N == 0)
        return st;
    const int es = element_size(out);
    if (!C || ldc < N || (K > 0 && (!A || !B || !scale_a || !scale_b || lda < K || ldb < K)))
        return BWGEMM_ERR_INVALID_ARG;
    if (!extent_ok(M, N, ldc) || (K > 0 && (!extent_ok(M, K, lda) || !extent_ok(N, K, ldb))))
        return BWGEMM_ERR_UNSUPPORTED;
    if (!aligned(C, 16) || ldc * es % 16 != 0 ||
        (K > 0 && (!aligned(A, 16) || lda % 16 != 0 || !aligned(B, 16) || ldb % 16 != 0 || !aligned(scale_a, 4) ||
                   !aligned(scale_b, 4) || (need > 0 && !aligned(workspace, 256)))))
        return BWGEMM_ERR_ALIGNMENT;
    if (workspace_bytes < need || (need > 0 && !workspace))
        return BWGEMM_ERR_WORKSPACE;
    DeviceGuard guard(plan->device);
    if (!guard.ok)
        return BWGEMM_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) {
        if ((st = check_resident({C}, plan->device)) != BWGEMM_OK)
            return st;
        return zero(C, ldc, M, N, es, s);
    }
    if ((st = check_resident({A, scale_a, B, scale_b, C, need ? workspace : nullptr}, plan->device)) != BWGEMM_OK)
        return st;
    const bool pdl = plan->opts.pdl_off == 0;
    if (takes_few_rows(kLanesInt8, M, N, K)) {
        FewRowsParams p = {};
        p.w[0] = reinterpret_cast<const uint8_t*>(B);
        p.ldw[0] = ldb;
        p.x = reinterpret_cast<const uint8_t*>(A);
        p.ldx = lda;
        p.row_bytes = K;
        p.M = int32_t(M);
        p.N = int32_t(N);
        p.ls = scale_b;
        p.cs = scale_a;
        p.out_type = out;
        p.out[0] = C;
        p.ldo[0] = ldc;
        if (launch_few_rows(kFewInt8, few_warps(kFewInt8, N, p.row_bytes), p, s, pdl) != cudaSuccess)
            return BWGEMM_ERR_CUDA;
        plan->launches += 1;
        return BWGEMM_OK;
    }
    const bool turned = takes_turned(M, N, K);
    if (turned) {  // from here on "A" is the operand in the columns
        std::swap(M, N);
        std::swap(A, B);
        std::swap(lda, ldb);
        std::swap(scale_a, scale_b);
    }
    const LanesPlan sel = plan_lanes(kLanesInt8, plan->num_sms, pairs_of(plan), M, N, K, &plan->opts, plan->workspace_bytes);
    if (sel.workers == 0)
        return BWGEMM_ERR_UNSUPPORTED;
    const LanesVariant& v = kLanesVariants[sel.variant];
    const int64_t ldy = round_up(K, 128);
    LanesParams p = {};
    take_lanes(&p, sel, plan, M, N, K);
    p.c_chunks = int32_t(ldy / 64);
    p.turned = turned;
    p.ls = scale_b;
    p.cs = scale_a;
    p.dtype = BWGEMM_FP16;
    p.out_type = out;
    p.out[0] = C;
    p.ldo[0] = ldc;
    LanesMaps maps;
    p.l_chunks = int32_t(K / 128);
    if ((st = encode_bytes(&maps.w, &maps.w3, B, ldb, N, K, uint32_t(p.l_rows), CU_TENSOR_MAP_SWIZZLE_128B)) != BWGEMM_OK)
        return st;
    maps.w2 = maps.w23 = maps.w;
    if (v.widens) {
        if ((st = encode_bytes(&maps.x, &maps.x3, A, lda, M, K, uint32_t(v.bn), CU_TENSOR_MAP_SWIZZLE_NONE)) != BWGEMM_OK)
            return st;
    } else {
        if ((st = encode_operand16(&maps.x, &maps.x3, workspace, ldy, BWGEMM_FP16, M, ldy, uint32_t(v.bn / v.cg))) !=
            BWGEMM_OK)
            return st;
        const WidenParams wp = {A, lda, int32_t(M), int32_t(K), static_cast<uint16_t*>(workspace), ldy};
        if (launch_widen(wp, s, pdl) != cudaSuccess)
            return BWGEMM_ERR_CUDA;
        plan->launches += 1;
    }
    if (launch_lanes(sel.variant, maps, p, sel.workers * v.cg, s, pdl) != cudaSuccess)
        return BWGEMM_ERR_CUDA;
    plan->launches += 1;
    return BWGEMM_OK;
}

bwgemm_status_t bwgemm_select_gated(int32_t num_sms, int32_t max_pairs, int64_t M, int64_t N, int64_t K,
                                    const bwgemm_plan_options_t* opts, bwgemm_lanes_config_t* out)
{
    if (!out || num_sms < 1 || max_pairs < 0 || M < 1 || N < 1 || K < 1)
        return BWGEMM_ERR_INVALID_ARG;
    if (!fits(M) || !fits(N) || !fits(K))
        return BWGEMM_ERR_UNSUPPORTED;
    if (takes_few_rows(kLanesGated, M, N, K)) {
        *out = {2, 8, int32_t(M > 8 ? 16 : 8), 0, 0, 0};
        return BWGEMM_OK;
    }
    const GatedPlan g = plan_gated(num_sms, max_pairs ? max_pairs : num_sms / 2, M, N, K, opts, workspace_of(opts));
    if (g.lanes && g.l.workers == 0)
        return BWGEMM_ERR_UNSUPPORTED;
    if (g.lanes)
        *out = {1, g.l.l_rows, kLanesVariants[g.l.variant].bn, g.l.dp_tiles, g.l.sk_tiles, g.l.workers};
    else
        *out = {0, 128, 256, int32_t(g.num_r * g.num_c), 0, g.workers};
    return BWGEMM_OK;
}

bwgemm_status_t bwgemm_select_integer(int32_t num_sms, int32_t max_pairs, int64_t M, int64_t N, int64_t K,
                                   const bwgemm_plan_options_t* opts, bwgemm_lanes_config_t* out)
{
    if (!out || num_sms < 1 || max_pairs < 0 || M < 1 || N < 1 || K < 1)
        return BWGEMM_ERR_INVALID_ARG;
    if (!fits(M) || !fits(N) || !fits(K))
        return BWGEMM_ERR_UNSUPPORTED;
    if (takes_few_rows(kLanesInt8, M, N, K)) {
        *out = {2, 16, int32_t(M > 8 ? 16 : 8), 0, 0, 0};
        return BWGEMM_OK;
    }
    const bool turned = takes_turned(M, N, K);
    const LanesPlan s = plan_lanes(kLanesInt8, num_sms, max_pairs ? max_pairs : num_sms / 2, turned ? N : M, turned ? M : N, K,
                                   opts, workspace_of(opts));
    if (s.workers == 0)
        return BWGEMM_ERR_UNSUPPORTED;
    *out = {turned ? 3 : 1, s.l_rows, kLanesVariants[s.variant].bn, s.dp_tiles, s.sk_tiles, s.workers};
    return BWGEMM_OK;
}

bwgemm_status_t bwgemm_select_gated_backward(int32_t num_sms, int32_t max_pairs, int64_t M, int64_t N, int64_t K,
                                             const bwgemm_plan_options_t* opts, bwgemm_ortho_config_t out[2])
{
    if (!out || num_sms < 1 || max_pairs < 0 || M < 1 || N < 1 || K < 1)
        return BWGEMM_ERR_INVALID_ARG;
    if (!fits(M) || !fits(N) || !fits(K))
        return BWGEMM_ERR_UNSUPPORTED;
    const PairPlan s = plan_backward(M, N, K, true, true, capped(num_sms, 1, opts),
                                     capped(max_pairs ? max_pairs : num_sms / 2, 2, opts), workspace_of(opts));
    if (s.workers == 0)
        return BWGEMM_ERR_UNSUPPORTED;
    for (int i = 0; i < 2; ++i)
        out[i] = {pair_tile(s.cg), s.prod[i].splits, s.prod[i].units / s.prod[i].splits, s.workers};
    return BWGEMM_OK;
}

}  // extern "C"
