// feed_forward.h -- launch descriptions of the gated feed-forward layer and of
// the 8-bit integer product: shared by their kernels' translation units and
// feed_forward.cpp, which checks the arguments and fills them in.
#pragma once

#include "operators.h"

namespace bwgemm {

// ------------------------------------------- products in square tiles
// What a launch computes from 16-bit operands; `a` and `b` are the sides whose rows
// (columns, where stored transposed) are D's rows and columns.
enum : int {
    kPairGated = 0,    // H = act(X Wg^T) * (X Wu^T):  a = X, b = Wg and Wu
    kPairBackward = 1  // dX = dG Wg + dU Wu:          a = dG then dU, b = Wg then Wu, stored K x columns
                       // dWg = dG^T X, dWu = dU^T X:  a = dG or dU, b = X, both stored K x rows
};

// An operand in boxes of 64 elements x 128 rows, and in boxes of two whole 64-element
// chunks of those rows.
struct PairMaps {
    CUtensorMap a[2], a3[2];     // X | dG, dU
    CUtensorMap b[3], b3[3];     // Wg, Wu | Wg, Wu, X
    CUtensorMap out[3];          // H, G, U | dX, dWg, dWu in boxes of 64 columns x 32 rows
};

// One of a launch's products: H | dX, and dWg with dWu.
struct PairProduct {
    int32_t rows, cols;          // of one result
    int32_t steps;               // of 128 of K, of all terms
    int32_t results;             // results stacked along the tile rows (dWg, dWu: 2)
    int32_t num_r, num_c;        // tiles of one result
    int32_t splits;              // slices of K per tile (1: whole)
    int32_t units;               // tiles, or slices of them: 0 where it is not wanted
    int32_t join_share;          // warps that add the slices of one piece: 1, 2, 4 or 8
};

struct PairParams {
    PairProduct prod[2];
    int32_t early;               // units of the second product for who has fewer of the first's
    int32_t steps_k;             // of one term of dX: ceil(N / 128)
    int32_t chunks_a, chunks_b;  // whole 64-element chunks of the operands' rows (0: no a3 / b3)
    float* partials;             // the slices' fp32 sums, by unit
    int32_t dtype;
    int32_t activation;          // kPairGated
    uint16_t* out[3];            // results; kPairGated: G and U null where they are not kept
    int64_t ldo[3];
    uint64_t timeout_ns;
    uint32_t* status;
    int32_t stall_kblock;        // test hook, as in GemmParams
};

constexpr int pair_tile(int cg) { return 128 * cg; }
// The products, then for those in slices the kernel that adds them.
cudaError_t launch_pair(int form, int cg, const PairMaps& maps, const PairParams& p, int grid, cudaStream_t stream, bool pdl);

// ------------------------------------------------ gradients of G and U
struct GateGradParams {
    const uint16_t *dh, *g, *u;  // rows x cols, 16-byte rows
    uint16_t *dg, *du;
    int64_t lddh, ldg, ldu, ldd; // ldd: of both results
    int64_t rows, cols;
    int32_t dtype, activation;
};
cudaError_t launch_gate_grad(const GateGradParams& p, cudaStream_t stream, bool pdl);

// ------------------------------- products with the weights in the lanes
// For few rows of X, and for 8-bit integers at any size: the weights' rows are the
// MMA's M, X's rows its N, so the accumulator holds the result transposed.
enum : int {
    kLanesGated = 0,  // 16-bit weights Wg and Wu from shared memory, M = 64 each
    kLanesInt8 = 1    // 8-bit integer weights as fp16 through TMEM, M = 128 (256 over a CTA pair)
};

struct LanesParams {
    int32_t lrows, crows, K;     // rows of the weights and of X
    int32_t num_kb;              // ceil(K / 128)
    int32_t l_rows;              // weight rows per tile: a multiple of 8, at most 64, 128 or (pair) 256
    int32_t l_chunks, c_chunks;  // whole chunks of the weights' and X's rows: of 64 elements, of 128 integers
    int32_t num_l, num_c;        // tiles along the weights' rows and X's
    int32_t raster_group;
    int32_t dp_tiles, sk_tiles;  // as in ScaledParams
    int32_t sk_iters;
    const float* ls;             // kLanesInt8: a scale per weight row,
    const float* cs;             // and per row of X
    int32_t dtype;               // of 16-bit operands (kLanesInt8: fp16)
    int32_t out_type;
    int32_t activation;
    void* out[3];                // C; kLanesGated: H, G, U (G null: not kept)
    int64_t ldo[3];
    int32_t turned;              // kLanesInt8: the lanes are A's rows, "X" is B: lanes are rows of C
    uint64_t timeout_ns;
    uint32_t* status;
    float* partials;
    uint32_t* counters;
    int32_t stall_kblock;
};

struct LanesVariant {
    int mode, cg, bn;
    bool widens = false;  // takes X as 8-bit integers (else launch_widen's fp16)
};
constexpr LanesVariant kLanesVariants[] = {
    {kLanesGated, 1, 16},      {kLanesGated, 1, 32},      {kLanesGated, 1, 64}, {kLanesGated, 1, 128},
    {kLanesInt8, 1, 16, true}, {kLanesInt8, 1, 32, true}, {kLanesInt8, 1, 32},  {kLanesInt8, 1, 64},
    {kLanesInt8, 1, 128},      {kLanesInt8, 2, 256},
};
constexpr int kNumLanesVariants = int(sizeof(kLanesVariants) / sizeof(kLanesVariants[0]));

// w / w2: the weights (gated: of G and U) in boxes of a chunk x l_rows; w3, w23: of two whole
// chunks; x, x3: X so, in bn / cg rows.
struct LanesMaps {
    CUtensorMap w, w2, w3, w23, x, x3;
};
cudaError_t launch_lanes(int idx, const LanesMaps& maps, const LanesParams& p, int grid, cudaStream_t stream, bool pdl);
// Epilogue warps of a variant, each with an arrival counter per tile and CTA.
constexpr int lanes_epi_warps(int bn) { return bn >= 128 ? 8 : 4; }
// fp32 sums of a CTA's partial tile.
constexpr int lanes_partial_floats(int mode, int bn) { return mode == kLanesGated ? 2 * 128 * bn : 128 * bn; }

// ------------------------------------------------ at most 16 rows of X
enum : int { kFewInt8 = 0, kFewBf16 = 1, kFewFp16 = 2 };

struct FewRowsParams {
    const uint8_t* w[2];         // 8-bit weights, or Wg and Wu; rows ldw bytes apart
    int64_t ldw[2];
    const uint8_t* x;
    int64_t ldx;
    int64_t row_bytes;           // K in bytes
    int32_t M, N;
    const float* ls;             // kFewInt8: a scale per weight row,
    const float* cs;             // and per row of X
    int32_t out_type, activation;
    void* out[3];                // as in LanesParams
    int64_t ldo[3];
};
constexpr int kFewMost = 16;
constexpr int64_t kFewIntegerK = 131071;  // 2^14 each, sums in 32 bits
// Columns of the result per CTA, whose 8, 16 or 32 warps divide K.
#ifdef __CUDACC__
__host__ __device__
#endif
constexpr int few_rows(int kind) { return kind == kFewInt8 ? 16 : 8; }
cudaError_t launch_few_rows(int kind, int warps, const FewRowsParams& p, cudaStream_t stream, bool pdl);

// ------------------------------------------------------- 8-bit integers
struct RowsInt8Params {
    const void* x;               // rows x cols, ldx elements apart
    int64_t ldx;
    int64_t rows, cols;
    int8_t* q;                   // ldq bytes apart
    int64_t ldq;
    float* scales;
};
cudaError_t launch_quantize_int8(int dtype, const RowsInt8Params& p, cudaStream_t stream, bool pdl);

// X of 8-bit integers as fp16, rows of `ldy` elements (zeros past the end).
struct WidenParams {
    const int8_t* x;
    int64_t ldx;
    int32_t rows, cols;
    uint16_t* y;
    int64_t ldy;
};
cudaError_t launch_widen(const WidenParams& p, cudaStream_t stream, bool pdl);

}  // namespace bwgemm
