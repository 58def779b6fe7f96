// operators.h -- launch descriptions of the operators beside the 16-bit GEMM:
// quantising to blocks of 128, the product of such matrices, and the
// orthogonalisation.  Shared by their kernels' translation units and
// operators.cpp, which checks the arguments and fills them in.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/bwgemm.h"

namespace bwgemm {

constexpr int kBlock = 128;  // elements of K, or rows, that share a scale

// A block whose largest magnitude is below this is scaled as if it held it:
// limit / amax then stays finite in fp32 and an all-zero block needs no case
// of its own.
constexpr float kSmallestAmax = 7.8886090522101181e-31f;  // 2^-100

// Allow `kernel` its dynamic shared memory on the current device, once per
// device (the call costs more than looking it up).  `done`: a bit per device,
// one word per kernel.
template <typename Kernel>
inline cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<uint64_t>& done)
{
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_relaxed) & bit)
        return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess)
        done.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

// ------------------------------------------------------------------ quantise
struct QuantizeParams {
    const void* x;       // rows x cols, ldx elements apart
    int64_t ldx;
    int64_t rows, cols;
    uint8_t* q;          // rows x cols in 8 bits, ldq bytes apart
    int64_t ldq;
    float* s;            // [column block][row or row block], lds apart
    int64_t lds;
    uint8_t* qt;         // cols x rows in 8 bits (or null), ldqt bytes apart
    int64_t ldqt;
    float* st;           // [row block][column or column block], ldst apart
    int64_t ldst;
    int32_t pow2;        // 1: scales rounded up to powers of two
};

// fp8: 0 = e4m3, 1 = e5m2; square: one scale per 128 x 128 instead of 1 x 128.
cudaError_t launch_quantize(int dtype, int fp8, bool square, const QuantizeParams& p, cudaStream_t stream, bool pdl);

// ------------------------------------------------------------ scaled product
// C[M x N] = sum over K blocks of sa * sb * (A block)(B block)^T.  The kernel
// sees a lane-side operand (the MMA's M: one TMEM lane per row) and a
// column-side operand (the MMA's N).  In order the lane side is A; swapped,
// for few rows of A, it is B and the accumulator holds C transposed.
struct ScaledParams {
    int32_t lrows, crows, K;      // rows of the lane-side and column-side operands
    int32_t num_kb;               // ceil(K / 128)
    int32_t chunks;               // whole 128-element K chunks (0: no 3-D views)
    int32_t l_rows;               // lane rows per tile (swapped form: a multiple of 8, at most 128)
    int32_t stages;               // of the ring (swapped form)
    int32_t num_l, num_c;         // blocks of lane rows and of columns
    int32_t raster_group;         // lane blocks walked before stepping along the columns
    int32_t dp_tiles, sk_tiles;   // tiles computed whole; tiles whose K iterations are spread over the workers
    int32_t sk_iters;             // sk_tiles * num_kb
    const float* ls;              // scale of lane row r, K block kb: ls[kb * ls_ld + (r >> ls_shift)]
    int64_t ls_ld;
    const float* cs;              // and of column c
    int64_t cs_ld;
    int32_t ls_shift, cs_shift;   // 0: a scale per row, 7: one per 128 rows
    void* c;
    int64_t ldc;
    int32_t out_type;             // bwgemm_dtype_t of C
    int32_t accumulate;           // 1: C += (fp32 only)
    uint32_t idesc;
    uint64_t timeout_ns;
    uint32_t* status;
    float* partials;              // fp32 partial tiles of stream-K pieces
    uint32_t* counters;           // K blocks arrived per (tile, CTA, warp); zero between calls
    int32_t stall_kblock;         // test hook, as in GemmParams
};

// Compiled forms: columns per tile (128 lane rows each), operands swapped, and
// whether the column side has a scale per column (the swapped forms always take
// one per column and read one per 128 through it).
struct ScaledVariant {
    int bn;
    bool swap, colvec;
};
constexpr ScaledVariant kScaledVariants[] = {
    {256, false, false}, {256, false, true}, {128, false, false}, {128, false, true},
    {64, true, true},    {32, true, true},   {16, true, true},
};
constexpr int kNumScaledVariants = int(sizeof(kScaledVariants) / sizeof(kScaledVariants[0]));
// K blocks per ring stage and TMA copy, and the ring: stages of kps * (l_rows +
// bn) rows of 128 bytes
constexpr int scaled_kps(int bn, bool swap) { return swap && bn <= 32 ? 4 : 2; }
constexpr int kScaledRingBytes = 192 * 1024;
constexpr int kScaledMaxStages = 10;
constexpr int scaled_stages(int bn, bool swap, int l_rows)
{
    const int n = kScaledRingBytes / (scaled_kps(bn, swap) * (l_rows + bn) * kBlock);
    return n < kScaledMaxStages ? n : kScaledMaxStages;
}

// l / c: the operands in boxes of 128 bytes x (128 | bn) rows; l3 / c3:
// their 3-D views of scaled_kps() K blocks; out: C in 64-byte x 32-row boxes
// (operands in order only).
cudaError_t launch_scaled(int idx, const CUtensorMap& l, const CUtensorMap& c, const CUtensorMap& l3,
                          const CUtensorMap& c3, const CUtensorMap& out, const ScaledParams& p, int grid,
                          cudaStream_t stream, bool pdl);

// The same product for at most kScaledFewRows rows of A (scaled_few_sm103.cu).
struct FewParams {
    const uint8_t* w;            // weights, N x K, ldw bytes apart
    const uint8_t* x;            // A, M x K
    int64_t ldw, ldx;
    const float* ws;             // scales as in ScaledParams
    const float* xs;
    int64_t ws_ld, xs_ld;
    int32_t ws_shift, xs_shift;
    int32_t M, N, K, num_kb;
    void* c;
    int64_t ldc;
    int32_t out_type, accumulate;
};
constexpr int kScaledFewRows = 16;
cudaError_t launch_scaled_few(int w_type, int x_type, const FewParams& p, cudaStream_t stream, bool pdl);

// -------------------------------------------------------- orthogonalisation
// One product of the iteration over a stack of matrices, fp16 operands:
//   D = alpha * A B^T + beta * E + diag * I
// A and B: `rows` / `cols` wide on their output side and K deep, each K-major
// or (a_mn / b_mn) MN-major, i.e. stored transposed.
struct OrthoParams {
    int32_t rows, cols;          // of D
    int32_t steps_k;             // ceil(K / 128)
    int32_t terms;               // 1, or 2: A or B is the sum of two fp16 matrices (maps a2 / b2)
    int32_t low_side;            // 0: none; then a step per 128 of the tile's diagonal block with the
                                 // low part of A (1) or B (2), stored `batch` matrices further
    int32_t num_r, num_c;        // tiles along rows and columns
    int32_t tiles, batch;        // tiles per matrix; matrices
    int32_t splits;              // slices of K per tile (1: whole)
    float* partials;             // their fp32 sums
    int32_t join_share;          // warps that add the slices of one piece: 1, 2, 4 or 8
    int32_t symmetric;           // 1: only tiles on and below the diagonal, stored twice
    float alpha, beta, diag;
    const float* alpha_dev;      // a further factor per matrix (null: 1)
    const uint16_t* e;           // E, fp16 (null: none), lde elements apart, stride_e per matrix
    int64_t lde, stride_e;
    int32_t store_cols;          // columns that may be stored (D's padded width)
    int32_t low;                 // 1: also store what fp16 rounding lost (map out2; symmetric: of the
                                 // diagonal's tiles, `batch` matrices further)
    int32_t out_bf16;            // 1: D is bf16 instead of fp16
    int32_t plain_store;         // 1: D's rows cannot be written by TMA: element by element to `out`
    uint16_t* out;               // D, for plain stores and for slices
    int64_t ldo, stride_o;
    uint64_t timeout_ns;
    uint32_t* status;
    int32_t stall_kblock;
};

// Which side each operand of a product is stored along.
enum : int { kOrthoNT = 0, kOrthoNN = 1, kOrthoTN = 2 };  // A, B: K K | K MN | MN MN
constexpr int ortho_tile(int cg) { return 128 * cg; }

// out: D in 64 x 32 boxes; out2: its low part, or (symmetric) D in turned boxes
cudaError_t launch_ortho(int form, int cg, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& a2,
                         const CUtensorMap& b2, const CUtensorMap& out, const CUtensorMap& out2, const OrthoParams& p,
                         int grid, cudaStream_t stream, bool pdl);

// The input pass: sums of squares, then G as fp16 in the workspace.
struct OrthoInput {
    const void* g;               // rows x cols, ldg apart, stride_g per matrix
    int64_t ldg, stride_g;
    int32_t dtype;
    int32_t rows, cols, batch;
    int32_t vectors;             // 1: rows start on 16-byte boundaries
    float eps;
    int32_t log2_scale;          // X is stored times 2^log2_scale
    int32_t steps;
    int8_t growth[64];           // per step, powers of two that a small X grows by: ceil(log2 |a|)
    float* sums;                 // [batch][parts]
    int32_t parts;               // blocks per matrix of the first kernel
    uint16_t* hi;                // fp16, `ld` apart, `stride` per matrix; columns up to ld are zeroed
    uint16_t* lo;                // what fp16 lost (null: nothing is)
    int64_t ld, stride;
    float* factors;              // [step][2][batch]: further factors of S and of the next X
};
cudaError_t launch_ortho_input(const OrthoInput& p, cudaStream_t stream, bool pdl);

}  // namespace bwgemm
