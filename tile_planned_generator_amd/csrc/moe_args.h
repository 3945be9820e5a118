// moe_args.h - argument blocks and launchers of the 8-bit expert layer's kernels:
// the fp8 block quantiser, the block-scaled fp8 products, the sort of tokens by
// expert and the movement of their rows.  Internal to the library.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "fp8_rules.h"

namespace dg {

constexpr int MOE_MAX_EXPERTS = 512;

// Block-scaled fp8 product of A [M][K] and B [N][K] (K contiguous in both):
// C[i][j] = sum over blocks g of sa[g][i] * sb[g][j / b_block] * (a_g . b_g).
enum Fp8Mode : int {
    FP8_DENSE = 0,
    FP8_ROWS = 1,    // rows off[e] .. off[e+1]-1 of A against B + e * stride_b
    FP8_WGRAD = 2    // C + e * stride_c over the K range off[e] .. off[e+1]-1
};
struct Fp8Args {
    const void *A, *B;
    const float *sa, *sb;
    void *C;
    const int32_t *off;              // FP8_ROWS, FP8_WGRAD: experts + 1 device offsets
    int64_t lda, ldb, ld_sa, ld_sb, ldc;
    int64_t stride_b, stride_sb;     // FP8_ROWS: elements between experts
    int64_t stride_c;                // FP8_WGRAD: elements between experts
    int M, N, K, experts;
    int out_type;                    // Elt: T_F16, T_BF16 or T_F32
    int tiles_m, tiles_n;            // FP8_ROWS: tiles_m is the largest possible number of row tiles
    int split_k, k_slice;            // FP8_DENSE: K slices (k_slice a multiple of 128) into ws [split][M][N]
    float *ws;
};
struct Fp8Shape {
    int bm, bn, threads;
    bool stream;                     // K is cut over the waves of a workgroup
    const char *name;
};
const Fp8Shape &fp8_shape(int kernel);
hipError_t launch_fp8(int kernel, int mode, int b_block, const Fp8Args &a, hipStream_t s);

// fp8 quantiser: codes and scales of the rows (or, transposed, of the columns)
// of X, whose row r may be taken from row index[r] / index_div.
struct QuantFp8Args {
    const void *X;
    const int32_t *index;
    void *codes;
    float *scales;
    int64_t x_rows, ldx, ldq, ld_scale;
    int rows, cols;                  // rows after the index, columns of X
    int index_div;
    int x_type;                      // Elt
};
hipError_t launch_quant_fp8(const QuantFp8Args &a, bool transpose, hipStream_t s);

// Stable sort of tokens * topk pairs by expert.
struct MoeSortArgs {
    const int32_t *ids;
    int32_t *off, *src, *dst;
    int32_t *ws;                     // blocks * experts counts, unused when blocks is 1
    int pairs, experts, align, capacity;
    int blocks, per_block;           // workgroups and pairs of each (a multiple of the workgroup's threads)
};
void moe_sort_shape(int64_t pairs, int &blocks, int &per_block);
hipError_t launch_moe_sort(const MoeSortArgs &a, hipStream_t s);

// Movement of token rows; all matrices share the element type.
struct MoeMoveArgs {
    const void *x;                   // gather: X; combine: Y; gradient: Y
    const void *dout;                // gradient: dO
    void *out;                       // gather: Y; combine: O; gradient: dY
    const int32_t *src, *dst;
    const float *w;                  // router's weights [tokens][topk] or null (ones)
    float *dw;                       // gradient: [tokens][topk], or null
    int64_t ldx, ldout, ld_dout;
    int rows, tokens, topk, hidden;
    int type;                        // Elt
};
hipError_t launch_moe_gather(const MoeMoveArgs &a, hipStream_t s);
hipError_t launch_moe_combine(const MoeMoveArgs &a, hipStream_t s);
hipError_t launch_moe_combine_grad(const MoeMoveArgs &a, hipStream_t s);

}  // namespace dg
