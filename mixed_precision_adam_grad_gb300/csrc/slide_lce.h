// slide_lce.h — internal interface of the linear cross entropy's products
// (lce_gemm.cu) and the code that plans them (lce.cu).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace slide {

constexpr int kLceRows = 256;         // tokens of a tile: rows of the logits, and of d_x
constexpr float kLceSpread = 30.0f;   // how far a logit may lie above its row's reference

// What becomes of a product, with r a row and c a column of the result.
enum LceKind {
    kLceLogits = 0,  // e = exp(value - ref[r]), 0 for the target's column: written as BF16 (with `keep`), its sum and the
                     // largest value over 128 columns left in `sum` and `top`
    kLceScaled = 1,  // scale[r]*value as BF16
    kLcePlain = 2,   // value as BF16
    kLcePart = 3,    // value as FP32, part after part
    kLceAdd = 4      // value added to FP32
};

struct LceProduct {
    CUtensorMap a, b, out;
    CUtensorMap b_low;  // with `wrap`: second part of b, against the same steps of a
    int wrap;           // steps of a, where there are two parts of b (k64 is twice that), else 0
    int kind;
    int a_mn, b_mn;    // the operand lies with M (or N) innermost instead of K
    int rows, cols;    // of the result
    int k64;           // steps of 64 along K
    int parts;         // of K (kLcePart), each in a slice of its own of out
    int n_fast;        // consecutive tiles go along the columns
    // kLceLogits
    const float *ref;
    const int *target;     // column, or -1: the row is padding
    float *sum, *top;      // [2 * tile columns][pitch]
    int64_t pitch;
    int keep;
    const unsigned *again; // NULL, or whether any rows are wanted, and then per 256 rows whether they are
    const float *scale;    // kLceScaled; 0: the row is 0
    unsigned *status;
    int test_stall;
};

// Columns of a tile: 256.
constexpr int kLceCols = 256;

// Whether a product of so many rows runs on single CTAs (tiles of 128 rows)
// instead of pairs (256).
inline bool lce_single(int rows) { return rows <= 128; }

cudaError_t launch_lce_product(const LceProduct &p, int device, cudaStream_t stream);

// How many tiles run at once.
cudaError_t lce_groups(int rows, int device, int *groups);

// A matrix of rows x cols values, rows `stride` values apart, as boxes of
// box_cols x box_rows for the copy engine; 128-byte swizzle, so a box's row is
// 128 bytes.  fp32: FP32 values instead of BF16.  Slices `slice` values apart,
// if there is more than one.
cudaError_t lce_map(CUtensorMap *map, const void *base, bool fp32, int64_t rows, int64_t cols, int64_t stride, int box_rows,
                    int slices = 1, int64_t slice = 0);

}  // namespace slide
