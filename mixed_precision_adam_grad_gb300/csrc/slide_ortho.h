// slide_ortho.h — internal interface of the Newton-Schulz products
// (ortho_gemm.cu) and the code that plans them (ortho.cu).
//
// Tiled layouts of the workspace's matrices.  A matrix is cut into row blocks
// of 128; a T16 matrix (FP16) keeps, row block by row block, tiles of 128 rows
// x 64 columns of 16 KiB, a T32 matrix (FP32) tiles of 128 x 32, also 16 KiB.
// Inside a tile each row's 128 bytes are eight 16-byte chunks, and chunk c of
// row r lies at place c ^ (r & 7): the 128-byte swizzle the matrix unit reads,
// so a tile goes to shared memory as one linear bulk copy.  The same bytes
// serve as a K-major operand (rows along M or N) and as an MN-major one (rows
// along K), so no matrix is ever transposed.  A symmetric matrix keeps only
// its upper 128 x 128 blocks: block (i, j), i > j, is read as block (j, i)
// with the other major-ness.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace slide {

constexpr int kTileElems16 = 128 * 64;  // halves of a T16 tile
constexpr int kTileElems32 = 128 * 32;  // floats of a T32 tile

enum OperandKind { kOperandK = 0, kOperandMN = 1, kOperandSym = 2 };

enum EpilogueKind {
    kEpiGram = 0,    // G = acc: out16, and out32 if given
    kEpiPoly = 1,    // B = b*C16 + c*acc: out16 without the diagonal, dvec_out = a + diag; out32/out16b = aI + B if given
    kEpiSym = 2,     // Y = d_i*C32 + acc: out16 (diag_out: without the diagonal, which goes to dvec_out) and out32 if given
    kEpiApply = 3,   // X = d*C32 + acc: out32 and out16
    kEpiOut = 4,     // X as in kEpiApply, rounded to BF16 into the caller's array
    kEpiMuon = 5     // X as in kEpiApply, applied to the caller's master weights
};

struct OrthoOperands {
    const __half *a, *b;
    const float *c32;
    const __half *c16;
    const float *dvec;
    float *out32;
    __half *out16, *out16b;
    float *dvec_out;
};

struct OrthoGemm {
    OrthoOperands p[2];      // nprob products of one shape
    int nprob, batch;
    int a_kind, b_kind;      // OperandKind
    int a_c64, b_c64;        // tiles of a row block of each operand
    int64_t a_stride, b_stride;  // halves from one matrix of the batch to the next
    int k64;                 // steps of 64 along K
    int mblk, nblk;          // 128-blocks of the result
    int sym;                 // only the upper blocks of the result
    int out_c64;             // T16 tiles of a row block of the result (T32: twice as many)
    int64_t out_stride;      // elements from one matrix to the next
    int d_stride;            // floats of dvec per matrix
    int d_by_col;            // dvec scales columns
    int diag_out;
    float alpha;             // acc -> value
    float c16_scale;         // b / scale of C16
    float coef_a;
    float s16, s16b;         // scales of out16 and out16b
    const float *c_inv;      // per matrix factor of C32, or NULL
    // kEpiOut and kEpiMuon
    int rows, cols;
    uint16_t *w;
    int64_t w_row, w_batch;  // strides in elements
    float *theta;            // contiguous
    float decay, step;
    unsigned *status;
    int test_stall;
};

cudaError_t launch_ortho_gemm(const OrthoGemm &g, int epi, int device, cudaStream_t stream);

}  // namespace slide
