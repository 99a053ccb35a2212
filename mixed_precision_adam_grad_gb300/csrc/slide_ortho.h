// slide_ortho.h — internal interface of the Newton-Schulz products
// (ortho_gemm.cu) and the code that plans them (ortho.cu).
//
// Every m x n matrix of the iteration is a pair of FP16 matrices, hi and lo,
// for the value (hi + lo/2048) / s with s a power of two: 22 bits, and hi is
// at the same time the operand of the next product.  A matrix lies in tiles of
// 128 rows x 64 columns of 16 KiB, row block after row block.  Inside a tile
// each row's 128 bytes are eight 16-byte chunks, and chunk c of row r lies at
// place c ^ (r & 7): the 128-byte swizzle the matrix unit reads, so a tile
// goes to shared memory as one linear bulk copy.  The same bytes serve as a
// K-major operand (rows along M or N) and as an MN-major one (rows along K),
// so no matrix is ever transposed.  A symmetric matrix keeps only its upper
// 128 x 128 blocks: block (i, j), i > j, is read as block (j, i) with the
// other major-ness.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace slide {

constexpr int kTileElems = 128 * 64;   // values of a tile
constexpr float kLoScale = 2048.0f;    // lo holds the rounding error of hi times this

enum OperandKind { kOperandK = 0, kOperandMN = 1, kOperandSym = 2 };

// What becomes of the product: value = alpha*acc, then
enum EpilogueKind {
    kEpiGram = 0,    // G = value
    kEpiPoly = 1,    // B = c_scale*C.hi + value: out (hi only) without its diagonal, dvec_out = coef_a + diagonal
    kEpiSym = 2,     // Y = d_i*C + value.  With dvec2 (the product of two factors diag(d) + O that are kept as such):
                     // Y = d_i*C.hi + dvec2_j*C.lo + value, and d_i*dvec2_i on the diagonal.  With diag_out only hi,
                     // without the diagonal, which goes to dvec_out
    kEpiApply = 3,   // X = d*C + value
    kEpiOut = 4,     // X as in kEpiApply, rounded to BF16 into the caller's array
    kEpiMuon = 5     // X as in kEpiApply, applied to the caller's master weights
};

struct OrthoPair {
    __half *hi, *lo;
};

struct OrthoProduct {
    const __half *a, *b;
    OrthoPair c;          // read
    OrthoPair out;        // written
    const float *dvec, *dvec2;
    float *dvec_out;
    float alpha;
    float c_scale;        // of C (1/its scale; for kEpiPoly times b)
    float c_scale2;       // of C.lo, with dvec2
    float s_out;          // scale of out
    int diag_out;
};

struct OrthoGemm {
    OrthoProduct p[2];       // nprob products of one shape and kind
    int epi;                 // EpilogueKind
    int nprob;
    int a_kind, b_kind;      // OperandKind
    int a_c64, b_c64;        // tiles of a row block of each operand
    int64_t a_stride, b_stride;  // values from one matrix of the batch to the next
    int k64;                 // steps of 64 along K
    int mblk, nblk;          // 128-blocks of the result
    int sym;                 // only the upper blocks of the result
    int out_c64;             // tiles of a row block of C and the results
    int64_t out_stride;      // values from one matrix to the next
    int d_stride;            // floats of dvec per matrix
    int d_by_col;            // dvec scales columns
    float coef_a;
    int parts;               // of K, set by the launch (1 in a plan): for kEpiGram, joined by the last CTA to come
    int area;                // of a Gram matrix: the first area for its parts
    int narrow;              // tiles of 128 x 64 instead of 128 x 128, set by the launch (0 in a plan)
};

constexpr int kMaxPhases = 32;  // products of one launch, one after the other
constexpr int kJoinTiles = 80;  // most tiles, of all matrices, whose K is split: with two parts each they fill the SMs
constexpr int kJoinWords = kJoinTiles * 8;

struct OrthoPlan {
    OrthoGemm ph[kMaxPhases];
    int n_phases, batch;
    unsigned *status, *layer_status;  // layer_status may be NULL
    unsigned *count;         // [n_phases][batch] CTAs' tiles written so far, zero at the start
    unsigned *joined;        // [kJoinTiles][8] parts of a tile (a warp's rows and columns of it) so far, zero at the start
    // for parts, memory that nothing else uses during a Gram phase of the same
    // matrix: `areas` arrays from OrthoGemm::area on, each [batch] of area_slots
    // times 128 x 128 floats, a matrix's area_matrix floats from the next one's
    float *area[8];
    int areas, area_slots;
    int64_t area_matrix;
    // kEpiOut and kEpiMuon
    int rows, cols;
    uint16_t *w;
    int64_t w_row, w_batch;  // strides in elements
    int vec;                 // rows of w (and theta) can be written eight values at a time
    float *theta;            // contiguous
    float decay, step;
    int test_stall;
};

constexpr unsigned kStatusWaitLimit = 2u;  // bit of a status word: a wait ran out

__device__ __forceinline__ void report_wait_limit(unsigned *status, unsigned *layer_status)
{
    atomicOr(status, kStatusWaitLimit);
    if (layer_status)
        atomicOr(layer_status, kStatusWaitLimit);
}

// How a call computes, for tests that are written for one way.
enum OrthoForm {
    kFormSmall = 1,    // the kernels for a small side
    kFormGroups = 2,   // several steps on the Gram matrix
    kFormPairs = 4,    // pairs of CTAs
    kFormSplit = 8,    // K of the Gram matrix split
    kFormNarrow = 16   // tiles of 128 x 64 in some phase
};

// With `form` nothing is launched: its bits are added to *form.
cudaError_t launch_ortho_products(const OrthoPlan &plan, int device, cudaStream_t stream, int *form);

// 1/d as a power of two times a factor, for a d = |X|_F + eps that may lie
// anywhere among the norms of finite FP32 matrices (1/d itself need not be an
// FP32 value): x*pow2 is exact but for what lies 2^-126 below the norm, so
// (x*pow2)*rest is x times the rounded 1/d.  0 of zeros, whatever eps; NaN
// where the matrix has a NaN or an infinity.
struct InverseNorm {
    float pow2, rest;
};

__device__ __forceinline__ InverseNorm inverse_norm(double d)
{
    InverseNorm r = {1.0f, 0.0f};
    if (d == 0.0)
        return r;
    if (!(d < 1e300)) {
        r.rest = __int_as_float(0x7fffffff);
        return r;
    }
    const int e = min(126, max(-126, ilogb(d)));
    r.pow2 = exp2f((float)-e);
    r.rest = (float)(ldexp(1.0, e) / d);
    return r;
}

}  // namespace slide
