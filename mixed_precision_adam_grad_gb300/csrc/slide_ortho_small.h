// slide_ortho_small.h — internal interface of the Newton-Schulz kernels for
// matrices with a side of at most 128 (ortho_small.cu).
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "slide_kernels.h"
#include "slide_ortho.h"

namespace slide {

constexpr int kSmallSide = 128;
constexpr int kSmallMaxSteps = 6;
constexpr int kSmallMaxParts = 4;  // clusters along the long side, one partial Gram matrix each

constexpr int kVecHalves = 2;

struct SmallOrtho {
    // the matrices, or the R replicas of a Muon step
    ReplicaPtrs g;
    int R;
    int64_t row_stride, batch_stride;
    int batch, rows, cols;
    int m;                      // the smaller side
    int tall;
    int fp32;                   // type of the matrices or replicas
    int muon;
    int vec;                    // rows can be read eight values at a time (kVecHalves: as two vectors of four)
    int mom_vec;                // rows of mom and u can
    // Muon: contiguous
    float *mom, *u;
    float mu, one_minus_mu;
    float inv_r;                // 1/R where that is exact, else 0
    int nesterov;
    // the polynomial: G, R = aI + bG + cG^2, T = R G and Q, the product of the
    // R, are FP16 pairs times powers of two; per step the factors that take an
    // accumulator (of scaled factors) or G to the next scaled pair
    int steps;
    float g_first;                   // scale of the first G
    float r_eye[kSmallMaxSteps];     // a
    float r_g[kSmallMaxSteps];       // b
    float r_g2[kSmallMaxSteps];      // c
    float t_of[kSmallMaxSteps];      // R G -> T
    float g_of[kSmallMaxSteps];      // R T -> the next G
    float q_of[kSmallMaxSteps];      // R Q -> Q; for the first step R -> Q
    float q_last;                    // 1 / scale of the last Q
    float eps;
    // scratch
    float *parts;               // [batch][n_parts][128 x 128]
    __half *q;                  // [batch][hi, lo][128 x 128], tiles as in slide_ortho.h
    InverseNorm *inv;           // [batch]
    unsigned *status, *layer_status;  // layer_status may be NULL
    int keep_status;            // add to *status instead of clearing it first
    int n_parts;                // set by the launch
    // results
    uint16_t *w;
    int64_t w_row, w_batch;
    int w_vec;
    float *theta;
    float decay, step;
    int test_stall;
};

// Bytes of the scratch's three arrays for `batch` matrices.
inline int64_t small_parts_bytes(int batch) { return (int64_t)batch * kSmallMaxParts * 128 * 128 * 4; }
inline int64_t small_q_bytes(int batch) { return (int64_t)batch * 2 * 128 * 128 * 2; }

cudaError_t launch_ortho_small(SmallOrtho s, int device, cudaStream_t stream);

}  // namespace slide
