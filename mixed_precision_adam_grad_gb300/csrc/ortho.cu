// ortho.cu — slide_orthogonalize and slide_muon_step: the Newton-Schulz
// orthogonal factor of a batch of matrices, alone or as the update of the
// matrices' master weights.
//
// With X = G / (|G|_F + eps) and, per step, the quintic of the singular values
//     A = X X^T,  X <- (aI + bA + cA^2) X          (on the smaller side)
// the work is matrix products only, done by ortho_gemm.cu.  Two forms of the
// same polynomial are used:
//   - step by step, three products a step: A and A^2 are symmetric (half the
//     blocks), so a step costs 3 m^2 n + m^3 operations for an m x n matrix;
//   - several steps on the Gram matrix alone: with R = aI + bG + cG^2,
//     G <- R G R and Q <- R Q commute and stay symmetric m x m matrices, and
//     X is multiplied by Q once per group.  A group of p steps costs
//     3 m^2 n + (4p - 3) m^3 instead of p (3 m^2 n + m^3).
// The second form needs fewer operations as soon as n > m; shape_of says from
// where on it is used, groups_of how long a group is.  What limits that is
// accuracy: small singular values are multiplied by a in Q at each step while G
// still holds their squares, beside the roundings of its FP16 operands, which
// have the size of the large ones.  Worst of eight spectra (noise, and 4 to 128
// directions over noise of 1e-1 to 1e-4), 2-norm of the error over 2-norm, of
// five steps:
//     coefficients     m     3 + 2    2 + 2 + 1   step by step
//     quintic        200    8.4e-3      5.1e-3        1.7e-3
//                    500    5.4e-3      3.1e-3        1.0e-3
//                   2560    2.8e-3      1.4e-3        7.2e-4
//     a = 8.2 first  200    8.4e-2      1.8e-2        3.3e-3
//                   2560    1.1e-2      5.8e-3        1.1e-3
// A group of 3 later than the first, where many singular values are near 1, is
// up to 0.45 off (six steps of the quintic, m = 238).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdlib>
#include <cstring>

#include "slide.h"
#include "slide_ortho.h"
#include "slide_ortho_small.h"
#include "slide_state.h"
#include "sm103_ptx.h"

namespace slide {
namespace {

constexpr int kMaxSteps = 16;
constexpr int kGroupSteps = 3;       // at most; only the first group, from a smaller side of kLongGroups on, else 2
constexpr int kLongGroups = 512;
constexpr double kGroupSlope = 3.5;  // largest |a| of a step with others behind it in its group
constexpr int kMaxSide = 1 << 20;
constexpr int kMaxSmallSide = 16384;
constexpr int kMaxBatch = 65535;
constexpr int kNormParts = 512;  // partial sums of squares per matrix
constexpr int kPrepThreads = 256;

// ---- preparation ------------------------------------------------------------

struct SourceArgs {
    ReplicaPtrs g;            // the matrix, or the R replicas of a Muon step
    int R;
    int64_t row_stride, batch_stride;
    int rows, cols;
    int rblk, cblk;           // blocks of 128
    int vec;                  // rows can be read eight values at a time
    int vec4;                 // BF16: four at a time
    // Muon step only: contiguous
    float *mom, *u;
    float mu, one_minus_mu;
    float inv_r;              // 1/R where that is exact (a division of zeros takes long), else 0
    int nesterov;
    double *parts;            // [batch][kNormParts]
    unsigned *status, *count, *joined;
    int keep_status;          // add to *status instead of clearing it first
};

__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float widen(float x) { return x; }

// Values at .. at+7 of a row, of which n lie inside it.
template <typename T>
__device__ __forceinline__ void load8(const void *base, int64_t at, int n, bool vec, float (&v)[8])
{
    const T *p = static_cast<const T *>(base) + at;
    if (vec && n >= 8) {
        if constexpr (sizeof(T) == 2) {
            const uint4 w = *reinterpret_cast<const uint4 *>(p);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(u[e] << 16);
                v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
        } else {
            const float4 w = *reinterpret_cast<const float4 *>(p), x = *reinterpret_cast<const float4 *>(p + 4);
            v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w, v[4] = x.x, v[5] = x.y, v[6] = x.z, v[7] = x.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = e < n ? widen(p[e]) : 0.0f;
    }
}

// Sum of a block's values in a fixed order; thread 0 has it.
__device__ __forceinline__ double block_sum(double x)
{
    __shared__ double s[kPrepThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_down_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) == 0)
        s[threadIdx.x >> 5] = x;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int i = 0; i < kPrepThreads / 32; ++i)
            t += s[i];
    __syncthreads();
    return t;
}

// Squares are added up in FP32 a few at a time and those sums in double.  A
// sum outside this range (values beyond about 1e18, or all below 1e-15) may
// have lost squares to FP32's range: it is formed again in double, from memory
// (the values would take registers until then).
constexpr float kSquaresLow = 0x1p-100f, kSquaresHigh = 0x1p120f;

__device__ __forceinline__ bool squares_fit(float sum) { return sum >= kSquaresLow && sum <= kSquaresHigh; }

template <typename T>
__device__ __forceinline__ double squares_again(const T *p, int n)
{
    double sum = 0.0;
#pragma unroll 1
    for (int e = 0; e < n; ++e) {
        const float x = widen(p[e]);
        if (x != 0.0f)  // FP64 is slow, and zeros have nothing to add
            sum += (double)x * (double)x;
    }
    return sum;
}

constexpr int kRowsAtOnce = kPrepThreads / 16;  // rows of 128 columns, eight a thread

// V values from an address that is aligned to V of them.
template <int V>
__device__ __forceinline__ void load_vec(const uint16_t *p, float (&v)[V])
{
    uint32_t u[V / 2];
    if constexpr (V == 8) {
        const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p));
        u[0] = w.x, u[1] = w.y, u[2] = w.z, u[3] = w.w;
    } else {
        const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(p));
        u[0] = w.x, u[1] = w.y;
    }
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
        v[2 * e] = __uint_as_float(u[e] << 16);
        v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
}

template <int V>
__device__ __forceinline__ void load_vec(const float *p, float (&v)[V])
{
    static_assert(V == 4, "16 bytes");
    const float4 w = __ldcs(reinterpret_cast<const float4 *>(p));
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
}

// One value of a Muon step: the replicas' mean into the momentum, the update.
__device__ __forceinline__ float muon_value(const SourceArgs &a, float sum, float &m)
{
    const float g = __fmul_rn(a.one_minus_mu, a.inv_r > 0.0f ? sum * a.inv_r : __fdiv_rn(sum, (float)a.R));
    m = __fadd_rn(__fmul_rn(m, a.mu), g);
    return a.nesterov ? __fadd_rn(__fmul_rn(m, a.mu), g) : m;
}

__device__ __forceinline__ void begin_source(const SourceArgs &a)
{
    ptx::launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x < kMaxPhases)
        a.count[(int64_t)threadIdx.x * gridDim.y + blockIdx.y] = 0;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        for (int i = threadIdx.x; i < kJoinWords; i += kPrepThreads)
            a.joined[i] = 0;
        if (threadIdx.x == 0 && !a.keep_status)
            *a.status = 0;
    }
}

// A partial sum of a matrix's squares per block of threads, the matrices lying
// one after another without gaps: whole aligned vectors whatever the length of
// a row.  For a Muon step the squares are those of the update, which is formed
// on the way and kept in u.
template <typename T, bool MUON>
__global__ void __launch_bounds__(kPrepThreads) k_ortho_source(const __grid_constant__ SourceArgs a)
{
    begin_source(a);
    // vectors a thread reads whole: 16 bytes of each array it reads most from
    constexpr int V = !MUON && sizeof(T) == 2 ? 8 : 4, kAhead = MUON ? 2 : 4;
    const int b = blockIdx.y;
    const int64_t size = (int64_t)a.rows * a.cols, from = b * size, to = from + size;
    const T *x = static_cast<const T *>(a.g.p[0]);
    const int64_t v0 = (from + V - 1) / V, v1 = to / V;  // aligned vectors inside the matrix
    double sum = 0.0;
    auto square = [](const float(&v)[V]) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e)
            s = fmaf(v[e], v[e], s);
        return s;
    };
    for (int64_t k = v0 + (int64_t)blockIdx.x * (kPrepThreads * kAhead) + threadIdx.x; k < v1;
         k += (int64_t)gridDim.x * (kPrepThreads * kAhead)) {
        float v[kAhead][V], m[MUON ? kAhead : 1][V];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t at = (k + j * kPrepThreads) * V;
            if (at + V <= to) {
                load_vec<V>(x + at, v[j]);
                if constexpr (MUON)
                    load_vec<V>(a.mom + at, m[j]);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    v[j][e] = 0.0f;
            }
        }
        if constexpr (MUON) {
            for (int r = 1; r < a.R; ++r) {
                float w[kAhead][V];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int64_t at = (k + j * kPrepThreads) * V;
                    if (at + V <= to)
                        load_vec<V>(static_cast<const T *>(a.g.p[r]) + at, w[j]);
                }
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    if ((k + j * kPrepThreads) * V + V <= to)
#pragma unroll
                        for (int e = 0; e < V; ++e)
                            v[j][e] = __fadd_rn(v[j][e], w[j][e]);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int64_t at = (k + j * kPrepThreads) * V;
                if (at + V <= to) {
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        v[j][e] = muon_value(a, v[j][e], m[j][e]);
                    __stcs(reinterpret_cast<float4 *>(a.mom + at), make_float4(m[j][0], m[j][1], m[j][2], m[j][3]));
                    *reinterpret_cast<float4 *>(a.u + at) = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
                }
            }
        }
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            part += square(v[j]);
        if (squares_fit(part)) {
            sum += (double)part;
        } else {
#pragma unroll 1
            for (int j = 0; j < kAhead; ++j) {
                const int64_t at = (k + j * kPrepThreads) * V;
                if (at + V <= to) {
                    if constexpr (MUON)
                        sum += squares_again(a.u + at, V);
                    else
                        sum += squares_again(x + at, V);
                }
            }
        }
    }
    // the matrix's first and last values outside whole vectors
    const int head = (int)((v0 * V < to ? v0 * V : to) - from), tail = v1 >= v0 ? (int)(to - v1 * V) : 0;
    if (blockIdx.x == 0 && (int)threadIdx.x < head + tail) {
        const int i = threadIdx.x;
        const int64_t at = i < head ? from + i : v1 * V + (i - head);
        float u = widen(x[at]);
        if constexpr (MUON) {
            for (int r = 1; r < a.R; ++r)
                u = __fadd_rn(u, widen(static_cast<const T *>(a.g.p[r])[at]));
            float m = a.mom[at];
            u = muon_value(a, u, m);
            a.mom[at] = m;
            a.u[at] = u;
        }
        sum += (double)u * (double)u;
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0)
        a.parts[(int64_t)b * kNormParts + blockIdx.x] = sum;
}

// The same of matrices with strides.  A block of threads passes over 128 x 128
// blocks of a matrix; a thread has eight columns of every 16th row.
template <typename T>
__global__ void __launch_bounds__(kPrepThreads) k_ortho_source_strided(const __grid_constant__ SourceArgs a)
{
    begin_source(a);
    const int b = blockIdx.y, r0 = threadIdx.x >> 4, c0 = (threadIdx.x & 15) * 8;
    double sum = 0.0;
    for (int blk = blockIdx.x; blk < a.rblk * a.cblk; blk += gridDim.x) {
        const int rb = blk / a.cblk, cb = blk - rb * a.cblk;
        const int col = cb * 128 + c0, n = a.cols - col;
        float part = 0.0f;
        if (n > 0) {
#pragma unroll 4
            for (int r = r0; r < 128; r += kRowsAtOnce) {
                const int row = rb * 128 + r;
                float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                if (row < a.rows)
                    load8<T>(a.g.p[0], (int64_t)b * a.batch_stride + (int64_t)row * a.row_stride + col, n, a.vec, v);
                float s = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s = fmaf(v[e], v[e], s);
                if (squares_fit(s))
                    part += s;
                else if (row < a.rows)
                    sum += squares_again(static_cast<const T *>(a.g.p[0]) + (int64_t)b * a.batch_stride +
                                             (int64_t)row * a.row_stride + col, min(n, 8));
            }
        }
        sum += (double)part;
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0)
        a.parts[(int64_t)b * kNormParts + blockIdx.x] = sum;
}

struct ScaleArgs {
    const void *x;
    int64_t row_stride, batch_stride;
    int rows, cols, rblk, cblk, vec;
    OrthoPair out;
    int c64;           // tiles of a row block
    int64_t out_stride;
    int n_parts;
    const double *parts;
    float eps, scale;
};

// The 16 aligned bytes at p; what lies outside [lo, hi), the caller's array,
// is not read.
__device__ __forceinline__ uint4 load_granule(uintptr_t p, uintptr_t lo, uintptr_t hi)
{
    if (p >= lo && p + 16 <= hi)
        return *reinterpret_cast<const uint4 *>(p);
    uint32_t w[4] = {0, 0, 0, 0};
    for (int i = 0; i < 8; ++i)  // two bytes at a time: the elements are aligned to that
        if (p + 2 * i >= lo && p + 2 * i < hi)
            w[i >> 1] |= (uint32_t) * reinterpret_cast<const uint16_t *>(p + 2 * i) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight values from element c8*8 of the 128 of a row that begins anywhere: the
// row's 16 lanes read aligned vectors, take the next lane's first one too and
// shift.  `row`: address of the row's first of the 128 (in any case aligned to
// the type), n: how many there are; all 16 lanes call it with the same two.
template <typename T>
__device__ __forceinline__ void load8_shifted(uintptr_t row, int n, int c8, uintptr_t lo, uintptr_t hi, float (&v)[8])
{
    constexpr int kVecs = sizeof(T) / 2;  // 16-byte vectors of eight values
    const uint32_t off = (uint32_t)(row & 15);
    const uintptr_t base = row - off, end = row + (uintptr_t)n * sizeof(T);
    uint32_t w[4 * kVecs + 4];
#pragma unroll
    for (int i = 0; i <= kVecs; ++i) {
        // the last vector is the next lane's first; the last lane reads it itself
        const uintptr_t p = base + (uintptr_t)(c8 * kVecs + i) * 16;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (i < kVecs || c8 == 15)
            if (n > 0 && p < end)
                x = load_granule(p, lo, hi);
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t next = __shfl_down_sync(0xffffffffu, w[j], 1);
        if (c8 != 15)
            w[4 * kVecs + j] = next;
    }
    const bool two = off & 8, one = off & 4;
#pragma unroll
    for (int j = 0; j < 4 * kVecs + 2; ++j)
        w[j] = two ? w[j + 2] : w[j];
#pragma unroll
    for (int j = 0; j < 4 * kVecs + 1; ++j)
        w[j] = one ? w[j + 1] : w[j];
    if constexpr (sizeof(T) == 2) {
        const uint32_t s = (off & 2) * 8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t x = __funnelshift_r(w[j], w[j + 1], s);
            v[2 * j] = __uint_as_float(x << 16);
            v[2 * j + 1] = __uint_as_float(x & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = __uint_as_float(w[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = c8 * 8 + j < n ? v[j] : 0.0f;
}

// X = G / (|G|_F + eps) as a pair of FP16 matrices in tiles, zero beyond the
// matrix's edges.  SHIFTED: the rows do not begin at 16-byte boundaries.
template <typename T, bool SHIFTED>
__global__ void __launch_bounds__(kPrepThreads) k_ortho_scale(const __grid_constant__ ScaleArgs a)
{
    __shared__ InverseNorm s_inv;
    const int b = blockIdx.y, r0 = threadIdx.x >> 4, c8 = threadIdx.x & 15;
    ptx::launch_dependents();
    ptx::wait_for_previous_grid();
    double x = 0.0;
    for (int i = threadIdx.x; i < a.n_parts; i += kPrepThreads)
        x += a.parts[(int64_t)b * kNormParts + i];
    x = block_sum(x);
    if (threadIdx.x == 0)
        s_inv = inverse_norm(sqrt(x) + (double)a.eps);
    __syncthreads();
    const float pow2 = s_inv.pow2, rest = s_inv.rest * a.scale;
    const uintptr_t lo_at = (uintptr_t)a.x;
    const uintptr_t hi_at = (uintptr_t)(static_cast<const T *>(a.x) + (int64_t)(gridDim.y - 1) * a.batch_stride +
                                        (int64_t)(a.rows - 1) * a.row_stride + a.cols);
    for (int blk = blockIdx.x; blk < a.rblk * a.cblk; blk += gridDim.x) {
        const int rb = blk / a.cblk, cb = blk - rb * a.cblk;
        const int col = cb * 128 + c8 * 8, n = a.cols - col;
        const int64_t tile = (int64_t)b * a.out_stride + ((int64_t)rb * a.c64 + 2 * cb + (c8 >> 3)) * kTileElems;
#pragma unroll SHIFTED ? 2 : 4
        for (int r = r0; r < 128; r += kRowsAtOnce) {
            const int row = rb * 128 + r;
            const int64_t at_row = (int64_t)b * a.batch_stride + (int64_t)row * a.row_stride;
            float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (SHIFTED)
                load8_shifted<T>((uintptr_t)(static_cast<const T *>(a.x) + at_row + cb * 128),
                                 row < a.rows ? min(128, a.cols - cb * 128) : 0, c8, lo_at, hi_at, v);
            else if (row < a.rows && n > 0)
                load8<T>(a.x, at_row + col, n, true, v);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = v[2 * e] * pow2 * rest, z = v[2 * e + 1] * pow2 * rest;
                const __half2 p = __floats2half2_rn(y, z);
                const float2 f = __half22float2(p);
                const __half2 q = __floats2half2_rn((y - f.x) * kLoScale, (z - f.y) * kLoScale);
                hi[e] = *reinterpret_cast<const uint32_t *>(&p);
                lo[e] = *reinterpret_cast<const uint32_t *>(&q);
            }
            const int64_t at = tile + r * 64 + (((c8 & 7) ^ (r & 7)) * 8);
            *reinterpret_cast<uint4 *>(a.out.hi + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(a.out.lo + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
}

// ---- plan ---------------------------------------------------------------------

struct Shape {
    int batch, rows, cols;
    int rblk, cblk;      // 128-blocks
    int rpad, cpad;      // rounded up to even
    bool tall;
    int m, n, mblk, mpad;
    bool grouped;
};

Shape shape_of(int batch, int rows, int cols)
{
    Shape s;
    s.batch = batch;
    s.rows = rows;
    s.cols = cols;
    s.rblk = (rows + 127) / 128;
    s.cblk = (cols + 127) / 128;
    s.rpad = (s.rblk + 1) & ~1;
    s.cpad = (s.cblk + 1) & ~1;
    s.tall = rows > cols;
    s.m = s.tall ? cols : rows;
    s.n = s.tall ? rows : cols;
    s.mblk = s.tall ? s.cblk : s.rblk;
    s.mpad = s.tall ? s.cpad : s.rpad;
    // operations per five steps, in m^3: 15 n/m + 5 step by step, 6 n/m + 14
    // in groups of 3 + 2: equal at n = m.  Near there the groups gain nothing
    // and lose accuracy (a square matrix of noise has singular values near
    // zero: 2.7e-3 against 1e-3 at 1000 x 1001), so they start at n = 1.25 m.
    // Small matrices are bound by latency, and step by step there are 15
    // phases instead of 17 and 10 with a K of m instead of 15: 15 us + 0.026 m
    // less, against 0.0121 us n for three more Gram matrices and 0.9 ms for
    // each 1e12 operations more.  Fitted to 45 shapes from 200 x 260 to 4000 x
    // 32000: 200 x 600 95 us step by step, 110 in groups; 1000 x 3000 229 and
    // 197.  Of 163 shapes from 136 x 1000 to 8 of 500 x 16000 it misses one by
    // 9 % (30 of 320 x 1000), the others by at most 5 %.
    // (Of groups of 2 + 2 + 1 the third of these Gram matrices is one of theirs.)
    const double n = s.n, m = s.m, less = 15.0 + 0.026 * m, part = s.m < kLongGroups ? 2.0 / 3.0 : 1.0;
    const double more = part * (0.0121 * n + 0.9e-9 * 9.0 * (n - m) * m * m * batch);
    s.grouped = 4 * (int64_t)s.n >= 5 * (int64_t)s.m && more > less;
    return s;
}

struct Work {
    unsigned *status;
    unsigned *count;           // [kMaxPhases][batch]
    unsigned *joined;          // [kJoinWords]
    double *parts;
    __half *x_hi[2], *x_lo;
    float *u;                  // a Muon step's update
    OrthoPair g;
    __half *o[2];              // B without its diagonal, of this step and the one before
    float *d[2];               // a + the diagonal of B
    // grouped form
    OrthoPair t, q[2];
    float *dq;
    // the kernels for a small side, in the same place
    InverseNorm *inv;
    float *small_parts, *small_u;
    __half *small_q;
    int64_t x_elems, m_elems;  // per matrix
    int64_t bytes;
};

Work layout(const Shape &s, char *base)
{
    Work w{};
    int64_t off = 0;
    auto take = [&](int64_t bytes) {
        char *p = base ? base + off : nullptr;
        off += (int64_t)align_up((size_t)bytes);
        return (void *)p;
    };
    w.x_elems = (int64_t)s.rpad * s.cpad * 128 * 128;
    w.m_elems = (int64_t)s.mpad * s.mpad * 128 * 128;
    const int64_t xb = w.x_elems * s.batch, mb = w.m_elems * s.batch;
    auto pair = [&](int64_t n) {
        OrthoPair p;
        p.hi = (__half *)take(2 * n);
        p.lo = (__half *)take(2 * n);
        return p;
    };
    w.status = (unsigned *)take(4);
    w.count = (unsigned *)take(4 * (int64_t)kMaxPhases * s.batch);
    w.joined = (unsigned *)take(4 * kJoinWords);
    w.parts = (double *)take(8 * (int64_t)s.batch * kNormParts);
    w.x_hi[0] = (__half *)take(2 * xb);
    w.x_lo = (__half *)take(2 * xb);
    w.g = pair(mb);
    const int64_t db = 4 * (int64_t)s.batch * s.mpad * 128;
    w.o[0] = (__half *)take(2 * mb);
    w.d[0] = (float *)take(db);
    if (s.grouped) {
        w.o[1] = (__half *)take(2 * mb);
        w.d[1] = (float *)take(db);
        w.t = pair(mb);
        w.q[0] = pair(mb);
        w.q[1] = pair(mb);
        w.dq = (float *)take(db);
    }
    // the update is read before the first product writes the second copy of X
    w.x_hi[1] = (__half *)take(2 * xb > 4 * (int64_t)s.batch * s.rows * s.cols ? 2 * xb
                                                                               : 4 * (int64_t)s.batch * s.rows * s.cols);
    w.u = (float *)w.x_hi[1];
    w.bytes = off;
    if (s.m <= kSmallSide) {  // the status, then the other kernels' arrays
        off = (int64_t)align_up(4);
        w.inv = (InverseNorm *)take((int64_t)sizeof(InverseNorm) * s.batch);
        w.small_parts = (float *)take(small_parts_bytes(s.batch));
        w.small_q = (__half *)take(small_q_bytes(s.batch));
        w.small_u = (float *)take(4 * (int64_t)s.batch * s.rows * s.cols);
        w.bytes = off > w.bytes ? off : w.bytes;
    }
    return w;
}

// Scales and bounds of each step.  With the spectral norm of X at most
// norm_k, the FP16 operands of step k are stored times powers of two that
// bring typical entries (1/sqrt(m) of the norm) near 1 and keep the largest
// possible one below 2^15.
struct Schedule {
    int steps;
    float a[kMaxSteps], b[kMaxSteps], c[kMaxSteps];
    float sx[kMaxSteps];  // scale of X entering step k
    float sg[kMaxSteps];  // scale of the m x m operands of step k
    double norm[kMaxSteps], r_max[kMaxSteps], t_max[kMaxSteps];  // bounds of |X|, |R| and |R G|
    int group[kMaxSteps];  // steps of the group that begins with step k
};

// The groups of a shape that has them.  Q, the product of a group's R, has to
// stay in FP16's range.
void groups_of(Schedule &s, int m)
{
    for (int k = 0; k < s.steps; k += s.group[k]) {
        const int most = k == 0 && m >= kLongGroups ? kGroupSteps : 2;
        int p = 1;
        double q = s.r_max[k];
        while (p < most && k + p < s.steps && std::fabs(s.a[k + p - 1]) <= kGroupSlope && q * s.r_max[k + p] <= 16384.0)
            q *= s.r_max[k + p++];
        s.group[k] = p;
    }
}

float pow2_floor(double x) { return (float)std::exp2(std::floor(std::log2(x))); }

slide_status schedule_of(const slide_ortho_params *p, int m, Schedule *out)
{
    static const float kQuintic[3] = {3.4445f, -4.7750f, 2.0315f};
    if (!p)
        return fail(SLIDE_ERR_INVALID_ARG, "ortho params are NULL");
    if (p->steps < 1 || p->steps > kMaxSteps)
        return fail(SLIDE_ERR_INVALID_ARG, "ortho params: steps must lie in [1, 16]");
    if (!std::isfinite(p->eps) || p->eps < 0.0f)
        return fail(SLIDE_ERR_INVALID_ARG, "ortho params: eps must be finite and >= 0");
    out->steps = p->steps;
    double norm = 1.0, s = std::fmin(64.0, pow2_floor(std::sqrt((double)m)));
    for (int k = 0; k < p->steps; ++k) {
        const float *t = p->coeffs ? p->coeffs + 3 * k : kQuintic;
        for (int e = 0; e < 3; ++e)
            if (!std::isfinite(t[e]))
                return fail(SLIDE_ERR_INVALID_ARG, "ortho params: non-finite coefficient");
        const double a = out->a[k] = t[0], b = out->b[k] = t[1], c = out->c[k] = t[2];
        double next = 0.0, big = norm * norm, r_max = std::fabs(a), t_max = 0.0;
        for (int i = 1; i <= 1024; ++i) {  // the polynomials on [0, norm]
            const double x = norm * i / 1024.0, x2 = x * x, r = a + b * x2 + c * x2 * x2;
            next = std::fmax(next, std::fabs(x * r));
            big = std::fmax(big, std::fmax(std::fabs(r - a), std::fabs(x2 * r)));
            r_max = std::fmax(r_max, std::fabs(r));
            t_max = std::fmax(t_max, std::fabs(x2 * r));
        }
        out->norm[k] = norm;
        out->r_max[k] = r_max;
        out->t_max[k] = t_max;
        next *= 1.01;
        if (!(next <= 64.0) || !(r_max <= 16384.0) || !(big <= 16384.0))
            return fail(SLIDE_ERR_INVALID_ARG, "ortho params: the coefficients' polynomial grows beyond the range of "
                                               "the iteration (spectral norm 64)");
        double sx = s;
        while (sx > 1.0 && (sx * sx * big > 32768.0 || sx * norm > 32768.0))
            sx *= 0.5;
        out->sx[k] = (float)sx;
        out->sg[k] = (float)(sx * sx);
        s = std::fmax(1.0, s / std::fmax(1.0, std::exp2(std::ceil(std::log2(std::fmax(1.0, std::fabs(a)))))));
        norm = std::fmax(next, 1e-3);
    }
    groups_of(*out, m);
    return SLIDE_OK;
}

struct Finish {
    MuonBlock block;
    int epi;
    uint16_t *w;
    int64_t w_row, w_batch;
    float *theta;
    float decay, step;
};

// Tests only: whether the kernels issue no products, so that their waits run
// out.  "first": those of a layer's first block.
bool test_stall(const MuonBlock &block)
{
    const char *v = getenv("SLIDE_TEST_PIPELINE_STALL");
    return v && (block.index == 0 || strcmp(v, "first") != 0);
}

// The products, from the matrix in x_hi[0] and x_lo to the caller's array; with
// `form` only how they would be computed.
cudaError_t enqueue_products(const Shape &s, const Work &w, const Schedule &sc, const Finish &f, int device,
                             cudaStream_t stream, int *form)
{
    const int xc64 = 2 * s.cpad, mc64 = 2 * s.mpad, mdim = s.mpad * 128;
    const int kn = s.tall ? (s.rows + 63) / 64 : (s.cols + 63) / 64;
    const int km = (s.m + 63) / 64;

    OrthoPlan plan{};
    plan.batch = s.batch;
    plan.status = w.status;
    plan.layer_status = f.block.layer_status;
    plan.count = w.count;
    plan.joined = w.joined;
    if (s.grouped) {
        __half *const free[8] = {w.o[0], w.o[1], w.t.hi, w.t.lo, w.q[0].hi, w.q[0].lo, w.q[1].hi, w.q[1].lo};
        for (__half *p : free)
            plan.area[plan.areas++] = (float *)p;
        plan.area_slots = s.mpad * s.mpad / 2;
        plan.area_matrix = w.m_elems / 2;
    } else {  // the other copy of X
        plan.area[0] = (float *)w.x_hi[0];
        plan.area[1] = (float *)w.x_hi[1];
        plan.areas = 1;
        plan.area_slots = s.rpad * s.cpad / 2;
        plan.area_matrix = w.x_elems / 2;
    }
    plan.rows = s.rows;
    plan.cols = s.cols;
    plan.w = f.w;
    plan.w_row = f.w_row;
    plan.w_batch = f.w_batch;
    plan.vec = (uintptr_t)f.w % 16 == 0 && (f.epi == kEpiMuon ? s.cols % 8 == 0 && (uintptr_t)f.theta % 32 == 0
                                                              : f.w_row % 8 == 0 && (s.batch == 1 || f.w_batch % 8 == 0));
    plan.theta = f.theta;
    plan.decay = f.decay;
    plan.step = f.step;
    plan.test_stall = test_stall(f.block);

    OrthoGemm base{};
    base.nprob = 1;
    base.parts = 1;
    base.d_stride = mdim;

    OrthoGemm mm = base;  // a symmetric m x m product of symmetric factors
    mm.a_kind = mm.b_kind = kOperandSym;
    mm.a_c64 = mm.b_c64 = mm.out_c64 = mc64;
    mm.a_stride = mm.b_stride = mm.out_stride = w.m_elems;
    mm.k64 = km;
    mm.mblk = mm.nblk = s.mblk;
    mm.sym = 1;

    // From m = 512 on T and all but a group's first G are kept without their low
    // halves: 0.8e-3 to 1.0e-3 instead of 0.5e-3 to 0.8e-3 off there (noise with
    // or without strong directions), and half the epilogue's traffic; a smaller m
    // has fewer entries to average their roundings (1.6e-3 at m = 256).
    const bool lean = s.m >= 512;
    auto add = [&](const OrthoGemm &g, int epi) {
        plan.ph[plan.n_phases] = g;
        plan.ph[plan.n_phases++].epi = epi;
    };
    int cur = 0;
    for (int k0 = 0; k0 < sc.steps;) {
        const int p = s.grouped ? sc.group[k0] : 1;
        if (form && p > 1)
            *form |= kFormGroups;
        const bool last = k0 + p == sc.steps;
        if (plan.n_phases + 3 * kGroupSteps + 1 > kMaxPhases) {
            // the next group goes into a launch of its own, whose counts start at zero again
            cudaError_t e = launch_ortho_products(plan, device, stream, form);
            if (e == cudaSuccess && !form)
                e = cudaMemsetAsync(w.count, 0, sizeof(unsigned) * kMaxPhases * s.batch, stream);
            if (e != cudaSuccess)
                return e;
            plan.n_phases = 0;
        }
        // G = X X^T (wide) or X^T X (tall)
        OrthoGemm g = base;
        g.a_kind = g.b_kind = s.tall ? kOperandMN : kOperandK;
        g.a_c64 = g.b_c64 = xc64;
        g.a_stride = g.b_stride = w.x_elems;
        g.k64 = kn;
        g.mblk = g.nblk = s.mblk;
        g.sym = 1;
        g.out_c64 = mc64;
        g.out_stride = w.m_elems;
        g.area = s.grouped ? 0 : cur ^ 1;
        g.p[0].a = g.p[0].b = w.x_hi[cur];
        g.p[0].alpha = 1.0f / (sc.sx[k0] * sc.sx[k0]);
        g.p[0].out.hi = w.g.hi;
        g.p[0].out.lo = p > 1 ? w.g.lo : nullptr;
        g.p[0].s_out = sc.sg[k0];
        add(g, kEpiGram);
        int qcur = 0;
        for (int j = 0; j < p; ++j) {
            const int k = k0 + j, now = j & 1;
            const float sg = sc.sg[k];
            // B = bG + cG^2
            OrthoGemm b = mm;
            b.coef_a = sc.a[k];
            b.p[0].a = b.p[0].b = w.g.hi;
            b.p[0].c = w.g;
            b.p[0].alpha = sc.c[k] / (sg * sg);
            b.p[0].c_scale = sc.b[k] / sg;
            b.p[0].out.hi = w.o[now];
            b.p[0].s_out = sg;
            b.p[0].dvec_out = w.d[now];
            add(b, kEpiPoly);
            if (p == 1)
                break;
            // with R = aI + B = diag(d) + O: T = R G and Q <- R Q, in one launch
            OrthoGemm t = mm;
            t.nprob = 0;
            if (j + 1 < p) {
                OrthoProduct &x = t.p[t.nprob++];
                x.a = w.o[now];
                x.b = w.g.hi;
                x.c = w.g;
                x.c_scale = 1.0f / sg;
                x.dvec = w.d[now];
                x.alpha = 1.0f / (sg * sg);
                x.out = w.t;
                x.s_out = sg;
                if (lean) {
                    x.out.lo = nullptr;
                    if (j > 0)
                        x.c.lo = nullptr;
                }
            }
            if (j > 0) {
                OrthoProduct &x = t.p[t.nprob++];
                x.a = w.o[now];
                x.dvec = w.d[now];
                if (j == 1) {  // Q is the first step's R still: (d + O)(d' + O')
                    const float s0 = sc.sg[k0];
                    x.b = x.c.hi = w.o[0];
                    x.c.lo = w.o[1];
                    x.c_scale = 1.0f / s0;
                    x.c_scale2 = 1.0f / sg;
                    x.dvec2 = w.d[0];
                    x.alpha = 1.0f / (sg * s0);
                } else {
                    x.b = w.q[qcur].hi;
                    x.c = w.q[qcur];
                    x.c_scale = 1.0f;
                    x.alpha = 1.0f / sg;
                }
                x.out.hi = w.q[qcur ^ 1].hi;
                x.out.lo = j + 1 < p ? w.q[qcur ^ 1].lo : nullptr;
                x.s_out = 1.0f;
                x.diag_out = j + 1 == p;
                x.dvec_out = w.dq;
                qcur ^= 1;
            }
            if (t.nprob > 0)
                add(t, kEpiSym);
            if (j + 1 < p) {  // G <- R T
                OrthoGemm n = mm;
                OrthoProduct &x = n.p[0];
                x.a = w.o[now];
                x.b = w.t.hi;
                x.c = w.t;
                x.c_scale = 1.0f / sg;
                x.dvec = w.d[now];
                x.alpha = 1.0f / (sg * sg);
                x.out = w.g;
                x.s_out = sc.sg[k + 1];
                if (lean)
                    x.c.lo = x.out.lo = nullptr;
                add(n, kEpiSym);
            }
        }
        // X <- Q X, the diagonal of Q on both halves of X
        OrthoGemm x = base;
        const __half *q = p == 1 ? w.o[0] : w.q[qcur].hi;
        x.a_kind = s.tall ? kOperandK : kOperandSym;
        x.b_kind = s.tall ? kOperandSym : kOperandMN;
        x.a_c64 = s.tall ? xc64 : mc64;
        x.b_c64 = s.tall ? mc64 : xc64;
        x.a_stride = s.tall ? w.x_elems : w.m_elems;
        x.b_stride = s.tall ? w.m_elems : w.x_elems;
        x.k64 = km;
        x.mblk = s.rblk;
        x.nblk = s.cblk;
        x.out_c64 = xc64;
        x.out_stride = w.x_elems;
        x.d_by_col = s.tall;
        x.p[0].a = s.tall ? w.x_hi[cur] : q;
        x.p[0].b = s.tall ? q : w.x_hi[cur];
        x.p[0].alpha = 1.0f / ((p == 1 ? sc.sg[k0] : 1.0f) * sc.sx[k0]);
        x.p[0].c.hi = w.x_hi[cur];
        x.p[0].c.lo = w.x_lo;
        x.p[0].c_scale = 1.0f / sc.sx[k0];
        x.p[0].dvec = p == 1 ? w.d[0] : w.dq;
        if (!last) {
            x.p[0].out.hi = w.x_hi[cur ^ 1];
            x.p[0].out.lo = w.x_lo;
            x.p[0].s_out = sc.sx[k0 + p];
        }
        add(x, last ? f.epi : kEpiApply);
        cur ^= 1;
        k0 += p;
    }
    return launch_ortho_products(plan, device, stream, form);
}

template <typename Kernel, typename Args>
cudaError_t launch_behind(Kernel k, dim3 grid, const Args &a, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kPrepThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a);
}

// The kernels for a small side of at most 128, which run all steps on the Gram
// matrix; more than kSmallMaxSteps steps would let its rounding errors grow
// (times a^2 a step in directions that X does not have).  Five steps are at most
// 5e-3 off (spectra as above; 1.1e-2 if they begin with a = 8.2), six 2e-2: as
// the products step by step are with so small a side.
bool is_small(const Shape &s, const Schedule &sc) { return s.m <= kSmallSide && sc.steps <= kSmallMaxSteps; }

cudaError_t enqueue_small(const Shape &s, const Work &w, const Schedule &sc, const SourceArgs &a, const Finish &f,
                          bool fp32, bool muon, float eps, int device, cudaStream_t stream)
{
    SmallOrtho o{};
    o.g = a.g;
    o.R = a.R;
    o.row_stride = a.row_stride;
    o.batch_stride = a.batch_stride;
    o.batch = s.batch;
    o.rows = s.rows;
    o.cols = s.cols;
    o.m = s.m;
    o.tall = s.tall;
    o.fp32 = fp32;
    o.muon = muon;
    o.vec = a.vec ? 1 : a.vec4 ? kVecHalves : 0;
    o.mom_vec = s.cols % 4 == 0;
    o.mom = a.mom;
    o.u = w.small_u;
    o.inv_r = a.inv_r;
    o.mu = a.mu;
    o.one_minus_mu = a.one_minus_mu;
    o.nesterov = a.nesterov;
    o.steps = sc.steps;
    const auto scale = [](double bound) { return (double)pow2_floor(16384.0 / std::fmax(bound, 1.0)); };
    double q = 1.0, sq = 1.0;
    for (int k = 0; k < sc.steps; ++k) {
        const double sg = scale(sc.norm[k] * sc.norm[k]), sr = scale(sc.r_max[k]), st = scale(sc.t_max[k]);
        const double next_q = scale(q *= sc.r_max[k]);
        if (k == 0)
            o.g_first = (float)sg;
        o.r_eye[k] = (float)(sc.a[k] * sr);
        o.r_g[k] = (float)(sc.b[k] * sr / sg);
        o.r_g2[k] = (float)(sc.c[k] * sr / (sg * sg));
        o.t_of[k] = (float)(st / (sr * sg));
        if (k + 1 < sc.steps)
            o.g_of[k] = (float)(scale(sc.norm[k + 1] * sc.norm[k + 1]) / (sr * st));
        o.q_of[k] = (float)(k == 0 ? next_q / sr : next_q / (sr * sq));
        sq = next_q;
    }
    o.q_last = (float)(1.0 / sq);
    o.eps = eps;
    o.parts = w.small_parts;
    o.q = w.small_q;
    o.inv = w.inv;
    o.status = w.status;
    o.layer_status = f.block.layer_status;
    o.keep_status = f.block.index > 0;
    o.w = f.w;
    o.w_row = f.w_row;
    o.w_batch = f.w_batch;
    o.theta = f.theta;
    o.decay = f.decay;
    o.step = f.step;
    o.w_vec = muon ? s.cols % 4 == 0
                   : (uintptr_t)f.w % 8 == 0 && f.w_row % 4 == 0 && (s.batch == 1 || f.w_batch % 4 == 0);
    o.test_stall = test_stall(f.block);
    return launch_ortho_small(o, device, stream);
}

// The norms (and a Muon step's update), then the normalised operands.
cudaError_t enqueue_source(const Shape &s, const Work &w, const Schedule &sc, SourceArgs a, bool keep_status, bool fp32,
                           bool muon, float eps, cudaStream_t stream)
{
    a.keep_status = keep_status;
    a.rows = s.rows;
    a.cols = s.cols;
    a.rblk = s.rblk;
    a.cblk = s.cblk;
    a.u = w.u;
    a.parts = w.parts;
    a.status = w.status;
    a.count = w.count;
    a.joined = w.joined;
    const int64_t blocks = (int64_t)s.rblk * s.cblk;
    const int64_t per = (1216 + s.batch - 1) / s.batch;  // eight blocks of threads per SM
    const int64_t most = per < kNormParts ? per : kNormParts;
    const int parts = (int)(blocks < most ? blocks : most);
    const dim3 grid(parts, s.batch);
    const bool flat = a.row_stride == s.cols && (s.batch == 1 || a.batch_stride == (int64_t)s.rows * s.cols) &&
                      (uintptr_t)a.g.p[0] % 16 == 0;
    if (!muon && !flat) {
        if (fp32)
            k_ortho_source_strided<float><<<grid, kPrepThreads, 0, stream>>>(a);
        else
            k_ortho_source_strided<uint16_t><<<grid, kPrepThreads, 0, stream>>>(a);
    } else if (muon) {
        if (fp32)
            k_ortho_source<float, true><<<grid, kPrepThreads, 0, stream>>>(a);
        else
            k_ortho_source<uint16_t, true><<<grid, kPrepThreads, 0, stream>>>(a);
    } else {
        if (fp32)
            k_ortho_source<float, false><<<grid, kPrepThreads, 0, stream>>>(a);
        else
            k_ortho_source<uint16_t, false><<<grid, kPrepThreads, 0, stream>>>(a);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    ScaleArgs c{};
    c.x = muon ? w.u : a.g.p[0];
    c.row_stride = a.row_stride;
    c.batch_stride = a.batch_stride;
    c.rows = s.rows;
    c.cols = s.cols;
    c.rblk = s.rblk;
    c.cblk = s.cblk;
    c.vec = muon ? s.cols % 4 == 0 : a.vec;
    c.out.hi = w.x_hi[0];
    c.out.lo = w.x_lo;
    c.c64 = 2 * s.cpad;
    c.out_stride = w.x_elems;
    c.n_parts = parts;
    c.parts = w.parts;
    c.eps = eps;
    c.scale = sc.sx[0];
    const dim3 grid2((unsigned)(blocks < per ? blocks : per), s.batch);
    if (muon || fp32)
        return c.vec ? launch_behind(k_ortho_scale<float, false>, grid2, c, stream)
                     : launch_behind(k_ortho_scale<float, true>, grid2, c, stream);
    return c.vec ? launch_behind(k_ortho_scale<uint16_t, false>, grid2, c, stream)
                 : launch_behind(k_ortho_scale<uint16_t, true>, grid2, c, stream);
}

cudaError_t enqueue(const Shape &s, const Work &w, const Schedule &sc, const SourceArgs &a, const Finish &f, bool fp32,
                    bool muon, float eps, int device, cudaStream_t stream)
{
    if (is_small(s, sc))
        return enqueue_small(s, w, sc, a, f, fp32, muon, eps, device, stream);
    const cudaError_t e = enqueue_source(s, w, sc, a, f.block.index > 0, fp32, muon, eps, stream);
    return e == cudaSuccess ? enqueue_products(s, w, sc, f, device, stream, nullptr) : e;
}

slide_status check_shape(int32_t batch, int32_t rows, int32_t cols)
{
    if (batch < 0 || batch > kMaxBatch)
        return fail(SLIDE_ERR_INVALID_ARG, "batch must lie in [0, 65535]");
    if (rows < 0 || cols < 0 || rows > kMaxSide || cols > kMaxSide)
        return fail(SLIDE_ERR_INVALID_ARG, "rows and cols must lie in [0, 2^20]");
    if ((rows < cols ? rows : cols) > kMaxSmallSide)
        return fail(SLIDE_ERR_INVALID_ARG, "the smaller side of a matrix must be at most 16384");
    return SLIDE_OK;
}

bool empty(int32_t batch, int32_t rows, int32_t cols) { return batch == 0 || rows == 0 || cols == 0; }

slide_status check_type(int32_t type, const char *what)
{
    if (type != SLIDE_TYPE_BF16 && type != SLIDE_TYPE_FP32)
        return fail(SLIDE_ERR_INVALID_ARG, std::string(what) + " must be SLIDE_TYPE_BF16 or SLIDE_TYPE_FP32");
    return SLIDE_OK;
}

bool misaligned(const void *p, size_t to) { return ((uintptr_t)p % to) != 0; }

slide_status check_workspace(const Work &need, const void *workspace, int64_t bytes)
{
    if (!workspace || misaligned(workspace, 256))
        return fail(SLIDE_ERR_INVALID_ARG, "workspace is NULL or not 256-byte aligned");
    if (bytes < need.bytes)
        return fail(SLIDE_ERR_INVALID_ARG, "workspace is smaller than slide_ortho_workspace says");
    return SLIDE_OK;
}

}  // namespace

slide_status clear_ortho_status(void *workspace, int64_t workspace_bytes, slide_stream_t stream)
{
    if (workspace && !misaligned(workspace, 256) && workspace_bytes >= 256) {
        const cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(unsigned), (cudaStream_t)stream);
        if (e != cudaSuccess)
            return fail_cuda(e, "clearing the workspace's status word");
    }
    clear_error();
    return SLIDE_OK;
}

slide_status check_muon_hparams(const slide_muon_hparams *hp)
{
    if (!hp)
        return fail(SLIDE_ERR_INVALID_ARG, "muon hparams are NULL");
    const float vals[4] = {hp->lr, hp->momentum, hp->weight_decay, hp->scale};
    for (float x : vals)
        if (!std::isfinite(x))
            return fail(SLIDE_ERR_INVALID_ARG, "muon hparams: non-finite value");
    if (hp->lr < 0.0f || hp->weight_decay < 0.0f || hp->scale < 0.0f)
        return fail(SLIDE_ERR_INVALID_ARG, "muon hparams: lr, weight_decay and scale must be >= 0");
    if (hp->momentum < 0.0f || hp->momentum >= 1.0f)
        return fail(SLIDE_ERR_INVALID_ARG, "muon hparams: momentum must lie in [0, 1)");
    Schedule sc;
    return schedule_of(&hp->ortho, 1, &sc);
}

}  // namespace slide

using namespace slide;

extern "C" slide_status slide_ortho_workspace(int32_t batch, int32_t rows, int32_t cols, int64_t *bytes)
{
    slide_status rc = check_shape(batch, rows, cols);
    if (rc != SLIDE_OK)
        return rc;
    if (!bytes)
        return fail(SLIDE_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = empty(batch, rows, cols) ? 256 : layout(shape_of(batch, rows, cols), nullptr).bytes;
    clear_error();
    return SLIDE_OK;
}

extern "C" slide_status slide_orthogonalize(int32_t batch, int32_t rows, int32_t cols, const void *x, int32_t x_type,
                                            int64_t x_row_stride, int64_t x_batch_stride, void *bf16_out,
                                            int64_t out_row_stride, int64_t out_batch_stride,
                                            const slide_ortho_params *params, void *workspace,
                                            int64_t workspace_bytes, slide_stream_t stream)
{
    slide_status rc = check_shape(batch, rows, cols);
    if (rc == SLIDE_OK)
        rc = check_type(x_type, "x_type");
    Schedule sc;
    if (rc == SLIDE_OK)
        rc = schedule_of(params, rows < cols ? (rows > 0 ? rows : 1) : (cols > 0 ? cols : 1), &sc);
    if (rc != SLIDE_OK)
        return rc;
    if (empty(batch, rows, cols))
        return clear_ortho_status(workspace, workspace_bytes, stream);
    if (!x || misaligned(x, x_type == SLIDE_TYPE_FP32 ? 4 : 2) || !bf16_out || misaligned(bf16_out, 2))
        return fail(SLIDE_ERR_INVALID_ARG, "x or bf16_out is NULL or not aligned to its type");
    if (x_row_stride < cols || out_row_stride < cols)
        return fail(SLIDE_ERR_INVALID_ARG, "a row stride is smaller than cols");
    // one after another, or row by row beside one another
    const bool apart = out_batch_stride >= (int64_t)(rows - 1) * out_row_stride + cols ||
                       (out_batch_stride >= cols && out_batch_stride <= (out_row_stride - cols) / (batch > 1 ? batch - 1 : 1));
    if (batch > 1 && (x_batch_stride < 0 || !apart))
        return fail(SLIDE_ERR_INVALID_ARG, "x_batch_stride is negative, or the matrices of bf16_out overlap");
    const Shape s = shape_of(batch, rows, cols);
    const Work w = layout(s, (char *)workspace);
    if ((rc = check_workspace(w, workspace, workspace_bytes)) != SLIDE_OK)
        return rc;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess)
        return fail_cuda(e, "cudaGetDevice");
    SourceArgs a{};
    a.g.p[0] = x;
    a.row_stride = x_row_stride;
    a.batch_stride = x_batch_stride;
    const int64_t per16 = x_type == SLIDE_TYPE_FP32 ? 4 : 8;  // elements of 16 bytes
    a.vec = !misaligned(x, 16) && x_row_stride % per16 == 0 && (batch == 1 || x_batch_stride % per16 == 0);
    a.vec4 = x_type == SLIDE_TYPE_BF16 && !misaligned(x, 8) && x_row_stride % 4 == 0 && (batch == 1 || x_batch_stride % 4 == 0);
    Finish f{};
    f.epi = kEpiOut;
    f.w = (uint16_t *)bf16_out;
    f.w_row = out_row_stride;
    f.w_batch = out_batch_stride;
    e = enqueue(s, w, sc, a, f, x_type == SLIDE_TYPE_FP32, false, params->eps, device, (cudaStream_t)stream);
    if (e != cudaSuccess)
        return fail_cuda(e, "orthogonalisation launch");
    clear_error();
    return SLIDE_OK;
}

slide_status slide::muon_step(int32_t batch, int32_t rows, int32_t cols, int32_t n_replicas,
                              const void *const *grad_replicas, int32_t grads_type, float *master, float *momentum,
                              void *bf16_out, const slide_muon_hparams *hp, void *workspace, int64_t workspace_bytes,
                              const MuonBlock &block, slide_stream_t stream)
{
    slide_status rc = check_shape(batch, rows, cols);
    if (rc == SLIDE_OK)
        rc = check_type(grads_type, "grads_type");
    if (rc != SLIDE_OK)
        return rc;
    if (n_replicas < 1 || n_replicas > SLIDE_MAX_REPLICAS)
        return fail(SLIDE_ERR_INVALID_ARG, "n_replicas must lie in [1, 8]");
    if ((rc = check_muon_hparams(hp)) != SLIDE_OK)
        return rc;
    if (!grad_replicas)
        return fail(SLIDE_ERR_INVALID_ARG, "grad_replicas is NULL");
    if (empty(batch, rows, cols))
        return clear_ortho_status(workspace, workspace_bytes, stream);
    Schedule sc;
    if ((rc = schedule_of(&hp->ortho, rows < cols ? rows : cols, &sc)) != SLIDE_OK)
        return rc;
    SourceArgs a{};
    for (int r = 0; r < n_replicas; ++r) {
        a.g.p[r] = grad_replicas[r];
        if (!a.g.p[r] || misaligned(a.g.p[r], 16))
            return fail(SLIDE_ERR_INVALID_ARG, "gradient replica pointer is NULL or not 16-byte aligned");
    }
    const void *arrs[3] = {master, momentum, bf16_out};
    for (const void *p : arrs)
        if (!p || misaligned(p, 16))
            return fail(SLIDE_ERR_INVALID_ARG, "master, momentum and bf16_out must be 16-byte aligned device pointers");
    const Shape s = shape_of(batch, rows, cols);
    const Work w = layout(s, (char *)workspace);
    if ((rc = check_workspace(w, workspace, workspace_bytes)) != SLIDE_OK)
        return rc;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess)
        return fail_cuda(e, "cudaGetDevice");
    a.R = n_replicas;
    a.row_stride = cols;
    a.batch_stride = (int64_t)rows * cols;
    a.mom = momentum;
    a.inv_r = (n_replicas & (n_replicas - 1)) == 0 ? 1.0f / (float)n_replicas : 0.0f;
    a.mu = hp->momentum;
    a.one_minus_mu = (float)(1.0 - (double)hp->momentum);
    a.nesterov = hp->nesterov != 0;
    a.vec = cols % (grads_type == SLIDE_TYPE_FP32 ? 4 : 8) == 0;
    a.vec4 = grads_type == SLIDE_TYPE_BF16 && cols % 4 == 0;
    Finish f{};
    f.block = block;
    f.epi = kEpiMuon;
    f.w = (uint16_t *)bf16_out;
    f.theta = master;
    f.decay = (float)(1.0 - (double)hp->lr * (double)hp->weight_decay);
    const double scale = hp->scale > 0.0f ? (double)hp->scale : 0.2 * std::sqrt((double)(rows > cols ? rows : cols));
    f.step = (float)((double)hp->lr * scale);
    e = enqueue(s, w, sc, a, f, grads_type == SLIDE_TYPE_FP32, true, hp->ortho.eps, device, (cudaStream_t)stream);
    if (e != cudaSuccess)
        return fail_cuda(e, "muon step launch");
    clear_error();
    return SLIDE_OK;
}

extern "C" slide_status slide_muon_step(int32_t batch, int32_t rows, int32_t cols, int32_t n_replicas,
                                        const void *const *grad_replicas, int32_t grads_type, float *master,
                                        float *momentum, void *bf16_out, const slide_muon_hparams *hp,
                                        void *workspace, int64_t workspace_bytes, slide_stream_t stream)
{
    return muon_step(batch, rows, cols, n_replicas, grad_replicas, grads_type, master, momentum, bf16_out, hp, workspace,
                     workspace_bytes, MuonBlock{}, stream);
}

extern "C" slide_status slide_ortho_status(const void *workspace, slide_stream_t stream)
{
    if (!workspace || misaligned(workspace, 256))
        return fail(SLIDE_ERR_INVALID_ARG, "workspace is NULL or not 256-byte aligned");
    unsigned word = 0;
    cudaError_t e = cudaMemcpyAsync(&word, workspace, sizeof word, cudaMemcpyDeviceToHost, (cudaStream_t)stream);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess)
        return fail_cuda(e, "reading the workspace's status word");
    if (word & 2u)
        return fail(SLIDE_ERR_TIMEOUT, "a pipeline wait inside a product reached its limit; that call is incomplete");
    clear_error();
    return SLIDE_OK;
}

// Tests only: the OrthoForm of a call, or -1.
extern "C" SLIDE_API int32_t slide_test_ortho_form(int32_t batch, int32_t rows, int32_t cols, int32_t muon,
                                                   const slide_ortho_params *params)
{
    Schedule sc;
    if (check_shape(batch, rows, cols) != SLIDE_OK || empty(batch, rows, cols) ||
        schedule_of(params, rows < cols ? rows : cols, &sc) != SLIDE_OK)
        return -1;
    const Shape s = shape_of(batch, rows, cols);
    if (is_small(s, sc))
        return kFormSmall;
    Finish f{};
    f.epi = muon ? kEpiMuon : kEpiOut;
    int device = 0, form = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        enqueue_products(s, layout(s, nullptr), sc, f, device, nullptr, &form) != cudaSuccess)
        return -1;
    return form;
}
