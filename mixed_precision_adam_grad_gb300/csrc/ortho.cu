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
// The second form needs fewer operations as soon as n > m and is used from n =
// 1.25 m on.  A group is at most
// kGroupSteps = 3 steps: small singular values are multiplied by a^p in Q
// while G still holds their squares, and the FP16 operands then cost 6e-4 to
// 1.2e-3 (2-norm) with groups of 3 + 2, but up to 5e-3 with one group of 5
// when a few directions dominate.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "slide.h"
#include "slide_ortho.h"
#include "slide_state.h"

namespace slide {
namespace {

constexpr int kMaxSteps = 16;
constexpr int kGroupSteps = 3;
constexpr int kMaxSide = 1 << 20;
constexpr int kMaxSmallSide = 16384;
constexpr int kMaxBatch = 65535;
constexpr int kNormParts = 512;  // partial sums of squares per matrix
constexpr int kPrepThreads = 256;

// ---- preparation ------------------------------------------------------------

struct SourceArgs {
    // kSrcMatrix: x; kSrcMuon: g[0..R-1] and the momentum
    ReplicaPtrs g;
    int R;
    int64_t row_stride, batch_stride;
    float *mom;
    float mu, one_minus_mu;
    int nesterov;
    int rows, cols;
    int rblk, cblk, c32;      // blocks of 128; T32 tiles of a row block
    int64_t out_stride;
    float *out;               // T32, not normalised
    double *parts;            // [batch][kNormParts]
    int vec;                  // rows can be read four values at a time
    unsigned *status;
};

__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float widen(float x) { return x; }

template <typename T>
__device__ __forceinline__ void load4(const void *base, int64_t at, int n, bool vec, float (&v)[4])
{
    const T *p = static_cast<const T *>(base) + at;
    if (vec && n == 4) {
        if constexpr (sizeof(T) == 2) {
            const uint2 w = __ldcs(reinterpret_cast<const uint2 *>(p));
            v[0] = __uint_as_float(w.x << 16);
            v[1] = __uint_as_float(w.x & 0xffff0000u);
            v[2] = __uint_as_float(w.y << 16);
            v[3] = __uint_as_float(w.y & 0xffff0000u);
        } else {
            const float4 w = __ldcs(reinterpret_cast<const float4 *>(p));
            v[0] = w.x;
            v[1] = w.y;
            v[2] = w.z;
            v[3] = w.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
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

// Reads the matrix (or forms Muon's update from the replicas and the
// momentum), writes it in T32 tiles, zero beyond its edges, and a partial sum
// of its squares per block.
template <typename T, bool MUON>
__global__ void __launch_bounds__(kPrepThreads) k_ortho_source(const __grid_constant__ SourceArgs a)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
    if (blockIdx.x == 0 && b == 0 && threadIdx.x == 0)
        *a.status = 0;
    double sum = 0.0;
    for (int blk = blockIdx.x; blk < a.rblk * a.cblk; blk += gridDim.x) {
        const int rb = blk / a.cblk, cb = blk - rb * a.cblk;
        const int col = cb * 128 + lane * 4;
        const int n = min(4, a.cols - col);
        float part = 0.0f;
        for (int r = warp; r < 128; r += kPrepThreads / 32) {
            const int row = rb * 128 + r;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (row < a.rows && n > 0) {
                const int64_t at = (int64_t)b * a.batch_stride + (int64_t)row * a.row_stride + col;
                if constexpr (MUON) {
                    float m[4];
                    load4<T>(a.g.p[0], at, n, a.vec, v);
                    for (int k = 1; k < a.R; ++k) {
                        float w[4];
                        load4<T>(a.g.p[k], at, n, a.vec, w);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = __fadd_rn(v[e], w[e]);
                    }
                    load4<float>(a.mom, at, n, a.vec, m);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float g = __fmul_rn(a.one_minus_mu, __fdiv_rn(v[e], (float)a.R));
                        m[e] = __fadd_rn(__fmul_rn(m[e], a.mu), g);
                        v[e] = a.nesterov ? __fadd_rn(__fmul_rn(m[e], a.mu), g) : m[e];
                    }
                    if (a.vec && n == 4) {
                        __stcs(reinterpret_cast<float4 *>(a.mom + at), make_float4(m[0], m[1], m[2], m[3]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (e < n)
                                a.mom[at + e] = m[e];
                            else
                                v[e] = 0.0f;
                        }
                    }
                } else {
                    load4<T>(a.g.p[0], at, n, a.vec, v);
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                part = fmaf(v[e], v[e], part);
            float *tile = a.out + (int64_t)b * a.out_stride +
                          ((int64_t)rb * a.c32 + cb * 4 + (lane >> 3)) * kTileElems32 + r * 32;
            reinterpret_cast<float4 *>(tile)[(lane & 7) ^ (r & 7)] = make_float4(v[0], v[1], v[2], v[3]);
        }
        sum += (double)part;
    }
    sum = block_sum(sum);
    if (threadIdx.x == 0)
        a.parts[(int64_t)b * kNormParts + blockIdx.x] = sum;
}

struct ScaleArgs {
    const float *x;   // T32
    __half *out;      // T16
    int64_t x_stride;
    int tiles;        // T16 tiles per matrix (the padding's among them)
    int n_parts;
    const double *parts;
    float *inv;       // [batch]
    float eps, scale;
};

// inv = 1 / (|G|_F + eps), and the normalised matrix as FP16 operands.
__global__ void __launch_bounds__(kPrepThreads) k_ortho_scale(const ScaleArgs a)
{
    __shared__ float s_inv;
    const int b = blockIdx.y;
    double x = 0.0;
    for (int i = threadIdx.x; i < a.n_parts; i += kPrepThreads)
        x += a.parts[(int64_t)b * kNormParts + i];
    x = block_sum(x);
    if (threadIdx.x == 0) {
        s_inv = (float)(1.0 / (sqrt(x) + (double)a.eps));
        if (x == 0.0 && a.eps == 0.0f)
            s_inv = 0.0f;  // a matrix of zeros stays one
        if (blockIdx.x == 0)
            a.inv[b] = s_inv;
    }
    __syncthreads();
    const float inv = s_inv, scale = a.scale;
    for (int t = blockIdx.x; t < a.tiles; t += gridDim.x) {
        const float4 *src = reinterpret_cast<const float4 *>(a.x + (int64_t)b * a.x_stride + (int64_t)t * kTileElems16);
        uint4 *dst = reinterpret_cast<uint4 *>(a.out + (int64_t)b * a.x_stride + (int64_t)t * kTileElems16);
        for (int i = threadIdx.x; i < kTileElems16 / 8; i += kPrepThreads) {
            const int r = i >> 3, c = (i & 7) ^ (r & 7);  // chunk c (8 columns) of row r
            const float4 *row = src + (c >> 2) * (kTileElems32 / 4) + r * 8;
            const float4 u = row[(2 * (c & 3)) ^ (r & 7)], w = row[(2 * (c & 3) + 1) ^ (r & 7)];
            const float f[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __half2 p = __floats2half2_rn(f[2 * e] * inv * scale, f[2 * e + 1] * inv * scale);
                h[e] = *reinterpret_cast<const uint32_t *>(&p);
            }
            dst[i] = make_uint4(h[0], h[1], h[2], h[3]);
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
    s.grouped = 4 * (int64_t)s.n >= 5 * (int64_t)s.m;
    return s;
}

struct Work {
    unsigned *status;
    float *inv;
    double *parts;
    float *x32;
    __half *x16[2];
    __half *g16, *o16;
    float *d;
    // grouped form
    __half *t16, *q16[2];
    float *g32, *t32, *q32, *dq;
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
    w.status = (unsigned *)take(4);
    w.inv = (float *)take(4 * (int64_t)s.batch);
    w.parts = (double *)take(8 * (int64_t)s.batch * kNormParts);
    w.x32 = (float *)take(4 * xb);
    w.x16[0] = (__half *)take(2 * xb);
    w.x16[1] = (__half *)take(2 * xb);
    w.g16 = (__half *)take(2 * mb);
    w.o16 = (__half *)take(2 * mb);
    w.d = (float *)take(4 * (int64_t)s.batch * s.mpad * 128);
    if (s.grouped) {
        w.t16 = (__half *)take(2 * mb);
        w.q16[0] = (__half *)take(2 * mb);
        w.q16[1] = (__half *)take(2 * mb);
        w.g32 = (float *)take(4 * mb);
        w.t32 = (float *)take(4 * mb);
        w.q32 = (float *)take(4 * mb);
        w.dq = (float *)take(4 * (int64_t)s.batch * s.mpad * 128);
    }
    w.bytes = off;
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
};

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
    double q = 1.0;
    for (int k = 0; k < p->steps; ++k) {
        const float *t = p->coeffs ? p->coeffs + 3 * k : kQuintic;
        for (int e = 0; e < 3; ++e)
            if (!std::isfinite(t[e]))
                return fail(SLIDE_ERR_INVALID_ARG, "ortho params: non-finite coefficient");
        const double a = out->a[k] = t[0], b = out->b[k] = t[1], c = out->c[k] = t[2];
        double next = 0.0, big = norm * norm, r_max = std::fabs(a);
        for (int i = 1; i <= 1024; ++i) {  // the polynomials on [0, norm]
            const double x = norm * i / 1024.0, x2 = x * x, r = a + b * x2 + c * x2 * x2;
            next = std::fmax(next, std::fabs(x * r));
            big = std::fmax(big, std::fmax(std::fabs(r - a), std::fabs(x2 * r)));
            r_max = std::fmax(r_max, std::fabs(r));
        }
        next *= 1.01;
        q = (k % kGroupSteps == 0 ? 1.0 : q) * r_max;
        if (!(next <= 64.0) || !(q <= 16384.0) || !(big <= 16384.0))
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
    return SLIDE_OK;
}

struct Finish {
    int epi;
    uint16_t *w;
    int64_t w_row, w_batch;
    float *theta;
    float decay, step;
};

bool test_stall() { return getenv("SLIDE_TEST_PIPELINE_STALL") != nullptr; }

// The products, from the matrix in w.x32 and w.x16[0] to the caller's array.
cudaError_t enqueue_products(const Shape &s, const Work &w, const Schedule &sc, const Finish &f, int device,
                             cudaStream_t stream)
{
    const int xc64 = 2 * s.cpad, mc64 = 2 * s.mpad, mdim = s.mpad * 128;
    const int kn = s.tall ? (s.rows + 63) / 64 : (s.cols + 63) / 64;
    const int km = (s.m + 63) / 64;
    const bool stall = test_stall();

    OrthoGemm base{};
    base.nprob = 1;
    base.batch = s.batch;
    base.d_stride = mdim;
    base.status = w.status;
    base.test_stall = stall;

    OrthoGemm mm = base;  // a symmetric m x m product of symmetric factors
    mm.a_kind = mm.b_kind = kOperandSym;
    mm.a_c64 = mm.b_c64 = mm.out_c64 = mc64;
    mm.a_stride = mm.b_stride = mm.out_stride = w.m_elems;
    mm.k64 = km;
    mm.mblk = mm.nblk = s.mblk;
    mm.sym = 1;

    int cur = 0;
    cudaError_t e = cudaSuccess;
    for (int k0 = 0; k0 < sc.steps;) {
        const int p = s.grouped ? (sc.steps - k0 < kGroupSteps ? sc.steps - k0 : kGroupSteps) : 1;
        const bool last = k0 + p == sc.steps;
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
        g.alpha = 1.0f / (sc.sx[k0] * sc.sx[k0]);
        g.s16 = sc.sg[k0];
        g.p[0].a = g.p[0].b = w.x16[cur];
        g.p[0].out16 = w.g16;
        g.p[0].out32 = p > 1 ? w.g32 : nullptr;
        if ((e = launch_ortho_gemm(g, kEpiGram, device, stream)) != cudaSuccess)
            return e;
        int qcur = 0;
        for (int j = 0; j < p; ++j) {
            const int k = k0 + j;
            const float sg = sc.sg[k];
            // B = bG + cG^2
            OrthoGemm b = mm;
            b.alpha = sc.c[k] / (sg * sg);
            b.c16_scale = sc.b[k] / sg;
            b.coef_a = sc.a[k];
            b.s16 = sg;
            b.s16b = 1.0f;
            b.p[0].a = b.p[0].b = b.p[0].c16 = w.g16;
            b.p[0].out16 = w.o16;
            b.p[0].dvec_out = w.d;
            if (j == 0 && p > 1) {
                b.p[0].out32 = w.q32;
                b.p[0].out16b = w.q16[0];
            }
            if ((e = launch_ortho_gemm(b, kEpiPoly, device, stream)) != cudaSuccess)
                return e;
            if (p == 1)
                break;
            if (j > 0) {  // Q <- R Q
                OrthoGemm q = mm;
                q.alpha = 1.0f / sg;
                q.s16 = 1.0f;
                q.diag_out = j + 1 == p;
                q.p[0].a = w.o16;
                q.p[0].b = w.q16[qcur];
                q.p[0].c32 = w.q32;
                q.p[0].dvec = w.d;
                q.p[0].out32 = j + 1 == p ? nullptr : w.q32;
                q.p[0].out16 = w.q16[qcur ^ 1];
                q.p[0].dvec_out = w.dq;
                if ((e = launch_ortho_gemm(q, kEpiSym, device, stream)) != cudaSuccess)
                    return e;
                qcur ^= 1;
            }
            if (j + 1 < p) {
                OrthoGemm t = mm;  // T = R G
                t.alpha = 1.0f / (sg * sg);
                t.s16 = sg;
                t.p[0].a = w.o16;
                t.p[0].b = w.g16;
                t.p[0].c32 = w.g32;
                t.p[0].dvec = w.d;
                t.p[0].out32 = w.t32;
                t.p[0].out16 = w.t16;
                if ((e = launch_ortho_gemm(t, kEpiSym, device, stream)) != cudaSuccess)
                    return e;
                t.s16 = sc.sg[k + 1];  // G <- R T
                t.p[0].b = w.t16;
                t.p[0].c32 = w.t32;
                t.p[0].out32 = j + 2 < p ? w.g32 : nullptr;
                t.p[0].out16 = w.g16;
                if ((e = launch_ortho_gemm(t, kEpiSym, device, stream)) != cudaSuccess)
                    return e;
            }
        }
        // X <- Q X, the diagonal of Q on the FP32 copy of X
        OrthoGemm x = base;
        const __half *q16 = p == 1 ? w.o16 : w.q16[qcur];
        x.a_kind = s.tall ? kOperandK : kOperandSym;
        x.b_kind = s.tall ? kOperandSym : kOperandMN;
        x.a_c64 = s.tall ? xc64 : mc64;
        x.b_c64 = s.tall ? mc64 : xc64;
        x.a_stride = s.tall ? w.x_elems : w.m_elems;
        x.b_stride = s.tall ? w.m_elems : w.x_elems;
        x.p[0].a = s.tall ? w.x16[cur] : q16;
        x.p[0].b = s.tall ? q16 : w.x16[cur];
        x.k64 = km;
        x.mblk = s.rblk;
        x.nblk = s.cblk;
        x.out_c64 = xc64;
        x.out_stride = w.x_elems;
        x.d_by_col = s.tall;
        x.alpha = 1.0f / ((p == 1 ? sc.sg[k0] : 1.0f) * sc.sx[k0]);
        x.c_inv = k0 == 0 ? w.inv : nullptr;
        x.p[0].c32 = w.x32;
        x.p[0].dvec = p == 1 ? w.d : w.dq;
        if (last) {
            x.rows = s.rows;
            x.cols = s.cols;
            x.w = f.w;
            x.w_row = f.w_row;
            x.w_batch = f.w_batch;
            x.theta = f.theta;
            x.decay = f.decay;
            x.step = f.step;
        } else {
            x.s16 = sc.sx[k0 + p];
            x.p[0].out32 = w.x32;
            x.p[0].out16 = w.x16[cur ^ 1];
        }
        if ((e = launch_ortho_gemm(x, last ? f.epi : kEpiApply, device, stream)) != cudaSuccess)
            return e;
        cur ^= 1;
        k0 += p;
    }
    return cudaSuccess;
}

cudaError_t enqueue_source(const Shape &s, const Work &w, const Schedule &sc, SourceArgs a, bool fp32, bool muon,
                           float eps, cudaStream_t stream)
{
    a.rows = s.rows;
    a.cols = s.cols;
    a.rblk = s.rblk;
    a.cblk = s.cblk;
    a.c32 = 4 * s.cpad;
    a.out_stride = w.x_elems;
    a.out = w.x32;
    a.parts = w.parts;
    a.status = w.status;
    const int64_t blocks = (int64_t)s.rblk * s.cblk;
    const int parts = (int)(blocks < kNormParts ? blocks : kNormParts);
    const dim3 grid(parts, s.batch);
    if (muon) {
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
    c.x = w.x32;
    c.out = w.x16[0];
    c.x_stride = w.x_elems;
    c.tiles = s.rblk * 2 * s.cpad;
    c.n_parts = parts;
    c.parts = w.parts;
    c.inv = w.inv;
    c.eps = eps;
    c.scale = sc.sx[0];
    const int per = (1216 + s.batch - 1) / s.batch;
    const dim3 grid2(c.tiles < per ? c.tiles : per, s.batch);
    k_ortho_scale<<<grid2, kPrepThreads, 0, stream>>>(c);
    return cudaGetLastError();
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
    if (empty(batch, rows, cols)) {
        clear_error();
        return SLIDE_OK;
    }
    if (!x || misaligned(x, x_type == SLIDE_TYPE_FP32 ? 4 : 2) || !bf16_out || misaligned(bf16_out, 2))
        return fail(SLIDE_ERR_INVALID_ARG, "x or bf16_out is NULL or not aligned to its type");
    if (x_row_stride < cols || out_row_stride < cols)
        return fail(SLIDE_ERR_INVALID_ARG, "a row stride is smaller than cols");
    if (batch > 1 && (x_batch_stride < 0 || out_batch_stride < (int64_t)(rows - 1) * out_row_stride + cols))
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
    const size_t v4 = x_type == SLIDE_TYPE_FP32 ? 16 : 8;
    a.vec = !misaligned(x, v4) && x_row_stride % 4 == 0 && (batch == 1 || x_batch_stride % 4 == 0);
    e = enqueue_source(s, w, sc, a, x_type == SLIDE_TYPE_FP32, false, params->eps, (cudaStream_t)stream);
    if (e != cudaSuccess)
        return fail_cuda(e, "orthogonalisation: preparation launch");
    Finish f{};
    f.epi = kEpiOut;
    f.w = (uint16_t *)bf16_out;
    f.w_row = out_row_stride;
    f.w_batch = out_batch_stride;
    e = enqueue_products(s, w, sc, f, device, (cudaStream_t)stream);
    if (e != cudaSuccess)
        return fail_cuda(e, "orthogonalisation: product launch");
    clear_error();
    return SLIDE_OK;
}

extern "C" slide_status slide_muon_step(int32_t batch, int32_t rows, int32_t cols, int32_t n_replicas,
                                        const void *const *grad_replicas, int32_t grads_type, float *master,
                                        float *momentum, void *bf16_out, const slide_muon_hparams *hp,
                                        void *workspace, int64_t workspace_bytes, slide_stream_t stream)
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
    if (empty(batch, rows, cols)) {
        clear_error();
        return SLIDE_OK;
    }
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
    a.mu = hp->momentum;
    a.one_minus_mu = (float)(1.0 - (double)hp->momentum);
    a.nesterov = hp->nesterov != 0;
    a.vec = cols % 4 == 0;
    e = enqueue_source(s, w, sc, a, grads_type == SLIDE_TYPE_FP32, true, hp->ortho.eps, (cudaStream_t)stream);
    if (e != cudaSuccess)
        return fail_cuda(e, "muon step: preparation launch");
    Finish f{};
    f.epi = kEpiMuon;
    f.w = (uint16_t *)bf16_out;
    f.theta = master;
    f.decay = (float)(1.0 - (double)hp->lr * (double)hp->weight_decay);
    const double scale = hp->scale > 0.0f ? (double)hp->scale : 0.2 * std::sqrt((double)(rows > cols ? rows : cols));
    f.step = (float)((double)hp->lr * scale);
    e = enqueue_products(s, w, sc, f, device, (cudaStream_t)stream);
    if (e != cudaSuccess)
        return fail_cuda(e, "muon step: product launch");
    clear_error();
    return SLIDE_OK;
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
