// ortho_small.cu — the Newton-Schulz polynomial for matrices whose smaller side
// m is at most 128: the iteration runs on the m x m Gram matrix inside one
// CTA, and the matrix itself is read twice and written once.
//
//   1. k_small_gram: raw = X X^T (X^T X if tall), each CTA a stretch of the
//      long side, eight of them (a cluster) added up through distributed
//      shared memory; a Muon step's update is formed on the way.  FP32 values
//      enter as pairs of BF16, which need no scale, so no norm has to be known
//      before: |X|_F^2 is the trace of the result.
//   2. k_small_poly: one CTA per matrix: G = raw / (|X|_F + eps)^2, then per
//      step R = aI + bG + cG^2, G <- R G R, Q <- R Q.
//   3. k_small_apply: out = Q X / (|X|_F + eps).
//
// Operands of 2 and 3 are FP16 pairs (hi + lo, 22 bits), each product three
// tensor-core products (hi*hi + hi*lo + lo*hi) into one FP32 accumulator, so
// all steps can run on G without going back to X.  For a 64 x 2560 matrix the
// products themselves take a fifth of the time: what counts is the number of
// dependent steps, about 1.5 us each inside a CTA, where a product that goes
// through global memory and a count of all CTAs takes 6 us.  64 x 2560 takes 31
// us; 36 matrices of 64 x 16512 124 us for 380 MB, 3.1 TB/s: conversions to
// 16-bit pairs beside the loads.
#include <cuda_bf16.h>

#include <atomic>

#include "slide_ortho_small.h"
#include "sm103_ptx.h"

namespace slide {
namespace {

using namespace ptx;

constexpr int kThreads = 256;
constexpr int kCluster = 8;
constexpr int kTile = 16384;           // 128 rows x 64 columns of 16-bit values
constexpr int kGramStages = 3;
constexpr float kApplyScale = 1024.0f; // of X / |X| in k_small_apply: entries are at most 1

__device__ __forceinline__ uint32_t idesc_of(uint32_t n, bool a_mn, bool b_mn, bool bf16)
{
    return f16_idesc(128, n, a_mn, b_mn) | (bf16 ? (1u << 7) | (1u << 10) : 0u);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float widen(float x) { return x; }

// Values at .. at+7 of a row, of which n lie inside it (zero beyond).
template <typename T>
__device__ __forceinline__ void load8(const void *base, int64_t at, int n, int vec, float (&v)[8])
{
    const T *p = static_cast<const T *>(base) + at;
    if (vec && n >= 8) {
        if constexpr (sizeof(T) == 2) {
            uint4 w;
            if (vec == kVecHalves) {
                const uint2 x = reinterpret_cast<const uint2 *>(p)[0], y = reinterpret_cast<const uint2 *>(p)[1];
                w = make_uint4(x.x, x.y, y.x, y.y);
            } else {
                w = *reinterpret_cast<const uint4 *>(p);
            }
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

__device__ __forceinline__ void store8(float *p, int n, bool vec, const float (&v)[8])
{
    if (vec && n >= 8) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n)
                p[e] = v[e];
    }
}

// Eight values as a 16-byte chunk of FP16 (or BF16) and the chunk of what the
// rounding left.
template <bool BF>
__device__ __forceinline__ void split8(const float (&v)[8], uint4 &hi, uint4 &lo)
{
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float x = v[2 * e], y = v[2 * e + 1];
        if constexpr (BF) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
            const float2 f = __bfloat1622float2(p);
            const __nv_bfloat162 q = __floats2bfloat162_rn(x - f.x, y - f.y);
            h[e] = *reinterpret_cast<const uint32_t *>(&p);
            l[e] = *reinterpret_cast<const uint32_t *>(&q);
        } else {
            const __half2 p = __floats2half2_rn(x, y);
            const float2 f = __half22float2(p);
            const __half2 q = __floats2half2_rn(x - f.x, y - f.y);
            h[e] = *reinterpret_cast<const uint32_t *>(&p);
            l[e] = *reinterpret_cast<const uint32_t *>(&q);
        }
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Set-up shared by the three kernels: mbarriers, tensor memory of `cols` columns.
struct Base {
    uint64_t bar[kGramStages + 1];
    uint32_t tmem;
    volatile int abort;
};

__device__ __forceinline__ uint32_t set_up(Base &b, uint32_t cols)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i <= kGramStages; ++i)
            mbar_init(smem_addr(&b.bar[i]), 1);
        b.abort = 0;
        fence_async_shared();
    }
    if (threadIdx.x < 32)
        tmem_alloc<1>(smem_addr(&b.tmem), cols);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    return __shfl_sync(0xffffffffu, b.tmem, 0);
}

// The warp's number, in a form the compiler knows to be the same in all lanes:
// what is computed from it and the kernel's arguments stays in uniform
// registers, which the matrix instructions take (80 cycles each otherwise).
__device__ __forceinline__ int warp_number() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }

// Wait for a barrier that tensor-core products arrive on; a wait that runs out
// ends the CTA's work, which it reports at its end.
__device__ __forceinline__ void wait_products(Base &b, int i, uint32_t parity)
{
    if (!mbar_wait(smem_addr(&b.bar[i]), parity, &b.abort))
        b.abort = 1;
    tmem_fence_after();
}

// ---- 1: the Gram matrix ---------------------------------------------------------

// Grid: (8 * n_parts, batch), clusters of 8 along x.  A step takes 64 of the
// long side.  PAIR: the values need a second BF16.
template <typename T, bool MUON>
__global__ void __launch_bounds__(kThreads, 2) __cluster_dims__(kCluster, 1, 1)
    k_small_gram(const __grid_constant__ SmallOrtho a)
{
    constexpr bool kPair = sizeof(T) == 4 || MUON;
    constexpr int kStage = (kPair ? 2 : 1) * kTile;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Base sh;
    const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t tmem = set_up(sh, 128);
    const int tid = threadIdx.x, warp = warp_number(), lane = tid & 31, b = blockIdx.y;
    launch_dependents();
    if (blockIdx.x == 0 && b == 0 && tid == 0 && !a.keep_status)
        *a.status = 0;
    const int n_side = a.tall ? a.rows : a.cols;
    const int steps = (n_side + 63) / 64, per = (steps + gridDim.x - 1) / gridDim.x;
    const int k0 = min(steps, (int)blockIdx.x * per), k1 = min(steps, k0 + per);
    const uint32_t n16 = (uint32_t)((a.m + 15) & ~15);
    const uint32_t idesc = idesc_of(n16, a.tall, a.tall, true);
    const int mchunks = (a.m + 7) / 8;  // chunks along the short side (tall)

    // Chunk number tid + j*kThreads of step k, of 8 a row (16 if tall with m >
    // 64); n: how many of its eight values exist (0 or less: none).  place: in
    // the stage, negative where nothing is put (what lies in rows beyond n16
    // reaches only rows of the result that nobody reads).
    const int row_shift = a.tall && a.m > 64 ? 4 : 3, per_thread = a.m > 64 ? 4 : 2;
    struct Chunk {
        int64_t at;
        int n, place;
    };
    auto chunk = [&](int k, int j) {
        const int i = tid + j * kThreads, r = i >> row_shift, c = i & ((1 << row_shift) - 1);
        const int row = a.tall ? k * 64 + r : r, col = a.tall ? c * 8 : k * 64 + c * 8;
        Chunk x;
        if (a.tall)
            x.place = c < ((mchunks + 7) & ~7) ? (c >> 3) * (kTile / 2) + r * 128 + (((c & 7) ^ (r & 7)) << 4) : -1;
        else
            x.place = r < (int)n16 ? r * 128 + ((c ^ (r & 7)) << 4) : -1;
        x.n = x.place >= 0 && row < a.rows ? a.cols - col : 0;
        x.at = (int64_t)b * a.batch_stride + (int64_t)row * a.row_stride + col;
        return x;
    };
    auto put = [&](uint32_t stage, int place, const float (&v)[8]) {
        if (place < 0)
            return;
        uint4 hi, lo;
        split8<true>(v, hi, lo);
        sts128(stage + place, hi);
        if constexpr (kPair)
            sts128(stage + kTile + place, lo);
    };
    // A Muon step forms the update on the way, and writes it and the momentum:
    // a chunk at a time, in a loop, what the next step reads on its way into L2
    // meanwhile.  (All four at once in registers took longer, the instructions
    // had to be fetched: a step of six of 18 x 3696 61 us instead of 35.)
    auto muon_step = [&](int k, uint32_t stage) {
#pragma unroll 1
        for (int j = 0; j < per_thread && (a.tall || j * 32 < (int)n16); ++j) {
            const Chunk x = chunk(k, j);
            float v[8], m[8];
            load8<T>(a.g.p[0], x.at, x.n, a.vec, v);
            load8<float>(a.mom, x.at, x.n, a.mom_vec, m);
#pragma unroll 1
            for (int r = 1; r < a.R; ++r) {
                float w[8];
                load8<T>(a.g.p[r], x.at, x.n, a.vec, w);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = __fadd_rn(v[e], w[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = __fmul_rn(a.one_minus_mu, a.inv_r > 0.0f ? v[e] * a.inv_r : __fdiv_rn(v[e], (float)a.R));
                m[e] = __fadd_rn(__fmul_rn(m[e], a.mu), g);
                v[e] = a.nesterov ? __fadd_rn(__fmul_rn(m[e], a.mu), g) : m[e];
            }
            store8(a.mom + x.at, x.n, a.mom_vec, m);
            store8(a.u + x.at, x.n, a.mom_vec, v);
            put(stage, x.place, v);
        }
    };
    auto muon_prefetch = [&](int k) {
#pragma unroll 1
        for (int j = 0; j < per_thread; ++j) {
            const Chunk x = chunk(k, j);
            if (x.n <= 0)
                continue;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(a.mom + x.at));
#pragma unroll 1
            for (int r = 0; r < a.R; ++r)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const T *>(a.g.p[r]) + x.at));
        }
    };
    float v[4][8];  // of the next step (not for a Muon step)
    auto load_step = [&](int k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j >= per_thread)
                break;
            const Chunk x = chunk(k, j);
            load8<T>(a.g.p[0], x.at, x.n, a.vec, v[j]);
        }
    };
    if (k0 < k1) {
        if constexpr (MUON)
            muon_prefetch(k0);
        else
            load_step(k0);
    }
    for (int k = k0; k < k1; ++k) {
        const int it = k - k0, s = it % kGramStages;
        if (it >= kGramStages)
            wait_products(sh, s, (it / kGramStages - 1) & 1);
        const uint32_t stage = ring + s * kStage;
        if constexpr (MUON) {
            if (k + 1 < k1)
                muon_prefetch(k + 1);
            muon_step(k, stage);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < per_thread)
                    put(stage, chunk(k, j).place, v[j]);
            if (k + 1 < k1)
                load_step(k + 1);
        }
        fence_async_shared();
        __syncthreads();
        if (warp == 0 && elect_one() && !a.test_stall) {
            const uint32_t step = a.tall ? 2048u : 32u;
#pragma unroll
            for (int term = 0; term < (kPair ? 3 : 1); ++term) {
                const uint64_t da = operand_desc(stage + (term == 2 ? kTile : 0), kTile / 2);
                const uint64_t db = operand_desc(stage + (term == 1 ? kTile : 0), kTile / 2);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_f16<1>(tmem, da + j * (step >> 4), db + j * (step >> 4), idesc, it > 0 || term > 0 || j > 0);
            }
            mma_commit<1>(smem_addr(&sh.bar[s]));
        }
        __syncwarp();
    }
    // the last products of each stage
    for (int it = max(0, k1 - k0 - kGramStages); it < k1 - k0; ++it)
        wait_products(sh, it % kGramStages, (it / kGramStages) & 1);
    __syncthreads();

    // The cluster's sum: each CTA puts its part into shared memory (chunk c of
    // row r at c ^ (r & 31)), then adds up 16 rows of all of them.
    const int quad = warp & 3, half = warp >> 2, row = quad * 32 + lane;
    if (half * 64 < (int)n16) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            uint32_t acc[32];
            if (k1 > k0) {
                tmem_load32(tmem + ((uint32_t)(quad * 32) << 16) + half * 64 + h * 32, acc);
                tmem_wait_load();
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int c = half * 16 + h * 8 + q;
                const bool in = k1 > k0 && 4 * c < (int)n16;
                sts128(ring + row * 512 + ((c ^ (row & 31)) << 4),
                       in ? make_uint4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]) : make_uint4(0, 0, 0, 0));
            }
        }
    }
    tmem_fence_before();
    cluster_sync();
    const int part = blockIdx.x / kCluster;
    const uint32_t rank = cluster_rank();
    float4 *out = reinterpret_cast<float4 *>(a.parts) + ((int64_t)b * a.n_parts + part) * 4096;
    for (int i = tid; i < 16 * 32; i += kThreads) {
        const int r = rank * 16 + (i & 15), c = i >> 4;
        if (r >= a.m || 4 * c >= (int)n16)
            continue;
        const uint32_t at = ring + r * 512 + ((c ^ (r & 31)) << 4);
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (uint32_t p = 0; p < kCluster; ++p) {
            float4 x;
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                         : "r"(map_to_rank(at, p))
                         : "memory");
            sum.x += x.x;
            sum.y += x.y;
            sum.z += x.z;
            sum.w += x.w;
        }
        out[c * 128 + r] = sum;  // chunk after chunk, so that a thread per row reads along the rows
    }
    cluster_sync();
    tmem_fence_after();
    if (warp == 0)
        tmem_free<1>(tmem, 128);
    if (tid == 0 && sh.abort)
        report_wait_limit(a.status, a.layer_status);
}

// ---- 2: the polynomial ------------------------------------------------------------

// A symmetric m x m pair in shared memory, K-major tiles of 128 rows x 64
// columns.  TILES = 2 (m > 64): two tiles of hi, two of lo.  TILES = 1: one
// tile, hi in rows 0..63 and lo in rows 64..127, so that one instruction
// multiplies a factor by both.
template <int TILES>
__device__ __forceinline__ uint32_t pair_at(uint32_t m, int row, int chunk, bool lo)
{
    if constexpr (TILES == 1)
        row += lo ? 64 : 0;
    else
        m += (chunk >> 3) * kTile + (lo ? 2 * kTile : 0);
    return m + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// acc = A * B of pairs, without lo * lo.  TILES = 2: hi*hi + hi*lo + lo*hi in
// columns 0..n16-1.  TILES = 1: hi*hi + lo*hi there and hi*lo from column 64 on,
// eight instructions instead of twelve; each takes about 80 cycles whatever
// its size.
template <int TILES>
__device__ __forceinline__ void issue_pair(uint32_t tmem, uint32_t a, uint32_t b, uint32_t n16)
{
    const uint32_t k16 = n16 / 16;
    if constexpr (TILES == 1) {
        const uint64_t da = operand_desc(a, 16), db = operand_desc(b, 16);
        const uint32_t both = idesc_of(64 + n16, false, false, false), one = idesc_of(n16, false, false, false);
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
            if (j < k16)
                mma_f16<1>(tmem, da + j * 2, db + j * 2, both, j > 0);
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j)
            if (j < k16)
                mma_f16<1>(tmem, da + (64 * 128 >> 4) + j * 2, db + j * 2, one, true);
    } else {
        const uint32_t idesc = idesc_of(n16, false, false, false);
#pragma unroll
        for (int term = 0; term < 3; ++term) {
            const uint64_t da = operand_desc(a + (term == 2 ? 2 * kTile : 0), 16);
            const uint64_t db = operand_desc(b + (term == 1 ? 2 * kTile : 0), 16);
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                const uint32_t off = ((j >> 2) * kTile + (j & 3) * 32) >> 4;
                if (j < k16)
                    mma_f16<1>(tmem, da + off, db + off, idesc, term > 0 || j > 0);
            }
        }
    }
}

// Row `row`, columns 32*block.. of a pair, from 32 values.
template <int TILES>
__device__ __forceinline__ void put_pair(uint32_t m, int row, int block, const float (&v)[32])
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float x[8] = {v[8 * q], v[8 * q + 1], v[8 * q + 2], v[8 * q + 3],
                            v[8 * q + 4], v[8 * q + 5], v[8 * q + 6], v[8 * q + 7]};
        uint4 hi, lo;
        split8<false>(x, hi, lo);
        sts128(pair_at<TILES>(m, row, 4 * block + q, false), hi);
        sts128(pair_at<TILES>(m, row, 4 * block + q, true), lo);
    }
}

// The lane's 32 values of an accumulator.
template <int TILES>
__device__ __forceinline__ void read_acc(uint32_t at, float (&v)[32])
{
    uint32_t x[32];
    tmem_load32(at, x);
    if constexpr (TILES == 1) {
        uint32_t y[32];
        tmem_load32(at + 64, y);
        tmem_wait_load();
#pragma unroll
        for (int e = 0; e < 32; ++e)
            v[e] = __uint_as_float(x[e]) + __uint_as_float(y[e]);
    } else {
        tmem_wait_load();
#pragma unroll
        for (int e = 0; e < 32; ++e)
            v[e] = __uint_as_float(x[e]);
    }
}

constexpr int kPairBytes = 4 * kTile;  // room of a pair, in shared memory and in a.q
template <int TILES>
constexpr int kPolyPair = TILES == 2 ? kPairBytes : 2 * kTile;  // with TILES = 1 an instruction reads 192 rows
template <int TILES>
constexpr int kPolySmem = 1024 + 3 * kPolyPair<TILES>;

// Traces outside this range may have lost squares to FP32's range.  Below it
// that matters only where eps does not dwarf the norm (below 2^-45).
constexpr float kTraceHigh = 0x1p100f, kTraceLow = 0x1p-90f, kEpsLow = 0x1p-25f, kEpsHigh = 0x1p100f;

__device__ __forceinline__ bool trace_fits(float trace, float eps)
{
    return trace <= kTraceHigh && (trace >= kTraceLow || eps >= kEpsLow) && eps <= kEpsHigh;
}

// For a matrix whose trace does not fit: its Gram matrix once more, by this CTA
// alone, in FP32, from the values times the power of two that brings the
// largest one to 1.  It takes the place of the first part, and zeros that of the
// others; a.inv gets 1/(|X| + eps) and *inv that for the scaled values.
// `stage`: 64 rows of kStageRow floats of shared memory.  (No matrix
// instructions: with this 64 x 2560 takes 0.44 ms instead of 32 us, 128 x 16384
// 4.8 ms, which only such matrices pay.)
constexpr int kStageRow = 132;

__device__ __forceinline__ void gram_again(const SmallOrtho &a, uint32_t stage, int blocks, float *inv)
{
    __shared__ unsigned s_top;
    __shared__ float s_diag[128];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
    auto value = [&](int row, int col) {
        if (a.muon)
            return a.u[((int64_t)b * a.rows + row) * a.cols + col];
        const int64_t at = (int64_t)b * a.batch_stride + (int64_t)row * a.row_stride + col;
        return a.fp32 ? static_cast<const float *>(a.g.p[0])[at] : widen(static_cast<const uint16_t *>(a.g.p[0])[at]);
    };
    if (tid == 0)
        s_top = 0;
    if (tid < 128)
        s_diag[tid] = 0.0f;
    __syncthreads();
    unsigned top = 0;
    for (int row = warp; row < a.rows; row += (int)blockDim.x / 32)
        for (int col = lane; col < a.cols; col += 32)
            top = max(top, __float_as_uint(value(row, col)) & 0x7fffffffu);
    atomicMax(&s_top, top);
    __syncthreads();
    top = s_top;
    const bool finite = top < 0x7f800000u, some = finite && top != 0;
    const int e = some ? ilogbf(__uint_as_float(top)) : 0, e1 = max(-126, min(126, -e));
    const float f1 = exp2f((float)e1), f2 = exp2f((float)(-e - e1));
    const int row = tid & 127, block = tid >> 7, n_side = a.tall ? a.rows : a.cols;
    const bool mine = block < blocks && row < a.m;
    float4 *out = reinterpret_cast<float4 *>(a.parts) + (int64_t)b * a.n_parts * 4096 + block * 8 * 128 + row;
    for (int s0 = 0; s0 < n_side && some; s0 += 64) {
        __syncthreads();
        for (int i = tid; i < 64 * 128; i += blockDim.x) {
            const int k = a.tall ? i >> 7 : i & 63, j = a.tall ? i & 127 : i >> 6;
            const float x = j < a.m && s0 + k < n_side ? (a.tall ? value(s0 + k, j) : value(j, s0 + k)) : 0.0f;
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage + (k * kStageRow + j) * 4), "f"(x * f1 * f2) : "memory");
        }
        __syncthreads();
        for (int q = 0; q < 8 && mine; ++q) {  // four columns at a time, the sums of 64 to those before
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int k = 0; k < 64; ++k) {
                float x;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(stage + (k * kStageRow + row) * 4) : "memory");
                const uint4 y = lds128(stage + (k * kStageRow + block * 32 + 4 * q) * 4);
                sum.x = fmaf(x, __uint_as_float(y.x), sum.x);
                sum.y = fmaf(x, __uint_as_float(y.y), sum.y);
                sum.z = fmaf(x, __uint_as_float(y.z), sum.z);
                sum.w = fmaf(x, __uint_as_float(y.w), sum.w);
            }
            if (s0 > 0) {
                const float4 before = out[q * 128];
                sum.x += before.x;
                sum.y += before.y;
                sum.z += before.z;
                sum.w += before.w;
            }
            out[q * 128] = sum;
            if (block * 32 + 4 * q == (row & ~3))
                s_diag[row] = (row & 3) == 0 ? sum.x : (row & 3) == 1 ? sum.y : (row & 3) == 2 ? sum.z : sum.w;
        }
    }
    for (int part = 1; part < a.n_parts && mine && some; ++part)
        for (int q = 0; q < 8; ++q)
            out[part * 4096 + q * 128] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncthreads();
    if (tid == 0) {
        double trace = 0.0;
        for (int i = 0; i < a.m; ++i)
            trace += s_diag[i];
        const InverseNorm r = inverse_norm(finite ? ldexp(sqrt(trace), e) + (double)a.eps : NAN);
        a.inv[b] = r;
        *inv = (float)ldexp((double)r.pow2 * r.rest, e);
    }
    __syncthreads();
}

// 128 threads per 32 columns and a last warp that issues the products.  Warp
// (quad, block) has rows 32*quad.. and columns 32*block.. of every matrix; warps
// whose rows all lie beyond m rest.  Rows and columns beyond m inside a used
// block are zero, those of unused blocks hold anything: they only meet rows of
// results that nobody reads.
//
// A step is three products one after the other, G^2, T = R G and R T; Q <- R Q
// runs behind the third and is taken up while the next step's first is under
// way.
template <int TILES>
__global__ void __launch_bounds__(128 * 2 * TILES + 32) k_small_poly(const __grid_constant__ SmallOrtho a)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ Base sh;
    __shared__ double s_trace[4];
    __shared__ float s_inv;
    __shared__ int s_again;
    __shared__ float s_f[6][kSmallMaxSteps];  // the factors of the steps (from the arguments each would take 200 cycles)
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t G = base, R = base + kPolyPair<TILES>, Q = base + 2 * kPolyPair<TILES>;
    const uint32_t tmem = set_up(sh, 256);
    const int tid = threadIdx.x, warp = warp_number(), lane = tid & 31, b = blockIdx.x;
    const int blocks = (int)blockDim.x / 128;  // of 32 columns
    const bool issuer = warp == 4 * blocks;
    const int quad = warp & 3, block = warp >> 2, row = quad * 32 + lane;
    const uint32_t n16 = (uint32_t)((a.m + 15) & ~15);
    const uint32_t acc0 = tmem + ((uint32_t)(quad * 32) << 16) + block * 32, acc1 = acc0 + 128;
    const bool mine = !issuer && quad * 32 < a.m;
    const bool diag = mine && quad == block;  // the lane's diagonal element is its number `lane`
    const int eye_at = diag && row < a.m ? lane : -1;
    if (tid < a.steps) {
        s_f[0][tid] = a.r_eye[tid];
        s_f[1][tid] = a.r_g[tid];
        s_f[2][tid] = a.r_g2[tid];
        s_f[3][tid] = a.t_of[tid];
        s_f[4][tid] = a.g_of[tid];
        s_f[5][tid] = a.q_of[tid];
    }
    launch_dependents();
    wait_for_previous_grid();
    if (tid == 0) {
        s_again = 0;
        if (*(volatile unsigned *)a.status & kStatusWaitLimit)
            sh.abort = 1;  // the launch before gave up: no waits of the full length
    }
    uint32_t done[2] = {0, 0};  // products waited for on each of the two barriers

again:
    // the raw Gram matrix, zero beyond m; its trace is |X|_F^2
    float v[32];
    if (!issuer) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const int chunk = block * 8 + c;
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (row < a.m && 4 * chunk < (int)n16) {
                const float4 *p =
                    reinterpret_cast<const float4 *>(a.parts) + (int64_t)b * a.n_parts * 4096 + chunk * 128 + row;
                for (int k = 0; k < a.n_parts; ++k) {
                    const float4 x = p[(int64_t)k * 4096];
                    sum.x += x.x;
                    sum.y += x.y;
                    sum.z += x.z;
                    sum.w += x.w;
                }
            }
            v[4 * c] = sum.x, v[4 * c + 1] = sum.y, v[4 * c + 2] = sum.z, v[4 * c + 3] = sum.w;
        }
    }
    if (diag) {
        double trace = 0.0;
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (e == lane)
                trace = v[e];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            trace += __shfl_xor_sync(0xffffffffu, trace, o);
        if (lane == 0)
            s_trace[quad] = trace;
    }
    __syncthreads();
    if (tid == 0 && !s_again) {  // one thread: FP64 is slow
        double trace = 0.0;
        for (int i = 0; i < blocks; ++i)
            trace += s_trace[i];
        // a matrix of zeros stays one, whatever eps
        s_inv = trace == 0.0 && a.eps == 0.0f ? 0.0f : (float)(1.0 / (sqrt(trace) + (double)a.eps));
        a.inv[b] = InverseNorm{1.0f, s_inv};
    }
    __syncthreads();
    const float inv = s_inv;
    float r[32];  // bG + aI of the coming step, from G as it is written
    auto begin_r = [&](int k) {
        const float eye = s_f[0][k], bb = s_f[1][k];
#pragma unroll
        for (int e = 0; e < 32; ++e)
            r[e] = fmaf(bb, v[e], e == eye_at ? eye : 0.0f);
    };
    if (mine) {
#pragma unroll
        for (int e = 0; e < 32; ++e)
            v[e] = v[e] * inv * (inv * a.g_first);
        put_pair<TILES>(G, row, block, v);
        begin_r(0);
    }
    auto issue = [&](int bar, uint32_t x, uint32_t y) {
        if (issuer && !a.test_stall) {
            tmem_fence_after();
            if (elect_one()) {
                issue_pair<TILES>(tmem + bar * 128, x, y, n16);
                mma_commit<1>(smem_addr(&sh.bar[bar]));
            }
            __syncwarp();
        }
    };
    auto wait = [&](int bar) {
        wait_products(sh, bar, done[bar] & 1);
        ++done[bar];
    };
    // this thread's values of an accumulator, times f, into a pair
    auto keep = [&](uint32_t acc, float f, uint32_t to) {
        if (!mine)
            return;
        read_acc<TILES>(acc, v);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            v[e] *= f;
        put_pair<TILES>(to, row, block, v);
    };
    auto settle = [&] {
        tmem_fence_before();
        fence_async_shared();
        __syncthreads();
    };
    settle();

    for (int k = 0; k < a.steps && !sh.abort; ++k) {
        const bool more = k + 1 < a.steps;
        const float cc = s_f[2][k], t_of = s_f[3][k], g_of = s_f[4][k];
        issue(0, G, G);
        if (k > 1) {  // the Q of the step before
            wait(1);
            keep(acc1, s_f[5][k - 1], Q);
        }
        wait(0);
        if (mine) {  // R = aI + bG + cG^2; the first R is also Q
            read_acc<TILES>(acc0, v);
#pragma unroll
            for (int e = 0; e < 32; ++e)
                v[e] = fmaf(cc, v[e], r[e]);
            put_pair<TILES>(R, row, block, v);
            if (k == 0) {
                const float q_of = s_f[5][0];
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    v[e] *= q_of;
                put_pair<TILES>(Q, row, block, v);
            }
        }
        settle();
        if (more) {
            issue(0, R, G);  // T, in G's place
            wait(0);
            keep(acc0, t_of, G);
            settle();
            issue(0, R, G);  // the next G, from R and T
            if (k > 0)
                issue(1, R, Q);
            wait(0);
            keep(acc0, g_of, G);
            begin_r(k + 1);
            settle();
        } else if (k > 0) {
            issue(1, R, Q);
            wait(1);
            keep(acc1, s_f[5][k], Q);
            settle();
        }
    }
    // Q, as it lies; k_small_apply reads its rows below n16, or of lo from row 64 on
    uint4 *out = reinterpret_cast<uint4 *>(a.q) + (int64_t)b * (kPairBytes / 16);
    for (int i = tid; i < (TILES == 2 ? kPairBytes : kTile) / 16; i += blockDim.x)
        out[i] = lds128(Q + i * 16);
    // Only now, off the straight way (each CTA runs through its instructions
    // once, and fetching them counts): was the Gram matrix what it should be?
    if (!s_again && !sh.abort) {
        double trace = 0.0;
        for (int i = 0; i < blocks; ++i)
            trace += s_trace[i];
        if (!trace_fits((float)trace, a.eps)) {
            gram_again(a, base, blocks, &s_inv);
            if (tid == 0)
                s_again = 1;
            __syncthreads();
            goto again;
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == 0)
        tmem_free<1>(tmem, 256);
    if (tid == 0 && sh.abort)
        report_wait_limit(a.status, a.layer_status);
}

// ---- 3: the result ------------------------------------------------------------------

// A CTA takes stretches of 128 of the long side in turn.  Shared memory: Q
// (pair), X (pair), both only as many 64-column tiles (Q) and rows or tiles (X)
// as m needs; the result goes through X's place as FP32.
template <typename T, bool MUON, int TILES>
__global__ void __launch_bounds__(kThreads, TILES == 1 ? 3 : 1) k_small_apply(const __grid_constant__ SmallOrtho a)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ Base sh;
    const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const uint32_t tmem = set_up(sh, 128);
    const int tid = threadIdx.x, warp = warp_number(), lane = tid & 31, b = blockIdx.y;
    const uint32_t n16 = (uint32_t)((a.m + 15) & ~15), k16 = n16 / 16;
    constexpr int tiles = TILES;               // 64-column tiles along the short side
    const uint32_t q_lo = tiles * kTile;       // Q: tiles of hi, then tiles of lo
    // X: tall: 128 rows x m, tiles along m; wide: m rows x 128, two tiles of 64*tiles rows
    const uint32_t X = base + 2 * q_lo, x_lo = tiles * kTile, x_tile = a.tall ? kTile : tiles * (kTile / 2);
    const uint32_t idesc = a.tall ? idesc_of(n16, false, false, false) : idesc_of(128, false, true, false);
    const int quad = warp & 3, half = warp >> 2;
    launch_dependents();
    wait_for_previous_grid();
    if (tid == 0 && (*(volatile unsigned *)a.status & kStatusWaitLimit))
        sh.abort = 1;
    __syncthreads();
    const InverseNorm inverse = a.inv[b];
    const float pow2 = inverse.pow2, inv = inverse.rest * kApplyScale;  // pow2 is 1 wherever 1/norm has room in FP32
    const float back = a.q_last / kApplyScale;
    {
        const uint4 *q = reinterpret_cast<const uint4 *>(a.q) + (int64_t)b * (kPairBytes / 16);
        if constexpr (tiles == 2) {
            for (int i = tid; i < 2 * (kTile / 16); i += kThreads) {
                sts128(base + i * 16, q[i]);
                sts128(base + q_lo + i * 16, q[2 * (kTile / 16) + i]);
            }
        } else {  // 64 rows of each
            for (int i = tid; i < kTile / 32; i += kThreads) {
                sts128(base + i * 16, q[i]);
                sts128(base + q_lo + i * 16, q[kTile / 32 + i]);
            }
        }
    }
    const int n_side = a.tall ? a.rows : a.cols;
    uint32_t phase = 0;
    // tall: 128 rows of 8*tiles chunks; wide: 64*tiles rows of 16 chunks
    float v[4 * tiles][8];
    auto load_stretch = [&](int s0) {
#pragma unroll
        for (int j = 0; j < 4 * tiles; ++j) {
            const int i = tid + j * kThreads;
            const int row = a.tall ? s0 + (tiles == 2 ? i >> 4 : i >> 3) : i >> 4;
            const int col = a.tall ? (i & (8 * tiles - 1)) * 8 : s0 + (i & 15) * 8;
            const int n = a.cols - col;
            if (row < a.rows && n > 0) {
                const int64_t at = (int64_t)b * a.batch_stride + (int64_t)row * a.row_stride + col;
                if constexpr (MUON)
                    load8<float>(a.u, at, n, a.mom_vec, v[j]);
                else
                    load8<T>(a.g.p[0], at, n, a.vec, v[j]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[j][e] = 0.0f;
            }
        }
    };
    load_stretch(blockIdx.x * 128);
    for (int s0 = blockIdx.x * 128; s0 < n_side && !sh.abort; s0 += gridDim.x * 128, ++phase) {
#pragma unroll
        for (int j = 0; j < 4 * tiles; ++j) {
            const int i = tid + j * kThreads;
            const int r = a.tall ? (tiles == 2 ? i >> 4 : i >> 3) : i >> 4, c = a.tall ? i & (8 * tiles - 1) : i & 15;
            const uint32_t place = (c >> 3) * x_tile + r * 128 + (((c & 7) ^ (r & 7)) << 4);
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = v[j][e] * pow2 * inv;
            uint4 hi, lo;
            split8<false>(x, hi, lo);
            sts128(X + place, hi);
            sts128(X + x_lo + place, lo);
        }
        if (s0 + (int)gridDim.x * 128 < n_side)
            load_stretch(s0 + gridDim.x * 128);
        fence_async_shared();
        __syncthreads();
        if (warp == 0 && elect_one() && !a.test_stall) {
            tmem_fence_after();
            for (int term = 0; term < 3; ++term) {
                const uint32_t q = base + (term == 1 ? q_lo : 0), x = X + (term == 2 ? x_lo : 0);
                const uint64_t dq = operand_desc(q, 16), dx = operand_desc(x, x_tile);
                for (uint32_t j = 0; j < k16; ++j) {
                    const uint32_t kq = ((j >> 2) * kTile + (j & 3) * 32) >> 4;
                    if (a.tall)
                        mma_f16<1>(tmem, dx + kq, dq + kq, idesc, term > 0 || j > 0);
                    else
                        mma_f16<1>(tmem, dq + kq, dx + ((j * 2048) >> 4), idesc, term > 0 || j > 0);
                }
            }
            mma_commit<1>(smem_addr(&sh.bar[0]));
        }
        __syncwarp();
        wait_products(sh, 0, phase & 1);
        // rows x cols of the result: tall 128 x m, wide m x 128; FP32 in X's
        // place, chunk c of row r at c ^ (r & (chunks of a row - 1))
        const int d_cols = a.tall ? 64 * tiles : 128, d_rows = a.tall ? 128 : 64 * tiles, chunks = d_cols / 4;
        const int row = quad * 32 + lane;
        if (row < d_rows && half * 64 < d_cols) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                uint32_t x[32];
                tmem_load32(tmem + ((uint32_t)(quad * 32) << 16) + half * 64 + h * 32, x);
                tmem_wait_load();
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const int c = half * 16 + h * 8 + q;
                    sts128(X + row * d_cols * 4 + ((c ^ (row & (chunks - 1) & 31)) << 4),
                           make_uint4(__float_as_uint(__uint_as_float(x[4 * q]) * back),
                                      __float_as_uint(__uint_as_float(x[4 * q + 1]) * back),
                                      __float_as_uint(__uint_as_float(x[4 * q + 2]) * back),
                                      __float_as_uint(__uint_as_float(x[4 * q + 3]) * back)));
                }
            }
        }
        tmem_fence_before();
        __syncthreads();
        const int top = a.tall ? s0 : 0, left = a.tall ? 0 : s0;
        const int r_end = min(d_rows, a.rows - top), c_end = min(d_cols, a.cols - left);
        // four columns of a row at a time: 16 or 32 threads per row
        const int per_row = d_cols / 4, at_once = kThreads / per_row;
        const int c = (tid % per_row) * 4;
        constexpr int kAhead = MUON ? 4 : 1;
        for (int r0 = tid / per_row; r0 < r_end; r0 += at_once * kAhead) {
            float th[kAhead][4];
            if constexpr (MUON) {
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int r = r0 + j * at_once;
                    if (r < r_end && c < c_end) {
                        const float *p = a.theta + ((int64_t)b * a.rows + top + r) * a.cols + left + c;
                        if (a.w_vec && c + 4 <= c_end) {
                            const float4 w = *reinterpret_cast<const float4 *>(p);
                            th[j][0] = w.x, th[j][1] = w.y, th[j][2] = w.z, th[j][3] = w.w;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                th[j][e] = c + e < c_end ? p[e] : 0.0f;
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int r = r0 + j * at_once;
                if (r >= r_end || c >= c_end)
                    continue;
                const uint4 u = lds128(X + r * d_cols * 4 + (((c / 4) ^ (r & (chunks - 1) & 31)) << 4));
                float o[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
                int64_t at;
                if constexpr (MUON) {
                    at = ((int64_t)b * a.rows + top + r) * a.cols + left + c;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[e] = __fsub_rn(__fmul_rn(th[j][e], a.decay), __fmul_rn(a.step, o[e]));
                } else {
                    at = (int64_t)b * a.w_batch + (int64_t)(top + r) * a.w_row + left + c;
                }
                uint16_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = __bfloat16_as_ushort(__float2bfloat16_rn(o[e]));
                if (a.w_vec && c + 4 <= c_end) {
                    if constexpr (MUON)
                        *reinterpret_cast<float4 *>(a.theta + at) = make_float4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint2 *>(a.w + at) =
                        make_uint2((uint32_t)w[0] | (uint32_t)w[1] << 16, (uint32_t)w[2] | (uint32_t)w[3] << 16);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (c + e < c_end) {
                            if constexpr (MUON)
                                a.theta[at + e] = o[e];
                            a.w[at + e] = w[e];
                        }
                    }
                }
            }
        }
        fence_async_shared();
        __syncthreads();  // the next stretch takes X's place
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == 0)
        tmem_free<1>(tmem, 128);
    if (tid == 0 && sh.abort)
        report_wait_limit(a.status, a.layer_status);
}

constexpr int kMaxDevices = 64;

template <typename Kernel>
cudaError_t launch_kernel(Kernel k, dim3 grid, int threads, int smem, bool behind, const SmallOrtho &a, cudaStream_t stream,
                          std::atomic<int> &ready)
{
    if (!ready.load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kPolySmem<2>);
        if (e != cudaSuccess)
            return e;
        ready.store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = behind ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <typename T, bool MUON>
cudaError_t launch_all(SmallOrtho &a, int device, int sms, cudaStream_t stream)
{
    static std::atomic<int> ready[kMaxDevices][5];
    const int n_side = a.tall ? a.rows : a.cols;
    // a cluster of eight CTAs per 8 x 2 steps of 64, as long as all are resident (two a SM): with 8 x 4
    // a Muon step of 2 x 4096 x 100 took 76 us instead of 66
    const int steps = (n_side + 63) / 64;
    const int fit = 2 * sms / (kCluster * a.batch);
    int parts = (steps + 2 * kCluster - 1) / (2 * kCluster);
    parts = parts < fit ? parts : fit;
    parts = parts < 1 ? 1 : parts > kSmallMaxParts ? kSmallMaxParts : parts;
    a.n_parts = parts;
    const int pair = sizeof(T) == 4 || MUON ? 2 : 1;
    const int gram = 1024 + (kGramStages * pair * kTile > 65536 ? kGramStages * pair * kTile : 65536);
    cudaError_t e = launch_kernel(k_small_gram<T, MUON>, dim3(kCluster * parts, a.batch), kThreads, gram, false, a, stream,
                                  ready[device][0]);
    const int tiles = a.m > 64 ? 2 : 1, poly = (a.m + 31) / 32 * 128 + 32;
    if (e == cudaSuccess)
        e = tiles == 2 ? launch_kernel(k_small_poly<2>, dim3(a.batch), poly, kPolySmem<2>, true, a, stream, ready[device][1])
                       : launch_kernel(k_small_poly<1>, dim3(a.batch), poly, kPolySmem<1>, true, a, stream, ready[device][4]);
    if (e != cudaSuccess)
        return e;
    const int64_t stretches = (n_side + 127) / 128;
    const int64_t room = (int64_t)sms * (tiles == 2 ? 1 : 3) / a.batch;  // what is resident at once
    const dim3 grid((unsigned)(stretches < room ? stretches : room > 0 ? room : 1), a.batch);
    const int smem = 1024 + 4 * tiles * kTile;
    return tiles == 2 ? launch_kernel(k_small_apply<T, MUON, 2>, grid, kThreads, smem, true, a, stream, ready[device][2])
                      : launch_kernel(k_small_apply<T, MUON, 1>, grid, kThreads, smem, true, a, stream, ready[device][3]);
}

}  // namespace

cudaError_t launch_ortho_small(SmallOrtho a, int device, cudaStream_t stream)
{
    if (device < 0 || device >= kMaxDevices)
        return cudaErrorInvalidDevice;
    static std::atomic<int> count[kMaxDevices];
    int sms = count[device].load(std::memory_order_acquire);
    if (sms == 0) {
        const cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
        if (e != cudaSuccess)
            return e;
        count[device].store(sms, std::memory_order_release);
    }
    if (a.muon)
        return a.fp32 ? launch_all<float, true>(a, device, sms, stream) : launch_all<uint16_t, true>(a, device, sms, stream);
    return a.fp32 ? launch_all<float, false>(a, device, sms, stream) : launch_all<uint16_t, false>(a, device, sms, stream);
}

}  // namespace slide
