// lce_gemm.cu — the matrix products of the linear cross entropy on the
// fifth-generation tensor cores (tcgen05, accumulators in tensor memory), BF16
// operands and FP32 accumulators.
//
// A CTA is persistent over output tiles: warp 0 brings operand tiles by TMA
// into a ring of stages, warp 1 issues the matrix instructions, and warps 2-9
// read finished accumulators from tensor memory, which holds two of them, so
// an epilogue overlaps the next tile's products.  A pair of CTAs (cta_group::2)
// has a tile of 256 x 256, each CTA 128 of its rows and half of the operand
// that both need; both CTAs' copies are counted by the barriers of the first,
// which issues for both.  Up to 128 rows go to single CTAs on 128 x 256.
//
// The operands lie as the caller has them, row by row; either dimension may be
// the innermost one, since the matrix unit reads 128-byte swizzled tiles both
// ways, so nothing is transposed in memory.  What a box has beyond the matrix
// arrives as zeros, and is not written.
//
// Bound by the matrix instructions: 4096 x 5120 x 152064 takes 3.2 ms forwards
// (1.98 PFLOP/s), 3.4 and 3.2 ms for the gradients; at 2048 x 2560 x 50257 the
// tensor pipe is active 84, 87 and 84 % of the time.  In a series of calls the
// power limit sets the pace (11.5 ms for the three, 1.66 PFLOP/s).  A pair's step of
// 64 along K takes 0.34 us and brings 64 KiB from L2.
#include <cuda_bf16.h>

#include <atomic>

#include "slide_lce.h"
#include "sm103_ptx.h"

namespace slide {
namespace {

using namespace ptx;

constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kPiece = 4096;                      // 32 rows of 128 bytes
constexpr int kEpiBuffers = 2;                    // of an epilogue warp
constexpr int kEpiBytes = kEpiWarps * kEpiBuffers * kPiece;
constexpr int kBlock = 16384;                     // an operand of 128 x 64
constexpr unsigned kFullMask = 0xffffffffu;
constexpr unsigned kStatusWaitLimit = 2u;
// Steps of 64 that the accumulators add up.  The matrix unit cuts each of its
// additions, on average a quarter of 2^-24 of the sum so far, always towards 0, so
// a long sum comes out small: by 4.3e-6 of its value over 5120 random products, by
// 6.6e-5 over 65536; where all have one sign by 3.8e-4 over 65536 and 6.4e-3 over
// a million.  The epilogue's warps therefore take the sums of every kRun steps and
// add them in registers, rounded: 1.0e-6 of a logit of one sign's products at any
// length, 2e-7 of the magnitudes where signs are random.  For logits this costs the
// launch 1 to 2 % (loss of 1021 x 2560 over 50257 words 181 us instead of 179, with
// 8 steps 183).  The gradients' sums end as BF16 and may be longer: below 5e-5 over
// 4096 products of one sign, where BF16 rounds by up to 3.9e-3.
constexpr int kRun = 16, kGradientRun = 64;
constexpr float kLog2e = 1.4426950408889634f;

template <int CG>
struct Ring {
    static constexpr int kB = CG == 2 ? kBlock : 2 * kBlock;  // a CTA's columns: half of the pair's, or all 256
    static constexpr int kStage = kBlock + kB;
    static constexpr int kStages = CG == 2 ? 5 : 3;
    static constexpr int kSmem = 1024 + kStages * kStage + kEpiBytes;
};

struct Tile {
    int i, j, part;
};

template <int CG>
__host__ __device__ __forceinline__ int tile_rows(const LceProduct &p)
{
    return (p.rows + 128 * CG - 1) / (128 * CG);
}
__host__ __device__ __forceinline__ int tile_cols(const LceProduct &p) { return (p.cols + kLceCols - 1) / kLceCols; }

template <int CG>
__device__ __forceinline__ Tile decode(const LceProduct &p, int t)
{
    const int mt = tile_rows<CG>(p), nt = tile_cols(p);
    Tile x;
    x.part = t / (mt * nt);
    t -= x.part * (mt * nt);
    if (p.n_fast) {
        x.i = t / nt;
        x.j = t - x.i * nt;
    } else {
        x.j = t / mt;
        x.i = t - x.j * mt;
    }
    return x;
}

template <int CG>
__device__ __forceinline__ bool wanted(const LceProduct &p, const Tile &x)
{
    return !p.again || p.again[1 + x.i * CG / 2] != 0;
}

__device__ __forceinline__ int first_step(const LceProduct &p, int part)
{
    return (int)((int64_t)part * p.k64 / p.parts);
}

// A box from (x, y) of the matrix, counted by `bar`: for a pair the first
// CTA's, wherever the box goes.
template <int CG>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                dst),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
            "%3}], [%4];" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
}

__device__ __forceinline__ void store_box(const CUtensorMap *map, uint32_t src, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y),
                 "r"(src)
                 : "memory");
}

__device__ __forceinline__ void store_box3(const CUtensorMap *map, uint32_t src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
                 "r"(y), "r"(z), "r"(src)
                 : "memory");
}

__device__ __forceinline__ void add_box(const CUtensorMap *map, uint32_t src, int x, int y)
{
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
                 "r"(x), "r"(y), "r"(src)
                 : "memory");
}

// An operand's block of `count` rows along M (or N) from r0 on, step k of K.
template <int CG>
__device__ __forceinline__ void load_operand(uint32_t slot, const CUtensorMap *map, bool mn, int r0, int count, int k,
                                             uint32_t bar)
{
    if (mn) {
        for (int i = 0; i < count / 64; ++i)
            load_box<CG>(slot + i * (kBlock / 2), map, r0 + i * 64, k * 64, bar);
    } else {
        for (int i = 0; i < count / 128; ++i)
            load_box<CG>(slot + i * kBlock, map, k * 64, r0 + i * 128, bar);
    }
}

// Instruction descriptor: BF16 operands, FP32 accumulators.
__device__ __forceinline__ uint32_t bf16_idesc(uint32_t m, uint32_t n, bool a_mn, bool b_mn)
{
    return f16_idesc(m, n, a_mn, b_mn) | (1u << 7) | (1u << 10);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// 32 columns of the lane's row as BF16: columns 32h.. of a piece of 64.
__device__ __forceinline__ void put_bf16(uint32_t piece, int lane, int h, const float (&v)[32])
{
    const uint32_t row = piece + lane * 128;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v[8 * q + 2 * e], v[8 * q + 2 * e + 1]);
            u[e] = *reinterpret_cast<const uint32_t *>(&x);
        }
        sts128(row + (((4 * h + q) ^ (lane & 7)) << 4), u[0], u[1], u[2], u[3]);
    }
}

__device__ __forceinline__ float exp2_approx(float x)  // 2 ulp, ex2.approx
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct Shared {
    uint64_t full[5], empty[5], acc_full[2], acc_empty[2];
    uint32_t tmem;
    volatile int abort;
};

// A warp's buffer for the next piece: the copy out of it that was issued two
// pieces ago has read it.
__device__ __forceinline__ uint32_t next_piece(uint32_t mine, uint32_t &pieces)
{
    if (elect_one())
        bulk_wait_read<kEpiBuffers - 1>();
    __syncwarp();
    return mine + (pieces++ % kEpiBuffers) * kPiece;
}

// The sums of a run of products, an epilogue warp's accumulators, are added to z.
__device__ __forceinline__ void add_run(float (&z)[128], uint32_t acc)
{
#pragma unroll
    for (int i = 0; i < 128; i += 16) {
        uint32_t raw[16];
        tmem_load16(acc + i, raw);
        tmem_wait_load();
#pragma unroll
        for (int e = 0; e < 16; ++e)
            z[i + e] += __uint_as_float(raw[e]);
    }
}

// z is added to the accumulators.
__device__ __forceinline__ void add_back(const float (&z)[128], uint32_t acc)
{
#pragma unroll
    for (int i = 0; i < 128; i += 16) {
        uint32_t raw[16];
        tmem_load16(acc + i, raw);
        tmem_wait_load();
#pragma unroll
        for (int e = 0; e < 16; ++e)
            raw[e] = __float_as_uint(z[i + e] + __uint_as_float(raw[e]));
        tmem_store16(acc + i, raw);
    }
    tmem_wait_store();
}

// One epilogue warp's part of a tile: 32 rows from row0 on, 128 columns from
// col0 on.  acc: its accumulators.
__device__ __forceinline__ void epilogue_logits(const LceProduct &p, int row0, int col0, int lane, uint32_t acc, uint32_t mine,
                                                uint32_t &pieces)
{
    const int row = row0 + lane;
    const bool in = row < p.rows;
    const int target = in ? p.target[row] : -1;
    const float ref = in ? p.ref[row] : 0.0f;
    const bool none = target == -1;  // padding, or beyond the last row
    float sum = 0.0f, top = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
        const int col = col0 + c;
        if (col >= p.cols)
            break;
        uint32_t raw[32];
        tmem_load32(acc + c, raw);
        tmem_wait_load();
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
            v[e] = __uint_as_float(raw[e]);
        // what does not count: columns beyond the last, the target's, rows of padding
        const int lim = p.cols - col, at = target - col;
        if (__any_sync(kFullMask, none || (unsigned)at < 32u) || lim < 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (none || e == at || e >= lim)
                    v[e] = -INFINITY;
        }
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 32; ++e)
            top = fmaxf(top, v[e]);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            v[e] = exp2_approx((v[e] - ref) * kLog2e);
            s += v[e];
        }
        sum += s;
        if (p.keep) {
            const int h = (c >> 5) & 1;
            const uint32_t piece = h == 0 ? next_piece(mine, pieces) : mine + ((pieces - 1) % kEpiBuffers) * kPiece;
            put_bf16(piece, lane, h, v);
            if (h == 1 || col + 32 >= p.cols) {
                fence_async_shared();
                __syncwarp();
                if (elect_one()) {
                    if (row0 < p.rows)
                        store_box(&p.out, piece, col & ~63, row0);
                    bulk_commit();
                }
                __syncwarp();
            }
        }
    }
    if (in && col0 < p.cols) {
        const int64_t at = (int64_t)(col0 >> 7) * p.pitch + row;
        p.sum[at] = sum;
        p.top[at] = top;
    }
}

__device__ __forceinline__ void epilogue_bf16(const LceProduct &p, int row0, int col0, int lane, uint32_t acc, uint32_t mine,
                                              uint32_t &pieces)
{
    const int row = row0 + lane;
    const float scale = p.kind == kLceScaled ? (row < p.rows ? p.scale[row] : 0.0f) : 1.0f;
#pragma unroll 1
    for (int c = 0; c < 128; c += 64) {
        if (col0 + c >= p.cols || row0 >= p.rows)
            break;
        const uint32_t piece = next_piece(mine, pieces);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            uint32_t raw[32];
            tmem_load32(acc + c + 32 * h, raw);
            tmem_wait_load();
            float v[32];
#pragma unroll
            for (int e = 0; e < 32; ++e)
                v[e] = scale == 0.0f ? 0.0f : scale * __uint_as_float(raw[e]);
            put_bf16(piece, lane, h, v);
        }
        fence_async_shared();
        __syncwarp();
        if (elect_one()) {
            store_box(&p.out, piece, col0 + c, row0);
            bulk_commit();
        }
        __syncwarp();
    }
}

__device__ __forceinline__ void epilogue_fp32(const LceProduct &p, int row0, int col0, int part, int lane, uint32_t acc,
                                              uint32_t mine, uint32_t &pieces)
{
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
        if (col0 + c >= p.cols || row0 >= p.rows)
            break;
        const uint32_t piece = next_piece(mine, pieces);
        uint32_t raw[32];
        tmem_load32(acc + c, raw);
        tmem_wait_load();
#pragma unroll
        for (int q = 0; q < 8; ++q)
            sts128(piece + lane * 128 + ((q ^ (lane & 7)) << 4), raw[4 * q], raw[4 * q + 1], raw[4 * q + 2], raw[4 * q + 3]);
        fence_async_shared();
        __syncwarp();
        if (elect_one()) {
            if (p.kind == kLceAdd)
                add_box(&p.out, piece, col0 + c, row0);
            else if (p.parts > 1)
                store_box3(&p.out, piece, col0 + c, row0, part);
            else
                store_box(&p.out, piece, col0 + c, row0);
            bulk_commit();
        }
        __syncwarp();
    }
}

// Sums of one run, or logits' or gradients' of more: these take 168 registers
// instead of 84.
enum LceForm { kOneRun = 0, kLogitRuns = 1, kGradientRuns = 2 };

template <int CG, int FORM>
__global__ void __launch_bounds__(kThreads, 1) k_lce_product(const __grid_constant__ LceProduct p)
{
    using R = Ring<CG>;
    constexpr bool LONG = FORM != kOneRun;
    constexpr int RUN = FORM == kLogitRuns ? kRun : kGradientRun;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;

    const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int first = blockIdx.x / CG, stride = gridDim.x / CG;
    const int tiles = tile_rows<CG>(p) * tile_cols(p) * p.parts;
    constexpr uint32_t kCols = 2 * kLceCols;

    if (p.again) {  // mostly there is nothing to do
        launch_dependents();
        wait_for_previous_grid();
        if (p.again[0] == 0)
            return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < R::kStages; ++s) {
            mbar_init(smem_addr(&sh.full[s]), 1);
            mbar_init(smem_addr(&sh.empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_addr(&sh.acc_full[a]), 1);
            mbar_init(smem_addr(&sh.acc_empty[a]), CG * kEpiWarps);
        }
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_shared();
    }
    if (warp == 1)
        tmem_alloc<CG>(smem_addr(&sh.tmem), kCols);
    tmem_fence_before();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    launch_dependents();
    wait_for_previous_grid();
    fence_async();  // what the previous launch wrote is read by the copy engine

    if (warp == 0) {
        uint32_t it = 0;
        bool ok = true;
        for (int t = first; ok && !p.test_stall && t < tiles; t += stride) {
            const Tile x = decode<CG>(p, t);
            if (!wanted<CG>(p, x))
                continue;
            const int k1 = first_step(p, x.part + 1);
            for (int k = first_step(p, x.part); k < k1; ++k, ++it) {
                const uint32_t s = it % R::kStages, ph = (it / R::kStages) & 1;
                ok = __all_sync(kFullMask, mbar_wait(smem_addr(&sh.empty[s]), ph ^ 1, &sh.abort));
                if (!ok)
                    break;
                const uint32_t slot = ring + s * R::kStage;
                const uint32_t bar = CG == 2 ? map_to_rank(smem_addr(&sh.full[s]), 0) : smem_addr(&sh.full[s]);
                const bool low = p.wrap && k >= p.wrap;
                const int at = low ? k - p.wrap : k;
                if (elect_one()) {
                    if (rank == 0)
                        mbar_expect_tx(smem_addr(&sh.full[s]), CG * R::kStage);
                    load_operand<CG>(slot, &p.a, p.a_mn, (x.i * CG + rank) * 128, 128, at, bar);
                    load_operand<CG>(slot + kBlock, low ? &p.b_low : &p.b, p.b_mn, x.j * kLceCols + rank * 128, R::kB / 128, at, bar);
                }
                __syncwarp();
            }
        }
        if (!ok) {
            sh.abort = 1;
            if (lane == 0)
                atomicOr(p.status, kStatusWaitLimit);
        }
        // the products of the last stages are done, so no copy is in flight and
        // no instruction reads the ring when the CTA ends
        for (uint32_t d = it > R::kStages ? it - R::kStages : 0; d < it; ++d)
            mbar_wait(smem_addr(&sh.empty[d % R::kStages]), (d / R::kStages) & 1, nullptr);
    } else if (warp == 1) {
        if (rank == 0) {
            uint32_t it = 0, n = 0;
            bool ok = true;
            const uint32_t idesc = bf16_idesc(128 * CG, kLceCols, p.a_mn, p.b_mn);
            const uint32_t a_step = (p.a_mn ? 2048 : 32) >> 4, b_step = (p.b_mn ? 2048 : 32) >> 4;
            for (int t = first; ok && t < tiles; t += stride) {
                const Tile x = decode<CG>(p, t);
                if (!wanted<CG>(p, x))
                    continue;
                const int last = first_step(p, x.part + 1);
                for (int k0 = first_step(p, x.part), k1; ok && k0 < last; k0 = k1, ++n) {
                    k1 = LONG && last - k0 > RUN ? k0 + RUN : last;
                    const uint32_t buf = n & 1, use = n >> 1;
                    ok = __all_sync(kFullMask, mbar_wait(smem_addr(&sh.acc_empty[buf]), (use & 1) ^ 1, &sh.abort));
                    if (!ok)
                        break;
                    tmem_fence_after();
                    for (int k = k0; k < k1; ++k, ++it) {
                        const uint32_t s = it % R::kStages, ph = (it / R::kStages) & 1;
                        ok = __all_sync(kFullMask, mbar_wait(smem_addr(&sh.full[s]), ph, &sh.abort));
                        if (!ok)
                            break;
                        tmem_fence_after();
                        const uint32_t slot = ring + s * R::kStage;
                        const uint64_t a_desc = operand_desc(slot, kBlock / 2), b_desc = operand_desc(slot + kBlock, kBlock / 2);
                        if (elect_one()) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mma_f16<CG>(tmem + buf * kLceCols, a_desc + j * a_step, b_desc + j * b_step, idesc,
                                            k > k0 || j > 0);
                            mma_commit<CG>(smem_addr(&sh.empty[s]));
                            if (k + 1 == k1)
                                mma_commit<CG>(smem_addr(&sh.acc_full[buf]));
                        }
                        __syncwarp();
                    }
                }
            }
            if (!ok) {
                sh.abort = 1;
                if (lane == 0)
                    atomicOr(p.status, kStatusWaitLimit);
            }
            // instructions in flight end before the CTA does
            for (uint32_t d = it > R::kStages ? it - R::kStages : 0; d < it; ++d)
                mbar_wait(smem_addr(&sh.empty[d % R::kStages]), (d / R::kStages) & 1, nullptr);
        }
    } else {
        // a warp reads the 32 lanes of tensor memory of its number mod 4
        const int quad = warp & 3, half = (warp - 2) >> 2;
        const uint32_t mine = ring + R::kStages * R::kStage + ((warp - 2) * kEpiBuffers) * kPiece;
        uint32_t n = 0, pieces = 0;
        bool ok = true;
        auto acc = [&] { return tmem + ((uint32_t)(quad * 32) << 16) + (n & 1) * kLceCols + half * 128; };
        auto wait_acc = [&] {
            const bool got = __all_sync(kFullMask, mbar_wait(smem_addr(&sh.acc_full[n & 1]), (n >> 1) & 1, &sh.abort));
            tmem_fence_after();
            return got;
        };
        auto free_acc = [&] {
            tmem_fence_before();
            __syncwarp();
            if (elect_one())
                mbar_arrive_cluster(map_to_rank(smem_addr(&sh.acc_empty[n & 1]), 0));
            __syncwarp();
            ++n;
        };
        for (int t = first; t < tiles; t += stride) {
            const Tile x = decode<CG>(p, t);
            if (!wanted<CG>(p, x))
                continue;
            const int row0 = (x.i * CG + (int)rank) * 128 + quad * 32, col0 = x.j * kLceCols + half * 128;
            if constexpr (LONG) {
                const int runs = (first_step(p, x.part + 1) - first_step(p, x.part) + RUN - 1) / RUN;
                float z[128];
#pragma unroll
                for (int e = 0; e < 128; ++e)
                    z[e] = 0.0f;
#pragma unroll 1
                for (int r = 1; r < runs && (ok = wait_acc()); ++r) {
                    add_run(z, acc());
                    free_acc();
                }
                if (ok && (ok = wait_acc()))
                    add_back(z, acc());
            } else {
                ok = wait_acc();
            }
            if (!ok)
                break;
            if (FORM == kLogitRuns || (FORM == kOneRun && p.kind == kLceLogits))
                epilogue_logits(p, row0, col0, lane, acc(), mine, pieces);
            else if (p.kind == kLceScaled || p.kind == kLcePlain)
                epilogue_bf16(p, row0, col0, lane, acc(), mine, pieces);
            else
                epilogue_fp32(p, row0, col0, x.part, lane, acc(), mine, pieces);
            free_acc();
        }
        bulk_wait<0>();
        if (!ok) {
            sh.abort = 1;
            if (lane == 0)
                atomicOr(p.status, kStatusWaitLimit);
        }
    }
    __syncwarp();
    tmem_fence_before();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tmem_fence_after();
    if (warp == 1)
        tmem_free<CG>(tmem, kCols);
}

constexpr int kMaxDevices = 64;

template <int CG>
void configure(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&at)[2], int groups, cudaStream_t stream)
{
    cfg.gridDim = dim3(groups * CG);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Ring<CG>::kSmem;
    cfg.stream = stream;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
}

// How many groups of CG CTAs the device holds at once (asked once per device).
template <int CG>
cudaError_t resident_groups(int device, int *groups)
{
    static std::atomic<int> cache[kMaxDevices];
    if (device < 0 || device >= kMaxDevices)
        return cudaErrorInvalidDevice;
    *groups = cache[device].load(std::memory_order_acquire);
    if (*groups > 0)
        return cudaSuccess;
    int sms = 0;
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    for (auto *kernel : {k_lce_product<CG, kOneRun>, k_lce_product<CG, kLogitRuns>, k_lce_product<CG, kGradientRuns>})
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<CG>::kSmem);
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    configure<CG>(cfg, at, sms / CG, nullptr);
    cfg.numAttrs = 1;
    if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveClusters(groups, k_lce_product<CG, kLogitRuns>, &cfg);
    if (e != cudaSuccess)
        return e;
    if (*groups < 1)
        return cudaErrorLaunchOutOfResources;
    *groups = *groups < sms / CG ? *groups : sms / CG;
    cache[device].store(*groups, std::memory_order_release);
    return cudaSuccess;
}

template <int CG>
cudaError_t launch(const LceProduct &p, int device, cudaStream_t stream)
{
    int groups = 0;
    const cudaError_t e = resident_groups<CG>(device, &groups);
    if (e != cudaSuccess)
        return e;
    const int tiles = tile_rows<CG>(p) * tile_cols(p) * p.parts;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at[2];
    configure<CG>(cfg, at, tiles < groups ? tiles : groups, stream);
    const bool logits = p.kind == kLceLogits;
    const int most = (p.k64 + p.parts - 1) / p.parts;  // steps of a part
    return most <= (logits ? kRun : kGradientRun) ? cudaLaunchKernelEx(&cfg, k_lce_product<CG, kOneRun>, p)
           : logits                               ? cudaLaunchKernelEx(&cfg, k_lce_product<CG, kLogitRuns>, p)
                                                  : cudaLaunchKernelEx(&cfg, k_lce_product<CG, kGradientRuns>, p);
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

}  // namespace

cudaError_t launch_lce_product(const LceProduct &p, int device, cudaStream_t stream)
{
    return lce_single(p.rows) ? launch<1>(p, device, stream) : launch<2>(p, device, stream);
}

cudaError_t lce_groups(int rows, int device, int *groups)
{
    return lce_single(rows) ? resident_groups<1>(device, groups) : resident_groups<2>(device, groups);
}

cudaError_t lce_map(CUtensorMap *map, const void *base, bool fp32, int64_t rows, int64_t cols, int64_t stride, int box_rows,
                    int slices, int64_t slice)
{
    static std::atomic<EncodeTiled> encode;
    EncodeTiled f = encode.load(std::memory_order_acquire);
    if (!f) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess)
            return e;
        if (found != cudaDriverEntryPointSuccess || !p)
            return cudaErrorNotSupported;
        f = reinterpret_cast<EncodeTiled>(p);
        encode.store(f, std::memory_order_release);
    }
    const cuuint64_t size = fp32 ? 4 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)slices};
    const cuuint64_t strides[2] = {(cuuint64_t)stride * size, (cuuint64_t)slice * size};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / size), (cuuint32_t)box_rows, 1}, step[3] = {1, 1, 1};
    const CUresult r = f(map, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, slices > 1 ? 3 : 2,
                         const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace slide
