// ortho_gemm.cu — the matrix products of the Newton-Schulz iteration on the
// fifth-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// Each product is D = A*B with FP16 operands and FP32 accumulators, followed
// by an epilogue that adds the FP32 part of the iterate and forms the operands
// of the next product (slide_ortho.h lists them).  All operands lie in the
// tiled layouts of slide_ortho.h, so the producer needs plain bulk copies
// only.
//
// A CTA is persistent over output tiles: warp 0 streams operand tiles into a
// ring of kStages stages, warp 1 issues the matrix instructions, and warps 2-9
// read finished accumulators from tensor memory, which holds two output tiles,
// so an epilogue overlaps the next tile's products.
//
// Why FP16 and where FP32 stays: FP16 rounds 8 times finer than BF16 at the
// same rate, and the iterates are bounded (the matrix is normalised first), so
// each operand is stored times a power of two that keeps it in range.  What is
// rounded enters the result only through a product with off-diagonal values:
// the diagonal of every left factor is kept apart in FP32 and applied to the
// FP32 copy of the iterate.  Off by 5e-4 to 1.2e-3 (2-norm over 2-norm) from
// the polynomial in 64 bits for spectra from flat to a single spike, where
// BF16 operands are 1e-2 to 1e-1 off.
#include <cuda_bf16.h>

#include <atomic>

#include "slide_ortho.h"
#include "sm103_ptx.h"

namespace slide {
namespace {

using namespace ptx;

constexpr int kStages = 5;
constexpr int kSlot = 16384;                      // one operand block: 128 x 64 FP16
constexpr int kStageBytes = 2 * kSlot;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kBounce = 32 * 33;                  // floats of a warp's transposing buffer
constexpr int kSmem = 1024 + kStages * kStageBytes + kEpiWarps * kBounce * 4;
constexpr unsigned kStatusWaitLimit = 2u;

struct Tile {
    int prob, b, i, j;
};

template <int CG>
__device__ __forceinline__ Tile decode(const OrthoGemm &g, int t)
{
    const int mt = (g.mblk + CG - 1) / CG, nt = (g.nblk + CG - 1) / CG;
    const int per = g.sym ? mt * (mt + 1) / 2 : mt * nt;
    const int z = t / per, r = t - z * per;
    Tile x;
    x.prob = z / g.batch;
    x.b = z - x.prob * g.batch;
    if (g.sym) {
        int j = (int)((sqrtf(8.0f * (float)r + 1.0f) - 1.0f) * 0.5f);
        while (j * (j + 1) / 2 > r)
            --j;
        while ((j + 1) * (j + 2) / 2 <= r)
            ++j;
        x.j = j;
        x.i = r - j * (j + 1) / 2;
    } else if (mt <= nt) {
        x.j = r / mt;
        x.i = r - x.j * mt;
    } else {
        x.i = r / nt;
        x.j = r - x.i * nt;
    }
    return x;
}

template <int CG>
__device__ __forceinline__ int tile_count(const OrthoGemm &g)
{
    const int mt = (g.mblk + CG - 1) / CG, nt = (g.nblk + CG - 1) / CG;
    return (g.sym ? mt * (mt + 1) / 2 : mt * nt) * g.batch * g.nprob;
}

// Whether step k of the operand whose tile has index t (in units of CG blocks)
// is read MN-major: a symmetric matrix keeps block (k, t) for k <= t.
template <int CG>
__device__ __forceinline__ bool reads_mn(int kind, int t, int k)
{
    return kind == kOperandSym ? (k >> 1) <= CG * t : kind == kOperandMN;
}

// Copy the 128 x 64 operand block (blk along M or N, step k) into a slot.
__device__ __forceinline__ void load_operand(uint32_t slot, const __half *m, int c64, int blk, int k, bool mn,
                                             uint32_t bar)
{
    if (mn) {
        const __half *t = m + ((int64_t)(k >> 1) * c64 + 2 * blk) * kTileElems16 + (k & 1) * (kTileElems16 / 2);
        bulk_load(slot, t, kSlot / 2, bar);
        bulk_load(slot + kSlot / 2, t + kTileElems16, kSlot / 2, bar);
    } else {
        bulk_load(slot, m + ((int64_t)blk * c64 + k) * kTileElems16, kSlot, bar);
    }
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Row r's 32 values at chunk offset `c` (4 chunks of 8) of a T16 tile.
__device__ __forceinline__ void store16(__half *tile, int r, int c, const float (&v)[32], float s)
{
    uint4 *row = reinterpret_cast<uint4 *>(tile + r * 64);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint4 x;
        x.x = pack_half2(v[8 * q] * s, v[8 * q + 1] * s);
        x.y = pack_half2(v[8 * q + 2] * s, v[8 * q + 3] * s);
        x.z = pack_half2(v[8 * q + 4] * s, v[8 * q + 5] * s);
        x.w = pack_half2(v[8 * q + 6] * s, v[8 * q + 7] * s);
        row[(c + q) ^ (r & 7)] = x;
    }
}

__device__ __forceinline__ void store32(float *tile, int r, const float (&v)[32])
{
    float4 *row = reinterpret_cast<float4 *>(tile + r * 32);
#pragma unroll
    for (int q = 0; q < 8; ++q)
        row[q ^ (r & 7)] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
}

template <int CG, int EPI>
__device__ __forceinline__ void epilogue_chunk(const OrthoGemm &g, const Tile &x, int ib, int jb, int row, int q,
                                               const uint32_t (&acc)[32], float *bounce, int lane)
{
    // q: 32-column chunk of the 128-block jb
    const OrthoOperands &p = g.p[x.prob];
    const int64_t t16 = (int64_t)x.b * g.out_stride + ((int64_t)ib * g.out_c64 + 2 * jb + (q >> 1)) * kTileElems16;
    const int64_t t32 = (int64_t)x.b * g.out_stride + ((int64_t)ib * g.out_c64 * 2 + 4 * jb + q) * kTileElems32;
    const int gi = ib * 128 + row, gj = jb * 128 + q * 32;
    const int on_diag = g.sym && gi >= gj && gi < gj + 32 ? gi - gj : -1;
    float v[32];
#pragma unroll
    for (int e = 0; e < 32; ++e)
        v[e] = __uint_as_float(acc[e]) * g.alpha;

    if constexpr (EPI == kEpiPoly) {
        const uint4 *crow = reinterpret_cast<const uint4 *>(p.c16 + t16 + row * 64);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 w = crow[((q & 1) * 4 + c) ^ (row & 7)];
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[h]));
                v[8 * c + 2 * h] += g.c16_scale * f.x;
                v[8 * c + 2 * h + 1] += g.c16_scale * f.y;
            }
        }
    }
    if constexpr (EPI == kEpiSym || EPI == kEpiApply || EPI == kEpiOut || EPI == kEpiMuon) {
        const float4 *crow = reinterpret_cast<const float4 *>(p.c32 + t32 + row * 32);
        const float *d = p.dvec + (int64_t)x.b * g.d_stride;
        const float inv = g.c_inv ? g.c_inv[x.b] : 1.0f;
        const float dr = g.d_by_col ? inv : inv * d[gi];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float4 w = crow[c ^ (row & 7)];
            float4 dc = make_float4(dr, dr, dr, dr);
            if (g.d_by_col) {
                const float4 k = *reinterpret_cast<const float4 *>(d + gj + 4 * c);
                dc = make_float4(dr * k.x, dr * k.y, dr * k.z, dr * k.w);
            }
            v[4 * c] = fmaf(dc.x, w.x, v[4 * c]);
            v[4 * c + 1] = fmaf(dc.y, w.y, v[4 * c + 1]);
            v[4 * c + 2] = fmaf(dc.z, w.z, v[4 * c + 2]);
            v[4 * c + 3] = fmaf(dc.w, w.w, v[4 * c + 3]);
        }
    }

    if constexpr (EPI == kEpiPoly) {
        float dd = 0.0f;
        if (p.out32) {  // Q = aI + B, with its diagonal
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                if (e == on_diag) {
                    v[e] += g.coef_a;
                    dd = v[e];
                }
            }
            store32(p.out32 + t32, row, v);
            store16(p.out16b + t16, row, (q & 1) * 4, v, g.s16b);
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (e == on_diag)
                    v[e] = 0.0f;
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                if (e == on_diag) {
                    dd = v[e] + g.coef_a;
                    v[e] = 0.0f;
                }
            }
        }
        if (on_diag >= 0)
            p.dvec_out[(int64_t)x.b * g.d_stride + gi] = dd;
        store16(p.out16 + t16, row, (q & 1) * 4, v, g.s16);
    } else if constexpr (EPI == kEpiOut || EPI == kEpiMuon) {
        // through the warp's buffer, so that a warp writes along the rows
#pragma unroll
        for (int e = 0; e < 32; ++e)
            bounce[lane * 33 + e] = v[e];
        __syncwarp();
        const int col = gj + lane;
        const int row0 = ib * 128 + (row & ~31);
        const int lim = min(32, g.rows - row0);
        if (col < g.cols) {
            for (int r = 0; r < lim; ++r) {
                float o = bounce[r * 33 + lane];
                if constexpr (EPI == kEpiMuon) {
                    const int64_t at = ((int64_t)x.b * g.rows + row0 + r) * g.cols + col;
                    o = __fsub_rn(__fmul_rn(g.theta[at], g.decay), __fmul_rn(g.step, o));
                    g.theta[at] = o;
                    g.w[at] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
                } else {
                    g.w[(int64_t)x.b * g.w_batch + (int64_t)(row0 + r) * g.w_row + col] =
                        __bfloat16_as_ushort(__float2bfloat16_rn(o));
                }
            }
        }
        __syncwarp();
    } else {
        if (p.out32)
            store32(p.out32 + t32, row, v);
        if constexpr (EPI == kEpiSym) {
            if (g.diag_out && on_diag >= 0) {
                float dd = 0.0f;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    if (e == on_diag) {
                        dd = v[e];
                        v[e] = 0.0f;
                    }
                }
                p.dvec_out[(int64_t)x.b * g.d_stride + gi] = dd;
            }
        }
        store16(p.out16 + t16, row, (q & 1) * 4, v, g.s16);
    }
}

template <int CG, int EPI>
__global__ void __launch_bounds__(kThreads, 1) k_ortho_gemm(const __grid_constant__ OrthoGemm g)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages], s_peer[kStages], s_acc_full[2], s_acc_empty[2];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;

    const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
    float *bounce_all = reinterpret_cast<float *>(smem_raw + (ring - smem_addr(smem_raw)) + kStages * kStageBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int first = blockIdx.x / CG, stride = gridDim.x / CG;
    constexpr uint32_t kCols = 2 * 128 * CG;  // two accumulators of 128*CG columns

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&s_full[s]), 1);
            mbar_init(smem_addr(&s_empty[s]), 1);
            mbar_init(smem_addr(&s_peer[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_addr(&s_acc_full[a]), 1);
            mbar_init(smem_addr(&s_acc_empty[a]), CG * kEpiWarps);
        }
        s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_shared();
    }
    if (warp == 1)
        tmem_alloc<CG>(smem_addr(&s_tmem), kCols);
    tmem_fence_before();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = s_tmem;
    // a launch behind one whose wait ran out does nothing
    const int total = (*(volatile unsigned *)g.status & kStatusWaitLimit) ? 0 : tile_count<CG>(g);
    // both CTAs of a pair have to agree on that
    int n_tiles = total;
    if constexpr (CG == 2) {
        __shared__ int s_total;
        if (threadIdx.x == 0 && rank == 0) {
            const uint32_t mine = smem_addr(&s_total);
            for (uint32_t r = 0; r < 2; ++r)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_rank(mine, r)), "r"(total) : "memory");
        }
        cluster_sync();
        n_tiles = s_total;
    }

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = first; t < n_tiles && ok && !g.test_stall; t += stride) {
                const Tile x = decode<CG>(g, t);
                const __half *a = g.p[x.prob].a + (int64_t)x.b * g.a_stride;
                const __half *b = g.p[x.prob].b + (int64_t)x.b * g.b_stride;
                for (int k = 0; k < g.k64; ++k, ++it) {
                    const uint32_t s = it % kStages, ph = (it / kStages) & 1;
                    if (!mbar_wait(smem_addr(&s_empty[s]), ph ^ 1, &s_abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = smem_addr(&s_full[s]), slot = ring + s * kStageBytes;
                    mbar_expect_tx(bar, kStageBytes);
                    load_operand(slot, a, g.a_c64, x.i * CG + rank, k, reads_mn<CG>(g.a_kind, x.i, k), bar);
                    load_operand(slot + kSlot, b, g.b_c64, x.j * CG + rank, k, reads_mn<CG>(g.b_kind, x.j, k), bar);
                }
            }
            if (!ok)
                s_abort = 1;
            // copies in flight land before the CTA ends
            for (uint32_t d = it > kStages ? it - kStages : 0; d < it; ++d) {
                volatile int never = 0;
                mbar_wait(smem_addr(&s_full[d % kStages]), (d / kStages) & 1, &never);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (int t = first; t < n_tiles && ok; t += stride, ++n) {
                const Tile x = decode<CG>(g, t);
                const uint32_t buf = n & 1, use = n >> 1;
                if (rank == 0 && !mbar_wait(smem_addr(&s_acc_empty[buf]), (use & 1) ^ 1, &s_abort)) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                for (int k = 0; k < g.k64; ++k, ++it) {
                    const uint32_t s = it % kStages, ph = (it / kStages) & 1;
                    ok = mbar_wait(smem_addr(&s_full[s]), ph, &s_abort);
                    if (ok && CG == 2) {
                        if (rank == 0)
                            ok = mbar_wait(smem_addr(&s_peer[s]), ph, &s_abort);
                        else
                            mbar_arrive_cluster(map_to_rank(smem_addr(&s_peer[s]), 0));
                    }
                    if (!ok)
                        break;
                    if (rank != 0)
                        continue;
                    tmem_fence_after();
                    const bool a_mn = reads_mn<CG>(g.a_kind, x.i, k), b_mn = reads_mn<CG>(g.b_kind, x.j, k);
                    const uint32_t idesc = f16_idesc(128 * CG, 128 * CG, a_mn, b_mn);
                    const uint32_t slot = ring + s * kStageBytes;
                    const uint32_t a_step = a_mn ? 2048 : 32, b_step = b_mn ? 2048 : 32;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_f16<CG>(tmem + buf * 128 * CG, operand_desc(slot + j * a_step, kSlot / 2),
                                    operand_desc(slot + kSlot + j * b_step, kSlot / 2), idesc, k > 0 || j > 0);
                    mma_commit<CG>(smem_addr(&s_empty[s]));
                }
                if (ok && rank == 0)
                    mma_commit<CG>(smem_addr(&s_acc_full[buf]));
            }
            if (!ok) {
                s_abort = 1;
                atomicOr(g.status, kStatusWaitLimit);
            }
            // the matrix instructions in flight end before the CTA does: the
            // commits of the last stages have arrived
            for (uint32_t d = it > kStages ? it - kStages : 0; d < it; ++d) {
                volatile int never = 0;
                mbar_wait(smem_addr(&s_empty[d % kStages]), (d / kStages) & 1, &never);
            }
        }
    } else {
        const int quad = warp & 3, half = (warp - 2) >> 2;
        float *bounce = bounce_all + (warp - 2) * kBounce;
        const int row = quad * 32 + lane;
        uint32_t n = 0;
        for (int t = first; t < n_tiles; t += stride, ++n) {
            const Tile x = decode<CG>(g, t);
            const uint32_t buf = n & 1, use = n >> 1;
            const bool ok = mbar_wait(smem_addr(&s_acc_full[buf]), use & 1, &s_abort);
            if (!__all_sync(0xffffffffu, ok)) {
                s_abort = 1;
                if (lane == 0)
                    atomicOr(g.status, kStatusWaitLimit);
                break;
            }
            tmem_fence_after();
            const int ib = x.i * CG + rank;
            for (int c = half; c < 4 * CG; c += 2) {
                uint32_t acc[32];
                tmem_load32(tmem + ((uint32_t)(quad * 32) << 16) + buf * 128 * CG + c * 32, acc);
                tmem_wait_load();
                const int jb = x.j * CG + (c >> 2);
                if (ib >= g.mblk || jb >= g.nblk || (g.sym && ib > jb))
                    continue;
                epilogue_chunk<CG, EPI>(g, x, ib, jb, row, c & 3, acc, bounce, lane);
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(map_to_rank(smem_addr(&s_acc_empty[buf]), 0));
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

template <int CG, int EPI>
cudaError_t launch(const OrthoGemm &g, int device, cudaStream_t stream)
{
    static std::atomic<int> sms[kMaxDevices];
    int n = sms[device].load(std::memory_order_acquire);
    if (n == 0) {
        cudaError_t e = cudaFuncSetAttribute(k_ortho_gemm<CG, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e == cudaSuccess)
            e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device);
        if (e != cudaSuccess)
            return e;
        sms[device].store(n, std::memory_order_release);
    }
    const int mt = (g.mblk + CG - 1) / CG, nt = (g.nblk + CG - 1) / CG;
    const int64_t tiles = (int64_t)(g.sym ? mt * (mt + 1) / 2 : mt * nt) * g.batch * g.nprob;
    const int groups = (int)(tiles < n / CG ? tiles : n / CG);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(groups * CG);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_ortho_gemm<CG, EPI>, g);
}

template <int CG>
cudaError_t launch_epi(const OrthoGemm &g, int epi, int device, cudaStream_t stream)
{
    switch (epi) {
    case kEpiGram: return launch<CG, kEpiGram>(g, device, stream);
    case kEpiPoly: return launch<CG, kEpiPoly>(g, device, stream);
    case kEpiSym: return launch<CG, kEpiSym>(g, device, stream);
    case kEpiApply: return launch<CG, kEpiApply>(g, device, stream);
    case kEpiOut: return launch<CG, kEpiOut>(g, device, stream);
    default: return launch<CG, kEpiMuon>(g, device, stream);
    }
}

}  // namespace

cudaError_t launch_ortho_gemm(const OrthoGemm &g, int epi, int device, cudaStream_t stream)
{
    if (device < 0 || device >= kMaxDevices)
        return cudaErrorInvalidDevice;
    return launch_epi<1>(g, epi, device, stream);
}

}  // namespace slide
