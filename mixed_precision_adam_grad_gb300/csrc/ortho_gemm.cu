// ortho_gemm.cu — the matrix products of the Newton-Schulz iteration on the
// fifth-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// Each product is D = A*B with FP16 operands and FP32 accumulators, followed
// by an epilogue that adds the diagonal's part of the left factor times the
// iterate and forms the operands of the next product (slide_ortho.h lists
// them).  All operands lie in the
// tiled layouts of slide_ortho.h, so the producer needs plain bulk copies
// only.
//
// A CTA is persistent over output tiles: warp 0 streams operand tiles into a
// ring of kStages stages, warp 1 issues the matrix instructions, and warps 2-9
// read finished accumulators from tensor memory, which holds two output tiles,
// so an epilogue overlaps the next tile's products.  An epilogue warp takes 32
// rows x 64 columns at a time: it copies their C into its own buffer (for the
// first chunk of a tile before the product is ready, for both of its chunks
// where only the high half is kept), replaces it by the result and writes that
// from there, all with bulk copies of 4 KiB.  (Low halves through registers
// instead, in 32-byte sectors, made room for a sixth stage, but the phases that
// have them took 15 to 50 % longer.)
//
// One launch runs all the products of an iteration (a cooperative launch, so all
// CTAs are resident).  The tiles of all phases, phase after phase and matrix
// after matrix, form one sequence that the CTAs share out in turn.  A CTA whose
// tile is written counts it for its matrix and phase, and nobody reads for a tile
// of the next phase before that count is full: matrices of a batch do not wait
// for one another, and a phase's last, partly filled round of tiles runs beside
// the next phase's first.  (With a barrier of all CTAs after each phase 40
// matrices of 1000 x 2187 took 1476 us instead of 1320, with a launch for each
// phase another 2 us a phase.)  The counts are watched by a warp of its own,
// the last, which goes ahead of the others and tells them in shared memory how
// far they may read: the 0.7 us that a look at a count takes would otherwise
// stand between two tiles' loads (1428 us; with the look in the middle of the
// tile before, 1350).
//
// Bound by the matrix instructions, or what L2 delivers to them, where there are
// tiles for all SMs: 5120 x 17408 3.2 ms (1.14 PFLOP/s of the operations that
// the formula needs, more with whole blocks on the diagonals), 40 of 1000 x 2187
// 1.24 ms.  Few and small matrices are bound by the 15 to 17 dependent phases,
// about 4.5 us each besides their products: a Muon step of 228 x 705 107 us; the
// tensor pipe is busy 14 % of the time with 2 of 1024 x 2560.
//
// Why FP16 and where FP32 stays: FP16 rounds 8 times finer than BF16 at the
// same rate, and the iterates are bounded (the matrix is normalised first), so
// each operand is stored times a power of two that keeps it in range.  What is
// rounded enters the result only through a product with off-diagonal values:
// the diagonal of every left factor is kept apart in FP32 and applied to the
// iterate's full 22 bits.  Off by 5e-4 to 1.2e-3 (2-norm over 2-norm) from
// the polynomial in 64 bits for noise with or without strong directions, where
// BF16 operands are 1e-2 to 1e-1 off; ortho.cu says what a wider spectrum costs.
#include <cuda_bf16.h>

#include <atomic>
#include <cmath>

#include "slide_ortho.h"
#include "sm103_ptx.h"

namespace slide {
namespace {

using namespace ptx;

constexpr int kStages = 5;
constexpr int kSlot = 16384;                      // one operand block: 128 x 64 FP16
constexpr int kStageBytes = 2 * kSlot;
constexpr int kEpiWarps = 8;
constexpr int kWatchWarp = 2 + kEpiWarps;
constexpr int kThreads = (kWatchWarp + 1) * 32;
constexpr int kPiece = 4096;                      // 32 rows of a tile
constexpr int kEpiBytes = 2 * kPiece;             // an epilogue warp's buffer: hi and lo of a chunk, or hi of two
constexpr int kSmem = 1024 + kStages * kStageBytes + kEpiWarps * kEpiBytes;
constexpr int kMaxParts = 8;  // of a Gram matrix's K
constexpr unsigned kFullMask = 0xffffffffu;

struct Tile {
    int prob, b, i, j;
    int half;   // of the tile's columns, where it is narrow
    int part;   // of the K of the tile, where it is split
    int index;  // of the tile among those of all matrices (halves and parts not counted)
};

template <int CG>
__device__ __forceinline__ Tile decode(const OrthoGemm &g, int t)
{
    const int mt = (g.mblk + CG - 1) / CG, nt = (g.nblk + CG - 1) / CG;
    const int per = g.sym ? mt * (mt + 1) / 2 : mt * nt;
    Tile x;
    x.index = t;
    x.part = x.half = 0;
    if (CG == 1 && g.parts > 1) {
        x.index = t / g.parts;
        x.part = t - x.index * g.parts;
    }
    if (CG == 1 && g.narrow) {
        x.half = x.index & 1;
        x.index >>= 1;
    }
    const int z = x.index / per, r = x.index - z * per;
    x.b = z / g.nprob;
    x.prob = z - x.b * g.nprob;
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

// Tiles of one matrix, each half and part of one counted.
template <int CG>
__host__ __device__ __forceinline__ int tile_count(const OrthoGemm &g)
{
    const int mt = (g.mblk + CG - 1) / CG, nt = (g.nblk + CG - 1) / CG;
    return (g.sym ? mt * (mt + 1) / 2 : mt * nt) * g.nprob * g.parts * (g.narrow ? 2 : 1);
}

// The first step of a part of K (pairs of CTAs take all of it).
template <int CG>
__device__ __forceinline__ int first_step(const OrthoGemm &g, int part)
{
    return CG == 2 || g.parts == 1 ? part * g.k64 : part * g.k64 / g.parts;
}

// A position in the sequence of all tiles.
template <int CG>
struct Walk {
    int f = 0;          // phase
    int64_t base = 0;   // tiles before it
    int64_t here;       // tiles in it
    __device__ __forceinline__ explicit Walk(const OrthoPlan &plan) : here((int64_t)tile_count<CG>(plan.ph[0]) * plan.batch) {}
    // Moves on to tile t (never back); false beyond the last.
    __device__ __forceinline__ bool to(const OrthoPlan &plan, int64_t t)
    {
        while (t - base >= here) {
            base += here;
            if (++f == plan.n_phases)
                return false;
            here = (int64_t)tile_count<CG>(plan.ph[f]) * plan.batch;
        }
        return true;
    }
};

// Whether step k of the operand whose tile has index t (in units of CG blocks)
// is read MN-major: a symmetric matrix keeps block (k, t) for k <= t.
template <int CG>
__device__ __forceinline__ bool reads_mn(int kind, int t, int k)
{
    return kind == kOperandSym ? (k >> 1) <= CG * t : kind == kOperandMN;
}

// Copy the 128 x 64 operand block (blk along M or N, step k) into a slot, or of
// a narrow tile's B half of it, 64 x 64.
__device__ __forceinline__ void load_half_operand(uint32_t slot, const __half *m, int c64, int blk, int half, int k,
                                                  bool mn, uint32_t bar)
{
    const __half *t = mn ? m + ((int64_t)(k >> 1) * c64 + 2 * blk + half) * kTileElems + (k & 1) * (kTileElems / 2)
                         : m + ((int64_t)blk * c64 + k) * kTileElems + half * (kTileElems / 2);
    bulk_load(slot, t, kSlot / 2, bar);
}

__device__ __forceinline__ void load_operand(uint32_t slot, const __half *m, int c64, int blk, int k, bool mn,
                                             uint32_t bar)
{
    if (mn) {
        const __half *t = m + ((int64_t)(k >> 1) * c64 + 2 * blk) * kTileElems + (k & 1) * (kTileElems / 2);
        bulk_load(slot, t, kSlot / 2, bar);
        bulk_load(slot + kSlot / 2, t + kTileElems, kSlot / 2, bar);
    } else {
        bulk_load(slot, m + ((int64_t)blk * c64 + k) * kTileElems, kSlot, bar);
    }
}

__device__ __forceinline__ uint32_t pack_half2(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ float2 unpack_half2(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2 *>(&u)); }

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float lds32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint16_t lds16(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Columns 32h..32h+31 of the lane's row of a 64-column piece: the high halves.
__device__ __forceinline__ void put_hi(uint32_t piece, int lane, int h, const float (&v)[32], float s)
{
    const uint32_t row = piece + lane * 128;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            u[e] = pack_half2(__floats2half2_rn(v[8 * q + 2 * e] * s, v[8 * q + 2 * e + 1] * s));
        sts128(row + (((4 * h + q) ^ (lane & 7)) << 4), make_uint4(u[0], u[1], u[2], u[3]));
    }
}

// High and low halves, into the piece and the one behind it.
__device__ __forceinline__ void put_pair(uint32_t piece, int lane, int h, const float (&v)[32], float s)
{
    const uint32_t row = piece + lane * 128;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t u[4], w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = v[8 * q + 2 * e] * s, y = v[8 * q + 2 * e + 1] * s;
            const __half2 k = __floats2half2_rn(x, y);
            const float2 f = __half22float2(k);
            u[e] = pack_half2(k);
            w[e] = pack_half2(__floats2half2_rn((x - f.x) * kLoScale, (y - f.y) * kLoScale));
        }
        const uint32_t c = row + (((4 * h + q) ^ (lane & 7)) << 4);
        sts128(c, make_uint4(u[0], u[1], u[2], u[3]));
        sts128(c + kPiece, make_uint4(w[0], w[1], w[2], w[3]));
    }
}

// Four floats, loaded where they are used (all of a chunk's at once would not
// fit into the registers).
__device__ __forceinline__ float4 load_here(const float *p)
{
    float4 v;
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}

// Whether an epilogue has a C.
template <int EPI>
constexpr bool kHasC = EPI != kEpiGram;

// How C enters: hi times one factor; hi and lo times the row's factor; hi times
// the row's and lo times the column's (EpilogueKind: dvec2); hi and lo times
// the column's factor.
enum CMode { kCHigh = 0, kCRow = 1, kCTwo = 2, kCCol = 3, kCParts = 4 };

// What a warp needs of a product's arguments, in registers.
struct Local {
    float alpha, s_out, d_row, col_scale, eye;
    const float *d_col;   // of the matrix; kCTwo, kCCol
    float *d_out;         // of the matrix; NULL: the diagonal stays
    __half *out_hi, *out_lo;  // out_lo NULL: only the high half is kept
    int parts, slot, warp;    // of a Gram matrix: the first part's slot, the warp's place
};

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
        sts128(row + (((4 * h + q) ^ (lane & 7)) << 4), make_uint4(u[0], u[1], u[2], u[3]));
    }
}

// The orthogonal factor goes to the weights' update through 16-bit shared
// memory: FP16 times this, 2^-12 of the value off, a tenth of the factor's own
// error, and the weights stay in FP32.
constexpr float kMuonScale = 256.0f;

__device__ __forceinline__ float muon_weight(const OrthoPlan &plan, float th, float o)
{
    return __fsub_rn(__fmul_rn(th, plan.decay), __fmul_rn(plan.step, o * (1.0f / kMuonScale)));
}

// Writes a piece (32 rows from row0, 64 columns from gj) to the caller's
// array, along the rows: eight lanes a row where vectors fit, else one row at a
// time, 32 neighbouring columns together.  A Muon step's weights come through
// the place behind the piece, 16 rows at a time: that many loads in flight take
// no registers.  (Four rows and sixteen in registers made all epilogues spill
// them to memory, 40 matrices of 1000 x 2187 took 1360 us instead of 1235; one
// row and eight 464 us instead of 449 for a Muon step of 7 of 1001 x 2731.)
template <int EPI>
__device__ __forceinline__ void write_rows(const OrthoPlan &plan, int b, int row0, int gj, int lane, uint32_t buf)
{
    const int64_t next = EPI == kEpiMuon ? plan.cols : plan.w_row;
    const int64_t at0 = EPI == kEpiMuon ? ((int64_t)b * plan.rows + row0) * plan.cols + gj
                                        : (int64_t)b * plan.w_batch + (int64_t)row0 * plan.w_row + gj;
    const int lim = min(32, plan.rows - row0), n = plan.cols - gj;
    const bool vec = plan.vec && n >= 64;
    constexpr int kAtOnce = 16;
    const uint32_t stage = buf + kPiece;  // [kAtOnce][64] floats, each written and read by the same lane
#pragma unroll 1
    for (int r0 = 0; r0 < lim; r0 += kAtOnce) {
        const int r1 = min(kAtOnce, lim - r0);
        if (vec) {
            const int c = lane & 7;
            if constexpr (EPI == kEpiMuon) {
                for (int r = lane >> 3; r < r1; r += 4) {
                    const float *th = plan.theta + at0 + (r0 + r) * next + c * 8;
                    copy_async16(stage + r * 256 + c * 32, th);
                    copy_async16(stage + r * 256 + c * 32 + 16, th + 4);
                }
                copy_async_wait();
            }
            for (int r = lane >> 3; r < r1; r += 4) {
                const int64_t at = at0 + (r0 + r) * next + c * 8;
                uint4 w = lds128(buf + (r0 + r) * 128 + ((c ^ (r & 7)) << 4));
                if constexpr (EPI == kEpiMuon) {
                    const uint4 lo = lds128(stage + r * 256 + c * 32), hi = lds128(stage + r * 256 + c * 32 + 16);
                    uint32_t th[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                    uint32_t y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 o = unpack_half2(u[e]);
                        const float p = muon_weight(plan, __uint_as_float(th[2 * e]), o.x);
                        const float q = muon_weight(plan, __uint_as_float(th[2 * e + 1]), o.y);
                        th[2 * e] = __float_as_uint(p);
                        th[2 * e + 1] = __float_as_uint(q);
                        const __nv_bfloat162 z = __floats2bfloat162_rn(p, q);
                        y[e] = *reinterpret_cast<const uint32_t *>(&z);
                    }
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(plan.theta + at),
                                 "r"(th[0]), "r"(th[1]), "r"(th[2]), "r"(th[3]), "r"(th[4]), "r"(th[5]), "r"(th[6]), "r"(th[7])
                                 : "memory");
                    w = make_uint4(y[0], y[1], y[2], y[3]);
                }
                *reinterpret_cast<uint4 *>(plan.w + at) = w;
            }
        } else {
            if constexpr (EPI == kEpiMuon) {
                for (int col = lane; col < min(n, 64); col += 32)
                    for (int r = 0; r < r1; ++r)
                        copy_async4(stage + r * 256 + col * 4, plan.theta + at0 + (r0 + r) * next + col);
                copy_async_wait();
            }
            for (int col = lane; col < min(n, 64); col += 32) {
#pragma unroll 4
                for (int r = 0; r < r1; ++r) {
                    const int64_t at = at0 + (r0 + r) * next + col;
                    uint16_t u = lds16(buf + (r0 + r) * 128 + (((col >> 3) ^ (r & 7)) << 4) + (lane & 7) * 2);
                    if constexpr (EPI == kEpiMuon) {
                        const float p = muon_weight(plan, lds32(stage + r * 256 + col * 4), __half2float(__ushort_as_half(u)));
                        u = __bfloat16_as_ushort(__float2bfloat16_rn(p));
                        __stcs(plan.theta + at, p);
                    }
                    plan.w[at] = u;
                }
            }
        }
    }
}

__device__ __forceinline__ void read_half(uint32_t piece, int lane, int h, uint32_t *w)
{
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 x = lds128(piece + lane * 128 + (((4 * h + q) ^ (lane & 7)) << 4));
        w[4 * q] = x.x, w[4 * q + 1] = x.y, w[4 * q + 2] = x.z, w[4 * q + 3] = x.w;
    }
}

// A tile of a Gram matrix whose K is split: each part's sums of a warp's 32 rows
// x 64 columns, FP32, half after half, four columns of all lanes together.
constexpr int kPartElems = 32 * 64;

// Where a warp's lie: the slots of a matrix, of 128 x 128 values each, fill the
// areas one after another.
__device__ __forceinline__ float *part_at(const OrthoPlan &plan, int b, int slot, int warp)
{
    const int area = slot / plan.area_slots;
    return plan.area[area] + b * plan.area_matrix + (int64_t)(slot - area * plan.area_slots) * (kEpiWarps * kPartElems) +
           warp * kPartElems;
}

__device__ __forceinline__ void leave_part(float *to, int lane, uint32_t acc_addr)
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t acc[32];
        tmem_load32(acc_addr + h * 32, acc);
        tmem_wait_load();
#pragma unroll
        for (int q = 0; q < 8; ++q)
            __stcg(reinterpret_cast<uint4 *>(to) + (h * 8 + q) * 32 + lane,
                   make_uint4(acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]));
    }
}

// Half h of their sum, part after part.
__device__ __forceinline__ void add_parts(const OrthoPlan &plan, const Local &k, int b, int lane, int h, uint32_t (&sum)[32])
{
#pragma unroll
    for (int e = 0; e < 32; ++e)
        sum[e] = 0u;
#pragma unroll 2
    for (int p = 0; p < k.parts; ++p) {
        const float4 *from = reinterpret_cast<const float4 *>(part_at(plan, b, k.slot + p, k.warp)) + h * 256 + lane;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float4 w = __ldcg(from + q * 32);
            const float x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum[4 * q + e] = __float_as_uint(__uint_as_float(sum[4 * q + e]) + x[e]);
        }
    }
}

// One chunk: this warp's 32 rows (the lane's is gi) x 64 columns from gj on, in
// two halves; a loop, not unrolled, since a CTA that comes to a phase for a
// tile or two waits for its instructions (2 matrices of 1024 x 2560 234 us
// unrolled, 221 as a loop; a single piece of code for all kinds of epilogues
// again 230).
// buf holds C (hi, and lo behind it) and is where results leave from; at: the
// chunk's place in the operands, in values.
template <int EPI, int MODE>
__device__ __forceinline__ void epilogue_chunk(const OrthoPlan &plan, const Local &k, int b, int gi, int gj, int lane,
                                               uint32_t acc_addr, uint32_t buf, int64_t at)
{
    uint32_t chi[kHasC<EPI> ? 16 : 1], clo[MODE == kCHigh || MODE == kCParts ? 1 : 16];
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        uint32_t acc[32];
        if constexpr (MODE == kCParts)
            add_parts(plan, k, b, lane, h, acc);
        else
            tmem_load32(acc_addr + h * 32, acc);
        if constexpr (kHasC<EPI>)
            read_half(buf, lane, h, chi);
        if constexpr (MODE != kCHigh && MODE != kCParts)
            read_half(buf + kPiece, lane, h, clo);
        tmem_wait_load();
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
            v[e] = __uint_as_float(acc[e]) * k.alpha;
        if constexpr (kHasC<EPI>) {
#pragma unroll
            for (int e4 = 0; e4 < 8; ++e4) {
                float col[4];
                if constexpr (MODE == kCTwo || MODE == kCCol) {
                    const float4 w = load_here(k.d_col + gj + 32 * h + 4 * e4);
                    col[0] = w.x * k.col_scale, col[1] = w.y * k.col_scale, col[2] = w.z * k.col_scale, col[3] = w.w * k.col_scale;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 f = unpack_half2(chi[2 * e4 + e]);
                    float *y = v + 4 * e4 + 2 * e;
                    if constexpr (MODE == kCHigh) {
                        y[0] = fmaf(k.d_row, f.x, y[0]);
                        y[1] = fmaf(k.d_row, f.y, y[1]);
                    } else {
                        const float2 l = unpack_half2(clo[2 * e4 + e]);
                        if constexpr (MODE == kCTwo) {
                            y[0] = fmaf(k.d_row, f.x, fmaf(col[2 * e], l.x, y[0]));
                            y[1] = fmaf(k.d_row, f.y, fmaf(col[2 * e + 1], l.y, y[1]));
                        } else {
                            const float d0 = MODE == kCCol ? col[2 * e] : k.d_row, d1 = MODE == kCCol ? col[2 * e + 1] : k.d_row;
                            y[0] = fmaf(d0, fmaf(l.x, 1.0f / kLoScale, f.x), y[0]);
                            y[1] = fmaf(d1, fmaf(l.y, 1.0f / kLoScale, f.y), y[1]);
                        }
                    }
                }
            }
        }
        if constexpr (EPI == kEpiPoly || EPI == kEpiSym) {
            // the lane's diagonal element, if it lies among these columns
            const int on_diag = gi - gj - 32 * h;
            if ((MODE == kCTwo || k.d_out) && (unsigned)on_diag < 32u) {
                float dd = 0.0f;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    if (e == on_diag) {
                        dd = v[e] + k.eye;
                        v[e] = k.d_out ? 0.0f : dd;
                    }
                }
                if (k.d_out)
                    k.d_out[gi] = dd;
            }
        }
        // each half's result takes the place of its C
        if constexpr (EPI == kEpiOut)
            put_bf16(buf, lane, h, v);
        else if constexpr (EPI == kEpiMuon)
            put_hi(buf, lane, h, v, kMuonScale);
        else if (k.out_lo)
            put_pair(buf, lane, h, v, k.s_out);
        else
            put_hi(buf, lane, h, v, k.s_out);
    }
    if constexpr (EPI == kEpiOut || EPI == kEpiMuon) {
        __syncwarp();
        write_rows<EPI>(plan, b, gi & ~31, gj, lane, buf);
    }
    fence_async_shared();  // results leave the buffer, or the next C comes into it, by the copy engine
    __syncwarp();
    if constexpr (EPI != kEpiOut && EPI != kEpiMuon) {
        if (elect_one()) {
            bulk_store(k.out_hi + at, buf, kPiece);
            if (k.out_lo)
                bulk_store(k.out_lo + at, buf + kPiece, kPiece);
            bulk_commit();
        }
        __syncwarp();
    }
}

// A Muon step's master weights of a chunk, on their way into L2 while the
// product is not ready yet.
__device__ __forceinline__ void prefetch_theta(const OrthoPlan &plan, const Tile &x, int row0, int col, int lane)
{
    const int row = row0 + lane;
    if (row >= plan.rows || col >= plan.cols)
        return;
    const float *p = plan.theta + ((int64_t)x.b * plan.rows + row) * plan.cols + col;
    const int n = min(64, plan.cols - col);
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
    if (n > 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p + 32));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p + n - 1));
}

// Shared state of a CTA, besides the operand ring and the epilogue's buffers.
struct Shared {
    uint64_t full[kStages], empty[kStages], peer[kStages], acc_full[2], acc_empty[2], c[kEpiWarps][2];
    uint32_t tmem;
    unsigned written[4];     // epilogue warps that have written their part of a tile, of every fourth tile: while one
                             // warp still writes tile n, no other can be beyond tile n + 2
    unsigned clear;          // tiles of the CTA that may be read for: the phase before them is done
    volatile int abort;
};

// Before tile number n of this CTA is read for, by a whole warp; false if a wait
// ran out.
__device__ __forceinline__ bool clear_to_read(Shared &sh, uint32_t n)
{
    const bool ok = __all_sync(kFullMask, shared_wait(smem_addr(&sh.clear), n + 1, &sh.abort));
    fence_async();  // what is read was written, and comes, by the copy engine
    return ok;
}

// Tile number n of this CTA, x of phase g, by one epilogue warp.  asked: copies
// of C asked for so far on each of the two barriers.
template <int CG, int EPI>
__device__ __forceinline__ bool epilogue_tile(const OrthoPlan &plan, const OrthoGemm &g, const Tile &x, Shared &sh,
                                              uint32_t tmem, uint32_t mine, int warp, int lane, uint32_t rank, uint32_t n,
                                              uint32_t (&asked)[2])
{
    // warp (quad, half): rows 32*quad.., every second chunk of 64 columns; the
    // one chunk of a narrow tile is every second tile's for the same four warps
    const int quad = warp & 3, row = quad * 32 + lane;
    const bool narrow = CG == 1 && g.narrow;
    const int half = narrow ? x.half : warp >> 2, place_of = quad + 4 * half;
    {
        const OrthoProduct &p = g.p[x.prob];
        const uint32_t buf = n & 1, use = n >> 1;
        const int ib = x.i * CG + rank, gi = ib * 128 + row;
        // the chunks of the tile that exist (and, of a symmetric result, are
        // kept): c0 and c0 + 2
        const int c0 = (g.sym ? max(0, 2 * (ib - x.j * CG)) : 0) + half;
        const int c1 = ib < g.mblk && !(narrow && (warp >> 2) != (int)(n & 1)) ? min(2 * CG, 2 * (g.nblk - x.j * CG)) : 0;
        const bool has_lo = kHasC<EPI> && EPI != kEpiPoly && p.c.lo != nullptr;
        // both chunks fit side by side if they have no low halves
        const bool both = EPI == kEpiPoly || (EPI == kEpiSym && !has_lo && !p.out.lo);
        auto place = [&](int c) {  // of this warp's piece of chunk c
            return (int64_t)x.b * g.out_stride + ((int64_t)ib * g.out_c64 + 2 * x.j * CG + c) * kTileElems + quad * 32 * 64;
        };
        auto fetch = [&](int c, int i) {  // into buffer i
            if (elect_one()) {
                bulk_wait_read<0>();  // of the stores out of it
                if constexpr (kHasC<EPI>) {
                    const uint32_t bar = smem_addr(&sh.c[warp][i]);
                    mbar_expect_tx(bar, has_lo ? 2 * kPiece : kPiece);
                    bulk_load(mine + i * kPiece, p.c.hi + place(c), kPiece, bar);
                    if (has_lo)
                        bulk_load(mine + kPiece, p.c.lo + place(c), kPiece, bar);
                }
            }
            __syncwarp();
            if constexpr (kHasC<EPI>)
                ++asked[i];
        };
        if (c0 < c1)
            fetch(c0, 0);
        if (both && c0 + 2 < c1)
            fetch(c0 + 2, 1);
        Local k;
        k.alpha = p.alpha;
        k.s_out = p.s_out;
        k.out_hi = p.out.hi;
        k.out_lo = p.out.lo;
        k.d_row = p.c_scale;
        k.eye = EPI == kEpiPoly ? g.coef_a : 0.0f;
        k.col_scale = p.c_scale;
        k.d_col = nullptr;
        const bool two = EPI == kEpiSym && p.dvec2 != nullptr;
        const int64_t d_at = (int64_t)x.b * g.d_stride;
        k.d_out = (EPI == kEpiPoly || (EPI == kEpiSym && p.diag_out)) ? p.dvec_out + d_at : nullptr;
        if constexpr (kHasC<EPI> && EPI != kEpiPoly) {
            if (c0 < c1) {
                if (g.d_by_col) {
                    k.d_col = p.dvec + d_at;
                } else {
                    const float d = p.dvec[d_at + gi];
                    k.d_row = d * p.c_scale;
                    if (two) {
                        k.d_col = p.dvec2 + d_at;
                        k.col_scale = p.c_scale2;
                        k.eye = d * k.d_col[gi];
                    }
                }
                if (k.d_col && lane < 2)  // the factors of the columns, on their way
                    for (int c = c0; c < c1; c += 2)
                        asm volatile("prefetch.global.L1 [%0];" ::"l"(k.d_col + x.j * CG * 128 + c * 64 + lane * 32));
            }
        }
        if constexpr (EPI == kEpiMuon)
            for (int c = c0; c < c1; c += 2)
                prefetch_theta(plan, x, ib * 128 + quad * 32, x.j * CG * 128 + c * 64, lane);
        bool ok = __all_sync(kFullMask, mbar_wait(smem_addr(&sh.acc_full[buf]), use & 1, &sh.abort));
        tmem_fence_after();
        bool mine_to_do = true;
        if constexpr (EPI == kEpiGram) {
            k.parts = g.parts;
            if (CG == 1 && k.parts > 1 && ok && c0 < c1) {
                // (c0 is the warp's only chunk.)  The last part to come adds
                // them all up, in their order.
                k.slot = g.area * plan.area_slots + (x.index - x.b * (g.mblk * (g.mblk + 1) / 2)) * g.parts;
                k.warp = place_of;
                leave_part(part_at(plan, x.b, k.slot + x.part, place_of), lane,
                           tmem + ((uint32_t)(quad * 32) << 16) + buf * 128 * CG + (narrow ? 0 : c0) * 64);
                __syncwarp();
                unsigned before = 0;
                if (lane == 0)
                    before = add_acq_rel(plan.joined + x.index * kEpiWarps + place_of, 1u);
                mine_to_do = (int)(__shfl_sync(kFullMask, before, 0) % g.parts) == g.parts - 1;
                __syncwarp();
            }
        }
        for (int c = c0; c < c1 && ok && mine_to_do; c += 2) {
            const int i = both && c != c0;
            if constexpr (kHasC<EPI>)
                ok = __all_sync(kFullMask, mbar_wait(smem_addr(&sh.c[warp][i]), (asked[i] - 1) & 1, &sh.abort));
            if (!ok)
                break;
            const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + buf * 128 * CG + (narrow ? 0 : c) * 64;
            const int gj = x.j * CG * 128 + c * 64;
            if constexpr (EPI == kEpiGram || EPI == kEpiPoly) {
                if constexpr (CG == 1 && EPI == kEpiGram) {
                    if (k.parts > 1) {
                        epilogue_chunk<EPI, kCParts>(plan, k, x.b, gi, gj, lane, acc, mine + i * kPiece, place(c));
                        continue;
                    }
                }
                epilogue_chunk<EPI, kCHigh>(plan, k, x.b, gi, gj, lane, acc, mine + i * kPiece, place(c));
            } else if constexpr (EPI == kEpiSym) {
                if (two)
                    epilogue_chunk<EPI, kCTwo>(plan, k, x.b, gi, gj, lane, acc, mine + i * kPiece, place(c));
                else if (has_lo)
                    epilogue_chunk<EPI, kCRow>(plan, k, x.b, gi, gj, lane, acc, mine + i * kPiece, place(c));
                else
                    epilogue_chunk<EPI, kCHigh>(plan, k, x.b, gi, gj, lane, acc, mine + i * kPiece, place(c));
            } else {
                if (g.d_by_col)
                    epilogue_chunk<EPI, kCCol>(plan, k, x.b, gi, gj, lane, acc, mine + i * kPiece, place(c));
                else
                    epilogue_chunk<EPI, kCRow>(plan, k, x.b, gi, gj, lane, acc, mine + i * kPiece, place(c));
            }
            if (!both && c + 2 < c1)
                fetch(c + 2, 0);
        }
        if (!ok)
            return false;
        tmem_fence_before();
        __syncwarp();
        if (elect_one())
            mbar_arrive_cluster(map_to_rank(smem_addr(&sh.acc_empty[buf]), 0));
        __syncwarp();
    }
    return true;
}

template <int CG>
__global__ void __launch_bounds__(kThreads, 1) k_ortho_products(const __grid_constant__ OrthoPlan plan)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;

    const uint32_t ring = (smem_addr(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int first = blockIdx.x / CG, stride = gridDim.x / CG;
    constexpr uint32_t kCols = 2 * 128 * CG;  // two accumulators of 128*CG columns

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&sh.full[s]), 1);
            mbar_init(smem_addr(&sh.empty[s]), 1);
            mbar_init(smem_addr(&sh.peer[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_addr(&sh.acc_full[a]), 1);
            mbar_init(smem_addr(&sh.acc_empty[a]), CG * kEpiWarps);
        }
        for (int w = 0; w < kEpiWarps; ++w)
            for (int i = 0; i < 2; ++i)
                mbar_init(smem_addr(&sh.c[w][i]), 1);
        sh.abort = 0;
        sh.clear = 0;
        for (int i = 0; i < 4; ++i)
            sh.written[i] = 0;
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
    wait_for_previous_grid();
    fence_async();  // what the previous launch wrote is read by the copy engine

    if (warp == 0) {
        uint32_t it = 0;
        bool ok = true;
        Walk<CG> walk(plan);
        uint32_t n = 0;
        for (int64_t t = first; ok && !plan.test_stall && walk.to(plan, t); t += stride, ++n) {
            const OrthoGemm &g = plan.ph[walk.f];
            const Tile x = decode<CG>(g, (int)(t - walk.base));
            const __half *a = g.p[x.prob].a + (int64_t)x.b * g.a_stride;
            const __half *b = g.p[x.prob].b + (int64_t)x.b * g.b_stride;
            ok = clear_to_read(sh, n);
            const int k1 = first_step<CG>(g, x.part + 1);
            for (int k = first_step<CG>(g, x.part); k < k1 && ok; ++k, ++it) {
                const uint32_t s = it % kStages, ph = (it / kStages) & 1;
                ok = __all_sync(kFullMask, mbar_wait(smem_addr(&sh.empty[s]), ph ^ 1, &sh.abort));
                if (!ok)
                    break;
                const uint32_t bar = smem_addr(&sh.full[s]), slot = ring + s * kStageBytes;
                const bool a_mn = reads_mn<CG>(g.a_kind, x.i, k), b_mn = reads_mn<CG>(g.b_kind, x.j, k);
                if (elect_one()) {
                    mbar_expect_tx(bar, CG == 1 && g.narrow ? kSlot + kSlot / 2 : kStageBytes);
                    load_operand(slot, a, g.a_c64, x.i * CG + rank, k, a_mn, bar);
                    if (CG == 1 && g.narrow)
                        load_half_operand(slot + kSlot, b, g.b_c64, x.j, x.half, k, b_mn, bar);
                    else
                        load_operand(slot + kSlot, b, g.b_c64, x.j * CG + rank, k, b_mn, bar);
                }
                __syncwarp();
            }
        }
        if (!ok) {
            sh.abort = 1;
            if (lane == 0)
                report_wait_limit(plan.status, plan.layer_status);
        }
        // copies in flight land before the CTA ends
        for (uint32_t d = it > kStages ? it - kStages : 0; d < it; ++d)
            mbar_wait(smem_addr(&sh.full[d % kStages]), (d / kStages) & 1, nullptr);
    } else if (warp == 1) {
        uint32_t it = 0, n = 0;
        bool ok = true;
        Walk<CG> walk(plan);
        for (int64_t t = first; ok && walk.to(plan, t); t += stride, ++n) {
            const OrthoGemm &g = plan.ph[walk.f];
            const Tile x = decode<CG>(g, (int)(t - walk.base));
            const uint32_t buf = n & 1, use = n >> 1;
            if (rank == 0) {
                ok = __all_sync(kFullMask, mbar_wait(smem_addr(&sh.acc_empty[buf]), (use & 1) ^ 1, &sh.abort));
                if (!ok)
                    break;
                tmem_fence_after();
            }
            const int k0 = first_step<CG>(g, x.part), k1 = first_step<CG>(g, x.part + 1);
            for (int k = k0; k < k1; ++k, ++it) {
                const uint32_t s = it % kStages, ph = (it / kStages) & 1;
                ok = mbar_wait(smem_addr(&sh.full[s]), ph, &sh.abort);
                if (CG == 2 && rank == 0)
                    ok = ok && mbar_wait(smem_addr(&sh.peer[s]), ph, &sh.abort);
                ok = __all_sync(kFullMask, ok);
                if (!ok)
                    break;
                if (CG == 2 && rank != 0) {
                    if (elect_one())
                        mbar_arrive_cluster(map_to_rank(smem_addr(&sh.peer[s]), 0));
                    __syncwarp();
                    continue;
                }
                const bool a_mn = reads_mn<CG>(g.a_kind, x.i, k), b_mn = reads_mn<CG>(g.b_kind, x.j, k);
                const uint32_t idesc = f16_idesc(128 * CG, CG == 1 && g.narrow ? 64 : 128 * CG, a_mn, b_mn);
                const uint32_t slot = ring + s * kStageBytes;
                const uint64_t a_desc = operand_desc(slot, kSlot / 2), b_desc = operand_desc(slot + kSlot, kSlot / 2);
                const uint32_t a_step = (a_mn ? 2048 : 32) >> 4, b_step = (b_mn ? 2048 : 32) >> 4;
                if (elect_one()) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_f16<CG>(tmem + buf * 128 * CG, a_desc + j * a_step, b_desc + j * b_step, idesc,
                                    k > k0 || j > 0);
                    mma_commit<CG>(smem_addr(&sh.empty[s]));
                    if (k + 1 == k1)
                        mma_commit<CG>(smem_addr(&sh.acc_full[buf]));
                }
                __syncwarp();
            }
        }
        if (!ok) {
            sh.abort = 1;
            if (lane == 0)
                report_wait_limit(plan.status, plan.layer_status);
        }
        // the matrix instructions in flight end before the CTA does: the
        // commits of the last stages have arrived
        for (uint32_t d = it > kStages ? it - kStages : 0; d < it; ++d)
            mbar_wait(smem_addr(&sh.empty[d % kStages]), (d / kStages) & 1, nullptr);
    } else if (warp == kWatchWarp) {
        bool ok = true;
        int f = 0, b = -1;  // the phase and matrix that the last tile was of
        uint32_t n = 0;
        Walk<CG> walk(plan);
        for (int64_t t = first; ok && walk.to(plan, t); t += stride) {
            const Tile x = decode<CG>(plan.ph[walk.f], (int)(t - walk.base));
            if (walk.f > 0 && (walk.f != f || x.b != b)) {
                ok = __all_sync(kFullMask, counter_wait(plan.count + (int64_t)(walk.f - 1) * plan.batch + x.b,
                                                        tile_count<CG>(plan.ph[walk.f - 1]) * CG, plan.status,
                                                        kStatusWaitLimit, &sh.abort));
                f = walk.f;
                b = x.b;
            }
            ++n;
            if (ok && lane == 0)
                store_shared(smem_addr(&sh.clear), n);
            __syncwarp();
        }
        if (!ok) {
            sh.abort = 1;
            if (lane == 0)
                report_wait_limit(plan.status, plan.layer_status);
        }
    } else {
        const int w = warp - 2;
        const int ew = (warp & 3) | ((w >> 2) << 2);  // a warp reads the 32 lanes of tensor memory of its number mod 4
        const uint32_t mine = ring + kStages * kStageBytes + ew * kEpiBytes;
        uint32_t n = 0, asked[2] = {0, 0};
        bool ok = true;
        Walk<CG> walk(plan);
        for (int64_t t = first; walk.to(plan, t); t += stride, ++n) {
            const OrthoGemm &g = plan.ph[walk.f];
            const Tile x = decode<CG>(g, (int)(t - walk.base));
            ok = clear_to_read(sh, n);
            if (ok) {
                switch (g.epi) {
                case kEpiGram: ok = epilogue_tile<CG, kEpiGram>(plan, g, x, sh, tmem, mine, ew, lane, rank, n, asked); break;
                case kEpiPoly: ok = epilogue_tile<CG, kEpiPoly>(plan, g, x, sh, tmem, mine, ew, lane, rank, n, asked); break;
                case kEpiSym: ok = epilogue_tile<CG, kEpiSym>(plan, g, x, sh, tmem, mine, ew, lane, rank, n, asked); break;
                case kEpiApply: ok = epilogue_tile<CG, kEpiApply>(plan, g, x, sh, tmem, mine, ew, lane, rank, n, asked); break;
                case kEpiOut: ok = epilogue_tile<CG, kEpiOut>(plan, g, x, sh, tmem, mine, ew, lane, rank, n, asked); break;
                default: ok = epilogue_tile<CG, kEpiMuon>(plan, g, x, sh, tmem, mine, ew, lane, rank, n, asked); break;
                }
            }
            if (!ok)
                break;
            if (walk.f + 1 < plan.n_phases) {  // the CTA's last warp counts the tile
                bulk_wait<0>();
                __syncwarp();
                if (lane == 0 && add_shared(smem_addr(&sh.written[n & 3]), 1u) % kEpiWarps == kEpiWarps - 1)
                    add_release(plan.count + (int64_t)walk.f * plan.batch + x.b, 1u);
                __syncwarp();
            }
        }
        bulk_wait<0>();
        if (!ok) {
            sh.abort = 1;
            if (lane == 0)
                report_wait_limit(plan.status, plan.layer_status);
            for (int i = 0; i < 2; ++i)  // copies of C may be in flight
                if (asked[i] > 0)
                    mbar_wait(smem_addr(&sh.c[ew][i]), (asked[i] - 1) & 1, nullptr);
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

// Splits K of the Gram matrices where their tiles leave CTAs without work.  A
// step takes 0.33 us, the joining of parts 2 us and another 0.65 us a part (64
// KiB read at the rate of one SM): best with sqrt(K / 2 steps) parts, from 24
// steps on.  2 matrices of 238 x 14962 took 332 us without, 238 with it.
void split_gram(OrthoPlan &plan, int groups)
{
    for (int f = 0; f < plan.n_phases; ++f) {
        OrthoGemm &g = plan.ph[f];
        if (g.epi != kEpiGram || g.k64 < 24)
            continue;
        const int tiles = tile_count<1>(g), all = tiles * plan.batch;
        int parts = (int)std::sqrt(0.5 * g.k64);
        parts = parts < kMaxParts ? parts : kMaxParts;
        parts = parts < groups / all ? parts : groups / all;
        parts = parts < plan.areas * plan.area_slots / tiles ? parts : plan.areas * plan.area_slots / tiles;
        if (parts >= 2 && all <= kJoinTiles)
            g.parts = parts;
    }
}

// Halves the tiles of phases that leave two thirds of the CTAs without work all
// the same: less to load for a step and half the epilogue, whose time is that of
// its instructions.  A Muon step of 228 x 705 took 134 us without, 122 with it,
// 300 x 8000 157 and 147; with 72 tiles of 152 (2 matrices of 1024 x 2560) it
// gains nothing (222 and 224).
void narrow_tiles(OrthoPlan &plan, int groups)
{
    for (int f = 0; f < plan.n_phases; ++f)
        plan.ph[f].narrow = 3 * tile_count<1>(plan.ph[f]) * plan.batch <= groups;
}

template <int CG>
cudaError_t launch(const OrthoPlan &plan, int groups, cudaStream_t stream)
{
    int most = 1;
    for (int f = 0; f < plan.n_phases; ++f) {
        const int t = tile_count<CG>(plan.ph[f]) * plan.batch;
        most = t > most ? t : most;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((most < groups ? most : groups) * CG);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute at[3];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeCooperative;
    at[1].val.cooperative = 1;
    at[2].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[2].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 3;
    return cudaLaunchKernelEx(&cfg, k_ortho_products<CG>, plan);
}

// How many groups of CG CTAs the device holds at once (once per device: *cache).
template <int CG>
cudaError_t resident_groups(std::atomic<int> &cache, int device, int *groups)
{
    *groups = cache.load(std::memory_order_acquire);
    if (*groups > 0)
        return cudaSuccess;
    int sms = 0;
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_ortho_products<CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(sms / CG * CG);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CG;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveClusters(groups, k_ortho_products<CG>, &cfg);
    if (e != cudaSuccess)
        return e;
    if (*groups < 1)
        return cudaErrorLaunchOutOfResources;
    *groups = *groups < sms / CG ? *groups : sms / CG;
    cache.store(*groups, std::memory_order_release);
    return cudaSuccess;
}

// Steps of the ring on the busiest CTA.  Of a single matrix each phase waits
// for the one before; those of a batch run into one another.
template <int CG>
double steps(const OrthoPlan &plan, int groups)
{
    double sum = 0.0;
    for (int f = 0; f < plan.n_phases; ++f) {
        const int t = tile_count<CG>(plan.ph[f]) * plan.batch;
        const double rounds = plan.batch == 1 ? (t + groups - 1) / groups : t > groups ? (double)t / groups : 1.0;
        sum += rounds * ((plan.ph[f].k64 + plan.ph[f].parts - 1) / plan.ph[f].parts) * (plan.ph[f].narrow ? 0.76 : 1.0);
    }
    return sum;
}

}  // namespace

cudaError_t launch_ortho_products(const OrthoPlan &plan, int device, cudaStream_t stream, int *form)
{
    if (device < 0 || device >= kMaxDevices)
        return cudaErrorInvalidDevice;
    static std::atomic<int> singles[kMaxDevices], pairs[kMaxDevices];
    int n1 = 0, n2 = 0;
    cudaError_t e = resident_groups<1>(singles[device], device, &n1);
    if (e == cudaSuccess)
        e = resident_groups<2>(pairs[device], device, &n2);
    if (e != cudaSuccess)
        return e;
    // A pair of CTAs on a 256 x 256 tile takes 0.39 us a step, a single one on
    // 128 x 128 0.33 us with every SM at it (both bound by what L2 delivers,
    // 15 TB/s): pairs do 3.3 times the work per step, but a matrix has four
    // times fewer tiles for them.
    OrthoPlan split = plan;
    split_gram(split, n1);
    narrow_tiles(split, n1);
    const bool in_pairs = 0.39 * steps<2>(plan, n2) <= 0.33 * steps<1>(split, n1);
    if (form) {
        *form |= in_pairs ? kFormPairs : 0;
        for (int f = 0; f < split.n_phases && !in_pairs; ++f)
            *form |= (split.ph[f].parts > 1 ? kFormSplit : 0) | (split.ph[f].narrow ? kFormNarrow : 0);
        return cudaSuccess;
    }
    if (in_pairs)
        return launch<2>(plan, n2, stream);
    return launch<1>(split, n1, stream);
}

}  // namespace slide
