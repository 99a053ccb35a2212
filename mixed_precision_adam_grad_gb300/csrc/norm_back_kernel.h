// norm_back_kernel.h — the gradient of slide_norm: of the rows, and of weight and
// bias, whose sums go over the rows; included by a translation unit for each type
// of rows.
//
// A block takes tiles of 1 to 16 rows.  x and d_out of a tile lie in shared
// memory, the next tile's are on their way meanwhile.  First each row belongs
// to a team of warps (16 warps over the tile's rows), which forms the two sums
// of the row and then its gradient; then each thread takes columns and adds
// their terms over the tile's rows to its sums, which stay in registers for all
// of the block's tiles.  So every tensor is read from memory once, what a row
// costs besides its values is shared by many values of a thread, and nothing is
// added atomically.  A second kernel joins the blocks' sums, always in the same
// order.
//
// Bound by latency: 16 warps an SM (25 %) hide too little of it for the instructions
// that they have, 30 an element: x, d_out and the weight are read from shared memory
// and unpacked for the row's sums and again for its gradient, x and d_out a third
// time for the columns.  8192 x 8192 BF16 takes 110 us (floor 60), FP32 8192 x 5120
// 141 (75); with the residual's gradient and a dropout 16384 x 5120 takes 201 us
// (floor 126), 49 instructions an element, issue slots busy 57 % of the time.  The
// columns' part alone (no d_x) runs at the memory's rate: 55 us for 336 MB.  A block
// is 16 warps: 32 were slower (64 registers spill: 16384 x 5120 244 us instead of
// 227), two blocks of 8 faster by 3 to 8 % up to 4096 columns and slower beyond 8192;
// one form serves both.
#pragma once
#include <algorithm>
#include <atomic>

#include "norm_rows.h"

namespace slide {
namespace {

constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr size_t kMaxSmem = 224 * 1024;  // beside 2.3 KiB of sums
constexpr int kMaxDevices = 64;

// A tile's row in shared memory, its runs from c0 on: by copies that go past the
// registers, where they can be that small.
template <int MODE, typename T>
__device__ __forceinline__ void fetch_row(uint8_t *to, const T *row, int c0, int gap, int k, int end)
{
    uint32_t at = ptx::smem_addr(to) + c0 * (int)sizeof(T);
    row += c0;
    for (int c = c0; c < end; c += gap, at += gap * (int)sizeof(T), row += gap) {
        if constexpr (MODE != kSingle) {
            if (whole<MODE>(c, k, end)) {
#pragma unroll
                for (int h = 0; h < (int)sizeof(T) / 2; ++h)
                    ptx::copy_async16(at + h * 16, row + h * (16 / (int)sizeof(T)));
            } else {
                Run<T, 8> r;
                load_part(r, row, k - c, end - c);
                r.store(to + c * sizeof(T));
            }
        } else if constexpr (sizeof(T) == 4) {
            ptx::copy_async4(at, row);
        } else {
            reinterpret_cast<T *>(to)[c] = *row;
        }
    }
}

// J: runs of columns (eight, or one value unless kAligned) whose sums a thread
// keeps.  WHAT: what the kernel is compiled for (open questions cost predicates at
// every run: 8192 x 8192 BF16 took 132 us with all of them, 110 without).
enum What {
    kPlain = 0,     // a weight and d_x; no d_sum, d_residual or dropout
    kStream = 1,    // d_sum too
    kDropped = 2,   // d_sum, d_residual and a dropout
    kOpen = 3       // anything
};

template <typename T, int MODE, int J, int WIDE, int WHAT>
__global__ void __launch_bounds__(kThreads) k_norm_back(const NormBackArgs a)
{
    constexpr int VEC = MODE == kSingle ? 1 : 8, COLS = MODE == kAligned ? 8 : 1;
    using R = Run<T, VEC>;
    __shared__ __align__(16) float2 red[kWarps][kWarps];
    __shared__ __align__(16) float2 stats[2][kWarps];  // per stage and row: mean, reciprocal root
    extern __shared__ __align__(16) uint8_t smem[];
    const int warps = kWarps / a.tile, team = (threadIdx.x >> 5) / warps;
    const int gap = warps * 32 * VEC, c0 = (threadIdx.x - team * warps * 32) * VEC, cols = a.cols;
    const int lane = threadIdx.x & 31;
    const uint32_t step = WHAT == kDropped || WHAT == kOpen ? drop_step(a.drop) : 0;
    const int tensor = a.tile * a.pitch;  // bytes of a tile's x, and of its d_out behind it
    constexpr bool OPEN = WHAT == kOpen;
    const bool rows_too = !OPEN || a.d_x || a.d_residual, sums_too = a.part_w || a.part_b;
    const bool more_too = WHAT == kStream || WHAT == kDropped || (OPEN && a.d_sum);
    const bool res_too = WHAT == kDropped || (OPEN && a.d_residual), drops = WHAT == kDropped || (OPEN && a.drop.limit16);
    Params<MODE, WIDE> weight;
    weight.init(a.weight, a.wide, reinterpret_cast<float *>(smem + a.stages * 2 * tensor), cols);
    // where a row's values start in its first run
    auto offset = [&](int64_t r) { return MODE == kShifted ? (int)((uint32_t)r * (uint32_t)a.xs & 7) : 0; };
    // the row to ask for, and in step with the tiles the row at hand
    const int64_t r_step = (int64_t)gridDim.x * a.tile;
    int64_t asked = (int64_t)blockIdx.x * a.tile + team, r = asked;
    const T *ask_x = static_cast<const T *>(a.x) + asked * a.xs, *ask_g = static_cast<const T *>(a.d_out) + asked * a.gs;
    const T *more = static_cast<const T *>(a.d_sum) + r * a.ss, *ask_more = more;
    T *d_x = static_cast<T *>(a.d_x) + r * a.ds, *d_res = static_cast<T *>(a.d_residual) + r * a.rs;

    auto fetch = [&](int stage) {
        if (asked < a.rows) {
            const int k = offset(asked);
            uint8_t *to = smem + stage * 2 * tensor + team * a.pitch;
            fetch_row<MODE>(to, ask_x - k, c0, gap, k, cols + k);
            fetch_row<MODE>(to + tensor, ask_g - k, c0, gap, k, cols + k);
            if (c0 == 0) {
                ptx::copy_async4(ptx::smem_addr(&stats[stage][team].y), a.rstd + asked);
                if (!a.rms)
                    ptx::copy_async4(ptx::smem_addr(&stats[stage][team].x), a.mean + asked);
            }
            if (more_too && rows_too) {  // read later, from L2
                constexpr int kLine = 128 / (int)sizeof(T);
                for (int c = (c0 / VEC) * kLine; c < cols; c += warps * 32 * kLine)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(ask_more + c));
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        asked += r_step;
        ask_x += r_step * a.xs;
        ask_g += r_step * a.gs;
        if (more_too)
            ask_more += r_step * a.ss;
    };
    if (a.rms && threadIdx.x < 2 * kWarps)
        stats[threadIdx.x / kWarps][threadIdx.x % kWarps].x = 0.0f;
    Vals<COLS> dw[J], db[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        dw[j].clear();
        db[j].clear();
    }
    ptx::launch_dependents();
    const bool ahead = a.stages == 2;
    int stage = 0;
    if (ahead)
        fetch(0);
    for (int64_t first_row = (int64_t)blockIdx.x * a.tile; first_row < a.rows; first_row += r_step) {
        if (ahead) {
            fetch(stage ^ 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            fetch(0);
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const uint32_t tile = ptx::smem_addr(smem) + stage * 2 * tensor;
        if (rows_too && r < a.rows) {
            const int k = offset(r), end = cols + k;
            const uint32_t x = tile + team * a.pitch + c0 * (int)sizeof(T);  // the thread's first run
            const float mean = stats[stage][team].x, rstd = stats[stage][team].y;
            // x - mean and d_out*weight of the run at column c, which lies at p
            auto terms = [&](uint32_t p, int c, Vals<VEC> &xm, Vals<VEC> &gw) {
                R v, u;
                v.load_shared(p);
                u.load_shared(p + tensor);
                gw = u.get();
                if (!OPEN || a.weight)
                    gw = mul(gw, weight.template get<VEC>(c, k));
                xm = add(v.get(), -mean);
            };
            Vals<VEC> s0, s1;  // one sum for each place of a run
            s0.clear();
            s1.clear();
#pragma unroll 2
            for (uint32_t c = c0, p = x; (int)c < end; c += gap, p += gap * (int)sizeof(T)) {
                Vals<VEC> xm, gw;
                terms(p, c, xm, gw);
                s0 = add(s0, gw);
                s1 = fma(gw, xm, s1);
            }
            R next;  // of d_sum, a run ahead
            if (more_too && c0 < end)
                load_run<MODE>(next, more - k + c0, c0, k, end);
            float t0 = s0.sum(), t1 = s1.sum();
            team_sum2(t0, t1, red[team], team, warps);
            // rstd*(g - sum(g)/cols - h*sum(g*h)/cols), h = (x - mean)*rstd
            const float k0 = a.rms ? 0.0f : -t0 * a.inv_cols * rstd, k1 = -(t1 * rstd) * a.inv_cols * rstd * rstd;
            Dropper<VEC> drop;
            const uint64_t first = (uint64_t)a.drop.first + (uint64_t)r * cols - k;
            // whole warps: lanes beyond the row form masks for others
            constexpr int kStep = VEC == 8 ? 1 : 4;
            for (int c1 = c0; c1 - lane * VEC < end; c1 += kStep * gap) {
#pragma unroll
                for (int i = 0; i < kStep; ++i) {
                    const int c = c1 + i * gap;
                    const bool in = c < end;
                    Vals<VEC> gw;
                    if (in) {
                        Vals<VEC> xm;
                        const R v = next;
                        if (more_too && c + gap < end)
                            load_run<MODE>(next, more - k + c + gap, c + gap, k, end);
                        terms(x + (c - c0) * (int)sizeof(T), c, xm, gw);
                        gw = fma(gw, rstd, fma(xm, k1, k0));
                        if (more_too)
                            gw = add(gw, v.get());
                        if (res_too)
                            store_run<MODE>(gw, d_res - k + c, c, k, end);
                    }
                    if (!OPEN || a.d_x) {
                        if (drops)
                            drop.run(a.drop, step, first, i, c, gap, end, gw);
                        if (in)
                            store_run<MODE>(gw, d_x - k + c, c, k, end);
                    }
                }
            }
        }
        if (sums_too) {
            const int live = (int)min((int64_t)a.tile, a.rows - first_row);
            uint32_t p = tile + threadIdx.x * (COLS * (int)sizeof(T));
#pragma unroll 4
            for (int q = 0; q < live; ++q, p += a.pitch) {
                const float2 of = stats[stage][q];
                const int k = offset(first_row + q);
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if ((threadIdx.x + j * kThreads) * COLS < cols) {
                        const uint32_t at = p + (j * kThreads * COLS + k) * (int)sizeof(T);
                        Run<T, COLS> v, u;
                        v.load_shared(at);
                        u.load_shared(at + tensor);
                        const Vals<COLS> h = mul(add(v.get(), -of.x), of.y), d = u.get();
                        dw[j] = fma(d, h, dw[j]);
                        db[j] = add(db[j], d);
                    }
                }
            }
        }
        r += r_step;
        d_x += r_step * a.ds;
        if (res_too)
            d_res += r_step * a.rs;
        if (more_too)
            more += r_step * a.ss;
        __syncthreads();  // the tile's place is free
        stage ^= ahead;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (threadIdx.x + j * kThreads) * COLS;
        if (c < cols) {
            const int64_t at = (int64_t)blockIdx.x * cols + c;
            Run<float, COLS> o;
            if (a.part_w) {
                o.set(dw[j]);
                o.store(a.part_w + at);
            }
            if (a.part_b) {
                o.set(db[j]);
                o.store(a.part_b + at);
            }
        }
    }
}

// Sums of the parts, 32 columns to a block: warp after warp of the parts, then
// the warps' sums.
template <typename P>
__global__ void __launch_bounds__(512) k_norm_join(const float *part_w, const float *part_b, int parts, int cols, P *d_weight,
                                                   P *d_bias)
{
    __shared__ float sums[16][32];
    ptx::wait_for_previous_grid();
    const bool w = blockIdx.y == 0 && d_weight;
    const float *part = w ? part_w : part_b;
    P *out = w ? d_weight : d_bias;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 10
        for (int p = warp; p < parts; p += 16)
            s += part[(int64_t)p * cols + c];
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 16; ++i)
            s += sums[i][lane];
        out[c] = narrow<P>(s);
    }
}

// Bytes of a row in shared memory.
int row_pitch(int cols, size_t size, Mode mode) { return (int)(((cols + (mode == kShifted ? 7 : 0)) * size + 31) & ~(size_t)31); }

// Rows of a tile: as many as leave room for two tiles, but no more than give
// every block one, and no more warps to a row than have values.
int tile_rows(int64_t rows, int cols, size_t pitch, size_t room, int vec)
{
    int n = kWarps;
    while (n > 1 && (4 * n * pitch > room || (rows < (int64_t)n * kParts && (kWarps / n) * 32 * vec < cols)))
        n /= 2;
    return n;
}

template <typename T, int MODE, int J, int WIDE, int WHAT>
cudaError_t launch(const NormBackArgs &a, int64_t blocks, cudaStream_t s)
{
    static std::atomic<bool> allowed[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    if (!allowed[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(k_norm_back<T, MODE, J, WIDE, WHAT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
        if (e != cudaSuccess)
            return e;
        allowed[dev].store(true, std::memory_order_release);
    }
    const size_t smem = (size_t)a.stages * 2 * a.tile * a.pitch + Params<MODE>::words(a.cols) * sizeof(float);
    k_norm_back<T, MODE, J, WIDE, WHAT><<<(unsigned)blocks, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int WIDE, int WHAT>
cudaError_t launch_aligned(const NormBackArgs &a, int64_t blocks, cudaStream_t s)
{
    const int j = (a.cols / 8 + kThreads - 1) / kThreads;
    return j == 1   ? launch<T, kAligned, 1, WIDE, WHAT>(a, blocks, s)
           : j == 2 ? launch<T, kAligned, 2, WIDE, WHAT>(a, blocks, s)
                    : launch<T, kAligned, 4, WIDE, WHAT>(a, blocks, s);
}

// Columns of single values: 4, 8, 16 or 32 to a thread.  Plain calls have kernels of
// their own at each (8192 x 4099 BF16 135 us, with all questions open 160).
template <typename T, int MODE, int WHAT = kOpen>
cudaError_t launch_singles(const NormBackArgs &a, int64_t blocks, cudaStream_t s)
{
    const int j = (a.cols + kThreads - 1) / kThreads;
    return j <= 4    ? launch<T, MODE, 4, -1, WHAT>(a, blocks, s)
           : j <= 8  ? launch<T, MODE, 8, -1, WHAT>(a, blocks, s)
           : j <= 16 ? launch<T, MODE, 16, -1, WHAT>(a, blocks, s)
                     : launch<T, MODE, 32, -1, WHAT>(a, blocks, s);
}

template <typename T, typename P>
cudaError_t launch(NormBackArgs a, Mode mode, void *d_weight, void *d_bias, float *ws, cudaStream_t s)
{
    const size_t room = kMaxSmem - (mode == kShifted ? Params<kShifted>::words(a.cols) * sizeof(float) : 0);
    a.pitch = row_pitch(a.cols, sizeof(T), mode);
    a.tile = tile_rows(a.rows, a.cols, a.pitch, room, mode == kSingle ? 1 : 8);
    a.stages = 4 * (size_t)a.tile * a.pitch <= room ? 2 : 1;
    const int64_t blocks = parts_for(a.rows, a.tile);
    a.part_w = d_weight ? ws : nullptr;
    a.part_b = d_bias ? ws + blocks * a.cols : nullptr;
    if (a.rows > 0) {
        cudaError_t e;
        if (mode == kAligned) {
            constexpr int kWide = sizeof(T) == 4;  // the weight's type is the rows' (7 % off where it is found out at every load)
            const bool drop = a.drop.limit16 != 0;
            if (a.weight && a.d_x && (a.wide != 0) == (kWide != 0) && !drop && !a.d_residual)
                e = a.d_sum ? launch_aligned<T, kWide, kStream>(a, blocks, s) : launch_aligned<T, kWide, kPlain>(a, blocks, s);
            else if (a.weight && a.d_x && (a.wide != 0) == (kWide != 0) && drop && a.d_residual && a.d_sum)
                e = launch_aligned<T, kWide, kDropped>(a, blocks, s);
            else
                e = launch_aligned<T, -1, kOpen>(a, blocks, s);
        } else {
            const bool plain = a.weight && a.d_x && !a.d_sum && !a.d_residual && !a.drop.limit16;
            e = mode == kSingle ? launch_singles<T, kSingle>(a, blocks, s)
                : plain         ? launch_singles<T, kShifted, kPlain>(a, blocks, s)
                                : launch_singles<T, kShifted>(a, blocks, s);
        }
        if (e != cudaSuccess)
            return e;
    }
    if (!d_weight && !d_bias)
        return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((a.cols + 31) / 32, d_weight && d_bias ? 2 : 1);
    cfg.blockDim = dim3(512);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_norm_join<P>, (const float *)a.part_w, (const float *)a.part_b, (int)blocks, a.cols,
                              (P *)d_weight, (P *)d_bias);
}

}  // namespace
}  // namespace slide
