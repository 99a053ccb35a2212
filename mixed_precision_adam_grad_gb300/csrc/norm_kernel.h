// norm_kernel.h — the norm's forward kernel and its launch; included by a
// translation unit for each type of rows, with and without a sum (they compile
// side by side).
//
// A row belongs to a team of 1 to 8 warps, which keeps it in registers, as it
// is kept in memory, from the first sum to the last store: every tensor is read
// once.  The variance is that of the centred values, a second sum over the
// registers, so a large mean costs no digits.  Teams are small and a thread's
// share of a row large, since what a row costs besides its values (addresses,
// two sums over the team, a root) costs each of its threads the same.
//
// Bound by memory where rows are wide and plain: RMS of 8192 x 8192 BF16 48 us, 5.6
// TB/s of its 268 MB (83 % of a plain copy's rate), FP32 8192 x 5120 61 us (83 %);
// narrower ones by latency, since a team has no load in flight while it sums and
// stores (8192 x 2560 BF16 21 us, 60 %, x 4096 33 us, 61 %).  Dropout, residual and
// norm of 16384 x 5120 BF16 take 127 us (79 %): 35 instructions an element, eight of
// them the generator's integers, issue slots busy 62 % of the time with 24 warps an
// SM.
#pragma once
#include <atomic>

#include "norm_rows.h"

namespace slide {
namespace {

constexpr int kMaxWarps = 8, kThreads = kMaxWarps * 32;

__device__ __forceinline__ float team_sum(float v, float *red, int team, int warps)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(kFull, v, o);
    if (warps == 1)
        return v;
    if ((threadIdx.x & 31) == 0)
        red[(threadIdx.x >> 5) % warps] = v;
    team_sync(team, warps);
    v = 0.0f;
    for (int i = 0; i < warps; i += 2) {
        const float2 u = *reinterpret_cast<const float2 *>(red + i);
        v += u.x + u.y;
    }
    return v;
}

// What a kernel is compiled for.  A question that only the arguments answer costs
// instructions at every run, whose two answers stand there under predicates: the
// frequent calls have kernels of their own (residual and dropout, 16384 x 5120
// BF16: 143 us with all questions open, 127 without).
enum What { kNone = 0, kResidual = 1, kDropped = 2, kAnySum = 3 };  // s = x; residual + x; residual + dropout(x); any
enum Norm { kAnyNorm = 0, kLayer = 1, kRms = 2 };                   // any; with weight and bias; with weight alone

// Blocks that have to fit on an SM.  Other teams work while one waits for its
// row, so registers are given up for warps: BF16 rows of 2560 take 20.9 us with four
// blocks, 22.7 with three and 25.0 with two, a residual and a dropout 127 us with
// three, 132 with four (spilled) and 140 with two (16384 x 5120); FP32 rows need
// theirs (8192 x 1601: 26.7 us with two, 33.9 with three and 37.0 with four).  Single
// values: 8192 x 2561 113 us with three, 195 with one; 4096 x 8191 214 us with one,
// 296 with two.
template <typename T>
constexpr int min_blocks(int mode, int nv, int what)
{
    return mode == kSingle ? (nv <= 8 ? 4 : nv <= 16 ? 3 : 1) : sizeof(T) == 4 ? (nv <= 3 ? 3 : 2) : nv <= 5 && what == kNone ? 4 : 3;
}

// The thread's NV runs start VEC*32*warps values apart.
template <typename T, int MODE, int NV, int WHAT, int NORM, int WIDE>
__global__ void __launch_bounds__(kThreads, min_blocks<T>(MODE, NV, WHAT)) k_norm(const NormArgs a)
{
    constexpr int VEC = MODE == kSingle ? 1 : 8;
    using R = Run<T, VEC>;
    // of each team; its sums alternate: a warp is at most one ahead of another of its team
    __shared__ __align__(16) float red[2][kMaxWarps][kMaxWarps];
    extern __shared__ float staged[];
    const int warps = a.warps, team = (threadIdx.x >> 5) / warps, teams = kMaxWarps / warps;
    const int gap = warps * 32 * VEC, c0 = (threadIdx.x - team * warps * 32) * VEC;
    const bool res_too = WHAT == kResidual || WHAT == kDropped || (WHAT == kAnySum && a.residual);
    const bool drops = WHAT == kDropped || (WHAT == kAnySum && a.drop.limit16);
    const bool rms = NORM == kRms || (NORM == kAnyNorm && a.rms);
    const bool weighs = NORM != kAnyNorm || a.weight, biased = NORM == kLayer || (NORM == kAnyNorm && a.bias);
    const uint32_t step = drops ? drop_step(a.drop) : 0;
    Params<MODE, WIDE> weight, bias;
    weight.init(a.weight, a.wide, staged, a.cols);
    bias.init(a.bias, a.wide, staged + Params<MODE>::words(a.cols), a.cols);
    if (MODE == kShifted)
        __syncthreads();
    int half = 0;
    for (int64_t r = (int64_t)blockIdx.x * teams + team; r < a.rows; r += (int64_t)gridDim.x * teams) {
        // the row's values are those from k to end behind the start of its first run
        const int k = MODE == kShifted ? (int)((uint64_t)(r * a.xs) & 7) : 0, end = a.cols + k;
        const T *x = static_cast<const T *>(a.x) + r * a.xs - k;
        R s[NV];  // what is normed
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (c0 + i * gap < end)
                load_run<MODE>(s[i], x + c0 + i * gap, c0 + i * gap, k, end);
        if constexpr (WHAT != kNone) {
            const T *res = static_cast<const T *>(a.residual) + r * a.rs - k;
            T *sum = static_cast<T *>(a.sum) + r * a.ss - k;
            R q[NV];
            if (res_too) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (c0 + i * gap < end)
                        load_run<MODE>(q[i], res + c0 + i * gap, c0 + i * gap, k, end);
            }
            Dropper<VEC> drop;
            const uint64_t first = (uint64_t)a.drop.first + (uint64_t)r * a.cols - k;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * gap;
                Vals<VEC> v = s[i].get();
                if (drops)  // whole warps: lanes beyond the row form masks for others
                    drop.run(a.drop, step, first, i, c, gap, end, v);
                if (c < end) {
                    if (res_too)
                        v = add(q[i].get(), v);
                    store_run<MODE>(v, sum + c, c, k, end);
                    s[i].set(v);
                }
            }
        }
        float mean = 0.0f;
        Vals<VEC> part;  // one sum for each place of a run
        part.clear();
        if (!rms) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (c0 + i * gap < end)
                    part = add(part, s[i].get());
            }
            mean = quotient(team_sum(part.sum(), red[half][team], team, warps), (float)a.cols, a.inv_cols);
            half ^= 1;
            part.clear();
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * gap;
            if (c < end) {
                Vals<VEC> v = s[i].get();
                if (!rms)
                    v = add(v, -mean);
                if (!whole<MODE>(c, k, end)) {
                    float x[VEC];
                    v.split_to(x);
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        x[e] = c + e >= k && c + e < end ? x[e] : 0.0f;
                    v.set(x);
                }
                part = fma(v, v, part);
            }
        }
        const float rstd = inverse_root(team_sum(part.sum(), red[half][team], team, warps) * a.inv_cols + a.eps);
        half ^= 1;
        if (c0 == 0) {
            if (a.mean)
                a.mean[r] = mean;
            if (a.rstd)
                a.rstd[r] = rstd;
        }
        T *out = static_cast<T *>(a.out) + r * a.os - k;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * gap;
            if (c < end) {
                Vals<VEC> v = s[i].get();
                if (!rms)
                    v = add(v, -mean);
                v = mul(v, rstd);
                if (weighs)
                    v = mul(v, weight.template get<VEC>(c, k));
                if (biased)
                    v = add(v, bias.template get<VEC>(c, k));
                store_run<MODE>(v, out + c, c, k, end);
            }
        }
    }
}

// Runs of a thread and warps of a team: the fewest warps that hold the row, of
// those the fewest runs; more warps where there are too few rows to fill the
// device (32 warps an SM: RMS norms of 2048 x 4096 BF16 take 9.0 us, at 24 11.8; at
// 64 those of 2048 x 2560 took 10.3 instead of 8.6).  The warps that are resident of
// the kernel at hand, 16 of FP32 rows, are no better count: RMS of 4099 x 1601 FP32
// 18.5 us instead of 18.6, but 4096 x 2048 18.3 instead of 17.3, and 3000 x 2048 with
// a residual 30.8 instead of 21.8.
struct Form {
    int nv, warps;
};

template <int N>
Form form_for(const int (&runs_of)[N], int runs, int64_t rows, int sms)
{
    Form f{runs_of[N - 1], kMaxWarps};
    for (int w = kMaxWarps; w >= 1; w /= 2) {
        const int need = (runs + 32 * w - 1) / (32 * w);
        if (need > runs_of[N - 1] || (w < kMaxWarps && need > 1 && rows * w < (int64_t)sms * 32))
            break;
        f.warps = w;
        for (int i = N - 1; i >= 0; --i)
            if (runs_of[i] >= need)
                f.nv = runs_of[i];
    }
    return f;
}

constexpr int kMaxDevices = 64;

template <typename T, int MODE, int NV, int WHAT, int NORM, int WIDE>
cudaError_t launch(const NormArgs &a, int sms, cudaStream_t s)
{
    // blocks on an SM: asked again where their shared memory is another than last time
    static std::atomic<int64_t> cache[kMaxDevices];
    const int teams = kMaxWarps / a.warps, smem = 2 * Params<MODE>::words(a.cols) * (int)sizeof(float);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    int64_t known = cache[dev].load(std::memory_order_relaxed);
    if (known == 0 || known >> 8 != smem) {
        int n = 0;
        if (smem > 0)
            e = cudaFuncSetAttribute(k_norm<T, MODE, NV, WHAT, NORM, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     2 * Params<MODE>::words(kMaxCols) * (int)sizeof(float));
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_norm<T, MODE, NV, WHAT, NORM, WIDE>, kThreads, smem);
        if (e != cudaSuccess)
            return e;
        if (n < 1)
            return cudaErrorLaunchOutOfResources;
        known = (int64_t)smem << 8 | n;
        cache[dev].store(known, std::memory_order_relaxed);
    }
    const int64_t blocks = (a.rows + teams - 1) / teams, most = (int64_t)sms * (known & 255);
    k_norm<T, MODE, NV, WHAT, NORM, WIDE><<<(unsigned)(blocks < most ? blocks : most), kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int MODE, int WHAT, int NORM, int WIDE>
cudaError_t launch_runs(NormArgs a, int sms, cudaStream_t s)
{
    constexpr int kRuns[] = {1, 2, 3, 4, 5, 6, 8};
    const Form f = form_for(kRuns, (a.cols + (MODE == kShifted ? 14 : 0)) / 8, a.rows, sms);
    a.warps = f.warps;
    switch (f.nv) {
    case 1: return launch<T, MODE, 1, WHAT, NORM, WIDE>(a, sms, s);
    case 2: return launch<T, MODE, 2, WHAT, NORM, WIDE>(a, sms, s);
    case 3: return launch<T, MODE, 3, WHAT, NORM, WIDE>(a, sms, s);
    case 4: return launch<T, MODE, 4, WHAT, NORM, WIDE>(a, sms, s);
    case 5: return launch<T, MODE, 5, WHAT, NORM, WIDE>(a, sms, s);
    case 6: return launch<T, MODE, 6, WHAT, NORM, WIDE>(a, sms, s);
    default: return launch<T, MODE, 8, WHAT, NORM, WIDE>(a, sms, s);
    }
}

// Parameters of the rows' type.
template <typename T, int WHAT>
cudaError_t launch_native(const NormArgs &a, Norm norm, int sms, cudaStream_t s)
{
    constexpr int kWide = sizeof(T) == 4;
    return norm == kLayer ? launch_runs<T, kAligned, WHAT, kLayer, kWide>(a, sms, s)
                          : launch_runs<T, kAligned, WHAT, kRms, kWide>(a, sms, s);
}

template <typename T, bool SUM>
cudaError_t launch(NormArgs a, Mode mode, int sms, cudaStream_t s)
{
    constexpr int kOpen = SUM ? kAnySum : kNone;
    const Norm norm = !a.weight || (a.rms != 0) == (a.bias != nullptr) ? kAnyNorm : a.rms ? kRms : kLayer;
    if (mode == kAligned) {
        if (norm != kAnyNorm && (a.wide != 0) == (sizeof(T) == 4) && (!SUM || a.residual)) {
            if constexpr (SUM)
                return a.drop.limit16 ? launch_native<T, kDropped>(a, norm, sms, s) : launch_native<T, kResidual>(a, norm, sms, s);
            else
                return launch_native<T, kNone>(a, norm, sms, s);
        }
        return launch_runs<T, kAligned, kOpen, kAnyNorm, -1>(a, sms, s);
    }
    if (mode == kShifted && a.cols + 7 <= kMaxCols) {  // its runs, with those in part the row's, fit into a block
        if constexpr (!SUM) {
            if (norm != kAnyNorm)
                return norm == kLayer ? launch_runs<T, kShifted, kNone, kLayer, -1>(a, sms, s)
                                      : launch_runs<T, kShifted, kNone, kRms, -1>(a, sms, s);
        }
        return launch_runs<T, kShifted, kOpen, kAnyNorm, -1>(a, sms, s);
    }
    // value by value: as few to a thread as the row allows, since each has a load, an
    // address and two parameters of its own (8192 x 2561 BF16: 118 us, with two warps
    // and 64 values to a thread 419)
    constexpr int kRuns[] = {8};
    if (a.cols <= 8 * kThreads) {
        a.warps = form_for(kRuns, a.cols, a.rows, sms).warps;
        return launch<T, kSingle, 8, kOpen, kAnyNorm, -1>(a, sms, s);
    }
    a.warps = kMaxWarps;
    return a.cols <= 16 * kThreads   ? launch<T, kSingle, 16, kOpen, kAnyNorm, -1>(a, sms, s)
           : a.cols <= 32 * kThreads ? launch<T, kSingle, 32, kOpen, kAnyNorm, -1>(a, sms, s)
                                     : launch<T, kSingle, 64, kOpen, kAnyNorm, -1>(a, sms, s);
}

}  // namespace
}  // namespace slide
