// norm_rows.h — what the norm's forward pass (norm_kernel.h, norm.cu) and its
// gradient (norm_back_kernel.h, norm_back.cu) share: runs of values, teams of
// warps, the kernels' arguments and the checks of a call's.
#pragma once
#include <cmath>
#include <initializer_list>
#include <string>
#include <type_traits>

#include "slide.h"
#include "slide_rows.h"
#include "slide_state.h"
#include "sm103_ptx.h"

namespace slide {

constexpr int kMaxCols = 16384;
constexpr unsigned kFull = 0xffffffffu;

// VEC consecutive values as they lie in memory: 8, in 16-byte vectors, or one.
template <typename T, int VEC>
struct Run {
    static constexpr int kBytes = VEC * (int)sizeof(T);
    using Word = std::conditional_t<kBytes == 2, uint16_t, uint32_t>;
    static constexpr int kWords = kBytes <= 4 ? 1 : kBytes / 4;
    Word w[kWords];

    __device__ __forceinline__ void load(const void *p)
    {
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = static_cast<const uint4 *>(p)[i];
                w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
            }
        } else {
            w[0] = *static_cast<const Word *>(p);
        }
    }
    __device__ __forceinline__ void store(void *p) const
    {
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                static_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else {
            *static_cast<Word *>(p) = w[0];
        }
    }
    __device__ __forceinline__ void load_shared(uint32_t p)
    {
        if constexpr (kBytes >= 16) {
#pragma unroll
            for (int i = 0; i < kWords; i += 4)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                             : "r"(p + i * 4)
                             : "memory");
        } else if constexpr (kBytes == 4) {
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(p) : "memory");
        } else {
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w[0]) : "r"(p) : "memory");
        }
    }
    __device__ __forceinline__ Vals<VEC> get() const
    {
        Vals<VEC> v;
        float x[VEC];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                x[i] = __uint_as_float(w[i]);
        } else if constexpr (VEC == 1) {
            x[0] = __uint_as_float((uint32_t)w[0] << 16);
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
        v.set(x);
        return v;
    }
    __device__ __forceinline__ void set(const Vals<VEC> &v)
    {
        float x[VEC];
        v.split_to(x);
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                w[i] = __float_as_uint(x[i]);
        } else if constexpr (VEC == 1) {
            w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
    }
};

// How rows lie.
//   kAligned: every row starts on 16 bytes and is whole runs of eight.
//   kShifted: the tensors are alike (aligned bases, the same stride modulo 8),
//     but a row starts anywhere: its runs are those of the memory, eight values
//     from a multiple of eight on, and the row's first and last may be in part
//     another's.  Run C of a row that starts k values behind such a multiple
//     holds the columns 8*C - k ..., so weights are read at an offset.
//   kSingle: value by value, for anything else.
enum Mode { kAligned = 0, kShifted = 1, kSingle = 2 };

// Values lo .. hi - 1 of a run that is only in part the row's; zeros elsewhere.
template <typename T>
__device__ __forceinline__ void load_part(Run<T, 8> &r, const T *p, int lo, int hi)
{
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = e >= lo && e < hi ? widen(p[e]) : 0.0f;
    Vals<8> v;
    v.set(x);
    r.set(v);
}

template <typename T>
__device__ __forceinline__ void store_part(const Vals<8> &v, T *p, int lo, int hi)
{
    float x[8];
    v.split_to(x);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e >= lo && e < hi)
            p[e] = narrow<T>(x[e]);
}

// A row's run at c (in values from the run that holds the row's start), of a
// row from k to end there: whole, or in part.
template <int MODE>
__device__ __forceinline__ bool whole(int c, int k, int end)
{
    return MODE != kShifted || (c >= k && c + 8 <= end);
}

template <int MODE, typename T, int VEC>
__device__ __forceinline__ void load_run(Run<T, VEC> &r, const T *p, int c, int k, int end)
{
    if (whole<MODE>(c, k, end)) {
        r.load(p);
    } else {
        if constexpr (VEC == 8)
            load_part(r, p, k - c, end - c);
    }
}

template <int MODE, typename T, int VEC>
__device__ __forceinline__ void store_run(const Vals<VEC> &v, T *p, int c, int k, int end)
{
    if (whole<MODE>(c, k, end)) {
        Run<T, VEC> r;
        r.set(v);
        r.store(p);
    } else {
        if constexpr (VEC == 8)
            store_part(v, p, k - c, end - c);
    }
}

// The weight's or bias's values for a run.  kShifted reads them from shared
// memory, where column c stands, in FP32, at [c mod 8][c / 8 + 1]: the lanes of
// a warp read neighbouring words whatever the row's offset.
// WIDE: FP32 in memory, or BF16, or (-1) as the call says.
template <int MODE, int WIDE = -1>
struct Params {
    const void *p;
    const float *s;
    int pitch;
    bool wide_;
    __device__ __forceinline__ bool wide() const { return WIDE < 0 ? wide_ : WIDE != 0; }

    static __host__ __device__ int words(int cols) { return MODE == kShifted ? 8 * (cols / 8 + 3) : 0; }
    __device__ __forceinline__ float one(int c) const
    {
        return wide() ? static_cast<const float *>(p)[c] : widen(static_cast<const bf16 *>(p)[c]);
    }
    // By the whole block; a barrier is due before the first get.
    __device__ __forceinline__ void init(const void *from, bool fp32, float *to, int cols)
    {
        p = from;
        wide_ = fp32;
        s = to;
        pitch = cols / 8 + 3;
        if constexpr (MODE == kShifted) {
            if (p)
                for (int c = threadIdx.x; c < words(cols); c += blockDim.x)
                    to[(c & 7) * pitch + (c >> 3)] = c >= 8 && c - 8 < cols ? one(c - 8) : 0.0f;
        }
    }
    template <int VEC>
    __device__ __forceinline__ Vals<VEC> get(int c, int k) const
    {
        float x[VEC];
        if constexpr (MODE == kShifted) {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                x[e] = s[((e - k) & 7) * pitch + (c >> 3) + 1 - (e < k)];
        } else if constexpr (VEC == 8) {
            if (wide())
                unpack8(load_raw8(static_cast<const float *>(p) + c), x);
            else
                unpack8(load_raw8(static_cast<const bf16 *>(p) + c), x);
        } else {
            x[0] = one(c);
        }
        Vals<VEC> v;
        v.set(x);
        return v;
    }
};

// Dropout of a thread's runs, run by run in order; first: number of the value at
// c = 0, c: the thread's run i, gap: values between its runs, end: of the row.  A
// run of eight is one block of the generator where it starts on one, or lies in
// two.  The single values of a warp's lanes lie in at most five blocks: eight
// lanes form the masks of a run, the warp those of four runs at a time, and each
// value's bit comes from the lane that has it.
template <int VEC>
struct Dropper {
    uint32_t mask;
    __device__ __forceinline__ void run(const Drop &d, uint32_t step, uint64_t first, int i, int c, int gap, int end,
                                        Vals<VEC> &v)
    {
        if constexpr (VEC == 8) {
            if (c < end) {
                const uint64_t e = first + c;
                const int k = (int)(e & 7);
                if (k == 0) {
                    drop8(d, step, e >> 3, v);
                } else {
                    // (a row's first run may start before element 0)
                    const uint32_t m = (keep8(d, step, e >> 3) | keep8(d, step, (e + 8) >> 3) << 8) >> k;
                    float x[8];
                    v.split_to(x);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[j] = m >> j & 1 ? x[j] * d.scale : 0.0f;
                    v.set(x);
                }
            }
        } else {
            const int lane = threadIdx.x & 31, c0 = c - lane;
            if (c0 >= end)  // the same for the whole warp
                return;
            if (i % 4 == 0)
                mask = keep8(d, step, ((first + c0 + (lane >> 3) * gap) >> 3) + (lane & 7));
            const uint64_t f = first + c0, e = f + lane;
            const uint32_t m = __shfl_sync(kFull, mask, (i % 4) * 8 + (int)((e >> 3) - (f >> 3)));
            v.p[0] = m >> (e & 7) & 1 ? v.p[0] * d.scale : 0.0f;
        }
    }
};

// Wait for the `warps` warps of a team (its own barrier), or the warp's lanes.
__device__ __forceinline__ void team_sync(int team, int warps)
{
    if (warps == 1)
        __syncwarp();
    else
        asm volatile("barrier.cta.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
}

// Sums of two values over a team of `warps` warps, on every lane.  red: the
// team's 16 places; between two calls with the same ones the block's threads meet
// at a barrier, so that no warp writes its sums while another still reads.
__device__ __forceinline__ void team_sum2(float &a, float &b, float2 *red, int team, int warps)
{
    const int lane = threadIdx.x & 31;
    float v = lane & 1 ? b : a;  // each lane keeps one of the two
    v += __shfl_xor_sync(kFull, lane & 1 ? a : b, 1);
#pragma unroll
    for (int o = 16; o > 1; o >>= 1)
        v += __shfl_xor_sync(kFull, v, o);
    const float w = __shfl_xor_sync(kFull, v, 1);
    a = lane & 1 ? w : v;
    b = lane & 1 ? v : w;
    if (warps == 1)
        return;
    if (lane == 0)
        red[(threadIdx.x >> 5) % warps] = make_float2(a, b);
    team_sync(team, warps);
    a = b = 0.0f;
    for (int i = 0; i < warps; i += 2) {
        const float4 u = *reinterpret_cast<const float4 *>(red + i);
        a += u.x + u.z;
        b += u.y + u.w;
    }
}

// 1/sqrt: the approximation and a step of Newton's method on y^-2 = v.
__device__ __forceinline__ float inverse_root(float v)
{
    const float y = rsqrtf(v);
    const float e = fmaf(-v * y, y, 1.0f);
    return v > 0.0f && v <= 3.402823466e38f ? fmaf(0.5f * y, e, y) : y;
}

// s/n, given 1/n as FP32 rounds it: the product, and what it leaves of s added.
// An exact quotient comes out exactly, so a row of one value has no variance (a
// product alone made 1000 out of 1601 times 1000 a value 6e-5 above it, and 2 % of
// a deviation of the difference, at eps 1e-5).
__device__ __forceinline__ float quotient(float s, float n, float inv_n)
{
    const float q = s * inv_n;
    return fabsf(q) <= 3.402823466e38f ? fmaf(fmaf(-q, n, s), inv_n, q) : q;
}

struct NormArgs {
    int64_t rows;
    int cols, warps, rms, wide;  // wide: weight and bias are FP32
    float eps, inv_cols;
    const void *x, *residual, *weight, *bias;
    void *sum, *out;
    int64_t xs, rs, ss, os;
    float *mean, *rstd;
    Drop drop;
};

struct NormBackArgs {
    int64_t rows;
    int cols, tile, rms;  // rows of a tile: a power of two
    int wide;             // weight is FP32
    int stages;           // tiles in shared memory: 2, or 1 where two do not fit
    int pitch;            // bytes of a row there
    float inv_cols;
    const void *x, *weight, *d_out, *d_sum;
    const float *mean, *rstd;
    void *d_x, *d_residual;
    int64_t xs, gs, ss, ds, rs;
    float *part_w, *part_b;  // [blocks][cols], or NULL
    Drop drop;
};

constexpr int kParts = 152;  // most partial sums of a weight's gradient: a block on each SM
inline int64_t parts_for(int64_t rows, int tile) { return (rows + tile - 1) / tile < kParts ? (rows + tile - 1) / tile : kParts; }

// One translation unit each.
cudaError_t launch_norm_back_bf16(const NormBackArgs &a, Mode mode, void *d_weight, void *d_bias, float *ws, cudaStream_t s);
cudaError_t launch_norm_back_fp32(const NormBackArgs &a, Mode mode, void *d_weight, void *d_bias, float *ws, cudaStream_t s);
cudaError_t launch_norm_bf16(const NormArgs &a, Mode mode, int sms, cudaStream_t s);
cudaError_t launch_norm_bf16_sum(const NormArgs &a, Mode mode, int sms, cudaStream_t s);
cudaError_t launch_norm_fp32(const NormArgs &a, Mode mode, int sms, cudaStream_t s);
cudaError_t launch_norm_fp32_sum(const NormArgs &a, Mode mode, int sms, cudaStream_t s);

slide_status check_norm(int64_t rows, int32_t cols, const slide_norm_config *c);  // norm.cu

// A tensor of rows.
struct Tensor {
    const char *name;
    const void *p;
    int64_t stride;
    bool needed;
};

// What is wrong with tensors, and in *mode how their rows lie; params: whether
// weight and bias are aligned to 16 bytes (norm.cu).
slide_status check_tensors(std::initializer_list<Tensor> ts, int64_t rows, int32_t cols, size_t size, bool params, Mode *mode);

// What is written may be what is read, row by row in the same places (norm.cu).
bool in_step(const Tensor &w, std::initializer_list<Tensor> reads, int64_t rows);

}  // namespace slide
