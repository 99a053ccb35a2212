// slide_rows.h — what the row-wise operators share: the dropout's generator
// and vectors of eight values.  Device code, and the check of a dropout.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "slide.h"

namespace slide {

struct Drop {
    uint32_t key[20];  // of the ten rounds, two each
    uint32_t site, step;
    const uint32_t *step_dev;
    int64_t first;
    uint32_t limit16;  // limit << 16; 0: nothing is dropped
    float scale;
};

// Checks a dropout (NULL: nothing is dropped) and makes it a kernel's (dropout.cu).
slide_status make_drop(const slide_dropout_config *c, Drop *d);

inline bool misaligned(const void *p, size_t to) { return ((uintptr_t)p % to) != 0; }
inline size_t type_size(int32_t type) { return type == SLIDE_TYPE_FP32 ? 4 : 2; }

// The row that block b of eight values lies in, of rows of cols8 blocks.  The
// division, a sequence of instructions that is much longer in 64 bits, is one of
// 32 where both numbers have no more (a row may have 2^37 blocks).
inline __host__ __device__ int64_t row_of_block(int64_t b, int64_t cols8)
{
    return (uint64_t)(b | cols8) >> 32 ? b / cols8 : (uint32_t)b / (uint32_t)cols8;
}

// Multiprocessors of the current device (dropout.cu).
cudaError_t multiprocessors(int *n);

// VEC FP32 values, two to a register pair and to an instruction; each operation
// is rounded once, none contracted.  (A norm's gradient executes 10 % fewer
// instructions than with one value to an instruction.)
using Pair = unsigned long long;

__device__ __forceinline__ Pair pair(float lo, float hi)
{
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(Pair p, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p)); }

template <int VEC>
struct Vals {
    Pair p[VEC / 2];
    __device__ __forceinline__ static Pair all(float x) { return pair(x, x); }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            p[i] = 0;
    }
    __device__ __forceinline__ void split_to(float (&x)[VEC]) const
    {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            split(p[i], x[2 * i], x[2 * i + 1]);
    }
    __device__ __forceinline__ void set(const float (&x)[VEC])
    {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            p[i] = pair(x[2 * i], x[2 * i + 1]);
    }
    __device__ __forceinline__ float sum() const  // VEC is 8
    {
        Pair a, b, c;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(a) : "l"(p[0]), "l"(p[1]));
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(b) : "l"(p[2]), "l"(p[3]));
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(c) : "l"(a), "l"(b));
        float lo, hi;
        split(c, lo, hi);
        return lo + hi;
    }
};

template <>
struct Vals<1> {
    float p[1];
    __device__ __forceinline__ static float all(float x) { return x; }
    __device__ __forceinline__ void clear() { p[0] = 0.0f; }
    __device__ __forceinline__ void split_to(float (&x)[1]) const { x[0] = p[0]; }
    __device__ __forceinline__ void set(const float (&x)[1]) { p[0] = x[0]; }
    __device__ __forceinline__ float sum() const { return p[0]; }
};

__device__ __forceinline__ Pair add1(Pair a, Pair b)
{
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair mul1(Pair a, Pair b)
{
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair fma1(Pair a, Pair b, Pair c)
{
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float add1(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float mul1(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float fma1(float a, float b, float c) { return fmaf(a, b, c); }

template <int VEC>
constexpr int kPlaces = VEC == 1 ? 1 : VEC / 2;

template <int VEC>
__device__ __forceinline__ Vals<VEC> add(const Vals<VEC> &a, const Vals<VEC> &b)
{
    Vals<VEC> r;
#pragma unroll
    for (int i = 0; i < kPlaces<VEC>; ++i)
        r.p[i] = add1(a.p[i], b.p[i]);
    return r;
}
template <int VEC>
__device__ __forceinline__ Vals<VEC> add(const Vals<VEC> &a, float b)
{
    Vals<VEC> r;
#pragma unroll
    for (int i = 0; i < kPlaces<VEC>; ++i)
        r.p[i] = add1(a.p[i], Vals<VEC>::all(b));
    return r;
}
template <int VEC>
__device__ __forceinline__ Vals<VEC> mul(const Vals<VEC> &a, const Vals<VEC> &b)
{
    Vals<VEC> r;
#pragma unroll
    for (int i = 0; i < kPlaces<VEC>; ++i)
        r.p[i] = mul1(a.p[i], b.p[i]);
    return r;
}
template <int VEC>
__device__ __forceinline__ Vals<VEC> mul(const Vals<VEC> &a, float b)
{
    Vals<VEC> r;
#pragma unroll
    for (int i = 0; i < kPlaces<VEC>; ++i)
        r.p[i] = mul1(a.p[i], Vals<VEC>::all(b));
    return r;
}
template <int VEC>
__device__ __forceinline__ Vals<VEC> fma(const Vals<VEC> &a, const Vals<VEC> &b, const Vals<VEC> &c)
{
    Vals<VEC> r;
#pragma unroll
    for (int i = 0; i < kPlaces<VEC>; ++i)
        r.p[i] = fma1(a.p[i], b.p[i], c.p[i]);
    return r;
}
template <int VEC>
__device__ __forceinline__ Vals<VEC> fma(const Vals<VEC> &a, float b, const Vals<VEC> &c)
{
    Vals<VEC> r;
#pragma unroll
    for (int i = 0; i < kPlaces<VEC>; ++i)
        r.p[i] = fma1(a.p[i], Vals<VEC>::all(b), c.p[i]);
    return r;
}
template <int VEC>
__device__ __forceinline__ Vals<VEC> fma(const Vals<VEC> &a, float b, float c)
{
    Vals<VEC> r;
#pragma unroll
    for (int i = 0; i < kPlaces<VEC>; ++i)
        r.p[i] = fma1(a.p[i], Vals<VEC>::all(b), Vals<VEC>::all(c));
    return r;
}

__device__ __forceinline__ uint32_t drop_step(const Drop &d) { return d.step + (d.step_dev ? __ldg(d.step_dev) : 0u); }

// Philox4x32-10 of (block, site, step): Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC'11.
__device__ __forceinline__ uint4 drop_bits(const Drop &d, uint32_t step, uint64_t block)
{
    uint32_t a = (uint32_t)block, b = (uint32_t)(block >> 32), c = d.site, e = step;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = (uint64_t)a * 0xD2511F53u, q = (uint64_t)c * 0xCD9E8D57u;
        a = (uint32_t)(q >> 32) ^ b ^ d.key[2 * r];
        b = (uint32_t)q;
        c = (uint32_t)(p >> 32) ^ e ^ d.key[2 * r + 1];
        e = (uint32_t)p;
    }
    return make_uint4(a, b, c, e);
}

// The block's eight values through the mask.
__device__ __forceinline__ void drop8(const Drop &d, uint32_t step, uint64_t block, Vals<8> &v)
{
    const uint4 r = drop_bits(d, step, block);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        split(mul1(v.p[i], pair(d.scale, d.scale)), lo, hi);
        v.p[i] = pair((w[i] << 16) >= d.limit16 ? lo : 0.0f, w[i] >= d.limit16 ? hi : 0.0f);
    }
}

// Bit i: the block's value i stays.
__device__ __forceinline__ uint32_t keep8(const Drop &d, uint32_t step, uint64_t block)
{
    const uint4 r = drop_bits(d, step, block);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m |= (uint32_t)((w[i] << 16) >= d.limit16) << (2 * i);
        m |= (uint32_t)(w[i] >= d.limit16) << (2 * i + 1);
    }
    return m;
}

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(bf16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x)
{
    if constexpr (sizeof(T) == 2)
        return __float2bfloat16_rn(x);
    else
        return x;
}

// Eight values as they lie in memory, 16-byte aligned.
template <typename T>
struct Raw8 {
    uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T *p)
{
    Raw8<T> r;
    if constexpr (sizeof(T) == 2) {
        r.v[0] = *reinterpret_cast<const uint4 *>(p);
    } else {
        r.v[0] = *reinterpret_cast<const uint4 *>(p);
        r.v[1] = *(reinterpret_cast<const uint4 *>(p) + 1);
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T> &r, float (&x)[8])
{
    if constexpr (sizeof(T) == 2) {
        const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else {
        const uint32_t u[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = __uint_as_float(u[i]);
    }
}

template <typename T>
__device__ __forceinline__ Raw8<T> pack8(const float (&x)[8])
{
    Raw8<T> r;
    if constexpr (sizeof(T) == 2) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        r.v[0] = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        r.v[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        r.v[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void store_raw8(T *p, const Raw8<T> &r)
{
    *reinterpret_cast<uint4 *>(p) = r.v[0];
    if constexpr (sizeof(T) == 4)
        *(reinterpret_cast<uint4 *>(p) + 1) = r.v[1];
}

}  // namespace slide
