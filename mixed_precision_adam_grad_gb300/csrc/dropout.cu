// dropout.cu — slide_dropout: a mask of random bits by element number, formed
// where it is used, on a tensor or on what is added to the residual stream.
//
// A thread has the eight elements of one block of the generator, 16 bits each,
// so 10 rounds serve eight elements.  Sixteen bits instead of 32 halve the
// generator's work; the rate is rounded to 1/65536 and the scale is that of
// the rounded rate.
//
// Bound by memory: 16384 x 5120 BF16 added to the residual stream (503 MB) 75 us,
// 6.7 TB/s, the rate of a plain copy; 19 instructions an element, of which the
// issue slots are busy 58 % of the time; without a residual 64 us (5.3 TB/s).  Rows
// that no vector fits (an odd base, stride or `first`) go value by value, a block of
// the generator to a thread: 200 to 225 us, FP32 325 to 340.
#include <cmath>
#include <string>

#include <atomic>

#include "slide.h"
#include "slide_rows.h"
#include "slide_state.h"

namespace slide {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 2;  // blocks of eight elements

struct DropoutArgs {
    int64_t rows, cols;
    const void *x, *residual;
    void *out;
    int64_t xs, rs, os;  // strides of rows, in elements
    Drop drop;
};

// Whole blocks of eight within a row, each 16-byte aligned; with `flat` the
// rows lie one behind the other and count as one (cols8 blocks), of which
// `tail` elements behind the last block are left to the last thread.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_dropout_vec(const DropoutArgs a, int64_t blocks, int64_t cols8, int tail)
{
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    T *out = static_cast<T *>(a.out);
    const uint32_t step = drop_step(a.drop);
    const uint64_t first = (uint64_t)a.drop.first >> 3;
    const int64_t b0 = (int64_t)blockIdx.x * (kThreads * kPerThread) + threadIdx.x;
    Raw8<T> rx[kPerThread], rr[kPerThread];
    int64_t row[kPerThread], at[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int64_t b = b0 + i * kThreads;
        row[i] = 0;
        if (blocks != cols8)
            row[i] = row_of_block(b, cols8);
        at[i] = (b - row[i] * cols8) * 8;
        if (b < blocks) {
            rx[i] = load_raw8(x + row[i] * a.xs + at[i]);
            if (res)
                rr[i] = load_raw8(res + row[i] * a.rs + at[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int64_t b = b0 + i * kThreads;
        if (b < blocks) {
            float x[8];
            Vals<8> v, r;
            unpack8(rx[i], x);
            v.set(x);
            if (a.drop.limit16)
                drop8(a.drop, step, first + b, v);
            if (res) {
                unpack8(rr[i], x);
                r.set(x);
                v = add(r, v);
            }
            v.split_to(x);
            store_raw8(out + row[i] * a.os + at[i], pack8<T>(x));
        } else if (b == blocks && tail) {
            const uint32_t keep = a.drop.limit16 ? keep8(a.drop, step, first + b) : 0xffu;
            for (int e = 0; e < tail; ++e) {
                const float v = keep >> e & 1 ? widen(x[at[i] + e]) * a.drop.scale : 0.0f;
                out[at[i] + e] = narrow<T>(res ? __fadd_rn(widen(res[at[i] + e]), v) : v);
            }
        }
    }
}

// Any strides and alignment: a thread has one block of the generator, whose
// elements may lie in several rows.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_dropout_any(const DropoutArgs a, int64_t blocks)
{
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.residual);
    T *out = static_cast<T *>(a.out);
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= blocks)
        return;
    const int64_t n = a.rows * a.cols, block = (a.drop.first >> 3) + i;
    const uint32_t keep = a.drop.limit16 ? keep8(a.drop, drop_step(a.drop), (uint64_t)block) : 0xffu;
    int64_t e = block * 8 - a.drop.first;  // the tensor's element, negative before the first
    int64_t row = e > 0 ? e / a.cols : 0, col = e > 0 ? e - row * a.cols : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j, ++e) {
        if (e >= 0 && e < n) {
            const float v = keep >> j & 1 ? widen(x[row * a.xs + col]) * a.drop.scale : 0.0f;
            out[row * a.os + col] = narrow<T>(res ? __fadd_rn(widen(res[row * a.rs + col]), v) : v);
            if (++col == a.cols) {
                col = 0;
                ++row;
            }
        }
    }
}

template <typename T>
cudaError_t launch(const DropoutArgs &a, cudaStream_t s)
{
    const int64_t n = a.rows * a.cols;
    const bool flat = a.rows == 1 || (a.xs == a.cols && a.os == a.cols && (!a.residual || a.rs == a.cols));
    auto vec = [&](const void *p, int64_t stride) {
        return !misaligned(p, 16) && (flat || (stride * (int64_t)sizeof(T)) % 16 == 0);
    };
    if (a.drop.first % 8 == 0 && (flat || a.cols % 8 == 0) && vec(a.x, a.xs) && vec(a.out, a.os) &&
        (!a.residual || vec(a.residual, a.rs))) {
        const int64_t blocks = n / 8, cols8 = flat ? blocks : a.cols / 8;
        const int64_t grid = (blocks + 1 + kThreads * kPerThread - 1) / (kThreads * kPerThread);  // below 2^29
        k_dropout_vec<T><<<(unsigned)grid, kThreads, 0, s>>>(a, blocks, cols8, flat ? (int)(n % 8) : 0);
    } else {
        const int64_t blocks = ((a.drop.first + n - 1) >> 3) - (a.drop.first >> 3) + 1;
        const int64_t grid = (blocks + kThreads - 1) / kThreads;  // at most 2^29 + 1
        k_dropout_any<T><<<(unsigned)grid, kThreads, 0, s>>>(a, blocks);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t multiprocessors(int *n)
{
    static std::atomic<int> cache[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    *n = dev < 64 ? cache[dev].load(std::memory_order_relaxed) : 0;
    if (*n == 0) {
        e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess && dev < 64)
            cache[dev].store(*n, std::memory_order_relaxed);
    }
    return e;
}

slide_status make_drop(const slide_dropout_config *c, Drop *d)
{
    *d = Drop{};
    d->scale = 1.0f;
    if (!c)
        return SLIDE_OK;
    const double limit = std::floor((double)c->p * 65536.0 + 0.5);
    if (!(c->p >= 0.0f) || !(limit < 65536.0))
        return fail(SLIDE_ERR_INVALID_ARG, "dropout: p must be at least 0 and, rounded to 1/65536, below 1");
    if (c->first < 0 || c->first > ((int64_t)1 << 62))
        return fail(SLIDE_ERR_INVALID_ARG, "dropout: first must lie in [0, 2^62]");
    if (misaligned(c->step_dev, 4))
        return fail(SLIDE_ERR_INVALID_ARG, "dropout: step_dev is not aligned to its type");
    for (uint32_t r = 0; r < 10; ++r) {
        d->key[2 * r] = (uint32_t)c->seed + r * 0x9E3779B9u;
        d->key[2 * r + 1] = (uint32_t)(c->seed >> 32) + r * 0xBB67AE85u;
    }
    d->site = c->site;
    d->step = c->step;
    d->step_dev = c->step_dev;
    d->first = c->first;
    d->limit16 = (uint32_t)limit << 16;
    d->scale = (float)(65536.0 / (65536.0 - limit));
    return SLIDE_OK;
}

}  // namespace slide

using namespace slide;

extern "C" slide_status slide_dropout(int64_t rows, int64_t cols, int32_t type, const void *x, int64_t x_stride,
                                      const void *residual, int64_t residual_stride, void *out, int64_t out_stride,
                                      const slide_dropout_config *cfg, slide_stream_t stream)
{
    constexpr int64_t kMost = (int64_t)1 << 40;
    if (rows < 0 || cols < 0 || (cols > 0 && rows > kMost / cols))
        return fail(SLIDE_ERR_INVALID_ARG, "rows and cols must be >= 0, and rows*cols at most 2^40");
    if (type != SLIDE_TYPE_BF16 && type != SLIDE_TYPE_FP32)
        return fail(SLIDE_ERR_INVALID_ARG, "type must be SLIDE_TYPE_BF16 or SLIDE_TYPE_FP32");
    if (!cfg)
        return fail(SLIDE_ERR_INVALID_ARG, "dropout config is NULL");
    DropoutArgs a{};
    const slide_status rc = make_drop(cfg, &a.drop);
    if (rc != SLIDE_OK)
        return rc;
    if (x_stride < cols || out_stride < cols || (residual && residual_stride < cols))
        return fail(SLIDE_ERR_INVALID_ARG, "a row stride is smaller than cols");
    if (rows == 0 || cols == 0) {
        clear_error();
        return SLIDE_OK;
    }
    const size_t size = type_size(type);
    if (!x || misaligned(x, size) || !out || misaligned(out, size) || misaligned(residual, size))
        return fail(SLIDE_ERR_INVALID_ARG, "x or out is NULL, or x, residual or out is not aligned to its type");
    if (rows > 1 && ((x == out && x_stride != out_stride) || (residual == out && residual_stride != out_stride)))
        return fail(SLIDE_ERR_INVALID_ARG, "in place, the strides must be equal");
    a.rows = rows;
    a.cols = cols;
    a.x = x;
    a.xs = x_stride;
    a.residual = residual;
    a.rs = residual_stride;
    a.out = out;
    a.os = out_stride;
    const cudaError_t e = size == 4 ? launch<float>(a, (cudaStream_t)stream) : launch<bf16>(a, (cudaStream_t)stream);
    if (e != cudaSuccess)
        return fail_cuda(e, "dropout launch");
    clear_error();
    return SLIDE_OK;
}
