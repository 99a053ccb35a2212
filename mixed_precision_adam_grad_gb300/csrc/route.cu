// route.cu — routing of tokens to experts: scores, bias for balance, groups,
// top-k and renormalised weights (slide_route_experts), its gradient
// (slide_route_experts_backward) and the step of the balancing bias
// (slide_route_bias_step).
//
// One warp per token; lane l holds the NV = 1, 2, 4, ... 32 consecutive
// experts from l*NV on, in registers, so a row is read once.  Every choice is
// made on 32-bit keys whose unsigned order is the order of the FP32 values
// (0 = not available), so a pick is the maximum of the lane's keys, one
// warp-wide maximum and a ballot; the lowest lane holding it has the lowest
// expert, which decides ties.  The scores that enter a choice are single FP32
// operations, each rounded, with the accurate exponential: 1 / (1 + exp(-x)).
#include <cuda_runtime.h>
#include <float.h>

#include <atomic>
#include <cmath>
#include <string>

#include "slide.h"
#include "slide_state.h"

namespace slide {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kWarps = 8;
constexpr float kTiny = 1e-20f;
constexpr unsigned kFull = 0xffffffffu;

struct RouteArgs {
    int64_t tokens;
    const void *logits;
    int64_t row_stride;
    const float *bias;
    const uint8_t *mask;
    float *weights;
    int32_t *experts;
    unsigned long long *load;
    int E, K, groups, top_groups, group_size, group_max;
    int renorm;
    float scale;
    int vec;
};

__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 counts as 0
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float value_of(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <typename T>
__device__ __forceinline__ float widen(T x)
{
    if constexpr (sizeof(T) == 2)
        return __uint_as_float((uint32_t)x << 16);
    else
        return x;
}

// The lane's NV consecutive values of a row; -inf beyond its E experts.
template <typename T, int NV>
__device__ __forceinline__ void load_row(const T *row, int lane, int E, bool vec, float (&x)[NV])
{
    const int e0 = lane * NV;
    constexpr int kPer = 16 / sizeof(T);
    if constexpr (NV >= kPer) {
        if (vec && e0 + NV <= E) {
#pragma unroll
            for (int q = 0; q < NV / kPer; ++q) {
                const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(row + e0) + q);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if constexpr (sizeof(T) == 2) {
                        x[q * 8 + 2 * h] = __uint_as_float(u[h] << 16);
                        x[q * 8 + 2 * h + 1] = __uint_as_float(u[h] & 0xffff0000u);
                    } else {
                        x[q * 4 + h] = __uint_as_float(u[h]);
                    }
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        x[i] = e0 + i < E ? widen(row[e0 + i]) : -INFINITY;
}

__device__ __forceinline__ float sigmoid(float x) { return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-x))); }

__device__ __forceinline__ float warp_max(float x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
    return x;
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        x += __shfl_xor_sync(kFull, x, o);
    return x;
}

template <int NV>
__device__ __forceinline__ uint32_t lane_max(const uint32_t (&key)[NV])
{
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < NV; ++i)
        m = max(m, key[i]);
    return m;
}

// Rank of a group from its best two keys (0 = none).
__device__ __forceinline__ uint32_t group_rank(uint32_t k1, uint32_t k2, bool only_max)
{
    if (k1 == 0 || k2 == 0 || only_max)
        return k1;
    return key_of(__fadd_rn(value_of(k1), value_of(k2)));
}

// Drop the keys of all but the best groups.
template <int NV>
__device__ __forceinline__ void keep_groups(uint32_t (&key)[NV], const RouteArgs &a, int lane)
{
    const int gs = a.group_size, lanes = gs / NV;
    if (gs % NV == 0 && (lanes & (lanes - 1)) == 0 && lanes <= 32) {
        // a group is a run of 1, 2, 4, ... lanes: its best two by exchanges
        uint32_t k1 = 0, k2 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            k2 = max(k2, min(k1, key[i]));
            k1 = max(k1, key[i]);
        }
        for (int o = 1; o < lanes; o <<= 1) {
            const uint32_t o1 = __shfl_xor_sync(kFull, k1, o), o2 = __shfl_xor_sync(kFull, k2, o);
            k2 = max(max(k2, o2), min(k1, o1));
            k1 = max(k1, o1);
        }
        const uint32_t rank = group_rank(k1, k2, a.group_max);
        uint32_t left = rank;  // of the lane's group, 0 once it is taken
        for (int p = 0; p < a.top_groups; ++p) {
            const uint32_t m = __reduce_max_sync(kFull, left);
            if (m == 0)
                break;
            const int owner = __ffs(__ballot_sync(kFull, left == m)) - 1;
            if (lane / lanes == owner / lanes)
                left = 0;
        }
        const bool kept = left == 0;  // groups of rank 0 have nothing to drop
#pragma unroll
        for (int i = 0; i < NV; ++i)
            key[i] = kept ? key[i] : 0;
        return;
    }
    // any size: one group after the other; lane g holds the rank of groups g, g + 32, ...
    uint32_t ranks[kMaxExperts / 32];
    const int rounds = (a.groups + 31) / 32;
#pragma unroll
    for (int r = 0; r < kMaxExperts / 32; ++r)
        ranks[r] = 0;
    for (int g = 0; g < a.groups; ++g) {
        uint32_t k1 = 0, k2 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane * NV + i;
            const uint32_t k = e >= g * gs && e < (g + 1) * gs ? key[i] : 0;
            k2 = max(k2, min(k1, k));
            k1 = max(k1, k);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t o1 = __shfl_xor_sync(kFull, k1, o), o2 = __shfl_xor_sync(kFull, k2, o);
            k2 = max(max(k2, o2), min(k1, o1));
            k1 = max(k1, o1);
        }
        const uint32_t rank = group_rank(k1, k2, a.group_max);
#pragma unroll
        for (int r = 0; r < kMaxExperts / 32; ++r)
            if (g == r * 32 + lane)
                ranks[r] = rank;
    }
    uint32_t kept[kMaxExperts / 32];  // bit g of word g / 32, the same in every lane
#pragma unroll
    for (int r = 0; r < kMaxExperts / 32; ++r)
        kept[r] = 0;
    for (int p = 0; p < a.top_groups; ++p) {
        uint32_t mine = 0;
#pragma unroll
        for (int r = 0; r < kMaxExperts / 32; ++r)
            mine = max(mine, ranks[r]);
        const uint32_t m = __reduce_max_sync(kFull, mine);
        if (m == 0)
            break;
        int best = kMaxExperts;
#pragma unroll
        for (int r = kMaxExperts / 32 - 1; r >= 0; --r)
            if (r < rounds && ranks[r] == m)
                best = r * 32 + lane;
        best = __reduce_min_sync(kFull, best);
#pragma unroll
        for (int r = 0; r < kMaxExperts / 32; ++r) {
            if (best == r * 32 + lane)
                ranks[r] = 0;
            if (best >> 5 == r)
                kept[r] |= 1u << (best & 31);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int g = (lane * NV + i) / gs;
        uint32_t word = 0;
#pragma unroll
        for (int r = 0; r < kMaxExperts / 32; ++r)
            if (g >> 5 == r)
                word = kept[r];
        key[i] = word >> (g & 31) & 1 ? key[i] : 0;
    }
}

template <typename T, int NV, bool SIGMOID>
__global__ void __launch_bounds__(kWarps * 32) k_route(const RouteArgs a)
{
    __shared__ unsigned hist[kMaxExperts];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (a.load) {
        for (int e = threadIdx.x; e < a.E; e += kWarps * 32)
            hist[e] = 0;
        __syncthreads();
    }
    float bias[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        bias[i] = a.bias && lane * NV + i < a.E ? a.bias[lane * NV + i] : 0.0f;
    // a softmax keeps the order of the logits: the choice is made on them,
    // except where the scores' values matter (a bias, or sums of a group)
    const bool by_logit = !SIGMOID && !a.bias && (a.groups == 1 || a.group_max);

    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.tokens; t += (int64_t)gridDim.x * kWarps) {
        int my_expert = -1;
        float my_score = 0.0f;
        bool nan = false;
        if (!a.mask || a.mask[t]) {
            float score[NV];
            uint32_t key[NV];
            load_row<T, NV>(static_cast<const T *>(a.logits) + t * a.row_stride, lane, a.E, a.vec, score);
            if constexpr (SIGMOID) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const float x = score[i];
                    score[i] = sigmoid(x);
                    const float v = a.bias ? __fadd_rn(score[i], bias[i]) : score[i];
                    nan |= v != v;
                    key[i] = x == -INFINITY || v == -INFINITY ? 0 : key_of(v);
                }
            } else {
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    nan |= score[i] != score[i];
                    score[i] = fminf(score[i], FLT_MAX);
                    top = fmaxf(top, score[i]);
                }
                top = warp_max(top);
                float sum = 0.0f;
                if (top > -INFINITY) {
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        key[i] = score[i] == -INFINITY ? 0 : key_of(score[i]);
                        score[i] = expf(score[i] - top);
                        sum += score[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        key[i] = 0;
                        score[i] = 0.0f;
                    }
                    sum = 1.0f;
                }
                sum = warp_sum(sum);
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    score[i] = __fdiv_rn(score[i], sum);
                    if (!by_logit) {
                        const float v = a.bias ? __fadd_rn(score[i], bias[i]) : score[i];
                        nan |= v != v;
                        key[i] = key[i] == 0 || v == -INFINITY ? 0 : key_of(v);
                    }
                }
            }
            nan = __any_sync(kFull, nan);
            if (!nan) {
                if (a.groups > 1)
                    keep_groups<NV>(key, a, lane);
                uint32_t mine = lane_max<NV>(key);
                for (int p = 0; p < a.K; ++p) {
                    const uint32_t m = __reduce_max_sync(kFull, mine);
                    if (m == 0)
                        break;
                    const int owner = __ffs(__ballot_sync(kFull, mine == m)) - 1;
                    int at = 0;
                    float s = 0.0f;
                    if (lane == owner) {
#pragma unroll
                        for (int i = NV - 1; i >= 0; --i) {
                            if (key[i] == m) {
                                at = i;
                                s = score[i];
                            }
                        }
#pragma unroll
                        for (int i = 0; i < NV; ++i)
                            key[i] = i == at ? 0 : key[i];
                        mine = lane_max<NV>(key);
                    }
                    at = __shfl_sync(kFull, at, owner);
                    s = __shfl_sync(kFull, s, owner);
                    if (lane == p) {
                        my_expert = owner * NV + at;
                        my_score = s;
                    }
                }
                if (a.renorm)
                    my_score = __fdiv_rn(my_score, __fadd_rn(warp_sum(my_score), kTiny));
                my_score *= a.scale;
            }
        }
        if (lane < a.K) {
            a.experts[t * a.K + lane] = my_expert;
            a.weights[t * a.K + lane] = nan ? __int_as_float(0x7fffffff) : my_score;
            if (a.load && my_expert >= 0)
                atomicAdd(&hist[my_expert], 1u);
        }
    }
    if (a.load) {
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += kWarps * 32)
            if (hist[e])
                atomicAdd(a.load + e, (unsigned long long)hist[e]);
    }
}

struct BackArgs {
    int64_t tokens;
    const void *logits;
    int64_t row_stride;
    const int32_t *experts;
    const float *d_weights;
    const uint8_t *mask;
    void *d_logits;
    int64_t d_stride;
    int E, K, renorm;
    float scale;
    int vec, d_vec;
};

template <typename T>
__device__ __forceinline__ T narrow(float x)
{
    if constexpr (sizeof(T) == 2) {
        const uint32_t u = __float_as_uint(x);
        if ((u & 0x7fffffffu) > 0x7f800000u)
            return (T)((u >> 16) | 0x40u);
        return (T)((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);  // to nearest even
    } else {
        return x;
    }
}

// dlogits of one token per warp.  Only the chosen experts have a gradient,
// except for a softmax that is not renormalised, whose row is dense (DENSE).
template <typename T, int NV, bool SIGMOID, bool DENSE>
__global__ void __launch_bounds__(kWarps * 32) k_route_back(const BackArgs a)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kPer = 16 / sizeof(T);
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.tokens; t += (int64_t)gridDim.x * kWarps) {
        const T *row = static_cast<const T *>(a.logits) + t * a.row_stride;
        T *out = static_cast<T *>(a.d_logits) + t * a.d_stride;
        int e = -1;
        float dw = 0.0f;
        if ((!a.mask || a.mask[t]) && lane < a.K) {
            e = a.experts[t * a.K + lane];
            e = e < a.E ? e : -1;
            if (e >= 0)
                dw = a.d_weights[t * a.K + lane] * a.scale;
        }
        const bool any = __any_sync(kFull, e >= 0);
        float x[NV], top = -INFINITY, sum = 0.0f;
        const float xe = e >= 0 ? fminf(widen(row[e]), FLT_MAX) : -INFINITY;
        float dx = 0.0f, base = 0.0f;
        if (DENSE && any) {
            load_row<T, NV>(row, lane, a.E, a.vec, x);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                x[i] = fminf(x[i], FLT_MAX);
                top = fmaxf(top, x[i]);
            }
            top = warp_max(top);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                x[i] = expf(x[i] - top);
                sum += x[i];
            }
            sum = warp_sum(sum);
            const float p = e >= 0 ? expf(xe - top) / sum : 0.0f;
            base = warp_sum(dw * p);
            dx = p * (dw - base);
            base = -base / sum;
        } else if (any && SIGMOID) {
            const float p = e >= 0 ? sigmoid(xe) : 0.0f;
            float dp = dw;
            if (a.renorm) {
                const float total = warp_sum(p) + kTiny;
                dp = (dw - warp_sum(dw * p) / total) / total;
            }
            dx = dp * p * (1.0f - p);
        } else if (any) {
            top = warp_max(xe);
            float p = e >= 0 ? expf(xe - top) : 0.0f;
            p /= warp_sum(p);
            dx = p * (dw - warp_sum(dw * p));
        }
        // the row, then the chosen experts over it
        if (a.d_vec) {
            if constexpr (DENSE && NV >= kPer) {
#pragma unroll
                for (int q = 0; q < NV / kPer; ++q) {
                    const int at = lane * NV + q * kPer;
                    if (at < a.E) {
                        alignas(16) T w[kPer];
#pragma unroll
                        for (int i = 0; i < kPer; ++i)
                            w[i] = any ? narrow<T>(x[q * kPer + i] * base) : T(0);
                        *reinterpret_cast<uint4 *>(out + at) = *reinterpret_cast<uint4 *>(w);
                    }
                }
            } else if constexpr (!DENSE) {
                for (int at = lane * kPer; at < a.E; at += 32 * kPer)
                    *reinterpret_cast<uint4 *>(out + at) = make_uint4(0, 0, 0, 0);
            }
        }
        if (!a.d_vec || (DENSE && NV < kPer)) {
            if constexpr (DENSE) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (lane * NV + i < a.E)
                        out[lane * NV + i] = any ? narrow<T>(x[i] * base) : T(0);
            } else {
                for (int at = lane; at < a.E; at += 32)
                    out[at] = T(0);
            }
        }
        __syncwarp();
        if (e >= 0)
            out[e] = narrow<T>(dx);
    }
}

// bias += rate * sign(mean load - load); the load starts again from zero.
__global__ void __launch_bounds__(256) k_route_bias(int E, long long *load, float *bias, float rate)
{
    __shared__ long long part[256];
    long long sum = 0;
    for (int e = threadIdx.x; e < E; e += 256)
        sum += load[e];
    part[threadIdx.x] = sum;
    __syncthreads();
    for (int o = 128; o > 0; o >>= 1) {
        if (threadIdx.x < o)
            part[threadIdx.x] += part[threadIdx.x + o];
        __syncthreads();
    }
    const long long total = part[0];
    for (int e = threadIdx.x; e < E; e += 256) {
        const long long d = total - load[e] * E;
        bias[e] = __fadd_rn(bias[e], d > 0 ? rate : d < 0 ? -rate : 0.0f);
        load[e] = 0;
    }
}

cudaError_t sm_count(int *n)
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

template <typename T, int NV>
cudaError_t launch_route(const RouteArgs &a, bool sig, int grid, cudaStream_t s)
{
    if (sig)
        k_route<T, NV, true><<<grid, kWarps * 32, 0, s>>>(a);
    else
        k_route<T, NV, false><<<grid, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_route(const RouteArgs &a, bool sig, int grid, cudaStream_t s)
{
    const int nv = (a.E + 31) / 32;
    if (nv <= 1)
        return launch_route<T, 1>(a, sig, grid, s);
    if (nv <= 2)
        return launch_route<T, 2>(a, sig, grid, s);
    if (nv <= 4)
        return launch_route<T, 4>(a, sig, grid, s);
    if (nv <= 8)
        return launch_route<T, 8>(a, sig, grid, s);
    if (nv <= 16)
        return launch_route<T, 16>(a, sig, grid, s);
    return launch_route<T, 32>(a, sig, grid, s);
}

template <typename T, int NV>
cudaError_t launch_dense(const BackArgs &a, int grid, cudaStream_t s)
{
    k_route_back<T, NV, false, true><<<grid, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_back(const BackArgs &a, bool sig, int grid, cudaStream_t s)
{
    if (sig || a.renorm) {
        if (sig)
            k_route_back<T, 1, true, false><<<grid, kWarps * 32, 0, s>>>(a);
        else
            k_route_back<T, 1, false, false><<<grid, kWarps * 32, 0, s>>>(a);
        return cudaGetLastError();
    }
    const int nv = (a.E + 31) / 32;
    if (nv <= 1)
        return launch_dense<T, 1>(a, grid, s);
    if (nv <= 2)
        return launch_dense<T, 2>(a, grid, s);
    if (nv <= 4)
        return launch_dense<T, 4>(a, grid, s);
    if (nv <= 8)
        return launch_dense<T, 8>(a, grid, s);
    if (nv <= 16)
        return launch_dense<T, 16>(a, grid, s);
    return launch_dense<T, 32>(a, grid, s);
}

bool misaligned(const void *p, size_t to) { return ((uintptr_t)p % to) != 0; }

slide_status check_route(int64_t tokens, const slide_route_config *c, int32_t type)
{
    if (tokens < 0 || tokens > ((int64_t)1 << 40))
        return fail(SLIDE_ERR_INVALID_ARG, "tokens must lie in [0, 2^40]");
    if (type != SLIDE_TYPE_BF16 && type != SLIDE_TYPE_FP32)
        return fail(SLIDE_ERR_INVALID_ARG, "logits_type must be SLIDE_TYPE_BF16 or SLIDE_TYPE_FP32");
    if (!c)
        return fail(SLIDE_ERR_INVALID_ARG, "route config is NULL");
    if (c->n_experts < 1 || c->n_experts > kMaxExperts)
        return fail(SLIDE_ERR_INVALID_ARG, "route config: n_experts must lie in [1, 1024]");
    if (c->score != SLIDE_SCORE_SOFTMAX && c->score != SLIDE_SCORE_SIGMOID)
        return fail(SLIDE_ERR_INVALID_ARG, "route config: unknown score");
    if (c->group_score != SLIDE_GROUP_TOP2 && c->group_score != SLIDE_GROUP_MAX)
        return fail(SLIDE_ERR_INVALID_ARG, "route config: unknown group_score");
    if (c->n_groups < 1 || c->n_experts % c->n_groups != 0)
        return fail(SLIDE_ERR_INVALID_ARG, "route config: n_groups must divide n_experts");
    if (c->top_groups < 1 || c->top_groups > c->n_groups)
        return fail(SLIDE_ERR_INVALID_ARG, "route config: top_groups must lie in [1, n_groups]");
    if (c->top_k < 1 || c->top_k > kMaxTopK || c->top_k > c->n_experts / c->n_groups * c->top_groups)
        return fail(SLIDE_ERR_INVALID_ARG, "route config: top_k must lie in [1, 32] and not exceed the experts of "
                                           "top_groups groups");
    if (!std::isfinite(c->scale))
        return fail(SLIDE_ERR_INVALID_ARG, "route config: non-finite scale");
    return SLIDE_OK;
}

int grid_for(int64_t tokens, int sms, int per_sm)
{
    const int64_t blocks = (tokens + kWarps - 1) / kWarps;
    const int64_t most = (int64_t)sms * per_sm;
    return (int)(blocks < most ? blocks : most);
}

}  // namespace
}  // namespace slide

using namespace slide;

extern "C" slide_status slide_route_experts(int64_t tokens, const void *logits, int32_t logits_type,
                                            int64_t logits_stride, const float *bias, const uint8_t *token_mask,
                                            const slide_route_config *cfg, float *weights, int32_t *experts,
                                            int64_t *load, slide_stream_t stream)
{
    slide_status rc = check_route(tokens, cfg, logits_type);
    if (rc != SLIDE_OK)
        return rc;
    if (logits_stride < cfg->n_experts)
        return fail(SLIDE_ERR_INVALID_ARG, "logits_stride is smaller than n_experts");
    if (tokens == 0) {
        clear_error();
        return SLIDE_OK;
    }
    const size_t size = logits_type == SLIDE_TYPE_FP32 ? 4 : 2;
    if (!logits || misaligned(logits, size) || !weights || misaligned(weights, 4) || !experts || misaligned(experts, 4))
        return fail(SLIDE_ERR_INVALID_ARG, "logits, weights or experts is NULL or not aligned to its type");
    if (misaligned(bias, 4) || misaligned(load, 8))
        return fail(SLIDE_ERR_INVALID_ARG, "bias or load is not aligned to its type");
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess)
        return fail_cuda(e, "device query");
    RouteArgs a{};
    a.tokens = tokens;
    a.logits = logits;
    a.row_stride = logits_stride;
    a.bias = bias;
    a.mask = token_mask;
    a.weights = weights;
    a.experts = experts;
    a.load = reinterpret_cast<unsigned long long *>(load);
    a.E = cfg->n_experts;
    a.K = cfg->top_k;
    a.groups = cfg->n_groups;
    a.top_groups = cfg->top_groups;
    a.group_size = cfg->n_experts / cfg->n_groups;
    a.group_max = cfg->group_score == SLIDE_GROUP_MAX;
    a.renorm = cfg->renormalize != 0;
    a.scale = cfg->scale;
    a.vec = !misaligned(logits, 16) && (logits_stride * size) % 16 == 0;
    const int grid = grid_for(tokens, sms, 8);
    const bool sig = cfg->score == SLIDE_SCORE_SIGMOID;
    e = size == 4 ? launch_route<float>(a, sig, grid, (cudaStream_t)stream)
                  : launch_route<uint16_t>(a, sig, grid, (cudaStream_t)stream);
    if (e != cudaSuccess)
        return fail_cuda(e, "routing launch");
    clear_error();
    return SLIDE_OK;
}

extern "C" slide_status slide_route_experts_backward(int64_t tokens, const void *logits, int32_t logits_type,
                                                     int64_t logits_stride, const int32_t *experts,
                                                     const float *d_weights, const uint8_t *token_mask,
                                                     const slide_route_config *cfg, void *d_logits,
                                                     int64_t d_logits_stride, slide_stream_t stream)
{
    slide_status rc = check_route(tokens, cfg, logits_type);
    if (rc != SLIDE_OK)
        return rc;
    if (logits_stride < cfg->n_experts || d_logits_stride < cfg->n_experts)
        return fail(SLIDE_ERR_INVALID_ARG, "logits_stride or d_logits_stride is smaller than n_experts");
    if (tokens == 0) {
        clear_error();
        return SLIDE_OK;
    }
    const size_t size = logits_type == SLIDE_TYPE_FP32 ? 4 : 2;
    if (!logits || misaligned(logits, size) || !d_logits || misaligned(d_logits, size))
        return fail(SLIDE_ERR_INVALID_ARG, "logits or d_logits is NULL or not aligned to its type");
    if (!experts || misaligned(experts, 4) || !d_weights || misaligned(d_weights, 4))
        return fail(SLIDE_ERR_INVALID_ARG, "experts or d_weights is NULL or not aligned to its type");
    if (logits == d_logits)
        return fail(SLIDE_ERR_INVALID_ARG, "d_logits must not be the logits");
    int sms = 0;
    cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess)
        return fail_cuda(e, "device query");
    BackArgs a{};
    a.tokens = tokens;
    a.logits = logits;
    a.row_stride = logits_stride;
    a.experts = experts;
    a.d_weights = d_weights;
    a.mask = token_mask;
    a.d_logits = d_logits;
    a.d_stride = d_logits_stride;
    a.E = cfg->n_experts;
    a.K = cfg->top_k;
    a.renorm = cfg->renormalize != 0;
    a.scale = cfg->scale;
    const size_t per = 16 / size;
    a.vec = !misaligned(logits, 16) && (logits_stride * size) % 16 == 0;
    a.d_vec = !misaligned(d_logits, 16) && (d_logits_stride * size) % 16 == 0 && cfg->n_experts % per == 0;
    const int grid = grid_for(tokens, sms, 8);
    const bool sig = cfg->score == SLIDE_SCORE_SIGMOID;
    e = size == 4 ? launch_back<float>(a, sig, grid, (cudaStream_t)stream)
                  : launch_back<uint16_t>(a, sig, grid, (cudaStream_t)stream);
    if (e != cudaSuccess)
        return fail_cuda(e, "routing gradient launch");
    clear_error();
    return SLIDE_OK;
}

extern "C" slide_status slide_route_bias_step(int32_t n_experts, int64_t *load, float *bias, float rate,
                                              slide_stream_t stream)
{
    if (n_experts < 1 || n_experts > kMaxExperts)
        return fail(SLIDE_ERR_INVALID_ARG, "n_experts must lie in [1, 1024]");
    if (!load || misaligned(load, 8) || !bias || misaligned(bias, 4))
        return fail(SLIDE_ERR_INVALID_ARG, "load or bias is NULL or not aligned to its type");
    if (!std::isfinite(rate) || rate < 0.0f)
        return fail(SLIDE_ERR_INVALID_ARG, "rate must be finite and >= 0");
    k_route_bias<<<1, 256, 0, (cudaStream_t)stream>>>(n_experts, reinterpret_cast<long long *>(load), bias, rate);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return fail_cuda(e, "bias step launch");
    clear_error();
    return SLIDE_OK;
}
