// route.cu — routing of tokens to experts: scores, bias for balance, groups,
// top-k and renormalised weights (slide_route_experts), its gradient
// (slide_route_experts_backward) and the step of the balancing bias
// (slide_route_bias_step).
//
// A token has LPT = 8, 16 or 32 lanes of a warp (a warp 32/LPT tokens); its
// lane l holds the NV = 2, 4, 8, 16 or 32 consecutive experts from l*NV on, in
// registers, so a row is read once.  Every choice is
// made on 32-bit keys whose unsigned order is the order of the FP32 values
// (those up to the key of -inf: not available).  Each lane sorts its keys once, in runs of at most
// eight, so that a pick is one maximum of the runs' heads over the token's lanes, a ballot
// and a shift in the lane that held it; the lowest lane holding the maximum
// has the lowest expert, which decides ties.  Which experts they were is
// looked up at the end, all picks at once: lane p finds pick p's key among its
// owner's, and of equal ones takes the next that no earlier pick took.  The
// chosen experts' scores are formed again from their logits.
// The scores that enter a choice are single FP32 operations, each rounded,
// with the accurate exponential: 1 / (1 + exp(-x)).
//
// Bound by instructions: at 65536 tokens x 256 experts (8 groups, top 8) the
// rows take 11 us from memory, the kernel 64 us, 786 instructions a token: a
// quarter of them the FP32 sigmoids, 18 % the picks, 14 % the groups.  Eight experts per lane are best: 16 lanes
// of 16 there took 94 us (the sort and the pops of two runs), while 8 lanes of
// 8 need less than half the instructions of 32 lanes of 2 for 60 experts.
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
constexpr int kWarps = 8;      // of a block
constexpr int kAnyWarps = 4;   // where each needs shared memory
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
    int vec, bias_vec;
};

constexpr uint32_t kKeyNone = 0x007fffffu, kKeyInf = 0xff800000u;  // keys of -inf and inf

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

__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(__fadd_rn(1.0f, expf(-x))); }

// The bias of the lane's experts (0 beyond the last), four at a time where
// they are aligned.
template <int NV>
__device__ __forceinline__ void load_bias(const RouteArgs &a, int lane, float (&b)[NV])
{
    const int e0 = lane * NV;
    if constexpr (NV >= 4) {
        if (a.bias_vec && e0 + NV <= a.E) {
#pragma unroll
            for (int q = 0; q < NV / 4; ++q) {
                const float4 w = __ldg(reinterpret_cast<const float4 *>(a.bias + e0) + q);
                b[4 * q] = w.x, b[4 * q + 1] = w.y, b[4 * q + 2] = w.z, b[4 * q + 3] = w.w;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (e0 + i < a.E)
            b[i] = __ldg(a.bias + e0 + i);
}

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

// Sorted keys: L = 1, 2 or 4 runs of R = min(NV, 8), largest first.
template <int NV>
struct Runs {
    static constexpr int R = NV < 8 ? NV : 8, L = NV / R;
    uint32_t key[L][R];
};

template <int NV>
__device__ __forceinline__ void sort_runs(const uint32_t (&key)[NV], Runs<NV> &r)
{
    constexpr int R = Runs<NV>::R, L = Runs<NV>::L;
#pragma unroll
    for (int l = 0; l < L; ++l) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            r.key[l][i] = key[l * R + i];
        // odd-even merge sort
#pragma unroll
        for (int p = 1; p < R; p *= 2) {
#pragma unroll
            for (int k = p; k >= 1; k /= 2) {
#pragma unroll
                for (int j = k % p; j + k < R; j += 2 * k) {
#pragma unroll
                    for (int i = 0; i < k; ++i) {
                        if (i + j + k < R && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                            const uint32_t x = r.key[l][i + j], y = r.key[l][i + j + k];
                            r.key[l][i + j] = max(x, y);
                            r.key[l][i + j + k] = min(x, y);
                        }
                    }
                }
            }
        }
    }
}

template <int NV>
__device__ __forceinline__ uint32_t head(const Runs<NV> &r)
{
    uint32_t m = r.key[0][0];
#pragma unroll
    for (int l = 1; l < Runs<NV>::L; ++l)
        m = max(m, r.key[l][0]);
    return m;
}

// If `here`, takes the head m off one run that has it.
template <int NV>
__device__ __forceinline__ void pop(Runs<NV> &r, uint32_t m, bool here)
{
    constexpr int R = Runs<NV>::R, L = Runs<NV>::L;
#pragma unroll
    for (int l = 0; l < L; ++l) {
        const bool this_one = here && (L == 1 || r.key[l][0] == m);
        here = here && !this_one;
#pragma unroll
        for (int i = 0; i + 1 < R; ++i)
            r.key[l][i] = this_one ? r.key[l][i + 1] : r.key[l][i];
        r.key[l][R - 1] = this_one ? 0 : r.key[l][R - 1];
    }
}

// Rank of a group from its best two keys; 0: it has none.
__device__ __forceinline__ uint32_t group_rank(uint32_t k1, uint32_t k2, bool only_max)
{
    if (k1 <= kKeyNone)
        return 0;
    if (k2 <= kKeyNone || only_max)
        return k1;
    return key_of(__fadd_rn(value_of(k1), value_of(k2)));
}

// Maximum over the LPT lanes of a token.
template <int LPT>
__device__ __forceinline__ uint32_t token_max(uint32_t x)
{
    if constexpr (LPT == 32)
        return __reduce_max_sync(kFull, x);
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1)
        x = max(x, __shfl_xor_sync(kFull, x, o));
    return x;
}

template <int LPT>
__device__ __forceinline__ float token_sum(float x)
{
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1)
        x += __shfl_xor_sync(kFull, x, o);
    return x;
}

// The token's lanes for which `is` holds, as the lowest bits.
template <int LPT>
__device__ __forceinline__ uint32_t token_ballot(bool is, int lane)
{
    const uint32_t b = __ballot_sync(kFull, is);
    if constexpr (LPT == 32)
        return b;
    return (b >> (lane & ~(LPT - 1))) & ((1u << (LPT & 31)) - 1);
}

// For groups of 1, 2, 4, ... whole lanes: whether the lane's is one of the best,
// from the lane's sorted keys.
template <int LPT, int NV>
__device__ __forceinline__ bool lane_kept(const Runs<NV> &r, const RouteArgs &a, int lane)
{
    const int lanes = a.group_size / NV;
    uint32_t k1 = 0, k2 = 0;
#pragma unroll
    for (int l = 0; l < Runs<NV>::L; ++l) {
        k2 = max(max(k2, r.key[l][1]), min(k1, r.key[l][0]));
        k1 = max(k1, r.key[l][0]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(kFull, k1, o), o2 = __shfl_xor_sync(kFull, k2, o);
        k2 = max(max(k2, o2), min(k1, o1));
        k1 = max(k1, o1);
    }
    uint32_t left = group_rank(k1, k2, a.group_max);  // of the lane's group, 0 once it is taken
    const int my = lane & (LPT - 1);
    for (int p = 0; p < a.top_groups; ++p) {
        const uint32_t m = token_max<LPT>(left);
        const int owner = __ffs(token_ballot<LPT>(left == m, lane)) - 1;
        if (((my ^ owner) & ~(lanes - 1)) == 0)
            left = 0;
    }
    return left == 0;  // groups of rank 0 have nothing to drop
}

// Groups of any size: drop the keys of all but the best.  keys and ranks: the
// warp's shared memory, E and a.groups words.
template <int NV>
__device__ __forceinline__ void keep_groups(uint32_t (&key)[NV], const RouteArgs &a, int lane, uint32_t *keys,
                                            uint32_t *ranks)
{
    const int gs = a.group_size;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (lane * NV + i < a.E)
            keys[lane * NV + i] = key[i];
    __syncwarp();
    uint32_t mine = 0;  // best rank of the lane's groups lane, lane + 32, ...
    for (int g = lane; g < a.groups; g += 32) {
        uint32_t k1 = 0, k2 = 0;
        for (int e = g * gs; e < (g + 1) * gs; ++e) {
            k2 = max(k2, min(k1, keys[e]));
            k1 = max(k1, keys[e]);
        }
        ranks[g] = group_rank(k1, k2, a.group_max);
        mine = max(mine, ranks[g]);
    }
    for (int p = 0; p < a.top_groups; ++p) {
        const uint32_t m = __reduce_max_sync(kFull, mine);
        if (m == 0)
            break;
        int best = a.groups;
        if (mine == m)
            for (best = lane; ranks[best] != m; best += 32)
                ;
        best = __reduce_min_sync(kFull, best);
        if (lane == (best & 31)) {
            ranks[best] = 0;  // taken
            mine = 0;
            for (int g = lane; g < a.groups; g += 32)
                mine = max(mine, ranks[g]);
        }
    }
    __syncwarp();
    // a group that had a rank and was not taken is dropped
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (lane * NV + i < a.E && ranks[(lane * NV + i) / gs] != 0)
            key[i] = 0;
}

// ANY: the groups are not runs of lanes; each warp (LPT is 32) then has E +
// groups words of shared memory.
template <typename T, int LPT, int NV, bool SIGMOID, bool ANY>
__global__ void __launch_bounds__((ANY ? kAnyWarps : kWarps) * 32) k_route(const RouteArgs a)
{
    constexpr int kWarpsHere = ANY ? kAnyWarps : kWarps, kTokens = 32 / LPT;
    __shared__ unsigned hist[kMaxExperts];
    extern __shared__ uint32_t words[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, my = lane & (LPT - 1);
    if (a.load) {
        for (int e = threadIdx.x; e < a.E; e += kWarpsHere * 32)
            hist[e] = 0;
        __syncthreads();
    }
    // a softmax keeps the order of the logits: the choice is made on them,
    // except where the scores' values matter (a bias, or sums of a group)
    const bool by_logit = !SIGMOID && !a.bias && (a.groups == 1 || a.group_max);
    const bool by_lane = !ANY && a.groups > 1;

    for (int64_t t0 = ((int64_t)blockIdx.x * kWarpsHere + warp) * kTokens; t0 < a.tokens;
         t0 += (int64_t)gridDim.x * kWarpsHere * kTokens) {
        const int64_t t = t0 + lane / LPT;
        const bool in = t < a.tokens, live = in && (!a.mask || a.mask[t]);
        const T *row = static_cast<const T *>(a.logits) + t * a.row_stride;
        float x[NV], top = 0.0f, sum = 1.0f;
        uint32_t key[NV];
        bool nan = false;
        if (live) {
            load_row<T, NV>(row, my, a.E, a.vec, x);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                x[i] = -INFINITY;
        }
        if constexpr (SIGMOID) {
            float bias[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i)
                bias[i] = 0.0f;
            if (a.bias)
                load_bias<NV>(a, my, bias);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                // neither a score nor its sum with a bias is -0
                const uint32_t u = __float_as_uint(__fadd_rn(sigmoid(x[i]), bias[i]));
                key[i] = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
                key[i] = x[i] == -INFINITY ? 0 : key[i];
            }
        } else {
            top = -INFINITY;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                nan |= x[i] != x[i];
                x[i] = fminf(x[i], FLT_MAX);
                top = fmaxf(top, x[i]);
                key[i] = key_of(x[i]);
            }
#pragma unroll
            for (int o = LPT / 2; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
            top = fmaxf(top, -FLT_MAX);  // where nothing is available
            if (!(by_logit && a.renorm)) {
                // scores are needed: for the keys, or for the weights' scale
                sum = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    x[i] = expf(x[i] - top);
                    sum += x[i];
                }
                sum = token_sum<LPT>(sum);
                if (!by_logit) {
                    float bias[NV];
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        bias[i] = 0.0f;
                    if (a.bias)
                        load_bias<NV>(a, my, bias);
#pragma unroll
                    for (int i = 0; i < NV; ++i)
                        key[i] = key[i] <= kKeyNone ? 0 : key_of(__fadd_rn(__fdiv_rn(x[i], sum), bias[i]));
                }
            }
        }
        if constexpr (ANY) {
            uint32_t *mine = words + warp * (a.E + a.groups);
            keep_groups<NV>(key, a, lane, mine, mine + a.E);
        }
        Runs<NV> runs;
        sort_runs<NV>(key, runs);
        uint32_t mine = head<NV>(runs);
        nan = token_ballot<LPT>(nan || mine > kKeyInf, lane) != 0;
        const bool kept = !by_lane || lane_kept<LPT, NV>(runs, a, lane);
        mine = kept ? mine : 0;
        uint32_t my_key = 0;  // lane p: pick p's key and its owner
        int my_owner = 0;
        for (int p = 0; p < a.K; ++p) {
            const uint32_t m = token_max<LPT>(mine);
            const int owner = __ffs(token_ballot<LPT>(mine == m, lane)) - 1;
            my_key = my == p ? m : my_key;
            my_owner = my == p ? owner : my_owner;
            pop<NV>(runs, m, my == owner);
            mine = kept ? head<NV>(runs) : 0;
        }
        int best = -1;  // lane p: the expert of pick p
        const int from = (lane & ~(LPT - 1)) + my_owner;
        // equal keys of one lane are picked one after the other
        const bool same_key = __shfl_up_sync(kFull, my_key, 1) == my_key;
        const bool same_owner = __shfl_up_sync(kFull, my_owner, 1) == my_owner;
        const bool again = my > 0 && my < a.K && same_key && same_owner;
        if (!__any_sync(kFull, again)) {
#pragma unroll
            for (int i = NV - 1; i >= 0; --i)
                best = __shfl_sync(kFull, key[i], from) == my_key ? i : best;
        } else {
            int nth = 0;  // which of the owner's equal keys it is
            for (int p = 1; p < a.K; ++p) {
                const int before = __shfl_up_sync(kFull, nth, 1);
                nth = my == p ? (again ? before + 1 : 0) : nth;
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const bool is = __shfl_sync(kFull, key[i], from) == my_key;
                best = is && nth == 0 ? i : best;
                nth -= is;
            }
        }
        best += my_owner * NV;
        best = my_key <= kKeyNone || nan || !live ? -1 : best;
        const float y = best >= 0 ? widen(row[best]) : -INFINITY;
        float score = 0.0f;
        if constexpr (SIGMOID) {
            if (best >= 0)
                score = sigmoid(y);
        } else {
            if (a.renorm && !by_logit) {
                // a bias can leave the row's largest logit out: relative to the
                // largest chosen one, as the gradient has it
                top = fminf(y, FLT_MAX), sum = 1.0f;
#pragma unroll
                for (int o = LPT / 2; o > 0; o >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
            }
            if (best >= 0)
                score = __fdiv_rn(expf(fminf(y, FLT_MAX) - top), sum);
        }
        if (a.renorm)
            score = __fdiv_rn(score, __fadd_rn(token_sum<LPT>(score), kTiny));
        if (in && my < a.K) {
            a.experts[t * a.K + my] = best;
            a.weights[t * a.K + my] = nan && live ? __int_as_float(0x7fffffff) : score * a.scale;
            if (a.load && best >= 0)
                atomicAdd(&hist[best], 1u);
        }
    }
    if (a.load) {
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += kWarpsHere * 32)
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

// Gradients of normalised weights are differences: of an expert's upstream
// value g_i and the mean sum_j p_j g_j of the token's, times p_i.  The
// difference is formed as sum_j p_j (g_i - g_j), term by term: where one expert
// has nearly all the weight, g_i - sum_j p_j g_j keeps no digit of its gradient.

// Gradient where only the chosen experts have one: W = 1, 2, 4, ... 32 lanes
// (at least top_k) per token, 32/W tokens per warp at a time.  The rows are
// filled with zeros, then the chosen experts' values go over them.
template <typename T, bool SIGMOID>
__global__ void __launch_bounds__(kWarps * 32) k_route_back_sparse(const BackArgs a, int W)
{
    const int lane = threadIdx.x & 31;
    constexpr int kPer = 16 / sizeof(T);
    const int at_once = 32 / W, place = lane & (W - 1);
    const int64_t step = (int64_t)gridDim.x * kWarps * at_once;
    for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * at_once; t0 < a.tokens; t0 += step) {
        const int64_t t = t0 + lane / W;
        int e = -1;
        float dw = 0.0f;
        if (t < a.tokens && place < a.K && (!a.mask || a.mask[t])) {
            e = a.experts[t * a.K + place];
            dw = a.d_weights[t * a.K + place];
            if (e < 0 || e >= a.E) {
                e = -1;
                dw = 0.0f;
            }
        }
        const float x = e >= 0 ? fminf(widen(static_cast<const T *>(a.logits)[t * a.row_stride + e]), FLT_MAX) : -INFINITY;
        // the rows of the warp's tokens, in whole vectors where they are aligned
        const int rows = (int)(a.tokens - t0 < at_once ? a.tokens - t0 : at_once);
        for (int r = 0; r < rows; ++r) {
            T *out = static_cast<T *>(a.d_logits) + (t0 + r) * a.d_stride;
            if (a.d_vec) {
                for (int c = lane * kPer; c < a.E; c += 32 * kPer)
                    *reinterpret_cast<uint4 *>(out + c) = make_uint4(0, 0, 0, 0);
            } else {
                for (int c = lane; c < a.E; c += 32)
                    out[c] = T(0);
            }
        }
        auto sum_of = [&](float v) {  // over the token's lanes
            for (int o = 1; o < W; o <<= 1)
                v += __shfl_xor_sync(kFull, v, o);
            return v;
        };
        auto differences = [&](float p) {  // sum_j p_j (dw - dw_j)
            float v = 0.0f;
            auto add = [&](int o) {
                v = fmaf(__shfl_xor_sync(kFull, p, o), dw - __shfl_xor_sync(kFull, dw, o), v);
            };
            if (W > 1)
                add(1);
            if (W > 2)
                add(2), add(3);
            for (int o = 4; o < W; o += 4)
                add(o), add(o + 1), add(o + 2), add(o + 3);
            return v;
        };
        float dx;
        if constexpr (SIGMOID) {
            const float p = e >= 0 ? sigmoid(x) : 0.0f;
            const float q = x > 0.0f ? expf(-x) * p : 1.0f - p;  // 1 - p without cancellation
            float dp = dw;
            if (a.renorm) {
                const float total = sum_of(p) + kTiny;
                dp = fmaf(dw, kTiny, differences(p)) / total / total;
            }
            dx = dp * a.scale * p * q;
        } else {
            float top = x;
            for (int o = 1; o < W; o <<= 1)
                top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
            float p = e >= 0 ? expf(x - top) : 0.0f;
            const float total = sum_of(p);
            p = total > 0.0f ? p / total : 0.0f;
            dx = p * differences(p) * a.scale;
        }
        __syncwarp();
        if (e >= 0)
            static_cast<T *>(a.d_logits)[t * a.d_stride + e] = narrow<T>(dx);
    }
}

// Gradient of a softmax that is not renormalised: the whole row, one token per
// warp.  65536 x 256 FP32 33 us (134 MB): five sums over the warp a token, one
// after another; 28 us with the cancelling difference.
template <typename T, int NV>
__global__ void __launch_bounds__(kWarps * 32) k_route_back_dense(const BackArgs a)
{
    __shared__ unsigned chosen[kWarps][32];
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
                dw = a.d_weights[t * a.K + lane];
        }
        const bool any = __any_sync(kFull, e >= 0);
        float x[NV], dx = 0.0f, base = 0.0f;
        if (any) {
            chosen[warp][lane] = 0;  // a bit for each expert
            __syncwarp();
            if (e >= 0)
                atomicOr(&chosen[warp][e >> 5], 1u << (e & 31));
            const float xe = e >= 0 ? fminf(widen(row[e]), FLT_MAX) : -INFINITY;
            float top = -INFINITY, rest = 0.0f;
            load_row<T, NV>(row, lane, a.E, a.vec, x);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                x[i] = fminf(x[i], FLT_MAX);
                top = fmaxf(top, x[i]);
            }
            top = warp_max(top);
            __syncwarp();
            const unsigned mine = chosen[warp][lane * NV >> 5] >> (lane * NV & 31);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                x[i] = expf(x[i] - top);
                rest += mine >> i & 1 ? 0.0f : x[i];
            }
            float p = e >= 0 ? expf(xe - top) : 0.0f;
            rest = warp_sum(rest);
            float all = warp_sum(p);
            const float one = 1.0f / (rest + all);
            p *= one;
            all *= one;
            rest *= one;
            // g_i - sum_j p_j g_j = (g_i - g_r) sum_j p_j - sum_j p_j (g_j - g_r) + g_i (1 - sum_j p_j), r the
            // expert with the largest p
            const unsigned largest = __reduce_max_sync(kFull, __float_as_uint(p));
            const int at = __ffs(__ballot_sync(kFull, __float_as_uint(p) == largest)) - 1;
            const float dr = __shfl_sync(kFull, dw, at), h = e >= 0 ? dw - dr : 0.0f;
            const float mean = warp_sum(p * h);
            dx = p * fmaf(dw, rest, fmaf(h, all, -mean)) * a.scale;
            base = -fmaf(dr, all, mean) * one * a.scale;
        }
        // the row, then the chosen experts over it
        bool done = false;
        if constexpr (NV >= kPer) {
            if (a.d_vec) {
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
                done = true;
            }
        }
        if (!done) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (lane * NV + i < a.E)
                    out[lane * NV + i] = any ? narrow<T>(x[i] * base) : T(0);
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

// Launches `kernel` with blocks of `warps` warps for `units` warps' worth of
// work, but no more blocks than the device holds at once (*resident caches
// that number per kernel).
template <typename Kernel, typename... Args>
cudaError_t launch_warps(Kernel kernel, std::atomic<int> &resident, int64_t units, int warps, size_t smem, int sms,
                         cudaStream_t s, Args... args)
{
    int per_sm = resident.load(std::memory_order_relaxed);
    if (per_sm == 0) {
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, warps * 32, smem);
        if (e != cudaSuccess)
            return e;
        per_sm = per_sm > 0 ? per_sm : 1;
        if (smem == 0)
            resident.store(per_sm, std::memory_order_relaxed);
    }
    const int64_t blocks = (units + warps - 1) / warps, most = (int64_t)sms * per_sm;
    kernel<<<(unsigned)(blocks < most ? blocks : most), warps * 32, smem, s>>>(args...);
    return cudaGetLastError();
}

template <typename T, int LPT, int NV, bool ANY>
cudaError_t launch_route(const RouteArgs &a, bool sig, int sms, cudaStream_t s)
{
    static std::atomic<int> resident[2];
    const int warps = ANY ? kAnyWarps : kWarps;
    const size_t smem = ANY ? sizeof(uint32_t) * kAnyWarps * (a.E + a.groups) : 0;  // at most 32 KiB
    const int64_t units = (a.tokens + 32 / LPT - 1) / (32 / LPT);
    return sig ? launch_warps(k_route<T, LPT, NV, true, ANY>, resident[0], units, warps, smem, sms, s, a)
               : launch_warps(k_route<T, LPT, NV, false, ANY>, resident[1], units, warps, smem, sms, s, a);
}

// Whether groups of this size are runs of 1, 2, 4, ... lanes of nv experts.
bool runs_of_lanes(const RouteArgs &a, int nv)
{
    const int lanes = a.group_size / nv;
    return a.groups == 1 || (a.group_size % nv == 0 && (lanes & (lanes - 1)) == 0);
}

template <typename T>
cudaError_t launch_route(const RouteArgs &a, bool sig, int sms, cudaStream_t s)
{
    // as few lanes per token as hold its picks, with eight experts each
    if (a.K <= 8 && a.E <= 64) {
        if (a.E <= 16 && runs_of_lanes(a, 2))
            return launch_route<T, 8, 2, false>(a, sig, sms, s);
        if (a.E <= 32 && runs_of_lanes(a, 4))
            return launch_route<T, 8, 4, false>(a, sig, sms, s);
        if (runs_of_lanes(a, 8))
            return launch_route<T, 8, 8, false>(a, sig, sms, s);
    }
    if (a.K <= 16 && a.E <= 128) {
        if (a.E <= 64 && runs_of_lanes(a, 4))
            return launch_route<T, 16, 4, false>(a, sig, sms, s);
        if (runs_of_lanes(a, 8))
            return launch_route<T, 16, 8, false>(a, sig, sms, s);
    }
    if (a.E <= 64 && runs_of_lanes(a, 2))
        return launch_route<T, 32, 2, false>(a, sig, sms, s);
    if (a.E <= 256 && runs_of_lanes(a, 8))
        return launch_route<T, 32, 8, false>(a, sig, sms, s);
    if (a.E <= 512 && runs_of_lanes(a, 16))
        return launch_route<T, 32, 16, false>(a, sig, sms, s);
    if (runs_of_lanes(a, 32))
        return launch_route<T, 32, 32, false>(a, sig, sms, s);
    if (a.E <= 256)
        return launch_route<T, 32, 8, true>(a, sig, sms, s);
    return launch_route<T, 32, 32, true>(a, sig, sms, s);
}

template <typename T, int NV>
cudaError_t launch_dense(const BackArgs &a, int sms, cudaStream_t s)
{
    static std::atomic<int> resident;
    return launch_warps(k_route_back_dense<T, NV>, resident, a.tokens, kWarps, 0, sms, s, a);
}

template <typename T>
cudaError_t launch_back(const BackArgs &a, bool sig, int sms, cudaStream_t s)
{
    if (sig || a.renorm) {
        int W = 1;
        while (W < a.K)
            W *= 2;
        static std::atomic<int> resident[2];
        const int64_t units = (a.tokens + 32 / W - 1) / (32 / W);
        return sig ? launch_warps(k_route_back_sparse<T, true>, resident[0], units, kWarps, 0, sms, s, a, W)
                   : launch_warps(k_route_back_sparse<T, false>, resident[1], units, kWarps, 0, sms, s, a, W);
    }
    const int nv = (a.E + 31) / 32;
    if (nv <= 1)
        return launch_dense<T, 1>(a, sms, s);
    if (nv <= 2)
        return launch_dense<T, 2>(a, sms, s);
    if (nv <= 4)
        return launch_dense<T, 4>(a, sms, s);
    if (nv <= 8)
        return launch_dense<T, 8>(a, sms, s);
    if (nv <= 16)
        return launch_dense<T, 16>(a, sms, s);
    return launch_dense<T, 32>(a, sms, s);
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
    a.bias_vec = !misaligned(bias, 16);
    const bool sig = cfg->score == SLIDE_SCORE_SIGMOID;
    e = size == 4 ? launch_route<float>(a, sig, sms, (cudaStream_t)stream)
                  : launch_route<uint16_t>(a, sig, sms, (cudaStream_t)stream);
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
    const bool sig = cfg->score == SLIDE_SCORE_SIGMOID;
    e = size == 4 ? launch_back<float>(a, sig, sms, (cudaStream_t)stream)
                  : launch_back<uint16_t>(a, sig, sms, (cudaStream_t)stream);
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
