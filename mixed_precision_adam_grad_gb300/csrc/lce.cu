// lce.cu — linear cross entropy (slide_linear_cross_entropy): the projection to
// a vocabulary, the loss, and the gradients of both factors.
//
// The softmax needs no pass of its own over the logits.  A token's reference is
// its target's logit, a dot product that is formed first: e_v = exp(z_v - z_y)
// can then be written as soon as z_v is known, BF16 having FP32's range.  With
// S = 1 + sum_{v != y} e_v,
//   loss = log S,   d_x = (d_loss/S) * (sum_{v != y} e_v w_v - (S - 1) w_y),
// and likewise for d_weight, so the factor that is known last, d_loss/S, belongs
// to whole rows: d_x takes it in its epilogue, d_weight from rows of x that are
// multiplied by it (T x H values instead of T x V; in two BF16 parts of few
// tokens).  The target's e is left
// out of the sum and its place then holds -(S - 1): no difference of nearly
// equal numbers is formed anywhere, however sure the model is.
// Where a logit lies more than 30 above the target's, so that e might leave
// BF16's useful range, the 256 rows' logits are formed once more with the
// largest logit as reference; so they are where the target's is -inf, its
// reference therefore 0, and the largest lies more than 30 below that.  This is
// decided on the device: the launches are always there and end at once where
// nothing is flagged.
//
// Three products, 2*T*H*V operations each, as many as the formulas have; the
// alternatives that need no T x V memory at all form the logits twice.  The e
// of a group of tokens are kept: 2 GiB of them at most, or those of 256 tokens
// where these are more (from 4.2 million words on).
#include <float.h>
#include <math.h>
#include <stdlib.h>

#include <algorithm>
#include <string>

#include "slide.h"
#include "slide_lce.h"
#include "slide_rows.h"
#include "slide_state.h"
#include "sm103_ptx.h"

namespace slide {
namespace {

constexpr int64_t kMaxTokens = 1 << 24, kMaxVocab = 1 << 24;
constexpr int kMaxHidden = 65536;
constexpr int64_t kMaxStride = (int64_t)1 << 36;
constexpr int64_t kGroupBytes = (int64_t)2 << 30;
constexpr int kMaxParts = 64;
constexpr int kJoinRows = 8;  // tokens of a block of k_join
// Up to so many tokens d_weight's factor x*d_loss/S is taken in two BF16 parts.
// Writing d_weight bounds its product there (a tile of 256 x 256 is written in 1.5
// us, four steps of 64 tokens take 1.4), so the second part costs little (16 tokens,
// 32000 x 1024: 74 us instead of 72); with one part the 2-norm of few tokens' errors
// was up to 1.57 times that of the result's own rounding, with many tokens it is 1.4
// times, with two parts 1.0 to 1.05 times.
constexpr int kTwoParts = 128;
constexpr unsigned kFull = 0xffffffffu;

struct Head {           // the start of a workspace
    unsigned status;    // first, for slide_linear_cross_entropy_status
    float one_over;     // 1/(tokens that are not padding)
    unsigned joined;    // blocks of a group's second k_join that are done
};

struct GroupArgs {      // a group of tokens
    int tokens, hidden, vocab;
    const bf16 *x, *weight;
    int64_t xs, ws;
    const int64_t *targets;
    const float *d_loss;  // or NULL: head->one_over
    float *loss, *lse;
    Head *head;
    int *target;
    float *ref, *own, *scale;  // reference, target's logit, d_loss/S
    unsigned *again;       // whether any rows are formed again, then which 256 are
    const float *sum, *top;
    int parts;             // of a row's sums: 128 columns each
    int64_t pitch;
    bf16 *e;               // or NULL
    int64_t e_stride;
    bf16 *scaled;          // rows of x times scale, or NULL
    bf16 *scaled_low;      // what is rounded off them, or NULL
};

// What the whole call's tokens add up to.
struct All {
    int64_t tokens;
    const int64_t *targets;
    const float *loss, *d_loss;
    float *total;  // or NULL
    int last;      // this group is the last one
};

// Sum over the block (256 threads), on its first thread; in a fixed order.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T (&part)[256])
{
    part[threadIdx.x] = v;
    __syncthreads();
#pragma unroll
    for (int o = 128; o >= 32; o >>= 1) {
        if (threadIdx.x < o)
            part[threadIdx.x] += part[threadIdx.x + o];
        __syncthreads();
    }
    v = part[threadIdx.x & 31];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// The targets' logits, a warp to a token.  count: block 0 also counts the call's
// tokens that are not padding.
__global__ void __launch_bounds__(256) k_targets(const GroupArgs g, const All all, int count, int clear)
{
    __shared__ int part[256];
    ptx::launch_dependents();
    ptx::wait_for_previous_grid();
    const int t = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) {
            if (clear)
                g.head->status = 0;
            g.head->joined = 0;
            g.again[0] = 0;
        }
        if (count) {
            int n = 0;
#pragma unroll 8
            for (int64_t i = threadIdx.x; i < all.tokens; i += 256)
                n += all.targets[i] >= 0;
            n = block_sum(n, part);
            if (threadIdx.x == 0)
                g.head->one_over = 1.0f / (float)(n > 0 ? n : 1);
        }
    }
    if (t >= g.tokens)
        return;
    if (t % kLceRows == 0 && lane == 0)
        g.again[1 + t / kLceRows] = 0;
    const int64_t y = g.targets[t];
    float z = y < 0 ? 0.0f : __int_as_float(0x7fffffff);
    if (y >= 0 && y < g.vocab) {
        const bf16 *x = g.x + t * g.xs, *w = g.weight + y * g.ws;
        float s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s[i] = 0.0f;
#pragma unroll 5
        for (int c = lane * 8; c < g.hidden; c += 256) {
            float a[8], b[8];
            unpack8(load_raw8(x + c), a);
            unpack8(load_raw8(w + c), b);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[i] = fmaf(a[i], b[i], s[i]);
        }
        z = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            z += __shfl_xor_sync(kFull, z, o);
    }
    if (lane == 0) {
        g.target[t] = y < 0 ? -1 : y < g.vocab ? (int)y : -2;
        g.own[t] = z;
        g.ref[t] = isfinite(z) ? z : 0.0f;
    }
}

// Each token's sums over the vocabulary, its loss, and what the gradients need:
// the target's place among the e, and the row's factor.
__device__ __forceinline__ void join_rows(const GroupArgs &g, int second)
{
    __shared__ float sums[32][kJoinRows], tops[32][kJoinRows];
    const int row0 = blockIdx.x * kJoinRows, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    {
        const int r = lane & 7, slot = warp * 4 + (lane >> 3);
        float s = 0.0f, m = -INFINITY;
        if (row0 + r < g.tokens) {
#pragma unroll 8
            for (int p = slot; p < g.parts; p += 32) {
                s += g.sum[p * g.pitch + row0 + r];
                m = fmaxf(m, g.top[p * g.pitch + row0 + r]);
            }
        }
        sums[slot][r] = s;
        tops[slot][r] = m;
    }
    __syncthreads();
    const int t = row0 + warp;
    if (t >= g.tokens)
        return;
    float others = sums[lane][warp], top = tops[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        others += __shfl_xor_sync(kFull, others, o);
        top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    }
    const int y = g.target[t];
    const float ref = g.ref[t], own = g.own[t];
    const float total = expf(own - ref) + others;
    float loss = 0.0f, scale = 0.0f;
    if (y != -1) {
        loss = ref == own ? log1pf(others) : (ref - own) + logf(total);
        scale = (g.d_loss ? g.d_loss[t] : g.head->one_over) / total;
        // -(S - 1) stands rounded in the target's place, the largest term of the
        // row (as large as all others together): the factor takes its rounding
        // out again, for 2^-8 at most on the others.
        const float kept = __bfloat162float(__float2bfloat16_rn(others));
        if (kept >= FLT_MIN && kept <= FLT_MAX)
            scale *= others / kept;
        if (isnan(loss))  // the gradients too (d_loss/total is 0 where the target's logit is infinite)
            scale = loss;
    }
    if (lane == 0) {
        // a logit far above the reference, or (where that is 0, the target's being -inf) all far below it
        const bool far = top - ref > kLceSpread || (own == -INFINITY && top < -kLceSpread && top > -INFINITY);
        if (!second && far && y != -1) {
            g.again[0] = 1;
            g.again[1 + t / kLceRows] = 1;
            g.ref[t] = top;
        }
        g.loss[t] = loss;
        // (own + loss would lose lse's digits where the target lies far below, and all of them where it is -inf)
        if (g.lse)
            g.lse[t] = y == -1 ? 0.0f : ref == own || own == INFINITY ? own + loss : ref + logf(total);
        g.scale[t] = scale;
        if (g.e && y >= 0)
            g.e[t * g.e_stride + y] = __float2bfloat16_rn(-others);
    }
    if (g.scaled) {
        const bf16 *x = g.x + t * g.xs;
        const int64_t at = (int64_t)t * g.hidden;
#pragma unroll 5
        for (int c = lane * 8; c < g.hidden; c += 256) {
            float v[8];
            unpack8(load_raw8(x + c), v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = scale == 0.0f ? 0.0f : v[i] * scale;
            const Raw8<bf16> kept = pack8<bf16>(v);
            store_raw8(g.scaled + at + c, kept);
            if (g.scaled_low) {
                float k[8];
                unpack8(kept, k);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] -= k[i];
                store_raw8(g.scaled_low + at + c, pack8<bf16>(v));
            }
        }
    }
}

// second: only the rows whose logits were formed again; behind the last group's,
// total = sum of d_loss*loss, in 64 bits, by the block that is done last.
__global__ void __launch_bounds__(256) k_join(const GroupArgs g, const All all, int second)
{
    __shared__ double part[256];
    __shared__ unsigned before;
    ptx::launch_dependents();
    ptx::wait_for_previous_grid();
    if (!second || (g.again[0] && g.again[1 + blockIdx.x * kJoinRows / kLceRows]))
        join_rows(g, second);
    if (!second || !all.last || !all.total)
        return;
    __syncthreads();
    if (threadIdx.x == 0)
        before = ptx::add_acq_rel(&g.head->joined, 1u);
    __syncthreads();
    if (before + 1 != gridDim.x)
        return;
    __threadfence();
    double s = 0.0;
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < all.tokens; t += 256) {
        const float l = __ldcg(all.loss + t), d = all.d_loss ? all.d_loss[t] : g.head->one_over;
        s += all.targets[t] >= 0 ? (double)d * l : 0.0;
    }
    s = block_sum(s, part);
    if (threadIdx.x == 0)
        *all.total = (float)s;
}

// d_x from the parts of its sums, part after part.
__global__ void __launch_bounds__(256) k_join_d_x(int tokens, int hidden, int parts, const float *part, const float *scale,
                                                  bf16 *d_x, int64_t stride)
{
    ptx::launch_dependents();
    ptx::wait_for_previous_grid();
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4, n = (int64_t)tokens * hidden;
    if (i >= n)
        return;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int p = 0; p < parts; ++p) {
        const float4 w = __ldcs(reinterpret_cast<const float4 *>(part + p * n + i));
        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
    const int64_t t = i / hidden;
    const float s = scale[t];
    if (s == 0.0f)
        v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * s, v.y * s), b = __floats2bfloat162_rn(v.z * s, v.w * s);
    *reinterpret_cast<uint2 *>(d_x + t * stride + (i - t * hidden)) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// FP32 sums over the groups to BF16.
__global__ void __launch_bounds__(256) k_round(int64_t rows, int hidden, const float *in, bf16 *out, int64_t stride)
{
    ptx::launch_dependents();
    ptx::wait_for_previous_grid();
    const int64_t n = rows * hidden;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 256 * 8) {
        float v[8];
        unpack8(load_raw8(in + i), v);
        const int64_t r = i / hidden;
        store_raw8(out + r * stride + (i - r * hidden), pack8<bf16>(v));
    }
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), int64_t blocks, int threads, cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

// Sizes and places within a workspace.
struct Work {
    int64_t bytes;
    int groups, group;    // of tokens: how many, tokens of each (the last one may have fewer)
    int sum_parts;
    int64_t pitch, e_stride;
    int dx_parts;         // most parts of d_x's sums
    Head *head;
    int *target;
    float *ref, *own, *scale, *sum, *top, *part, *acc;
    unsigned *again;
    bf16 *e, *scaled, *scaled_low;
};

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Parts of K for d_x's tiles, each `steps` long: as many as make the rounds of
// the tiles come out best.  A tile costs about 8 steps besides its products, a
// part's sums are written and read (FP32) at the memory's rate: a step takes 0.34
// us, 0.38 under the power limit, in which the memory moves some 2.6 MB.
int parts_of_d_x(int tokens, int hidden, int64_t vocab, int groups)
{
    const int64_t rows = lce_single(tokens) ? 128 : 256;
    const int64_t tiles = ((tokens + rows - 1) / rows) * ((hidden + kLceCols - 1) / kLceCols), steps = (vocab + 63) / 64;
    int best = 1;
    double least = 0.0;
    for (int p = 1; p <= kMaxParts && (p == 1 || steps / p >= 16); ++p) {
        const int64_t rounds = (tiles * p + groups - 1) / groups;
        double cost = (double)rounds * ((steps + p - 1) / p + 8);
        if (p > 1)
            cost += 10.0 + (double)p * tokens * hidden * 8.0 / 2.6e6;
        if (p == 1 || cost < least) {
            best = p;
            least = cost;
        }
    }
    return best;
}

Work layout(int64_t tokens, int hidden, int64_t vocab, bool d_x, bool d_weight, char *base)
{
    Work w{};
    const bool keep = d_x || d_weight;
    w.sum_parts = (int)((vocab + 127) / 128);
    w.e_stride = up(vocab, 64);
    const int64_t each = (keep ? 2 * w.e_stride : 0) + (int64_t)w.sum_parts * 8;
    const int64_t most = std::max<int64_t>(kLceRows, kGroupBytes / each / kLceRows * kLceRows);
    w.groups = (int)((tokens + most - 1) / most);
    w.group = (int)std::min<int64_t>(tokens, up((tokens + w.groups - 1) / w.groups, kLceRows));
    w.pitch = up(w.group, 32);
    int64_t at = 0;
    auto take = [&](int64_t n) {
        char *p = base ? base + at : nullptr;
        at += up(n, 256);
        return p;
    };
    w.head = (Head *)take(sizeof(Head));
    w.target = (int *)take(4 * w.pitch);
    w.ref = (float *)take(4 * w.pitch);
    w.own = (float *)take(4 * w.pitch);
    w.scale = (float *)take(4 * w.pitch);
    w.again = (unsigned *)take(4 * (1 + (w.group + kLceRows - 1) / kLceRows));
    w.sum = (float *)take(4 * w.pitch * w.sum_parts);
    w.top = (float *)take(4 * w.pitch * w.sum_parts);
    if (keep)
        w.e = (bf16 *)take(2 * w.e_stride * w.group);
    if (d_weight) {
        w.scaled = (bf16 *)take((int64_t)2 * w.group * hidden);
        if (w.group <= kTwoParts)
            w.scaled_low = (bf16 *)take((int64_t)2 * w.group * hidden);
    }
    if (d_x) {
        // for as many groups of CTAs as there may be on a device like this one
        w.dx_parts = parts_of_d_x(w.group, hidden, vocab, lce_single(w.group) ? 152 : 76);
        if (w.dx_parts > 1)
            w.part = (float *)take((int64_t)4 * w.dx_parts * w.group * hidden);
    }
    if (d_weight && w.groups > 1)
        w.acc = (float *)take((int64_t)4 * vocab * hidden);
    w.bytes = at;
    return w;
}

struct Call {
    int64_t tokens;
    int hidden, vocab;
    const bf16 *x, *weight;
    int64_t xs, ws;
    const int64_t *targets;
    const float *d_loss;
    float *loss, *lse, *total;
    bf16 *d_x, *d_weight;
    int64_t dxs, dws;
};

cudaError_t enqueue_group(const Call &c, const Work &w, int64_t t0, int n, int device, bool stall, cudaStream_t s)
{
    const bool first = t0 == 0, last = t0 + n == c.tokens;
    GroupArgs g{};
    g.tokens = n;
    g.hidden = c.hidden;
    g.vocab = c.vocab;
    g.x = c.x + t0 * c.xs;
    g.xs = c.xs;
    g.weight = c.weight;
    g.ws = c.ws;
    g.targets = c.targets + t0;
    g.d_loss = c.d_loss ? c.d_loss + t0 : nullptr;
    g.loss = c.loss + t0;
    g.lse = c.lse ? c.lse + t0 : nullptr;
    g.head = w.head;
    g.target = w.target;
    g.ref = w.ref, g.own = w.own, g.scale = w.scale;
    g.again = w.again;
    g.sum = w.sum, g.top = w.top;
    g.parts = w.sum_parts;
    g.pitch = w.pitch;
    g.e = w.e;
    g.e_stride = w.e_stride;
    g.scaled = w.scaled;
    g.scaled_low = w.scaled_low;
    const All all{c.tokens, c.targets, c.loss, c.d_loss, c.total, last};

    // the products first: nothing is enqueued if one cannot be described
    LceProduct logits{};
    logits.kind = kLceLogits;
    logits.rows = n;
    logits.cols = c.vocab;
    logits.k64 = (c.hidden + 63) / 64;
    logits.parts = 1;
    logits.ref = w.ref;
    logits.target = w.target;
    logits.sum = w.sum;
    logits.top = w.top;
    logits.pitch = w.pitch;
    logits.keep = w.e != nullptr;
    logits.status = &w.head->status;
    logits.test_stall = stall;
    cudaError_t e = lce_map(&logits.a, g.x, false, n, c.hidden, c.xs, 128);
    if (e == cudaSuccess)
        e = lce_map(&logits.b, c.weight, false, c.vocab, c.hidden, c.ws, 128);
    if (e == cudaSuccess && logits.keep)
        e = lce_map(&logits.out, w.e, false, n, c.vocab, w.e_stride, 32);

    LceProduct dx{};
    bf16 *dx_out = c.d_x + (c.d_x ? t0 * c.dxs : 0);
    if (c.d_x && e == cudaSuccess) {
        int groups = 0;
        e = lce_groups(n, device, &groups);
        dx.rows = n;
        dx.cols = c.hidden;
        dx.k64 = (c.vocab + 63) / 64;
        dx.b_mn = 1;
        dx.n_fast = 1;
        dx.scale = w.scale;
        dx.status = &w.head->status;
        dx.parts = e == cudaSuccess ? std::min(w.dx_parts, parts_of_d_x(n, c.hidden, c.vocab, groups)) : 1;
        dx.kind = dx.parts > 1 ? kLcePart : kLceScaled;
        if (e == cudaSuccess)
            e = lce_map(&dx.a, w.e, false, n, c.vocab, w.e_stride, 128);
        if (e == cudaSuccess)
            e = lce_map(&dx.b, c.weight, false, c.vocab, c.hidden, c.ws, 64);
        if (e == cudaSuccess)
            e = dx.parts > 1
                    ? lce_map(&dx.out, w.part, true, n, c.hidden, c.hidden, 32, dx.parts, (int64_t)n * c.hidden)
                    : lce_map(&dx.out, dx_out, false, n, c.hidden, c.dxs, 32);
    }

    LceProduct dw{};
    if (c.d_weight && e == cudaSuccess) {
        int groups = 0;
        e = lce_groups(c.vocab, device, &groups);
        dw.rows = c.vocab;
        dw.cols = c.hidden;
        dw.k64 = (n + 63) / 64;
        dw.a_mn = dw.b_mn = 1;
        dw.n_fast = 1;
        dw.parts = 1;
        dw.status = &w.head->status;
        dw.kind = !w.acc ? kLcePlain : first ? kLcePart : kLceAdd;
        if (e == cudaSuccess)
            e = lce_map(&dw.a, w.e, false, n, c.vocab, w.e_stride, 64);
        if (e == cudaSuccess)
            e = lce_map(&dw.b, w.scaled, false, n, c.hidden, c.hidden, 64);
        if (e == cudaSuccess && w.scaled_low) {
            dw.wrap = dw.k64;
            dw.k64 *= 2;
            e = lce_map(&dw.b_low, w.scaled_low, false, n, c.hidden, c.hidden, 64);
        }
        if (e == cudaSuccess)
            e = w.acc ? lce_map(&dw.out, w.acc, true, c.vocab, c.hidden, c.hidden, 32)
                      : lce_map(&dw.out, c.d_weight, false, c.vocab, c.hidden, c.dws, 32);
    }

    const int64_t join_blocks = (n + kJoinRows - 1) / kJoinRows;
    if (e == cudaSuccess)
        e = launch(k_targets, (n + 7) / 8, 256, s, g, all, first && !c.d_loss, first);
    if (e == cudaSuccess)
        e = launch_lce_product(logits, device, s);
    if (e == cudaSuccess)
        e = launch(k_join, join_blocks, 256, s, g, all, 0);
    logits.again = w.again;
    if (e == cudaSuccess)
        e = launch_lce_product(logits, device, s);
    if (e == cudaSuccess)
        e = launch(k_join, join_blocks, 256, s, g, all, 1);
    if (c.d_x) {
        if (e == cudaSuccess)
            e = launch_lce_product(dx, device, s);
        if (e == cudaSuccess && dx.parts > 1)
            e = launch(k_join_d_x, ((int64_t)n * c.hidden / 4 + 255) / 256, 256, s, n, c.hidden, dx.parts, w.part, w.scale, dx_out,
                       c.dxs);
    }
    if (c.d_weight) {
        if (e == cudaSuccess)
            e = launch_lce_product(dw, device, s);
        if (e == cudaSuccess && w.acc && last)
            e = launch(k_round, std::min<int64_t>(((int64_t)c.vocab * c.hidden / 8 + 255) / 256, 65536), 256, s,
                       (int64_t)c.vocab, c.hidden, w.acc, c.d_weight, c.dws);
    }
    return e;
}

cudaError_t enqueue(const Call &c, const Work &w, int device, bool stall, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    for (int64_t t = 0; t < c.tokens && e == cudaSuccess; t += w.group)
        e = enqueue_group(c, w, t, (int)std::min<int64_t>(w.group, c.tokens - t), device, stall, s);
    return e;
}

slide_status check_sizes(int64_t tokens, int32_t hidden, int32_t vocab)
{
    if (tokens < 0 || tokens > kMaxTokens)
        return fail(SLIDE_ERR_INVALID_ARG, "tokens must lie in [0, 2^24]");
    if (hidden < 8 || hidden > kMaxHidden || hidden % 8 != 0)
        return fail(SLIDE_ERR_INVALID_ARG, "hidden must be a multiple of 8 in [8, 65536]");
    if (vocab < 1 || vocab > kMaxVocab)
        return fail(SLIDE_ERR_INVALID_ARG, "vocab must lie in [1, 2^24]");
    return SLIDE_OK;
}

}  // namespace
}  // namespace slide

using namespace slide;

extern "C" slide_status slide_linear_cross_entropy_workspace(int64_t tokens, int32_t hidden, int32_t vocab, int32_t d_x,
                                                             int32_t d_weight, int64_t *bytes)
{
    const slide_status rc = check_sizes(tokens, hidden, vocab);
    if (rc != SLIDE_OK)
        return rc;
    if (!bytes)
        return fail(SLIDE_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = tokens == 0 ? 256 : layout(tokens, hidden, vocab, d_x != 0, d_weight != 0, nullptr).bytes;
    clear_error();
    return SLIDE_OK;
}

extern "C" slide_status slide_linear_cross_entropy(int64_t tokens, int32_t hidden, int32_t vocab, const void *x,
                                                   int64_t x_stride, const void *weight, int64_t weight_stride,
                                                   const int64_t *targets, const float *d_loss, float *loss, float *lse,
                                                   float *total, void *d_x, int64_t d_x_stride, void *d_weight,
                                                   int64_t d_weight_stride, void *workspace, int64_t workspace_bytes,
                                                   slide_stream_t stream)
{
    slide_status rc = check_sizes(tokens, hidden, vocab);
    if (rc != SLIDE_OK)
        return rc;
    struct Matrix {
        const char *name;
        const void *p;
        int64_t stride;
        bool needed;
    };
    for (const Matrix &m : {Matrix{"x", x, x_stride, tokens > 0}, Matrix{"weight", weight, weight_stride, tokens > 0},
                            Matrix{"d_x", d_x, d_x_stride, false}, Matrix{"d_weight", d_weight, d_weight_stride, false}}) {
        if (m.needed && !m.p)
            return fail(SLIDE_ERR_INVALID_ARG, std::string(m.name) + " is NULL");
        if (!m.p)
            continue;
        if (misaligned(m.p, 16))
            return fail(SLIDE_ERR_INVALID_ARG, std::string(m.name) + " is not 16-byte aligned");
        if (m.stride < hidden || m.stride % 8 != 0 || m.stride >= kMaxStride)
            return fail(SLIDE_ERR_INVALID_ARG,
                        std::string(m.name) + ": the row stride must be a multiple of 8, at least hidden and below 2^36");
    }
    const cudaStream_t s = (cudaStream_t)stream;
    if (!workspace || misaligned(workspace, 256))
        return fail(SLIDE_ERR_INVALID_ARG, "workspace is NULL or not 256-byte aligned");
    if (tokens == 0) {  // nothing to sum: the gradient of the weight is 0
        if (workspace_bytes < 256)
            return fail(SLIDE_ERR_INVALID_ARG, "workspace is smaller than slide_linear_cross_entropy_workspace says");
        if (misaligned(total, 4))
            return fail(SLIDE_ERR_INVALID_ARG, "total is not aligned to its type");
        cudaError_t e = cudaMemsetAsync(workspace, 0, sizeof(Head), s);
        if (e == cudaSuccess && d_weight)
            e = cudaMemset2DAsync(d_weight, (size_t)d_weight_stride * 2, 0, (size_t)hidden * 2, vocab, s);
        if (e == cudaSuccess && total)
            e = cudaMemsetAsync(total, 0, sizeof(float), s);
        if (e != cudaSuccess)
            return fail_cuda(e, "clearing the results of no tokens");
        clear_error();
        return SLIDE_OK;
    }
    if (!targets || misaligned(targets, 8) || !loss || misaligned(loss, 4))
        return fail(SLIDE_ERR_INVALID_ARG, "targets or loss is NULL or not aligned to its type");
    if (misaligned(d_loss, 4) || misaligned(lse, 4) || misaligned(total, 4))
        return fail(SLIDE_ERR_INVALID_ARG, "d_loss, lse or total is not aligned to its type");
    if ((d_x && (d_x == x || d_x == weight)) || (d_weight && (d_weight == x || d_weight == weight || d_weight == d_x)))
        return fail(SLIDE_ERR_INVALID_ARG, "d_x and d_weight must not be x, weight or each other");
    const Work w = layout(tokens, hidden, vocab, d_x, d_weight, (char *)workspace);
    if (workspace_bytes < w.bytes)
        return fail(SLIDE_ERR_INVALID_ARG, "workspace is smaller than slide_linear_cross_entropy_workspace says");
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess)
        return fail_cuda(e, "cudaGetDevice");
    const Call c{tokens, hidden, vocab, (const bf16 *)x, (const bf16 *)weight, x_stride, weight_stride, targets, d_loss,
                 loss,   lse,    total, (bf16 *)d_x,     (bf16 *)d_weight,     d_x_stride, d_weight_stride};
    const char *v = getenv("SLIDE_TEST_PIPELINE_STALL");
    e = enqueue(c, w, device, v && v[0] && v[0] != '0', s);
    if (e != cudaSuccess)
        return fail_cuda(e, "linear cross entropy launch");
    clear_error();
    return SLIDE_OK;
}

extern "C" slide_status slide_linear_cross_entropy_status(const void *workspace, slide_stream_t stream)
{
    if (!workspace || misaligned(workspace, 256))
        return fail(SLIDE_ERR_INVALID_ARG, "workspace is NULL or not 256-byte aligned");
    unsigned word = 0;
    cudaError_t e = cudaMemcpyAsync(&word, workspace, sizeof word, cudaMemcpyDeviceToHost, (cudaStream_t)stream);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess)
        return fail_cuda(e, "reading the workspace's status word");
    if (word & 2u)
        return fail(SLIDE_ERR_TIMEOUT, "a pipeline wait inside a product reached its limit; that call is incomplete");
    clear_error();
    return SLIDE_OK;
}
