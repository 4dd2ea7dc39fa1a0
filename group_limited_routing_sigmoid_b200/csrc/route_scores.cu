// Routing from given logits under either score function (beam_route_scores).
//
// A warp per token.  With groups in play every group gets L lanes (a power of
// two, L * n_group <= 32), else one group of 32; a lane owns `epl` consecutive
// experts of its group, in registers.  The choice is made among candidates: the
// experts whose key reaches the n-th largest of the lanes' best keys (n the
// experts wanted) hold the n largest and are few (about 13 of 256 for n = 9).
// They are packed, one to a lane, and ranked by counting the larger ones.
// 32768 x 256, 8 groups of which 4 stay, bias, top 8: 33 to 35 us (1.0 TB/s); without
// groups and bias 20 us.  Lists sorted in the lanes with one maximum over their
// heads per expert wanted took 49 and 26 us.
//
// Decisions are those of 64-bit arithmetic: an FP32 score is off by a few
// ulps, so a row in which two keys (neighbours of the chosen ranking) or two
// group scores (last kept, first dropped) are closer than that error, and not
// exactly equal, is decided again from 64-bit scores (decide_row, the same
// warp).  Without a bias the keys are the logits themselves, which are exact.
//
// A lane owns up to 60 experts where n_group is no power of two (route_layout.h).
// 4096 x 720, 10 groups of which 4 stay: 17 us, 50 with a bias (sigmoid; 23 and
// 58 at one block an SM and twice the registers, which only 60 experts a lane
// gain from: 4096 x 1020, 17 groups, bias 77 and 66 us).
//
// Bound by instruction issue at large T, by the latency of a row's chain of
// warp-wide steps at small T.
#include "ops_common.cuh"
#include "route_layout.h"

namespace beam {
namespace {

using namespace ops;

constexpr int kRouteWarps = 8;

struct RouteArgs {
    const float *logits, *bias;
    int32_t *idx;
    float *w;
    long long ldl;
    int T, E;
    int lanes_log, size, epl;   // RouteLayout
    int keep;       // groups that stay, 0: all
    int group_top, top_k, renorm;
    int vec;        // rows and lanes start on 16-byte boundaries
    float scale;
};

__device__ __forceinline__ float redux_max(float v)
{
    float r;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

__device__ __forceinline__ Span span_of(const RouteArgs &p, int lane)
{
    return Span(lane, p.lanes_log, p.size, p.epl, p.E);
}

constexpr float kLog2e = 1.4426950408889634f;

// The approximations below flush subnormals (3 instructions less each): what
// they are used for is compared with margins far above 2^-126.

__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_fast(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Sigmoid to about 2^-22 absolute: enough to rank by, with the margins below.
__device__ __forceinline__ float sigmoid_fast(float x) { return rcp_fast(1.0f + exp2_fast(x * -kLog2e)); }

// exp(x - y) to some 3 ulps: the difference's rounding, which alone would cost
// |x - y| half ulps (64 for scores next to 2^-92), is put back as a factor.
__device__ __forceinline__ float exp_of_difference(float x, float y)
{
    const float d = x - y, z = d - x, lost = (x - (d - z)) - (y + z);
    const float e = expf(d);
    return e > 0.f ? fmaf(e, lost, e) : 0.f;   // d = -inf has no such factor
}

// From e^-|x|, which does not overflow: scores down to the least subnormal.
__device__ __forceinline__ float sigmoid(float x)
{
    const float e = expf(-fabsf(x));
    return (x < 0.f ? e : 1.0f) / (1.0f + e);
}

// --- a row in 64 bits ------------------------------------------------------------

// Slow and rare.  Writes the row's outputs; every tie that is left is one of
// equal keys.
template <int EPL, bool SOFTMAX, bool BIAS>
__device__ __noinline__ void decide_row(const RouteArgs &p, long long row)
{
    const int lane = threadIdx.x & 31;
    const Span my = span_of(p, lane);
    const float *l = p.logits + row * p.ldl;
    const int lanes = 1 << p.lanes_log;
    double top = -INFINITY, sum = 1.0;
    double key[EPL];
    if (SOFTMAX) {
#pragma unroll 1
        for (int i = 0; i < my.mine; ++i) top = fmax(top, (double)l[my.e0 + i]);
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, d));
        sum = 0.0;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const double x = i < my.mine ? (double)l[my.e0 + i] : -INFINITY;
        key[i] = SOFTMAX ? exp(x - top) : 1.0 / (1.0 + exp(-x));
        if (SOFTMAX) sum += key[i];
    }
    if (SOFTMAX) sum = warp_sum(sum);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const bool in = i < my.mine && l[my.e0 + i] > -INFINITY;
        const double b = BIAS && in ? (double)p.bias[my.e0 + i] : 0.0;
        key[i] = in ? (SOFTMAX ? key[i] / sum : key[i]) + b : -INFINITY;
    }
    bool kept = true;
    if (p.keep) {
        double a = -INFINITY, b = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) b = fmax(b, fmin(a, key[i])), a = fmax(a, key[i]);
        for (int d = 1; d < lanes; d <<= 1) {
            const double oa = __shfl_xor_sync(0xffffffffu, a, d), ob = __shfl_xor_sync(0xffffffffu, b, d);
            b = fmax(fmin(a, oa), fmax(b, ob));
            a = fmax(a, oa);
        }
        const double score = p.group_top == 2 && b > -INFINITY ? a + b : a;
        int rank = 0;
        for (int g = 0; g < 32; g += lanes) {
            const double o = __shfl_sync(0xffffffffu, score, g);
            rank += o > score || (o == score && g < (lane & -lanes));
        }
        kept = rank < p.keep;
    }
    // Keys as integers that order as they do, 0: not eligible; a round's
    // largest is found in two halves and the lowest index in a third step.
    // Without a bias the logits order the scores, also where those saturate.
    unsigned long long ord[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        ord[i] = 0;
        if (kept && key[i] > -INFINITY) {
            const long long v = __double_as_longlong(BIAS ? key[i] + 0.0 : (double)l[my.e0 + i] + 0.0);   // -0 as 0
            ord[i] = (unsigned long long)(v < 0 ? ~v : v ^ (1ll << 63));
        }
    }
    int my_idx = -1;
    for (int j = 0; j < p.top_k; ++j) {
        unsigned long long m = 0;
        int at = p.E;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (ord[i] > m) m = ord[i], at = my.e0 + i;
        const uint32_t hi = (uint32_t)(m >> 32), best = __reduce_max_sync(0xffffffffu, hi);
        if (best == 0u) break;
        const uint32_t lo = __reduce_max_sync(0xffffffffu, hi == best ? (uint32_t)m : 0u);
        at = (int)__reduce_min_sync(0xffffffffu, hi == best && (uint32_t)m == lo ? (uint32_t)at : 0x7fffffffu);
        if (lane == j) my_idx = at;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (my.e0 + i == at) ord[i] = 0;
    }
    const double x = my_idx >= 0 ? (double)l[my_idx] : 0.0;
    double w = my_idx < 0 ? 0.0 : SOFTMAX ? exp(x - top) / sum : 1.0 / (1.0 + exp(-x));
    if (p.renorm) {
        double s = warp_sum(w);
        if (s < 1e-200) {   // scores that underflow still share: from their logarithms
            const double log_w = my_idx < 0 ? -INFINITY : SOFTMAX ? x - top : x < 0 ? x - log1p(exp(x)) : -log1p(exp(-x));
            double most = log_w;
#pragma unroll
            for (int d = 16; d; d >>= 1) most = fmax(most, __shfl_xor_sync(0xffffffffu, most, d));
            w = my_idx >= 0 ? exp(log_w - most) : 0.0;
            s = warp_sum(w);
        }
        w = s > 0.0 ? w / s : 0.0;
    }
    if (lane < p.top_k) {
        p.idx[row * p.top_k + lane] = my_idx;
        p.w[row * p.top_k + lane] = (float)(w * (double)p.scale);
    }
}

// ---------------------------------------------------------------------------------

template <int EPL, bool SOFTMAX, bool BIAS>
__global__ void __launch_bounds__(32 * kRouteWarps, EPL <= 8 ? 4 : 2) route_scores_kernel(const RouteArgs p)
{
    __shared__ __align__(16) float s_key[kRouteWarps][36];   // candidates' keys, then the chosen order's
    __shared__ int s_expert[kRouteWarps][32];
    __shared__ float2 s_tie[kRouteWarps][BIAS ? 32 : 1];      // logit and bias in the chosen order
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t below = (1u << lane) - 1u;
    const Span my = span_of(p, lane);
    float *cand = s_key[warp];
    int *expert = s_expert[warp];
    // with a bias one more than top_k: the best that is not chosen (33 have no
    // lane each: top_k 32 looks for that one by itself, 4096 x 256: 17 us, 43
    // with every such row decided in 64 bits)
    const int want = BIAS && p.top_k < 32 ? p.top_k + 1 : p.top_k;
    float bias[BIAS ? EPL : 1];
    bool nan_bias = false;
    if constexpr (BIAS) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            bias[i] = i < my.mine ? p.bias[my.e0 + i] : 0.f;
            nan_bias |= bias[i] != bias[i];
        }
        nan_bias = __any_sync(0xffffffffu, nan_bias);
    }
    for (long long row = (long long)blockIdx.x * kRouteWarps + warp; row < p.T;
         row += (long long)gridDim.x * kRouteWarps) {
        const float *l = p.logits + row * p.ldl;
        float key[EPL];   // logits, then keys
        if (EPL % 4 == 0 && p.vec) {
#pragma unroll
            for (int i = 0; i < EPL; i += 4) {
                const float4 v = i < my.mine ? *reinterpret_cast<const float4 *>(l + my.e0 + i)
                                             : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                key[i] = v.x;
                if constexpr (EPL >= 4) key[i + 1] = v.y, key[i + 2] = v.z, key[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = i < my.mine ? l[my.e0 + i] : -INFINITY;
        }
        float top = key[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) top = max_nan(top, key[i]);
        float head = top;
        top = redux_max(top);
        if (top != top || (SOFTMAX && top == INFINITY) || nan_bias) {
            if (lane < p.top_k) {
                p.idx[row * p.top_k + lane] = -1;
                p.w[row * p.top_k + lane] = __uint_as_float(0x7fffffffu);
            }
            continue;
        }
        // softmax: the sum, where keys or weights need it.  (Weights divided by
        // a sum of expf are no better: 60 to 1024 experts 5.5e-8 to 1.1e-7 of
        // their norm, 5.6e-8 to 1.1e-7 so, at 5% more time; 2.5e-8 is the
        // rounding of the result alone.)
        float sum = 1.f;
        const float ref = top > -INFINITY ? top : 0.f;
        if constexpr (SOFTMAX && !BIAS) {
            if (!p.renorm) {
                sum = 0.f;
#pragma unroll
                for (int i = 0; i < EPL; ++i) sum += exp2_fast((key[i] - ref) * kLog2e);
                sum = warp_sum(sum);
            }
        }
        if constexpr (BIAS) {
            float inv = 1.f;
            if constexpr (SOFTMAX) {
                sum = 0.f;
#pragma unroll
                for (int i = 0; i < EPL; ++i) sum += exp2_fast((key[i] - ref) * kLog2e);
                sum = warp_sum(sum);
                inv = rcp_fast(sum);
            }
            head = -INFINITY;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const float s = SOFTMAX ? exp2_fast((key[i] - ref) * kLog2e) * inv : sigmoid_fast(key[i]);
                key[i] = key[i] > -INFINITY ? s + bias[i] : -INFINITY;
                head = fmaxf(head, key[i]);
            }
        }
        // How far two FP32 keys may be off together.  Sigmoid: 2^-22 each
        // (s(1-s) times the exponential's 2^-22 and its argument's rounding,
        // half an ulp of the sum, an ulp of the reciprocal).  Softmax, in
        // units of 2^-24 / sum (the largest score is 1 / sum): the keys' own
        // exponentials 4 and 1 for its argument, and what both share, the
        // sum's partial sums EPL + 4 (EPL - 1 in the lane, 5 across), its
        // exponentials 4, their arguments 10 (3 roundings of the weighted mean
        // distance from the top, at most 3.4 for 1024 experts), its reciprocal
        // 2 and a product 1, all times the scores' difference: up to 30 for
        // 8 experts a lane, 54 for 32, 86 for 64.  And the rounding of the
        // added bias.
        constexpr float kSoftmaxTol = EPL <= 8 ? 0x1p-19f : EPL <= 32 ? 0x1p-18f : 0x1p-17f;
        const float tol_score = SOFTMAX ? kSoftmaxTol * rcp_fast(sum) : 0x1p-20f;
        bool close = false;
        if (p.keep) {
            float a = key[0], b = -INFINITY;
#pragma unroll
            for (int i = 1; i < EPL; ++i) b = fmaxf(b, fminf(a, key[i])), a = fmaxf(a, key[i]);
            for (int d = 1; d < 1 << p.lanes_log; d <<= 1) {
                const float oa = __shfl_xor_sync(0xffffffffu, a, d), ob = __shfl_xor_sync(0xffffffffu, b, d);
                b = fmaxf(fminf(a, oa), fmaxf(b, ob));
                a = fmaxf(a, oa);
            }
            float pa = a, pb = b;
            if constexpr (!BIAS) {   // softmax: up to the common factor
                pa = a > -INFINITY ? (SOFTMAX ? exp2_fast((a - top) * kLog2e) : sigmoid_fast(a)) : -INFINITY;
                pb = b > -INFINITY ? (SOFTMAX ? exp2_fast((b - top) * kLog2e) : sigmoid_fast(b)) : -INFINITY;
            }
            const float score = p.group_top == 2 && pb > -INFINITY ? pa + pb : pa;
            float left = score, lo = -INFINITY;
            for (int i = 0; i < p.keep; ++i) {
                lo = redux_max(left);
                const int first = __ffs(__ballot_sync(0xffffffffu, left == lo)) - 1;   // a group's first lane
                if (lane >> p.lanes_log == first >> p.lanes_log) left = -INFINITY;
            }
            const float hi = redux_max(left);   // the best that is dropped
            const float tol = (BIAS ? 2.f * tol_score : 0x1p-19f) + 0x1p-21f * (fabsf(lo) + fabsf(hi));
            if (hi > -INFINITY && !(lo - hi > tol)) {
                close = true;
                if constexpr (!BIAS) {
                    // groups that tie with the last kept by equal logits are
                    // decided by their indexes; nothing else may be near
                    const int at = __ffs(__ballot_sync(0xffffffffu, score == lo)) - 1;
                    const float ta = __shfl_sync(0xffffffffu, a, at), tb = __shfl_sync(0xffffffffu, b, at);
                    const bool near = score > -INFINITY && fabsf(score - lo) <= tol;
                    close = __any_sync(0xffffffffu, near && !(a == ta && (b == tb || p.group_top == 1)));
                }
            }
            if (left > -INFINITY) {   // dropped
                head = -INFINITY;
#pragma unroll
                for (int i = 0; i < EPL; ++i) key[i] = -INFINITY;
            }
        }
        // candidates: keys of the want-th largest head and more (equal heads
        // leave together, which only lowers the bound); -inf is none
        float bound = -INFINITY;
        for (int i = 0; i < want; ++i) {
            bound = redux_max(head);
            if (head == bound) head = -INFINITY;
        }
        bound = fmaxf(bound, -3.402823466e38f);
        uint32_t has[EPL];
        int n = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            has[i] = __ballot_sync(0xffffffffu, key[i] >= bound);
            n += __popc(has[i]);
        }
        if (n > 32) {
            // halve the gap up to the largest key, as integers of the floats'
            // order, until at least `want` and at most 32 are left
            const auto ordered = [](float v) {
                const int b = __float_as_int(v);
                return b < 0 ? b ^ 0x7fffffff : b;
            };
            float most = key[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) most = fmaxf(most, key[i]);
            int low = ordered(bound), high = ordered(redux_max(most)) + 1;
            for (int it = 0; it < 24 && n > 32; ++it) {
                const int mid = low + (int)(((uint32_t)high - (uint32_t)low) >> 1);
                const float v = __int_as_float(mid < 0 ? mid ^ 0x7fffffff : mid);
                int m = 0;
#pragma unroll
                for (int i = 0; i < EPL; ++i) m += __popc(__ballot_sync(0xffffffffu, key[i] >= v));
                if (m < want) high = mid;
                else low = mid, bound = v, n = m;
            }
#pragma unroll
            for (int i = 0; i < EPL; ++i) has[i] = __ballot_sync(0xffffffffu, key[i] >= bound);
        }
        if (close || n > 32) {
            decide_row<EPL, SOFTMAX, BIAS>(p, row);
            continue;
        }
        __syncwarp();   // the last row's reads of cand
        int base = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (has[i]) {
                if ((has[i] >> lane) & 1u) {
                    const int at = base + __popc(has[i] & below);
                    cand[at] = key[i];
                    expert[at] = my.e0 + i;
                }
                base += __popc(has[i]);
            }
        }
        if (lane < 4) cand[n + lane] = -INFINITY;   // whole fours below
        __syncwarp();
        const bool in = lane < n;
        const float mine = cand[in ? lane : 0];
        const int e = in ? expert[lane] : 0;
        const float xe = in ? l[e] : -INFINITY;
        int rank = 0;
        for (int m = 0; m < n; m += 4) {
            const float4 o = *reinterpret_cast<const float4 *>(cand + m);
            rank += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
        }
        if (__popc(__reduce_or_sync(0xffffffffu, in ? 1u << rank : 0u)) != n) {
            // equal keys: the lower index first
            rank = 0;
            for (int m = 0; m < n; ++m) rank += cand[m] > mine || (cand[m] == mine && expert[m] < e);
        }
        if constexpr (BIAS) {
            // neighbours of the ranking too close to tell, unless their
            // logits and biases are equal (across the border such a pair may
            // hide a third); and the last chosen too close to what is no
            // candidate
            const float be = in ? p.bias[e] : 0.f;
            float2 *tie = s_tie[warp];
            __syncwarp();
            if (in) cand[rank] = mine, tie[rank] = make_float2(xe, be);
            __syncwarp();
            const bool check = lane < p.top_k && in;
            const float k0 = check ? cand[lane] : 0.f;
            float border = bound;   // no key that is no candidate is above it
            if (want == p.top_k) {
                border = -3.402823466e38f;
#pragma unroll
                for (int i = 0; i < EPL; ++i) border = fmaxf(border, key[i] < bound ? key[i] : border);
                border = redux_max(border);
            }
            const float k1 = check && lane + 1 < n ? cand[lane + 1] : border;
            const float tol = tol_score + 0x1p-22f * (fabsf(k0) + fabsf(k1));
            const bool outside = check && lane == p.top_k - 1 && !(k0 - border > tol);
            const bool near = check && lane + 1 < n && !(k0 - k1 > tol) &&
                              !(lane + 1 < p.top_k && tie[lane].x == tie[lane + 1].x && tie[lane].y == tie[lane + 1].y);
            if (__any_sync(0xffffffffu, outside)) {
                decide_row<EPL, SOFTMAX, BIAS>(p, row);
                continue;
            }
            if (__any_sync(0xffffffffu, near)) {
                // all that may be chosen are candidates: rank those in 64 bits
                double total = 1.0;
                if constexpr (SOFTMAX) {
                    double part = 0.0;
#pragma unroll 1
                    for (int i = 0; i < my.mine; ++i) part += exp((double)l[my.e0 + i] - (double)top);
                    total = warp_sum(part);
                }
                const double exact = in ? (SOFTMAX ? exp((double)xe - (double)top) / total : 1.0 / (1.0 + exp(-(double)xe))) + (double)be
                                        : -INFINITY;
                rank = 0;
                for (int m = 0; m < n; ++m) {
                    const double o = __shfl_sync(0xffffffffu, exact, m);
                    const int oe = __shfl_sync(0xffffffffu, e, m);
                    rank += o > exact || (o == exact && oe < e);
                }
            }
        }
        if (!in) rank = 32;
        const bool chosen = rank < p.top_k;
        float w = 0.f;
        if constexpr (SOFTMAX) {
            const float most = p.renorm ? redux_max(chosen ? xe : -INFINITY) : top;
            w = chosen ? exp_of_difference(xe, most) : 0.f;
            if (!p.renorm && chosen) w = w / sum;
        } else {
            w = chosen ? sigmoid(xe) : 0.f;
        }
        if (p.renorm && n > 0) {
            const float s = warp_sum(w);
            if (!(s > 0x1p-90f)) {   // FP32 holds no full precision of it: from logarithms
                decide_row<EPL, SOFTMAX, BIAS>(p, row);
                continue;
            }
            w = w / s;
        }
        if (chosen) {
            p.idx[row * p.top_k + rank] = e;
            p.w[row * p.top_k + rank] = w * p.scale;
        }
        if (lane >= n && lane < p.top_k) {   // no expert left
            p.idx[row * p.top_k + lane] = -1;
            p.w[row * p.top_k + lane] = 0.f;
        }
    }
}

template <int EPL>
cudaError_t launch(const RouteArgs &a, bool softmax, dim3 grid, cudaStream_t s)
{
    const dim3 block(32 * kRouteWarps);
    if (softmax)
        return a.bias ? launch_pdl(route_scores_kernel<EPL, true, true>, grid, block, 0, s, a)
                      : launch_pdl(route_scores_kernel<EPL, true, false>, grid, block, 0, s, a);
    return a.bias ? launch_pdl(route_scores_kernel<EPL, false, true>, grid, block, 0, s, a)
                  : launch_pdl(route_scores_kernel<EPL, false, false>, grid, block, 0, s, a);
}

}  // namespace
}  // namespace beam

extern "C" int beam_route_scores(void *stream, const float *logits, int T, int E, long long ldl, int score,
                                 const float *bias, int n_group, int topk_group, int group_top, int top_k,
                                 int renormalize, float scale, int32_t *topk_idx, float *topk_w)
{
    using namespace beam;
    using namespace beam::ops;
    if (T < 0 || E < 1 || E > 1024) return fail(BEAM_ERR_INVALID_ARG, "T must be >= 0 and E in 1 .. 1024");
    if (score != BEAM_SCORE_SIGMOID && score != BEAM_SCORE_SOFTMAX) return fail(BEAM_ERR_INVALID_ARG, "score %d", score);
    if (n_group < 1 || n_group > 32 || E % n_group != 0)
        return fail(BEAM_ERR_INVALID_ARG, "n_group must divide E and be in 1 .. 32, got %d", n_group);
    if (topk_group < 1 || topk_group > n_group) return fail(BEAM_ERR_INVALID_ARG, "topk_group %d", topk_group);
    if (group_top != 1 && group_top != 2) return fail(BEAM_ERR_INVALID_ARG, "group_top must be 1 or 2");
    if (top_k < 1 || top_k > 32 || top_k > topk_group * (E / n_group))
        return fail(BEAM_ERR_INVALID_ARG, "top_k must be in 1 .. min(32, topk_group * E / n_group), got %d", top_k);
    if (!(scale - scale == 0.f)) return fail(BEAM_ERR_INVALID_ARG, "scale must be finite");
    if (T == 0) return BEAM_OK;
    if (!logits || !topk_idx || !topk_w) return fail(BEAM_ERR_INVALID_ARG, "logits, topk_idx and topk_w are required");
    if (ldl < E) return fail(BEAM_ERR_INVALID_ARG, "ldl is below E");
    if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4))
        return fail(BEAM_ERR_INVALID_ARG, "a pointer is not aligned");
    const int sms = sm_count();
    if (!sms) return fail(BEAM_ERR_CUDA, "no CUDA device");
    RouteArgs a{};
    a.logits = logits, a.bias = bias, a.idx = topk_idx, a.w = topk_w;
    a.ldl = ldl, a.T = T, a.E = E;
    a.group_top = group_top, a.top_k = top_k, a.renorm = renormalize != 0, a.scale = scale;
    a.keep = topk_group < n_group ? topk_group : 0;
    const RouteLayout how = route_layout(E, n_group, topk_group);
    a.lanes_log = how.lanes_log, a.size = how.size, a.epl = how.epl;
    a.vec = a.size % 4 == 0 && a.epl % 4 == 0 && rows_aligned16(logits, ldl, BEAM_F32);
    // twice the resident blocks: the second half starts where rows decided in
    // 64 bits leave room (when measured, 34 us; 38 with resident blocks only)
    const long long need = ((long long)T + kRouteWarps - 1) / kRouteWarps;
    const dim3 grid((unsigned)(need < 8LL * sms ? need : 8LL * sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool softmax = score == BEAM_SCORE_SOFTMAX;
    cudaError_t e;
    switch (how.regs) {
        case 1: e = launch<1>(a, softmax, grid, s); break;
        case 2: e = launch<2>(a, softmax, grid, s); break;
        case 4: e = launch<4>(a, softmax, grid, s); break;
        case 8: e = launch<8>(a, softmax, grid, s); break;
        case 16: e = launch<16>(a, softmax, grid, s); break;
        case 32: e = launch<32>(a, softmax, grid, s); break;
        case 64: e = launch<64>(a, softmax, grid, s); break;
        default: return fail(BEAM_ERR_UNSUPPORTED, "%d experts in %d groups", E, n_group);
    }
    return check_cuda(e, "beam_route_scores");
}
