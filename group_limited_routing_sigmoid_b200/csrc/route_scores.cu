// Routing from given logits under either score function (beam_route_scores).
//
// A warp per token.  With groups in play every group gets L lanes (a power of
// two, L * n_group <= 32), else one group of 32; a lane owns `epl` consecutive
// experts of its group, in registers.  A lane sorts its keys once (a network
// of minima and maxima, no indexes carried); a group's best two are then the
// heads of its lanes' lists, and each of the top_k rounds is one redux.max
// over the 32 heads, a ballot for the lowest lane that holds it and a shift of
// the winner's list.  The rounds' winners are turned into expert indexes
// together at the end, lane j finding key j among its owner's keys.
//
// Decisions are those of exact arithmetic: an FP32 score is off by a few
// ulps, so a row in which two keys (neighbours of the chosen ranking) or two
// group scores (last kept, first dropped) are closer than that error, and not
// exactly equal, is decided again from 64-bit scores (decide_row, the same
// warp).  Without a bias the keys are the logits themselves, which are exact.
//
// Bound by instruction issue at large T (some 350 instructions a token of 256
// grouped experts against 1 KB read), by the rounds' latency at small T.
#include "ops_common.cuh"

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
    int lanes;      // lanes a group (32 when no groups are dropped)
    int size;       // experts a group (E when no groups are dropped)
    int epl;        // experts a lane
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

// The lane's experts: `mine` of them from e0.
struct Span {
    int e0, mine;
    __device__ __forceinline__ Span(const RouteArgs &p, int lane)
    {
        const int sub = (lane & (p.lanes - 1)) * p.epl, g = lane / p.lanes;
        e0 = g * p.size + sub;
        mine = e0 < p.E ? max(min(p.size - sub, p.epl), 0) : 0;
    }
};

// Sigmoid to about 2^-22 absolute: enough to rank by, with the margins below.
__device__ __forceinline__ float sigmoid_fast(float x)
{
    float e, r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// --- sorting in registers, descending -------------------------------------------

__device__ __forceinline__ void order(float &a, float &b)
{
    const float hi = fmaxf(a, b);
    b = fminf(a, b);
    a = hi;
}

template <int N>
__device__ __forceinline__ void sort(float *v)
{
    if constexpr (N == 2) {
        order(v[0], v[1]);
    } else if constexpr (N == 4) {
        order(v[0], v[1]), order(v[2], v[3]), order(v[0], v[2]), order(v[1], v[3]), order(v[1], v[2]);
    } else if constexpr (N == 8) {   // 19 comparisons
        order(v[0], v[2]), order(v[1], v[3]), order(v[4], v[6]), order(v[5], v[7]);
        order(v[0], v[4]), order(v[1], v[5]), order(v[2], v[6]), order(v[3], v[7]);
        order(v[0], v[1]), order(v[2], v[3]), order(v[4], v[5]), order(v[6], v[7]);
        order(v[2], v[4]), order(v[3], v[5]);
        order(v[1], v[4]), order(v[3], v[6]);
        order(v[1], v[2]), order(v[3], v[4]), order(v[5], v[6]);
    }
}

// The eight largest of two sorted lists of eight, sorted, into a.
__device__ __forceinline__ void merge8(float *a, const float *b)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = fmaxf(a[i], b[7 - i]);   // bitonic
#pragma unroll
    for (int d = 4; d; d >>= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) order(a[i], a[i + d]);
}

// --- a row in 64 bits ------------------------------------------------------------

// Slow and rare.  Writes the row's outputs; every tie that is left is one of
// equal keys.
template <int EPL, bool SOFTMAX, bool BIAS>
__device__ __noinline__ void decide_row(const RouteArgs &p, long long row)
{
    const int lane = threadIdx.x & 31;
    const Span my(p, lane);
    const float *l = p.logits + row * p.ldl;
    double top = -INFINITY, log_sum = 0.0;
    double key[EPL];
    if (SOFTMAX) {
#pragma unroll 1
        for (int i = 0; i < my.mine; ++i) top = fmax(top, (double)l[my.e0 + i]);
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, d));
        double sum = 0.0;
#pragma unroll 1
        for (int i = 0; i < my.mine; ++i) sum += exp((double)l[my.e0 + i] - top);
        log_sum = log(warp_sum(sum));
    }
    // log of the score of the expert with logit x
    const auto log_score = [&](double x) {
        return SOFTMAX ? x - top - log_sum : (x < 0 ? x - log1p(exp(x)) : -log1p(exp(-x)));
    };
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        key[i] = -INFINITY;
        if (i < my.mine) {
            const double x = l[my.e0 + i];
            const double b = BIAS ? (double)p.bias[my.e0 + i] : 0.0;
            if (x > -INFINITY && b > -INFINITY) key[i] = exp(log_score(x)) + b;
        }
    }
    bool kept = true;
    if (p.keep) {
        double a = -INFINITY, b = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) b = fmax(b, fmin(a, key[i])), a = fmax(a, key[i]);
        for (int d = 1; d < p.lanes; d <<= 1) {
            const double oa = __shfl_xor_sync(0xffffffffu, a, d), ob = __shfl_xor_sync(0xffffffffu, b, d);
            b = fmax(fmin(a, oa), fmax(b, ob));
            a = fmax(a, oa);
        }
        const double score = p.group_top == 2 && b > -INFINITY ? a + b : a;
        int rank = 0;
        for (int g = 0; g < 32; g += p.lanes) {
            const double o = __shfl_sync(0xffffffffu, score, g);
            rank += o > score || (o == score && g < (lane & ~(p.lanes - 1)));
        }
        kept = rank < p.keep;
    }
    // without a bias the logits order the scores, also where those saturate
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if (!kept) key[i] = -INFINITY;
        if (!BIAS && key[i] > -INFINITY) key[i] = l[my.e0 + i];
    }
    int my_idx = -1;
    for (int j = 0; j < p.top_k; ++j) {
        double best = -INFINITY;
        int at = p.E;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > best) best = key[i], at = my.e0 + i;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const double o = __shfl_xor_sync(0xffffffffu, best, d);
            const int oa = __shfl_xor_sync(0xffffffffu, at, d);
            if (o > best || (o == best && oa < at)) best = o, at = oa;
        }
        if (at == p.E) break;
        if (lane == j) my_idx = at;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (my.e0 + i == at) key[i] = -INFINITY;
    }
    // weights from the logarithms, so that scores that underflow still share
    const double my_log = my_idx >= 0 ? log_score(l[my_idx]) : -INFINITY;
    double w = my_idx >= 0 ? exp(my_log) : 0.0;
    if (p.renorm) {
        double m = my_log;
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, d));
        w = my_idx >= 0 ? exp(my_log - m) : 0.0;
        const double s = warp_sum(w);
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
    // A lane's list holds its best eight; one that is used up in the rounds
    // sends the row to decide_row.
    constexpr int D = EPL < 8 ? EPL : 8;
    __shared__ __align__(16) float s_keys[kRouteWarps][32 * EPL];
    __shared__ float2 s_won[kRouteWarps][33];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Span my(p, lane);
    float *keys = s_keys[warp];
    float2 *won = s_won[warp];
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
        float x[EPL];
        if (EPL % 4 == 0 && p.vec) {
#pragma unroll
            for (int i = 0; i < EPL; i += 4) {
                const float4 v = i < my.mine ? *reinterpret_cast<const float4 *>(l + my.e0 + i)
                                             : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                x[i] = v.x;
                if constexpr (EPL >= 4) x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) x[i] = i < my.mine ? l[my.e0 + i] : -INFINITY;
        }
        float top = x[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) top = max_nan(top, x[i]);
        top = redux_max(top);
        if (top != top || (SOFTMAX && top == INFINITY) || nan_bias) {
            if (lane < p.top_k) {
                p.idx[row * p.top_k + lane] = -1;
                p.w[row * p.top_k + lane] = __uint_as_float(0x7fffffffu);
            }
            continue;
        }
        // softmax: the sum, where keys or weights need it
        float sum = 1.f;
        float key[EPL];
        if constexpr (SOFTMAX) {
            if (BIAS || !p.renorm) {
                sum = 0.f;
#pragma unroll
                for (int i = 0; i < EPL; ++i) {
                    key[i] = x[i] > -INFINITY ? expf(x[i] - top) : 0.f;
                    sum += key[i];
                }
                sum = warp_sum(sum);
            }
        }
        const float inv = 1.0f / sum;   // the largest softmax score
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if constexpr (BIAS) {
                const float k = (SOFTMAX ? key[i] * inv : sigmoid_fast(x[i])) + bias[i];
                key[i] = x[i] > -INFINITY ? k : -INFINITY;
            } else {
                key[i] = x[i];
            }
        }
        // How far two FP32 keys may be off together.  Sigmoid: 2^-22 each
        // (s(1-s) times the exponential's 2^-22 and its argument's rounding,
        // half an ulp of the sum, an ulp of the reciprocal).  Softmax: some
        // ulps of the largest score each (exponential 2, its argument's
        // rounding, 37 partial sums, two products).  And the rounding of the
        // added bias.
        const float tol_score = SOFTMAX ? 0x1p-19f * inv : 0x1p-20f;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < EPL; ++i) keys[lane * EPL + i] = key[i];
        if constexpr (EPL == 16) {
            sort<8>(key), sort<8>(key + 8);
            merge8(key, key + 8);
        } else if constexpr (EPL == 32) {
            sort<8>(key), sort<8>(key + 8), sort<8>(key + 16), sort<8>(key + 24);
            merge8(key, key + 8), merge8(key + 16, key + 24), merge8(key, key + 16);
        } else {
            sort<EPL>(key);
        }
        bool close = false;
        if (p.keep) {
            float a = key[0], b = D > 1 ? key[D > 1 ? 1 : 0] : -INFINITY;
            for (int d = 1; d < p.lanes; d <<= 1) {
                const float oa = __shfl_xor_sync(0xffffffffu, a, d), ob = __shfl_xor_sync(0xffffffffu, b, d);
                b = fmaxf(fminf(a, oa), fmaxf(b, ob));
                a = fmaxf(a, oa);
            }
            float pa = a, pb = b;
            if constexpr (!BIAS) {   // softmax: up to the common factor
                pa = a > -INFINITY ? (SOFTMAX ? expf(a - top) : sigmoid(a)) : -INFINITY;
                pb = b > -INFINITY ? (SOFTMAX ? expf(b - top) : sigmoid(b)) : -INFINITY;
            }
            const float score = p.group_top == 2 && pb > -INFINITY ? pa + pb : pa;
            float left = score, lo = -INFINITY;
            bool kept = false;
            for (int i = 0; i < p.keep; ++i) {
                lo = redux_max(left);
                if (lo == -INFINITY) break;
                const int first = __ffs(__ballot_sync(0xffffffffu, left == lo)) - 1;   // a group's first lane
                if ((lane & ~(p.lanes - 1)) == first) kept = true, left = -INFINITY;
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
            if (!kept) key[0] = -INFINITY;
        }
        __syncwarp();
        // with a bias one round more than top_k: the best that is not chosen
        const int rounds = BIAS ? p.top_k + 1 : p.top_k;
        int found = 0, popped = 0;
        if (!close) {
            for (; found < rounds; ++found) {
                const float best = redux_max(key[0]);
                if (best == -INFINITY) break;
                const uint32_t m = __ballot_sync(0xffffffffu, key[0] == best);
                if ((m & ((2u << lane) - 1u)) == (1u << lane)) {   // the lowest of them
                    won[found] = make_float2(best, __int_as_float(lane));
#pragma unroll
                    for (int i = 0; i + 1 < D; ++i) key[i] = key[i + 1];
                    key[D - 1] = -INFINITY;
                    if (EPL > D) ++popped;
                }
            }
            if (EPL > D) close = __any_sync(0xffffffffu, popped >= D && my.mine > D);
        }
        if (close) {
            decide_row<EPL, SOFTMAX, BIAS>(p, row);
            continue;
        }
        __syncwarp();
        // lane j: the expert of round j
        const bool in = lane < found;
        const float2 wj = won[in ? lane : 0];
        const int owner = in ? __float_as_int(wj.y) : 0;
        const float pk = __shfl_up_sync(0xffffffffu, wj.x, 1);
        const int po = __shfl_up_sync(0xffffffffu, owner, 1);
        const uint32_t repeat = __ballot_sync(0xffffffffu, in && lane > 0 && pk == wj.x && po == owner);
        int at = 0;
        if (repeat == 0u) {
#pragma unroll
            for (int i = EPL - 1; i >= 0; --i)
                if (keys[owner * EPL + i] == wj.x) at = i;
        } else {
            // equal keys of one lane: the r-th of them in index order
            int r = 0;
            for (int j = lane; j > 0 && ((repeat >> j) & 1u); --j) ++r;
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (keys[owner * EPL + i] == wj.x && r-- == 0) at = i;
        }
        const int e = owner / p.lanes * p.size + (owner & (p.lanes - 1)) * p.epl + at;
        const float xe = in && found > 0 ? l[e] : -INFINITY;
        if constexpr (BIAS) {
            // neighbours of the ranking too close to tell, unless their
            // logits and biases are equal; an equal pair across the border
            // may hide a third
            const float be = in ? p.bias[e] : 0.f;
            const float nk = lane + 1 < found ? won[lane + 1].x : -INFINITY;
            const float nx = __shfl_down_sync(0xffffffffu, xe, 1), nb = __shfl_down_sync(0xffffffffu, be, 1);
            const float tol = tol_score + 0x1p-22f * (fabsf(wj.x) + fabsf(nk));
            const bool tied = nx == xe && nb == be && lane + 1 < p.top_k;
            if (__any_sync(0xffffffffu, lane + 1 < found && !(wj.x - nk > tol) && !tied)) {
                decide_row<EPL, SOFTMAX, BIAS>(p, row);
                continue;
            }
        }
        const bool chosen = in && lane < p.top_k;
        float w = 0.f;
        if constexpr (SOFTMAX) {
            const float ref = p.renorm ? redux_max(chosen ? xe : -INFINITY) : top;
            w = chosen ? expf(xe - ref) : 0.f;
            if (!p.renorm && chosen) w = w / sum;
        } else {
            w = chosen ? sigmoid(xe) : 0.f;
        }
        if (p.renorm && found > 0) {
            const float s = warp_sum(w);
            if (!(s > 0x1p-90f)) {   // FP32 holds no full precision of it: from logarithms
                decide_row<EPL, SOFTMAX, BIAS>(p, row);
                continue;
            }
            w = w / s;
        }
        if (lane < p.top_k) {
            p.idx[row * p.top_k + lane] = chosen ? e : -1;
            p.w[row * p.top_k + lane] = w * p.scale;
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
    const bool groups = topk_group < n_group;
    a.keep = groups ? topk_group : 0;
    a.lanes = 32;
    while (groups && a.lanes * n_group > 32) a.lanes /= 2;
    a.size = groups ? E / n_group : E;
    a.epl = (a.size + a.lanes - 1) / a.lanes;
    if (a.epl > 2) a.epl = (a.epl + 3) / 4 * 4;   // whole 16-byte loads
    a.vec = a.size % 4 == 0 && a.epl % 4 == 0 && rows_aligned16(logits, ldl, BEAM_F32);
    const long long need = ((long long)T + kRouteWarps - 1) / kRouteWarps;
    const dim3 grid((unsigned)(need < 4LL * sms ? need : 4LL * sms));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool softmax = score == BEAM_SCORE_SOFTMAX;
    cudaError_t e;
    if (a.epl <= 1) e = launch<1>(a, softmax, grid, s);
    else if (a.epl <= 2) e = launch<2>(a, softmax, grid, s);
    else if (a.epl <= 4) e = launch<4>(a, softmax, grid, s);
    else if (a.epl <= 8) e = launch<8>(a, softmax, grid, s);
    else if (a.epl <= 16) e = launch<16>(a, softmax, grid, s);
    else e = launch<32>(a, softmax, grid, s);
    return check_cuda(e, "beam_route_scores");
}
