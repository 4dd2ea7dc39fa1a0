// Routing from given logits under either score function (beam_route_scores).
//
// A warp per token.  Lane l owns the `epl` = ceil(E / 32) consecutive experts
// from l * epl, kept in registers.  Scores in FP32, groups ranked by the sum
// of their best keys, then top_k rounds of a warp-wide maximum (redux) over
// order-preserving integer keys, ties to the lower index.
//
// Decisions are those of exact arithmetic: an FP32 score is off by a few
// ulps, so a row in which two keys (neighbours of the chosen ranking) or two
// group scores (last kept, first dropped) are closer than that error is
// decided again from 64-bit scores (decide_row, the same warp).  Without a
// bias the keys are ranked by the logits themselves, which are exact.
//
// Bound by HBM at large T (4 bytes an expert), by the top-k rounds' latency
// at small T.
#include "ops_common.cuh"

namespace beam {
namespace {

using namespace ops;

constexpr int kRouteWarps = 4;

struct RouteArgs {
    const float *logits, *bias;
    int32_t *idx;
    float *w;
    long long ldl;
    int T, E, epl, n_group, topk_group, group_top, top_k, softmax, renorm;
    float scale;
};

// Unsigned key that orders as the float does; NaN is excluded beforehand.
// 0 is below every float's key: "not eligible".
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t b = __float_as_uint(v);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    return v;
}

template <typename F>
__device__ __forceinline__ F warp_sum(F v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// Decide a row in 64 bits, from shared memory: slow and rare.  key[e] and
// logp[e] (log of the score) are this warp's E doubles each.  Writes the
// row's outputs; every tie that is left is one of equal keys.
__device__ __noinline__ void decide_row(const RouteArgs &p, long long row, double *key, double *logp)
{
    const int lane = threadIdx.x & 31;
    const float *l = p.logits + row * p.ldl;
    double top = -INFINITY;
    for (int e = lane; e < p.E; e += 32) top = fmax(top, (double)l[e]);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, d));
    double log_sum = 0.0;
    if (p.softmax) {
        double sum = 0.0;
        for (int e = lane; e < p.E; e += 32) sum += exp((double)l[e] - top);
        log_sum = log(warp_sum(sum));
    }
    for (int e = lane; e < p.E; e += 32) {
        const double x = l[e];
        const double b = p.bias ? (double)p.bias[e] : 0.0;
        const bool ok = x > -INFINITY && b > -INFINITY;
        const double lp = p.softmax ? x - top - log_sum
                                    : (x < 0 ? x - log1p(exp(x)) : -log1p(exp(-x)));
        logp[e] = lp;
        // without a bias the logits order the scores, also where those
        // saturate
        key[e] = !ok ? -INFINITY : exp(lp) + b;
    }
    __syncwarp();
    if (p.topk_group < p.n_group) {
        const int size = p.E / p.n_group;
        double score = -INFINITY;
        if (lane < p.n_group) {
            double a = -INFINITY, b = -INFINITY;
            for (int e = lane * size; e < (lane + 1) * size; ++e) {
                const double k = key[e];
                if (k > a) b = a, a = k;
                else if (k > b) b = k;
            }
            score = a;
            if (p.group_top == 2 && b > -INFINITY) score += b;
        }
        int rank = 0;
        for (int g = 0; g < p.n_group; ++g) {
            const double o = __shfl_sync(0xffffffffu, score, g);
            rank += o > score || (o == score && g < lane);
        }
        const uint32_t kept = __ballot_sync(0xffffffffu, lane < p.n_group && rank < p.topk_group);
        __syncwarp();
        for (int e = lane; e < p.E; e += 32)
            if (!((kept >> (e / size)) & 1u)) key[e] = -INFINITY;
        __syncwarp();
    }
    int my_idx = -1;
    double my_log = -INFINITY;
    for (int j = 0; j < p.top_k; ++j) {
        double best = -INFINITY;
        float bl = -INFINITY;
        int at = p.E;
        for (int e = lane; e < p.E; e += 32) {
            const float x = p.bias ? 0.f : l[e];
            if (key[e] > -INFINITY && (p.bias ? key[e] > best : (x > bl || at == p.E))) best = key[e], bl = x, at = e;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const double o = __shfl_xor_sync(0xffffffffu, best, d);
            const float ol = __shfl_xor_sync(0xffffffffu, bl, d);
            const int oa = __shfl_xor_sync(0xffffffffu, at, d);
            const bool more = p.bias ? o > best : ol > bl;
            const bool same = p.bias ? o == best : ol == bl;
            if (oa < p.E && (at == p.E || more || (same && oa < at))) best = o, bl = ol, at = oa;
        }
        if (at == p.E) break;
        if (lane == j) my_idx = at, my_log = logp[at];
        __syncwarp();
        if (lane == 0) key[at] = -INFINITY;
        __syncwarp();
    }
    // weights from the logarithms, so that scores that underflow still share
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

template <int EPL>
__global__ void __launch_bounds__(32 * kRouteWarps) route_scores_kernel(const RouteArgs p)
{
    extern __shared__ double s_route[];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double *s_key = s_route + (size_t)warp * 2 * p.E;
    float *s_f = reinterpret_cast<float *>(s_key);
    const int e0 = lane * p.epl;
    const int mine = min(max(p.E - e0, 0), p.epl);
    for (long long row = (long long)blockIdx.x * kRouteWarps + warp; row < p.T;
         row += (long long)gridDim.x * kRouteWarps) {
        const float *l = p.logits + row * p.ldl;
        float x[EPL], sc[EPL], key[EPL];   // logit, score, key
        bool nan = false;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            x[i] = i < mine ? l[e0 + i] : -INFINITY;
            nan |= x[i] != x[i] || (p.softmax && x[i] == INFINITY);
            top = fmaxf(top, x[i]);
        }
        float inv = 1.f, pmax = 1.f;
        if (p.softmax) {
            top = warp_max(top);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                sc[i] = x[i] > -INFINITY ? expf(x[i] - top) : 0.f;
                sum += sc[i];
            }
            sum = warp_sum(sum);
            inv = 1.0f / sum;
            pmax = inv;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (p.softmax) sc[i] *= inv;
            else sc[i] = 1.0f / (1.0f + expf(-x[i]));
            const float b = p.bias && i < mine ? p.bias[e0 + i] : 0.f;
            nan |= b != b;
            if (b == -INFINITY) x[i] = -INFINITY;   // never chosen
            key[i] = x[i] > -INFINITY ? sc[i] + b : -INFINITY;
        }
        if (__any_sync(0xffffffffu, nan)) {
            if (lane < p.top_k) {
                p.idx[row * p.top_k + lane] = -1;
                p.w[row * p.top_k + lane] = __uint_as_float(0x7fffffffu);
            }
            continue;
        }
        // How far two FP32 keys may be off together: a score carries a few
        // ulps (exponential 2, division and sum 1 each, 32 partial sums in
        // the softmax), the added bias half an ulp of the key.
        const float tol_score = 0x1p-20f * pmax;
        bool close = false;
        uint32_t kept_mask = 0xffffffffu;
        if (p.topk_group < p.n_group) {
            const int size = p.E / p.n_group;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i < mine) s_f[e0 + i] = key[i];
            __syncwarp();
            float score = -INFINITY;
            if (lane < p.n_group) {
                float a = -INFINITY, b = -INFINITY;
                for (int e = lane * size; e < (lane + 1) * size; ++e) {
                    const float k = s_f[e];
                    b = fmaxf(b, fminf(a, k));
                    a = fmaxf(a, k);
                }
                score = a;
                if (p.group_top == 2 && b > -INFINITY) score += b;
            }
            __syncwarp();
            int rank = 0;
            for (int g = 0; g < p.n_group; ++g) {
                const float o = __shfl_sync(0xffffffffu, score, g);
                rank += o > score || (o == score && g < lane);
            }
            const bool in = lane < p.n_group && rank < p.topk_group;
            kept_mask = __ballot_sync(0xffffffffu, in);
            // last kept against first dropped
            const float lo = -warp_max(in ? -score : -INFINITY);
            const float hi = warp_max(lane < p.n_group && !in ? score : -INFINITY);
            const float tol = 2.f * tol_score + 0x1p-21f * (fabsf(lo) + fabsf(hi));
            close = hi > -INFINITY && !(lo - hi > tol);
        }
        // keys to integers: the logits' order without a bias
        uint32_t ord[EPL];
        const int size = p.E / p.n_group;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const bool ok = i < mine && key[i] > -INFINITY && ((kept_mask >> ((e0 + i) / size)) & 1u);
            ord[i] = ok ? order_key(p.bias ? key[i] : x[i]) : 0u;
        }
        int my_idx = -1;
        float my_w = 0.f;
        float last = INFINITY, last_x = 0.f, last_b = 0.f;
        // one round more than top_k: the best that was not chosen
        for (int j = 0; j <= p.top_k && !close; ++j) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) m = max(m, ord[i]);
            const uint32_t best = __reduce_max_sync(0xffffffffu, m);
            if (best == 0u) break;
            int at = 0x7fffffff;
            if (m == best) {
#pragma unroll
                for (int i = EPL - 1; i >= 0; --i)
                    if (ord[i] == best) at = e0 + i;
            }
            const int e = (int)__reduce_min_sync(0xffffffffu, (uint32_t)at);
            const int owner = e / p.epl;
            float ks = 0.f, kk = 0.f, kx = 0.f;
            if (lane == owner) {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (e0 + i == e) {
                        ks = sc[i], kk = key[i], kx = x[i];
                        ord[i] = 0u;
                    }
            }
            if (p.bias) {
                kk = __shfl_sync(0xffffffffu, kk, owner);
                kx = __shfl_sync(0xffffffffu, kx, owner);
                const float kb = p.bias[e];
                const float tol = tol_score + 0x1p-22f * (fabsf(last) + fabsf(kk));
                // equal logits and biases tie exactly: the index has decided
                if (j > 0 && !(last - kk > tol) && !(kx == last_x && kb == last_b)) close = true;
                last = kk, last_x = kx, last_b = kb;
            }
            if (j < p.top_k) {
                ks = __shfl_sync(0xffffffffu, ks, owner);
                if (lane == j) my_idx = e, my_w = ks;
            }
        }
        if (p.renorm && !close) {
            const float s = warp_sum(my_w);
            // a sum that FP32 holds no full precision of: from logarithms
            if (__shfl_sync(0xffffffffu, my_idx, 0) >= 0 && !(s > 0x1p-90f)) close = true;
            my_w = my_w / s;
        }
        if (close) {
            __syncwarp();
            decide_row(p, row, s_key, s_key + p.E);
            __syncwarp();
            continue;
        }
        if (lane < p.top_k) {
            p.idx[row * p.top_k + lane] = my_idx;
            p.w[row * p.top_k + lane] = my_idx >= 0 ? my_w * p.scale : 0.f;
        }
    }
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
    RouteArgs a{logits, bias, topk_idx, topk_w, ldl, T, E, (E + 31) / 32, n_group, topk_group, group_top,
                top_k, score == BEAM_SCORE_SOFTMAX, renormalize != 0, scale};
    const size_t smem = (size_t)kRouteWarps * 2 * E * sizeof(double);
    const long long need = ((long long)T + kRouteWarps - 1) / kRouteWarps;
    const dim3 grid((unsigned)(need < 16LL * sms ? need : 16LL * sms)), block(32 * kRouteWarps);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
#define BEAM_R(N)                                                                                          \
    do {                                                                                                   \
        if (smem > 48 * 1024)                                                                              \
            e = cudaFuncSetAttribute(route_scores_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize,  \
                                     (int)smem);                                                           \
        if (e == cudaSuccess) e = launch_pdl(route_scores_kernel<N>, grid, block, smem, s, a);             \
    } while (0)
    if (a.epl <= 1) BEAM_R(1);
    else if (a.epl <= 2) BEAM_R(2);
    else if (a.epl <= 4) BEAM_R(4);
    else if (a.epl <= 8) BEAM_R(8);
    else if (a.epl <= 16) BEAM_R(16);
    else BEAM_R(32);
#undef BEAM_R
    return check_cuda(e, "beam_route_scores");
}
