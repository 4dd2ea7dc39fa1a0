// Residual addition and root-mean-square norm, with the normalised rows in
// 16 or 32 bits and / or as MXFP8 (beam_rms_norm).
//
//   s = alpha r + beta x,   y = s rsqrt(mean(s^2) + eps) gamma
//
// One pass: a row is loaded once, kept in registers as FP32 between the sum
// of squares and the outputs, and everything written from there.  Bound by
// HBM (8 operations an element against 6 to 11 bytes).
#include "ops_common.cuh"

namespace beam {
namespace {

using namespace ops;

struct NormArgs {
    const void *x, *r;
    void *ro;
    const float *gamma;
    void *out;
    uint8_t *codes, *scales;
    long long ldx, ldr, ldro, ldo;
    int T, H, out_dtype, gamma_vec;   // gamma_vec: gamma starts on 16 bytes
    float alpha, beta, eps;
    ScaleMap map;
};

// --- eight elements at any address ------------------------------------------------
//
// Rows of an odd length, or of a strided view, start anywhere.  Their vectors
// of 8 elements are read as the aligned 16-byte units that hold them and
// shifted into place (all vectors of a row by the same `o` bytes), and
// written the same way, with the part that lies in a lane's first unit taken
// from the lane below.  1000 x 2563 fp16: 6.3 us; 10.0 us with 2-byte accesses.

template <typename T> struct Units { uint32_t w[2 * sizeof(T) + 4]; };

// Elements e .. e + 7 of a row of n elements that starts at `row`.  [lo, hi)
// is the tensor: units that reach out of it, and elements past the row's
// end, are not read.  o: bytes to shift by.
template <typename T>
__device__ __forceinline__ Units<T> load_units(const T *row, int e, int n, const void *lo, const void *hi, uint32_t &o)
{
    constexpr int NU = sizeof(T) / 2;
    Units<T> u = {};
    const T *p = row + e;
    o = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
    const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) - o);
    const int units = o ? NU + 1 : NU;
    if (e + 8 <= n && static_cast<const void *>(q) >= lo && static_cast<const void *>(q + units) <= hi) {
#pragma unroll
        for (int i = 0; i <= NU; ++i)
            if (i < units) {
                const uint4 v = q[i];
                u.w[4 * i] = v.x, u.w[4 * i + 1] = v.y, u.w[4 * i + 2] = v.z, u.w[4 * i + 3] = v.w;
            }
    } else {
        o = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e + i < n) {
                if constexpr (sizeof(T) == 4) u.w[i] = reinterpret_cast<const uint32_t *>(p)[i];
                else u.w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(p)[i] << (16 * (i & 1));
            }
    }
    return u;
}

template <typename T>
__device__ __forceinline__ Raw8<T> shift_units(const Units<T> &u, uint32_t o)
{
    constexpr int N = 2 * sizeof(T);
    uint32_t w[N + 4];
#pragma unroll
    for (int i = 0; i < N + 4; ++i) w[i] = u.w[i];
#pragma unroll
    for (int i = 0; i < N + 2; ++i) w[i] = o & 8u ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < N + 1; ++i) w[i] = o & 4u ? w[i + 1] : w[i];
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = sizeof(T) == 2 && (o & 2u) ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
    return r;
}

// v to elements e .. e + 7 of the row (those below n).  Whole warps call it,
// lane l + 1 with the vector behind lane l's where both have one.
template <typename T>
__device__ __forceinline__ void store_any8(T *row, int e, int n, const float (&v)[8])
{
    constexpr int N = 2 * sizeof(T);
    T *p = row + e;
    const uint32_t o = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
    const int lane = threadIdx.x & 31;
    const bool whole = e + 8 <= n;
    const uint32_t wholes = __ballot_sync(0xffffffffu, whole);
    uint32_t c[N + 4];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (sizeof(T) == 4) c[i + 4] = __float_as_uint(v[i]);
        else if constexpr (std::is_same<T, __nv_bfloat16>::value) c[i + 4] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        else c[i + 4] = pack_f16x2(v[2 * i], v[2 * i + 1]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __shfl_up_sync(0xffffffffu, c[N + i], 1);
    if (!whole) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e + i < n) p[i] = from_f32<T>(v[i]);
        return;
    }
    // bytes 16 - o and on of (the lane below's last 16 bytes, this lane's)
    const uint32_t s = 16u - o;
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = s & 16u ? c[i + 4] : c[i];
    const bool below = lane > 0 && ((wholes >> (lane - 1)) & 1u);
    const bool above = lane < 31 && ((wholes >> (lane + 1)) & 1u);
    if (o) {
#pragma unroll
        for (int i = 0; i < N + 2; ++i) c[i] = s & 8u ? c[i + 2] : c[i];
#pragma unroll
        for (int i = 0; i < N + 1; ++i) c[i] = s & 4u ? c[i + 1] : c[i];
        if constexpr (sizeof(T) == 2)
#pragma unroll
            for (int i = 0; i < N; ++i) c[i] = s & 2u ? __funnelshift_r(c[i], c[i + 1], 16) : c[i];
    }
    uint4 *q = reinterpret_cast<uint4 *>(reinterpret_cast<uintptr_t>(p) - o);
    if (!o || below) q[0] = make_uint4(c[0], c[1], c[2], c[3]);
    if constexpr (sizeof(T) == 4) q[1] = make_uint4(c[4], c[5], c[6], c[7]);
    if (o) {
        // the ends of a run of lanes, element by element
        const int first = (int)(s / sizeof(T));   // elements of this lane in its first unit
        const int last = 8 - (int)(o / sizeof(T));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((!below && i < first) || (!above && i >= last)) p[i] = from_f32<T>(v[i]);
    }
}

// --- the kernel -------------------------------------------------------------------

struct Bounds {
    const void *x_end, *r_end;   // one past the last element of x and residual
};

// A row per block (WARP_ROWS = 0) or per warp.  Thread t of the row's `nt`
// holds the 8-element vectors t, t + nt, ...: NV of them at most.  ALIGNED:
// every row of every matrix starts on 16 bytes and H is a multiple of 8.  A
// 32-element MXFP8 block is four neighbouring lanes.  EARLY: gamma is read
// before the row's sum is known, which shortens a row's chain of waits (64 x
// 5120: 2.7 us, 3.3 without) but takes registers that many rows need more as
// rows in flight (8192 x 5120, no residual: 46 us, 32 without, at the four blocks
// an SM that the launch bounds ask for there; 38 with three).
template <typename XT, typename RT, bool HAS_R, bool ALIGNED, int NV, bool WARP_ROWS, bool EARLY>
__global__ void __launch_bounds__(WARP_ROWS ? 128 : NV == 2 ? 512 : 1024,
                                  NV == 2 && !EARLY && !HAS_R && ALIGNED ? 4 : 1) rms_norm_kernel(const NormArgs p, const Bounds end)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int nt = WARP_ROWS ? 32 : blockDim.x;
    const int t = WARP_ROWS ? lane : threadIdx.x;
    const int row = WARP_ROWS ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= p.T) {
        // rows of the last scale tile past T: their scale bytes are zero
        if (p.codes && p.map.tiled && row < (p.T + 127) / 128 * 128)
            for (int j = t; j < p.map.n4; j += nt)
                *reinterpret_cast<uint32_t *>(p.scales + p.map.at(row, 4 * j)) = 0;
        return;
    }
    float s[NV][8];
    float sum = 0.f;
    const XT *x = static_cast<const XT *>(p.x) + (size_t)row * p.ldx;
    const RT *r = HAS_R ? static_cast<const RT *>(p.r) + (size_t)row * p.ldr : nullptr;
    RT *ro = HAS_R ? static_cast<RT *>(p.ro) + (size_t)row * p.ldro : nullptr;
    float g[EARLY ? NV : 1][8];
    const auto load_gamma = [&](int e, float (&v)[8]) {
        if (ALIGNED || (p.gamma_vec && e + 8 <= p.H)) {
            const float4 a = *reinterpret_cast<const float4 *>(p.gamma + e), b = *reinterpret_cast<const float4 *>(p.gamma + e + 4);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = e + q < p.H ? p.gamma[e + q] : 0.f;
        }
    };
    if constexpr (ALIGNED) {
        Raw8<XT> xr[NV];
        Raw8<RT> rr[HAS_R ? NV : 1];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (t + i * nt) * 8;
            if (e < p.H) {
                xr[i] = load_raw8<true>(x + e);
                if constexpr (HAS_R) rr[i] = load_raw8<true>(r + e);
            }
        }
#pragma unroll
        for (int i = 0; EARLY && i < NV; ++i) {
            const int e = (t + i * nt) * 8;
            if (e < p.H) load_gamma(e, g[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (t + i * nt) * 8;
            if (e < p.H) {
                unpack8(xr[i], s[i]);
                if constexpr (HAS_R) {
                    float rv[8];
                    unpack8(rr[i], rv);
#pragma unroll
                    for (int q = 0; q < 8; ++q) s[i][q] = fmaf(p.alpha, rv[q], p.beta * s[i][q]);
                    store8<true>(ro + e, s[i]);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) s[i][q] *= p.beta;
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) sum = fmaf(s[i][q], s[i][q], sum);
            }
        }
    } else {
        Units<XT> xu[NV];
        Units<RT> ru[HAS_R ? NV : 1];
        uint32_t xo[NV], rs[HAS_R ? NV : 1];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (t + i * nt) * 8;
            xu[i] = load_units(x, e, p.H, p.x, end.x_end, xo[i]);
            if constexpr (HAS_R) ru[i] = load_units(r, e, p.H, p.r, end.r_end, rs[i]);
        }
#pragma unroll
        for (int i = 0; EARLY && i < NV; ++i) load_gamma((t + i * nt) * 8, g[i]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            unpack8(shift_units(xu[i], xo[i]), s[i]);   // zeros past the row's end
            if constexpr (HAS_R) {
                float rv[8];
                unpack8(shift_units(ru[i], rs[i]), rv);
#pragma unroll
                for (int q = 0; q < 8; ++q) s[i][q] = fmaf(p.alpha, rv[q], p.beta * s[i][q]);
                store_any8(ro, (t + i * nt) * 8, p.H, s[i]);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) s[i][q] *= p.beta;
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) sum = fmaf(s[i][q], s[i][q], sum);
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if constexpr (!WARP_ROWS) {
        __shared__ float part[32];
        if (lane == 0) part[threadIdx.x >> 5] = sum;
        __syncthreads();
        const int nw = blockDim.x >> 5;
        sum = lane < nw ? part[lane] : 0.f;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    }
    const float scale = 1.0f / sqrtf(sum / (float)p.H + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        // an MXFP8 block's lanes are all in or all out of the row (H a
        // multiple of 32 then), so its shuffles run on whole groups
        const int e = (t + i * nt) * 8;
        const bool in = e < p.H;
        float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        uint32_t m = 0;
        if (in) {
            float gl[8];
            if constexpr (!EARLY) load_gamma(e, gl);
#pragma unroll
            for (int q = 0; q < 8; ++q) y[q] = s[i][q] * scale * (EARLY ? g[EARLY ? i : 0][q] : gl[q]);
            m = amax_bits8(y);
        }
        if (p.out) {
            const size_t at = (size_t)row * p.ldo;
            if constexpr (ALIGNED) {
                if (in) {
                    if (p.out_dtype == BEAM_BF16) store8<true>(static_cast<__nv_bfloat16 *>(p.out) + at + e, y);
                    else if (p.out_dtype == BEAM_F16) store8<true>(static_cast<__half *>(p.out) + at + e, y);
                    else store8<true>(static_cast<float *>(p.out) + at + e, y);
                }
            } else {
                if (p.out_dtype == BEAM_BF16) store_any8(static_cast<__nv_bfloat16 *>(p.out) + at, e, p.H, y);
                else if (p.out_dtype == BEAM_F16) store_any8(static_cast<__half *>(p.out) + at, e, p.H, y);
                else store_any8(static_cast<float *>(p.out) + at, e, p.H, y);
            }
        }
        if (p.codes) {
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            if (in) {
                const bool bad = m >= kInfBits;
                const uint32_t b = ue8m0_byte<kTop448>(__uint_as_float(m));
                const float inv = ue8m0_inverse(b);
#pragma unroll
                for (int q = 0; q < 8; ++q) y[q] = bad ? 0.f : y[q] * inv;
                *reinterpret_cast<uint2 *>(p.codes + (size_t)row * p.H + e) = e4m3x8(y);
                if ((lane & 3) == 0) p.scales[p.map.at(row, e >> 5)] = bad ? 0xff : (uint8_t)b;
            }
        }
    }
    // scale bytes past the row's last scale in its last tile
    if (p.codes && p.map.tiled && t < 4 * p.map.n4 - p.map.n) p.scales[p.map.at(row, p.map.n + t)] = 0;
}

template <typename XT, typename RT, bool HAS_R, bool ALIGNED>
cudaError_t launch(const NormArgs &a, const Bounds &end, cudaStream_t stream)
{
    const int rows = a.codes && a.map.tiled ? (a.T + 127) / 128 * 128 : a.T;
    const int nvec = (a.H + 7) / 8;
#define BEAM_NORM(NV, WARP, EARLY, grid, block) \
    launch_pdl(rms_norm_kernel<XT, RT, HAS_R, ALIGNED, NV, WARP, EARLY>, dim3(grid), dim3(block), 0, stream, a, end)
    if (nvec <= 32) return BEAM_NORM(1, true, true, (rows + 3) / 4, 128);
    // unaligned rows of 1001: four vectors a lane take 156 registers (31 us for
    // 8000 rows), a block of two vectors a thread 23 us
    if (ALIGNED && nvec <= 32 * 4) return BEAM_NORM(4, true, false, (rows + 3) / 4, 128);
    const int nv = nvec <= 1024 ? 2 : 4;
    const int block = ((nvec + nv - 1) / nv + 31) / 32 * 32;
    if (nv == 4) return BEAM_NORM(4, false, false, rows, block);
    if (rows <= 16 * sm_count()) return BEAM_NORM(2, false, true, rows, block);
    return BEAM_NORM(2, false, false, rows, block);
#undef BEAM_NORM
}

template <typename XT, typename RT, bool HAS_R>
cudaError_t launch_any(const NormArgs &a, bool vec, cudaStream_t stream)
{
    Bounds end{static_cast<const XT *>(a.x) + (size_t)(a.T - 1) * a.ldx + a.H,
               HAS_R ? static_cast<const RT *>(a.r) + (size_t)(a.T - 1) * a.ldr + a.H : nullptr};
    return vec ? launch<XT, RT, HAS_R, true>(a, end, stream) : launch<XT, RT, HAS_R, false>(a, end, stream);
}

template <typename XT, int XD>
cudaError_t launch_x(const NormArgs &a, int residual_dtype, bool vec, cudaStream_t stream)
{
    if (!a.r) return launch_any<XT, XT, false>(a, vec, stream);
    if (residual_dtype == XD) return launch_any<XT, XT, true>(a, vec, stream);
    return launch_any<XT, float, true>(a, vec, stream);
}

}  // namespace
}  // namespace beam

extern "C" int beam_rms_norm(void *stream, const void *x, int x_dtype, long long ldx,
                             const void *residual, int residual_dtype, long long ldr,
                             void *residual_out, long long ldro, float alpha, float beta,
                             const float *gamma, float eps, int T, int H, void *out, int out_dtype,
                             long long ldo, uint8_t *codes, uint8_t *scales, int layout)
{
    using namespace beam;
    using namespace beam::ops;
    if (T < 0 || H < 1) return fail(BEAM_ERR_INVALID_ARG, "T must be >= 0 and H >= 1");
    if (!dtype_ok(x_dtype)) return fail(BEAM_ERR_INVALID_ARG, "x_dtype %d", x_dtype);
    if ((residual == nullptr) != (residual_out == nullptr) && T > 0)
        return fail(BEAM_ERR_INVALID_ARG, "residual and residual_out go together");
    if (residual && residual_dtype != BEAM_F32 && residual_dtype != x_dtype)
        return fail(BEAM_ERR_INVALID_ARG, "residual_dtype must be BEAM_F32 or x_dtype");
    if ((codes == nullptr) != (scales == nullptr)) return fail(BEAM_ERR_INVALID_ARG, "codes and scales go together");
    if (out && !dtype_ok(out_dtype)) return fail(BEAM_ERR_INVALID_ARG, "out_dtype %d", out_dtype);
    if (codes && !layout_ok(layout)) return fail(BEAM_ERR_INVALID_ARG, "layout %d", layout);
    if (codes && H % 32 != 0) return fail(BEAM_ERR_INVALID_ARG, "H must be a multiple of 32 for MXFP8, got %d", H);
    if (!(eps >= 0.f) || !(alpha - alpha == 0.f) || !(beta - beta == 0.f))
        return fail(BEAM_ERR_INVALID_ARG, "eps must be >= 0, alpha and beta finite");
    if (T > 0x7fffff00) return fail(BEAM_ERR_UNSUPPORTED, "T must be at most 2^31 - 256, got %d", T);
    if (H > 32768) return fail(BEAM_ERR_UNSUPPORTED, "H must be at most 32768, got %d", H);
    if (T == 0) return BEAM_OK;
    if (!x || !gamma || (!out && !codes)) return fail(BEAM_ERR_INVALID_ARG, "x, gamma and an output are required");
    if (ldx < H || (residual && (ldr < H || ldro < H)) || (out && ldo < H))
        return fail(BEAM_ERR_INVALID_ARG, "a row stride is below H");
    if (!aligned(x, dtype_size(x_dtype)) || !aligned(gamma, 4) ||
        (residual && (!aligned(residual, dtype_size(residual_dtype)) || !aligned(residual_out, dtype_size(residual_dtype)))) ||
        (out && !aligned(out, dtype_size(out_dtype))) || (codes && (!aligned(codes, 16) || !aligned(scales, 4))))
        return fail(BEAM_ERR_INVALID_ARG, "a pointer is not aligned");
    const bool vec = H % 8 == 0 && rows_aligned16(x, ldx, x_dtype) && aligned(gamma, 16) &&
                     (!residual || (rows_aligned16(residual, ldr, residual_dtype) &&
                                    rows_aligned16(residual_out, ldro, residual_dtype))) &&
                     (!out || rows_aligned16(out, ldo, out_dtype));
    NormArgs a{x, residual, residual_out, gamma, out, codes, scales, ldx, ldr, ldro, ldo, T, H, out_dtype, aligned(gamma, 16),
               alpha, beta, eps, ScaleMap(codes ? layout : 0, H / 32)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (x_dtype == BEAM_BF16) e = launch_x<__nv_bfloat16, BEAM_BF16>(a, residual_dtype, vec, s);
    else if (x_dtype == BEAM_F16) e = launch_x<__half, BEAM_F16>(a, residual_dtype, vec, s);
    else e = launch_x<float, BEAM_F32>(a, residual_dtype, vec, s);
    return check_cuda(e, "beam_rms_norm");
}
