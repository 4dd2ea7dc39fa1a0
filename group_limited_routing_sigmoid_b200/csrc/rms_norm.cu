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
    int T, H, out_dtype;
    float alpha, beta, eps;
    ScaleMap map;
};

// Store V (8 or 1) consecutive output elements in the output's type.
template <int V>
__device__ __forceinline__ void store_out(void *out, int dtype, size_t at, const float (&y)[V])
{
    if constexpr (V == 8) {
        if (dtype == BEAM_BF16) store8<true>(static_cast<__nv_bfloat16 *>(out) + at, y);
        else if (dtype == BEAM_F16) store8<true>(static_cast<__half *>(out) + at, y);
        else store8<true>(static_cast<float *>(out) + at, y);
    } else {
        if (dtype == BEAM_BF16) static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(y[0]);
        else if (dtype == BEAM_F16) static_cast<__half *>(out)[at] = __float2half_rn(y[0]);
        else static_cast<float *>(out)[at] = y[0];
    }
}

// A row per block (WARP_ROWS = 0) or per warp.  Thread t of the row's `nt`
// holds the V-element vectors t, t + nt, ...: NV of them at most.
//   V = 8   16-byte aligned rows, H a multiple of 8; a 32-element MXFP8 block
//           is four neighbouring lanes;
//   V = 1   everything else; a block is one warp-wide step.
template <typename XT, typename RT, bool HAS_R, int V, int NV, bool WARP_ROWS>
__global__ void __launch_bounds__(WARP_ROWS ? 128 : V == 8 && NV == 2 ? 512 : 1024) rms_norm_kernel(const NormArgs p)
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
    const int nvec = p.H / V;   // V = 8 only with H a multiple of 8
    float s[NV][V];
    float sum = 0.f;
    const XT *x = static_cast<const XT *>(p.x) + (size_t)row * p.ldx;
    const RT *r = HAS_R ? static_cast<const RT *>(p.r) + (size_t)row * p.ldr : nullptr;
    RT *ro = HAS_R ? static_cast<RT *>(p.ro) + (size_t)row * p.ldro : nullptr;
    if constexpr (V == 8) {
        Raw8<XT> xr[NV];
        Raw8<RT> rr[HAS_R ? NV : 1];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t + i * nt < nvec) {
                xr[i] = load_raw8<true>(x + (size_t)(t + i * nt) * 8);
                if constexpr (HAS_R) rr[i] = load_raw8<true>(r + (size_t)(t + i * nt) * 8);
            }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t + i * nt < nvec) {
                float xv[8];
                unpack8(xr[i], xv);
                if constexpr (HAS_R) {
                    float rv[8];
                    unpack8(rr[i], rv);
#pragma unroll
                    for (int q = 0; q < 8; ++q) s[i][q] = fmaf(p.alpha, rv[q], p.beta * xv[q]);
                    store8<true>(ro + (size_t)(t + i * nt) * 8, s[i]);
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) s[i][q] = p.beta * xv[q];
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) sum = fmaf(s[i][q], s[i][q], sum);
            }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = t + i * nt;
            s[i][0] = 0.f;
            if (e < nvec) {
                s[i][0] = p.beta * to_f32(x[e]);
                if constexpr (HAS_R) s[i][0] = fmaf(p.alpha, to_f32(r[e]), s[i][0]);
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = t + i * nt;
            if constexpr (HAS_R)
                if (e < nvec) ro[e] = from_f32<RT>(s[i][0]);
            sum = fmaf(s[i][0], s[i][0], sum);
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
        const int vec = t + i * nt;
        // an MXFP8 block's lanes are all in or all out of the row (H a
        // multiple of 32 then), so its shuffles run on whole groups
        if constexpr (V == 8) {
            float y[8];
            uint32_t m = 0;
            if (vec < nvec) {
                const float4 g0 = reinterpret_cast<const float4 *>(p.gamma)[2 * vec];
                const float4 g1 = reinterpret_cast<const float4 *>(p.gamma)[2 * vec + 1];
                const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
                for (int q = 0; q < 8; ++q) y[q] = s[i][q] * scale * g[q];
                if (p.out) store_out<8>(p.out, p.out_dtype, (size_t)row * p.ldo + (size_t)vec * 8, y);
                m = amax_bits8(y);
            }
            if (p.codes) {
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                if (vec < nvec) {
                    const bool bad = m >= kInfBits;
                    const uint32_t b = ue8m0_byte<kTop448>(__uint_as_float(m));
                    const float inv = ue8m0_inverse(b);
#pragma unroll
                    for (int q = 0; q < 8; ++q) y[q] = bad ? 0.f : y[q] * inv;
                    *reinterpret_cast<uint2 *>(p.codes + (size_t)row * p.H + (size_t)vec * 8) = e4m3x8(y);
                    if ((lane & 3) == 0) p.scales[p.map.at(row, vec >> 2)] = bad ? 0xff : (uint8_t)b;
                }
            }
        } else {
            const bool in = vec < nvec;
            float y[1] = {in ? s[i][0] * scale * p.gamma[vec] : 0.f};
            if (in && p.out) store_out<1>(p.out, p.out_dtype, (size_t)row * p.ldo + vec, y);
            if (p.codes) {
                const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(y[0]) & 0x7fffffffu);
                if (in) {
                    const bool bad = m >= kInfBits;
                    const uint32_t b = ue8m0_byte<kTop448>(__uint_as_float(m));
                    const float v = bad ? 0.f : y[0] * ue8m0_inverse(b);
                    uint16_t d;
                    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.0f), "f"(v));
                    p.codes[(size_t)row * p.H + vec] = (uint8_t)d;
                    if (lane == 0) p.scales[p.map.at(row, vec >> 5)] = bad ? 0xff : (uint8_t)b;
                }
            }
        }
    }
    // scale bytes past the row's last scale in its last tile
    if (p.codes && p.map.tiled && t < 4 * p.map.n4 - p.map.n) p.scales[p.map.at(row, p.map.n + t)] = 0;
}

template <typename XT, typename RT, bool HAS_R>
cudaError_t launch(const NormArgs &a, bool vec, cudaStream_t stream)
{
    const int rows = a.codes && a.map.tiled ? (a.T + 127) / 128 * 128 : a.T;
    if (vec) {
        const int nvec = a.H / 8;
        if (nvec <= 32 * 4) {
            const dim3 grid((rows + 3) / 4), block(128);
            if (nvec <= 32) return launch_pdl(rms_norm_kernel<XT, RT, HAS_R, 8, 1, true>, grid, block, 0, stream, a);
            return launch_pdl(rms_norm_kernel<XT, RT, HAS_R, 8, 4, true>, grid, block, 0, stream, a);
        }
        const int nv = nvec <= 1024 ? 2 : 4;
        const dim3 block(((nvec + nv - 1) / nv + 31) / 32 * 32);
        if (nv == 2) return launch_pdl(rms_norm_kernel<XT, RT, HAS_R, 8, 2, false>, dim3(rows), block, 0, stream, a);
        return launch_pdl(rms_norm_kernel<XT, RT, HAS_R, 8, 4, false>, dim3(rows), block, 0, stream, a);
    }
    if (a.H <= 8 * 1024) {
        const dim3 block(((a.H + 7) / 8 + 31) / 32 * 32);
        return launch_pdl(rms_norm_kernel<XT, RT, HAS_R, 1, 8, false>, dim3(rows), block, 0, stream, a);
    }
    return launch_pdl(rms_norm_kernel<XT, RT, HAS_R, 1, 32, false>, dim3(rows), dim3(1024), 0, stream, a);
}

template <typename XT, int XD>
cudaError_t launch_x(const NormArgs &a, int residual_dtype, bool vec, cudaStream_t stream)
{
    if (!a.r) return launch<XT, XT, false>(a, vec, stream);
    if (residual_dtype == XD) return launch<XT, XT, true>(a, vec, stream);
    return launch<XT, float, true>(a, vec, stream);
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
    NormArgs a{x, residual, residual_out, gamma, out, codes, scales, ldx, ldr, ldro, ldo, T, H, out_dtype,
               alpha, beta, eps, ScaleMap(codes ? layout : 0, H / 32)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (x_dtype == BEAM_BF16) e = launch_x<__nv_bfloat16, BEAM_BF16>(a, residual_dtype, vec, s);
    else if (x_dtype == BEAM_F16) e = launch_x<__half, BEAM_F16>(a, residual_dtype, vec, s);
    else e = launch_x<float, BEAM_F32>(a, residual_dtype, vec, s);
    return check_cuda(e, "beam_rms_norm");
}
