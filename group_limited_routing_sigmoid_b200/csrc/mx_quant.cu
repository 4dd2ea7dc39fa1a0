// Microscaled operands (beam_mx_*): making them from 16- or 32-bit rows,
// reading them back, and laying their scales out for the tensor cores.
//
// All of it is bound by HBM: a 16-bit element is 2 bytes in and 0.53 to 1.03
// out.  A warp takes 256 consecutive elements of a row, 8 a lane (one 16-byte
// load of 16-bit elements); a block of 16 or 32 elements is 2 or 4
// neighbouring lanes, whose largest magnitude is found by shuffles.  Where
// rows are contiguous and the scales lie row by row, the whole tensor is
// taken as one row (blocks divide rows, so they do not notice).
#include "ops_common.cuh"

namespace beam {
namespace {

using namespace ops;

constexpr int kWarps = 8;          // warps a block
constexpr int kUnit = 256;         // elements a warp takes at a time

// NVFP4 tensor scales outside this range would leave the exact range of the
// arithmetic below (block scale * tensor scale, its reciprocal, residuals).
constexpr float kMinTensorScale = 0x1p-112f, kMaxTensorScale = 0x1p112f;

struct QuantArgs {
    const void *x;
    const float *tensor_scale;
    uint8_t *codes, *scales;
    long long rows, ldx;    // rows of the tensor (or 1)
    long long K;            // elements a row
    long long units;        // warp units: rows (padded to the tile) x units a row
    long long units_row;
    ScaleMap map;
};

// x / d correctly rounded, from r = 1/d rounded: one step of Markstein's
// residual correction (IBM J. Res. Dev. 34, 1990).  Ties of the 4-bit grid
// are exact quotients and stay exact.
__device__ __forceinline__ float quotient(float x, float d, float r)
{
    const float q = x * r;
    return fmaf(fmaf(-q, d, x), r, q);
}

// One unit: 8 elements a lane, at element k of `row`.  `live`: the elements
// exist; otherwise only a scale byte past the end may have to be zeroed.
template <typename T, int FMT>
__device__ __forceinline__ void quantize_unit(const QuantArgs &p, const Raw8<T> &raw, long long row,
                                              long long k, bool live, int lane, float g)
{
    float v[8];
    uint32_t m = 0;
    if (live) {
        unpack8(raw, v);
        m = amax_bits8(v);
    }
    constexpr int GROUP = FMT == BEAM_NVFP4 ? 2 : 4;
#pragma unroll
    for (int d = 1; d < GROUP; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    bool bad = m >= kInfBits;
    uint32_t sb;
    if constexpr (FMT == BEAM_NVFP4) {
        bad |= !(g >= kMinTensorScale && g <= kMaxTensorScale);
        sb = bad ? 0x7fu : e4m3_byte(__uint_as_float(m) / (6.0f * g));
        const float d = e4m3x2_values(sb).x * g;
        const float r = 1.0f / d;
        const bool zero = bad || sb == 0;
        // a block whose scale saturated (a tensor scale found on other data):
        // its large quotients only have to stay large, and may be infinite
        const bool over = !(__uint_as_float(m) * r < 8.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = over ? v[i] * r : quotient(v[i], d, r);
            v[i] = zero ? 0.f : q;
        }
    } else {
        constexpr uint32_t TOP = FMT == BEAM_MXFP4 ? kTop6 : kTop448;
        sb = bad ? 0xffu : ue8m0_byte<TOP>(__uint_as_float(m));
        const float inv = bad ? 0.f : ue8m0_inverse(sb);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = bad ? 0.f : v[i] * inv;
    }
    if (live) {
        const size_t at = (size_t)row * p.K + k;
        if constexpr (FMT == BEAM_MXFP8) *reinterpret_cast<uint2 *>(p.codes + at) = e4m3x8(v);
        else *reinterpret_cast<uint32_t *>(p.codes + at / 2) = e2m1x8(v);
    }
    constexpr int BLOCK = 8 * GROUP;
    const long long j = k / BLOCK;
    if ((lane & (GROUP - 1)) == 0) {
        if (live) p.scales[p.map.at(row, j)] = (uint8_t)sb;
        else if (p.map.tiled && j < 4 * p.map.n4) p.scales[p.map.at(row, j)] = 0;
    }
}

template <typename T, int FMT, bool ALIGNED>
__global__ void __launch_bounds__(32 * kWarps) mx_quantize_kernel(const QuantArgs p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const float g = FMT == BEAM_NVFP4 ? *p.tensor_scale : 1.0f;
    const T *x = static_cast<const T *>(p.x);
    const long long step = (long long)gridDim.x * kWarps;
    for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < p.units; u += step) {
        const long long row = p.units_row == p.units ? 0 : u / p.units_row;
        const long long k = (u - row * p.units_row) * kUnit + lane * 8;
        const bool live = row < p.rows && k < p.K;
        Raw8<T> raw = {};
        if (live) raw = load_raw8<ALIGNED>(x + row * p.ldx + k);
        quantize_unit<T, FMT>(p, raw, row, k, live, lane, g);
    }
}

// Tensor scale: the least power of two g with amax <= 2688 g over the finite
// magnitudes.  g grows with amax, so blocks join theirs with an integer
// maximum of its bits, in any order.
__device__ __forceinline__ float tensor_scale_of(uint32_t amax_bits)
{
    const uint32_t b = max(amax_bits, __float_as_uint(0x1p-100f));
    constexpr uint32_t top = 0x45280000u;   // 2688 = 1.3125 x 2^11
    const int e = (int)(b >> 23) - 11 + ((b & 0x7fffffu) > (top & 0x7fffffu) ? 1 : 0);
    return __uint_as_float((uint32_t)e << 23);
}

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(32 * kWarps) mx_amax_kernel(const QuantArgs p, float *out)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const T *x = static_cast<const T *>(p.x);
    const long long step = (long long)gridDim.x * kWarps;
    uint32_t m = 0;
    for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < p.units; u += step) {
        const long long row = p.units_row == p.units ? 0 : u / p.units_row;
        const long long k = (u - row * p.units_row) * kUnit + lane * 8;
        const T *at = x + row * p.ldx + k;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (k + 8 <= p.K) {
            unpack8(load_raw8<ALIGNED>(at), v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (k + i < p.K) v[i] = to_f32(at[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
            m = max(m, b >= kInfBits ? 0u : b);
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    __shared__ uint32_t part[kWarps];
    if (lane == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < kWarps; ++i) m = max(m, part[i]);
        atomicMax(reinterpret_cast<int *>(out), __float_as_int(tensor_scale_of(m)));
    }
}

struct DequantArgs {
    const uint8_t *codes, *scales;
    const float *tensor_scale;
    void *out;
    long long rows, ldo, K, units, units_row;
    ScaleMap map;
};

template <typename T, int FMT, bool ALIGNED>
__global__ void __launch_bounds__(32 * kWarps) mx_dequantize_kernel(const DequantArgs p)
{
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const float g = p.tensor_scale ? *p.tensor_scale : 1.0f;
    const long long step = (long long)gridDim.x * kWarps;
    constexpr int BLOCK = FMT == BEAM_NVFP4 ? 16 : 32;
    for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < p.units; u += step) {
        const long long row = p.units_row == p.units ? 0 : u / p.units_row;
        const long long k = (u - row * p.units_row) * kUnit + lane * 8;
        if (k >= p.K) continue;
        const size_t at = (size_t)row * p.K + k;
        const uint32_t sb = p.scales[p.map.at(row, k / BLOCK)];
        const float s = FMT == BEAM_NVFP4 ? e4m3x2_values(sb).x : ue8m0_value(sb);
        float v[8];
        if constexpr (FMT == BEAM_MXFP8) {
            const uint2 c = *reinterpret_cast<const uint2 *>(p.codes + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = e4m3x2_values((i < 2 ? c.x : c.y) >> (16 * (i & 1)) & 0xffffu);
                v[2 * i] = f.x, v[2 * i + 1] = f.y;
            }
        } else {
            const uint32_t c = *reinterpret_cast<const uint32_t *>(p.codes + at / 2);
            uint32_t h[4];
            asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
                "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
                "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
                "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
                "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
                "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
                : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
                : "r"(c));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
                v[2 * i] = f.x, v[2 * i + 1] = f.y;
            }
        }
        // element * block scale first: exact in FP32 (it may only leave the
        // normal range for power-of-two scales next to 2^-127), then the
        // tensor scale, rounded once
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * s * g;
        store8<ALIGNED>(static_cast<T *>(p.out) + row * p.ldo + k, v);
    }
}

// Scales from rows to tiles: a thread per 4-byte group of a tile row.
__global__ void mx_tile_scales_kernel(const uint8_t *scales, uint8_t *tiled, long long rows, ScaleMap map,
                                      long long groups)
{
    pdl_launch_dependents();
    pdl_wait();
    const long long step = (long long)gridDim.x * blockDim.x;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < groups; i += step) {
        const long long row = i / map.n4;
        const int j4 = (int)(i - row * map.n4);
        uint32_t v = 0;
        if (row < rows)
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (4 * j4 + b < map.n) v |= (uint32_t)scales[row * map.n + 4 * j4 + b] << (8 * b);
        *reinterpret_cast<uint32_t *>(tiled + map.at(row, 4 * j4)) = v;
    }
}

// Blocks for `units` warp units: every SM's 8 resident blocks at most.
int grid_for(long long units)
{
    const long long need = (units + kWarps - 1) / kWarps;
    const long long most = (long long)sm_count() * 8;
    return (int)(need < most ? need : most);
}

template <int FMT>
cudaError_t launch_quantize(const QuantArgs &a, int dtype, bool al, cudaStream_t s)
{
    const dim3 grid(grid_for(a.units)), block(32 * kWarps);
#define BEAM_Q(T) (al ? launch_pdl(mx_quantize_kernel<T, FMT, true>, grid, block, 0, s, a) \
                      : launch_pdl(mx_quantize_kernel<T, FMT, false>, grid, block, 0, s, a))
    if (dtype == BEAM_BF16) return BEAM_Q(__nv_bfloat16);
    if (dtype == BEAM_F16) return BEAM_Q(__half);
    return BEAM_Q(float);
#undef BEAM_Q
}

template <int FMT>
cudaError_t launch_dequantize(const DequantArgs &a, int dtype, bool al, cudaStream_t s)
{
    const dim3 grid(grid_for(a.units)), block(32 * kWarps);
#define BEAM_D(T) (al ? launch_pdl(mx_dequantize_kernel<T, FMT, true>, grid, block, 0, s, a) \
                      : launch_pdl(mx_dequantize_kernel<T, FMT, false>, grid, block, 0, s, a))
    if (dtype == BEAM_BF16) return BEAM_D(__nv_bfloat16);
    if (dtype == BEAM_F16) return BEAM_D(__half);
    return BEAM_D(float);
#undef BEAM_D
}

int check_shape(int format, long long rows, int K, int layout)
{
    if (!format_ok(format)) return fail(BEAM_ERR_INVALID_ARG, "format %d", format);
    if (!layout_ok(layout)) return fail(BEAM_ERR_INVALID_ARG, "layout %d", layout);
    if (rows < 0 || rows > (1LL << 40)) return fail(BEAM_ERR_INVALID_ARG, "rows %lld", rows);
    if (K <= 0 || K % block_of(format) != 0)
        return fail(BEAM_ERR_INVALID_ARG, "K must be a positive multiple of %d, got %d", block_of(format), K);
    return BEAM_OK;
}

}  // namespace
}  // namespace beam

extern "C" {

long long beam_mx_scale_bytes(int format, long long rows, int K, int layout)
{
    using namespace beam;
    if (int rc = check_shape(format, rows, K, layout)) return rc;
    const long long n = K / ops::block_of(format);
    if (layout == BEAM_SCALES_ROWS) return rows * n;
    return (rows + 127) / 128 * ((n + 3) / 4) * 512;
}

int beam_mx_tensor_scale(void *stream, const void *x, int dtype, long long rows, int K, long long ldx,
                         float *tensor_scale)
{
    using namespace beam;
    using namespace beam::ops;
    if (rows < 0 || rows > (1LL << 40) || K < 1) return fail(BEAM_ERR_INVALID_ARG, "rows must be >= 0 and K >= 1");
    if (!dtype_ok(dtype)) return fail(BEAM_ERR_INVALID_ARG, "dtype %d", dtype);
    if (!tensor_scale || !aligned(tensor_scale, 4)) return fail(BEAM_ERR_INVALID_ARG, "tensor_scale is NULL or not aligned");
    if (rows > 0 && (!x || !aligned(x, dtype_size(dtype)))) return fail(BEAM_ERR_INVALID_ARG, "x is NULL or not aligned");
    if (rows > 0 && ldx < K) return fail(BEAM_ERR_INVALID_ARG, "ldx is below K");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!sm_count()) return fail(BEAM_ERR_CUDA, "no CUDA device");
    if (int rc = check_cuda(cudaMemsetAsync(tensor_scale, 0, sizeof(float), s), "cudaMemsetAsync")) return rc;
    const bool flat = rows == 1 || ldx == K;
    const long long n = flat ? rows * (long long)K : K;
    const bool al = rows_aligned16(x, flat ? 8 : ldx, dtype);
    const long long per = (n + kUnit - 1) / kUnit;
    const QuantArgs a{x, nullptr, nullptr, nullptr, flat ? 1 : rows, ldx, n, flat ? per : per * rows, per, ScaleMap(0, 1)};
    const dim3 grid(a.units ? grid_for(a.units) : 1), block(32 * kWarps);
    cudaError_t e;
#define BEAM_A(T) (al ? launch_pdl(mx_amax_kernel<T, true>, grid, block, 0, s, a, tensor_scale) \
                      : launch_pdl(mx_amax_kernel<T, false>, grid, block, 0, s, a, tensor_scale))
    if (dtype == BEAM_BF16) e = BEAM_A(__nv_bfloat16);
    else if (dtype == BEAM_F16) e = BEAM_A(__half);
    else e = BEAM_A(float);
#undef BEAM_A
    return check_cuda(e, "beam_mx_tensor_scale");
}

int beam_mx_quantize(void *stream, const void *x, int dtype, long long rows, int K, long long ldx,
                     int format, int layout, const float *tensor_scale, uint8_t *codes, uint8_t *scales)
{
    using namespace beam;
    using namespace beam::ops;
    if (int rc = check_shape(format, rows, K, layout)) return rc;
    if (!dtype_ok(dtype)) return fail(BEAM_ERR_INVALID_ARG, "dtype %d", dtype);
    if (rows == 0) return BEAM_OK;
    if (!x || !codes || !scales) return fail(BEAM_ERR_INVALID_ARG, "x, codes and scales are required");
    if ((format == BEAM_NVFP4) != (tensor_scale != nullptr))
        return fail(BEAM_ERR_INVALID_ARG, "tensor_scale is required for NVFP4 and must be NULL for the others");
    if (ldx < K) return fail(BEAM_ERR_INVALID_ARG, "ldx is below K");
    if (!aligned(x, dtype_size(dtype)) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(tensor_scale, 4))
        return fail(BEAM_ERR_INVALID_ARG, "a pointer is not aligned");
    if (!sm_count()) return fail(BEAM_ERR_CUDA, "no CUDA device");
    const int n = K / block_of(format);
    const bool flat = layout == BEAM_SCALES_ROWS && (rows == 1 || ldx == K);
    QuantArgs a{x, tensor_scale, codes, scales, rows, ldx, K, 0, 0, ScaleMap(layout, n)};
    if (flat) {
        a.rows = 1;
        a.K = rows * (long long)K;
        a.units = a.units_row = (a.K + kUnit - 1) / kUnit;
    } else {
        // tiled: the unit range covers the padding rows and scales too
        const long long span = layout == BEAM_SCALES_TILED ? (long long)a.map.n4 * 4 * block_of(format) : K;
        a.units_row = (span + kUnit - 1) / kUnit;
        a.units = a.units_row * (layout == BEAM_SCALES_TILED ? (rows + 127) / 128 * 128 : rows);
    }
    const bool al = rows_aligned16(x, flat ? 8 : ldx, dtype);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (format == BEAM_NVFP4) e = launch_quantize<BEAM_NVFP4>(a, dtype, al, s);
    else if (format == BEAM_MXFP4) e = launch_quantize<BEAM_MXFP4>(a, dtype, al, s);
    else e = launch_quantize<BEAM_MXFP8>(a, dtype, al, s);
    return check_cuda(e, "beam_mx_quantize");
}

int beam_mx_dequantize(void *stream, const uint8_t *codes, const uint8_t *scales,
                       const float *tensor_scale, int format, int layout, long long rows, int K,
                       void *out, int dtype, long long ldo)
{
    using namespace beam;
    using namespace beam::ops;
    if (int rc = check_shape(format, rows, K, layout)) return rc;
    if (!dtype_ok(dtype)) return fail(BEAM_ERR_INVALID_ARG, "dtype %d", dtype);
    if (rows == 0) return BEAM_OK;
    if (!codes || !scales || !out) return fail(BEAM_ERR_INVALID_ARG, "codes, scales and out are required");
    if (ldo < K) return fail(BEAM_ERR_INVALID_ARG, "ldo is below K");
    if (!aligned(out, dtype_size(dtype)) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(tensor_scale, 4))
        return fail(BEAM_ERR_INVALID_ARG, "a pointer is not aligned");
    if (!sm_count()) return fail(BEAM_ERR_CUDA, "no CUDA device");
    const bool flat = layout == BEAM_SCALES_ROWS && (rows == 1 || ldo == K);
    DequantArgs a{codes, scales, tensor_scale, out, rows, ldo, K, 0, 0, ScaleMap(layout, K / block_of(format))};
    if (flat) a.rows = 1, a.K = rows * (long long)K;
    a.units_row = (a.K + kUnit - 1) / kUnit;
    a.units = a.units_row * a.rows;
    const bool al = rows_aligned16(out, flat ? 8 : ldo, dtype);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (format == BEAM_NVFP4) e = launch_dequantize<BEAM_NVFP4>(a, dtype, al, s);
    else if (format == BEAM_MXFP4) e = launch_dequantize<BEAM_MXFP4>(a, dtype, al, s);
    else e = launch_dequantize<BEAM_MXFP8>(a, dtype, al, s);
    return check_cuda(e, "beam_mx_dequantize");
}

int beam_mx_tile_scales(void *stream, int format, const uint8_t *scales, long long rows, int K,
                        uint8_t *tiled)
{
    using namespace beam;
    using namespace beam::ops;
    if (int rc = check_shape(format, rows, K, BEAM_SCALES_TILED)) return rc;
    if (rows == 0) return BEAM_OK;
    if (!scales || !tiled || !aligned(tiled, 4)) return fail(BEAM_ERR_INVALID_ARG, "scales or tiled is NULL or not aligned");
    if (!sm_count()) return fail(BEAM_ERR_CUDA, "no CUDA device");
    const ScaleMap map(BEAM_SCALES_TILED, K / block_of(format));
    const long long groups = (rows + 127) / 128 * 128 * map.n4;
    return check_cuda(launch_pdl(mx_tile_scales_kernel, dim3(grid_for(groups / 32 + 1)), dim3(256), 0,
                                 static_cast<cudaStream_t>(stream), scales, tiled, rows, map, groups),
                      "beam_mx_tile_scales");
}

}  // extern "C"
