// Shared pieces of the handle-free operators (beam_ops.h): element types,
// 8-element loads and stores, the microscaled block formats.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "beam_ops.h"
#include "kernels.cuh"

namespace beam {
namespace ops {

// Record a host-side error text for beam_ops_error and return `code`.
int fail(int code, const char *fmt, ...);
int check_cuda(cudaError_t e, const char *what);

inline bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int dtype_size(int dtype) { return dtype == BEAM_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype >= BEAM_BF16 && dtype <= BEAM_F32; }
constexpr int block_size(int format) { return format == BEAM_NVFP4 ? 16 : 32; }
inline int block_of(int format) { return format == BEAM_NVFP4 ? 16 : 32; }
inline bool format_ok(int format) { return format >= BEAM_NVFP4 && format <= BEAM_MXFP8; }
inline bool layout_ok(int layout) { return layout == BEAM_SCALES_ROWS || layout == BEAM_SCALES_TILED; }

// Whether rows of `ld` elements from `p` all start on 16-byte boundaries.
inline bool rows_aligned16(const void *p, long long ld, int dtype)
{
    return aligned(p, 16) && (ld * dtype_size(dtype)) % 16 == 0;
}

// SMs of the current device (looked up once per device), or 0 on an error.
int sm_count();

template <int DT> struct TypeOf;
template <> struct TypeOf<BEAM_BF16> { using type = __nv_bfloat16; };
template <> struct TypeOf<BEAM_F16> { using type = __half; };
template <> struct TypeOf<BEAM_F32> { using type = float; };

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f32(float v) { return v; }

// Eight consecutive elements as they lie in memory: 16-byte loads when the
// address allows it (ALIGNED), element loads otherwise.
template <typename T> struct Raw8 { uint32_t w[2 * sizeof(T)]; };   // 4 words of 16 bits x 2, or 8

template <bool ALIGNED, typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T *p)
{
    Raw8<T> r;
    if constexpr (ALIGNED) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
            r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
        }
    } else if constexpr (sizeof(T) == 2) {
        const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = (uint32_t)q[2 * i] | ((uint32_t)q[2 * i + 1] << 16);
    } else {
        const uint32_t *q = reinterpret_cast<const uint32_t *>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) r.w[i] = q[i];
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T> &r, float (&v)[8])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(r.w[i] << 16);
            v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[i]));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

template <bool ALIGNED, typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8])
{
    if constexpr (!ALIGNED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = from_f32<T>(v[i]);
    } else if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint4 o;
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
            o = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                           pack_bf16x2(v[6], v[7]));
        else
            o = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]),
                           pack_f16x2(v[6], v[7]));
        *reinterpret_cast<uint4 *>(p) = o;
    }
}

// ---------------------------------------------------------------------------
// Microscaled blocks
// ---------------------------------------------------------------------------

// Where the scale byte (row, j) lies.
struct ScaleMap {
    int tiled;
    int n;       // scales per row
    int n4;      // ceil(n / 4)
    __host__ __device__ ScaleMap(int layout, int n_) : tiled(layout), n(n_), n4((n_ + 3) / 4) {}
    __device__ __forceinline__ size_t at(long long row, long long j) const
    {
        if (!tiled) return (size_t)(row * n + j);
        return (size_t)((row >> 7) * n4 + (j >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (j & 3);
    }
};

// UE8M0 scale of a block of finite amax: the least k with amax <= top 2^k,
// top = 6 (0x40c00000) or 448 (0x43e00000), clamped to [-127, 127]; as the
// byte k + 127.  With amax = 1.m 2^e and top = 1.t 2^f this is e - f, or
// e - f + 1 where m > t.  amax below 2^-126 (exponent field 0) gives 0.
template <uint32_t TOP_BITS>
__device__ __forceinline__ uint32_t ue8m0_byte(float amax)
{
    const uint32_t b = __float_as_uint(amax);
    constexpr int f = (int)(TOP_BITS >> 23) - 127;
    constexpr uint32_t t = TOP_BITS & 0x7fffffu;
    const int k = (int)(b >> 23) - f + ((b & 0x7fffffu) > t ? 1 : 0);   // biased by 127
    return (uint32_t)max(k, 0);
}

// 2^-(byte - 127) for a byte in 0 .. 253: exact, normal.
__device__ __forceinline__ float ue8m0_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// 2^(byte - 127): byte 0 is the subnormal 2^-127, 255 is NaN.
__device__ __forceinline__ float ue8m0_value(uint32_t byte)
{
    return byte == 0 ? __uint_as_float(0x00400000u)
                     : byte == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float(byte << 23);
}

// E4M3 byte of v >= 0, to nearest even, saturating at 448.
__device__ __forceinline__ uint32_t e4m3_byte(float v)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.0f), "f"(v));
    return d & 0xffu;
}

// Two E4M3 bytes (lo in bits 0-7) to floats; every E4M3 value is exact in f16.
__device__ __forceinline__ float2 e4m3x2_values(uint32_t two)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<__half2 *>(&h));
}

// Eight values to eight E2M1 codes (element 0 in the low nibble) / E4M3 bytes.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8])
{
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    return make_uint2((uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16));
}

// Largest magnitude of eight floats as a bit pattern (NaN above infinity
// above every finite value).
__device__ __forceinline__ uint32_t amax_bits8(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

constexpr uint32_t kInfBits = 0x7f800000u;
constexpr uint32_t kTop6 = 0x40c00000u, kTop448 = 0x43e00000u;

}  // namespace ops
}  // namespace beam
