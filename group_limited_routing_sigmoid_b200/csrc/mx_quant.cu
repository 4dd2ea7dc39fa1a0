// Microscaled operands (beam_mx_*): making them from 16- or 32-bit rows,
// reading them back, and laying their scales out for the tensor cores.
//
// Bound by HBM: a 16-bit element is 2 bytes in and 0.53 to 1.03 out.  A lane
// takes 16 consecutive elements of a row (a 32-byte load of 16-bit ones): an
// NVFP4 block is one lane's, a block of 32 two neighbouring lanes', whose
// largest magnitude meets in one shuffle.  Chunks of 16 are numbered through
// all rows, so short rows fill warps as well as long ones; where rows are
// contiguous and the scales lie row by row, the whole tensor is one row.  Two
// chunks a lane are loaded before either is worked on.  Quotients go two an
// instruction (fma.rn.f32x2), else NVFP4 is bound by issue.  Chunks are taken
// from the last to the first: what a kernel before this one touched last (the
// tensor scale's pass, the producer's stores) is still in L2.
//
// 20480 x 5120 bf16 on a B200: tensor scale 35 us (6.0 TB/s), NVFP4 46 us
// (5.8 TB/s; tiled scales 55 us), MXFP8 tiled 53 us (6.0 TB/s), NVFP4 back to
// bf16 45 to 48 us (5.6 to 6.0 TB/s).  Tiled scales of short rows cost more: at
// 64 elements an MX row's two scales are padded to four, so half of the chunks
// are padding (400000 x 64 MXFP4: 27 us tiled, 10.5 in rows).  With 8 elements a
// lane, one load ahead and scalar arithmetic tensor scale, NVFP4 and read-back
// took 195 us together, now 133.
#include "ops_common.cuh"

namespace beam {
namespace {

using namespace ops;

constexpr int kThreadsQ = 256;
constexpr int kChunk = 16;         // elements a lane takes at a time
constexpr int kAhead = 2;          // chunks a lane loads at once
constexpr int kCluster = 8;
constexpr long long kMostElements = 1ll << 60;   // sizes in bytes and chunks stay below 2^63
// Up to this many chunks one cluster finds the tensor scale, without the
// memset that atomics want before them (64 x 5120: 3.4 us, 4.4 us with it).
constexpr int kOneCluster = 32768;

// NVFP4 tensor scales outside this range would leave the exact range of the
// arithmetic below (block scale * tensor scale, its reciprocal, residuals).
constexpr float kMinTensorScale = 0x1p-112f, kMaxTensorScale = 0x1p112f;

// Chunk number -> row and chunk in the row.  Numbers stay below 2^31: larger
// tensors go in slices of rows (kSlice chunks, or a row where that has more).
constexpr long long kSlice = 1ll << 27;

struct Chunks {
    uint32_t magic;   // ceil(2^(31 + s) / per_row), s = ceil(log2 per_row)
    int shift;        // s - 1
    int total, per_row;
    Chunks() = default;
    Chunks(int rows, int per) : magic(0), shift(0), total(rows * per), per_row(per)
    {
        if (per <= 1) return;
        while ((1ll << (shift + 1)) < per) ++shift;
        magic = (uint32_t)(((1ull << (32 + shift)) + (unsigned long long)per - 1) / (unsigned long long)per);
    }
    template <int AL>
    __device__ __forceinline__ void at(int c, int &row, int &in_row) const
    {
        if constexpr (AL == 64) {   // kFlat
            row = 0, in_row = c;
        } else {
            row = per_row == 1 ? c : (int)(__umulhi((uint32_t)c, magic) >> shift);
            in_row = c - row * per_row;
        }
    }
};

struct QuantArgs {
    const void *x;
    const float *tensor_scale;
    uint8_t *codes, *scales;
    long long rows, ldx;    // rows of the tensor (or 1)
    long long K;            // elements a row
    long long row0;         // first row of this slice
    Chunks chunks;
    ScaleMap map;
};

// How chunks lie: kFlat, one row of 32-byte aligned chunks (no division, no
// row strides: 20480 x 5120 to NVFP4 52 us, 59 without), else the alignment
// known of every chunk in bytes (32, 16, or 0: the element's).
constexpr int kFlat = 64;

// Sixteen consecutive elements.
template <typename T> struct Raw16 { uint32_t w[4 * sizeof(T)]; };

template <int AL, typename T>
__device__ __forceinline__ Raw16<T> load_raw16(const T *p)
{
    Raw16<T> r;
    if constexpr (AL >= 32) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(r.w[8 * i]), "=r"(r.w[8 * i + 1]), "=r"(r.w[8 * i + 2]), "=r"(r.w[8 * i + 3]),
                           "=r"(r.w[8 * i + 4]), "=r"(r.w[8 * i + 5]), "=r"(r.w[8 * i + 6]), "=r"(r.w[8 * i + 7])
                         : "l"(reinterpret_cast<const uint32_t *>(p) + 8 * i));
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const Raw8<T> v = load_raw8<AL == 16>(p + 8 * h);
#pragma unroll
            for (int i = 0; i < (int)(2 * sizeof(T)); ++i) r.w[h * 2 * sizeof(T) + i] = v.w[i];
        }
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void unpack16(const Raw16<T> &r, float (&v)[16])
{
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        Raw8<T> q;
#pragma unroll
        for (int i = 0; i < (int)(2 * sizeof(T)); ++i) q.w[i] = r.w[h * 2 * sizeof(T) + i];
        float f[8];
        unpack8(q, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * h + i] = f[i];
    }
}

// Largest magnitude of the chunk as the bits of a float (NaN above infinity
// above every finite value).  16-bit types are compared in pairs, in their own
// bits: their order is that of the floats.
template <typename T>
__device__ __forceinline__ uint32_t amax_bits16(const Raw16<T> &r)
{
    uint32_t m = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, r.w[i] & 0x7fffffffu);
        return m;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, r.w[i] & 0x7fff7fffu);
        m = max(m & 0xffffu, m >> 16);
        if constexpr (std::is_same<T, __nv_bfloat16>::value) return m << 16;
        return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
    }
}

template <int AL, typename T>
__device__ __forceinline__ void store16(T *p, const float (&v)[16])
{
    if constexpr (AL >= 32) {
        uint32_t w[4 * sizeof(T)];
#pragma unroll
        for (int i = 0; i < (int)(4 * sizeof(T)); ++i) {
            if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
            else if constexpr (std::is_same<T, __nv_bfloat16>::value) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
            else w[i] = pack_f16x2(v[2 * i], v[2 * i + 1]);
        }
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             reinterpret_cast<uint32_t *>(p) + 8 * i),
                         "r"(w[8 * i]), "r"(w[8 * i + 1]), "r"(w[8 * i + 2]), "r"(w[8 * i + 3]), "r"(w[8 * i + 4]),
                         "r"(w[8 * i + 5]), "r"(w[8 * i + 6]), "r"(w[8 * i + 7])
                         : "memory");
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = v[8 * h + i];
            store8<AL == 16>(p + 8 * h, f);
        }
    }
}

__device__ __forceinline__ const float (&half_of(const float (&v)[16], int h))[8]
{
    return *reinterpret_cast<const float(*)[8]>(v + 8 * h);
}

// Two FP32 operations an instruction.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ void scale16(float (&v)[16], float s)
{
    const uint64_t ss = pair(s, s);
#pragma unroll
    for (int i = 0; i < 16; i += 2) unpair(mul2(pair(v[i], v[i + 1]), ss), v[i], v[i + 1]);
}

// x / d correctly rounded, from r = 1/d rounded: one step of Markstein's
// residual correction (IBM J. Res. Dev. 34, 1990).  Ties of the 4-bit grid
// are exact quotients and stay exact.
__device__ __forceinline__ float quotient(float x, float d, float r)
{
    const float q = x * r;
    return fmaf(fmaf(-q, d, x), r, q);
}

// The same for sixteen.
__device__ __forceinline__ void quotient16(float (&v)[16], float d, float r)
{
    const uint64_t rr = pair(r, r), nd = pair(-d, -d);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const uint64_t x = pair(v[i], v[i + 1]), q = mul2(x, rr);
        unpair(fma2(fma2(q, nd, x), rr, q), v[i], v[i + 1]);
    }
}

// One chunk of a row, at element k.  `live`: the elements exist; otherwise
// only a scale byte past the end may have to be zeroed.  Whole warps call it.
template <typename T, int FMT, int AL>
__device__ __forceinline__ void quantize_chunk(const QuantArgs &p, const Raw16<T> &raw, long long row, long long k,
                                               bool live, float g, float r6)
{
    uint32_t m = amax_bits16(raw);
    if constexpr (FMT != BEAM_NVFP4) m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    float v[16];
    unpack16(raw, v);
    const bool bad = m >= kInfBits || (FMT == BEAM_NVFP4 && !(g >= kMinTensorScale && g <= kMaxTensorScale));
    uint32_t sb;
    if constexpr (FMT == BEAM_NVFP4) {
        // amax / (6 g), correctly rounded where it is below the largest scale
        float q = __uint_as_float(m) * r6;
        if (q < 512.f) q = quotient(__uint_as_float(m), 6.0f * g, r6);
        sb = bad ? 0x7fu : e4m3_byte(q);
        const float d = e4m3x2_values(sb).x * g;
        const float r = 1.0f / d;
        if (bad || sb == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0.f;
        } else if (!(__uint_as_float(m) * r < 8.0f)) {
            // the scale saturated (a tensor scale found on other data): large
            // quotients only have to stay large, and may be infinite
            scale16(v, r);
        } else {
            quotient16(v, d, r);
        }
    } else {
        constexpr uint32_t TOP = FMT == BEAM_MXFP4 ? kTop6 : kTop448;
        sb = bad ? 0xffu : ue8m0_byte<TOP>(__uint_as_float(m));
        if (bad) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0.f;
        } else {
            scale16(v, ue8m0_inverse(sb));
        }
    }
    const long long j = k / block_size(FMT);
    const bool first = FMT == BEAM_NVFP4 || (k & 16) == 0;
    if (live) {
        const size_t at = AL == kFlat ? (size_t)k : (size_t)row * p.K + k;
        if constexpr (FMT == BEAM_MXFP8) {
            const uint2 a = e4m3x8(half_of(v, 0)), b = e4m3x8(half_of(v, 1));
            *reinterpret_cast<uint4 *>(p.codes + at) = make_uint4(a.x, a.y, b.x, b.y);
        } else {
            *reinterpret_cast<uint2 *>(p.codes + at / 2) = make_uint2(e2m1x8(half_of(v, 0)), e2m1x8(half_of(v, 1)));
        }
        if (first) p.scales[AL == kFlat ? (size_t)j : p.map.at(row, j)] = (uint8_t)sb;
    } else if (AL != kFlat && first && p.map.tiled && j < 4 * p.map.n4) {
        p.scales[p.map.at(row, j)] = 0;
    }
}

template <typename T, int FMT, int AL>
__global__ void __launch_bounds__(kThreadsQ) mx_quantize_kernel(const QuantArgs p)
{
    pdl_launch_dependents();
    pdl_wait();
    const float g = FMT == BEAM_NVFP4 ? *p.tensor_scale : 1.0f;
    const float r6 = 1.0f / (6.0f * g);
    const T *x = static_cast<const T *>(p.x);
    const int step = (int)gridDim.x * kThreadsQ, total = p.chunks.total;
    // whole warps stay together: lanes past the end have nothing live
    const int lane = threadIdx.x & 31;
    for (int c0 = (int)blockIdx.x * kThreadsQ + (int)threadIdx.x; c0 - lane < total; c0 += kAhead * step) {
        Raw16<T> raw[kAhead];
        long long row[kAhead], k[kAhead];
        bool live[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int c = total - 1 - (c0 + i * step);
            raw[i] = Raw16<T>{};
            if (c >= 0) {
                int r, in_row;
                p.chunks.at<AL>(c, r, in_row);
                row[i] = p.row0 + r;
                k[i] = (long long)in_row * kChunk;
                live[i] = AL == kFlat || (row[i] < p.rows && k[i] < p.K);
                if (live[i]) raw[i] = load_raw16<AL>(x + (AL == kFlat ? 0 : row[i] * p.ldx) + k[i]);
            } else {   // nothing to write: past the end of the last tile's scales
                row[i] = 0, k[i] = (long long)4 * p.map.n4 * block_size(FMT) + 16, live[i] = false;
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (c0 - lane + i * step < total)
                quantize_chunk<T, FMT, AL>(p, raw[i], row[i], k[i], live[i], g, r6);
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

// ONE: the grid is one cluster, which joins its blocks' maxima itself; else out
// holds zero beforehand and takes them by atomics.  The scale is `most` at most.
template <typename T, bool ONE, int AL>
__global__ void __launch_bounds__(kThreadsQ) mx_amax_kernel(const QuantArgs p, float *out, const float most)
{
    constexpr int AHEAD = sizeof(T) == 4 ? 2 : 4;
    // every block of the cluster has started before one writes into another's
    // shared memory (waited for below, when the data has been read)
    if constexpr (ONE) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    pdl_launch_dependents();
    pdl_wait();
    const T *x = static_cast<const T *>(p.x);
    const int step = (int)gridDim.x * kThreadsQ, total = p.chunks.total;
    uint32_t m = 0;
    for (int c0 = (int)blockIdx.x * kThreadsQ + (int)threadIdx.x; c0 < total; c0 += AHEAD * step) {
        Raw16<T> raw[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            raw[i] = Raw16<T>{};
            const int c = c0 + i * step;
            if (c < total) {
                int row, in_row;
                p.chunks.at<AL>(c, row, in_row);
                const long long k = (long long)in_row * kChunk;
                const T *at = x + (AL == kFlat ? 0 : (p.row0 + row) * p.ldx) + k;
                if (k + kChunk <= p.K) {
                    raw[i] = load_raw16<AL>(at);
                } else {
                    for (int e = 0; k + e < p.K; ++e) {
                        const uint32_t b = __float_as_uint(to_f32(at[e])) & 0x7fffffffu;
                        m = max(m, b >= kInfBits ? 0u : b);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const uint32_t b = amax_bits16(raw[i]);
            if (b < kInfBits) {
                m = max(m, b);
            } else {   // the finite ones among infinities and NaN
                float v[16];
                unpack16(raw[i], v);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t f = __float_as_uint(v[e]) & 0x7fffffffu;
                    m = max(m, f >= kInfBits ? 0u : f);
                }
            }
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    __shared__ uint32_t part[kThreadsQ / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < kThreadsQ / 32; ++i) m = max(m, part[i]);
        if constexpr (!ONE) atomicMax(reinterpret_cast<int *>(out), __float_as_int(fminf(tensor_scale_of(m), most)));
    }
    if constexpr (ONE) {
        __shared__ uint32_t all[kCluster];
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (threadIdx.x == 0)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&all[cluster_ctarank()]), 0)), "r"(m)
                         : "memory");
        __syncwarp();
        cluster_sync();
        if (threadIdx.x == 0 && cluster_ctarank() == 0) {
#pragma unroll
            for (int i = 0; i < kCluster; ++i) m = max(m, all[i]);
            *out = fminf(tensor_scale_of(m), most);
        }
    }
}

struct DequantArgs {
    const uint8_t *codes, *scales;
    const float *tensor_scale;
    void *out;
    long long ldo, K, row0;
    Chunks chunks;
    ScaleMap map;
};

template <typename T, int FMT, int AL>
__global__ void __launch_bounds__(kThreadsQ) mx_dequantize_kernel(const DequantArgs p)
{
    pdl_launch_dependents();
    pdl_wait();
    const float g = p.tensor_scale ? *p.tensor_scale : 1.0f;
    const int step = (int)gridDim.x * kThreadsQ, total = p.chunks.total;
    for (int c0 = (int)blockIdx.x * kThreadsQ + (int)threadIdx.x; c0 < total; c0 += kAhead * step) {
        uint4 codes[kAhead];
        uint32_t sb[kAhead];
        long long row[kAhead], k[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int c = c0 + i * step;
            codes[i] = make_uint4(0u, 0u, 0u, 0u), sb[i] = 0u, row[i] = 0, k[i] = 0;
            if (c < total) {
                int r, in_row;
                p.chunks.at<AL>(c, r, in_row);
                row[i] = p.row0 + r;
                k[i] = (long long)in_row * kChunk;
                const size_t at = AL == kFlat ? (size_t)k[i] : (size_t)row[i] * p.K + k[i];
                if constexpr (FMT == BEAM_MXFP8) {
                    codes[i] = *reinterpret_cast<const uint4 *>(p.codes + at);
                } else {
                    const uint2 q = *reinterpret_cast<const uint2 *>(p.codes + at / 2);
                    codes[i].x = q.x, codes[i].y = q.y;
                }
                const long long j = k[i] / block_size(FMT);
                sb[i] = p.scales[AL == kFlat ? (size_t)j : p.map.at(row[i], j)];
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (c0 + i * step >= total) break;
            const float s = FMT == BEAM_NVFP4 ? e4m3x2_values(sb[i]).x : ue8m0_value(sb[i]);
            float v[16];
            if constexpr (FMT == BEAM_MXFP8) {
                const uint32_t w[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 f = e4m3x2_values(w[e / 2] >> (16 * (e & 1)) & 0xffffu);
                    v[2 * e] = f.x, v[2 * e + 1] = f.y;
                }
            } else {
                const uint32_t w[2] = {codes[i].x, codes[i].y};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t h[4];
                    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
                        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
                        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
                        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
                        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
                        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
                        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
                        : "r"(w[q]));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
                        v[8 * q + 2 * e] = f.x, v[8 * q + 2 * e + 1] = f.y;
                    }
                }
            }
            // element * block scale first: exact in FP32 (it may only leave the
            // normal range for power-of-two scales next to 2^-127), then the
            // tensor scale, rounded once
            scale16(v, s);
            if (p.tensor_scale) scale16(v, g);
            store16<AL>(static_cast<T *>(p.out) + (AL == kFlat ? 0 : row[i] * p.ldo) + k[i], v);
        }
    }
}

// Scales from rows to tiles: a thread per 4-byte group of a tile row.  Run once
// for a checkpoint: 20480 x 5120 NVFP4 12.5 us for 13.1 MB in and out, MXFP4 7.6
// us for 6.6 MB (1 TB/s: single-byte loads, 4-byte stores 16 bytes apart).
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

// Blocks for `n` threads' work, at most `per_sm` an SM: 8, or 16 where the
// stores are most of the traffic (reading back 20480 x 5120 NVFP4: 44 us, 50 with 8).
int grid_for(long long n, int per_sm = 8)
{
    const long long need = (n + kThreadsQ - 1) / kThreadsQ;
    const long long most = (long long)sm_count() * per_sm;
    return (int)(need < most ? need : most);
}

// How the chunks of a matrix lie.
int chunk_alignment(const void *p, bool flat, long long ld, int dtype)
{
    if (flat && aligned(p, 32)) return kFlat;
    const long long pitch = (flat ? 32 : ld) * dtype_size(dtype);
    return aligned(p, 32) && pitch % 32 == 0 ? 32 : aligned(p, 16) && pitch % 16 == 0 ? 16 : 0;
}

#define BEAM_ALIGNED(kernel, T, ...)                                    \
    (al == kFlat ? launch_pdl(kernel<T, ##__VA_ARGS__, kFlat>, grid, dim3(kThreadsQ), 0, s, BEAM_ARGS) \
     : al == 32 ? launch_pdl(kernel<T, ##__VA_ARGS__, 32>, grid, dim3(kThreadsQ), 0, s, BEAM_ARGS) \
     : al == 16 ? launch_pdl(kernel<T, ##__VA_ARGS__, 16>, grid, dim3(kThreadsQ), 0, s, BEAM_ARGS) \
                : launch_pdl(kernel<T, ##__VA_ARGS__, 0>, grid, dim3(kThreadsQ), 0, s, BEAM_ARGS))
#define BEAM_TYPED(kernel, ...)                                         \
    (dtype == BEAM_BF16 ? BEAM_ALIGNED(kernel, __nv_bfloat16, ##__VA_ARGS__) \
     : dtype == BEAM_F16 ? BEAM_ALIGNED(kernel, __half, ##__VA_ARGS__)  \
                         : BEAM_ALIGNED(kernel, float, ##__VA_ARGS__))

template <int FMT>
cudaError_t launch_quantize(const QuantArgs &a, int dtype, int al, cudaStream_t s)
{
    const dim3 grid(grid_for(a.chunks.total));
#define BEAM_ARGS a
    return BEAM_TYPED(mx_quantize_kernel, FMT);
#undef BEAM_ARGS
}

template <int FMT>
cudaError_t launch_dequantize(const DequantArgs &a, int dtype, int al, cudaStream_t s)
{
    const dim3 grid(grid_for(a.chunks.total, 16));
#define BEAM_ARGS a
    return BEAM_TYPED(mx_dequantize_kernel, FMT);
#undef BEAM_ARGS
}

cudaError_t launch_amax(const QuantArgs &a, int dtype, int al, float *out, float most, cudaStream_t s)
{
    const dim3 grid(grid_for(a.chunks.total));
#define BEAM_ARGS a, out, most
    return BEAM_TYPED(mx_amax_kernel, false);
#undef BEAM_ARGS
}

// The same on one cluster.
template <typename... K, typename... Args>
cudaError_t launch_cluster(void (*kernel)(K...), cudaStream_t s, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreadsQ);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {kCluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<K>(args)...);
}

template <typename T>
cudaError_t launch_amax_one(const QuantArgs &a, int al, float *out, float most, cudaStream_t s)
{
    if (al == kFlat) return launch_cluster(mx_amax_kernel<T, true, kFlat>, s, a, out, most);
    if (al == 32) return launch_cluster(mx_amax_kernel<T, true, 32>, s, a, out, most);
    if (al == 16) return launch_cluster(mx_amax_kernel<T, true, 16>, s, a, out, most);
    return launch_cluster(mx_amax_kernel<T, true, 0>, s, a, out, most);
}

// launch(a) over slices of rows of `per` chunks each (rows == 1: over chunks;
// `step` advances a's pointers by that many then).
template <typename Args, typename Step, typename Launch>
cudaError_t in_slices(Args a, long long rows, long long per, Step step, Launch launch)
{
    if (rows == 1) {
        for (long long done = 0; done < per; done += kSlice) {
            Args part = a;
            step(part, done);
            part.chunks = Chunks(1, (int)(per - done < kSlice ? per - done : kSlice));
            if (cudaError_t e = launch(part)) return e;
        }
        return cudaSuccess;
    }
    const long long most = per < kSlice ? kSlice / per : 1;
    for (a.row0 = 0; a.row0 < rows; a.row0 += most) {
        a.chunks = Chunks((int)(rows - a.row0 < most ? rows - a.row0 : most), (int)per);
        if (cudaError_t e = launch(a)) return e;
    }
    return cudaSuccess;
}

int check_shape(int format, long long rows, int K, int layout)
{
    if (!format_ok(format)) return fail(BEAM_ERR_INVALID_ARG, "format %d", format);
    if (!layout_ok(layout)) return fail(BEAM_ERR_INVALID_ARG, "layout %d", layout);
    if (rows < 0 || rows > (1LL << 40)) return fail(BEAM_ERR_INVALID_ARG, "rows %lld", rows);
    if (K <= 0 || K % block_of(format) != 0)
        return fail(BEAM_ERR_INVALID_ARG, "K must be a positive multiple of %d, got %d", block_of(format), K);
    if (rows > kMostElements / K) return fail(BEAM_ERR_INVALID_ARG, "%lld x %d elements are too many", rows, K);
    return BEAM_OK;
}

// What the arguments of a tensor scale have to hold.
int check_scale(const void *x, int dtype, long long rows, int K, long long ldx, const float *tensor_scale)
{
    if (rows < 0 || rows > (1LL << 40) || K < 1) return fail(BEAM_ERR_INVALID_ARG, "rows must be >= 0 and K >= 1");
    if (rows > kMostElements / K) return fail(BEAM_ERR_INVALID_ARG, "%lld x %d elements are too many", rows, K);
    if (!dtype_ok(dtype)) return fail(BEAM_ERR_INVALID_ARG, "dtype %d", dtype);
    if (!tensor_scale || !aligned(tensor_scale, 4)) return fail(BEAM_ERR_INVALID_ARG, "tensor_scale is NULL or not aligned");
    if (rows > 0 && (!x || !aligned(x, dtype_size(dtype)))) return fail(BEAM_ERR_INVALID_ARG, "x is NULL or not aligned");
    if (rows > 0 && ldx < K) return fail(BEAM_ERR_INVALID_ARG, "ldx is below K");
    return BEAM_OK;
}

int find_scale(cudaStream_t s, const void *x, int dtype, long long rows, int K, long long ldx, float *tensor_scale, float most)
{
    if (!sm_count()) return fail(BEAM_ERR_CUDA, "no CUDA device");
    const bool flat = rows == 1 || ldx == K;
    QuantArgs a{x, nullptr, nullptr, nullptr, rows, ldx, K, 0, Chunks(0, 1), ScaleMap(0, 1)};
    const int al = chunk_alignment(x, flat, ldx, dtype);
    if (flat) a.rows = 1, a.K = rows * (long long)K;
    const long long per = (a.K + kChunk - 1) / kChunk;
    if (a.rows * per <= kOneCluster) {
        if (a.rows > 0) a.chunks = Chunks((int)a.rows, (int)per);
        const cudaError_t one = dtype == BEAM_BF16  ? launch_amax_one<__nv_bfloat16>(a, al, tensor_scale, most, s)
                                : dtype == BEAM_F16 ? launch_amax_one<__half>(a, al, tensor_scale, most, s)
                                                    : launch_amax_one<float>(a, al, tensor_scale, most, s);
        return check_cuda(one, "beam_mx_tensor_scale");
    }
    if (int rc = check_cuda(cudaMemsetAsync(tensor_scale, 0, sizeof(float), s), "cudaMemsetAsync")) return rc;
    const auto launch = [&](const QuantArgs &part) { return launch_amax(part, dtype, al, tensor_scale, most, s); };
    const cudaError_t e = in_slices(a, a.rows, per, [&](QuantArgs &part, long long c) {
        part.x = static_cast<const uint8_t *>(x) + c * kChunk * dtype_size(dtype);
        part.K -= c * kChunk;
    }, launch);
    return check_cuda(e, "beam_mx_tensor_scale");
}

// What the arguments of a quantisation of one row and more have to hold.
int check_quantize(const void *x, int dtype, int K, long long ldx, int format, const float *tensor_scale, const uint8_t *codes,
                   const uint8_t *scales)
{
    if (!x || !codes || !scales) return fail(BEAM_ERR_INVALID_ARG, "x, codes and scales are required");
    if ((format == BEAM_NVFP4) != (tensor_scale != nullptr))
        return fail(BEAM_ERR_INVALID_ARG, "tensor_scale is required for NVFP4 and must be NULL for the others");
    if (ldx < K) return fail(BEAM_ERR_INVALID_ARG, "ldx is below K");
    if (!aligned(x, dtype_size(dtype)) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(tensor_scale, 4))
        return fail(BEAM_ERR_INVALID_ARG, "a pointer is not aligned");
    return BEAM_OK;
}

cudaError_t quantize(cudaStream_t s, const void *x, int dtype, long long rows, int K, long long ldx, int format, int layout,
                     const float *tensor_scale, uint8_t *codes, uint8_t *scales)
{
    const int n = K / block_of(format);
    const bool flat = layout == BEAM_SCALES_ROWS && (rows == 1 || ldx == K);
    QuantArgs a{x, tensor_scale, codes, scales, rows, ldx, K, 0, Chunks(), ScaleMap(layout, n)};
    const int al = chunk_alignment(x, flat, ldx, dtype);
    const auto launch = [&](const QuantArgs &part) {
        return format == BEAM_NVFP4   ? launch_quantize<BEAM_NVFP4>(part, dtype, al, s)
               : format == BEAM_MXFP4 ? launch_quantize<BEAM_MXFP4>(part, dtype, al, s)
                                      : launch_quantize<BEAM_MXFP8>(part, dtype, al, s);
    };
    // tiled: the chunks cover the tiles' padding rows and scales too
    const bool tiled = layout == BEAM_SCALES_TILED;
    if (flat) a.rows = 1, a.K = rows * (long long)K;
    const long long all = flat ? 1 : tiled ? (rows + 127) / 128 * 128 : rows;
    const long long per = tiled ? (long long)a.map.n4 * 4 * block_of(format) / kChunk : a.K / kChunk;
    return in_slices(a, all, per, [&](QuantArgs &part, long long c) {
        part.x = static_cast<const uint8_t *>(x) + c * kChunk * dtype_size(dtype);
        part.codes = codes + (format == BEAM_MXFP8 ? c * kChunk : c * kChunk / 2);
        part.scales = scales + c * kChunk / block_of(format);
        part.K -= c * kChunk;
    }, launch);
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
    if (int rc = check_scale(x, dtype, rows, K, ldx, tensor_scale)) return rc;
    return find_scale(static_cast<cudaStream_t>(stream), x, dtype, rows, K, ldx, tensor_scale, INFINITY);
}

int beam_mx_quantize(void *stream, const void *x, int dtype, long long rows, int K, long long ldx,
                     int format, int layout, const float *tensor_scale, uint8_t *codes, uint8_t *scales)
{
    using namespace beam;
    using namespace beam::ops;
    if (int rc = check_shape(format, rows, K, layout)) return rc;
    if (!dtype_ok(dtype)) return fail(BEAM_ERR_INVALID_ARG, "dtype %d", dtype);
    if (rows == 0) return BEAM_OK;
    if (int rc = check_quantize(x, dtype, K, ldx, format, tensor_scale, codes, scales)) return rc;
    if (!sm_count()) return fail(BEAM_ERR_CUDA, "no CUDA device");
    return check_cuda(quantize(static_cast<cudaStream_t>(stream), x, dtype, rows, K, ldx, format, layout, tensor_scale, codes, scales),
                      "beam_mx_quantize");
}

int beam_mx_quantize_nvfp4(void *stream, const void *x, int dtype, long long rows, int K, long long ldx, int layout,
                           float *tensor_scale, uint8_t *codes, uint8_t *scales)
{
    using namespace beam;
    using namespace beam::ops;
    if (int rc = check_shape(BEAM_NVFP4, rows, K, layout)) return rc;
    if (int rc = check_scale(x, dtype, rows, K, ldx, tensor_scale)) return rc;
    if (rows > 0)
        if (int rc = check_quantize(x, dtype, K, ldx, BEAM_NVFP4, tensor_scale, codes, scales)) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // at most what quantize_chunk's arithmetic takes: larger values saturate
    if (int rc = find_scale(s, x, dtype, rows, K, ldx, tensor_scale, kMaxTensorScale)) return rc;
    if (rows == 0) return BEAM_OK;
    return check_cuda(quantize(s, x, dtype, rows, K, ldx, BEAM_NVFP4, layout, tensor_scale, codes, scales), "beam_mx_quantize_nvfp4");
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
    DequantArgs a{codes, scales, tensor_scale, out, ldo, K, 0, Chunks(), ScaleMap(layout, K / block_of(format))};
    const int al = chunk_alignment(out, flat, ldo, dtype);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const auto launch = [&](const DequantArgs &part) {
        return format == BEAM_NVFP4   ? launch_dequantize<BEAM_NVFP4>(part, dtype, al, s)
               : format == BEAM_MXFP4 ? launch_dequantize<BEAM_MXFP4>(part, dtype, al, s)
                                      : launch_dequantize<BEAM_MXFP8>(part, dtype, al, s);
    };
    if (flat) a.K = rows * (long long)K;
    const cudaError_t e = in_slices(a, flat ? 1 : rows, a.K / kChunk, [&](DequantArgs &part, long long c) {
        part.codes = codes + (format == BEAM_MXFP8 ? c * kChunk : c * kChunk / 2);
        part.scales = scales + c * kChunk / block_of(format);
        part.out = static_cast<uint8_t *>(out) + c * kChunk * dtype_size(dtype);
        part.K -= c * kChunk;
    }, launch);
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
    return check_cuda(launch_pdl(mx_tile_scales_kernel, dim3(grid_for(groups)), dim3(256), 0,
                                 static_cast<cudaStream_t>(stream), scales, tiled, rows, map, groups),
                      "beam_mx_tile_scales");
}

}  // extern "C"
