// Shared pieces of the microscaled product's kernels (mx_matmul.cu: one CTA a
// tile; mx_matmul_pair.cu: a CTA pair a tile).
#pragma once

#include "mx_plan.h"
#include "ops_common.cuh"

namespace beam {
namespace mx {

using namespace ops;

constexpr int kRowBytes = 128;            // bytes of a row in a stage
constexpr int kEpiWarps = 8;
constexpr int kCopyWarp = 2 + kEpiWarps;
constexpr int kThreads = 32 * (kCopyWarp + 1);
constexpr long long kWaitLimitNs = 2000000000ll;
constexpr uint32_t kWithheldBytes = 16;

// 512-byte scale tiles (128 rows x 4 scales) per stage and 128 rows.
constexpr int tiles_per_stage(int kind) { return kind == kNv ? 4 : kind == kMx4 ? 2 : 1; }
// K elements of a stage and of one MMA.
constexpr int stage_k(int kind) { return kind == kMx8 ? 128 : 256; }
constexpr int step_k(int kind) { return kind == kMx8 ? 32 : 64; }

struct Maps {
    CUtensorMap p, q;      // codes of the A and B side: boxes of 128 bytes x rows
    CUtensorMap sp, sq;    // their scale tiles: [128-row blocks][tiles along K][512 bytes]
};

struct MatmulArgs {
    const float *ga, *gw;
    void *out;
    long long ldo;
    int *status;
    int P, Q;              // rows of the A and B side
    int p_tiles, q_tiles;
    int nst;               // stages of K
    int ksteps;            // MMA K steps in all
    int split;             // CTAs that share a tile's K steps (the cluster)
    int single;            // 1: every CTA has one tile (or its share of one)
    int swap;              // 1: the A side holds the weights
    int dtype;
    int vec;               // 1: rows of out start on 16-byte boundaries
    uint32_t idesc;
    uint32_t tx;           // bytes one CTA's copies of a stage complete
    int withheld;          // the stage of K that waits for more than that (beam_ops_debug_withhold), or -1
    long long limit_ns;    // of a wait
};

cudaError_t launch_pair(int kind, const Maps &m, const MatmulArgs &a, int sms, cudaStream_t s);

// Byte offset of a stage's scale tiles and the tensor-memory columns they
// take, for `nqb` 128-row blocks of the B side.
constexpr int scale_bytes(int kind, int nqb) { return tiles_per_stage(kind) * 512 * (1 + nqb); }
constexpr int scale_cols(int kind, int nqb) { return tiles_per_stage(kind) * 4 * (1 + nqb); }

// 3-D tile load of scale tiles: box {512 bytes, tiles of a stage, blocks}.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int32_t y, int32_t z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(bar) : "memory");
}

// The same for a CTA pair: the barrier (a shared::cluster address) may be the other CTA's.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, int32_t y, int32_t z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(z), "r"(bar) : "memory");
}

// tcgen05.cp of one 512-byte scale tile: 32 rows of 16 bytes to lanes 0-31,
// four columns, replicated to the other three lane quadrants; for a pair, in
// either CTA from its own shared memory.
template <int CTAS>
__device__ __forceinline__ void scale_copy(uint32_t taddr, uint32_t smem)
{
    // no swizzle, 8 x 16-byte core matrices 128 bytes apart
    const uint64_t d = (uint64_t)((smem >> 4) & 0x3FFFu) | ((uint64_t)8u << 16) | ((uint64_t)8u << 32) |
                       ((uint64_t)1u << 46);
    if constexpr (CTAS == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

#define BEAM_MMA_SCALED(group, kind)                                                                        \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                          \
                 "tcgen05.mma.cta_group::" group "." kind " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),  \
                 "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                             \
                 : "memory")

template <int KIND, int CTAS>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                           uint32_t sfb, uint32_t accumulate)
{
    if constexpr (CTAS == 1) {
        if constexpr (KIND == kNv) BEAM_MMA_SCALED("1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
        else if constexpr (KIND == kMx4) BEAM_MMA_SCALED("1", "kind::mxf4.block_scale.scale_vec::2X");
        else BEAM_MMA_SCALED("1", "kind::mxf8f6f4.block_scale.scale_vec::1X");
    } else {
        if constexpr (KIND == kNv) BEAM_MMA_SCALED("2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
        else if constexpr (KIND == kMx4) BEAM_MMA_SCALED("2", "kind::mxf4.block_scale.scale_vec::2X");
        else BEAM_MMA_SCALED("2", "kind::mxf8f6f4.block_scale.scale_vec::1X");
    }
}
#undef BEAM_MMA_SCALED

// A stage's scale tiles (at sf in shared memory) to its columns tsf.
template <int KIND, int CTAS, int NQB>
__device__ __forceinline__ void copy_scales(uint32_t sf, uint32_t tsf)
{
    constexpr int CPS = tiles_per_stage(KIND);
    const uint32_t tsfq = tsf + CPS * 4;
#pragma unroll
    for (int c = 0; c < CPS; ++c) {
        scale_copy<CTAS>(tsf + c * 4, sf + c * 512);
#pragma unroll
        for (int b = 0; b < NQB; ++b) scale_copy<CTAS>(tsfq + (c * NQB + b) * 4, sf + (CPS * (1 + b) + c) * 512);
    }
}

// The first column, within its 128-row block's four, of the scales of a B tile
// that starts at `row`, a multiple of 64: 32 rows' scales are one column.  (An
// odd column -- a tile at an odd multiple of 32 rows -- is no scale address
// that the MMA takes.)
__device__ __forceinline__ uint32_t scale_column(int row) { return (uint32_t)(row >> 5) & 2u; }

// A stage's MMAs.  sp, sq: its codes in shared memory; tsf: its scales'
// columns; qcol: scale_column of the B tile.
template <int KIND, int CTAS, int NQB>
__device__ __forceinline__ void mma_stage(uint32_t d, uint32_t sp, uint32_t sq, uint32_t tsf, uint32_t qcol, uint32_t idesc,
                                          int steps, bool first)
{
    const uint32_t tsfq = tsf + tiles_per_stage(KIND) * 4 + qcol;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j < steps) {
            const int c = KIND == kNv ? j : KIND == kMx4 ? j / 2 : 0;
            const uint32_t id = KIND == kNv ? 0u : KIND == kMx4 ? (uint32_t)(j & 1) * 2u : (uint32_t)j;
            mma_scaled<KIND, CTAS>(d, umma_desc_sw128(sp + j * 32), umma_desc_sw128(sq + j * 32),
                                   idesc | (id << 4) | (id << 29), tsf + c * 4, tsfq + c * NQB * 4,
                                   (!first || j > 0) ? 1u : 0u);
        }
    }
}

__device__ __forceinline__ void put(void *out, int dtype, size_t at, float v)
{
    if (dtype == BEAM_BF16) static_cast<__nv_bfloat16 *>(out)[at] = __float2bfloat16_rn(v);
    else if (dtype == BEAM_F16) static_cast<__half *>(out)[at] = __float2half_rn(v);
    else static_cast<float *>(out)[at] = v;
}

// A warp's 32 rows x 32 columns of results (lane: row; v: its columns, scaled)
// to rows row0 .. of out at column col, through the warp's 4 KB block of
// shared memory so that a row's columns leave together: 16-byte units of a row
// at their index xor the row's low bits, no bank met twice.
//   elements of 2 bytes fill half a 128-byte line a row: `half_line` 0 or 1,
//   and `flush` writes both halves (64 columns) out; 4 bytes: one line.
__device__ __forceinline__ void stage_columns(const float (&v)[32], uint8_t *stg, int lane, int dtype, int half_line)
{
    uint4 *line = reinterpret_cast<uint4 *>(stg + lane * 128);
    if (dtype == BEAM_F32) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            line[u ^ (lane & 7)] = make_uint4(__float_as_uint(v[4 * u]), __float_as_uint(v[4 * u + 1]),
                                              __float_as_uint(v[4 * u + 2]), __float_as_uint(v[4 * u + 3]));
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float *f = v + 8 * u;
            line[(half_line * 4 + u) ^ (lane & 7)] =
                dtype == BEAM_BF16
                    ? make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]))
                    : make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]), pack_f16x2(f[6], f[7]));
        }
    }
}

// Write the staged lines out: `rows` rows of `cols` columns (at most a line)
// from out[at], rows ldo apart.  vec: every row starts on 16 bytes.  Rows that
// do not are stored as the aligned 16-byte units they cover, each from the two
// staged units that hold it, and their ends element by element (2-byte stores
// of whole lines took 13 of 29 us of 1021 x 5123 x 2560).
template <int ES>
__device__ __forceinline__ void flush_row(const uint8_t *line, int row, int u, uint8_t *o, int cols)
{
    constexpr int PER = 16 / ES;
    const auto unit = [&](int i) { return *reinterpret_cast<const uint4 *>(line + ((i ^ (row & 7)) * 16)); };
    const auto value = [&](int c) -> uint32_t {
        const uint8_t *s = line + (((c / PER) ^ (row & 7)) * 16) + c % PER * ES;
        if constexpr (ES == 4) return *reinterpret_cast<const uint32_t *>(s);
        else return *reinterpret_cast<const uint16_t *>(s);
    };
    const auto store = [&](int c, uint32_t v) {
        if constexpr (ES == 4) *reinterpret_cast<uint32_t *>(o + c * 4) = v;
        else *reinterpret_cast<uint16_t *>(o + c * 2) = (uint16_t)v;
    };
    const int off = (int)(reinterpret_cast<uintptr_t>(o) & 15u);
    if (off == 0) {
        if ((u + 1) * PER <= cols) *reinterpret_cast<uint4 *>(o + u * 16) = unit(u);
        else
            for (int c = u * PER; c < cols; ++c) store(c, value(c));
        return;
    }
    // unit u of memory: bytes 16 u - off and on of the line; its ends, before
    // the first and past the last whole unit, element by element.  All reads
    // first, so that the rows of an unrolled loop overlap.
    const int head = (16 - off) / ES;                 // elements before the first whole unit
    const int tail = cols <= head ? cols : head + (cols - head) / PER * PER;
    const uint4 a = unit(u > 0 ? u - 1 : 0), b = unit(u);
    const int t = min(tail + u, 8 * PER - 1);
    const uint32_t first = value(u), last = value(t);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const int s = 16 - off;
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = s & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = s & 4 ? w[i + 1] : w[i];
    if constexpr (ES == 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = s & 2 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
    if (u > 0 && head + u * PER <= cols) *reinterpret_cast<uint4 *>(o + u * 16 - off) = make_uint4(w[0], w[1], w[2], w[3]);
    if (u < head && u < cols) store(u, first);
    if (tail + u < cols) store(tail + u, last);
}

__device__ __forceinline__ void flush_lines(const uint8_t *stg, int lane, int dtype, void *out, size_t at, long long ldo,
                                            int rows, int cols, bool vec)
{
    if (rows <= 0 || cols <= 0) return;   // the tile reaches past out; no lane has lines to share
    const int es = dtype == BEAM_F32 ? 4 : 2, per = 16 / es;
    __syncwarp();
    uint8_t *o = static_cast<uint8_t *>(out) + at * es;
    const size_t pitch = (size_t)ldo * es;
    const int u = lane & 7;
    if (vec && cols % per == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = 4 * i + (lane >> 3);
            if (row < rows && u * per < cols)
                *reinterpret_cast<uint4 *>(o + row * pitch + u * 16) =
                    *reinterpret_cast<const uint4 *>(stg + row * 128 + ((u ^ (row & 7)) * 16));
        }
    } else {
#pragma unroll 4
        for (int i = 0; i < 8; ++i) {
            const int row = 4 * i + (lane >> 3);
            if (row >= rows) continue;
            if (es == 4) flush_row<4>(stg + row * 128, row, u, o + row * pitch, cols);
            else flush_row<2>(stg + row * 128, row, u, o + row * pitch, cols);
        }
    }
    __syncwarp();
}

}  // namespace mx
}  // namespace beam
