// Product of two microscaled operands on the block-scaled tensor cores
// (beam_mx_matmul):  out[t][n] = ga gw sum_k a[t][k] w[n][k].
//
// The MMA multiplies elements and block scales itself (tcgen05.mma
// .block_scale): codes come from shared memory, scales from tensor memory,
// sums stay in FP32 there.  The side with more rows (or the tokens, when both
// sides have more than 128) is the MMA's A operand, in tiles of 128 rows; the
// other is B, in tiles of BN = 16 .. 256 rows.
//
//   warp 0      one lane loads stages: a 128-byte wide box of codes of either
//               side (128B swizzle) and the 512-byte scale tiles that go with
//               it, by TMA and bulk copies into a ring
//   warp 10     one lane copies a stage's scale tiles to tensor memory
//               (tcgen05.cp, replicated to the four lane quadrants)
//   warp 1      one lane issues a stage's four MMAs
//   warps 2-9   epilogue: tensor memory to registers, tensor scales, rounding,
//               stores
//
// Where there are few tiles, the K steps of a tile are split over the CTAs of a
// cluster; each leaves its FP32 tile in its own shared memory and writes a
// share of the rows, summed over all of them in rank order, so results do not
// depend on timing and no workspace is needed.
//
// Bound, on a B200:
//   one sequence, NVFP4 5120 x 20480 (59 MB): 13.5 us = 4.4 TB/s.  About 3 us
//     are launch, set-up and the sum over a cluster; the stream itself runs at
//     5.5 TB/s (37888 x 20480: 79 us), the scales' copies taking 8% of it.
//   64 tokens, MXFP8 x MXFP4, 20480 x 5120 (56 MB): 22.4 us = 2.6 TB/s.  The TMA
//     unit takes about 3 clocks a row of a box, 64 bytes of 4-bit codes (spread
//     or not, the time is the same) as long as 128 bytes of others, and the
//     token rows cost as many again by half; and 160 tiles leave 12 of 148 SMs
//     with two.  Weights on the B side in tiles of 192, tokens on A, took 25.6 us.
//   L2 prefetches of the codes 6 or 12 stages ahead made all of them slower
//     (79 -> 95 us, 27 -> 32 us).
#include <atomic>

#include "mx_matmul.cuh"

namespace beam {
namespace {

using namespace mx;

// Sticky status word of the device (beam_ops_status), and where callers that
// take it, each with a slot of its own, find what it held.
constexpr int kTakers = 1024;
__device__ int g_ops_status;
__device__ int g_ops_taken[kTakers];

// Read and cleared in one step: of several callers one gets an event.
__global__ void take_status_kernel(int slot) { g_ops_taken[slot] = atomicExch(&g_ops_status, 0); }

template <int KIND, int BN>
struct Cfg {
    static constexpr int NQB = 1;                                        // BN <= 128: one scale block of B
    static constexpr int P_BYTES = kTileP * kRowBytes;
    static constexpr int Q_BYTES = BN * kRowBytes;
    static constexpr int STAGE = P_BYTES + Q_BYTES + (scale_bytes(KIND, NQB) + 1023) / 1024 * 1024;
    static constexpr int SF_COLS = scale_cols(KIND, NQB);
    static constexpr int STAGING = BN == 128 ? kEpiWarps * 4096 : 0;
    // tiles of up to 64 columns: half an SM, so that two CTAs share one
    static constexpr int BUDGET = BN <= 64 ? 110 * 1024 : 224 * 1024 - STAGING;
    static constexpr int FIT = BUDGET / STAGE;
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    static constexpr int TMEM_COLS = BN <= 64 ? 256 : 512;
    static constexpr int NBUF = 2;
    static constexpr int SF0 = NBUF * BN;
    static constexpr int SMEM = 1024 + STAGES * STAGE + STAGING + 384;
    static constexpr int CTAS_PER_SM = BN <= 64 ? 2 : 1;
    static constexpr int RED_LD = BN + 4;   // floats a row of a tile in shared memory: no bank met twice
    static_assert(STAGES >= 3 && SF0 + STAGES * SF_COLS <= TMEM_COLS, "tensor memory");
    static_assert(SMEM <= 232448 && RED_LD * kTileP * 4 <= STAGES * STAGE, "shared memory");
};

// Instruction descriptor of the block-scaled kinds: bits 4-5 scale id of B,
// 7-9 / 10-12 element types of A / B (E2M1: 1 in the 4-bit kinds, 5 in
// mxf8f6f4; E4M3: 0), 17-22 N >> 3, 23 scale type (1: UE8M0, 0: E4M3), 27-28
// M >> 7, 29-30 scale id of A.
uint32_t idesc_of(int kind, int m, int n, bool a_fp4, bool b_fp4)
{
    const uint32_t fa = kind == kMx8 ? (a_fp4 ? 5u : 0u) : 1u, fb = kind == kMx8 ? (b_fp4 ? 5u : 0u) : 1u;
    return (fa << 7) | (fb << 10) | ((uint32_t)(n >> 3) << 17) | (kind == kNv ? 0u : 1u << 23) |
           ((uint32_t)(m >> 7) << 27);
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// A CTA's share of a tile: every (8 split)-th group of rows of out, each the
// sum over the cluster's FP32 tiles ([rows][LD] at `base`, COLS columns) in
// rank order.  Four columns a lane; the loads of 8 / S rows from up to S ranks
// are in flight together, since another CTA's shared memory is some 500 clocks
// away (row by row 1000 x 100 x 512 took 7.4 us, 6.4 us so).
template <int COLS, int LD, int S>
__device__ __forceinline__ void write_rows(const MatmulArgs &p, uint32_t base, int rank, int w, int lane, int row0, int rows,
                                           int col0, int cols)
{
    constexpr int LANES = COLS / 4, GROUP = 32 / LANES, U = 8 / S;   // lanes a row, rows a warp takes at once
    static_assert(LANES * GROUP == 32, "whole warps");
    const float ga = p.ga ? *p.ga : 1.0f, gw = p.gw ? *p.gw : 1.0f;
    const int c = lane % LANES * 4, step = kEpiWarps * p.split * GROUP;
    for (int first = (rank * kEpiWarps + w) * GROUP + lane / LANES; first < rows; first += U * step) {
        float4 v[U][S];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = first + u * step;
            if (r >= rows || c >= cols) continue;
            const uint32_t at = base + (uint32_t)(r * LD + c) * 4u;
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (s < p.split) v[u][s] = ld_cluster_f32x4(S > 1 ? mapa_shared(at, (uint32_t)s) : at);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = first + u * step;
            if (r >= rows || c >= cols) continue;
            float4 y = v[u][0];
#pragma unroll
            for (int s = 1; s < S; ++s)
                if (s < p.split) y.x += v[u][s].x, y.y += v[u][s].y, y.z += v[u][s].z, y.w += v[u][s].w;
            const float o[4] = {y.x * ga * gw, y.y * ga * gw, y.z * ga * gw, y.w * ga * gw};
            const size_t to = (size_t)(row0 + r) * p.ldo + col0 + c;
            if (p.dtype == BEAM_F32) {
                float *out = static_cast<float *>(p.out) + to;
                if (c + 4 <= cols && (reinterpret_cast<uintptr_t>(out) & 15u) == 0) {
                    *reinterpret_cast<float4 *>(out) = make_float4(o[0], o[1], o[2], o[3]);
                    continue;
                }
            } else {
                uint16_t *out = static_cast<uint16_t *>(p.out) + to;
                if (c + 4 <= cols && (reinterpret_cast<uintptr_t>(out) & 7u) == 0) {
                    *reinterpret_cast<uint2 *>(out) = p.dtype == BEAM_BF16 ? make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]))
                                                                           : make_uint2(pack_f16x2(o[0], o[1]), pack_f16x2(o[2], o[3]));
                    continue;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < cols) put(p.out, p.dtype, to + j, o[j]);
        }
    }
}

template <int COLS, int LD>
__device__ __forceinline__ void write_tile(const MatmulArgs &p, uint32_t base, int rank, int w, int lane, int row0, int rows,
                                           int col0, int cols)
{
    if (p.split == 1) write_rows<COLS, LD, 1>(p, base, rank, w, lane, row0, rows, col0, cols);
    else if (p.split == 2) write_rows<COLS, LD, 2>(p, base, rank, w, lane, row0, rows, col0, cols);
    else if (p.split <= 4) write_rows<COLS, LD, 4>(p, base, rank, w, lane, row0, rows, col0, cols);
    else write_rows<COLS, LD, 8>(p, base, rank, w, lane, row0, rows, col0, cols);
}

template <int KIND, int BN>
__global__ void __launch_bounds__(kThreads, (Cfg<KIND, BN>::CTAS_PER_SM))
    mx_matmul_kernel(const __grid_constant__ Maps maps, const MatmulArgs p)
{
    using C = Cfg<KIND, BN>;
    constexpr int CPS = tiles_per_stage(KIND);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    uint8_t *staging = base_ptr + C::STAGES * C::STAGE;
    uint64_t *full = reinterpret_cast<uint64_t *>(staging + C::STAGING);
    uint64_t *empty = full + C::STAGES;
    uint64_t *tfull = empty + C::STAGES;
    uint64_t *tempty = tfull + 2;
    uint64_t *drain = tempty + 2;
    uint64_t *scaled = drain + 2;   // a stage's scales are in tensor memory (and its codes in shared)
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(scaled + C::STAGES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WaitCtl ctl{p.status, p.limit_ns};
    const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
            mbar_init(smem_u32(&scaled[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&tfull[a]), 1);
            mbar_init(smem_u32(&tempty[a]), 32 * kEpiWarps);
        }
        for (int a = 0; a < 2; ++a) mbar_init(smem_u32(&drain[a]), 1);
        fence_barrier_init();
        tma_prefetch_desc(&maps.p);
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.sp);
        tma_prefetch_desc(&maps.sq);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int total = status_is_set(ctl.status) ? 0 : p.p_tiles * p.q_tiles;
    const int first = blockIdx.x / p.split, stride = gridDim.x / p.split;
    const int ks0 = (int)((long long)p.nst * rank / p.split), ks1 = (int)((long long)p.nst * (rank + 1) / p.split);

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ loads
            const uint64_t pol_p = p.swap ? l2_policy_evict_first() : l2_policy_evict_normal();
            const uint64_t pol_q = l2_policy_evict_normal();
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            for (int item = first; item < total && ok; item += stride) {
                const int pt = item % p.p_tiles, qt = item / p.p_tiles;
                for (int ks = ks0; ks < ks1; ++ks) {
                    if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, ctl)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sp = base + stage * C::STAGE, sq = sp + C::P_BYTES, sf = sq + C::Q_BYTES;
                    const uint32_t fb = smem_u32(&full[stage]);
                    mbar_arrive_expect_tx(fb, ks == p.withheld ? p.tx + kWithheldBytes : p.tx);
                    // x: bytes for the byte maps, elements for the 4-bit map (both 128 a stage)
                    tma_load_2d(sp, &maps.p, ks * kRowBytes, pt * kTileP, fb, pol_p);
                    tma_load_2d(sq, &maps.q, ks * kRowBytes, qt * BN, fb, pol_q);
                    tma_load_3d(sf, &maps.sp, ks * CPS, pt, fb);
                    tma_load_3d(sf + CPS * 512, &maps.sq, ks * CPS, qt * BN >> 7, fb);
                    ++issued;
                    if (++stage == C::STAGES) stage = 0, phase ^= 1u;
                }
            }
            // copies in flight land before the CTA leaves, also those whose
            // readers gave up after this thread had issued its last
            for (long long n = issued < C::STAGES ? issued : C::STAGES; n > 0; --n) {
                if (stage == 0) stage = C::STAGES - 1, phase ^= 1u;
                else --stage;
                mbar_wait_drain(smem_u32(&full[stage]), phase, ctl.limit_ns);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------------------------ MMAs
            int stage = 0, iter = 0;
            uint32_t phase = 0;
            bool ok = true, any = false;
            for (int item = first; item < total && ok; item += stride, ++iter) {
                const int acc = iter % C::NBUF;
                const uint32_t d = tmem + acc * BN;
                const uint32_t qcol = BN == 64 ? scale_column(item / p.p_tiles * BN) : 0u;   // smaller: one tile of B
                if (!mbar_wait(smem_u32(&tempty[acc]), ((uint32_t)(iter / C::NBUF) & 1u) ^ 1u, ctl)) break;
                tc_fence_after();
                for (int ks = ks0; ks < ks1; ++ks) {
                    if (!mbar_wait(smem_u32(&full[stage]), phase, ctl) || !mbar_wait(smem_u32(&scaled[stage]), phase, ctl)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sp = base + stage * C::STAGE;
                    mma_stage<KIND, 1, C::NQB>(d, sp, sp + C::P_BYTES, tmem + C::SF0 + stage * C::SF_COLS, qcol, p.idesc,
                                               min(4, p.ksteps - ks * 4), ks == ks0);
                    any = true;
                    umma_commit(smem_u32(&empty[stage]));
                    if (++stage == C::STAGES) stage = 0, phase ^= 1u;
                }
                if (ok) umma_commit(smem_u32(&tfull[acc]));
            }
            if (any) {   // every MMA is complete before tensor memory is released
                umma_commit(smem_u32(drain));
                mbar_wait_drain(smem_u32(drain), 0, ctl.limit_ns);
            }
        }
    } else if (warp == kCopyWarp) {
        if (lane == 0) {
            // ------------------------------------------------ scales
            // In a thread of their own: in the MMAs' they took as long again
            // as those (a single tile of K = 20480: NVFP4 44 -> 33 us).
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true, any = false;
            for (int item = first; item < total && ok; item += stride) {
                for (int ks = ks0; ks < ks1; ++ks) {
                    if (!mbar_wait(smem_u32(&full[stage]), phase, ctl)) {
                        ok = false;
                        break;
                    }
                    // a column set per ring stage: a copy never meets an
                    // earlier stage's MMAs still reading
                    copy_scales<KIND, 1, C::NQB>(base + stage * C::STAGE + C::P_BYTES + C::Q_BYTES,
                                                 tmem + C::SF0 + stage * C::SF_COLS);
                    any = true;
                    umma_commit(smem_u32(&scaled[stage]));
                    if (++stage == C::STAGES) stage = 0, phase ^= 1u;
                }
            }
            if (any) {
                umma_commit(smem_u32(&drain[1]));
                mbar_wait_drain(smem_u32(&drain[1]), 0, ctl.limit_ns);
            }
        }
    } else {
        // ---------------------------------------------------- epilogue
        const int quad = warp & 3, half = (warp - 2) >> 2;
        constexpr int CH = BN >= 64 ? 32 : 16;          // columns read at a time
        constexpr int SPAN = BN == 128 ? 64 : CH;       // columns a warp takes in turn
        const float ga = p.ga ? *p.ga : 1.0f, gw = p.gw ? *p.gw : 1.0f;
        int iter = 0;
        for (int item = first; item < total; item += stride, ++iter) {
            const int acc = iter % C::NBUF;
            const bool ok = mbar_wait(smem_u32(&tfull[acc]), (uint32_t)(iter / C::NBUF) & 1u, ctl);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const int pt = item % p.p_tiles, qt = item / p.p_tiles;
            const int prow0 = pt * kTileP + quad * 32;
            const uint32_t taddr = tmem + acc * BN + ((uint32_t)(quad * 32) << 16);
#pragma unroll 1
            for (int c0 = half * SPAN; c0 < BN; c0 += 2 * SPAN) {
#pragma unroll 1
                for (int c1 = c0; c1 < c0 + SPAN; c1 += CH) {
                    uint32_t r[CH];
                    if constexpr (CH == 32) tmem_ld32(taddr + c1, r);
                    else tmem_ld16(taddr + c1, r);
                    tmem_ld_wait();
                    if (p.single) {   // the ring is free: its one tile goes there, in rows of out
                        float *red = reinterpret_cast<float *>(base_ptr);
                        if (p.swap) {
#pragma unroll
                            for (int j = 0; j < CH; ++j) red[(c1 + j) * kTileP + quad * 32 + lane] = __uint_as_float(r[j]);
                        } else {
                            uint4 *row = reinterpret_cast<uint4 *>(red + (quad * 32 + lane) * C::RED_LD + c1);
#pragma unroll
                            for (int j = 0; j < CH; j += 4) row[j / 4] = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
                        }
                        continue;
                    }
                    float v[CH];
#pragma unroll
                    for (int j = 0; j < CH; ++j) v[j] = __uint_as_float(r[j]) * ga * gw;
                    const int q0 = qt * BN + c1;
                    if constexpr (BN == 128) {
                        if (!p.swap) {
                            const int span = p.dtype == BEAM_F32 ? 32 : 64;
                            const int line = (c1 - c0) % span;   // column of the staged line
                            stage_columns(v, staging + (warp - 2) * 4096, lane, p.dtype, line / 32);
                            if (line + 32 == span)
                                flush_lines(staging + (warp - 2) * 4096, lane, p.dtype, p.out,
                                            (size_t)prow0 * p.ldo + q0 - line, p.ldo, min(32, p.P - prow0),
                                            min(span, p.Q - (q0 - line)), p.vec);
                            continue;
                        }
                    }
                    if (prow0 + lane < p.P) {
#pragma unroll
                        for (int j = 0; j < CH; ++j)
                            if (q0 + j < p.Q)
                                put(p.out, p.dtype,
                                    p.swap ? (size_t)(q0 + j) * p.ldo + prow0 + lane : (size_t)(prow0 + lane) * p.ldo + q0 + j,
                                    v[j]);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(smem_u32(&tempty[acc]));
        }
    }

    if (p.single) {
        // every CTA's FP32 tile is in its shared memory
        __syncwarp();
        if (p.split > 1) cluster_sync();
        else __syncthreads();
        if (warp >= 2 && warp < kCopyWarp && first < total) {
            const int pt = first % p.p_tiles, qt = first / p.p_tiles;
            if (p.swap) write_tile<kTileP, kTileP>(p, base, rank, warp - 2, lane, qt * BN, min(BN, p.Q - qt * BN), pt * kTileP, min(kTileP, p.P - pt * kTileP));
            else write_tile<BN, C::RED_LD>(p, base, rank, warp - 2, lane, pt * kTileP, min(kTileP, p.P - pt * kTileP), qt * BN, min(BN, p.Q - qt * BN));
        }
        __syncwarp();
        if (p.split > 1) cluster_sync();   // no CTA leaves while another may read its tile
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static std::atomic<EncodeTiledFn> fn{nullptr};
    EncodeTiledFn f = fn.load(std::memory_order_acquire);
    if (!f) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            f = reinterpret_cast<EncodeTiledFn>(p);
            fn.store(f, std::memory_order_release);
        }
    }
    return f;
}

// Codes as a 2-D tensor of 128-byte wide boxes, 128B swizzle.  Bytes, except
// 4-bit codes beside 8-bit ones: those are spread by the copy to the 16-byte
// groups (8 bytes of codes, 8 of padding) that the mixed MMA reads.
bool code_map(CUtensorMap *m, const uint8_t *codes, int format, bool spread, long long rows, int K, int box_rows)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t pitch = format == BEAM_MXFP8 ? K : K / 2;
    cuuint64_t dims[2] = {spread ? (cuuint64_t)K : pitch, (cuuint64_t)rows};
    cuuint64_t strides[1] = {pitch};
    cuuint32_t box[2] = {kRowBytes, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return enc(m, spread ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
               const_cast<uint8_t *>(codes), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles as a 3-D tensor {128 words, tiles along K, 128-row blocks}; the
// box is a stage's tiles of `blocks` blocks.  Tiles past the end read as zero.
bool scale_map(CUtensorMap *m, const uint8_t *scales, long long rows, int n4, int tiles, int blocks)
{
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {128, (cuuint64_t)n4, (cuuint64_t)((rows + 127) / 128)};
    cuuint64_t strides[2] = {512, (cuuint64_t)n4 * 512};
    cuuint32_t box[3] = {128, (cuuint32_t)tiles, (cuuint32_t)blocks};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<uint8_t *>(scales), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KIND, int BN>
cudaError_t launch(const Maps &m, const MatmulArgs &a, int ctas, cudaStream_t s)
{
    using C = Cfg<KIND, BN>;
    cudaError_t e = cudaFuncSetAttribute(mx_matmul_kernel<KIND, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)a.split, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = a.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, mx_matmul_kernel<KIND, BN>, m, a);
}

template <int KIND>
cudaError_t launch_bn(int bn, const Maps &m, const MatmulArgs &a, int ctas, cudaStream_t s)
{
    switch (bn) {
        case 16: return launch<KIND, 16>(m, a, ctas, s);
        case 32: return launch<KIND, 32>(m, a, ctas, s);
        case 64: return launch<KIND, 64>(m, a, ctas, s);
        default: return launch<KIND, 128>(m, a, ctas, s);
    }
}

// beam_ops_debug_withhold's, for the thread's next product.
thread_local int t_withheld = -1, t_limit_ms = 0;

// Device address of the status word, looked up once per device.
std::atomic<int *> g_status_ptr[64];

int *status_ptr()
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    int *p = g_status_ptr[dev].load(std::memory_order_acquire);
    if (!p) {
        void *v = nullptr;
        if (cudaGetSymbolAddress(&v, g_ops_status) != cudaSuccess) return nullptr;
        p = static_cast<int *>(v);
        g_status_ptr[dev].store(p, std::memory_order_release);
    }
    return p;
}

}  // namespace
}  // namespace beam

extern "C" int beam_mx_matmul(void *stream, int a_format, const uint8_t *a_codes, const uint8_t *a_scales,
                              const float *a_tensor_scale, int w_format, const uint8_t *w_codes,
                              const uint8_t *w_scales, const float *w_tensor_scale, int T, int N, int K,
                              void *out, int dtype, long long ldo)
{
    using namespace beam;
    using namespace beam::ops;
    if (!format_ok(a_format) || !format_ok(w_format)) return fail(BEAM_ERR_INVALID_ARG, "format %d x %d", a_format, w_format);
    if (!dtype_ok(dtype)) return fail(BEAM_ERR_INVALID_ARG, "dtype %d", dtype);
    if (T < 0 || N < 0 || T >= (1 << 27) || N >= (1 << 27) || K <= 0)
        return fail(BEAM_ERR_INVALID_ARG, "T and N must be in 0 .. 2^27 - 1 and K positive");
    int kind;
    if (a_format == BEAM_NVFP4 && w_format == BEAM_NVFP4) kind = kNv;
    else if (a_format == BEAM_MXFP4 && w_format == BEAM_MXFP4) kind = kMx4;
    else if (a_format == BEAM_MXFP8 && (w_format == BEAM_MXFP4 || w_format == BEAM_MXFP8)) kind = kMx8;
    else return fail(BEAM_ERR_UNSUPPORTED, "formats %d x %d have no product", a_format, w_format);
    const int k_unit = kind == kMx8 ? 128 : 64;
    if (K % k_unit != 0) return fail(BEAM_ERR_UNSUPPORTED, "K must be a multiple of %d, got %d", k_unit, K);
    if (T == 0 || N == 0) return BEAM_OK;
    if (!a_codes || !a_scales || !w_codes || !w_scales || !out)
        return fail(BEAM_ERR_INVALID_ARG, "codes, scales and out are required");
    if (ldo < N) return fail(BEAM_ERR_INVALID_ARG, "ldo is below N");
    if (!aligned(a_codes, 32) || !aligned(a_scales, 32) || !aligned(w_codes, 32) || !aligned(w_scales, 32) ||
        !aligned(out, dtype_size(dtype)) || !aligned(a_tensor_scale, 4) || !aligned(w_tensor_scale, 4))
        return fail(BEAM_ERR_INVALID_ARG, "a pointer is not aligned");
    const int sms = sm_count();
    if (!sms) return fail(BEAM_ERR_CUDA, "no CUDA device");

    // the A side (128-row tiles): the tokens when both sides have more than
    // 128 rows (their stores are rows of out), else the longer side
    const bool swap = T <= 128 || N <= 128 ? N >= T : false;
    MatmulArgs a{};
    a.swap = swap;
    a.P = swap ? N : T;
    a.Q = swap ? T : N;
    a.ga = a_tensor_scale;
    a.gw = w_tensor_scale;
    a.out = out;
    a.ldo = ldo;
    a.dtype = dtype;
    a.vec = rows_aligned16(out, ldo, dtype);
    a.status = status_ptr();
    if (!a.status) return fail(BEAM_ERR_CUDA, "no device address of the status word");
    a.nst = (K + stage_k(kind) - 1) / stage_k(kind);
    a.ksteps = K / step_k(kind);
    const int n4 = (K / block_of(a_format) + 3) / 4;
    const Plan how = plan(kind, a.P, a.Q, a.nst, swap, a.vec != 0, sms);
    if (how.bn == 0) return fail(BEAM_ERR_UNSUPPORTED, "no plan for %d x %d x %d on %d SMs", T, N, K, sms);
    const int bn = how.bn, slots = sms * (bn <= 64 ? 2 : 1);
    const bool pair = how.pair;
    a.split = how.split;
    a.p_tiles = (a.P + (pair ? 255 : kTileP - 1)) / (pair ? 256 : kTileP);
    a.q_tiles = (a.Q + bn - 1) / bn;
    const long long tiles = (long long)a.p_tiles * a.q_tiles;
    const bool p_fp4 = (swap ? w_format : a_format) != BEAM_MXFP8, q_fp4 = (swap ? a_format : w_format) != BEAM_MXFP8;
    const bool p_spread = kind == kMx8 && p_fp4, q_spread = kind == kMx8 && q_fp4;
    a.idesc = idesc_of(kind, pair ? 256 : 128, bn, p_fp4, q_fp4);
    const int q_box = pair ? 128 : bn, cps = tiles_per_stage(kind), q_blocks = pair ? 2 : 1;
    // a spread copy counts the bytes of its packed codes
    a.tx = (uint32_t)(kTileP * (p_spread ? kRowBytes / 2 : kRowBytes) + q_box * (q_spread ? kRowBytes / 2 : kRowBytes) +
                      cps * 512 * (1 + q_blocks));
    a.withheld = t_withheld;
    a.limit_ns = t_withheld < 0 ? kWaitLimitNs : t_limit_ms * 1000000ll;
    t_withheld = -1;
    Maps m;
    if (!code_map(&m.p, swap ? w_codes : a_codes, swap ? w_format : a_format, p_spread, a.P, K, kTileP) ||
        !code_map(&m.q, swap ? a_codes : w_codes, swap ? a_format : w_format, q_spread, a.Q, K, q_box) ||
        !scale_map(&m.sp, swap ? w_scales : a_scales, a.P, n4, cps, 1) ||
        !scale_map(&m.sq, swap ? a_scales : w_scales, a.Q, n4, cps, q_blocks))
        return fail(BEAM_ERR_CUDA, "cuTensorMapEncodeTiled failed");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    // weights on the A side leave tensor memory in rows of out as they are
    a.single = !pair && (a.split > 1 || (tiles <= slots && !swap));
    const int ctas = (int)(tiles * a.split < slots || a.split > 1 ? tiles * a.split : slots);
    if (pair) e = launch_pair(kind, m, a, sms, s);
    else if (kind == kNv) e = launch_bn<kNv>(bn, m, a, ctas, s);
    else if (kind == kMx4) e = launch_bn<kMx4>(bn, m, a, ctas, s);
    else e = launch_bn<kMx8>(bn, m, a, ctas, s);
    return check_cuda(e, "beam_mx_matmul");
}

extern "C" int beam_ops_debug_withhold(int stage, int limit_ms)
{
    using namespace beam;
    using namespace beam::ops;
    if (stage < -1 || limit_ms < 1 || limit_ms > 2000)
        return fail(BEAM_ERR_INVALID_ARG, "stage must be >= -1 and limit_ms in 1 .. 2000, got %d, %d", stage, limit_ms);
    t_withheld = stage, t_limit_ms = limit_ms;
    return BEAM_OK;
}

extern "C" int beam_ops_status(void *stream)
{
    using namespace beam;
    using namespace beam::ops;
    static std::atomic<unsigned> ticket{0};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
    if (int rc = check_cuda(cudaStreamIsCapturing(s, &capturing), "beam_ops_status")) return rc;
    if (capturing != cudaStreamCaptureStatusNone) return fail(BEAM_ERR_INVALID_ARG, "beam_ops_status: the stream is being captured");
    const int slot = (int)(ticket.fetch_add(1, std::memory_order_relaxed) % kTakers);
    int host = 0;
    take_status_kernel<<<1, 1, 0, s>>>(slot);
    if (int rc = check_cuda(cudaGetLastError(), "beam_ops_status")) return rc;
    if (int rc = check_cuda(cudaMemcpyFromSymbolAsync(&host, g_ops_taken, sizeof(int), slot * sizeof(int), cudaMemcpyDeviceToHost, s),
                            "beam_ops_status")) return rc;
    if (int rc = check_cuda(cudaStreamSynchronize(s), "beam_ops_status")) return rc;
    return host;
}
