// Microscaled product on CTA pairs (cta_group::2): 256 x 256 tiles of out.
//
// Either CTA holds 128 of the tile's A rows (tokens) and 128 of its B rows
// (weights) a stage; the pair's MMAs read both halves, so a stage's 32 KB of
// codes serve 256 x 256 x 256 products -- half the fill of a single CTA's
// 128 x 256 tile, which the L2 could not feed at the 4-bit MMA rate (64 bytes
// a clock and SM here).  Accumulators: 256 columns of either CTA's tensor
// memory, one buffer (the scales of the ring's stages take the rest): the
// epilogue empties it into registers first (128 a thread), hands it back, and
// rounds and stores while the next tile's MMAs run.
//
// 4096 x 10240 x 5120, and the same kernel with parts left out (us): NVFP4 110,
// 85 without the scale copies, 98 without the MMAs, 70 with the loads alone;
// MXFP4 88, 84, 75, 69; MXFP8 x MXFP4 155, 140, 111, 108.  So the loads (64 KB
// a pair and stage) are the largest part of the 4-bit kinds' time; NVFP4's 12
// copies a stage share the tensor pipe with the MMAs and add 26 us, MXFP4's
// 6 add 4, MXFP8's 3 (in twice the stages) 15.
#include "mx_matmul.cuh"

namespace beam {
namespace mx {

namespace {

constexpr uint16_t kBoth = 0x3;

template <int KIND>
struct PairCfg {
    static constexpr int HALF = 128 * kRowBytes;          // codes of 128 rows
    static constexpr int STAGE = 2 * HALF + (scale_bytes(KIND, 2) + 1023) / 1024 * 1024;
    static constexpr int STAGES = 5;
    static constexpr int STAGING = kEpiWarps * 4096;
    static constexpr int SF_COLS = scale_cols(KIND, 2);
    static constexpr int SF0 = 256;
    static constexpr int SMEM = 1024 + STAGES * STAGE + STAGING + 256;
    static_assert(SMEM <= 232448 && SF0 + STAGES * SF_COLS <= 512, "one CTA an SM");
};

}  // namespace

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mx_matmul_pair_kernel(const __grid_constant__ Maps maps, const MatmulArgs p)
{
    using C = PairCfg<KIND>;
    constexpr int CPS = tiles_per_stage(KIND);
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *base_ptr = smem_raw + (base - raw);
    uint8_t *staging = base_ptr + C::STAGES * C::STAGE;
    uint64_t *full = reinterpret_cast<uint64_t *>(staging + C::STAGING);
    uint64_t *empty = full + C::STAGES;
    uint64_t *tfull = empty + C::STAGES;
    uint64_t *tempty = tfull + 1;
    uint64_t *drain = tempty + 1;
    uint64_t *scaled = drain + 2;   // a stage's scales are in both CTAs' tensor memory
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(scaled + C::STAGES);
    volatile uint32_t *gave_up = tmem_slot + 1;   // a wait of this CTA ran out
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();   // 0 issues the MMAs
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const WaitCtl ctl{p.status, p.limit_ns};

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
            mbar_init(smem_u32(&scaled[s]), 1);
        }
        mbar_init(smem_u32(tfull), 1);
        mbar_init(smem_u32(tempty), 2 * 32 * kEpiWarps);
        for (int a = 0; a < 2; ++a) mbar_init(smem_u32(&drain[a]), 1);
        *gave_up = 0;
        fence_barrier_init();
        tma_prefetch_desc(&maps.p);
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.sp);
        tma_prefetch_desc(&maps.sq);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc_pair(smem_u32(tmem_slot), 512);
        tmem_relinquish_pair();
    }
    pdl_launch_dependents();
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();   // both CTAs' barriers exist before either signals the other
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int total = status_is_set(ctl.status) ? 0 : p.p_tiles * p.q_tiles;

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------ loads
            const uint64_t pol = l2_policy_evict_normal();
            int stage = 0;
            uint32_t phase = 0;
            long long issued = 0;
            bool ok = true;
            for (int item = pair; item < total && ok; item += npairs) {
                const int pt = item % p.p_tiles, qt = item / p.p_tiles;
                const int prow = pt * 256 + (int)rank * 128, qrow = qt * 256 + (int)rank * 128;
                for (int ks = 0; ks < p.nst; ++ks) {
                    if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, ctl)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sp = base + stage * C::STAGE, sq = sp + C::HALF, sf = sq + C::HALF;
                    const uint32_t fl = smem_u32(&full[stage]), f = mapa_shared(fl, 0);   // CTA 0's barrier
                    if (rank == 0) mbar_arrive_expect_tx(fl, 2u * p.tx + (ks == p.withheld ? kWithheldBytes : 0u));
                    tma_load_2d_pair(sp, &maps.p, ks * kRowBytes, prow, f, pol);
                    tma_load_2d_pair(sq, &maps.q, ks * kRowBytes, qrow, f, pol);
                    tma_load_3d_pair(sf, &maps.sp, ks * CPS, prow >> 7, f);
                    // the scales of all 256 B rows, in either CTA
                    tma_load_3d_pair(sf + CPS * 512, &maps.sq, ks * CPS, qt * 2, f);
                    ++issued;
                    if (++stage == C::STAGES) stage = 0, phase ^= 1u;
                }
            }
            if (!ok) *gave_up = 1;
            // copies in flight (CTA 0's barriers count both CTAs') land before the pair leaves, also
            // those whose readers gave up after this thread had issued its last
            for (long long n = rank != 0 ? 0 : issued < C::STAGES ? issued : C::STAGES; n > 0; --n) {
                if (stage == 0) stage = C::STAGES - 1, phase ^= 1u;
                else --stage;
                mbar_wait_drain(smem_u32(&full[stage]), phase, ctl.limit_ns);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ------------------------------------------------ MMAs
            int stage = 0;
            uint32_t phase = 0, iter = 0;
            bool ok = true, any = false;
            for (int item = pair; item < total && ok; item += npairs, ++iter) {
                if (!mbar_wait_cluster(smem_u32(tempty), (iter & 1u) ^ 1u, ctl)) break;
                tc_fence_after();
                for (int ks = 0; ks < p.nst; ++ks) {
                    if (!mbar_wait(smem_u32(&full[stage]), phase, ctl) || !mbar_wait(smem_u32(&scaled[stage]), phase, ctl)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sp = base + stage * C::STAGE;
                    mma_stage<KIND, 2, 2>(tmem, sp, sp + C::HALF, tmem + C::SF0 + stage * C::SF_COLS, 0, p.idesc,
                                          min(4, p.ksteps - ks * 4), ks == 0);
                    any = true;
                    umma_commit_pair(smem_u32(&empty[stage]), kBoth);
                    if (++stage == C::STAGES) stage = 0, phase ^= 1u;
                }
                if (ok) umma_commit_pair(smem_u32(tfull), kBoth);
            }
            if (any) umma_commit_pair(smem_u32(drain), kBoth);
        }
    } else if (warp == kCopyWarp) {
        if (lane == 0 && rank == 0) {
            // ------------------------------------------------ scales
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true, any = false;
            for (int item = pair; item < total && ok; item += npairs) {
                for (int ks = 0; ks < p.nst; ++ks) {
                    if (!mbar_wait(smem_u32(&full[stage]), phase, ctl)) {
                        ok = false;
                        break;
                    }
                    copy_scales<KIND, 2, 2>(base + stage * C::STAGE + 2 * C::HALF, tmem + C::SF0 + stage * C::SF_COLS);
                    any = true;
                    umma_commit_pair(smem_u32(&scaled[stage]), 1);
                    if (++stage == C::STAGES) stage = 0, phase ^= 1u;
                }
            }
            if (any) umma_commit_pair(smem_u32(&drain[1]), kBoth);
        }
    } else {
        // ---------------------------------------------------- epilogue (both CTAs)
        const int quad = warp & 3, half = (warp - 2) >> 2;
        uint8_t *stg = staging + (warp - 2) * 4096;
        const uint32_t release = mapa_shared(smem_u32(tempty), 0);
        const float ga = p.ga ? *p.ga : 1.0f, gw = p.gw ? *p.gw : 1.0f;
        uint32_t iter = 0;
        for (int item = pair; item < total; item += npairs, ++iter) {
            const bool ok = mbar_wait(smem_u32(tfull), iter & 1u, ctl);
            if (!__all_sync(0xffffffffu, ok)) {
                *gave_up = 1;
                break;
            }
            tc_fence_after();
            const int pt = item % p.p_tiles, qt = item / p.p_tiles;
            const int prow0 = pt * 256 + (int)rank * 128 + quad * 32;
            const uint32_t taddr = tmem + half * 128 + ((uint32_t)(quad * 32) << 16);
            uint32_t r[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(taddr + c * 32, r[c]);
            tmem_ld_wait();
            tc_fence_before();
            mbar_arrive_cluster(release);
            const int span = p.dtype == BEAM_F32 ? 1 : 2;   // 32-column pieces of a staged line
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[c][j]) * ga * gw;
                stage_columns(v, stg, lane, p.dtype, c % span);
                if (c % span == span - 1) {
                    const int q0 = qt * 256 + half * 128 + (c - span + 1) * 32;
                    flush_lines(stg, lane, p.dtype, p.out, (size_t)prow0 * p.ldo + q0, p.ldo, min(32, p.P - prow0),
                                min(span * 32, p.Q - q0), p.vec);
                }
            }
        }
    }

    // no tensor memory is released before CTA 0's copies and MMAs are complete
    if (warp == 1 && lane == 0 && pair < total) {
        mbar_wait_drain(smem_u32(drain), 0, ctl.limit_ns);
        mbar_wait_drain(smem_u32(&drain[1]), 0, ctl.limit_ns);
    }
    tc_fence_before();
    __syncthreads();
    // a copy of CTA 1 that CTA 0 no longer counted has no barrier to wait on:
    // 0.1 ms for it to land
    if (*gave_up && threadIdx.x == 0)
        for (int i = 0; i < 100; ++i) __nanosleep(1000);
    __syncwarp();
    cluster_sync();   // no CTA leaves while the other may still signal it
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

namespace {

template <int KIND>
cudaError_t launch(const Maps &m, const MatmulArgs &a, int sms, cudaStream_t s)
{
    const cudaError_t e = cudaFuncSetAttribute(mx_matmul_pair_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               PairCfg<KIND>::SMEM);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)a.p_tiles * a.q_tiles;
    const int pairs = (int)(tiles < sms / 2 ? tiles : sms / 2);
    return launch_pdl(mx_matmul_pair_kernel<KIND>, dim3(2 * pairs), dim3(kThreads), PairCfg<KIND>::SMEM, s, m, a);
}

}  // namespace

cudaError_t launch_pair(int kind, const Maps &m, const MatmulArgs &a, int sms, cudaStream_t s)
{
    if (kind == kNv) return launch<kNv>(m, a, sms, s);
    if (kind == kMx4) return launch<kMx4>(m, a, sms, s);
    return launch<kMx8>(m, a, sms, s);
}

}  // namespace mx
}  // namespace beam
