// Tile width and split of a microscaled product (mx_matmul.cu).  Plain C++, so
// that plans can be walked on the host for every size and SM count.
#pragma once

namespace beam {
namespace mx {

// Kinds of block-scaled MMA: NVFP4 (a scale per 16), MXFP4 (per 32) and
// MXFP8 x MXFP8 / MXFP4 (per 32, 8-bit operands in shared memory).
enum Kind { kNv = 0, kMx4 = 1, kMx8 = 2 };

constexpr int kTileP = 128;               // rows of the A side per CTA

// Clusters of 1 to 8 CTAs that a B200 holds at once, at one and two CTAs an SM
// (cudaOccupancyMaxActiveClusters with these kernels' threads and shared
// memory).  More clusters than fit only wait for their turn.
constexpr int kSms = 148;
constexpr int kClusters[2][8] = {{148, 74, 45, 33, 26, 22, 15, 15}, {296, 148, 93, 71, 56, 45, 37, 33}};

struct Plan {
    int bn, split;
    bool pair;
    long long cost;   // ns
};

// Tile width and split of K with the least estimated time.  The estimate: 2.5
// us of launch; a tile's set-up and epilogue; its stages one after another (a
// stage of a lone CTA waits on its loads and scale copies, 0.3 us + 2 ns a
// column, longer where two CTAs share an SM); the sum over a cluster; and for
// more tiles than CTAs the waves of them.  It was fitted to tiles of 32 to
// 128 columns split 1 to 8 times (500 x 500 x 512: 5.0 us at 64 columns, 6.2 at
// 128; 300 x 1000 x 5120: 9.9 us split 4 ways, 18.3 whole; 1 x 5120 x 20480:
// 13.5 us split 6 ways, 16.3 four ways, 25 two ways) and pairs (2048 x 5120 x
// 5120 MXFP8 x MXFP4: 50 us, 70 on single CTAs; 1021 x 5123 x 2560: 20.7 us,
// 17.5 on single CTAs, whose many tiles hide the odd rows' stores better).  It
// is off where 137 to 148 weight tiles meet at most 64 tokens: one CTA a tile is
// taken, two are faster (64 x 18944 x 5120: MXFP8 x MXFP4 20.1 and 16.7 us, NVFP4
// 16.8 and 14.6).
inline Plan plan(int kind, int P, int Q, int nst, bool swap, bool vec, int sms)
{
    const long long p_tiles = (P + kTileP - 1) / kTileP;
    Plan best{0, 1, false, 0};
    const auto offer = [&](int bn, int split, bool pair, long long cost) {
        if (best.bn == 0 || cost < best.cost) best = Plan{bn, split, pair, cost};
    };
    for (int bn = 16; bn <= 128; bn *= 2) {
        if (bn < 64 && bn < Q) continue;        // one tile of B, or scales at even columns
        const long long tiles = p_tiles * ((Q + bn - 1) / bn);
        const int per_sm = bn <= 64 ? 2 : 1;
        const long long fixed = 900 + 12 * bn;
        if (tiles > (long long)sms * per_sm) {   // persistent, the epilogue beside the next tile
            if (bn < 128 && !swap) continue;     // whose stores are then by columns
            const long long waves = (tiles + sms * per_sm - 1) / (sms * per_sm);
            offer(bn, 1, false, 2500 + fixed + waves * (nst * 410ll * per_sm + (vec ? 0 : 800)));
        } else {
            // whole tiles, or clusters that all fit at once
            for (int s = 1; s <= 8 && s <= nst && (s == 1 || tiles <= (long long)kClusters[per_sm - 1][s - 1] * sms / kSms); ++s) {
                // CTAs an SM, in thousandths: 8-bit stages mostly wait, 4-bit
                // ones (twice the K) are held up by the SM's other CTA
                const int ctas = (int)tiles * s, mean = ctas > sms ? ctas * 1000 / sms : 1000;
                const int share = kind == kMx8 || mean == 1000 ? mean : (mean + 2000) / 2;
                const int stage = (300 + 2 * bn) * share / 1000;
                offer(bn, s, false, 2500 + fixed + (s > 1 ? 300 + 100 * s : 0) + (long long)((nst + s - 1) / s) * stage);
            }
        }
        if (bn >= Q) break;
    }
    if (!swap && P > 128 && Q > 128 && sms >= 2) {
        const long long tiles = (long long)((P + 255) / 256) * ((Q + 255) / 256), waves = (tiles + sms / 2 - 1) / (sms / 2);
        offer(256, 1, true, 5000 + waves * (nst * 500ll + (vec ? 0 : 2900)));
    }
    return best;
}

}  // namespace mx
}  // namespace beam
