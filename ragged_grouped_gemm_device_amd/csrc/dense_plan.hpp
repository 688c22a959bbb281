// How a dense product is cut into tiles and pieces of K. Plain host code.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moe {

enum DensePass { kForward, kDgrad, kWgrad };

constexpr int DBK = 64;  // K elements per slab (128 bytes)

// Tile and split of a product: the cheapest by a model of the time (us) fitted to
// 54 products measured with operands from HBM, between 16 x 704 x 704 and 16384 x 7168
// x 4096 (it picks the fastest of 14 candidates there, or mostly one within 8%):
//   's' 64 x 64 tiles (small kernel): a round over the compute units takes 3.0, plus 1.05
//       for every slab of a wavefront (a quarter of the split's slabs), 0.55 with at most
//       32 rows;
//   'M' 128 x 128 tiles, two stages: 0.85 a slab for one on a compute unit, 0.95 for two
//       side by side (an eighth more in the dgrad, which reads W from HBM in 128-byte
//       pieces of its rows), 3.5 for the prologue and epilogue;
//   'D' 128 x 128 tiles, four stages, one on a compute unit: 0.53 to 0.73 a slab, 4.0;
//   'H' 256 x 128 tiles, three stages, one on a compute unit: 0.82 to 0.92 a slab, 5.0 (9.0
//       in the forward, whose activation no neighbour's products cover: 1000 x 2880 x 5760
//       51.1 us with GeGLU, M 47.2). The plan does not see the activation: a forward without
//       one would be 8% faster as H there (45.4 and 49.6) and takes M all the same. About
//       one forward shape in 2000 takes H (10959 x 3360 x 320);
//   'L' 256 x 256 tiles, two stages: 1.05 a slab with few of them at work up to 1.7 with
//       all (clock and L2), 8.0;
//   any: no less than 1.0 and the operands' read, at 5.2 TB/s with every compute unit at
//       work down to 2.6 with few;
//   splits: 1.8 for the joining launch and the partial sums' write and read, 3.5 TB/s for
//       the two together (they mostly stay in the last-level cache);
//   'L' with a part of a round left over: only those tiles' K in pieces (wgrad 8192 x 2880
//       x 5760, 276 tiles: 261 us, 370 as two rounds, 346 as M; 32768 x 2880 x 5760: 936,
//       1506, 1460; forward 4300 x 6000 x 4160: 222, 302 as two rounds; 9000 x 2880 x 5760:
//       259, 267; dgrad 4300 x 4104 x 4160: 147, 187).
// E.g. forward 2048 x 2048 x 2048: s 40.6 us, M 35.4, D 25.7, H 32.8, L 52.0; forward
// 16384 x 512 x 512: 37.8, 15.0, 19.2, 15.0, 19.1; dgrad 8192 x 2880 x 5760: 679, 287, 325,
// 254, 288; forward 4096 x 2048 x 7168: 256, 133, 154, 135, 114. 128 x 256 tiles measured
// like 256 x 128; with two stages instead of three neither was ever the fastest.
struct DensePlan {
    char kind;
    int ntm, ntn, splits, split_slabs;
    int tail_first, tail_splits, tail_slabs;  // tail_splits > 1: see DenseArgs
};
constexpr int kDenseCus = 256;

inline DensePlan dense_plan(int64_t M, int64_t N, int64_t K, DensePass pass) {
    const int64_t slabs = (K + DBK - 1) / DBK;
    DensePlan best{};
    double least = 0;
    for (const char kind : {'s', 'M', 'D', 'H', 'L'}) {
        const int64_t er = kind == 's' ? 64 : kind == 'L' || kind == 'H' ? 256 : 128;
        const int64_t ec = kind == 's' ? 64 : kind == 'L' ? 256 : 128;
        const int64_t ntm = (M + er - 1) / er, ntn = (N + ec - 1) / ec;
        for (int64_t want = 1; want <= 16 && want <= slabs; want *= 2) {
            const int64_t ss = (slabs + want - 1) / want, s = (slabs + ss - 1) / ss;
            const int64_t tiles = ntm * ntn * s, rounds = (tiles + kDenseCus - 1) / kDenseCus;
            const double fill = std::min(1.0, (double)tiles / kDenseCus);
            double t;
            if (kind == 's')
                t = (double)rounds * (3.0 + (M <= 32 ? 0.55 : 1.05) * (double)((ss + 3) / 4));
            else if (kind == 'M')
                t = (pass == kDgrad ? 1.12 : 1.0) * (double)ss * ((double)(rounds / 2) * 0.95 + (double)(rounds % 2) * 0.85) +
                    3.5 * (double)((rounds + 1) / 2);
            else if (kind == 'D')
                t = (double)rounds * ((double)ss * (0.53 + 0.2 * fill * fill) + 4.0);
            else if (kind == 'L')
                t = (double)rounds * ((double)ss * (1.05 + 0.65 * fill * fill) + 8.0);
            else
                t = (double)rounds * ((double)ss * (0.82 + 0.1 * fill * fill) + (pass == kForward ? 9.0 : 5.0));
            t = std::max(t, 1.0 + (double)(M + N) * (double)K * 2.0 / (5.2e6 * (0.5 + 0.5 * fill)));
            if (s > 1) t += 1.8 + (double)s * (double)M * (double)N * 4.0 / 3.5e6;
            if (best.splits && t >= least) continue;
            least = t;
            best = {kind, (int)ntm, (int)ntn, (int)s, (int)ss, 0, 1, 0};
        }
        // a part of a round left over: its tiles' K in pieces over all compute units
        const int64_t tiles = ntm * ntn, whole = tiles / kDenseCus, rem = tiles % kDenseCus;
        if (kind != 'L' || whole == 0 || rem == 0) continue;
        for (int64_t want = 2; want <= 16 && want <= slabs; ++want) {
            const int64_t ss = (slabs + want - 1) / want, s = (slabs + ss - 1) / ss;
            const int64_t units = rem * s, rounds = (units + kDenseCus - 1) / kDenseCus;
            const double fill = std::min(1.0, (double)units / kDenseCus);
            const double t = (double)whole * ((double)slabs * 1.7 + 8.0) +
                             (double)rounds * ((double)ss * (1.05 + 0.65 * fill * fill) + 8.0) + 1.8 +
                             (double)units * 65536.0 * 4.0 / 3.5e6;
            if (t >= least) continue;
            least = t;
            best = {kind, (int)ntm, (int)ntn, 1, (int)slabs, (int)(whole * kDenseCus), (int)s, (int)ss};
        }
    }
    return best;
}

// Joining K splits: eight lanes side by side on an output where outputs are few and splits
// many, else one.
inline bool dense_join_wide(int64_t items, int splits) { return items <= 8192 && splits >= 4; }

}  // namespace moe
