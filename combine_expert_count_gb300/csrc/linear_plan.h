// linear_plan.h -- which kernel a product of 16-bit rows and weights goes to, and in how
// many CTAs.  Plain host code of sizes alone (sms: the device's SMs), so that tests can
// ask it.
#pragma once

#include <cmath>
#include <cstdint>

namespace moe {

// How a product runs.
struct LinearPlan {
    int width;   // > 0: pairs of CTAs, tiles of 256 rows by so many weight rows
    int at;      // else: rows of a CTA
    int parts;   // CTAs of a cluster that share its k, where width is 0
    int stages;  // of a CTA's ring, where width is 0
};

constexpr int kLinearBlock = 64;  // elements of k in 128 bytes
constexpr int kSmem = 232448;  // a CTA's, which has an SM for itself
constexpr int kFewHead = 1280;   // bytes before the ring of a CTA of few rows, at most
constexpr int kFewTile = 16384;  // of weights in a block
// Up to so many rows the parts' sums have room of their own; with more they go where the
// ring was, once all parts are done with theirs.
constexpr int kLinearApart = 64;

// What the kernels take, in ns, fitted to 1560 measured times of 176 sizes, each of which
// went every way (a seventh off as a rule); what is chosen is 1.5% slower than the fastest
// way on average, 27% at most.
//   Few rows: 2.3 us and 24 ns a row that a CTA has (26 with fp32 results), 0.5 us for sums
//   that cross the cluster; the bytes of a CTA's stages at 163 KB/us, or 0.28 us a stage, in
//   quadrature with the operands at 7.1 MB/us; for each further round of CTAs 2.7 us and 22
//   ns a row, or half that where two fit an SM.
//   Tiles: 2.8 us and 15.6 ns an output of the tile; for each block of 64 along k what its
//   products take (1.07 ns an output; with fp32 results 4% more), 0.22 us at least, or its
//   bytes at the pair's share of 15 MB/us; a further tile of the pair's no less than storing
//   one does (1.9 us and 12.4 ns an output).  Rows of outputs that do not start on 16 bytes
//   are stored in 1.28 times as long, of an odd number in 1.9 times.
// us estimated and measured: 61 rows of gate/up of 768 by 2048 5.0 and 5.0, 2048 rows 13.6
// and 14.4; 64 x 256 x 7168 5.2 and 5.2; 2048 x 256 x 7168 in fp32 13.4 and 14.4; 200 x 2048 x
// 2048 7.1 and 7.0.  It is low for the largest tiles: 509 x 7168 x 7168 35.7 and 40.9, 8191 x
// 7168 x 7168 447 and 483 (there the clock falls), 8191 x 256 x 7168 in fp32 30.4 and 36.5, 8191 x
// 2048 x 768 with a residual, which it does not count, 26.0 and 30.1.
// A CTA's shared memory without its ring, a stage's, and its stages.
inline int few_fixed(int at, int parts) {
    const int rows = at / parts < 4 ? 4 : at / parts;
    return kFewHead + (at <= kLinearApart ? parts * rows * 512 : 0);
}
constexpr int few_stage(int at) { return 2 * (kFewTile + at * 128); }
inline int few_stages(int at, int parts, int64_t stages, bool f32) {
    const int fixed = few_fixed(at, parts), stage = few_stage(at);
    const int64_t mine = (stages + parts - 1) / parts;
    int got = (kSmem - fixed) / stage;
    if (got > 6) got = 6;
    if (got > mine) got = (int)mine;
    // Tensor memory goes with shared memory: CTAs that fit an SM by the one fit by the
    // other, and none waits for columns that a later kernel's CTAs hold.
    const int columns = f32 ? 2 * at : at;
    const int sums = at <= kLinearApart ? 1 : (at * 512 + stage - 1) / stage;  // their room
    while (got < sums || fixed + got * stage < columns * (kSmem / 512)) ++got;
    return got;
}

inline double few_cost(int at, int parts, int64_t tiles, int64_t stages, double bytes, bool f32,
                       int sms) {
    const int64_t ctas = tiles * parts;
    const int smem = few_fixed(at, parts) + few_stages(at, parts, stages, f32) * few_stage(at);
    const double waves = (double)((ctas + sms - 1) / sms), fed = few_stage(at) / 163.0;
    const double loop =
        waves * (double)((stages + parts - 1) / parts) * (fed > 280.0 ? fed : 280.0);
    const double hbm = bytes / 7100.0;
    return 2300.0 + (f32 ? 26.0 : 24.0) * at + (parts == 1 ? 0.0 : 500.0) +
           std::sqrt(loop * loop + hbm * hbm) +
           (waves - 1.0) * (2700.0 + 22.0 * at) * (2 * (smem + 1024) <= 233472 ? 0.5 : 1.0);
}

inline double tile_cost(int width, int64_t n, int64_t tiles, int64_t blocks, bool f32, int sms) {
    const int64_t room = sms / 2, full = tiles / room, rest = tiles % room;
    const double stored = width * (n % 8 == 0 ? 1.0 : n % 2 == 0 ? 1.28 : 1.9);
    const double next = 1900.0 + 12.4 * stored;
    const auto loop = [&](int64_t pairs) {
        const double fed = (16384.0 + 64.0 * width) * 2.0 * (double)pairs / 15000.0;
        const double done = 1.07 * width > 220.0 ? 1.07 * width : 220.0;
        return (double)blocks * (fed > done ? fed : done) * (f32 ? 1.04 : 1.0);
    };
    double cost = 2800.0 + 15.6 * stored;
    if (full) cost += loop(room) + (double)(full - 1) * (loop(room) > next ? loop(room) : next);
    if (rest) cost += full && loop(rest) < next ? next : loop(rest);
    return cost;
}

// n: outputs (of each half, where there is a pair of them).
inline LinearPlan linear_plan(int64_t rows, int64_t n, int64_t k, bool pair, bool f32, int sms) {
    const int64_t blocks = (k + kLinearBlock - 1) / kLinearBlock, stages = (blocks + 1) / 2;
    LinearPlan best = {0, 16, 1, 0};
    double least = -1.0;
    const auto take = [&](double cost, int width, int at, int parts) {
        if (least >= 0.0 && cost >= least) return;
        least = cost;
        best = {width, at, parts, 0};
    };
    const double bytes = 2.0 * (double)k * (double)(rows + (pair ? 2 * n : n));
    const int64_t few_n = (n + (pair ? 63 : 127)) / (pair ? 64 : 128);
    for (int at = 16; at <= 128; at *= 2) {
        const int64_t tiles = few_n * ((rows + at - 1) / at);
        take(few_cost(at, 1, tiles, stages, bytes, f32, sms), 0, at, 1);
        // clusters that are on the SMs together: of four all but two of them, of eight all
        // but four (of 152 SMs in groups of 16 to 20)
        for (int parts = 2; parts <= 8; parts *= 2)
            if (parts <= stages && tiles * parts <= sms - (parts == 4 ? 8 : parts == 8 ? 32 : 0))
                take(few_cost(at, parts, tiles, stages, bytes, f32, sms), 0, at, parts);
        if (at >= rows) break;
    }
    if (rows > 128)
        for (int width = pair ? 64 : 32; width <= (f32 ? 128 : 256); width += pair ? 64 : 32) {
            const int64_t outs = pair ? width / 2 : width;
            const int64_t tiles = (n + outs - 1) / outs * ((rows + 255) / 256);
            take(tile_cost(width, n, tiles, blocks, f32, sms), width, 0, 1);
        }
    if (best.width) return best;
    best.stages = few_stages(best.at, best.parts, stages, f32);
    return best;
}

}  // namespace moe
