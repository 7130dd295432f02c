// linear_plan.h -- which kernel a product of 16-bit rows and weights goes to, and in how
// many CTAs.  Plain host code of sizes alone (sms: the device's SMs), so that tests can
// ask it.
#pragma once

#include <cstdint>

namespace moe {

// How a product runs.
struct LinearPlan {
    int width;   // > 0: pairs of CTAs, tiles of 256 rows by so many weight rows
    int at;      // else: rows of a CTA
    int parts;   // CTAs (pairs) of a cluster that share its k
    int stages;  // of a CTA's ring, where width is 0
};

constexpr int kLinearBlock = 64;  // elements of k in 128 bytes
constexpr int kSmem = 232448;  // a CTA's, which has an SM for itself
constexpr int kLinearApart = 64;  // rows of a CTA up to which sums have room beside the ring

// What the kernels take, in ns, from what was measured of them: SMs take in 14.5 MB/us
// together at most (kFabric) and one 150 KB/us.
//   Few rows: 2.6 us and 22 ns a row that a CTA has, 0.3 us for sums that cross the
//   cluster (and 15 ns a row beyond 32, which wait for the ring), and the bytes of a CTA's
//   stages.
//   Tiles: 4.5 us and 13 ns an output of the tile, and for each block of 64 along k what
//   its products take (1.06 ns an output; fp32 results, whose sums are taken out on the
//   way, a quarter more), 170 ns at least, or its bytes.
// us estimated and measured: 61 rows of gate/up of 768 by 2048 5.3 and 5.9; 64 x 256 x 7168
// 5.3 and 5.4; 2048 x 256 x 7168 in fp32 14.6 and 15.7; 200 x 2048 x 2048 11.2 and 10.4; 768 x
// 7168 x 7168 62 and 61; 2048 x 7168 x 7168 120 and 126.  Of 47
// sizes, each measured in every way, the choice is within 13% of the best.
constexpr double kFabric = 14500.0;

inline double few_cost(int at, int parts, int64_t tiles, int64_t stages, int sms) {
    const int64_t ctas = tiles * parts;
    const double active = (double)(ctas < sms ? ctas : sms);
    const double rate = kFabric / active < 150.0 ? kFabric / active : 150.0;
    const double waves = (double)((ctas + sms - 1) / sms);
    return 2600.0 + 22.0 * at + (parts == 1 ? 0.0 : at <= 32 ? 300.0 : 300.0 + 15.0 * at) +
           waves * (double)((stages + parts - 1) / parts) * (32768.0 + 256.0 * at) / rate;
}

inline double tile_block_ns(int width, double pairs, bool f32) {
    const double fed = (16384.0 + 64.0 * width) * 2.0 * pairs / kFabric;
    const double done = 1.06 * width > 170.0 ? 1.06 * width : 170.0;
    return (fed > done ? fed : done) * (f32 ? 1.25 : 1.0);
}

inline double tile_cost(int width, int parts, int64_t tiles, int64_t blocks, bool f32, int sms) {
    const int64_t room = sms / 2, units = tiles * parts, full = units / room, rest = units % room;
    const double per = (double)((blocks + parts - 1) / parts);
    return 4500.0 + 13.0 * width + (parts > 1 ? 1500.0 : 0.0) +
           full * per * tile_block_ns(width, (double)room, f32) +
           (rest ? per * tile_block_ns(width, (double)rest, f32) : 0.0);
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
    const int64_t few_n = (n + (pair ? 63 : 127)) / (pair ? 64 : 128);
    for (int at = 16; at <= 128; at *= 2) {
        const int64_t tiles = few_n * ((rows + at - 1) / at);
        take(few_cost(at, 1, tiles, stages, sms), 0, at, 1);
        // clusters that are on the SMs together: of four all but two of them, of eight all
        // but four (of 152 SMs in groups of 16 to 20)
        for (int parts = 2; parts <= 8; parts *= 2)
            if (parts <= stages && tiles * parts <= sms - (parts == 4 ? 8 : parts == 8 ? 32 : 0))
                take(few_cost(at, parts, tiles, stages, sms), 0, at, parts);
        if (at >= rows) break;
    }
    if (rows > 128)
        for (int width = pair ? 64 : 32; width <= (f32 ? 128 : 256); width += pair ? 64 : 32) {
            const int64_t outs = pair ? width / 2 : width;
            const int64_t tiles = (n + outs - 1) / outs * ((rows + 255) / 256);
            take(tile_cost(width, 1, tiles, blocks, f32, sms), width, 0, 1);
            if (blocks >= 8 && 4 * tiles <= sms - 8)
                take(tile_cost(width, 2, tiles, blocks, f32, sms), width, 0, 2);
        }
    if (best.width) return best;
    const int rows_of = best.at / best.parts < 4 ? 4 : best.at / best.parts;
    const int apart = best.at <= kLinearApart ? best.parts * rows_of * 512 : 0;
    const int stage = 2 * (16384 + best.at * 128);
    const int64_t mine = (stages + best.parts - 1) / best.parts;
    best.stages = (kSmem - 1280 - apart) / stage;
    if (best.stages > 6) best.stages = 6;
    if (best.stages > mine) best.stages = (int)mine;
    // Tensor memory goes with shared memory: CTAs that fit an SM by the one fit by the
    // other, and none waits for columns that a later kernel's CTAs hold.
    const int columns = f32 ? 2 * best.at : best.at;
    const int sums = apart ? 1 : (best.at * 512 + stage - 1) / stage;  // their room
    while (best.stages < sums || 1280 + apart + best.stages * stage < columns * (kSmem / 512))
        ++best.stages;
    return best;
}

}  // namespace moe
