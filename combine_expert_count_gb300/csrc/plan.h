// plan.h -- which kernel a grouped product goes to, and in how many CTAs.  Plain
// host code of sizes alone (sms: the device's SMs), so that tests can ask it.
#pragma once

#include <cstdint>

namespace moe {

constexpr int kTileRows = 128;  // rows of a tile: the lanes of tensor memory

// Rows of an expert that meet its weights at a time in the kernels for few rows, a
// product's columns.  More are several CTAs, whose reads of the weights meet in L2.
constexpr int kThinRowsAt = 16;

// Groups of `at` rows of one expert that there can be, each expert's last being part
// full: at least one for each expert with rows.
inline int64_t row_groups(int64_t N, int64_t cap, int64_t E, int at) {
    const int64_t rows = N * cap, used = rows < E ? rows : E;
    return (rows - used) / at + used;
}

// Whether a product goes to the kernels for few rows.  us there against the 128-row
// tiles:
//   32 rows in all: 7168 x 2048 8.5 : 9.8; 7168 x 7168 16.1 : 19.2; 16 experts of
//   7168 x 2048 39 : 41; gate/up of 2048 by 7168 11.8 : 20.2
//   or all CTAs on the SMs at once: 4096 x 4096, 64 rows 10.6 : 14.1; 128 x 7168, 1024
//   rows 10.4 : 17.4; gate/up of 2048 by 7168, 64 rows 13.9 : 20.3; (not so) 7168 x
//   2048, 96 rows 16.3 : 10.1
//   or at most eight rows an expert, and 512 KB of weights to each CTA: 32 experts'
//   gate/up of 2048 by 7168, 128 rows 145 : 157, of 128 uneven ones of 768 by 2048, 1021
//   rows 64.7 : 65.4; 32 of 2048 x 7168, 256 rows 76.5 : 80.1; (not so, 12 rows each)
//   the last, uneven 83.8 : 80.3; (not so, 96 KB) 128 of 2048 x 768, 512 rows 48 : 43
inline bool few_rows(int64_t N, int64_t cap, int64_t E, int64_t n, int64_t k, bool pair, int sms) {
    const int64_t rows = N * cap;
    return rows <= 32 || (n >> 7) * row_groups(N, cap, E, kThinRowsAt) < sms ||
           (rows <= 8 * E && (pair ? 2 : 1) * k >= 4096);
}

// CTAs that share a unit's k blocks there: as many as the SMs hold at two each, eight
// at most, with a block each at least and one CTA for two or three blocks (us: 2048 x
// 256 3.6 and 4.1 with two; 2048 x 512 4.4 with two and 4.1 with four).  Powers of
// two: clusters of five for four cost a layer of four tokens 211 us for 185 (hidden
// 7168), their CTAs not filling the SMs in pairs.
inline int thin_parts(int64_t units, int64_t blocks, int sms) {
    int parts = 1;
    while (parts < 8 && blocks >= 4 && blocks >= 2 * parts && units * parts * 2 <= 2 * (int64_t)sms)
        parts *= 2;
    return parts;
}

// How a product runs.
struct ProductPlan {
    bool few;       // the kernels for few rows; else tiles of 128 rows
    int64_t units;  // groups of rows: of kThinRowsAt, or of kTileRows
    int wide;       // tiles: column blocks of a tile, 1 or 2
    int64_t tiles;  // as many as there can be
    int parts;      // CTAs that share k
};

// n: all outputs, gate and up (pair) together.
inline ProductPlan product_plan(int64_t N, int64_t cap, int64_t E, int64_t n, int64_t k, bool pair,
                                int sms) {
    const int64_t nb = n >> 7, kb = k >> 7;
    ProductPlan p = {few_rows(N, cap, E, n, k, pair, sms), 0, 1, 0, 1};
    if (p.few) {
        p.units = row_groups(N, cap, E, kThinRowsAt);
        p.tiles = p.units * (pair ? nb >> 1 : nb);
        p.parts = thin_parts(p.tiles, kb, sms);
        return p;
    }
    p.units = row_groups(N, cap, E, kTileRows);
    // one column block a tile where even those have an SM each: half the sums of a k
    // block, and its bound where an SM has one tile (7168 x 2048 at 128 rows 9.6 us,
    // 12.3 with two; 7168 x 7168 22.6, 29.5; 512 x 1024 6.9, 8.6; with up to twice
    // the SMs' tiles 16.5, 13.1 and 40, 30.4 at 512 rows)
    p.wide = pair || p.units * nb > sms ? 2 : 1;
    p.tiles = p.units * ((nb + p.wide - 1) / p.wide);
    // two CTAs to a tile where an SM each is left for them and k is long.  us with one
    // and two: gate/up of 2048 by 7168, 128 rows, 27.4 and 20.5; 7168 x 7168 (narrow
    // tiles) 22.5 and 19.3; k = 4096 14.4 and 13.7; k = 2048 12.0 and 12.3; k = 1024
    // 8.3 and 10.0.  Four: 19.2, 22.6 (wide), 14.0, 15.1, 10.0.
    p.parts = p.tiles * 2 <= sms && kb >= 32 ? 2 : 1;
    return p;
}

}  // namespace moe
