// Which bytes of an operand the int8 products may load, and which tile shape a
// product takes. Plain C++, constexpr, so that the kernels (gemm_i8.hip) and a
// test on the host take the same functions.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moe {

// Byte offset, from a tile's first row on, of K byte `at` of the tile's row r;
// rows past the operand's last one (`last`, counted from the tile's first) are
// that one again.
constexpr uint32_t row_offset(int r, int last, int K, int at) { return (uint32_t)(r < last ? r : last) * (uint32_t)K + (uint32_t)at; }

// Record count of an operand of n bytes from a tile's first row on. (2^31 - 16
// at most: 256 rows of the longest K end far below that.)
constexpr int records(size_t n) { return n > 0x7FFFFFF0u ? 0x7FFFFFF0 : (int)n; }

// The records that are left from K position k0 >= 0 on. Lane offsets below this
// are loaded, the rest is dropped; offsets, positions and operands are
// multiples of 16 bytes, so a 16-byte access lies on one side. From NOWHERE on
// no operand has any.
constexpr int NOWHERE = 0x7FFFFFF0;
constexpr int records_from(int all, int k0) { return all - k0 > 0 ? all - k0 : 0; }

// The tile shapes, and what they cost (us): a K step of 128 with at most one
// workgroup on each CU (`one`) and with all `per_cu` of them (`full`), and a
// round's prologue and epilogue (`round`). K <= 128 counts as one step; the
// persistent tiles run a second one there, of zeros. One `round` stands for plain
// and gated epilogues, with and without addends, on rows of every
// kind. Large tiles move fewer bytes per output, small ones reach more CUs. The
// figures are a fit to 1100 products
// with random sizes (1..16384 rows, 64..8192 columns, K 128..8192), each timed
// with every shape: where the best takes 5.5 us and more, the shape picked by
// them is 0.6% slower than it on average (below, the five differ by little more
// than two runs of one). E.g. 333 x 1000 x 4112: 32x64 8.9 us, 64x64 11.4,
// 128x128 22; 400 x 2048 x 2048: 64x64 6.7, 32x32 8.3, 128x128 11; 2048^3:
// 128x128 12.6 us, 64x64 21, 256x256 24; 16384 x 2048 x 2048: 256x256 59 us,
// 128x128 71. 256x128 tiles were measured beside these and gain nothing.
struct Shape {
    int tm, tn, per_cu;
    float one, full, round;
};
enum { S_256x256, S_128x128, S_64x64, S_32x64, S_32x32, S_COUNT };
constexpr Shape kShapes[S_COUNT] = {{256, 256, 1, 1.17f, 1.17f, 2.45f},
                                    {128, 128, 2, 0.41f, 0.79f, 1.09f},
                                    {64, 64, 2, 0.10f, 0.41f, 1.13f},
                                    {32, 64, 3, 0.06f, 0.42f, 0.70f},
                                    {32, 32, 2, 0.012f, 0.19f, 1.06f}};

// Tiles of a shape for this many output rows and B rows.
constexpr long long shape_tiles(int shape, int M, long long rows_b) {
    return (M + kShapes[shape].tm - 1LL) / kShapes[shape].tm * ((rows_b + kShapes[shape].tn - 1) / kShapes[shape].tn);
}

// Waves of a workgroup that share one small tile; 0 for the persistent tiles.
// At most one workgroup a CU (`few`): more waves in it (us with eight waves /
// with four: 400 x 2048 x 2048 6.8 / 7.2 and 333 x 1000 x 4112 9.0 / 9.5 so; 978
// x 704 x 5248 gated 21.0 / 17.4 and 481 x 2496 x 1632 11.9 / 9.6 with more
// tiles than CUs).
constexpr int split_waves(int shape, bool few) {
    return shape == S_32x32 ? 8 : shape == S_64x64 || shape == S_32x64 ? (few ? 8 : 4) : 0;
}

// The shape that the costs above make the fastest for this many output rows
// and B rows. Small tiles have a workgroup each, and a launch holds fewer than
// 2^32 threads: where theirs would hold more (2^23 tiles of eight waves, 2^24 of
// four: some 2^29 rows on one side) they are left out; a persistent grid takes
// any number of tiles.
constexpr int pick_shape(int M, long long rows_b, int K, long long cus) {
    const float steps = (float)((K + 127) / 128);
    int best = 0;
    float least = 3.4e38f;
    for (int i = 0; i < S_COUNT; ++i) {
        const Shape& c = kShapes[i];
        const long long tiles = shape_tiles(i, M, rows_b), slots = cus * c.per_cu;
        if (tiles * 64 * split_waves(i, tiles <= cus) >= 1LL << 32) continue;
        const long long rounds = tiles / slots, rest = tiles % slots;
        const float t = (float)rounds * (c.full * steps + c.round) +
                        (rest ? (rest <= cus ? c.one : c.full) * steps + c.round : 0.f);
        if (t < least) {
            least = t;
            best = i;
        }
    }
    return best;
}

}  // namespace moe
