// adapters_plan.hpp -- how a call of the adapters is cut into workgroups: host
// code, a function of the call's sizes alone.
#pragma once

#include <stdint.h>

namespace mnb {
namespace adapters {

constexpr int kDownWaves = 4;        // waves of the first product's workgroup
constexpr int kUpWaves = 4;          // of the second's, 64 columns each
constexpr int kOneWaves = 8;         // of the kernel of both
constexpr int kMaxRank = 128;

struct Plan {
    bool one;                        // both products in one launch
    int splits;                      // workgroups that share k
    int64_t k_per;                   // k of a split, a multiple of a step
    int down_tile, up_tile;          // rows of a workgroup: 16, 32, 64
    int down_ranks;                  // 16-rank tiles of one: 1, 2, 4
    int one_slots, down_slots, up_slots;   // workgroups that share the adapters of its rows
    int up_blocks;                   // 256-column blocks of a workgroup of the second product
    int pitch;                       // floats of a row between the products
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline Plan plan_of(int64_t m, int64_t n, int64_t k, int rank, int count, int f16)
{
    Plan c = {};
    const int step = f16 ? 64 : 32;  // k of a wave's step
    c.pitch = rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128;
    const int64_t tiles = ceil_div(m, 64);
    // more splits fill the chip, and each adds a row of h to what the second product reads (8416
    // rows, rank 32, k = 4096: 91.9, 89.0, 90.7, 95.9 us with 1, 2, 4, 8; 82 rows, rank 64, k = 11008: 19.3, 16.1, 16.0
    // with 4, 8, 16; 64 rows of 64 adapters, rank 16, k = 8192: 17.9, 15.8, 14.1, 16.8 with 2, 4, 8, 16)
    const int64_t most = ceil_div(k, (int64_t)step * kDownWaves);
    int64_t splits = ceil_div(512, tiles);
    splits = splits > most ? most : splits;
    splits = splits > 8 ? 8 : splits;
    // every 256 columns of the second product read all of h: past 48 MB that costs more than the splits
    // gain (4000 rows, k = n = 4096, fp16: rank 64 in eight 43.3 us, in four 39.2, in two 38.7;
    // rank 128 64.8, 54.4, 52.3, in one 53.8; 1000 fp32 rows of rank 64, 33 MB, 26.9 in eight, 25.7 in four)
    const int64_t fewest = rank > 64 ? 2 : 4;
    while (splits > fewest && m * splits * c.pitch * 4 * ceil_div(n, 64 * kUpWaves) > ((int64_t)48 << 20))
        splits = (splits + 1) / 2 < fewest ? fewest : (splits + 1) / 2;
    c.k_per = ceil_div(ceil_div(k, splits), step) * step;
    c.splits = (int)ceil_div(k, c.k_per);
    // adapters that `rows` rows can have
    auto distinct = [&](int64_t rows) {
        const int64_t d = m < rows ? m : rows;
        return count < 1 ? (int64_t)1 : d < count ? d : count;
    };
    // One launch while a CU has one adapter to see to and reads its A quickly: from 64 KB on it takes as long as
    // two, and few rows still gain the enqueue that their caller is spared (k = n = 4096, rank 16, in a graph and
    // call by call: one token 6.8 and 7.0 us against 7.0 and 9.6, 32 rows of 24 adapters 8.5 and 7.6 against 8.8 and 11.0,
    // 32 rows of one 9.0 against 7.3; k = n = 1024 5.9 against 8.1; 575 fp32 rows, 131 KB, 15.1 against 13.2).
    // Above it two are better, in a graph, one launch and two, one token and 32 rows of 24 adapters: 163 KB (k = 5120) 8.5
    // and 8.3, 9.8 and 10.1; 262 KB as k = 8192 10.2 and 8.6, as rank 32 9.4 and 8.3, 10.8 and 10.7, in fp32 12.3 and 8.8,
    // 14.0 and 11.0.
    const int64_t sets = ceil_div(m, 32) * ceil_div(n, 64 * kOneWaves);
    c.one = rank <= 32 && k * c.pitch * (f16 ? 2 : 4) <= (m <= 64 ? 144 : 64) * 1024 && sets * distinct(32) <= 256;
    auto slots = [&](int64_t workgroups, int64_t most, int64_t rows) {
        const int64_t s = most / workgroups < 1 ? 1 : most / workgroups;
        return (int)(s < distinct(rows) ? s : distinct(rows));
    };
    c.one_slots = slots(sets, 256, 32);
    // slots for the workgroups that the CUs hold at once (512 rows of 64 adapters, k = n = 4096: rank 16
    // 38 us with 1024, 46 with 512; rank 64 75 with 512, 81 with 1024)
    const int64_t held = rank <= 32 ? 1024 : 512;
    // 64 rows read A and B least often; with fewer workgroups than keep the memory busy 32 are
    // better (1000 rows of one adapter, k = n = 4096: second product 7.8 and 6.9 us, 8416 rows 83
    // and 88; first, 3100 rows 10.8 and 9.0, 8416 rows 18.0 and 19.9), and 16, then fewer ranks, until
    // there is one for every CU (121 rows, rank 64 in fp32: first 18 and 6.5 us, second 17 and 8)
    c.down_ranks = rank <= 16 ? 1 : rank <= 32 ? 2 : 4;
    auto down = [&] { return ceil_div(m, c.down_tile) * c.splits * ceil_div(rank, 16 * c.down_ranks); };
    c.down_tile = 64;
    if (down() <= 384) c.down_tile = 32;
    c.down_slots = slots(down(), held, c.down_tile);
    if (down() * c.down_slots < 256) {
        c.down_tile = 16;
        c.down_slots = slots(down(), held, c.down_tile);
    }
    while (c.down_ranks > 1 && down() * c.down_slots < 256) c.down_ranks /= 2;
    auto up = [&] { return ceil_div(m, c.up_tile) * ceil_div(n, 64 * kUpWaves); };
    c.up_tile = 64;
    if (up() < 1024) c.up_tile = 32;
    c.up_slots = slots(up(), held, c.up_tile);
    if (up() * c.up_slots < 256) {
        c.up_tile = 16;
        c.up_slots = slots(up(), held, c.up_tile);
    }
    // At ranks above 32 h is long to read: two blocks of columns a workgroup where there is more than a
    // round of workgroups, two a CU (4000 rows, rank 128: 57 us and 50; 1500 rows 29.0 and 27.8; rank 64 41.3
    // and 39.7; 1000 rows, 512 workgroups, 17.3 and 20.1.  Rank 32 gains nothing)
    c.up_blocks = rank > 32 && up() * c.up_slots > 512 ? 2 : 1;
    return c;
}

}  // namespace adapters
}  // namespace mnb
