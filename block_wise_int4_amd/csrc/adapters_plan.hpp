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
    int one_slots;                   // workgroups that share the adapters of 32 rows,
    int down_slots, up_slots;        // and of 64
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
    // rows, rank 32, k = 4096: 110, 105, 111 us with 2, 4, 8; 32 rows, rank 16: 11.3, 9.7, 9.2, and 9.7 with 16)
    const int64_t most = ceil_div(k, (int64_t)step * kDownWaves);
    int64_t splits = ceil_div(512, tiles);
    splits = splits > most ? most : splits;
    splits = splits > 8 ? 8 : splits;
    c.k_per = ceil_div(ceil_div(k, splits), step) * step;
    c.splits = (int)ceil_div(k, c.k_per);
    // adapters that `rows` rows can have
    auto distinct = [&](int64_t rows) {
        const int64_t d = m < rows ? m : rows;
        return count < 1 ? (int64_t)1 : d < count ? d : count;
    };
    // one launch while a CU has one adapter to see to and reads its A quickly (one token, k = n = 4096,
    // rank 16: 6.6 us against 7.0; 32 rows of 24 adapters 8.5 against 9.2, with k = 1024 columns 7.5
    // against 8.5; n = 11008, 22 sets of columns, 14.7 against 11.2; fp32, 256 KB, 13.4 against 11.5).  A call of one
    // launch also spares its caller an enqueue.
    const int64_t sets = ceil_div(m, 32) * ceil_div(n, 64 * kOneWaves);
    c.one = rank <= 32 && k * c.pitch * (f16 ? 2 : 4) <= 144 * 1024 && sets * distinct(32) <= 256;
    // a workgroup without an adapter costs a quarter of a microsecond of its CU: few where there are many tiles
    auto slots = [&](int64_t workgroups, int64_t most, int64_t rows) {
        const int64_t s = most / workgroups < 1 ? 1 : most / workgroups;
        return (int)(s < distinct(rows) ? s : distinct(rows));
    };
    c.one_slots = slots(sets, 256, 32);
    c.down_slots = slots(tiles * c.splits, 1024, 64);
    c.up_slots = slots(tiles * ceil_div(n, 64 * kUpWaves), 1024, 64);
    return c;
}

}  // namespace adapters
}  // namespace mnb
