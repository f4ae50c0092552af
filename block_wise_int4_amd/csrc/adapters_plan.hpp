// adapters_plan.hpp -- how a call of the adapters is cut into workgroups: host
// code, a function of the call's sizes alone.
#pragma once

#include <stdint.h>

namespace mnb {
namespace adapters {

constexpr int kDownWaves = 8;        // waves of the first product's workgroup
constexpr int kUpWaves = 4;          // of the second's, 64 columns each
constexpr int kMaxRank = 128;

struct Plan {
    int splits;                      // workgroups that share k
    int64_t k_per;                   // k of a split, a multiple of a step
    int down_slots, up_slots;        // workgroups that share the adapters of 64 rows
    int pitch;                       // floats of a row between the products
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline Plan plan_of(int64_t m, int64_t n, int64_t k, int rank, int count, int f16)
{
    Plan c = {};
    const int step = f16 ? 64 : 32;  // k of a wave's step
    c.pitch = (rank + 15) / 16 * 16;
    const int64_t tiles = ceil_div(m, 64);
    const int64_t most = ceil_div(k, (int64_t)step * kDownWaves);
    int64_t splits = ceil_div(512, tiles);
    splits = splits > most ? most : splits;
    splits = splits > 8 ? 8 : splits;
    c.k_per = ceil_div(ceil_div(k, splits), step) * step;
    c.splits = (int)ceil_div(k, c.k_per);
    // adapters that 64 rows can have
    int64_t distinct = m < 64 ? m : 64;
    distinct = distinct < count ? distinct : count;
    auto slots = [&](int64_t workgroups) {
        const int64_t s = ceil_div(1024, workgroups);
        return (int)(s > distinct ? (distinct < 1 ? 1 : distinct) : s);
    };
    c.down_slots = slots(tiles * c.splits);
    c.up_slots = slots(tiles * ceil_div(n, 64 * kUpWaves));
    return c;
}

}  // namespace adapters
}  // namespace mnb
