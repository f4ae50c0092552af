// adapters_plan.hpp -- how a call of the adapters is cut into workgroups: host
// code, a function of the call's sizes alone.
#pragma once

#include <stdint.h>

namespace mnb {
namespace adapters {

constexpr int kDownWaves = 8;        // waves of the first product's workgroup
constexpr int kMaxRank = 128;

struct Plan {
    int tiles16;                     // 16-row tiles of the first product's workgroup: 1, 2
    int splits;                      // workgroups that share k
    int64_t k_per;                   // k of a split, a multiple of a step
    int down_slots;                  // workgroups that share a tile's adapters
    int span;                        // 16-row tiles of the second product's workgroup
    int up_waves;                    // its waves, 64 columns each
    int up_slots;
    int pitch;                       // floats of a row between the products
};

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline Plan plan_of(int64_t m, int64_t n, int64_t k, int rank, int count, int f16)
{
    Plan c = {};
    const int step = f16 ? 64 : 32;  // k of a wave's step
    c.pitch = (rank + 15) / 16 * 16;
    c.tiles16 = m >= 4096 ? 2 : 1;
    const int64_t rows = 16 * c.tiles16, tiles = ceil_div(m, rows);
    const int64_t most = ceil_div(k, (int64_t)step * kDownWaves);
    int64_t splits = ceil_div(512, tiles);
    splits = splits > most ? most : splits;
    splits = splits > 8 ? 8 : splits;
    c.k_per = ceil_div(ceil_div(k, splits), step) * step;
    c.splits = (int)ceil_div(k, c.k_per);
    const int64_t distinct = rows < count ? (rows < m ? rows : m) : (count < m ? count : m);
    int64_t slots = ceil_div(2048, tiles * c.splits);
    c.down_slots = (int)(slots < distinct ? slots : distinct);
    if (c.down_slots < 1) c.down_slots = 1;      // an empty set
    c.span = m >= 1024 ? 8 : 1;
    c.up_waves = m >= 1024 ? 4 : 1;
    const int64_t wgs = ceil_div(ceil_div(m, 16), c.span) * ceil_div(n, 64 * c.up_waves);
    const int64_t distinct16 = distinct < 16 ? distinct : 16;
    slots = ceil_div(2048, wgs);
    c.up_slots = (int)(slots < distinct16 ? slots : distinct16);
    if (c.span > 1 || c.up_slots < 1) c.up_slots = 1;
    return c;
}

}  // namespace adapters
}  // namespace mnb
