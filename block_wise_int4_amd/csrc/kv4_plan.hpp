// kv4_plan.hpp -- how an attention call is cut into workgroups: host code, a
// function of the call's shapes alone.
#pragma once

#include "mnb_kv4.hpp"

namespace mnb {
namespace kv4 {

constexpr int kPromptWaves = 8;       // waves of the many-rows kernel's workgroup
constexpr int kMaxSplits = 512;

// How a call is cut.
struct Plan {
    int kind;                         // 0: one workgroup a row set; 1: few rows; 2: many rows
    int group;                        // few rows: column groups (4, 2, 1), 0 for two row tiles
    int tiles;                        // many rows: column tiles of a wave
    int rows;                         // rows per workgroup
    int row_tiles, splits, chunk;
};

inline Plan plan_of(const AttentionArgs& a)
{
    Plan c = {};
    const int64_t rows = a.max_q * (a.v.q_heads / a.v.kv_heads);
    const bool wide = a.v.head_dim == 256;
    // keys worth a split, in steps of grain; workgroups that fill the chip
    int64_t least = 256, grain = 256, want;
    if (rows <= (wide || a.v.groups > 2 ? 16 : 32)) {   // two column tiles where the registers hold them
        // few rows: the waves of a workgroup cut the keys between them (32 rows, 16
        // sequences of 4000 keys: 37 us, 55 with the many-rows kernel).  Rows repeated over the
        // idle columns, against 16 columns of which 4 are used: 82 and 125 us for 16
        // sequences of 8192 keys at head_dim 256, groups of 32, fp32; 32.5 and 36.7 for 32 at
        // head_dim 64; 42.7 and 42.9 at head_dim 128 with groups of 128, which memory bounds
        c.group = rows <= 4 ? 4 : rows <= 8 ? 2 : rows <= 16 ? 1 : 0;
        c.rows = c.group ? 16 / c.group : 32;
        // up to 1024 keys one workgroup of 8 waves does without the join (1000 keys: 10.1 us
        // against 11.4, 64 sequences of them 20.4 against 23.4; 2000 keys: 14.0 against 10.7)
        c.kind = !wide && a.v.groups <= 2 && c.group && a.max_kv <= 1024 ? 0 : 1;
        // one sequence: its pieces are alike, and two workgroups a CU in one round
        // are best (131072 keys: 34 us with 512, 44 with 2048); several of unknown
        // lengths: more and shorter pieces even them out (32 sequences of up to 8192 keys:
        // 45 us with 512, 41 with 3072)
        want = a.v.batch == 1 ? 512 : 3072;
    } else {
        c.kind = 2;
        // two column tiles a wave where that leaves a workgroup for every CU (1000
        // rows of 32 key heads: 90 us with two, 34 with one; 2048 and 1100 tokens of 8
        // key heads by 4: 233 us with two, 306 with one) and the registers hold them
        const int64_t wgs = (rows + 255) / 256 * a.v.kv_heads * a.v.batch;
        c.tiles = wide || a.v.groups > 2 || wgs < 256 ? 1 : 2;
        c.rows = kPromptWaves * 16 * c.tiles;
        // one workgroup a CU, so splits that make a second round gain nothing (800 new
        // tokens of 8000 keys, 200 workgroups: 196 us whole, 271 in two)
        want = 256;
        // and many rows' partials cost as much as some hundred keys (300 tokens of 32 heads,
        // no prefix: 14.8 us whole, 21 in two; 33 tokens with 1000 keys: 17 us in four, 23 in two)
        least = a.max_q * a.v.q_heads * a.v.batch <= 4096 ? 256 : 512;
        grain = 128;                           // a stage of the kernel, or more
    }
    c.row_tiles = (int)((rows + c.rows - 1) / c.rows);
    const int64_t units = (int64_t)c.row_tiles * a.v.kv_heads * a.v.batch;
    const int64_t most = (a.max_kv + least - 1) / least;
    int64_t splits = c.kind == 0 ? 1 : c.kind == 1 ? (want + units - 1) / units : want / units;
    splits = splits > most ? most : splits;
    splits = splits > kMaxSplits ? kMaxSplits : splits < 1 ? 1 : splits;
    c.chunk = (int)(((a.max_kv + splits - 1) / splits + grain - 1) / grain * grain);
    if (c.chunk < grain) c.chunk = (int)grain;
    c.splits = (int)((a.max_kv + c.chunk - 1) / c.chunk);
    if (c.splits < 1) c.splits = 1;
    return c;
}

}  // namespace kv4
}  // namespace mnb
