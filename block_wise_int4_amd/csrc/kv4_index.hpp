// kv4_index.hpp -- which rows and keys belong to a sequence: arithmetic on
// values of device memory, which may hold anything.  The same code on the host,
// where it is tested over the values' whole range.
#pragma once

#include "mnb_kv4.hpp"

namespace mnb {
namespace kv4 {

// Length and new tokens of a sequence, within the bounds of the call.
struct Sequence {
    int len, first, count;            // keys; first row and number of new tokens that are computed
    int before;                       // position of the first new token
};
__host__ __device__ __forceinline__ Sequence sequence_of(const KvView& v, int b, int max_q, int max_kv)
{
    Sequence s;
    // a cache without pages holds no keys (elsewhere a page out of range is read as page 0)
    const int64_t room = v.num_pages > 0 ? v.table_stride << v.page_shift : 0;
    int len = v.kv_len[b];
    len = len < 0 ? 0 : len > max_kv ? max_kv : len;
    s.len = (int64_t)len > room ? (int)room : len;
    int first = b, end = b + 1;
    if (v.q_start) {
        first = v.q_start[b];
        end = v.q_start[b + 1];
    }
    // offsets from 0 on have a difference that fits, and one that decreases means no tokens.
    // Positions are below zero however far they are, so they stop at -2^30: max_q is less than that
    first = first < 0 ? 0 : first;
    end = end < first ? first : end;
    const int before = s.len - (end - first);
    s.before = before < -(1 << 30) ? -(1 << 30) : before;
    end = end > v.tokens ? v.tokens : end;
    const int n = end - first;
    s.count = n <= 0 ? 0 : n > max_q ? max_q : n;
    s.first = first;
    return s;
}

// The window as the kernels take it: one that no position of max_kv keys passes is none.
__host__ __device__ __forceinline__ int window_of(int64_t window, int64_t max_kv)
{
    return window < max_kv ? (int)window : 0;
}

// The keys rows of tokens i0..i1 of a sequence can see: [lo, hi).  A window below 2^30
// and positions from -2^30 on keep the differences in 32 bits.
__host__ __device__ __forceinline__ void key_range(int causal, int window, const Sequence& s, int i0, int i1, int& lo, int& hi)
{
    lo = 0;
    hi = s.len;
    if (causal) {
        const int end = s.before + i1 + 1;
        hi = end < hi ? end : hi;
        if (window > 0) {
            const int from = s.before + i0 - window + 1;
            lo = from > 0 ? from : 0;
        }
    }
    hi = hi < lo ? lo : hi;
}

// The keys that rows i0..i1 of a sequence can see, counted without the gap between the
// first tokens that stay visible (`sinks`) and the window: block c of 32 keys in this count is
// block at(c) of the sequence.  lo and hi are in the count's keys, end is the last row's end in the
// sequence's.  Without sinks (negative: none, counted from the sequence's first key) at(c) is c.
struct Span {
    int lead, gap;                    // blocks before the gap, blocks left out
    int lo, hi, end;
    __host__ __device__ __forceinline__ int at(int c) const { return c + (c >= lead ? gap : 0); }
};
__host__ __device__ __forceinline__ Span span_of(int causal, int window, int sinks, const Sequence& s, int i0, int i1)
{
    Span r;
    key_range(causal, window, s, i0, i1, r.lo, r.hi);
    r.lead = r.gap = 0;
    r.end = r.hi;
    if (sinks < 0) return r;
    const int first = r.lo >> 5, most = (int)(((uint32_t)sinks + 31) >> 5);
    r.lead = most < first ? most : first;
    if (r.hi <= r.lo) r.lead = first;          // no row sees a key
    r.gap = first - r.lead;
    r.lo = r.lead > 0 && r.hi > r.lo ? 0 : r.lo - 32 * r.gap;
    r.hi -= 32 * r.gap;
    return r;
}

// No row set of this many rows, of heads that share a key head by `gqa`, has keys past this many
// in its count.
__host__ __device__ __forceinline__ int64_t longest_span(int window, int sinks, int64_t max_kv, int64_t rows, int gqa)
{
    if (sinks < 0 || window == 0) return max_kv;
    const int64_t tokens = (rows + gqa - 2) / gqa + 1;
    const int64_t most = ((int64_t)sinks + 31) / 32 * 32 + 31 + window + tokens - 1;
    return most < max_kv ? most : max_kv;
}

// A round of a wave's search among `batch` ends of sequences: lane i looks at
// the end of sequence at(i) - 1 if the range holds it, and keep() takes the number of lanes
// whose end is not past the token.  Unsigned: 64 steps may pass 2^31.
struct Search {
    uint32_t lo, n, step;             // ends of sequences lo .. lo + n - 1 are open
    __host__ __device__ __forceinline__ uint32_t at(int lane) const { return lo + (uint32_t)(lane + 1) * step; }
    __host__ __device__ __forceinline__ bool holds(uint32_t at) const { return at <= lo + n; }
    __host__ __device__ __forceinline__ void keep(int lanes)
    {
        const uint32_t left = lo + n;
        lo += (uint32_t)lanes * step;
        n = left - lo < step - 1 ? left - lo : step - 1;
        step = (n + 63) / 64;
    }
};
__host__ __device__ __forceinline__ Search search_of(int batch)
{
    return Search{0, (uint32_t)batch, ((uint32_t)batch + 63) / 64};
}

}  // namespace kv4
}  // namespace mnb
