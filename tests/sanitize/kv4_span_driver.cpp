// Host-side run, under AddressSanitizer and UndefinedBehaviorSanitizer, of the
// attention's count of keys without the gap between the first tokens that stay
// visible and the window: small shapes against the definition key by key, wide
// ones for their bounds, and the plan that cuts the count.  Built as plain C++.
#include <cstdio>
#include <cstring>
#include <vector>

#include "kv4_plan.hpp"

using namespace mnb;

static int failures = 0;
static void expect(bool good, const char* what)
{
    if (!good && ++failures < 20) std::printf("FAIL %s\n", what);
}

static kv4::Sequence sequence(int len, int tokens, int max_q)
{
    kv4::Sequence s;
    s.len = len;
    s.first = 0;
    s.count = tokens < max_q ? tokens : max_q;
    s.before = len - tokens < -(1 << 30) ? -(1 << 30) : len - tokens;
    return s;
}

// The blocks of the count are those with a key that a row sees, and no other, each once.
static void blocks()
{
    for (int len : {0, 1, 31, 32, 33, 100, 257, 300})
        for (int tokens : {1, 2, 40, 90, 320})
            for (int window : {0, 1, 2, 31, 32, 33, 64, 90, 200})
                for (int sinks : {0, 1, 4, 31, 32, 33, 64, 95, 96, 97, 150, 299, 1000})
                    for (int i0 : {0, 1, 30, 63})
                        for (int i1 : {i0, i0 + 1, i0 + 31, i0 + 100}) {
                            const kv4::Sequence s = sequence(len, tokens, 1000);
                            if (i1 >= s.count) continue;
                            const int w = kv4::window_of(window, len);
                            const kv4::Span p = kv4::span_of(1, w, sinks, s, i0, i1);
                            std::vector<char> want(400 / 32 + 1, 0), got(want);
                            int end = 0;
                            for (int i = i0; i <= i1; ++i)
                                for (int j = 0; j < len; ++j) {
                                    const int at = len - tokens + i;
                                    if (j <= at && (window == 0 || j > at - window || j < sinks)) {
                                        want[j / 32] = 1;
                                        end = j + 1 > end ? j + 1 : end;
                                    }
                                }
                            expect(p.lo <= p.hi && p.lo >= 0 && p.gap >= 0 && p.lead >= 0, "the count's ends");
                            if (p.lo < p.hi) {
                                expect(p.end == end, "the last key");
                                for (int c = p.lo >> 5; c < (p.hi + 31) >> 5; ++c) {
                                    expect(!got[p.at(c)], "once");
                                    got[p.at(c)] = 1;
                                }
                                const int last = p.at(((p.hi + 31) >> 5) - 1);
                                expect(last == (end - 1) / 32 && p.hi - 1 - (p.hi - 1) / 32 * 32 == (end - 1) % 32, "its place");
                            }
                            // first keys that no row sees may share the window's blocks only
                            expect(got == want, "the blocks");
                            const int64_t most = kv4::longest_span(w, sinks, len, i1 - i0 + 1, 1);
                            expect(p.hi <= most, "the longest count");
                        }
}

// Without sinks (-1) the count is the sequence's own.
static void alone()
{
    for (int len : {0, 1, 100, 300})
        for (int window : {0, 1, 33, 90})
            for (int i : {0, 5}) {
                const kv4::Sequence s = sequence(len, 9, 9);
                int lo, hi;
                key_range(1, window, s, i, i + 2, lo, hi);
                const kv4::Span p = kv4::span_of(1, window, -1, s, i, i + 2);
                expect(p.lo == lo && p.hi == hi && p.end == hi && p.gap == 0 && p.at(7) == 7, "as it was");
            }
}

// Lengths, windows and sinks over their range: the count stays inside the sequence.
static void wide()
{
    const int v[] = {0, 1, 31, 32, 33, 1000, (1 << 30) - 33, (1 << 30) - 1, 1 << 30};
    for (int len : v)
        for (int tokens : {1, 7, 1000, 1 << 30, INT32_MAX})
            for (int window : v)
                for (int sinks : v)
                    for (int i0 : {0, 5, 900, (1 << 29) - 300})
                        for (int i1 : {i0, i0 + 255}) {
                            const kv4::Sequence s = sequence(len, tokens, (1 << 29) - 1);
                            if (i1 >= s.count) continue;
                            const int w = kv4::window_of(window, len);
                            const kv4::Span p = kv4::span_of(1, w, sinks, s, i0, i1);
                            expect(p.lo >= 0 && p.lo <= p.hi && p.hi <= len && p.end <= len, "inside");
                            if (p.lo < p.hi) expect(p.at(((p.hi + 31) >> 5) - 1) * 32 < len, "its last block");
                            expect(p.hi <= kv4::longest_span(w, sinks, len, (int64_t)(i1 - i0 + 1) * 8, 8), "the longest count");
                        }
}

// Every key of the longest count is in a split, whatever the row set.
static void plans()
{
    for (int heads : {1, 2, 7, 8, 96})
        for (int kv_heads : {1, 8})
            for (int dim : {64, 128, 256})
                for (int groups : {1, 2, 4, 8})
                    for (int64_t batch : {1, 3, 64, 65535})
                        for (int64_t max_q : {1, 2, 5, 33, 2048, 100000})
                            for (int64_t max_kv : {(int64_t)0, (int64_t)1, (int64_t)700, (int64_t)5000, (int64_t)1 << 17, (int64_t)1 << 30})
                                for (int64_t window : {(int64_t)0, (int64_t)1, (int64_t)100, (int64_t)4096, (int64_t)1 << 40})
                                    for (int64_t sinks : {(int64_t)0, (int64_t)4, (int64_t)300, (int64_t)1 << 40}) {
                                        AttentionArgs a = {};
                                        a.v.q_heads = heads * kv_heads;
                                        a.v.kv_heads = kv_heads;
                                        a.v.head_dim = dim;
                                        a.v.groups = groups;
                                        a.v.batch = (int)batch;
                                        a.max_q = max_q;
                                        a.max_kv = max_kv;
                                        a.window = window;
                                        a.sinks = sinks;
                                        const kv4::Plan c = kv4::plan_of(a);
                                        const int w = kv4::window_of(window, max_kv);
                                        const int k = (int)(sinks < max_kv ? sinks : max_kv);
                                        const int64_t rows = max_q * heads;
                                        const int64_t set = c.rows < rows ? c.rows : rows;
                                        expect(c.splits >= 1 && c.splits <= kv4::kMaxSplits && c.chunk % 128 == 0, "splits");
                                        expect((int64_t)c.splits * c.chunk >= kv4::longest_span(w, k, max_kv, set, heads), "all keys");
                                        expect((int64_t)c.row_tiles * c.rows >= rows, "all rows");
                                        if (c.kind == 0) expect(c.splits == 1, "one workgroup");
                                    }
}

int main(int argc, char** argv)
{
    struct { const char* name; void (*run)(); } parts[] = {{"blocks", blocks}, {"alone", alone}, {"wide", wide}, {"plans", plans}};
    for (auto& p : parts)
        if (argc < 2 || !std::strcmp(argv[1], p.name)) p.run();
    std::printf("%s: %d failures\n", failures ? "FAILED" : "ok", failures);
    return failures ? 1 : 0;
}
