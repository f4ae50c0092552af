// Host-side run, under AddressSanitizer and UndefinedBehaviorSanitizer, of the
// arithmetic that the cache's and the attention's kernels do on lengths and
// offsets from device memory: whatever these hold, rows and keys stay inside
// the call's arrays.  Built as plain C++.
#include <cstdio>
#include <cstring>
#include <vector>

#include "kv4_index.hpp"

using namespace mnb;

static int failures = 0;
static void expect(bool good, const char* what)
{
    if (!good && ++failures < 20) std::printf("FAIL %s\n", what);
}

static KvView view(const int32_t* kv_len, const int32_t* q_start, int batch, int tokens, int64_t table_stride, int num_pages)
{
    KvView v = {};
    v.kv_len = kv_len;
    v.q_start = q_start;
    v.batch = batch;
    v.tokens = tokens;
    v.table_stride = table_stride;
    v.page_shift = 5;
    v.num_pages = num_pages;
    return v;
}

// A cache without pages has no keys, whatever the lengths say.
static void no_pages()
{
    const int32_t lens[] = {100, 1, INT32_MAX, 0, -3};
    for (int b = 0; b < 5; ++b) {
        const kv4::Sequence s = kv4::sequence_of(view(lens, nullptr, 5, 5, 40, 0), b, 1, 1000);
        expect(s.len == 0 && s.first == b && s.count == 1 && s.before == -1, "no pages");
        const kv4::Sequence one = kv4::sequence_of(view(lens, nullptr, 5, 5, 40, 1), b, 1, 1000);
        expect(one.len == (lens[b] < 0 ? 0 : lens[b] < 1000 ? lens[b] : 1000), "a page");
    }
}

// Offsets of any two values: rows inside the call's, none where the offsets
// decrease, positions by the formula as far as 32 bits hold them.
static void offsets()
{
    const int32_t v[] = {INT32_MIN, INT32_MIN + 1, INT32_MIN + 7, -(1 << 30), -100, -1, 0, 1, 5, 60, 99, 100, 101, 1 << 30,
                         INT32_MAX - 1, INT32_MAX};
    const int32_t lens[] = {INT32_MIN, -1, 0, 1, 77, 1 << 30, INT32_MAX};
    for (int32_t len : lens)
        for (int32_t first : v)
            for (int32_t end : v)
                for (int max_q : {1, 40, (1 << 29) - 1})
                    for (int max_kv : {0, 50, 1 << 30}) {
                        const int32_t q_start[] = {first, end};
                        const int tokens = 100;
                        const kv4::Sequence s = kv4::sequence_of(view(&len, q_start, 1, tokens, 1 << 26, 9), 0, max_q, max_kv);
                        expect(s.len >= 0 && s.len <= max_kv, "length");
                        expect(s.count >= 0 && s.count <= max_q, "count");
                        expect(s.count == 0 || (s.first >= 0 && s.first + s.count <= tokens), "rows");
                        expect(first < end || s.count == 0, "decreasing offsets");
                        expect(s.before >= -(1 << 30) && s.before <= s.len, "position");
                        if (first >= 0 && end >= first && end <= tokens) {
                            expect(s.before == s.len - (end - first), "the formula");
                            expect(s.count == (end - first < max_q ? end - first : max_q), "all rows");
                            expect(s.count == 0 || s.first == first, "first row");
                        }
                    }
}

// The search for a token's sequence by 64 lanes, for batches up to the largest:
// every offset looked at is one of the batch's, and the sequence is found.
static void search()
{
    for (int batch : {1, 2, 63, 64, 65, 700, 4096, 4097, 1 << 24, INT32_MAX - 65, INT32_MAX - 64, INT32_MAX - 2, INT32_MAX - 1})
        for (int per : {1, 3, 200, 1 << 28})                       // sequences to a token
            for (int64_t token : {(int64_t)0, (int64_t)1, (int64_t)5, (int64_t)batch / per / 2, (int64_t)batch / per - 1,
                                  (int64_t)batch / per, (int64_t)batch / per + 1}) {
                if (token < 0) continue;
                auto q_start = [&](uint32_t i) {
                    expect(i >= 1 && i <= (uint32_t)batch, "an offset of the batch");
                    return (int64_t)(i / (uint32_t)per);
                };
                kv4::Search s = kv4::search_of(batch);
                int rounds = 0;
                while (s.n > 0 && ++rounds < 20) {
                    int lanes = 0;
                    for (int lane = 0; lane < 64; ++lane) {
                        const uint32_t at = s.at(lane);
                        lanes += s.holds(at) && q_start(at) <= token;
                    }
                    s.keep(lanes);
                }
                const int64_t ends = (token + 1) * per - 1;        // of i / per <= token
                expect(rounds <= 6 && s.lo == (uint32_t)(ends < batch ? ends : batch), "the sequence");
            }
}

// The keys of rows under a window of any width, against the definition.
static void windows()
{
    const int64_t widths[] = {0, 1, 2, 31, 32, 1000, (1 << 30) - 1, 1 << 30, INT32_MAX - 1000, INT32_MAX - 1, INT32_MAX,
                              (int64_t)INT32_MAX + 1, INT64_MAX};
    const int32_t lens[] = {0, 1, 5, 33, 100, 1 << 30, INT32_MAX};
    for (int32_t len : lens)
        for (int32_t tokens : {1, 3, 20, 1000, INT32_MAX})
            for (int max_kv : {0, 1, 33, 1 << 30})
                for (int64_t width : widths)
                    for (int i0 : {0, 1, 19, 511, (1 << 29) - 2})
                        for (int i1 : {i0, i0 + 1, (1 << 29) - 1}) {
                            const int32_t q_start[] = {0, tokens};
                            const KvView v = view(&len, q_start, 1, tokens, 1 << 26, 9);
                            const kv4::Sequence s = kv4::sequence_of(v, 0, (1 << 29) - 1, max_kv);
                            if (i1 >= s.count) continue;
                            const int window = kv4::window_of(width, max_kv);
                            int lo, hi;
                            kv4::key_range(1, window, s, i0, i1, lo, hi);
                            const int64_t first = (int64_t)s.len - tokens;
                            int64_t from = 0, to = first + i1 + 1;     // of every row i0..i1 together
                            if (width > 0 && first + i0 + 1 > width) from = first + i0 + 1 - width;
                            to = to > s.len ? s.len : to;
                            expect(lo <= hi && (lo == hi ? to <= from : lo == from && hi == to), "keys of the rows");
                        }
}

int main(int argc, char** argv)
{
    struct { const char* name; void (*run)(); } parts[] = {{"no_pages", no_pages}, {"offsets", offsets}, {"search", search}, {"windows", windows}};
    for (auto& p : parts)
        if (argc < 2 || !std::strcmp(argv[1], p.name)) p.run();
    std::printf("%s: %d failures\n", failures ? "FAILED" : "ok", failures);
    return failures ? 1 : 0;
}
