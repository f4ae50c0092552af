// Host-side run of the calls between the products under AddressSanitizer and
// UndefinedBehaviorSanitizer: argument checks with random and extreme values,
// and the attention's plan over its whole range.  Built as plain C++: the
// launchers are stubs that are never reached, because the device check fails.
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "kv4_plan.hpp"
#include "mnb.h"
#include "mnb_api_common.hpp"
#include "mnb_kv4.hpp"

static char last[600];

namespace mnb {
namespace api {
mnb_status fail(mnb_status s, const char* fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(last, sizeof(last), fmt, ap);
    va_end(ap);
    return s;
}
mnb_status ok(const char*) { last[0] = 0; return MNB_OK; }
mnb_status check_ptr(const void* p, uintptr_t align, const char* name)
{
    if (!p || (reinterpret_cast<uintptr_t>(p) & (align - 1))) return fail(MNB_ERR_INVALID_ARGUMENT, "%s", name);
    return MNB_OK;
}
mnb_status check_device() { return fail(MNB_ERR_DEVICE, "no device"); }
mnb_status launched(hipError_t, const char*) { std::abort(); }
}  // namespace api
hipError_t launch_rms_norm(const NormArgs&, hipStream_t, const char**) { std::abort(); }
hipError_t launch_kv4_append(const AppendArgs&, hipStream_t, const char**) { std::abort(); }
hipError_t launch_kv4_read(const ReadArgs&, hipStream_t, const char**) { std::abort(); }
hipError_t launch_kv4_attention(const AttentionArgs&, hipStream_t, const char**) { std::abort(); }
size_t kv4_attention_workspace(const AttentionArgs& a)
{
    const kv4::Plan c = kv4::plan_of(a);
    return c.splits == 1 ? 0 : (size_t)c.splits * a.v.tokens * a.v.q_heads * (a.v.head_dim + 2) * 4;
}
}  // namespace mnb

static int failures = 0;
static uint64_t seed = 88172645463325252ull;
static uint64_t next()
{
    seed ^= seed << 13;
    seed ^= seed >> 7;
    seed ^= seed << 17;
    return seed;
}
static int64_t wild()
{
    static const int64_t v[] = {0, 1, -1, 2, 16, 31, 32, 64, 127, 128, 255, 256, 1000, 4096, 65535, 65536, 1 << 24,
                                INT32_MAX, (int64_t)INT32_MAX + 1, (int64_t)1 << 40, INT64_MAX, INT64_MIN, INT32_MIN};
    return v[next() % (sizeof(v) / sizeof(v[0]))];
}
static int64_t mild(int64_t most) { return 1 + (int64_t)(next() % (uint64_t)most); }
template <typename T> static T pick(std::initializer_list<T> l) { return l.begin()[next() % l.size()]; }

static void expect(bool good, const char* what)
{
    if (!good) {
        std::printf("FAIL %s\n", what);
        ++failures;
    }
}

int main()
{
    const char* base = reinterpret_cast<const char*>((uintptr_t)1 << 20);
    auto ptr = [&] { return const_cast<char*>(next() % 8 ? base : next() % 2 ? nullptr : base + 1 + next() % 15); };
    for (int i = 0; i < 200000; ++i) {
        const bool w = next() % 2;             // all fields wild, or a sound call with one wild field
        mnb_kv4_desc c = {};
        c.kv_heads = (int32_t)(w ? wild() : mild(16));
        c.q_heads = w ? (int32_t)wild() : c.kv_heads * (int32_t)mild(8);
        c.head_dim = pick<int32_t>({64, 128, 256});
        c.group_size = pick<int32_t>({32, 64});
        c.page_size = pick<int32_t>({32, 64, 128, 256});
        c.num_pages = w ? wild() : mild(1 << 20);
        if (next() % 16 == 0) c.reserved = 1;
        (void)mnb_kv4_cache_bytes(&c);
        const int64_t batch = w ? wild() : mild(64), tokens = w ? wild() : mild(1 << 16);
        const int64_t mq = w ? wild() : mild(4096), mk = w ? wild() : mild((int64_t)1 << 30);
        (void)mnb_attention_kv4_workspace_bytes(&c, batch, tokens, mq, mk);
        auto i32 = [&] { return reinterpret_cast<int32_t*>(ptr()); };
        auto f32 = [&] { return reinterpret_cast<float*>(ptr()); };
        const mnb_status a = mnb_attention_kv4(&c, ptr(), i32(), wild(), i32(), i32(), batch, tokens, mq, mk,
                                               (int32_t)(next() % 3), ptr(), wild(), 0.1f, (int32_t)(next() % 3), wild(),
                                               ptr(), f32(), ptr(), (size_t)wild(), nullptr);
        const mnb_status p = mnb_kv4_append(&c, ptr(), i32(), wild(), i32(), i32(), batch, tokens, (int32_t)(next() % 3),
                                            ptr(), wild(), ptr(), wild(), ptr(), wild(), f32(), f32(), wild(),
                                            (int32_t)wild(), (int32_t)(next() % 3), ptr(), nullptr);
        const mnb_status r = mnb_kv4_read(&c, ptr(), i32(), wild(), i32(), i32(), batch, tokens, (int32_t)(next() % 3),
                                          ptr(), ptr(), nullptr);
        const mnb_status n = mnb_rms_norm(ptr(), wild(), ptr(), wild(), ptr(), wild(), wild(), (int32_t)(next() % 3), 1e-5f,
                                          (int32_t)(next() % 5) - 1, ptr(), f32(), ptr(), nullptr);
        for (mnb_status s : {a, p, r, n}) expect(s >= MNB_OK && s <= MNB_ERR_DEVICE, "a status");
    }
    // the plan: every key in a split, every row in a tile, a grid that can be launched
    for (int i = 0; i < 400000; ++i) {
        mnb::AttentionArgs a = {};
        a.v.head_dim = pick<int>({64, 128, 256});
        a.v.groups = a.v.head_dim / pick<int>({32, 64});
        a.v.kv_heads = (int)mild(next() % 4 ? 32 : 4096);
        a.v.q_heads = a.v.kv_heads * (int)mild(16);
        a.v.batch = (int)mild(next() % 4 ? 64 : 65535);
        a.max_q = next() % 3 ? mild(8) : mild(((int64_t)1 << 29) / a.v.q_heads);
        a.max_kv = next() % 2 ? mild(5000) : mild((int64_t)1 << 30);
        if (next() % 50 == 0) a.max_kv = 0;
        const mnb::kv4::Plan c = mnb::kv4::plan_of(a);
        const int64_t rows = a.max_q * (a.v.q_heads / a.v.kv_heads);
        expect(c.splits >= 1 && c.splits <= mnb::kv4::kMaxSplits, "splits");
        expect(c.chunk > 0 && c.chunk % 64 == 0 && (int64_t)c.chunk * c.splits >= a.max_kv, "keys");
        expect((int64_t)c.row_tiles * c.rows >= rows && (int64_t)(c.row_tiles - 1) * c.rows < rows, "rows");
        expect((uint64_t)a.v.kv_heads * c.splits * c.row_tiles * 512 < ((uint64_t)1 << 32) + 512 || rows * a.v.kv_heads > ((int64_t)1 << 29), "grid");
        expect(c.splits == 1 || (uint64_t)a.max_q * a.v.q_heads * 256 < ((uint64_t)1 << 32), "join grid");
        expect(c.kind != 1 || c.group == 0 || c.rows == 16 / c.group, "group");
    }
    std::printf("%s: %d failures\n", failures ? "FAILED" : "ok", failures);
    return failures ? 1 : 0;
}
