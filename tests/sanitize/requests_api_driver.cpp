// Host-side run of the calls that serve many requests at once under
// AddressSanitizer and UndefinedBehaviorSanitizer: argument checks with random and
// extreme values, and the adapters' plan over its whole range.  Built as plain C++: the
// launchers are stubs that are never reached, because the device check fails.
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <initializer_list>

#include "adapters_plan.hpp"
#include "mnb.h"
#include "mnb_api_common.hpp"
#include "mnb_requests.hpp"

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
hipError_t launch_adapters(const AdapterArgs&, hipStream_t, const char**) { std::abort(); }
hipError_t launch_verify(const VerifyArgs&, hipStream_t, const char**) { std::abort(); }
size_t adapters_workspace(int64_t m, int64_t n, int64_t k, int rank, int count, int f16)
{
    const adapters::Plan c = adapters::plan_of(m, n, k, rank, count, f16);
    return c.one ? 0 : (size_t)c.splits * m * c.pitch * 4;
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
    static const int64_t v[] = {0, 1, -1, 2, 16, 31, 32, 64, 127, 128, 129, 255, 256, 1000, 1023, 1024, 4096, 65536, 1 << 24,
                                (1 << 24) + 1, 1 << 30, INT32_MAX, (int64_t)INT32_MAX + 1, (int64_t)1 << 40, INT64_MAX, INT64_MIN, INT32_MIN};
    return v[next() % (sizeof(v) / sizeof(v[0]))];
}
static int64_t mild(int64_t most) { return 1 + (int64_t)(next() % (uint64_t)most); }
static void expect(bool good, const char* what)
{
    if (!good && ++failures < 20) std::printf("FAIL %s\n", what);
}

int main()
{
    const char* base = reinterpret_cast<const char*>((uintptr_t)1 << 20);
    auto ptr = [&] { return const_cast<char*>(next() % 8 ? base : next() % 2 ? nullptr : base + 1 + next() % 15); };
    auto i32 = [&] { return reinterpret_cast<int32_t*>(ptr()); };
    auto f32 = [&] { return reinterpret_cast<float*>(ptr()); };
    int reached = 0;
    for (int i = 0; i < 300000; ++i) {
        const bool w = next() % 2;             // all fields wild, or a sound call with one wild field
        mnb_adapter_desc d = {};
        d.n = w ? wild() : mild(1 << 24);
        d.k = w ? wild() : mild(1 << 24);
        d.rank = (int32_t)(w ? wild() : mild(128));
        d.count = (int32_t)(w ? wild() : mild(1000));
        d.dtype = (int32_t)(next() % 16 ? next() % 2 : 2);
        d.reserved = next() % 16 == 0;
        const int64_t m = w ? wild() : mild(1 << 13);
        const size_t need = mnb_adapters_workspace_bytes(&d, m);
        const mnb_status a = mnb_adapters_add(&d, ptr(), ptr(), f32(), i32(), i32(), m, ptr(), w ? wild() : d.k + mild(9), ptr(),
                                              w ? wild() : d.n + mild(9), ptr(), w ? wild() : d.n + mild(9), ptr(),
                                              w ? (size_t)wild() : need, nullptr);
        const int64_t batch = w ? wild() : mild(64), vocab = w ? wild() : mild(300000), tokens = w ? wild() : mild(1000);
        const size_t size = mnb_verify_workspace_bytes(batch, vocab);
        const mnb_status v = mnb_verify_drafts(ptr(), w ? wild() : vocab + mild(9), ptr(), w ? wild() : vocab + mild(9), i32(), i32(),
                                               batch, tokens, vocab, (int32_t)(next() % 3), f32(), f32(), i32(), i32(), ptr(),
                                               w ? (size_t)wild() : size, nullptr);
        for (mnb_status s : {a, v}) expect(s >= MNB_OK && s <= MNB_ERR_DEVICE, "a status");
        reached += (a == MNB_ERR_DEVICE) + (v == MNB_ERR_DEVICE);
    }
    expect(reached > 1000, "sound calls reach the device check");
    // the plan: all of k in a split, whole steps, slots for no more adapters than there can be, grids that can be launched
    for (int i = 0; i < 400000; ++i) {
        const int64_t n = mild(next() % 2 ? 20000 : 1 << 24), k = mild(next() % 2 ? 20000 : 1 << 24);
        int64_t m = mild(next() % 3 ? 300 : (1 << 24) - 1);
        if (m * n >= (int64_t)1 << 37) m = ((int64_t)1 << 37) / n - 1;
        const int rank = (int)mild(128), f16 = (int)(next() % 2), count = (int)(next() % 20 ? mild(2000) : 0);
        const mnb::adapters::Plan c = mnb::adapters::plan_of(m, n, k, rank, count, f16);
        const int64_t blocks = (n + 255) / 256, ranks = 16 * c.down_ranks;
        expect((c.down_tile == 16 || c.down_tile == 32 || c.down_tile == 64) && (c.up_tile == 16 || c.up_tile == 32 || c.up_tile == 64), "tiles");
        expect(c.down_ranks == 1 || c.down_ranks == 2 || c.down_ranks == 4, "ranks");
        expect(c.pitch >= rank && c.pitch <= 128 && c.pitch % 16 == 0, "pitch");
        expect(c.splits >= 1 && c.splits <= 8 && c.k_per % (f16 ? 64 : 32) == 0, "splits");
        expect(c.k_per * c.splits >= k && c.k_per * (c.splits - 1) < k, "all of k");
        for (int s : {c.one_slots, c.down_slots, c.up_slots}) expect(s >= 1 && s <= 64 && (s <= count || s == 1) && s <= m, "slots");
        expect((uint64_t)((m + c.down_tile - 1) / c.down_tile) * c.splits * c.down_slots * ((rank + ranks - 1) / ranks) * 256 < (uint64_t)1 << 32, "first grid");
        expect((uint64_t)((m + c.up_tile - 1) / c.up_tile) * blocks * c.up_slots * 256 < (uint64_t)1 << 32, "second grid");
        if (c.one) expect((m + 31) / 32 * ((n + 511) / 512) * c.one_slots <= 256 && rank <= 32, "one launch");
    }
    std::printf("%s: %d failures\n", failures ? "FAILED" : "ok", failures);
    return failures ? 1 : 0;
}
