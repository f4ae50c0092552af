// mnb_requests_api.cpp -- the C ABI of the operators that serve many requests at
// once (low-rank adapters, drafted tokens): host-side validation, then one
// launcher call on the caller's stream.
#include <hip/hip_runtime.h>

#include "../../include/mnb.h"
#include "adapters_plan.hpp"
#include "mnb_api_common.hpp"
#include "mnb_requests.hpp"

namespace {

using mnb::api::check_device;
using mnb::api::check_ptr;
using mnb::api::fail;
using mnb::api::launched;
using mnb::api::ok;

mnb_status check_dtype(int32_t dtype)
{
    if (dtype != MNB_F16 && dtype != MNB_F32)
        return fail(MNB_ERR_INVALID_ARGUMENT, "dtype must be MNB_F16 or MNB_F32 (got %d)", dtype);
    return MNB_OK;
}

mnb_status check_stride(int64_t stride, int64_t row, int64_t rows, const char* name)
{
    if (stride < row)
        return fail(MNB_ERR_INVALID_ARGUMENT, "%s must be at least %lld (got %lld)", name, (long long)row,
                    (long long)stride);
    if (rows > 1 && stride > INT64_MAX / 8 / rows)
        return fail(MNB_ERR_INVALID_ARGUMENT, "%s times the rows overflows", name);
    return MNB_OK;
}

mnb_status check_adapters(const mnb_adapter_desc* d, int64_t m)
{
    if (!d) return fail(MNB_ERR_INVALID_ARGUMENT, "adapter descriptor is NULL");
    MNB_TRY(check_dtype(d->dtype));
    if (d->reserved != 0) return fail(MNB_ERR_INVALID_ARGUMENT, "reserved field must be 0");
    if (d->n < 0 || d->k < 1)
        return fail(MNB_ERR_INVALID_ARGUMENT, "N must be >= 0 and K >= 1 (got %lld, %lld)", (long long)d->n, (long long)d->k);
    if (d->rank < 1 || d->count < 0)
        return fail(MNB_ERR_INVALID_ARGUMENT, "rank must be >= 1 and count >= 0 (got %d, %d)", d->rank, d->count);
    if (m < 0) return fail(MNB_ERR_INVALID_ARGUMENT, "M must be >= 0 (got %lld)", (long long)m);
    if (d->rank > mnb::adapters::kMaxRank)
        return fail(MNB_ERR_UNSUPPORTED, "rank %d not supported (at most %d)", d->rank, mnb::adapters::kMaxRank);
    if (d->n > (1 << 24) || d->k > (1 << 24))
        return fail(MNB_ERR_UNSUPPORTED, "N=%lld, K=%lld not supported (at most 2^24)", (long long)d->n, (long long)d->k);
    if ((int64_t)d->count * d->rank > INT64_MAX / 8 / (d->n > d->k ? d->n : d->k))
        return fail(MNB_ERR_INVALID_ARGUMENT, "count=%d times rank=%d times N or K overflows", d->count, d->rank);
    // a workgroup of 256 threads takes 64 rows of 256 columns, in a grid of less than 2^32 threads
    if (m >= (1 << 24) || m * d->n >= (int64_t(1) << 37))
        return fail(MNB_ERR_UNSUPPORTED, "M=%lld not supported (below 2^24, and M*N below 2^37)", (long long)m);
    return MNB_OK;
}

mnb_status check_verify(int64_t batch, int64_t vocab)
{
    if (batch < 0 || vocab < 1)
        return fail(MNB_ERR_INVALID_ARGUMENT, "batch must be >= 0 and vocab >= 1 (got %lld, %lld)", (long long)batch,
                    (long long)vocab);
    if (vocab > (1 << 30)) return fail(MNB_ERR_UNSUPPORTED, "vocab %lld not supported (at most 2^30)", (long long)vocab);
    // a wave a chunk and at most three idle ones a sequence, in a grid of less than 2^32 threads
    if (batch >= (1 << 24) || mnb::verify_chunks(vocab) * batch >= (1 << 24))
        return fail(MNB_ERR_UNSUPPORTED, "batch %lld with vocab %lld not supported", (long long)batch, (long long)vocab);
    return MNB_OK;
}

}  // namespace

extern "C" {

size_t mnb_adapters_workspace_bytes(const mnb_adapter_desc* d, int64_t m)
{
    if (check_adapters(d, m) != MNB_OK) return 0;
    ok(nullptr);
    if (m == 0 || d->n == 0 || d->count == 0) return 0;
    return mnb::adapters_workspace(m, d->n, d->k, d->rank, d->count, d->dtype == MNB_F16);
}

mnb_status mnb_adapters_add(const mnb_adapter_desc* d, const void* a, const void* b, const float* scales,
                            const int32_t* ranks, const int32_t* adapter, int64_t m, const void* x, int64_t x_stride,
                            const void* base, int64_t base_stride, void* y, int64_t y_stride, void* workspace,
                            size_t workspace_bytes, void* stream)
{
    MNB_TRY(check_adapters(d, m));
    MNB_TRY(check_stride(x_stride, d->k, m, "x_stride"));
    MNB_TRY(check_stride(y_stride, d->n, m, "y_stride"));
    if (base) MNB_TRY(check_stride(base_stride, d->n, m, "base_stride"));
    if (m == 0 || d->n == 0) return ok("noop");
    if (base && base == y && base_stride != y_stride && m > 1)
        return fail(MNB_ERR_INVALID_ARGUMENT, "y is base, but their strides differ (%lld, %lld)", (long long)y_stride,
                    (long long)base_stride);
    const uintptr_t elem = d->dtype == MNB_F16 ? 2 : 4;
    if (d->count > 0) {
        MNB_TRY(check_ptr(a, 16, "a"));
        MNB_TRY(check_ptr(b, 16, "b"));
    }
    if (scales) MNB_TRY(check_ptr(scales, 4, "scales"));
    if (ranks) MNB_TRY(check_ptr(ranks, 4, "ranks"));
    MNB_TRY(check_ptr(adapter, 4, "adapter"));
    MNB_TRY(check_ptr(x, elem, "x"));
    if (base) MNB_TRY(check_ptr(base, elem, "base"));
    MNB_TRY(check_ptr(y, elem, "y"));
    const size_t need = d->count > 0 ? mnb::adapters_workspace(m, d->n, d->k, d->rank, d->count, d->dtype == MNB_F16) : 0;
    if (workspace_bytes < need)
        return fail(MNB_ERR_INVALID_ARGUMENT, "workspace too small: %zu bytes given, %zu needed", workspace_bytes, need);
    if (need > 0) MNB_TRY(check_ptr(workspace, 256, "workspace"));
    MNB_TRY(check_device());
    mnb::AdapterArgs g;
    g.a = a;
    g.b = b;
    g.scales = scales;
    g.ranks = ranks;
    g.adapter = adapter;
    g.x = x;
    g.base = base;
    g.y = y;
    g.m = m;
    g.n = d->n;
    g.k = d->k;
    g.rank = d->rank;
    g.count = d->count;
    g.x_stride = x_stride;
    g.base_stride = base_stride;
    g.y_stride = y_stride;
    g.workspace = workspace;
    g.f16 = d->dtype == MNB_F16;
    const char* variant = "";
    const hipError_t e = mnb::launch_adapters(g, static_cast<hipStream_t>(stream), &variant);
    return launched(e, variant);
}

size_t mnb_verify_workspace_bytes(int64_t batch, int64_t vocab)
{
    if (check_verify(batch, vocab) != MNB_OK) return 0;
    ok(nullptr);
    return mnb::verify_workspace(batch, vocab);
}

mnb_status mnb_verify_drafts(const void* target, int64_t target_stride, const void* draft, int64_t draft_stride,
                             const int32_t* ids, const int32_t* q_start, int64_t batch, int64_t tokens, int64_t vocab,
                             int32_t dtype, const float* accept, const float* pick, int32_t* out, int32_t* accepted,
                             void* workspace, size_t workspace_bytes, void* stream)
{
    MNB_TRY(check_dtype(dtype));
    MNB_TRY(check_verify(batch, vocab));
    if (tokens < 0 || tokens > INT32_MAX)
        return fail(MNB_ERR_INVALID_ARGUMENT, "tokens must be in 0..2^31-1 (got %lld)", (long long)tokens);
    MNB_TRY(check_stride(target_stride, vocab, tokens, "target_stride"));
    if (draft) MNB_TRY(check_stride(draft_stride, vocab, tokens, "draft_stride"));
    if (!q_start && tokens != batch)
        return fail(MNB_ERR_INVALID_ARGUMENT, "without q_start tokens must equal batch (got %lld, %lld)",
                    (long long)tokens, (long long)batch);
    if (batch == 0) return ok("noop");
    if (q_start) MNB_TRY(check_ptr(q_start, 4, "q_start"));
    const uintptr_t elem = dtype == MNB_F16 ? 2 : 4;
    MNB_TRY(check_ptr(accepted, 4, "accepted"));
    MNB_TRY(check_ptr(pick, 4, "pick"));
    if (tokens > 0) {
        MNB_TRY(check_ptr(target, elem, "target"));
        if (draft) MNB_TRY(check_ptr(draft, elem, "draft"));
        MNB_TRY(check_ptr(ids, 4, "ids"));
        MNB_TRY(check_ptr(accept, 4, "accept"));
        MNB_TRY(check_ptr(out, 4, "out"));
    }
    const size_t need = mnb::verify_workspace(batch, vocab);
    if (workspace_bytes < need)
        return fail(MNB_ERR_INVALID_ARGUMENT, "workspace too small: %zu bytes given, %zu needed", workspace_bytes, need);
    MNB_TRY(check_ptr(workspace, 256, "workspace"));
    MNB_TRY(check_device());
    mnb::VerifyArgs g;
    g.target = target;
    g.draft = draft;
    g.target_stride = target_stride;
    g.draft_stride = draft_stride;
    g.ids = ids;
    g.q_start = q_start;
    g.accept = accept;
    g.pick = pick;
    g.out = out;
    g.accepted = accepted;
    g.batch = batch;
    g.tokens = tokens;
    g.vocab = vocab;
    g.workspace = workspace;
    g.f16 = dtype == MNB_F16;
    const char* variant = "";
    const hipError_t e = mnb::launch_verify(g, static_cast<hipStream_t>(stream), &variant);
    return launched(e, variant);
}

}  // extern "C"
