// mnb_decoder_api.cpp -- the C ABI of the operators between a decoder layer's
// products (RMS norm, 4-bit cache, attention): host-side validation, then one
// launcher call on the caller's stream.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/mnb.h"
#include "mnb_api_common.hpp"
#include "mnb_kv4.hpp"

namespace {

using mnb::api::check_device;
using mnb::api::check_ptr;
using mnb::api::fail;
using mnb::api::launched;
using mnb::api::ok;

constexpr int64_t kMaxInt = INT32_MAX;

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

int64_t page_bytes(const mnb_kv4_desc* c)
{
    return (int64_t)c->kv_heads * (c->page_size / mnb::kKvBlock) * mnb::kv_block_bytes(c->head_dim, c->head_dim / c->group_size);
}

mnb_status check_kv_desc(const mnb_kv4_desc* c)
{
    if (!c) return fail(MNB_ERR_INVALID_ARGUMENT, "cache descriptor is NULL");
    if (c->kv_heads < 1 || c->q_heads < 1)
        return fail(MNB_ERR_INVALID_ARGUMENT, "q_heads and kv_heads must be >= 1 (got %d, %d)", c->q_heads, c->kv_heads);
    if (c->q_heads % c->kv_heads != 0)
        return fail(MNB_ERR_INVALID_ARGUMENT, "q_heads %d is not a multiple of kv_heads %d", c->q_heads, c->kv_heads);
    if (c->reserved != 0) return fail(MNB_ERR_INVALID_ARGUMENT, "reserved field must be 0");
    if (c->num_pages < 0 || c->num_pages > kMaxInt)
        return fail(MNB_ERR_INVALID_ARGUMENT, "num_pages must be in 0..2^31-1 (got %lld)", (long long)c->num_pages);
    if (c->q_heads > 65536)
        return fail(MNB_ERR_UNSUPPORTED, "q_heads %d not supported (at most 65536)", c->q_heads);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(MNB_ERR_UNSUPPORTED, "head_dim %d not supported (64, 128 or 256)", c->head_dim);
    if (c->group_size != 32 && c->group_size != 64 && c->group_size != 128)
        return fail(MNB_ERR_UNSUPPORTED, "group_size %d not supported (32, 64 or 128)", c->group_size);
    if (c->group_size > c->head_dim)
        return fail(MNB_ERR_UNSUPPORTED, "group_size %d exceeds head_dim %d", c->group_size, c->head_dim);
    if (c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256)
        return fail(MNB_ERR_UNSUPPORTED, "page_size %d not supported (32, 64, 128 or 256)", c->page_size);
    if (c->num_pages > INT64_MAX / page_bytes(c)) return fail(MNB_ERR_INVALID_ARGUMENT, "cache size overflows");
    return MNB_OK;
}

mnb_status check_sequences(const int32_t* block_table, int64_t table_stride, const int32_t* kv_len,
                           const int32_t* q_start, int64_t batch, int64_t tokens)
{
    MNB_TRY(check_ptr(block_table, 4, "block_table"));
    MNB_TRY(check_ptr(kv_len, 4, "kv_len"));
    if (q_start)
        MNB_TRY(check_ptr(q_start, 4, "q_start"));
    else if (tokens != batch)
        return fail(MNB_ERR_INVALID_ARGUMENT, "without q_start tokens must equal batch (got %lld, %lld)",
                    (long long)tokens, (long long)batch);
    if (table_stride < 1 || table_stride > kMaxInt)
        return fail(MNB_ERR_INVALID_ARGUMENT, "table_stride must be in 1..2^31-1 (got %lld)", (long long)table_stride);
    return MNB_OK;
}

mnb_status check_counts(int64_t batch, int64_t tokens)
{
    if (batch < 0 || tokens < 0)
        return fail(MNB_ERR_INVALID_ARGUMENT, "batch and tokens must be >= 0 (got %lld, %lld)", (long long)batch,
                    (long long)tokens);
    if (batch >= kMaxInt || tokens > kMaxInt)
        return fail(MNB_ERR_INVALID_ARGUMENT, "batch and tokens must fit in 32 bits");
    return MNB_OK;
}

// A workgroup of up to 256 threads each, in a grid of less than 2^32 threads.
mnb_status check_tokens(int64_t tokens)
{
    if (tokens >= (int64_t(1) << 24))
        return fail(MNB_ERR_UNSUPPORTED, "%lld tokens not supported (below 2^24)", (long long)tokens);
    return MNB_OK;
}

mnb::KvView view_of(const mnb_kv4_desc* c, const void* cache, const int32_t* block_table, int64_t table_stride,
                    const int32_t* kv_len, const int32_t* q_start, int64_t batch, int64_t tokens)
{
    mnb::KvView v;
    v.cache = static_cast<unsigned char*>(const_cast<void*>(cache));
    v.table = block_table;
    v.table_stride = table_stride;
    v.kv_len = kv_len;
    v.q_start = q_start;
    v.batch = (int)batch;
    v.tokens = (int)tokens;
    v.q_heads = c->q_heads;
    v.kv_heads = c->kv_heads;
    v.head_dim = c->head_dim;
    v.groups = c->head_dim / c->group_size;
    v.page_shift = c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : c->page_size == 128 ? 7 : 8;
    v.num_pages = (int)c->num_pages;
    return v;
}

// The attention's bounds, and the arguments its plan depends on.
mnb_status check_bounds(const mnb_kv4_desc* c, int64_t batch, int64_t tokens, int64_t max_q, int64_t max_kv)
{
    MNB_TRY(check_kv_desc(c));
    MNB_TRY(check_counts(batch, tokens));
    if (max_q < 0 || max_kv < 0)
        return fail(MNB_ERR_INVALID_ARGUMENT, "max_q and max_kv must be >= 0 (got %lld, %lld)", (long long)max_q,
                    (long long)max_kv);
    if (batch > 65535) return fail(MNB_ERR_UNSUPPORTED, "batch %lld not supported (at most 65535)", (long long)batch);
    if (max_kv > (int64_t(1) << 30))
        return fail(MNB_ERR_UNSUPPORTED, "max_kv %lld not supported (at most 2^30)", (long long)max_kv);
    if (max_q > kMaxInt / 4 / c->q_heads)
        return fail(MNB_ERR_UNSUPPORTED, "max_q %lld times q_heads %d not supported (below 2^29)", (long long)max_q,
                    c->q_heads);
    return MNB_OK;
}

mnb::AttentionArgs plan_args(const mnb_kv4_desc* c, int64_t batch, int64_t tokens, int64_t max_q, int64_t max_kv)
{
    mnb::AttentionArgs a = {};
    a.v = view_of(c, nullptr, nullptr, 0, nullptr, nullptr, batch, tokens);
    a.max_q = max_q;
    a.max_kv = max_kv;
    return a;
}

}  // namespace

extern "C" {

mnb_status mnb_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                        const void* weight, int64_t m, int64_t k, int32_t dtype, float eps, int32_t out_kind,
                        void* out, float* scales, void* residual_out, void* stream)
{
    MNB_TRY(check_dtype(dtype));
    if (out_kind != MNB_NORM_VALUES && out_kind != MNB_NORM_CODES_F16 && out_kind != MNB_NORM_CODES_I8)
        return fail(MNB_ERR_INVALID_ARGUMENT, "out_kind must be an mnb_norm_out (got %d)", out_kind);
    if (m < 0 || k < 1) return fail(MNB_ERR_INVALID_ARGUMENT, "M must be >= 0 and K >= 1 (got %lld, %lld)", (long long)m, (long long)k);
    if (m > kMaxInt || k > kMaxInt - 15) return fail(MNB_ERR_INVALID_ARGUMENT, "M and K must fit in 32 bits");
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(MNB_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
    if (out_kind == MNB_NORM_VALUES && scales)
        return fail(MNB_ERR_INVALID_ARGUMENT, "scales given but out_kind is MNB_NORM_VALUES");
    MNB_TRY(check_stride(x_stride, k, m, "x_stride"));
    if (residual) MNB_TRY(check_stride(residual_stride, k, m, "residual_stride"));
    if (m == 0) return ok("noop");
    const uintptr_t elem = dtype == MNB_F16 ? 2 : 4;
    MNB_TRY(check_ptr(x, elem, "x"));
    MNB_TRY(check_ptr(weight, elem, "weight"));
    if (residual) MNB_TRY(check_ptr(residual, elem, "residual"));
    if (residual_out) MNB_TRY(check_ptr(residual_out, elem, "residual_out"));
    MNB_TRY(check_ptr(out, out_kind == MNB_NORM_VALUES ? elem : out_kind == MNB_NORM_CODES_F16 ? 2 : 1, "out"));
    if (out_kind != MNB_NORM_VALUES) MNB_TRY(check_ptr(scales, 4, "scales"));
    MNB_TRY(check_device());
    mnb::NormArgs a;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.out = out;
    a.scales = scales;
    a.residual_out = residual_out;
    a.m = m;
    a.k = k;
    a.x_stride = x_stride;
    a.residual_stride = residual_stride;
    a.eps = eps;
    a.f16 = dtype == MNB_F16;
    a.out_kind = out_kind;
    const char* variant = "";
    const hipError_t e = mnb::launch_rms_norm(a, static_cast<hipStream_t>(stream), &variant);
    return launched(e, variant);
}

size_t mnb_kv4_cache_bytes(const mnb_kv4_desc* c)
{
    if (check_kv_desc(c) != MNB_OK) return 0;
    if (c->num_pages == 0) {
        fail(MNB_ERR_INVALID_ARGUMENT, "the cache has no pages");
        return 0;
    }
    ok(nullptr);
    return (size_t)(page_bytes(c) * c->num_pages);
}

mnb_status mnb_kv4_append(const mnb_kv4_desc* c, void* cache, const int32_t* block_table, int64_t table_stride,
                          const int32_t* kv_len, const int32_t* q_start, int64_t batch, int64_t tokens,
                          int32_t dtype, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const float* cos, const float* sin, int64_t rope_rows,
                          int32_t rotary_dim, int32_t interleaved, void* q_out, void* stream)
{
    MNB_TRY(check_kv_desc(c));
    MNB_TRY(check_dtype(dtype));
    MNB_TRY(check_counts(batch, tokens));
    if ((cos == nullptr) != (sin == nullptr))
        return fail(MNB_ERR_INVALID_ARGUMENT, "cos and sin must both be given or both be NULL");
    if (interleaved != 0 && interleaved != 1)
        return fail(MNB_ERR_INVALID_ARGUMENT, "interleaved must be 0 or 1 (got %d)", interleaved);
    if (cos) {
        if (rotary_dim < 1 || rotary_dim > c->head_dim)
            return fail(MNB_ERR_INVALID_ARGUMENT, "rotary_dim must be in 1..%d (got %d)", c->head_dim, rotary_dim);
        if (rotary_dim % 16 != 0)
            return fail(MNB_ERR_UNSUPPORTED, "rotary_dim %d not supported (a multiple of 16)", rotary_dim);
        if (rope_rows < 1) return fail(MNB_ERR_INVALID_ARGUMENT, "rope_rows must be >= 1 (got %lld)", (long long)rope_rows);
        MNB_TRY(check_ptr(cos, 4, "cos"));
        MNB_TRY(check_ptr(sin, 4, "sin"));
    }
    if ((q == nullptr) != (q_out == nullptr))
        return fail(MNB_ERR_INVALID_ARGUMENT, "q and q_out must both be given or both be NULL");
    const int64_t kv_row = (int64_t)c->kv_heads * c->head_dim, q_row = (int64_t)c->q_heads * c->head_dim;
    MNB_TRY(check_stride(k_stride, kv_row, tokens, "k_stride"));
    MNB_TRY(check_stride(v_stride, kv_row, tokens, "v_stride"));
    if (q) MNB_TRY(check_stride(q_stride, q_row, tokens, "q_stride"));
    if (tokens == 0 || batch == 0) return ok("noop");
    MNB_TRY(check_tokens(tokens));
    MNB_TRY(check_sequences(block_table, table_stride, kv_len, q_start, batch, tokens));
    const uintptr_t elem = dtype == MNB_F16 ? 2 : 4;
    MNB_TRY(check_ptr(k, elem, "k"));
    MNB_TRY(check_ptr(v, elem, "v"));
    if (q) MNB_TRY(check_ptr(q, elem, "q"));
    if (q) MNB_TRY(check_ptr(q_out, elem, "q_out"));
    MNB_TRY(check_ptr(cache, 256, "cache"));
    MNB_TRY(check_device());
    mnb::AppendArgs a;
    a.v = view_of(c, cache, block_table, table_stride, kv_len, q_start, batch, tokens);
    a.q = q;
    a.k = k;
    a.val = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.cos = cos;
    a.sin = sin;
    a.rope_rows = rope_rows;
    a.rotary_dim = cos ? rotary_dim : 0;
    a.interleaved = interleaved;
    a.q_out = q_out;
    a.f16 = dtype == MNB_F16;
    const char* variant = "";
    const hipError_t e = mnb::launch_kv4_append(a, static_cast<hipStream_t>(stream), &variant);
    return launched(e, variant);
}

mnb_status mnb_kv4_read(const mnb_kv4_desc* c, const void* cache, const int32_t* block_table, int64_t table_stride,
                        const int32_t* kv_len, const int32_t* q_start, int64_t batch, int64_t tokens,
                        int32_t dtype, void* k_out, void* v_out, void* stream)
{
    MNB_TRY(check_kv_desc(c));
    MNB_TRY(check_dtype(dtype));
    MNB_TRY(check_counts(batch, tokens));
    if (tokens == 0 || batch == 0 || (!k_out && !v_out)) return ok("noop");
    MNB_TRY(check_tokens(tokens));
    MNB_TRY(check_sequences(block_table, table_stride, kv_len, q_start, batch, tokens));
    const uintptr_t elem = dtype == MNB_F16 ? 2 : 4;
    if (k_out) MNB_TRY(check_ptr(k_out, elem, "k_out"));
    if (v_out) MNB_TRY(check_ptr(v_out, elem, "v_out"));
    MNB_TRY(check_ptr(cache, 256, "cache"));
    MNB_TRY(check_device());
    mnb::ReadArgs a;
    a.v = view_of(c, cache, block_table, table_stride, kv_len, q_start, batch, tokens);
    a.k_out = k_out;
    a.v_out = v_out;
    a.f16 = dtype == MNB_F16;
    const char* variant = "";
    const hipError_t e = mnb::launch_kv4_read(a, static_cast<hipStream_t>(stream), &variant);
    return launched(e, variant);
}

size_t mnb_attention_kv4_workspace_bytes(const mnb_kv4_desc* c, int64_t batch, int64_t tokens, int64_t max_q,
                                         int64_t max_kv)
{
    if (check_bounds(c, batch, tokens, max_q, max_kv) != MNB_OK) return 0;
    ok(nullptr);
    if (batch == 0 || tokens == 0 || max_q == 0) return 0;
    return mnb::kv4_attention_workspace(plan_args(c, batch, tokens, max_q, max_kv));
}

mnb_status mnb_attention_kv4(const mnb_kv4_desc* c, const void* cache, const int32_t* block_table,
                             int64_t table_stride, const int32_t* kv_len, const int32_t* q_start, int64_t batch,
                             int64_t tokens, int64_t max_q, int64_t max_kv, int32_t dtype, const void* q,
                             int64_t q_stride, float scale, int32_t causal, int64_t window, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, void* stream)
{
    MNB_TRY(check_bounds(c, batch, tokens, max_q, max_kv));
    MNB_TRY(check_dtype(dtype));
    if (causal != 0 && causal != 1) return fail(MNB_ERR_INVALID_ARGUMENT, "causal must be 0 or 1 (got %d)", causal);
    if (window < 0) return fail(MNB_ERR_INVALID_ARGUMENT, "window must be >= 0 (got %lld)", (long long)window);
    if (window > 0 && !causal) return fail(MNB_ERR_INVALID_ARGUMENT, "a window needs causal = 1");
    if (!std::isfinite(scale * mnb::kLog2E))
        return fail(MNB_ERR_INVALID_ARGUMENT, "scale must be finite, and times log2(e) too");
    MNB_TRY(check_stride(q_stride, (int64_t)c->q_heads * c->head_dim, tokens, "q_stride"));
    if (tokens == 0 || batch == 0 || max_q == 0) return ok("noop");
    MNB_TRY(check_sequences(block_table, table_stride, kv_len, q_start, batch, tokens));
    const uintptr_t elem = dtype == MNB_F16 ? 2 : 4;
    MNB_TRY(check_ptr(q, elem, "q"));
    MNB_TRY(check_ptr(out, elem, "out"));
    if (lse) MNB_TRY(check_ptr(lse, 4, "lse"));
    MNB_TRY(check_ptr(cache, 256, "cache"));
    mnb::AttentionArgs a = plan_args(c, batch, tokens, max_q, max_kv);
    const size_t need = mnb::kv4_attention_workspace(a);
    if (workspace_bytes < need)
        return fail(MNB_ERR_INVALID_ARGUMENT, "workspace too small: %zu bytes given, %zu needed", workspace_bytes, need);
    if (need > 0) MNB_TRY(check_ptr(workspace, 256, "workspace"));
    MNB_TRY(check_device());
    a.v = view_of(c, cache, block_table, table_stride, kv_len, q_start, batch, tokens);
    a.q = q;
    a.q_stride = q_stride;
    a.out = out;
    a.lse = lse;
    a.scale = scale;
    a.causal = causal;
    a.window = window;
    a.workspace = workspace;
    a.f16 = dtype == MNB_F16;
    const char* variant = "";
    const hipError_t e = mnb::launch_kv4_attention(a, static_cast<hipStream_t>(stream), &variant);
    return launched(e, variant);
}

}  // extern "C"
