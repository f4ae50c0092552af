// mnb_kv4.hpp -- the paged 4-bit key/value cache (layout in include/mnb.h) and
// the launchers of the operators between a decoder layer's products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mnb {

constexpr int kKvBlock = 32;   // tokens of one block: keys and values of one head

// Bytes of one block: 4-bit keys and values, then one word (fp16 scale, zero
// point) per token and group for each.
__host__ __device__ __forceinline__ int64_t kv_block_bytes(int D, int NG)
{
    return (int64_t)kKvBlock * D + 2 * kKvBlock * 4 * NG;
}

// The cache and the sequences in it, as the kernels take them.
struct KvView {
    unsigned char* cache;
    const int32_t* table;     // [batch, table_stride] page numbers
    int64_t table_stride;
    const int32_t* kv_len;    // [batch]
    const int32_t* q_start;   // [batch + 1], or NULL: one new token per sequence
    int batch;
    int tokens;               // rows of the new tokens' arrays
    int q_heads, kv_heads;
    int head_dim, groups;     // groups per head
    int page_shift;           // log2(page_size)
    int num_pages;
};

// ---- RMS norm ----
enum NormOut { kNormValues = 0, kNormCodesF16 = 1, kNormCodesI8 = 2 };
struct NormArgs {
    const void* x;
    const void* residual;
    const void* weight;
    void* out;
    float* scales;
    void* residual_out;
    int64_t m, k, x_stride, residual_stride;
    float eps;
    int f16;
    int out_kind;
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream, const char** variant);

// ---- append, read ----
struct AppendArgs {
    KvView v;
    const void* q;            // NULL: no queries
    const void* k;
    const void* val;
    int64_t q_stride, k_stride, v_stride;   // elements between tokens
    const float* cos;         // [rope_rows, rotary_dim / 2]; NULL: no rotation
    const float* sin;
    int64_t rope_rows;
    int rotary_dim, interleaved;
    void* q_out;
    int f16;
};
hipError_t launch_kv4_append(const AppendArgs& a, hipStream_t stream, const char** variant);

struct ReadArgs {
    KvView v;
    void* k_out;
    void* v_out;
    int f16;
};
hipError_t launch_kv4_read(const ReadArgs& a, hipStream_t stream, const char** variant);

// ---- attention ----
constexpr float kLog2E = 1.4426950408889634f;   // the kernels' logits are in units of log2
struct AttentionArgs {
    KvView v;
    const void* q;
    int64_t q_stride;
    void* out;
    float* lse;
    float scale;
    int causal;
    int64_t window;           // 0: none
    int64_t sinks = -1;       // first keys that stay visible; -1: none, splits cut from the whole length
    int64_t max_q, max_kv;
    void* workspace;
    int f16;
};
// Workspace bytes for a batch of these bounds.
size_t kv4_attention_workspace(const AttentionArgs& a);
hipError_t launch_kv4_attention(const AttentionArgs& a, hipStream_t stream, const char** variant);

}  // namespace mnb
