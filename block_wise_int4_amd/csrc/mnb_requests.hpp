// mnb_requests.hpp -- launchers of the operators that serve many requests at
// once: their low-rank adapters and the verification of their drafted tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mnb {

// ---- low-rank adapters beside a projection ----
struct AdapterArgs {
    const void* a;            // [count, rank, k]
    const void* b;            // [count, n, rank]
    const float* scales;      // [count], or NULL: 1
    const int32_t* ranks;     // [count], or NULL: rank
    const int32_t* adapter;   // [m]
    const void* x;
    const void* base;         // NULL: zeros
    void* y;
    int64_t m, n, k;
    int rank, count;
    int64_t x_stride, base_stride, y_stride;
    void* workspace;
    int f16;
};
size_t adapters_workspace(int64_t m, int64_t n, int64_t k, int rank, int count, int f16);
hipError_t launch_adapters(const AdapterArgs& a, hipStream_t stream, const char** variant);

// ---- drafted tokens against the target's probabilities ----
struct VerifyArgs {
    const void* target;       // [tokens, vocab]
    const void* draft;        // the same, or NULL: the drafts are certain
    int64_t target_stride, draft_stride;
    const int32_t* ids;       // [tokens]
    const int32_t* q_start;   // [batch + 1], or NULL
    const float* accept;      // [tokens]
    const float* pick;        // [batch]
    int32_t* out;             // [tokens]
    int32_t* accepted;        // [batch]
    int64_t batch, tokens, vocab;
    void* workspace;
    int f16;
};
constexpr int kVerifyChunk = 1024;   // tokens of a wave
inline int64_t verify_chunks(int64_t vocab) { return (vocab + kVerifyChunk - 1) / kVerifyChunk; }
// Two sums in 64 bits per sequence and chunk.
inline size_t verify_workspace(int64_t batch, int64_t vocab) { return (size_t)(batch * verify_chunks(vocab)) * 16; }
hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream, const char** variant);

}  // namespace mnb
