// kv4_attention.hpp -- device pieces shared by the two attention kernels over
// the 4-bit cache (few rows: kv4_attention.hip, many: kv4_prompt.hip).
#pragma once

#include <type_traits>

#include "kv4_index.hpp"
#include "kv4_plan.hpp"
#include "mnb_device.hpp"
#include "mnb_kv4.hpp"

namespace mnb {
namespace kv4 {

constexpr float kLow = -3.402823466e38f;   // "no key yet": below any logit, finite, so that differences are numbers
// The running reference M of a row is raised when the logit of a key plus the exponent
// of its value scale (the largest of its groups) passes M + kRaise, to kBelow under the
// largest such sum.  So p s' stays below 2^kRaise (fp16 ends at 2^16), and the largest
// p s' of the row is at least 2^(kBelow - 1), 2^23 above fp16's smallest normal value: a term
// keeps its bits unless it is that much smaller than the row's largest.  Of a key with
// groups of far different scales, the small groups' dims may lose theirs.
constexpr float kRaise = 15.9f, kBelow = 10.0f;

struct AttnParams {
    KvView v;
    const void* q;
    int64_t q_stride;
    void* out;
    float* lse;
    float* part_o;                    // [splits][tokens * q_heads][D] unnormalised
    float* part_ml;                   // [splits][tokens * q_heads][2]: M, sum
    float scale_log2;
    int causal;
    int window;                       // 0: none; else below max_kv
    int max_q, max_kv;
    int gqa;                          // query heads per key head
    int splits, chunk;                // keys per split, a multiple of 32
    int row_tiles, rows_per_wg;
};

hipError_t launch_prompt(const AttnParams& p, const Plan& c, int f16, hipStream_t s);
hipError_t launch_join(const AttnParams& p, int f16, hipStream_t s);

typedef uint16_t us2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f4_t mfma(const h8_t& a, const h8_t& b, const f4_t& c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ h8_t join(const h2_t q[4])
{
    return h8_t{q[0][0], q[0][1], q[1][0], q[1][1], q[2][0], q[2][1], q[3][0], q[3][1]};
}

__device__ __forceinline__ float scale_of(uint32_t m) { return (float)__builtin_bit_cast(_Float16, (uint16_t)m); }

// e with s < 2^e of an fp16 scale (low half of a word): -14 for zero and
// subnormals, 17 for infinity and NaN
__device__ __forceinline__ float top_exponent(uint32_t word) { return (float)((int)((word >> 10) & 31u) - 14); }

// the largest of a column's four lanes (16 and 32 apart), without a trip through LDS
__device__ __forceinline__ float of_quarters(float x)
{
    uint32_t u = __builtin_bit_cast(uint32_t, x);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    uint32_t lo = a[0], hi = a[1];             // an element by itself: a bit cast of a[1] takes a[0]
    u = __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)));
    const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    lo = b[0];
    hi = b[1];
    return fmaxf(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
}

// the larger of both halves each: of two words, the larger scale in the low half
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2_t, a), __builtin_bit_cast(us2_t, b)));
}

// The queries of a lane's row as the B operand of the first product: dims 32 j +
// 8 quarter .. + 7.  fp16 rows as they are.  fp32 rows as two fp16 parts: the
// row scaled by a power of two to a maximum in [2^14, 2^15), hi = fp16(q), lo =
// fp16(q - hi); the factor taken out is returned.
template <int NJ> __device__ __forceinline__ float load_query(const _Float16* q, h8_t (&f)[1][NJ])
{
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2), may_alias));
#pragma unroll
    for (int j = 0; j < NJ; ++j) f[0][j] = __builtin_bit_cast(h8_t, (u4_t)*reinterpret_cast<const raw*>(q + 32 * j));
    return 1.0f;
}
template <int NJ> __device__ __forceinline__ float load_query(const float* q, h8_t (&f)[2][NJ])
{
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
    float x[NJ][8], mx = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        const raw a = *reinterpret_cast<const raw*>(q + 32 * j), b = *reinterpret_cast<const raw*>(q + 32 * j + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[j][i] = a[i];
            x[j][4 + i] = b[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(x[j][i]) < __builtin_inff() ? fabsf(x[j][i]) : 0.0f);
    }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    int e = mx > 0.0f ? (int)(__builtin_bit_cast(uint32_t, mx) >> 23) - 127 - 14 : 0;
    e = e < -126 ? -126 : e;
    const float down = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = x[j][i] * down;
            const _Float16 top = (_Float16)s;
            f[0][j][i] = top;
            f[1][j][i] = fabsf(s) < __builtin_inff() ? (_Float16)(s - (float)top) : (_Float16)0.0f;
        }
    return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
}

// The pages of 64 blocks k0, k0 + step, ... , a lane each.  Entries past the
// table or outside the cache are replaced, so a load ahead of the sequence's end
// stays inside both.
__device__ __forceinline__ int pages_from(const KvView& v, const int32_t* table, int k0, int step, int lane)
{
    int64_t at = (int64_t)(k0 + lane * step) >> (v.page_shift - 5);
    at = at < v.table_stride ? at : v.table_stride - 1;
    return table[at];
}
__device__ __forceinline__ int page_in(const KvView& v, int pages, int i)   // i uniform
{
    const int page = __builtin_amdgcn_readlane(pages, i);
    return page < 0 || page >= v.num_pages ? 0 : page;
}

// Four outputs of a row, rounded once.
template <typename T> __device__ __forceinline__ void store4(T* out, const f4_t& y, float factor)
{
    typedef T out4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
    out4 t;
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = (T)(y[i] * factor);
    *reinterpret_cast<out4*>(out) = t;
}

__device__ __forceinline__ float log_sum(float M, float l)
{
    return l == 0.0f ? -__builtin_inff() : (M + log2f(l)) * 0.69314718055994531f;
}

}  // namespace kv4
}  // namespace mnb
