// kv4_append.hip -- new keys and values into the paged 4-bit cache, with the
// position rotation of queries and keys on the way, and stored rows back out.
//
// A group of `group` consecutive values of one head and token is stored as
//   s = fp16((hi - lo) / 15), lo = min(0, min x), hi = max(0, max x),
//   z = clamp(rne(-lo / s), 0, 15), c = clamp(rne(x / s) + z, 0, 15),
// and stands for (c - z) s.  All steps are binary32, each rounded once (no
// contraction), with 1 / s formed once per group.  s = 0 stores zeros; a group
// that holds a NaN or an infinity, or whose scale passes fp16, gets s = NaN or
// infinity and reads back as NaN.
//
// A workgroup takes one token: its sequence, position and page are found once,
// in scalar registers, and cos and sin are loaded once.  head_dim / 8 lanes take a
// head, 8 values a lane, and go through the heads in turn: a lane's 8 key codes
// are one word of the layout, and its 8 value codes are 8 bytes once the lane two
// over has lent its nibbles (a value byte holds two dims of one token, so no
// byte is shared between tokens and nothing is read back).
//
// Few tokens are bound by the chain q_start -> kv_len -> page table -> store, and
// get a lane group for every head; many by their traffic, most of it the
// queries' and the activations' own.
//
// Measured, head_dim 128, fp16, 32 heads by 8: 9665 prompt tokens with
// groups of 64, 52 us (append, 209 MB, and 216 counted in memory, so the L2 joins the parts of
// lines: 4.0 TB/s, where a large copy moves 5.15; the values' single bytes are four stores a
// lane) and 18.8 us (read, 51 MB: 2.7 TB/s; a lane loads eight single bytes for its values and
// uses one nibble of each); one token of each of 16 sequences 4.6 and 3.2 us, the chain's latency.
#include "kv4_index.hpp"
#include "mnb_device.hpp"
#include "mnb_kv4.hpp"

namespace mnb {

namespace {

// 8 consecutive elements as fp32, at any element alignment
__device__ __forceinline__ void load8(const _Float16* p, float* f)
{
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2), may_alias));
    const u4_t r = *reinterpret_cast<const raw*>(p);
    const h8_t h = __builtin_bit_cast(h8_t, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = (float)h[i];
}
__device__ __forceinline__ void load8(const float* p, float* f)
{
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
    const raw a = *reinterpret_cast<const raw*>(p), b = *reinterpret_cast<const raw*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = a[i];
        f[4 + i] = b[i];
    }
}
__device__ __forceinline__ void store8(_Float16* p, const float* f)
{
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2), may_alias));
    h8_t h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (_Float16)f[i];
    *reinterpret_cast<raw*>(p) = __builtin_bit_cast(u4_t, h);
}
__device__ __forceinline__ void store8(float* p, const float* f)
{
    typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
    *reinterpret_cast<raw*>(p) = raw{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<raw*>(p + 4) = raw{f[4], f[5], f[6], f[7]};
}

// The sequence of a token, searched by the wave: each round compares 64 spread
// offsets and keeps one 64th of the range.  Returns the number of sequences
// whose tokens all come before it (batch when the token is past the last).
__device__ __forceinline__ int find_sequence(const int32_t* q_start, int batch, int token, int lane)
{
    kv4::Search s = kv4::search_of(batch);
    while (s.n > 0) {
        const uint32_t at = s.at(lane);
        const bool before = s.holds(at) && q_start[at] <= token;
        s.keep(__builtin_popcountll(__builtin_amdgcn_ballot_w64(before)));
    }
    return uniform((int)s.lo);
}

// The token of a workgroup.  A token's codes are single bytes and words of lines that
// its block's other tokens share, and consecutive workgroups go to the 8 XCDs in turn:
// 64 tokens in a row stay on one XCD, whose L2 joins their parts of a line (append
// and read of 9665 tokens of 32 heads by 8: 56 us against 63.5 in order, 58 with 128).
// Tokens past the last whole round keep their order.
__device__ __forceinline__ int token_of(int wg, int tokens)
{
    constexpr int XCDS = 8, RUN = 64;
    const int i = wg % (XCDS * RUN);
    return wg - i + XCDS * RUN > tokens ? wg : wg - i + i % XCDS * RUN + i / XCDS;
}

struct Place {
    int64_t pos;              // position in the sequence, < 0: none
    unsigned char* page;      // block of head 0 in its page; NULL: no page
    int key;                  // token's place in its block
};

// Where a token of the workgroup is kept.  Rows of no sequence have no position,
// and page numbers and positions outside their ranges give no page.
__device__ __forceinline__ Place place_of(const KvView& v, int token, int64_t block_bytes)
{
    Place r{-1, nullptr, 0};
    int b = token, behind = 1;    // tokens of the sequence from this one on
    if (v.q_start) {
        b = find_sequence(v.q_start, v.batch, token, threadIdx.x & 63);
        if (b >= v.batch) return r;
        const int first = v.q_start[b], end = v.q_start[b + 1];
        if (token < first || token >= end) return r;   // before the first sequence, or offsets that decrease
        behind = end - token;
    }
    r.pos = (int64_t)v.kv_len[b] - behind;
    if (r.pos < 0) return r;
    const int64_t page_at = r.pos >> v.page_shift;
    if (page_at >= v.table_stride) return r;
    const int page = v.table[b * v.table_stride + page_at];
    if (page < 0 || page >= v.num_pages) return r;
    const int in_page = (int)(r.pos & ((1 << v.page_shift) - 1));
    const int nblk = 1 << (v.page_shift - 5);
    r.page = v.cache + ((int64_t)page * v.kv_heads * nblk + (in_page >> 5)) * block_bytes;
    r.key = in_page & 31;
    return r;
}

// Byte offsets inside a block (D = 8 LPR).
template <int LPR> __device__ __forceinline__ int key_word_at(int key, int l)
{
    const int w = (key >> 4) * (LPR / 4) + (l >> 2);
    return (w >> 2) * 1024 + ((l & 3) * 16 + (key & 15)) * 16 + (w & 3) * 4;
}
template <int LPR> __device__ __forceinline__ int value_byte_at(int key, int l)   // of the lane's first dim; 16 apart
{
    const int u = l >> 2, i = key & 3;
    return LPR * 128 + (u >> 1) * 1024 + (((key & 15) >> 2) * 16 + (l & 1) * 8) * 16 + (u & 1) * 8 + (key >> 4) * 4 +
           ((i & 1) * 2 + (i >> 1));
}

// The 8 values of a lane to codes, and the codes, scale and zero point of its
// group into a block.  The lanes of a head come together.
template <int LPR>
__device__ __forceinline__ void store_head(const float* x, unsigned char* block, int key, bool is_v, int l, int NG, int GL)
{
#pragma clang fp contract(off)
    constexpr int D = 8 * LPR;
    float lo = 0.0f, hi = 0.0f;
    int bad = 0;                                  // a NaN, which min and max skip
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        bad |= x[i] != x[i];
    }
    for (int off = 1; off < GL; off <<= 1) {
        lo = fminf(lo, __shfl_xor(lo, off));
        hi = fmaxf(hi, __shfl_xor(hi, off));
        bad |= __shfl_xor(bad, off);
    }
    _Float16 s16 = (_Float16)((hi - lo) * (1.0f / 15.0f));
    if (bad) s16 = (_Float16)__builtin_nanf("");
    const float s = (float)s16;
    const float inv = s > 0.0f && s < __builtin_inff() ? 1.0f / s : 0.0f;
    const float z = inv > 0.0f ? fminf(fmaxf(rintf(-lo * inv), 0.0f), 15.0f) : 0.0f;
    uint32_t nat = 0;                             // nibble i: dim d0 + i
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = fminf(fmaxf(rintf(x[i] * inv) + z, 0.0f), 15.0f);
        nat |= (uint32_t)c << (4 * i);
    }
    const uint32_t other = (uint32_t)__shfl_xor((int)nat, 2);
    if (l % GL == 0) {
        const int meta = 32 * D + (is_v ? 128 * NG : 0) + (key * NG + l / GL) * 4;
        *reinterpret_cast<uint32_t*>(block + meta) =
            (uint32_t)__builtin_bit_cast(uint16_t, s16) | ((uint32_t)z << 16);
    }
    if (!is_v) {
        // k-offsets 0,2,4,6 in the low four nibbles, 1,3,5,7 in the high four
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= ((nat >> (4 * i)) & 15u) << (4 * nibble_slot(i));
        *reinterpret_cast<uint32_t*>(block + key_word_at<LPR>(key, l)) = w;
    } else {
        // lanes l and l ^ 2 hold dims 16 apart: the low and the high nibble of 8
        // bytes, of which each writes four
        const bool upper = (l & 2) != 0;
        const uint32_t lo4 = upper ? other : nat, hi4 = upper ? nat : other;
        unsigned char* dst = block + value_byte_at<LPR>(key, l);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = j + (upper ? 4 : 0);
            dst[16 * i] = (unsigned char)(((lo4 >> (4 * i)) & 15u) | (((hi4 >> (4 * i)) & 15u) << 4));
        }
    }
}

template <typename T, int LPR>
__global__ __launch_bounds__(1024) void kv4_append_kernel(AppendArgs a)
{
#pragma clang fp contract(off)
    constexpr int D = 8 * LPR;
    const KvView& v = a.v;
    const int token = token_of(blockIdx.x, v.tokens);
    const int l = threadIdx.x % LPR, d0 = 8 * l;
    const int hq = a.q ? v.q_heads : 0;
    const int items = hq + 2 * v.kv_heads;       // heads of q, then of k, then of v
    const int step = blockDim.x / LPR;
    const int NG = v.groups, GL = LPR / NG;      // lanes of a group
    const int half = a.rotary_dim >> 1;
    const bool turn = a.cos && d0 < a.rotary_dim;
    const bool second = turn && !a.interleaved && d0 >= half;
    const T* const srcs[3] = {static_cast<const T*>(a.q) + token * a.q_stride, static_cast<const T*>(a.k) + token * a.k_stride,
                              static_cast<const T*>(a.val) + token * a.v_stride};
    // 8 values of an item, and the 8 they are turned with
    auto fetch = [&](int item, float* x, float* y) {
        const int kind = item < hq ? 0 : item < hq + v.kv_heads ? 1 : 2;
        const T* src = (kind == 0 ? srcs[0] : kind == 1 ? srcs[1] : srcs[2]) +
                       (int64_t)(item - (kind == 0 ? 0 : kind == 1 ? hq : hq + v.kv_heads)) * D;
        load8(src + d0, x);
        if (kind < 2 && turn && !a.interleaved) load8(src + (second ? d0 - half : d0 + half), y);
    };
    int item = threadIdx.x / LPR;
    float x[8], y[8];
    if (item < items) fetch(item, x, y);

    const int64_t block_bytes = kv_block_bytes(D, NG);
    const int64_t head_bytes = block_bytes << (v.page_shift - 5);
    const Place at = place_of(v, token, block_bytes);
    float c[8], s[8];                            // interleaved: four of each
    if (turn) {
        int64_t row = at.pos < 0 ? 0 : at.pos;
        row = (row < a.rope_rows ? row : a.rope_rows - 1) * half;
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = a.cos[row + (d0 >> 1) + i];
                s[i] = a.sin[row + (d0 >> 1) + i];
            }
        } else {
            load8(a.cos + row + (second ? d0 - half : d0), c);
            load8(a.sin + row + (second ? d0 - half : d0), s);
        }
    }
    for (; item < items; item += step) {
        const bool is_q = item < hq, is_v = item >= hq + v.kv_heads;
        if (turn && !is_v) {
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = x[2 * i], o = x[2 * i + 1];
                    x[2 * i] = e * c[i] - o * s[i];
                    x[2 * i + 1] = o * c[i] + e * s[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p = x[i] * c[i], t = y[i] * s[i];
                    x[i] = second ? p + t : p - t;
                }
            }
        }
        if (is_q)
            store8(static_cast<T*>(a.q_out) + ((int64_t)token * v.q_heads + item) * D + d0, x);
        else if (at.page)
            store_head<LPR>(x, at.page + (item - hq - (is_v ? v.kv_heads : 0)) * head_bytes, at.key, is_v, l, NG, GL);
        if (item + step < items) fetch(item + step, x, y);
    }
}

template <typename T, int LPR>
__global__ __launch_bounds__(1024) void kv4_read_kernel(ReadArgs a)
{
    constexpr int D = 8 * LPR;
    const KvView& v = a.v;
    const int token = token_of(blockIdx.x, v.tokens);
    const int l = threadIdx.x % LPR;
    const int NG = v.groups, GL = LPR / NG;
    const int step = blockDim.x / LPR;
    const int64_t block_bytes = kv_block_bytes(D, NG);
    const int64_t head_bytes = block_bytes << (v.page_shift - 5);
    const Place at = place_of(v, token, block_bytes);
    for (int item = threadIdx.x / LPR; item < 2 * v.kv_heads; item += step) {
        const bool is_v = item >= v.kv_heads;
        const int h = is_v ? item - v.kv_heads : item;
        void* out = is_v ? a.v_out : a.k_out;
        if (!out) continue;
        float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (at.page) {
            const unsigned char* block = at.page + h * head_bytes;
            const uint32_t m = *reinterpret_cast<const uint32_t*>(block + 32 * D + (is_v ? 128 * NG : 0) +
                                                                  (at.key * NG + l / GL) * 4);
            const float s = (float)__builtin_bit_cast(_Float16, (uint16_t)m);
            const int z = (int)((m >> 16) & 15u);
            int c[8];
            if (!is_v) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(block + key_word_at<LPR>(at.key, l));
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = (int)code_at(w, i);
            } else {
                const unsigned char* src = block + value_byte_at<LPR>(at.key, l);
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = (src[16 * i] >> ((l & 2) * 2)) & 15;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = (float)(c[i] - z) * s;
        }
        store8(static_cast<T*>(out) + ((int64_t)token * v.kv_heads + h) * D + 8 * l, x);
    }
}

// Threads of a token's workgroup: a lane group for every head while there are few
// tokens (each then goes through its chain of loads once), up to 256 threads
// otherwise (9665 tokens, append and read: 63 us; with 1024 threads 106, with 512 72, and
// with 128 as fast, but 17.5 against 15.5 us for 1200 tokens of 64 heads).
inline dim3 threads_for(int tokens, int items, int lanes)
{
    const int most = tokens <= 512 ? 1024 : 256;
    const int want = (items * lanes + 63) / 64 * 64;
    return dim3((unsigned)(want < most ? want : most));
}

}  // namespace

hipError_t launch_kv4_append(const AppendArgs& a, hipStream_t stream, const char** variant)
{
    const int lpr = a.v.head_dim / 8;
    const dim3 grid((unsigned)a.v.tokens);
    const dim3 block = threads_for(a.v.tokens, (a.q ? a.v.q_heads : 0) + 2 * a.v.kv_heads, lpr);
    *variant = "kv4_append";
    switch (lpr) {
    case 8:
        if (a.f16) kv4_append_kernel<_Float16, 8><<<grid, block, 0, stream>>>(a);
        else kv4_append_kernel<float, 8><<<grid, block, 0, stream>>>(a);
        break;
    case 16:
        if (a.f16) kv4_append_kernel<_Float16, 16><<<grid, block, 0, stream>>>(a);
        else kv4_append_kernel<float, 16><<<grid, block, 0, stream>>>(a);
        break;
    default:
        if (a.f16) kv4_append_kernel<_Float16, 32><<<grid, block, 0, stream>>>(a);
        else kv4_append_kernel<float, 32><<<grid, block, 0, stream>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_kv4_read(const ReadArgs& a, hipStream_t stream, const char** variant)
{
    const int lpr = a.v.head_dim / 8;
    const dim3 grid((unsigned)a.v.tokens);
    const dim3 block = threads_for(a.v.tokens, 2 * a.v.kv_heads, lpr);
    *variant = "kv4_read";
    switch (lpr) {
    case 8:
        if (a.f16) kv4_read_kernel<_Float16, 8><<<grid, block, 0, stream>>>(a);
        else kv4_read_kernel<float, 8><<<grid, block, 0, stream>>>(a);
        break;
    case 16:
        if (a.f16) kv4_read_kernel<_Float16, 16><<<grid, block, 0, stream>>>(a);
        else kv4_read_kernel<float, 16><<<grid, block, 0, stream>>>(a);
        break;
    default:
        if (a.f16) kv4_read_kernel<_Float16, 32><<<grid, block, 0, stream>>>(a);
        else kv4_read_kernel<float, 32><<<grid, block, 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace mnb
