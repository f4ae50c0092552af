// kv4_attention.hip -- attention over the paged 4-bit cache.
//
//   x_tk = scale * sum_d q_td (c_kd - z_k) s_k,   p_tk = exp(x_tk - max),
//   o_t  = sum_k p_tk (c'_kd - z'_k) s'_k / sum_k p_tk,
// over the keys a query may see, in one pass with a running maximum and sum.
//
// A code minus its zero point is an integer of at most 15 in magnitude: exact
// in fp16.  So the products run on the fp16 matrix cores on exact operands: q as
// it is (fp32 queries as a (hi, lo) pair of fp16), scales applied in fp32 to the
// logits, and the value's scale multiplied into p before p is rounded to
// fp16.  That rounding and the output's are the only ones to 16 bits; with SPLIT,
// p too is a (hi, lo) pair.
//
// Layout.  A wave computes S^T = K Q^T on v_mfma_f32_16x16x32_f16: 16 keys by
// 16 query rows, the key codes of a lane being one word per 32 dims.  The
// result puts keys 4q..4q+3 of a row in the registers of lane (row, q), which is
// the operand distribution that O^T = V^T P^T wants for P if the 32 keys of a block
// are counted (q, i, tile).  The cache stores the value codes in that count, so p
// goes from the softmax to the product without leaving its lane.
//
// Rows are (token, head) pairs that share a key head, token-major, so grouped
// heads fill the 16 columns.  The running reference M is common to a row's
// four lanes and is raised only when some lane's logit passes it by 2^14 (a
// branch of the whole wave), so the usual block needs no exchange between
// lanes.  M also bounds the value scale's exponent: p s' stays below 2^14.
//
// Work split: a workgroup is four waves, KW of them sharing the keys of one
// set of rows (joined through LDS), and `splits` workgroups share a
// sequence's keys (joined by a second kernel over fp32 partials), so that a
// few long sequences fill the chip.
#include <type_traits>

#include "mnb_device.hpp"
#include "mnb_kv4.hpp"

namespace mnb {

namespace {

constexpr float kLow = -1e30f;        // "no key yet": finite, so differences stay numbers

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
    int window;                       // 0: none
    int max_q, max_kv;
    int gqa;                          // query heads per key head
    int splits, chunk;                // keys per split, a multiple of 32
    int row_tiles, rows_per_wg;
};

__device__ __forceinline__ f4_t mfma(const h8_t& a, const h8_t& b, const f4_t& c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ h8_t join(const h2_t q[4])
{
    return h8_t{q[0][0], q[0][1], q[1][0], q[1][1], q[2][0], q[2][1], q[3][0], q[3][1]};
}

// e with s < 2^e of an fp16 scale (low half of a word): -14 for zero and
// subnormals, 17 for infinity and NaN
__device__ __forceinline__ float top_exponent(uint32_t word) { return (float)((int)((word >> 10) & 31u) - 14); }

typedef uint16_t us2_t __attribute__((ext_vector_type(2)));
// the larger of both halves each: of two words, the larger scale in the low half
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2_t, a), __builtin_bit_cast(us2_t, b)));
}

// Length and new tokens of a sequence, within the bounds of the call.
struct Sequence {
    int len, first, count;            // keys; first row and number of new tokens
};
__device__ __forceinline__ Sequence sequence_of(const KvView& v, int b, int max_q, int max_kv)
{
    Sequence s;
    int64_t room = v.table_stride << v.page_shift;
    int len = v.kv_len[b];
    len = len < 0 ? 0 : len > max_kv ? max_kv : len;
    s.len = (int64_t)len > room ? (int)room : len;
    int first = b, end = b + 1;
    if (v.q_start) {
        first = v.q_start[b];
        end = v.q_start[b + 1];
    }
    first = first < 0 ? 0 : first;
    end = end > v.tokens ? v.tokens : end;
    int n = end - first;
    s.first = first;
    s.count = n < 0 ? 0 : n > max_q ? max_q : n;
    return s;
}

// The keys rows of tokens i0..i1 of a sequence can see: [lo, hi).
__device__ __forceinline__ void key_range(const AttnParams& p, const Sequence& s, int i0, int i1, int& lo, int& hi)
{
    lo = 0;
    hi = s.len;
    if (p.causal) {
        const int end = s.len - s.count + i1 + 1;
        hi = end < hi ? end : hi;
        if (p.window > 0) {
            const int from = s.len - s.count + i0 - p.window + 1;
            lo = from > 0 ? from : 0;
        }
    }
    hi = hi < lo ? lo : hi;
}

template <typename T> struct Frag8;
template <> struct Frag8<_Float16> {
    static __device__ __forceinline__ void load(const _Float16* p, float* f)
    {
        typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2), may_alias));
        const u4_t r = *reinterpret_cast<const raw*>(p);
        const h8_t h = __builtin_bit_cast(h8_t, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)h[i];
    }
};
template <> struct Frag8<float> {
    static __device__ __forceinline__ void load(const float* p, float* f)
    {
        typedef float raw __attribute__((ext_vector_type(4), aligned(4)));
        const raw a = *reinterpret_cast<const raw*>(p), b = *reinterpret_cast<const raw*>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
    }
};

// One block of 32 keys as it arrives from memory: codes in the products' own
// distribution, and the block's 64 NG scale and zero-point words, NG to a
// lane (they pass through a slot of the wave in LDS to the lanes that use them).
template <int D, int NG> struct RawBlock {
    u4_t k[D / 64], v[D / 64];
    uint32_t meta[NG];
};

// Requests a block, or nothing where `there` is 0: buffer loads past their
// range fetch no memory, so the instructions are issued in any case and the
// number of loads in flight is known when the code is compiled.
template <int D, int NG>
__device__ __forceinline__ void load_block(unsigned char* blk, bool there, int lane, RawBlock<D, NG>& r)
{
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc(blk, 0, there ? 32 * D + 256 * NG : 0, 0x00020000);
    const int v16 = lane * 16, v4 = lane * 4;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) r.k[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, v16, i * 1024, 0);
#pragma unroll
    for (int i = 0; i < NG; ++i) r.meta[i] = __builtin_amdgcn_raw_buffer_load_b32(rs, v4, 32 * D + i * 256, 0);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) r.v[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, v16, 16 * D + i * 1024, 0);
}

// Words of keys 4q .. 4q+3 (NG each) from the wave's slot.
template <int NG> __device__ __forceinline__ void four_keys(const uint32_t* slot, uint32_t* w)
{
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        const u4_t r = reinterpret_cast<const u4_t*>(slot)[i];
        w[4 * i] = r.x;
        w[4 * i + 1] = r.y;
        w[4 * i + 2] = r.z;
        w[4 * i + 3] = r.w;
    }
}

__device__ __forceinline__ float scale_of(uint32_t m) { return (float)__builtin_bit_cast(_Float16, (uint16_t)m); }

// KW waves share the keys of a row set, RW row sets make a workgroup; PF blocks
// of a wave are in registers, all but the one in work still on their way.
// WPE: waves per SIMD that the registers are held to.
template <int D, int NG, bool F32, bool SPLIT, int NR, int KW, int RW, int PF, int WPE>
__global__ __launch_bounds__(KW * RW * 64, WPE) void kv4_attention_kernel(AttnParams p)
{
    constexpr int kWaves = KW * RW;
    typedef typename std::conditional<F32, float, _Float16>::type T;
    constexpr int NJ = D / 32;                 // 32-dim steps of the first product
    constexpr int NT = D / 16;                 // 16-dim tiles of the second
    constexpr int NQ = F32 ? 2 : 1;            // fp16 parts of q
    constexpr int JG = NJ / NG;                // steps per group
    constexpr int kRows = RW * NR * 16;

    const KvView& v = p.v;
    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int kw = wave % KW, rw = wave / KW;
    const int col = lane & 15, quarter = lane >> 4;
    const int h = blockIdx.x % v.kv_heads;
    const int split = (blockIdx.x / v.kv_heads) % p.splits;
    const int tile = p.row_tiles - 1 - (int)(blockIdx.x / v.kv_heads / p.splits);   // longest key ranges first
    const int b = blockIdx.y;

    // The pages of the wave's next 64 blocks from k0 on, a lane each; entries
    // past the table or outside the cache are replaced, so a load ahead of the
    // sequence's end stays inside both.  Without a window the first block does not
    // depend on the length: the table is requested beside it.
    const int32_t* table = v.table + (int64_t)b * v.table_stride;
    auto pages_from = [&](int k0) {
        int64_t at = (int64_t)(k0 + lane * KW) >> (v.page_shift - 5);
        at = at < v.table_stride ? at : v.table_stride - 1;
        return table[at];
    };
    auto page_in = [&](int pages, int i) {     // i uniform
        const int page = __builtin_amdgcn_readlane(pages, i);
        return page < 0 || page >= v.num_pages ? 0 : page;
    };
    const int c0 = split * p.chunk, c1 = c0 + p.chunk;
    int pages = 0;
    if (p.window == 0) pages = pages_from((c0 >> 5) + kw);

    const Sequence s = sequence_of(v, b, p.max_q, p.max_kv);
    const int rows = s.count * p.gqa;
    const int row0 = tile * kRows;
    if (row0 >= rows) return;                  // the whole workgroup
    const int last_row = row0 + kRows <= rows ? row0 + kRows - 1 : rows - 1;
    int lo, hi;
    key_range(p, s, row0 / p.gqa, last_row / p.gqa, lo, hi);
    // this split's part, in blocks
    const int from = lo > c0 ? lo : c0, to = hi < c1 ? hi : c1;
    const bool any = from < to;
    if (p.splits > 1 && !any) return;          // the join reads only splits with keys
    const int blk0 = from >> 5, blk1 = any ? (to + 31) >> 5 : blk0;
    if (p.window > 0) pages = pages_from(blk0 + kw);

    // the rows of this wave: queries as the B operand, row = column of the lane
    h8_t qf[NR][NQ][NJ];
    float qs[NR];                              // fp32 queries: the factor that was taken out of the lane's row
    int64_t out_row[NR];                       // (token, head) index, < 0: none
    int pos[NR];                               // last key the row sees
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        int r = row0 + (rw * NR + n) * 16 + col;
        const bool live = r < rows;
        r = live ? r : rows - 1;
        const int token = r / p.gqa, head = h * p.gqa + r % p.gqa;
        const T* q = static_cast<const T*>(p.q) + (int64_t)(s.first + token) * p.q_stride + (int64_t)head * D + 8 * quarter;
        out_row[n] = live ? (int64_t)(s.first + token) * v.q_heads + head : -1;
        pos[n] = p.causal ? s.len - s.count + token : s.len - 1;
        if constexpr (!F32) {
            typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2), may_alias));
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                qf[n][0][j] = __builtin_bit_cast(h8_t, (u4_t)*reinterpret_cast<const raw*>(q + 32 * j));
        } else {
            // the row scaled by a power of two to a maximum in [2^14, 2^15), then
            // hi = fp16(q), lo = fp16(q - hi)
            float f[NJ][8], mx = 0.0f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                Frag8<T>::load(q + 32 * j, f[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(f[j][i]) < __builtin_inff() ? fabsf(f[j][i]) : 0.0f);
            }
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            int e = mx > 0.0f ? (int)(__builtin_bit_cast(uint32_t, mx) >> 23) - 127 - 14 : 0;
            e = e < -126 ? -126 : e;
            const float down = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
            qs[n] = __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = f[j][i] * down;
                    const _Float16 top = (_Float16)x;
                    qf[n][0][j][i] = top;
                    qf[n][NQ - 1][j][i] = fabsf(x) < __builtin_inff() ? (_Float16)(x - (float)top) : (_Float16)0.0f;
                }
        }
    }

    f4_t o[NR][NT];
    float M[NR], l[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        M[n] = kLow;
        l[n] = 0.0f;
#pragma unroll
        for (int t = 0; t < NT; ++t) o[n][t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }

    const int nblk = 1 << (v.page_shift - 5);
    const int64_t block_bytes = kv_block_bytes(D, NG);
    auto block_at = [&](int page, int blk) {
        return v.cache + (((int64_t)page * v.kv_heads + h) * nblk + (blk & (nblk - 1))) * block_bytes;
    };
    // every row of the workgroup sees the whole of a block below `whole`, from `open` on
    int whole = s.len, open = 0;
    if (p.causal) {
        whole = s.len - s.count + row0 / p.gqa + 1;
        if (p.window > 0) open = s.len - s.count + last_row / p.gqa - p.window + 1;
    }

    __shared__ __align__(16) uint32_t meta[kWaves][64 * NG];
    uint32_t* slot = meta[wave];

    auto compute = [&](const RawBlock<D, NG>& r, int blk) {
        // a wave's LDS operations complete in order: no barrier between its lanes
#pragma unroll
        for (int i = 0; i < NG; ++i) slot[i * 64 + lane] = r.meta[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        // ---- logits of 32 keys by 16 NR rows ----
        float x[NR][2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t kw4[4 * NG];
            four_keys<NG>(slot + (t * 16 + 4 * quarter) * NG, kw4);
            f4_t acc[NR][NG];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint32_t zr = zp_pair((slot[(t * 16 + col) * NG + g] >> 16) & 15u);
#pragma unroll
                for (int n = 0; n < NR; ++n) acc[n][g] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int jj = 0; jj < JG; ++jj) {
                    const int j = g * JG + jj, w = t * NJ + j;
                    h2_t a4[4];
                    unpack_zr(r.k[w >> 2][w & 3], zr, a4);
                    const h8_t a = join(a4);
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int c = 0; c < NQ; ++c) acc[n][g] = mfma(a, qf[n][c][j], acc[n][g]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float ks = scale_of(kw4[i * NG + g]) * p.scale_log2;
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        x[n][t][i] = g == 0 ? acc[n][g][i] * ks : __builtin_fmaf(acc[n][g][i], ks, x[n][t][i]);
                }
                if constexpr (F32) {
#pragma unroll
                    for (int n = 0; n < NR; ++n) x[n][t][i] *= qs[n];
                }
            }
        }
        // ---- masks, and the running reference: the largest logit plus the exponent of its value scale ----
        uint32_t vw[2][4 * NG];
#pragma unroll
        for (int t = 0; t < 2; ++t) four_keys<NG>(slot + (32 + t * 16 + 4 * quarter) * NG, vw[t]);
        const bool edge = blk * 32 + 32 > whole || blk * 32 < open;
        uint32_t seen[NR];                     // bit 4 t + i: the row sees the key
        float mxs[NR];
        if (edge) {                            // key by key: a hidden key's scale is not looked at
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                seen[n] = 0;
                mxs[n] = -__builtin_inff();
                const int below = p.causal && p.window > 0 ? pos[n] - p.window : -1;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = blk * 32 + t * 16 + 4 * quarter + i;
                        uint32_t w = vw[t][i * NG];
#pragma unroll
                        for (int g = 1; g < NG; ++g) w = max_halves(w, vw[t][i * NG + g]);
                        if (key <= pos[n] && key > below && key < s.len)
                            seen[n] |= 1u << (4 * t + i);
                        else
                            x[n][t][i] = -__builtin_inff();
                        mxs[n] = fmaxf(mxs[n], x[n][t][i] + top_exponent(w));
                    }
            }
        } else {
            uint32_t w = vw[0][0];
#pragma unroll
            for (int k = 1; k < 8 * NG; ++k) w = max_halves(w, vw[k / (4 * NG)][k % (4 * NG)]);
            const float top = top_exponent(w);
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                float m = x[n][0][0];
#pragma unroll
                for (int k = 1; k < 8; ++k) m = fmaxf(m, x[n][k >> 2][k & 3]);
                mxs[n] = m + top;
            }
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            float mx = mxs[n];
            if (__builtin_amdgcn_ballot_w64(mx > M[n] + 14.0f)) {
                mx = fmaxf(mx, __shfl_xor(mx, 16));
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                const float next = fmaxf(M[n], mx - 10.0f);
                const float alpha = exp2f(M[n] - next);
                M[n] = next;
                l[n] *= alpha;
#pragma unroll
                for (int t = 0; t < NT; ++t) o[n][t] *= alpha;
            }
        }
        // ---- p ----
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[n][t][i] = __builtin_amdgcn_exp2f(x[n][t][i] - M[n]);
                    l[n] += x[n][t][i];
                }
        // ---- O^T += V^T (p s')^T, group by group ----
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            h8_t pb[NR], pl[NR];               // p s' as the B operand, its second part
            float f[NR][8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float vs = scale_of(vw[k >> 2][(k & 3) * NG + g]);
#pragma unroll
                for (int n = 0; n < NR; ++n) f[n][k] = x[n][k >> 2][k & 3] * vs;
            }
            if (edge) {                        // a hidden key adds nothing whatever its scale is
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[n][k] = (seen[n] >> k) & 1u ? f[n][k] : 0.0f;
            }
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    pb[n][k] = (_Float16)f[n][k];
                    if constexpr (SPLIT) pl[n][k] = (_Float16)(f[n][k] - (float)pb[n][k]);
                }
            // zero points of the lane's 8 keys, in the pairs of the unpack
            h2_t zl[4], zh[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t m0 = vw[k >> 1][(2 * (k & 1)) * NG + g], m1 = vw[k >> 1][(2 * (k & 1) + 1) * NG + g];
                const uint32_t z2 = __builtin_amdgcn_perm(m1, m0, 0x07060302u);
                zl[k] = as_h2(__builtin_amdgcn_bitop3_b32(z2, 0x000F000Fu, 0xE400E400u, 0xEA));
                zh[k] = as_h2(__builtin_amdgcn_bitop3_b32(z2 << 4, 0x00F000F0u, 0xD400D400u, 0xEA));
            }
            const h2_t sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
#pragma unroll
            for (int uu = 0; uu < JG; ++uu) {
                const int u = g * JG + uu;     // dims 32u .. 32u+31: tiles 2u and 2u+1
                h2_t lo4[4], hi4[4];
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t d = r.v[u >> 1][2 * (u & 1) + w], d8 = d >> 8;
                    const uint32_t ml = 0x000F000Fu, mh = 0x00F000F0u, magic = 0x64006400u;
                    lo4[2 * w] = as_h2(__builtin_amdgcn_bitop3_b32(d, ml, magic, 0xEA)) + zl[2 * w];
                    lo4[2 * w + 1] = as_h2(__builtin_amdgcn_bitop3_b32(d8, ml, magic, 0xEA)) + zl[2 * w + 1];
                    hi4[2 * w] = as_h2(__builtin_amdgcn_bitop3_b32(d, mh, magic, 0xEA)) * sixteenth + zh[2 * w];
                    hi4[2 * w + 1] = as_h2(__builtin_amdgcn_bitop3_b32(d8, mh, magic, 0xEA)) * sixteenth + zh[2 * w + 1];
                }
                const h8_t al = join(lo4), ah = join(hi4);
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    o[n][2 * u] = mfma(al, pb[n], o[n][2 * u]);
                    o[n][2 * u + 1] = mfma(ah, pb[n], o[n][2 * u + 1]);
                    if constexpr (SPLIT) {
                        o[n][2 * u] = mfma(al, pl[n], o[n][2 * u]);
                        o[n][2 * u + 1] = mfma(ah, pl[n], o[n][2 * u + 1]);
                    }
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // before the slot's next words
    };

    // ---- the wave's blocks, PF register sets in turn ----
    int blk = blk0 + kw;
    if (blk < blk1) {
        RawBlock<D, NG> set[PF];
#pragma unroll
        for (int i = 0; i < PF; ++i)
            load_block<D, NG>(block_at(page_in(pages, i), blk + i * KW), blk + i * KW < blk1, lane, set[i]);
        // whole turns of the sets, then what is left: no branch between a load and
        // its use but the refill's, whose load is waited for where it is made
        const int steps = (blk1 - blk + KW - 1) / KW;
        int at = PF;                           // lane of `pages` with the next load's page
        for (int turn = 0; turn < steps / PF; ++turn) {
            if (at > 64 - PF) {
                pages = pages_from(blk + PF * KW);
                at = 0;
                asm volatile("" : "+v"(pages));
            }
#pragma unroll
            for (int i = 0; i < PF; ++i) {
                compute(set[i], blk);
                const int next = blk + PF * KW;
                load_block<D, NG>(block_at(page_in(pages, at), next), next < blk1, lane, set[i]);
                ++at;
                blk += KW;
            }
        }
#pragma unroll
        for (int i = 0; i < PF - 1; ++i)
            if (i < steps % PF) compute(set[i], blk + i * KW);
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        l[n] += __shfl_xor(l[n], 16);
        l[n] += __shfl_xor(l[n], 32);
    }

    // ---- waves of the same rows join through LDS, 16 rows by up to 128 dims at a time ----
    if constexpr (KW > 1) {
        constexpr int kMost = KW > 4 ? 64 : 128;           // at most 34 KB
        constexpr int kDims = D < kMost ? D : kMost, kPitch = kDims + 4;   // rows start in different banks
        constexpr int kParts = D / kDims;
        __shared__ __align__(16) float so[kWaves][16][kPitch];
        __shared__ float ml[kWaves][NR][16][2];
        if (quarter == 0) {
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                ml[wave][n][col][0] = M[n];
                ml[wave][n][col][1] = l[n];
            }
        }
        // wave kw takes every KW-th tile of its rows: M, l and o become the sums
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            float w[KW];
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                if (n + part > 0) __syncthreads();         // the last part has been read
#pragma unroll
                for (int t = 0; t < kDims / 16; ++t)
                    *reinterpret_cast<f4_t*>(&so[wave][col][16 * t + 4 * quarter]) = o[n][part * (kDims / 16) + t];
                __syncthreads();
                if (part == 0) {
                    float m = kLow, sum = 0.0f;
#pragma unroll
                    for (int k = 0; k < KW; ++k) m = fmaxf(m, ml[rw * KW + k][n][col][0]);
#pragma unroll
                    for (int k = 0; k < KW; ++k) {
                        w[k] = exp2f(ml[rw * KW + k][n][col][0] - m);
                        sum = __builtin_fmaf(ml[rw * KW + k][n][col][1], w[k], sum);
                    }
                    M[n] = m;
                    l[n] = sum;
                }
#pragma unroll
                for (int t = 0; t < kDims / 16; ++t) {
                    if ((part * (kDims / 16) + t) % KW != kw) continue;
                    f4_t a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = 0; k < KW; ++k)
                        a += *reinterpret_cast<const f4_t*>(&so[rw * KW + k][col][16 * t + 4 * quarter]) * w[k];
                    o[n][part * (kDims / 16) + t] = a;
                }
            }
        }
    }

    // ---- results or partials ----
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        if (out_row[n] < 0) continue;
        if (p.splits == 1) {
            const float inv = l[n] == 0.0f ? 0.0f : 1.0f / l[n];   // a row that sees nothing gives zeros
            T* out = static_cast<T*>(p.out) + out_row[n] * D + 4 * quarter;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t % KW != kw) continue;
                typedef T out4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
                out4 y;
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = (T)(o[n][t][i] * inv);
                *reinterpret_cast<out4*>(out + 16 * t) = y;
            }
            if (p.lse && kw == 0 && quarter == 0)
                p.lse[out_row[n]] = l[n] == 0.0f ? -__builtin_inff() : (M[n] + log2f(l[n])) * 0.69314718055994531f;
        } else {
            const int64_t at = (int64_t)split * v.tokens * v.q_heads + out_row[n];
            float* part = p.part_o + at * D + 4 * quarter;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t % KW != kw) continue;
                *reinterpret_cast<f4_t*>(part + 16 * t) = o[n][t];
            }
            if (kw == 0 && quarter == 0) {
                p.part_ml[2 * at] = M[n];
                p.part_ml[2 * at + 1] = l[n];
            }
        }
    }
}

// Joins the splits of one (token, head).  D / 4 lanes take one split's partial
// in 16-byte loads; the workgroup's 4 to 16 such groups take one split in as many
// and meet in LDS.  The weights are formed once, one split to a thread.
constexpr int kJoinThreads = 256;
constexpr int kMaxSplits = 512;

template <int D, bool F32>
__global__ __launch_bounds__(kJoinThreads) void kv4_join_kernel(AttnParams p)
{
    typedef typename std::conditional<F32, float, _Float16>::type T;
    constexpr int LPR = D / 4, GR = kJoinThreads / LPR;
    __shared__ float wgt[kMaxSplits];
    __shared__ float red[2][kJoinThreads / 64];
    __shared__ __align__(16) float sums[GR][D];
    const KvView& v = p.v;
    const int tid = threadIdx.x;
    const int h = blockIdx.x % v.q_heads;
    const int i = blockIdx.x / v.q_heads;      // token of the sequence
    const Sequence s = sequence_of(v, blockIdx.y, p.max_q, p.max_kv);
    if (i >= s.count) return;
    const int64_t row = (int64_t)(s.first + i) * v.q_heads + h;
    // the splits that wrote this row: those with a key of its workgroup
    int lo, hi;
    const int r = i * p.gqa + h % p.gqa;
    const int rows = s.count * p.gqa;
    const int r0 = r / p.rows_per_wg * p.rows_per_wg;
    const int r1 = r0 + p.rows_per_wg <= rows ? r0 + p.rows_per_wg - 1 : rows - 1;
    key_range(p, s, r0 / p.gqa, r1 / p.gqa, lo, hi);
    const int s0 = lo / p.chunk, n = hi > lo ? (hi + p.chunk - 1) / p.chunk - s0 : 0;
    const int64_t step = (int64_t)v.tokens * v.q_heads;

    const float* ml = p.part_ml + 2 * (s0 * step + row);
    float M[kMaxSplits / kJoinThreads], L[kMaxSplits / kJoinThreads], m = kLow;
#pragma unroll
    for (int k = 0; k < kMaxSplits / kJoinThreads; ++k) {
        const int at = k * kJoinThreads + tid;
        M[k] = at < n ? ml[2 * at * step] : kLow;
        L[k] = at < n ? ml[2 * at * step + 1] : 0.0f;
        m = fmaxf(m, M[k]);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    if ((tid & 63) == 0) red[0][tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kJoinThreads / 64; ++k) m = fmaxf(m, red[0][k]);
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kMaxSplits / kJoinThreads; ++k) {
        const int at = k * kJoinThreads + tid;
        const float w = exp2f(M[k] - m);
        if (at < n) wgt[at] = w;
        sum = __builtin_fmaf(L[k], w, sum);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    if ((tid & 63) == 0) red[1][tid >> 6] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kJoinThreads / 64; ++k) sum += red[1][k];

    const int g = tid / LPR, d = tid % LPR * 4;
    const float* o = p.part_o + (s0 * step + row) * D + d;
    f4_t a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int k = g; k < n; k += GR) a += *reinterpret_cast<const f4_t*>(o + k * step * D) * wgt[k];
    *reinterpret_cast<f4_t*>(&sums[g][d]) = a;
    __syncthreads();
    if (tid < D) {
        float y = 0.0f;
#pragma unroll
        for (int k = 0; k < GR; ++k) y += sums[k][tid];
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        static_cast<T*>(p.out)[row * D + tid] = (T)(y * inv);
    }
    if (p.lse && tid == 0) p.lse[row] = sum == 0.0f ? -__builtin_inff() : (m + log2f(sum)) * 0.69314718055994531f;
}

// How a call is cut: row tiles per wave, waves that share keys, waves with rows
// of their own, splits.
struct Plan {
    int nr, kw, rw, rows;             // rows per workgroup
    int row_tiles, splits, chunk;
};

Plan plan_of(const AttentionArgs& a)
{
    Plan c;
    const int64_t rows = a.max_q * (a.v.q_heads / a.v.kv_heads);
    c.nr = rows <= 16 || a.v.head_dim == 256 ? 1 : 2;
    // few rows: all waves on the same rows, the keys cut between them
    const bool few = rows <= 16 * c.nr;
    const bool brief = few && c.nr == 1 && a.v.head_dim < 256 && a.max_kv <= 1024;
    c.kw = brief ? 8 : few ? 4 : 1;
    c.rw = few ? 1 : 4;
    c.rows = c.nr * 16 * c.rw;
    c.row_tiles = (int)((rows + c.rows - 1) / c.rows);
    const int64_t units = (int64_t)c.row_tiles * a.v.kv_heads * a.v.batch;
    const int64_t least = 64 * c.kw;           // keys that give every wave two blocks
    const int64_t most = (a.max_kv + least - 1) / least;
    int64_t splits = brief ? 1 : ((few ? 2048 : 256) + units - 1) / units;
    splits = splits > most ? most : splits;
    splits = splits > kMaxSplits ? kMaxSplits : splits < 1 ? 1 : splits;
    c.chunk = (int)(((a.max_kv + splits - 1) / splits + least - 1) / least * least);
    if (c.chunk < least) c.chunk = (int)least;
    c.splits = (int)((a.max_kv + c.chunk - 1) / c.chunk);
    if (c.splits < 1) c.splits = 1;
    return c;
}

template <int D, int NG, bool F32, int NR, int KW, int RW>
hipError_t launch_rows(const AttnParams& p, const Plan& c, hipStream_t s)
{
    const dim3 grid((unsigned)(p.v.kv_heads * c.splits * c.row_tiles), (unsigned)p.v.batch);
    // as many as the registers hold without spilling
    constexpr int PF = KW == 8 ? 4 - 2 * (D == 128 && F32) : D == 256 || (D == 128 && NR == 2 && (F32 || (NG == 4 && KW > 1))) ? 1
                       : KW == 1 || (D == 128 && (F32 || NR == 2)) ? 2 : 3;
    constexpr int WPE = NR == 1 && KW == 4 && D == 128 && NG == 1 && !F32 ? 3 : 1;
    // few rows: the matrix cores have time for p in two parts
    kv4_attention_kernel<D, NG, F32, F32 || KW >= 4, NR, KW, RW, PF, WPE><<<grid, dim3(KW * RW * 64), 0, s>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || c.splits == 1) return e;
    kv4_join_kernel<D, F32><<<dim3((unsigned)(p.max_q * p.v.q_heads), (unsigned)p.v.batch), dim3(kJoinThreads), 0, s>>>(p);
    return hipGetLastError();
}

template <int D, int NG, bool F32>
hipError_t launch_groups(const AttnParams& p, const Plan& c, hipStream_t s)
{
    // head_dim 256 keeps one row tile a wave: two do not fit the registers
    constexpr int NR = D == 256 ? 1 : 2;
    if (c.kw == 1) return launch_rows<D, NG, F32, NR, 1, 4>(p, c, s);
    if constexpr (D < 256)
        if (c.kw == 8) return launch_rows<D, NG, F32, 1, 8, 1>(p, c, s);
    return c.nr == 1 ? launch_rows<D, NG, F32, 1, 4, 1>(p, c, s) : launch_rows<D, NG, F32, NR, 4, 1>(p, c, s);
}

template <int D, int NG> hipError_t launch_type(const AttnParams& p, const Plan& c, int f16, hipStream_t s)
{
    return f16 ? launch_groups<D, NG, false>(p, c, s) : launch_groups<D, NG, true>(p, c, s);
}

}  // namespace

size_t kv4_attention_workspace(const AttentionArgs& a)
{
    const Plan c = plan_of(a);
    if (c.splits == 1) return 0;
    return (size_t)c.splits * a.v.tokens * a.v.q_heads * (a.v.head_dim + 2) * 4;
}

hipError_t launch_kv4_attention(const AttentionArgs& a, hipStream_t stream, const char** variant)
{
    const Plan c = plan_of(a);
    AttnParams p;
    p.v = a.v;
    p.q = a.q;
    p.q_stride = a.q_stride;
    p.out = a.out;
    p.lse = a.lse;
    p.part_o = static_cast<float*>(a.workspace);
    p.part_ml = p.part_o ? p.part_o + (int64_t)c.splits * a.v.tokens * a.v.q_heads * a.v.head_dim : nullptr;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.causal = a.causal;
    p.window = (int)(a.window > 0x7fffffff ? 0 : a.window);
    p.max_q = (int)a.max_q;
    p.max_kv = (int)a.max_kv;
    p.gqa = a.v.q_heads / a.v.kv_heads;
    p.splits = c.splits;
    p.chunk = c.chunk;
    p.row_tiles = c.row_tiles;
    p.rows_per_wg = c.rows;
    *variant = c.splits > 1 ? "attention_kv4_split" : "attention_kv4";
    const int ng = a.v.groups;
    switch (a.v.head_dim) {
    case 64:
        return ng == 1 ? launch_type<64, 1>(p, c, a.f16, stream) : launch_type<64, 2>(p, c, a.f16, stream);
    case 128:
        return ng == 1 ? launch_type<128, 1>(p, c, a.f16, stream)
                       : ng == 2 ? launch_type<128, 2>(p, c, a.f16, stream) : launch_type<128, 4>(p, c, a.f16, stream);
    default:
        return ng == 2 ? launch_type<256, 2>(p, c, a.f16, stream)
                       : ng == 4 ? launch_type<256, 4>(p, c, a.f16, stream) : launch_type<256, 8>(p, c, a.f16, stream);
    }
}

}  // namespace mnb
