// kv4_attention.hip -- attention over the paged 4-bit cache: the kernel for few
// query rows per key head, the join of splits, and the choice between kernels.
//
//   x_tk = scale * sum_d q_td (c_kd - z_k) s_k,   p_tk = exp(x_tk - max),
//   o_t  = sum_k p_tk (c'_kd - z'_k) s'_k / sum_k p_tk,
// over the keys a query may see, in one pass with a running maximum and sum.
//
// A code minus its zero point is an integer of at most 15 in magnitude: exact
// in fp16.  So the products run on the fp16 matrix cores on exact operands: q as
// it is (fp32 queries as a (hi, lo) pair of fp16, 22 bits), scales applied in fp32 to
// the logits, and the value's scale multiplied into p before p is rounded to fp16.
// That rounding (2^-12 on average over many keys) and the output's are the only
// ones to 16 bits; in fp32 calls p too is a (hi, lo) pair: the matrix cores' fp32 products
// run at a sixteenth of their fp16 rate, and two parts cost twice the products.
//
// Layout.  A wave computes S^T = K Q^T on v_mfma_f32_16x16x32_f16: 16 keys by
// 16 columns, the key codes of a lane being one word per 32 dims.  The result
// puts keys 4q..4q+3 of a column in the registers of lane (column, q), which is
// the operand distribution that O^T = V^T P^T wants for P if the 32 keys of a block
// are counted (q, i, tile).  The cache stores the value codes in that count, so p
// goes from the softmax to the product without leaving its lane.
//
// Rows are (token, head) pairs that share a key head.  With at most 4 (8) rows
// the 16 columns hold them 4 (2) times over, and each copy takes a quarter (half)
// of the keys through the softmax: its other entries of P are zeros, and
// the copies' sums are added at the end.  The vector work of the softmax, which
// bounds the kernel at full occupancy, then falls with the rows.  (The value's zero
// points are taken off in the unpack: as one sum p s' z' per row, subtracted at
// the end, they would cost 14 instructions a block less, but the difference of
// the two sums loses what a row of equal codes and zero points leaves.)
//
// The running reference M of a column is common to its four lanes and is looked at
// only when some lane's logit and value scale may pass it by 2^kRaise (a branch of the whole
// wave), so the usual block needs no exchange between lanes.
//
// Work split: the waves of a workgroup share the keys of one set of rows (joined
// through LDS), and `splits` workgroups share a sequence's keys (joined by a second
// kernel over fp32 partials), so that a few long sequences fill the chip.
//
// Measured, head_dim 128, fp16, 8 key heads by 4: 32 sequences of up to 8192 keys 44.4 us and
// 5.3 for the join (182 MB asked for and counted from memory: 4.1 TB/s without the join, where a large
// copy moves 5.15); one of 131072 keys with groups of 64, 30.7 and 4.7 us (151 MB: 4.9 TB/s); one of
// 1000 keys 9.9 us, without a join: launch, the chain to the first block, a wave's 4 blocks one
// after the other (their loads are asked for at once) and the join in LDS, on 8 workgroups: a
// wave waits 37% of its cycles for data and 25% for an issue slot.
// 8 sequences of 5 new tokens, 3 heads to a key head, a window of 3000 keys, in fp32 at
// head_dim 64, 12.0 and 4.6 us: bound by the latency of
// the chain to the first block, two blocks' work a wave, and the second launch.
#include "kv4_attention.hpp"

namespace mnb {
namespace kv4 {

namespace {

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

// N consecutive words from the wave's slot.
template <int N> __device__ __forceinline__ void words(const uint32_t* slot, uint32_t* w)
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const u4_t r = reinterpret_cast<const u4_t*>(slot)[i];
            w[4 * i] = r.x;
            w[4 * i + 1] = r.y;
            w[4 * i + 2] = r.z;
            w[4 * i + 3] = r.w;
        }
    } else if constexpr (N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const uint64_t r = reinterpret_cast<const uint64_t*>(slot)[i];
            w[2 * i] = (uint32_t)r;
            w[2 * i + 1] = (uint32_t)(r >> 32);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = slot[i];
    }
}

// f is called with the rotations of a row of 16 lanes that bring the copies of a
// column together (each leaves twice as many of them summed).
template <int N> struct Turn {
    __device__ __forceinline__ float operator()(float x) const
    {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x120 + N, 0xF, 0xF, false));
    }
};
template <int GRP, typename F> __device__ __forceinline__ void for_copies(F f)
{
    f(Turn<8>());
    if constexpr (GRP == 4) f(Turn<4>());
}

// GRP column groups (4: up to 4 rows, 2: up to 8, 1: up to 16 NR).  KW waves
// share the keys; PF blocks of a wave are in registers, all but the one in work
// still on their way.  Head size 256 is held to two waves a SIMD where that costs no more than 2
// registers in memory: with groups of 32 in fp32 and up to 4 rows (8 sequences of 4000 keys 26.6 us,
// 31.8 with one wave), and with larger groups.
template <int D, int NG, bool F32, int GRP, int NR, int KW, int PF>
__global__ __launch_bounds__(KW * 64, D == 256 && (GRP == 4 || NG <= 4) ? 2 : 1) void kv4_attention_kernel(AttnParams p)
{
    static_assert(GRP == 1 || NR == 1, "copies of the rows need one column tile");
    typedef typename std::conditional<F32, float, _Float16>::type T;
    constexpr bool SPLIT = F32;                // p in two parts
    constexpr int NJ = D / 32;                 // 32-dim steps of the first product
    constexpr int NT = D / 16;                 // 16-dim tiles of the second
    constexpr int NQ = F32 ? 2 : 1;            // fp16 parts of q
    constexpr int JG = NJ / NG;                // steps per group
    constexpr int I = 4 / GRP;                 // keys per tile that a lane takes through the softmax
    constexpr int R = 16 / GRP;                // rows of a column tile
    constexpr int kRows = NR * R;

    const KvView& v = p.v;
    const int lane = threadIdx.x & 63;
    const int kw = uniform(threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int copy = col / R;                  // which quarter (half) of the keys
    const int h = blockIdx.x % v.kv_heads;
    const int split = (blockIdx.x / v.kv_heads) % p.splits;
    const int tile = blockIdx.x / v.kv_heads / p.splits;
    const int b = blockIdx.y;

    // without a window the first block does not depend on the length: the table is
    // requested beside it
    const int32_t* table = v.table + (int64_t)b * v.table_stride;
    const int c0 = split * p.chunk, c1 = c0 + p.chunk;
    int pages = 0;
    if (p.window == 0) pages = pages_from(v, table, (c0 >> 5) + kw, KW, lane);

    const Sequence s = sequence_of(v, b, p.max_q, p.max_kv);
    const int rows = s.count * p.gqa;
    const int row0 = tile * kRows;
    if (row0 >= rows) return;                  // the whole workgroup
    const int last_row = row0 + kRows <= rows ? row0 + kRows - 1 : rows - 1;
    int lo, hi;
    key_range(p.causal, p.window, s, row0 / p.gqa, last_row / p.gqa, lo, hi);
    // this split's part, in blocks
    const int from = lo > c0 ? lo : c0, to = hi < c1 ? hi : c1;
    const bool any = from < to;
    if (p.splits > 1 && !any) return;          // the join reads only splits with keys
    const int blk0 = from >> 5, blk1 = any ? (to + 31) >> 5 : blk0;
    if (p.window > 0) pages = pages_from(v, table, blk0 + kw, KW, lane);

    const int nblk = 1 << (v.page_shift - 5);
    const int64_t block_bytes = kv_block_bytes(D, NG);
    auto block_at = [&](int page, int blk) {
        return v.cache + (((int64_t)page * v.kv_heads + h) * nblk + (blk & (nblk - 1))) * block_bytes;
    };

    h8_t qf[NR][NQ][NJ];
    float qs[NR];                              // fp32 queries: the factor that was taken out of the row
    int pos[NR];                               // last key the row sees
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        int r = row0 + n * 16 + col % R;
        r = r < rows ? r : rows - 1;
        const int token = r / p.gqa, head = h * p.gqa + r % p.gqa;
        pos[n] = p.causal ? s.before + token : s.len - 1;
        qs[n] = load_query<NJ>(static_cast<const T*>(p.q) + (int64_t)(s.first + token) * p.q_stride + (int64_t)head * D +
                                   8 * quarter, qf[n]);
    }
    // every row of the workgroup sees the whole of a block below `whole`, from `open` on
    int whole = s.len, open = 0;
    if (p.causal) {
        whole = s.before + row0 / p.gqa + 1;
        if (p.window > 0) open = s.before + last_row / p.gqa - p.window + 1;
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
    // where the lane's two (four, eight) entries of P go among its 8 keys: masks
    // of the halves of the four registers
    uint32_t put[2] = {0, 0};
    if constexpr (GRP == 4) {
        const uint32_t half = (copy & 1) ? 0xFFFF0000u : 0x0000FFFFu;
        put[0] = copy < 2 ? half : 0u;
        put[1] = copy < 2 ? 0u : half;
    } else if constexpr (GRP == 2) {
        put[0] = copy == 0 ? 0xFFFFFFFFu : 0u;
        put[1] = ~put[0];
    }

    __shared__ __align__(16) uint32_t meta[KW][64 * NG];
    uint32_t* slot = meta[kw];

    auto compute = [&](const RawBlock<D, NG>& r, int blk) {
        // a wave's LDS operations complete in order: no barrier between its lanes
#pragma unroll
        for (int i = 0; i < NG; ++i) slot[i * 64 + lane] = r.meta[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        uint32_t kwd[2][I * NG], vwd[2][I * NG];   // words of the lane's own keys
        const int mine = 4 * quarter + copy * I;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            words<I * NG>(slot + (t * 16 + mine) * NG, kwd[t]);
            words<I * NG>(slot + (32 + t * 16 + mine) * NG, vwd[t]);
        }
        // ---- logits less M ----
        float x[NR][2][I], Mu[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) Mu[n] = M[n] == kLow ? 0.0f : M[n];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint32_t zr = zp_pair((slot[(t * 16 + col) * NG + g] >> 16) & 15u);
                f4_t acc[NR];
#pragma unroll
                for (int n = 0; n < NR; ++n) acc[n] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int jj = 0; jj < JG; ++jj) {
                    const int j = g * JG + jj, w = t * NJ + j;
                    h2_t a4[4];
                    unpack_zr(r.k[w >> 2][w & 3], zr, a4);
                    const h8_t k8 = join(a4);
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int c = 0; c < NQ; ++c) acc[n] = mfma(k8, qf[n][c][j], acc[n]);
                }
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int i = 0; i < I; ++i) {
                        float dot = acc[n][i];         // of the lane's own keys
                        if constexpr (GRP == 2) dot = copy ? acc[n][2 + i] : acc[n][i];
                        if constexpr (GRP == 4) {
                            const float e0 = (copy & 1) ? acc[n][1] : acc[n][0], e1 = (copy & 1) ? acc[n][3] : acc[n][2];
                            dot = (copy & 2) ? e1 : e0;
                        }
                        const float ks = scale_of(kwd[t][i * NG + g]) * p.scale_log2;
                        // fp32 queries come back to their scale last, with M
                        const float add = g == 0 ? (F32 ? 0.0f : -Mu[n]) : x[n][t][i];
                        x[n][t][i] = __builtin_fmaf(dot, ks, add);
                    }
            }
        }
        if constexpr (F32) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int k = 0; k < 2 * I; ++k) x[n][k / I][k % I] = __builtin_fmaf(x[n][k / I][k % I], qs[n], -Mu[n]);
        }
        // ---- masks, and what the running reference must not fall too far below: of each key its
        // logit plus the exponent of its value scale, or, where no key is hidden, the largest of
        // either as a bound ----
        const bool edge = blk * 32 + 32 > whole || blk * 32 < open;
        uint32_t seen[NR];                     // bit t I + i: the row sees the key
        float mxs[NR];
        auto largest = [&](int n) {
            float mx = -__builtin_inff();
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < I; ++i) {
                    uint32_t w = vwd[t][i * NG];
#pragma unroll
                    for (int g = 1; g < NG; ++g) w = max_halves(w, vwd[t][i * NG + g]);
                    mx = fmaxf(mx, x[n][t][i] + top_exponent(w));
                }
            return mx;
        };
        if (edge) {
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                seen[n] = 0;
                const int below = p.causal && p.window > 0 ? pos[n] - p.window : -1;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < I; ++i) {
                        const int key = blk * 32 + t * 16 + mine + i;
                        if (key <= pos[n] && key > below && key < s.len)
                            seen[n] |= 1u << (I * t + i);
                        else
                            x[n][t][i] = -__builtin_inff();    // whatever its scale is
                    }
                mxs[n] = largest(n);
            }
        } else {
            uint32_t w = vwd[0][0];
#pragma unroll
            for (int k = 1; k < 2 * I * NG; ++k) w = max_halves(w, vwd[k / (I * NG)][k % (I * NG)]);
            const float top = top_exponent(w);
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                float m = x[n][0][0];
#pragma unroll
                for (int k = 1; k < 2 * I; ++k) m = fmaxf(m, x[n][k / I][k % I]);
                mxs[n] = m + top;
            }
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const bool first = M[n] == kLow;
            if (__builtin_amdgcn_ballot_w64(mxs[n] > (first ? -__builtin_inff() : kRaise))) {
                const float mx = of_quarters(edge ? mxs[n] : largest(n));
                // by the row's own visible keys alone: neither the rows beside it nor hidden keys
                // decide a bit of it
                const bool up = mx > (first ? -__builtin_inff() : kRaise);
                const float next = up ? Mu[n] + mx - kBelow : Mu[n];
                const float alpha = first ? 1.0f : exp2f(Mu[n] - next);   // nothing was summed before the first
                const float by = next - Mu[n];
                M[n] = up ? next : M[n];
                l[n] *= alpha;
#pragma unroll
                for (int t = 0; t < NT; ++t) o[n][t] *= alpha;
#pragma unroll
                for (int k = 0; k < 2 * I; ++k) x[n][k / I][k % I] -= by;
            }
        }
        // ---- p ----
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int k = 0; k < 2 * I; ++k) {
                float& e = x[n][k / I][k % I];
                e = __builtin_amdgcn_exp2f(e);
                l[n] += e;
            }
        // ---- O^T += V^T (p s')^T, group by group ----
        uint32_t vall[2][4 * NG];
#pragma unroll
        for (int t = 0; t < 2; ++t) words<4 * NG>(slot + (32 + t * 16 + 4 * quarter) * NG, vall[t]);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            h8_t pb[NR], pl[NR];               // p s' as the B operand, its second part
            float f[NR][2 * I];
#pragma unroll
            for (int k = 0; k < 2 * I; ++k) {
                const float vs = scale_of(vwd[k / I][(k % I) * NG + g]);
#pragma unroll
                for (int n = 0; n < NR; ++n) f[n][k] = x[n][k / I][k % I] * vs;
            }
            if (edge) {                        // a hidden key adds nothing whatever its scale is
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int k = 0; k < 2 * I; ++k) f[n][k] = (seen[n] >> k) & 1u ? f[n][k] : 0.0f;
            }
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                _Float16 top[2 * I], low[2 * I];
#pragma unroll
                for (int k = 0; k < 2 * I; ++k) {
                    top[k] = (_Float16)f[n][k];
                    low[k] = SPLIT ? (_Float16)(f[n][k] - (float)top[k]) : (_Float16)0.0f;
                }
                auto spread = [&](const _Float16* e) {
                    u4_t w;
                    if constexpr (GRP == 1) {
                        h8_t b8;
#pragma unroll
                        for (int k = 0; k < 2 * I; ++k) b8[k] = e[k];
                        return b8;
                    } else {
                        const uint32_t d0 = as_u32(GRP == 4 ? h2_t{e[0], e[0]} : h2_t{e[0], e[1]});
                        const uint32_t d1 = as_u32(GRP == 4 ? h2_t{e[1], e[1]} : h2_t{e[2], e[3]});
                        w.x = d0 & put[0];
                        w.y = d0 & put[1];
                        w.z = d1 & put[0];
                        w.w = d1 & put[1];
                        return __builtin_bit_cast(h8_t, w);
                    }
                };
                pb[n] = spread(top);
                if constexpr (SPLIT) pl[n] = spread(low);
            }
            const h2_t sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
            // zero points of all 8 keys of the lane's quarter, in the pairs of the unpack
            h2_t zl[4], zh[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t m0 = vall[k >> 1][(2 * (k & 1)) * NG + g], m1 = vall[k >> 1][(2 * (k & 1) + 1) * NG + g];
                const uint32_t z2 = __builtin_amdgcn_perm(m1, m0, 0x07060302u);
                zl[k] = as_h2(__builtin_amdgcn_bitop3_b32(z2, 0x000F000Fu, 0xE400E400u, 0xEA));
                zh[k] = as_h2(__builtin_amdgcn_bitop3_b32(z2 << 4, 0x00F000F0u, 0xD400D400u, 0xEA));
            }
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
            load_block<D, NG>(block_at(page_in(v, pages, i), blk + i * KW), blk + i * KW < blk1, lane, set[i]);
        // whole turns of the sets, then what is left: no branch between a load and
        // its use but the refill's, whose load is waited for where it is made
        const int steps = (blk1 - blk + KW - 1) / KW;
        int at = PF;                           // lane of `pages` with the next load's page
        for (int turn = 0; turn < steps / PF; ++turn) {
            if (at > 64 - PF) {
                pages = pages_from(v, table, blk + PF * KW, KW, lane);
                at = 0;
                asm volatile("" : "+v"(pages));
            }
#pragma unroll
            for (int i = 0; i < PF; ++i) {
                compute(set[i], blk);
                const int next = blk + PF * KW;
                load_block<D, NG>(block_at(page_in(v, pages, at), next), next < blk1, lane, set[i]);
                ++at;
                blk += KW;
            }
        }
#pragma unroll
        for (int i = 0; i < PF - 1; ++i)
            if (i < steps % PF) compute(set[i], blk + i * KW);
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {             // the sum of a column over its lanes
        l[n] += __shfl_xor(l[n], 16);
        l[n] += __shfl_xor(l[n], 32);
    }

    // ---- the copies of a row join by rotations of the 16 columns ----
    if constexpr (GRP > 1) {
        float m = M[0];
        for_copies<GRP>([&](auto turn) { m = fmaxf(m, turn(m)); });
        const float w = exp2f(M[0] - m);
        M[0] = m;
        l[0] *= w;
        for_copies<GRP>([&](auto turn) { l[0] += turn(l[0]); });
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y = o[0][t][i] * w;
                for_copies<GRP>([&](auto turn) { y += turn(y); });
                o[0][t][i] = y;
            }
    }
    // ---- the waves join through LDS, R rows by up to 128 dims at a time ----
    constexpr int kMost = KW * R > 64 ? 64 : 128;          // at most 34 KB
    constexpr int kDims = D < kMost ? D : kMost, kPitch = kDims + 4;   // rows start in different banks
    constexpr int kParts = D / kDims, kTiles = kDims / 16, kQuads = kDims / 4;
    __shared__ __align__(16) float so[KW][R][kPitch];
    __shared__ float ml[KW][NR][R][2];
    if (quarter == 0 && copy == 0) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            ml[kw][n][col][0] = M[n];
            ml[kw][n][col][1] = l[n];
        }
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
            if (n + part > 0) __syncthreads();             // the last part has been read
            if (copy == 0) {
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
                    *reinterpret_cast<f4_t*>(&so[kw][col][16 * t + 4 * quarter]) = o[n][part * kTiles + t];
            }
            __syncthreads();
            // four dims of a row to a thread
            for (int i = threadIdx.x; i < R * kQuads; i += KW * 64) {
                const int row = i / kQuads, d = i % kQuads * 4;
                const int r = row0 + n * 16 + row;
                if (r >= rows) continue;
                float m = kLow, sum = 0.0f;
                f4_t y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < KW; ++k) m = fmaxf(m, ml[k][n][row][0]);
#pragma unroll
                for (int k = 0; k < KW; ++k) {
                    const float w = exp2f(ml[k][n][row][0] - m);
                    sum = __builtin_fmaf(ml[k][n][row][1], w, sum);
                    y += *reinterpret_cast<const f4_t*>(&so[k][row][d]) * w;
                }
                const int64_t out_row = (int64_t)(s.first + r / p.gqa) * v.q_heads + h * p.gqa + r % p.gqa;
                const int64_t part_row = (int64_t)split * v.tokens * v.q_heads + out_row;
                if (p.splits == 1)                         // a row that sees nothing gives zeros
                    store4(static_cast<T*>(p.out) + out_row * D + part * kDims + d, y, sum == 0.0f ? 0.0f : 1.0f / sum);
                else
                    *reinterpret_cast<f4_t*>(p.part_o + part_row * D + part * kDims + d) = y;
                if (part == 0 && d == 0) {
                    if (p.splits > 1) {
                        p.part_ml[2 * part_row] = m;
                        p.part_ml[2 * part_row + 1] = sum;
                    } else if (p.lse) {
                        p.lse[out_row] = log_sum(m, sum);
                    }
                }
            }
        }
    }
}

// The splits that wrote row h of token i: those with a key of its workgroup.
// Returns how many, the first one in s0.
__device__ __forceinline__ int splits_of(const AttnParams& p, const Sequence& s, int i, int h, int& s0)
{
    int lo, hi;
    const int r = i * p.gqa + h % p.gqa;
    const int rows = s.count * p.gqa;
    const int r0 = r / p.rows_per_wg * p.rows_per_wg;
    const int r1 = r0 + p.rows_per_wg <= rows ? r0 + p.rows_per_wg - 1 : rows - 1;
    key_range(p.causal, p.window, s, r0 / p.gqa, r1 / p.gqa, lo, hi);
    s0 = lo / p.chunk;
    return hi > lo ? (hi + p.chunk - 1) / p.chunk - s0 : 0;
}

constexpr int kJoinThreads = 256;
constexpr int kWaveSplits = 16;       // most splits that a wave joins alone

// Joins the splits of one (token, head), one wave to each: lane k forms split k's
// weight, and D / 4 lanes take one split's partial in 16-byte loads.
template <int D, bool F32>
__global__ __launch_bounds__(kJoinThreads) void kv4_join_rows_kernel(AttnParams p)
{
    typedef typename std::conditional<F32, float, _Float16>::type T;
    constexpr int LPR = D / 4, GR = 64 / LPR;
    const KvView& v = p.v;
    const int lane = threadIdx.x & 63;
    const int at = uniform(blockIdx.x * (kJoinThreads / 64) + (threadIdx.x >> 6));
    const int h = at % v.q_heads, i = at / v.q_heads;      // token of the sequence
    const Sequence s = sequence_of(v, blockIdx.y, p.max_q, p.max_kv);
    if (i >= s.count) return;
    const int64_t row = (int64_t)(s.first + i) * v.q_heads + h;
    int s0;
    const int n = splits_of(p, s, i, h, s0);               // at most kWaveSplits
    const int64_t step = (int64_t)v.tokens * v.q_heads;
    const float* ml = p.part_ml + 2 * (s0 * step + row);
    const float M = lane < n ? ml[2 * lane * step] : kLow;
    const float L = lane < n ? ml[2 * lane * step + 1] : 0.0f;
    float m = M;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    const float w = exp2f(M - m);
    float sum = L * w;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);

    const int g = lane / LPR, d = lane % LPR * 4;
    const float* o = p.part_o + (s0 * step + row) * D + d;
    f4_t a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int k0 = 0; k0 < n; k0 += GR) {
        const int k = k0 + g;
        const float wk = __shfl(w, k);
        if (k < n) a += *reinterpret_cast<const f4_t*>(o + k * step * D) * wk;
    }
#pragma unroll
    for (int off = LPR; off < 64; off <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] += __shfl_xor(a[e], off);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    if (g == 0) store4(static_cast<T*>(p.out) + row * D + d, a, inv);
    if (p.lse && lane == 0) p.lse[row] = log_sum(m, sum);
}

// The same with a workgroup to each: its 4 to 16 groups of D / 4 lanes take a split
// each in turn and meet in LDS.  The weights are formed once, one split to a thread.
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
    int s0;
    const int n = splits_of(p, s, i, h, s0);
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
    if (p.lse && tid == 0) p.lse[row] = log_sum(m, sum);
}

template <int D, int NG, bool F32, int GRP, int NR, int KW>
hipError_t launch_rows(const AttnParams& p, const Plan& c, hipStream_t s)
{
    const dim3 grid((unsigned)(p.v.kv_heads * c.splits * c.row_tiles), (unsigned)p.v.batch);
    // as many register sets as the registers hold without spilling
    constexpr bool big = D == 256 || (NR == 2 && F32) || (D == 128 && NG == 4 && (F32 || GRP == 1));
    constexpr int PF = KW == 8 ? 4 - 2 * (D == 128 && F32) : big ? 1 : D == 128 && (F32 || NR == 2) ? 2 : 3;
    kv4_attention_kernel<D, NG, F32, GRP, NR, KW, PF><<<grid, dim3(KW * 64), 0, s>>>(p);
    return hipGetLastError();
}

template <int D, int NG, bool F32, int KW>
hipError_t launch_group(const AttnParams& p, const Plan& c, hipStream_t s)
{
    switch (c.group) {
    case 4: return launch_rows<D, NG, F32, 4, 1, KW>(p, c, s);
    case 2: return launch_rows<D, NG, F32, 2, 1, KW>(p, c, s);
    default: return launch_rows<D, NG, F32, 1, 1, KW>(p, c, s);
    }
}

template <int D, int NG, bool F32>
hipError_t launch_few(const AttnParams& p, const Plan& c, hipStream_t s)
{
    if constexpr (D < 256 && NG <= 2) {
        if (c.group == 0) return launch_rows<D, NG, F32, 1, 2, 4>(p, c, s);
        if (c.kind == 0) return launch_group<D, NG, F32, 8>(p, c, s);
    }
    return launch_group<D, NG, F32, 4>(p, c, s);
}

template <int D, int NG> hipError_t launch_type(const AttnParams& p, const Plan& c, int f16, hipStream_t s)
{
    return f16 ? launch_few<D, NG, false>(p, c, s) : launch_few<D, NG, true>(p, c, s);
}

hipError_t launch_few_rows(const AttnParams& p, const Plan& c, int f16, hipStream_t s)
{
    const int ng = p.v.groups;
    switch (p.v.head_dim) {
    case 64: return ng == 1 ? launch_type<64, 1>(p, c, f16, s) : launch_type<64, 2>(p, c, f16, s);
    case 128:
        return ng == 1 ? launch_type<128, 1>(p, c, f16, s)
                       : ng == 2 ? launch_type<128, 2>(p, c, f16, s) : launch_type<128, 4>(p, c, f16, s);
    default:
        return ng == 2 ? launch_type<256, 2>(p, c, f16, s)
                       : ng == 4 ? launch_type<256, 4>(p, c, f16, s) : launch_type<256, 8>(p, c, f16, s);
    }
}

template <int D> hipError_t launch_join_dim(const AttnParams& p, int f16, hipStream_t s)
{
    const unsigned rows = (unsigned)(p.max_q * p.v.q_heads), waves = kJoinThreads / 64;
    // A wave a row up to 16 splits: 1200 rows of 8 splits 52 us with its attention kernel
    // against 65, 9600 of 3 splits 89 against 102; past that the few rows there are leave
    // the chip idle (16 splits of 128 rows and 64 of 32: 22.1 against 27.9, 32 against 39).
    if (p.splits <= kWaveSplits) {
        const dim3 grid((rows + waves - 1) / waves, (unsigned)p.v.batch);
        if (f16) kv4_join_rows_kernel<D, false><<<grid, dim3(kJoinThreads), 0, s>>>(p);
        else kv4_join_rows_kernel<D, true><<<grid, dim3(kJoinThreads), 0, s>>>(p);
        return hipGetLastError();
    }
    const dim3 grid(rows, (unsigned)p.v.batch);
    if (f16) kv4_join_kernel<D, false><<<grid, dim3(kJoinThreads), 0, s>>>(p);
    else kv4_join_kernel<D, true><<<grid, dim3(kJoinThreads), 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_join(const AttnParams& p, int f16, hipStream_t s)
{
    switch (p.v.head_dim) {
    case 64: return launch_join_dim<64>(p, f16, s);
    case 128: return launch_join_dim<128>(p, f16, s);
    default: return launch_join_dim<256>(p, f16, s);
    }
}

}  // namespace kv4

size_t kv4_attention_workspace(const AttentionArgs& a)
{
    const kv4::Plan c = kv4::plan_of(a);
    if (c.splits == 1) return 0;
    return (size_t)c.splits * a.v.tokens * a.v.q_heads * (a.v.head_dim + 2) * 4;
}

hipError_t launch_kv4_attention(const AttentionArgs& a, hipStream_t stream, const char** variant)
{
    const kv4::Plan c = kv4::plan_of(a);
    kv4::AttnParams p;
    p.v = a.v;
    p.q = a.q;
    p.q_stride = a.q_stride;
    p.out = a.out;
    p.lse = a.lse;
    p.part_o = static_cast<float*>(a.workspace);
    p.part_ml = p.part_o ? p.part_o + (int64_t)c.splits * a.v.tokens * a.v.q_heads * a.v.head_dim : nullptr;
    p.scale_log2 = a.scale * kLog2E;
    p.causal = a.causal;
    p.window = kv4::window_of(a.window, a.max_kv);
    p.max_q = (int)a.max_q;
    p.max_kv = (int)a.max_kv;
    p.gqa = a.v.q_heads / a.v.kv_heads;
    p.splits = c.splits;
    p.chunk = c.chunk;
    p.row_tiles = c.row_tiles;
    p.rows_per_wg = c.rows;
    *variant = c.kind == 2 ? (c.splits > 1 ? "attention_kv4_prompt_split" : "attention_kv4_prompt")
                           : (c.splits > 1 ? "attention_kv4_split" : "attention_kv4");
    const hipError_t e = c.kind == 2 ? kv4::launch_prompt(p, c, a.f16, stream) : kv4::launch_few_rows(p, c, a.f16, stream);
    if (e != hipSuccess || c.splits == 1) return e;
    return kv4::launch_join(p, a.f16, stream);
}

}  // namespace mnb
