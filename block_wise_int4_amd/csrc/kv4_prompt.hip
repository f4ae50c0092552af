// kv4_prompt.hip -- attention over the paged 4-bit cache for many query rows
// per key head (prompts and long chunks): the mathematics and the operand
// layout of kv4_attention.hip, with the unpacked keys and values shared.
//
// A workgroup of RW waves holds RW x 16 NR rows; its waves unpack a stage of
// 8192 / D keys together, once, into fp16 fragments in LDS, and every wave reads
// all of them as its A operands.  (Unpacked by each wave for itself, the codes
// cost as many vector instructions as the softmax.)
//
// The next stages' codes are requested a stage ahead and unpacked into the other
// half of LDS, with one barrier for two stages.  With two waves a SIMD (the
// registers allow no more) the kernel is bound by the latencies inside a wave, so a wave takes up
// to 64 keys through its softmax at once: one look at the masks, one at the running
// reference, and long runs of independent products and exponentials.  LDS reads,
// products and vector work take about 155, 145 and 200 of 485 thousand cycles of a SIMD at
// the long case below: nearly their sum, which the two waves' opposite order and
// priorities bring down (from 233 us to 217 when they came in).
//
// Measured, head_dim 128, groups of 128, fp16: 2048 and 1100 new tokens of 32 heads by 8
// key heads 214 us (150 GFLOP: 700 TFLOP/s, where a large fp16 product
// of the library reaches 1139); 1000 tokens of 32 heads by 32 key
// heads 33 us, one round of workgroups that lasts as long as its longest key range.  Two more
// fp32 parts of q and p: 337 us for the first.  Head size 256 has one column tile a wave: 200
// us with groups of 128 for 1024 and 640 tokens of 16 heads by 4 after a prefix, 388 with groups of
// 32, whose zero points and scales are loaded late, 469 in fp32 (which holds 6 registers in memory
// until after the loop; head size 64 in groups of 32 holds two words of a stage there).
#include "kv4_attention.hpp"

namespace mnb {
namespace kv4 {

namespace {

template <int D, int NG, bool F32, int NR, int RW>
__global__ __launch_bounds__(RW * 64, 2) void kv4_prompt_kernel(AttnParams p)
{
    typedef typename std::conditional<F32, float, _Float16>::type T;
    constexpr bool SPLIT = F32;
    constexpr int NJ = D / 32, NT = D / 16, NQ = F32 ? 2 : 1, JG = NJ / NG;
    constexpr int kRows = RW * NR * 16;
    constexpr int SB = 256 / D > 0 ? 256 / D : 1;      // blocks of 32 keys in a stage: 8192 / D keys
    constexpr int QB = D / 64;                         // 1 KB quads of a block's keys (and of its values)
    constexpr int IT = 8 / RW;                         // quads a wave unpacks: 4 of keys, 4 of values in all
    static_assert(SB * QB == 4, "four quads of each a stage");

    // Stages in LDS: half of them in use, half being filled.  One barrier serves
    // EP stages.
    constexpr int EP = 2, NB = 2 * EP;
    __shared__ __align__(16) h8_t kf[NB][SB][2][NJ][64];    // key fragments: tile, 32-dim step, lane
    __shared__ __align__(16) h8_t vf[NB][SB][NT][64];       // value fragments: 16-dim tile, lane
    __shared__ __align__(16) float ks[NB][SB][NG][32];      // scale * key scale, in log2 units
    __shared__ __align__(16) float vs[NB][SB][NG][32];
    __shared__ float vtop[NB][SB];                          // a block's largest value scale, as its exponent

    const KvView& v = p.v;
    const int lane = threadIdx.x & 63;
    const int wave = uniform(threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int h = blockIdx.x % v.kv_heads;
    const int split = (blockIdx.x / v.kv_heads) % p.splits;
    const int tile = p.row_tiles - 1 - (int)(blockIdx.x / v.kv_heads / p.splits);   // longest key ranges first
    const int b = blockIdx.y;

    const Sequence s = sequence_of(v, b, p.max_q, p.max_kv);
    const int rows = s.count * p.gqa;
    const int row0 = tile * kRows;
    if (row0 >= rows) return;                          // the whole workgroup
    const int last_row = row0 + kRows <= rows ? row0 + kRows - 1 : rows - 1;
    int lo, hi;
    key_range(p.causal, p.window, s, row0 / p.gqa, last_row / p.gqa, lo, hi);
    const int c0 = split * p.chunk, c1 = c0 + p.chunk;
    const int from = lo > c0 ? lo : c0, to = hi < c1 ? hi : c1;
    const bool any = from < to;
    if (p.splits > 1 && !any) return;                  // the join reads only splits with keys
    const int blk0 = from >> 5, blk1 = any ? (to + 31) >> 5 : blk0;
    const int stages = (blk1 - blk0 + SB - 1) / SB;

    const int nblk = 1 << (v.page_shift - 5);
    const int64_t block_bytes = kv_block_bytes(D, NG);
    const int32_t* table = v.table + (int64_t)b * v.table_stride;
    int pages = pages_from(v, table, blk0, 1, lane);   // of blocks page0 ..
    int page0 = blk0;

    // the rows of this wave
    const int wrow0 = row0 + wave * NR * 16;
    const bool busy = wrow0 < rows;                    // a wave past the rows only unpacks
    h8_t qf[NR][NQ][NJ];
    float qs[NR];
    int pos[NR];
    int64_t out_row[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        int r = wrow0 + n * 16 + col;
        const bool live = r < rows;
        r = live ? r : rows - 1;
        const int token = r / p.gqa, head = h * p.gqa + r % p.gqa;
        out_row[n] = live ? (int64_t)(s.first + token) * v.q_heads + head : -1;
        pos[n] = p.causal ? s.before + token : s.len - 1;
        qs[n] = load_query<NJ>(static_cast<const T*>(p.q) + (int64_t)(s.first + token) * p.q_stride + (int64_t)head * D +
                                   8 * quarter, qf[n]);
    }
    // every row of the wave sees the whole of a block below `whole`, from `open`
    // on, and none of a block from `none` on
    int whole = s.len, open = 0, none = s.len;
    if (p.causal) {
        const int wlast = wrow0 + NR * 16 <= rows ? wrow0 + NR * 16 - 1 : rows - 1;
        whole = s.before + wrow0 / p.gqa + 1;
        none = s.before + wlast / p.gqa + 1;
        if (p.window > 0) open = s.before + wlast / p.gqa - p.window + 1;
    }
    whole = whole < to ? whole : to;           // past the split's end LDS holds zeros

    f4_t o[NR][NT];
    float M[NR], l[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        M[n] = kLow;
        l[n] = 0.0f;
#pragma unroll
        for (int t = 0; t < NT; ++t) o[n][t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // ---- a stage's codes: requested, then unpacked into LDS ----
    // Item it of a wave: quad Q = wave + it RW; Q < 4 keys, else values.  A key quad
    // needs the zero points of the lane's own keys (both tiles where the quad spans
    // them), a value quad those of the lane's 8 keys.
    constexpr int kTilesOfQuad = D == 64 ? 2 : 1;      // key tiles in a quad
    u4_t code[IT];
    uint32_t zw[IT][8 * NG];
    constexpr bool LATE = NG >= 8;                     // too many words to hold for a stage: loaded at the unpack
    __amdgpu_buffer_rsrc_t rs[IT];

    // Zero points and scales that item it needs.
    auto words_of = [&](int it, bool is_v, int qi) {
        const int meta = 32 * D + (is_v ? 128 * NG : 0);
        if (is_v) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < NG; ++i) {
                    const u4_t r = __builtin_amdgcn_raw_buffer_load_b128(rs[it], 16 * NG * quarter + 16 * i, meta + t * 64 * NG, 0);
                    zw[it][t * 4 * NG + 4 * i] = r.x;
                    zw[it][t * 4 * NG + 4 * i + 1] = r.y;
                    zw[it][t * 4 * NG + 4 * i + 2] = r.z;
                    zw[it][t * 4 * NG + 4 * i + 3] = r.w;
                }
        } else {
#pragma unroll
            for (int t = 0; t < kTilesOfQuad; ++t) {
                const int tt = D == 64 ? t : qi * 4 / NJ;      // key tile
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    zw[it][t * NG + g] = __builtin_amdgcn_raw_buffer_load_b32(rs[it], (col * NG + g) * 4, meta + tt * 64 * NG, 0);
            }
        }
    };
    auto request = [&](int st) {
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int Q = wave + it * RW;
            const bool is_v = Q >= 4;
            const int qq = Q & 3, bi = qq / QB, qi = qq % QB;
            const int blk = blk0 + st * SB + bi;
            const bool there = blk < blk1;
            int at = blk - page0;
            at = at < 0 ? 0 : at > 63 ? 63 : at;
            unsigned char* base = v.cache + (((int64_t)page_in(v, pages, at) * v.kv_heads + h) * nblk + (blk & (nblk - 1))) * block_bytes;
            rs[it] = __builtin_amdgcn_make_buffer_rsrc(base, 0, there ? 32 * D + 256 * NG : 0, 0x00020000);
            code[it] = __builtin_amdgcn_raw_buffer_load_b128(rs[it], lane * 16, (is_v ? 16 * D : 0) + qi * 1024, 0);
            if constexpr (!LATE) words_of(it, is_v, qi);
        }
    };
    auto unpack = [&](int buf) {
        const h2_t sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
#pragma unroll
        for (int it = 0; it < IT; ++it) {
            const int Q = wave + it * RW;
            const int qq = Q & 3, bi = qq / QB, qi = qq % QB;
            if constexpr (LATE) words_of(it, Q >= 4, qi);
            if (Q < 4) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int W = qi * 4 + w, t = W / NJ, j = W % NJ;
                    uint32_t m;                // zero point of the lane's key in tile t, group of step j
                    if constexpr (D == 64) {
                        m = zw[it][(w / 2) * NG + (w % 2) / JG];
                    } else {
                        m = zw[it][0];
#pragma unroll
                        for (int g = 1; g < NG; ++g) m = j / JG == g ? zw[it][g] : m;
                    }
                    h2_t a4[4];
                    unpack_zr(code[it][w], zp_pair((m >> 16) & 15u), a4);
                    kf[buf][bi][t][j][lane] = join(a4);
                }
            } else {
#pragma unroll
                for (int uu = 0; uu < 2; ++uu) {
                    const int u = 2 * qi + uu, g = u / JG;
                    h2_t lo4[4], hi4[4];
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const uint32_t d = code[it][2 * uu + w], d8 = d >> 8;
                        const uint32_t ml = 0x000F000Fu, mh = 0x00F000F0u, magic = 0x64006400u;
                        uint32_t z[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            uint32_t m0 = zw[it][(4 * w + 2 * k) * NG], m1 = zw[it][(4 * w + 2 * k + 1) * NG];
#pragma unroll
                            for (int e = 1; e < NG; ++e) {
                                m0 = g == e ? zw[it][(4 * w + 2 * k) * NG + e] : m0;
                                m1 = g == e ? zw[it][(4 * w + 2 * k + 1) * NG + e] : m1;
                            }
                            z[k] = __builtin_amdgcn_perm(m1, m0, 0x07060302u);
                        }
                        auto zl = [&](uint32_t z2) { return as_h2(__builtin_amdgcn_bitop3_b32(z2, ml, 0xE400E400u, 0xEA)); };
                        auto zh = [&](uint32_t z2) { return as_h2(__builtin_amdgcn_bitop3_b32(z2 << 4, mh, 0xD400D400u, 0xEA)); };
                        lo4[2 * w] = as_h2(__builtin_amdgcn_bitop3_b32(d, ml, magic, 0xEA)) + zl(z[0]);
                        lo4[2 * w + 1] = as_h2(__builtin_amdgcn_bitop3_b32(d8, ml, magic, 0xEA)) + zl(z[1]);
                        hi4[2 * w] = as_h2(__builtin_amdgcn_bitop3_b32(d, mh, magic, 0xEA)) * sixteenth + zh(z[0]);
                        hi4[2 * w + 1] = as_h2(__builtin_amdgcn_bitop3_b32(d8, mh, magic, 0xEA)) * sixteenth + zh(z[1]);
                    }
                    vf[buf][bi][2 * u][lane] = join(lo4);
                    vf[buf][bi][2 * u + 1][lane] = join(hi4);
                }
            }
            // the scales: a key quad's lanes of quarter 0 hold their tile's own keys,
            // a value quad's first column all 32 keys; the first quad of a block that
            // has a tile writes it
            if (Q < 4) {
                if (quarter == 0) {
#pragma unroll
                    for (int t = 0; t < kTilesOfQuad; ++t) {
                        const int tt = D == 64 ? t : qi * 4 / NJ;
                        if (D == 64 || qi * 4 % NJ == 0) {
#pragma unroll
                            for (int g = 0; g < NG; ++g)
                                ks[buf][bi][g][tt * 16 + col] = scale_of(zw[it][t * NG + g]) * p.scale_log2;
                        }
                    }
                }
            } else if (qi == 0) {
                uint32_t most = zw[it][0];
#pragma unroll
                for (int k = 1; k < 8 * NG; ++k) most = max_halves(most, zw[it][k]);
                most = max_halves(most, (uint32_t)__shfl_xor((int)most, 16));
                most = max_halves(most, (uint32_t)__shfl_xor((int)most, 32));
                if (lane == 0) vtop[buf][bi] = top_exponent(most);
                if (col == 0) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
#pragma unroll
                        for (int g = 0; g < NG; ++g)
                            vs[buf][bi][g][(k >> 2) * 16 + 4 * quarter + (k & 3)] = scale_of(zw[it][k * NG + g]);
                }
            }
        }
    };

    // KB blocks from b0 of a stage; the first is block blk of the sequence.
    constexpr int KB = SB < 2 || NG >= 4 || (F32 && NG > 1) ? 1 : 2;   // two where the registers hold them (249 us with one, 233 with two)
    auto compute = [&](int buf, int b0, int blk) {
        // ---- logits less M, 32 KB keys by 16 NR rows ----
        float y[NR][8 * KB], Mu[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) Mu[n] = M[n] == kLow ? 0.0f : M[n];
#pragma unroll
        for (int t = 0; t < 2 * KB; ++t) {
            const int bi = b0 + t / 2;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                f4_t acc[NR];
#pragma unroll
                for (int n = 0; n < NR; ++n) acc[n] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int jj = 0; jj < JG; ++jj) {
                    const int j = g * JG + jj;
                    const h8_t k8 = kf[buf][bi][t % 2][j][lane];
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int c = 0; c < NQ; ++c) acc[n] = mfma(k8, qf[n][c][j], acc[n]);
                }
                const f4_t k4 = *reinterpret_cast<const f4_t*>(&ks[buf][bi][g][t % 2 * 16 + 4 * quarter]);
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float& e = y[n][4 * t + i];
                        // fp32 queries come back to their scale last, with M
                        const float add = g == 0 ? (F32 ? 0.0f : -Mu[n]) : e;
                        e = __builtin_fmaf(acc[n][i], k4[i], add);
                        if (F32 && g == NG - 1) e = __builtin_fmaf(e, qs[n], -Mu[n]);
                    }
            }
        }
        // ---- masks: a hidden key's logit is -infinity ----
        const bool edge = (blk + KB) * 32 > whole || blk * 32 < open;
        uint32_t seen[NR];                     // bit 4 t + i: the row sees the key
        if (edge) {
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                const int below = p.causal && p.window > 0 ? pos[n] - p.window : -1;
                seen[n] = 0;
#pragma unroll
                for (int k = 0; k < 8 * KB; ++k) {
                    const int key = blk * 32 + (k >> 2) * 16 + 4 * quarter + (k & 3);
                    const bool ok = key <= pos[n] && key > below && key < to;
                    seen[n] |= ok ? 1u << k : 0u;
                    y[n][k] = ok ? y[n][k] : -__builtin_inff();
                }
            }
        }
        // ---- the running reference, of 16 rows at a time ----
        float top[KB];
#pragma unroll
        for (int k = 0; k < KB; ++k) top[k] = vtop[buf][b0 + k];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            float mx = -__builtin_inff();
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                float m = y[n][8 * kb];
#pragma unroll
                for (int k = 1; k < 8; ++k) m = fmaxf(m, y[n][8 * kb + k]);
                mx = fmaxf(mx, m + top[kb]);
            }
            const bool first = M[n] == kLow;
            if (__builtin_amdgcn_ballot_w64(mx > (first ? -__builtin_inff() : kRaise))) {
                // key by key: a logit plus the exponent of its own scale, so that the largest
                // product of a row sets its reference
                mx = -__builtin_inff();
                int own = 4 * quarter;         // opaque: else the scales read here stay in registers until the
                asm volatile("" : "+v"(own));  // products (37 spilled at head_dim 256, groups of 64, fp32)
#pragma unroll
                for (int t = 0; t < 2 * KB; ++t) {
                    u4_t most = {0, 0, 0, 0};  // fp32 scales: their exponents with a bias of 126
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const f4_t v4 = *reinterpret_cast<const f4_t*>(&vs[buf][b0 + t / 2][g][t % 2 * 16 + own]);
                        most = __builtin_elementwise_max(most, __builtin_bit_cast(u4_t, v4));
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mx = fmaxf(mx, y[n][4 * t + i] + __builtin_amdgcn_fmed3f((float)(most[i] >> 23), 112.0f, 143.0f));
                }
                mx = of_quarters(mx) - 126.0f;                     // as top_exponent
                // a row moves by its own visible keys alone: neither the rows beside it nor hidden
                // keys, whose scales are in top, decide a bit of it
                const bool up = mx > (first ? -__builtin_inff() : kRaise);
                if (!__builtin_amdgcn_ballot_w64(up)) continue;
                const float next = up ? Mu[n] + mx - kBelow : Mu[n];
                const float alpha = first ? 1.0f : exp2f(Mu[n] - next);   // nothing was summed before the first
                const float by = next - Mu[n];
                M[n] = up ? next : M[n];
                l[n] *= alpha;
#pragma unroll
                for (int t = 0; t < NT; ++t) o[n][t] *= alpha;
#pragma unroll
                for (int k = 0; k < 8 * KB; ++k) y[n][k] -= by;
            }
        }
        // ---- p ----
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int k = 0; k < 8 * KB; ++k) {
                y[n][k] = __builtin_amdgcn_exp2f(y[n][k]);
                l[n] += y[n][k];
            }
        // ---- O^T += V^T (p s')^T, block by block and group by group ----
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                h8_t pb[NR], pl[NR];
                float f[NR][8];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const f4_t v4 = *reinterpret_cast<const f4_t*>(&vs[buf][b0 + kb][g][t * 16 + 4 * quarter]);
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[n][4 * t + i] = y[n][8 * kb + 4 * t + i] * v4[i];
                }
                if (edge) {                    // a hidden key adds nothing whatever its scale is
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int k = 0; k < 8; ++k) f[n][k] = (seen[n] >> (8 * kb + k)) & 1u ? f[n][k] : 0.0f;
                }
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        pb[n][k] = (_Float16)f[n][k];
                        if constexpr (SPLIT) pl[n][k] = (_Float16)(f[n][k] - (float)pb[n][k]);
                    }
#pragma unroll
                for (int tt = 0; tt < 2 * JG; ++tt) {
                    const int t = 2 * JG * g + tt;
                    const h8_t v8 = vf[buf][b0 + kb][t][lane];
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        o[n][t] = mfma(v8, pb[n], o[n][t]);
                        if constexpr (SPLIT) o[n][t] = mfma(v8, pl[n], o[n][t]);
                    }
                }
            }
        }
    };

    auto ask = [&](int st) {
        // pages of the blocks to request: refilled before they leave the register
        if (blk0 + (st + 1) * SB > page0 + 64) {
            page0 = blk0 + st * SB;
            pages = pages_from(v, table, page0, 1, lane);
        }
        request(st);
    };
    // A SIMD's two waves are w and w + RW / 2: one unpacks before its products, the other
    // after them and goes first where both can issue, so that one's products run beside
    // the other's softmax.
    const bool first_half = wave < RW / 2;
    if (!first_half) __builtin_amdgcn_s_setprio(1);
    if (stages > 0) {
        request(0);
#pragma unroll
        for (int i = 0; i < EP; ++i) {
            unpack(i);                         // past the end: the last codes again, unused
            if (i + 1 < stages) ask(i + 1);
        }
        __syncthreads();
        for (int st = 0; st < stages; ++st) {
            const int buf = st & (NB - 1);
            const bool more = st + EP < stages, further = st + EP + 1 < stages;
            if (first_half && more) unpack((st + EP) & (NB - 1));
            if (first_half && further) ask(st + EP + 1);
#pragma unroll
            for (int b0 = 0; b0 < SB; b0 += KB) {
                const int blk = blk0 + st * SB + b0;
                // blocks past the end hold zeros and are masked
                if (busy && blk < blk1 && blk * 32 < none) compute(buf, b0, blk);
            }
            if (!first_half && more) unpack((st + EP) & (NB - 1));
            if (!first_half && further) ask(st + EP + 1);
            if ((st & (EP - 1)) == EP - 1) __syncthreads();
        }
    }

#pragma unroll
    for (int n = 0; n < NR; ++n) {
        l[n] += __shfl_xor(l[n], 16);
        l[n] += __shfl_xor(l[n], 32);
        if (out_row[n] < 0) continue;
        if (p.splits == 1) {
            const float inv = l[n] == 0.0f ? 0.0f : 1.0f / l[n];   // a row that sees nothing gives zeros
            T* out = static_cast<T*>(p.out) + out_row[n] * D + 4 * quarter;
#pragma unroll
            for (int t = 0; t < NT; ++t) store4(out + 16 * t, o[n][t], inv);
            if (p.lse && quarter == 0) p.lse[out_row[n]] = log_sum(M[n], l[n]);
        } else {
            const int64_t at = (int64_t)split * v.tokens * v.q_heads + out_row[n];
            float* part = p.part_o + at * D + 4 * quarter;
#pragma unroll
            for (int t = 0; t < NT; ++t) *reinterpret_cast<f4_t*>(part + 16 * t) = o[n][t];
            if (quarter == 0) {
                p.part_ml[2 * at] = M[n];
                p.part_ml[2 * at + 1] = l[n];
            }
        }
    }
}

template <int D, int NG, bool F32> hipError_t launch_tiles(const AttnParams& p, const Plan& c, hipStream_t s)
{
    const dim3 grid((unsigned)(p.v.kv_heads * c.splits * c.row_tiles), (unsigned)p.v.batch);
    if constexpr (D < 256 && NG <= 2) {
        if (c.tiles == 2) {
            kv4_prompt_kernel<D, NG, F32, 2, kPromptWaves><<<grid, dim3(kPromptWaves * 64), 0, s>>>(p);
            return hipGetLastError();
        }
    }
    kv4_prompt_kernel<D, NG, F32, 1, kPromptWaves><<<grid, dim3(kPromptWaves * 64), 0, s>>>(p);
    return hipGetLastError();
}

template <int D, int NG> hipError_t launch_type(const AttnParams& p, const Plan& c, int f16, hipStream_t s)
{
    return f16 ? launch_tiles<D, NG, false>(p, c, s) : launch_tiles<D, NG, true>(p, c, s);
}

}  // namespace

hipError_t launch_prompt(const AttnParams& p, const Plan& c, int f16, hipStream_t s)
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

}  // namespace kv4
}  // namespace mnb
