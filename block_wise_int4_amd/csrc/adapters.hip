// adapters.hip -- low-rank adapters of many requests beside one projection:
//
//   y[t] = base[t] + s_a B_a (A_a x[t]),   a = adapter[t],
//
// A_a [rank, k], B_a [n, rank]; rows of a call may have any adapters in any
// order.  Two products, h = A x in fp32, then y = base + s B h, in two launches, or in one for few
// rows (every workgroup then forms the h of its adapters by itself).
//
// What bounds it: x, base and y read and written once, for few rows A and B of the adapters that
// occur; the products are small (rank 32: 32 operations a byte).  So both kernels are built
// around their loads.
//
// Rows are gathered by adapter inside a tile of 16, 32 or 64 (a lane a row: a ballot names the rows of an
// adapter, a move between lanes lists them), so the matrix cores see 16 rows of one adapter where
// the tile has them, in whatever order they came, and nothing is sorted beforehand.  The adapters of a
// tile are shared out to `slots` workgroups; a slot takes every slots-th of the tile's adapters.
//
// First product: the waves share k.  A load takes 128 neighbouring bytes of 8 rows and the
// operands of v_mfma_f32_16x16x32_f16 form in the wave's own LDS (loaded as operands, each of a load's
// lanes goes to another row, at 16 bytes a cycle and CU: 8416 rows, k = 4096, rank 32 18 us, 60 so).
// Second product: h is prepared once a workgroup, as operands in LDS: in fp16 calls as two fp16 parts of the row
// scaled by a power of two, 22 bits, so that h is not rounded to 16 bits (at rank 16 and below one product takes both
// parts; both have h's sign, so that an infinite B meets no difference of infinities); in fp32 calls as it is, for v_mfma_f32_16x16x4f32.  The result turns through
// LDS so that base is read and y is written 128 bytes or more of a row at a time.
//
// Measured, call by call.  k = n = 4096, rank 16, fp16: one token 7.1 us, 32 tokens of 24 adapters 8.1 (6.2
// MB asked for), both one launch and the time of its chain: adapter, rank, A and x, two meetings in LDS,
// base and y (fp32, two launches: 8.8 and 10.9).  8416 rows, k = 4096, n = 11008, rank 32: 89 us for 443 MB, 5.0 TB/s
// where a large copy moves 5.1; the first kernel a fifth of it (69 MB).  4000 rows, k = n = 4096: rank 16 25.6 us,
// 32 27.5, 64 39.6, 128 52.3 (floor 20), of which the first kernel takes 9, 10, 13 and 21: every 32 rows
// read all of A, above rank 64 x is read twice, and every 512 columns read h and part it anew.  In
// fp32 rank 64 takes 77 us (floor 39), 30 + 48: its products run at a sixteenth of the fp16 rate, two waves a SIMD.
// No instance keeps a vector register in memory.
#include <type_traits>

#include "adapters_plan.hpp"
#include "mnb_device.hpp"
#include "mnb_requests.hpp"
#include "mnb_vec.hpp"

namespace mnb {
namespace adapters {

namespace {

struct Params {
    const void* a;
    const void* b;
    const float* scales;
    const int32_t* ranks;
    const int32_t* adapter;
    const void* x;
    const void* base;
    void* y;
    float* h;                         // [splits][m][pitch]
    int64_t m, n, k, x_stride, base_stride, y_stride, k_per;
    int rank, count, splits, slots, pitch, rblocks, nblocks, blocks, tile;
};

__device__ __forceinline__ f4_t mfma16(const h8_t& a, const h8_t& b, const f4_t& c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// One 16-byte piece of both operands into a 16 x 16 product.  The sum's order is
// free, so the quarters of a wave take neighbouring pieces of a row.
__device__ __forceinline__ f4_t product(const h8_t& a, const h8_t& b, const f4_t& c) { return mfma16(a, b, c); }
__device__ __forceinline__ f4_t product(const f4_t& a, const f4_t& b, f4_t c)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
}

// The rows of a tile of up to 64, a lane each: adapter (-1: none, out of range or of rank 0) and its rank.
struct Rows {
    int adapter, rank;
    bool there;
};
__device__ __forceinline__ Rows rows_of(const Params& p, int64_t row0, int lane)
{
    const int64_t row = row0 + lane;
    Rows r = {-1, p.rank, lane < p.tile && row < p.m};
    if (r.there) {
        const int a = p.adapter[row];
        if (a >= 0 && a < p.count) {
            if (p.ranks) r.rank = p.ranks[a] < p.rank ? p.ranks[a] : p.rank;
            r.adapter = r.rank > 0 ? a : -1;
        }
    }
    return r;
}

// The slot of a workgroup, and which of the slot's it is.  Slots that may find no adapter come
// last: the first ones' work spreads over all XCDs, whatever the number of slots is a multiple of.
struct Place {
    int slot;
    uint32_t rest;
};
__device__ __forceinline__ Place place_of(const Params& p)
{
    const uint32_t per = gridDim.x / p.slots;
    return Place{(int)(blockIdx.x / per), blockIdx.x % per};
}

// The same with all of a slot's workgroups on one XCD, since each reads all of the slot's A (32 rows of
// 24 adapters: 8.0 us, 10.4 with them spread).  Fewer slots than XCDs are spread.
__device__ __forceinline__ Place place_near(const Params& p)
{
    if (p.slots < 8) return place_of(p);
    const uint32_t per = gridDim.x / ((p.slots + 7) / 8 * 8), on = blockIdx.x / 8;
    return Place{(int)(on / per * 8 + blockIdx.x % 8), on % per};
}

// Lane n of the result holds the n-th row of a set of rows (the others behind them).
__device__ __forceinline__ int gathered(uint64_t set, int lane)
{
    const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(set >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)set, 0));
    const int to = (set >> lane & 1) ? before : __builtin_popcountll(set) + lane - before;
    return __builtin_amdgcn_ds_permute(4 * to, lane);
}

// Calls f(adapter, rank, rows) for the adapters of a tile that are the slot's.
template <typename F> __device__ __forceinline__ void for_adapters(const Rows& r, int slot, int slots, F f)
{
    uint64_t todo = __builtin_amdgcn_ballot_w64(r.adapter >= 0);
    int skip = slot;
    while (todo) {
        const int at = __builtin_ctzll(todo);
        const int ad = __builtin_amdgcn_readlane(r.adapter, at);
        const uint64_t same = __builtin_amdgcn_ballot_w64(r.adapter == ad);
        todo &= ~same;
        if (skip > 0) {
            --skip;
            continue;
        }
        skip = slots - 1;
        f(ad, __builtin_amdgcn_readlane(r.rank, at), same);
    }
}

// A step's 128 bytes of a row, in the wave's LDS: piece i of row r lies at i ^ (r % 8), so that
// neither the rows' pieces, as they arrive, nor the operands' columns meet in a bank.
__device__ __forceinline__ int in_row(int row, int piece) { return row * 8 + (piece ^ (row & 7)); }

// Ranks rank0 .. of h = A x for up to 16 CU rows of one adapter, the waves sharing k.
// Eight neighbouring lanes take 128 neighbouring bytes of a row, and the operands form in LDS: loaded
// as operands, each of a load's lanes would go to another row, and the cache looks up four times
// as often.  sink(n, r, sum) takes element r of the n-th row.
template <typename T, int CU, int RT, int KW, typename F>
__device__ __forceinline__ void down_rows(const Params& p, int ad, int rank0, int rank, int order, int rows, int64_t row0,
                                          int split, u4_t* lds, F sink)
{
    constexpr int E = Vec<T>::E, STEP = 8 * E;
    constexpr int R = 16 * (CU + RT), IT = R / 8;       // rows of x, then of A; loads of a step
    constexpr int S = 4 < CU * RT ? 4 : CU * RT;        // 16 x 16 tiles that meet at once
    typedef typename Vec<T>::type V;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int64_t k0 = split * p.k_per, k1 = k0 + p.k_per < p.k ? k0 + p.k_per : p.k;
    const int full = (int)((k1 - k0) / STEP);
    const int left = (int)((k1 - k0) % STEP);
    u4_t* mine = lds + wave * (R * 8);

    const T* from[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        int r = 8 * i + (lane >> 3);
        if (i < 2 * CU) {
            r = r < rows ? r : rows - 1;                // not written
            from[i] = static_cast<const T*>(p.x) + (row0 + __shfl(order, r)) * p.x_stride;
        } else {
            r -= 16 * CU;
            r = r < rank ? r : rank - 1;                // not written
            from[i] = static_cast<const T*>(p.a) + ((int64_t)ad * p.rank + rank0 + r) * p.k;
        }
        from[i] += k0 + (lane & 7) * E;
    }
    f4_t acc[CU][RT];
#pragma unroll
    for (int u = 0; u < CU; ++u)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[u][t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};

    V next[IT];
    auto request = [&](int s) {
        if (s < full) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                // one 16-row tile may hold few rows: the others' loads would cost as much
                if (CU > 1 || i >= 2 || 8 * i + (lane >> 3) < rows) next[i] = load(from[i] + (int64_t)s * STEP);
                else next[i] = V{};
            }
        } else {
#pragma unroll
            for (int i = 0; i < IT; ++i) next[i] = load_some(from[i] + (int64_t)s * STEP, left - (lane & 7) * E);
        }
    };
    const int steps = full + (left > 0 ? 1 : 0);
    if (wave < steps) request(wave);
    __syncthreads();                                    // LDS held the last adapter's sums
    for (int s = wave; s < steps; s += KW) {
#pragma unroll
        for (int i = 0; i < IT; ++i)
            mine[in_row(8 * i + (lane >> 3), lane & 7)] = __builtin_bit_cast(u4_t, next[i]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // a wave's LDS operations complete in order
        if (s + KW < steps) request(s + KW);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            V xv[CU], av[RT];
#pragma unroll
            for (int u = 0; u < CU; ++u) xv[u] = __builtin_bit_cast(V, mine[in_row(16 * u + col, 2 * quarter + e)]);
#pragma unroll
            for (int t = 0; t < RT; ++t) av[t] = __builtin_bit_cast(V, mine[in_row(16 * (CU + t) + col, 2 * quarter + e)]);
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int u = 0; u < CU; ++u) acc[u][t] = product(av[t], xv[u], acc[u][t]);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // before the next step's
    }
    // the waves' sums meet in LDS
    float(*red)[64][20] = reinterpret_cast<float(*)[64][20]>(lds);
#pragma unroll
    for (int i0 = 0; i0 < CU * RT; i0 += S) {
        if (i0 / CU * 16 >= rank) break;
        __syncthreads();                                // the operands, or the last sums, have been read
#pragma unroll
        for (int i = 0; i < S; ++i)
            *reinterpret_cast<f4_t*>(&red[wave][16 * i + col][4 * quarter]) = acc[(i0 + i) % CU][(i0 + i) / CU];
        __syncthreads();
#pragma unroll
        for (int part = 0; part < (4 * S + KW - 1) / KW; ++part) {
            const int at = (threadIdx.x >> 4) + 4 * KW * part, r0 = threadIdx.x & 15;
            const int i = i0 + at / 16, n = 16 * (i % CU) + at % 16, r = 16 * (i / CU) + r0;
            float sum = 0.0f;
            if (at < 16 * S) {
#pragma unroll
                for (int w = 0; w < KW; ++w) sum += red[w][at][r0];
            }
            sink(n, r, sum, at < 16 * S && n < rows && r < rank);
        }
    }
}

// h = A x for a tile of rows, 16 RT ranks and the adapters of one slot.
template <typename T, int RT> __global__ __launch_bounds__(kDownWaves * 64, RT <= 2 ? 3 : 2) void adapters_down_kernel(Params p)
{
    constexpr int KW = kDownWaves;
    __shared__ __align__(16) u4_t lds[KW * 16 * (4 + RT) * 8];
    static_assert(sizeof(lds) >= sizeof(float) * KW * 64 * 20, "the sums fit");
    const int lane = threadIdx.x & 63;
    const Place at = place_of(p);
    const int slot = at.slot, split = at.rest % p.splits, rank0 = at.rest / p.splits % p.rblocks * (16 * RT);
    const int64_t row0 = (int64_t)(at.rest / p.splits / p.rblocks) * p.tile;
    const Rows mine = rows_of(p, row0, lane);
    for_adapters(mine, slot, p.slots, [&](int ad, int rank, uint64_t same) {
        const int order = gathered(same, lane), rows = __builtin_popcountll(same);
        const int here = rank - rank0 < 16 * RT ? rank - rank0 : 16 * RT;
        if (here <= 0) return;
        float* h = p.h + ((int64_t)split * p.m + row0) * p.pitch + rank0;
        auto sink = [&](int n, int r, float sum, bool there) {
            const int row = __shfl(order, n & 63);
            if (there) h[row * p.pitch + r] = sum;
        };
        if (rows > 32) down_rows<T, 4, RT, KW>(p, ad, rank0, here, order, rows, row0, split, lds, sink);
        else if (rows > 16) down_rows<T, 2, RT, KW>(p, ad, rank0, here, order, rows, row0, split, lds, sink);
        else down_rows<T, 1, RT, KW>(p, ad, rank0, here, order, rows, row0, split, lds, sink);
    });
}

// The second product's operands.  RC: 32-rank chunks; 0: up to 16 ranks, both fp16 parts
// of h in one product.  Four ranks r0 .. of a row of h, summed over the splits, go into LDS
// as operands; PITCH / 4 neighbouring lanes hold a row.
template <typename T, int RC> struct Up;

template <int RC> struct Up<_Float16, RC> {
    static constexpr int PITCH = RC == 0 ? 16 : 32 * RC, NC = RC == 0 ? 1 : RC, PARTS = RC == 0 ? 1 : 2, NH = NC * PARTS;
    typedef h8_t piece;
    typedef _Float16 h4 __attribute__((ext_vector_type(4)));
    static __device__ __forceinline__ int rank0(int c, int quarter) { return RC == 0 ? 8 * (quarter & 1) : 32 * c + 8 * quarter; }
    // h as two fp16 parts, 22 bits, of the row scaled to below 2^16; the power of two taken out.  Both parts have h's
    // sign and are 0 only where h is, so that their products with an infinite B are of one sign: the first is cut
    // off below h, and neither is less than fp16's least number, 2^-39 of the row's largest (rounded to nearest
    // the second was 0 or of the other sign in half of all places, and the sum NaN).
    static __device__ __forceinline__ float put(const f4_t& v, int row, int r0, piece (*hf)[NH][64])
    {
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fabsf(v[i]) < __builtin_inff() ? fabsf(v[i]) : 0.0f);
#pragma unroll
        for (int off = 1; off < PITCH / 4; off <<= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
        int e = mx > 0.0f ? (int)(__builtin_bit_cast(uint32_t, mx) >> 23) - 127 - 15 : 0;
        e = e < -126 ? -126 : e;
        const float down = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
        typedef __fp16 rz2 __attribute__((ext_vector_type(2)));
        h4 hi, lo;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            float s[2], least[2];
            rz2 cut;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                s[k] = fabsf(v[i + k] * down);
                least[k] = v[i + k] != 0.0f ? 1.25f / (1 << 24) : 0.0f;    // rounds to 2^-24, also less an ulp
                s[k] = __builtin_elementwise_maximum(s[k], least[k]);      // NaN stays
            }
            const float below = 1.0f - 1.0f / (1 << 23);
            cut = __builtin_amdgcn_cvt_pkrtz(s[0] * below, s[1] * below);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                hi[i + k] = (_Float16)__builtin_copysignf((float)cut[k], v[i + k]);
                lo[i + k] = (_Float16)__builtin_copysignf(fmaxf(s[k] - (float)cut[k], least[k]), v[i + k]);
            }
        }
        const int u = row / 16, at = 16 * (r0 % 32 / 8) + row % 16, half = r0 / 4 & 1;
        if constexpr (RC == 0) {
            reinterpret_cast<h4*>(&hf[u][0][at])[half] = hi;
            reinterpret_cast<h4*>(&hf[u][0][at + 32])[half] = lo;
        } else {
            reinterpret_cast<h4*>(&hf[u][r0 / 32 * 2][at])[half] = hi;
            reinterpret_cast<h4*>(&hf[u][r0 / 32 * 2 + 1][at])[half] = lo;
        }
        return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
    }
};

template <int RC> struct Up<float, RC> {
    static constexpr int PITCH = RC == 0 ? 16 : 32 * RC, NC = PITCH / 16, PARTS = 1, NH = NC;   // 16-rank chunks
    typedef f4_t piece;
    static __device__ __forceinline__ int rank0(int c, int quarter) { return 16 * c + 4 * quarter; }
    static __device__ __forceinline__ float put(const f4_t& v, int row, int r0, piece (*hf)[NH][64])
    {
        hf[row / 16][r0 / 16][16 * (r0 % 16 / 4) + row % 16] = v;
        return 1.0f;
    }
};

// A lane's pieces of base in N 16-row tiles.
template <typename T, int NT> struct Base {
    static constexpr int N = NT;
    typename Vec<T>::type v[N][16 / Vec<T>::E];
    int row[N][16 / Vec<T>::E];
};

// A wave's 64 columns of y = base + s B h, for rows of a tile of 64.  The products leave a column
// of 16 rows to a quarter of the wave; through LDS they come back as whole pieces of a row, and base
// and y are read and written 128 (fp32: 256) neighbouring bytes at a time.
template <typename T, int RC> struct Columns {
    typedef Up<T, RC> O;
    typedef typename Vec<T>::type V;
    static constexpr int E = Vec<T>::E, LANES = 64 / E, STEP = 64 / LANES;   // lanes to a row's 64 columns, rows at a time
    static constexpr int PIECES = 16 / STEP;            // of a lane in a 16-row tile

    const Params& p;
    int64_t n0, left;
    int lane, c0, r0;                                   // column and row of the lane's first piece
    bool busy;                                          // a wave past the columns only prepares h
    const T* base;
    T* y;
    V b[O::NC][4];
    float scale;

    __device__ __forceinline__ Columns(const Params& q, int64_t row0, int64_t first, int of) : p(q), n0(first), lane(of)
    {
        c0 = lane % LANES * E;
        r0 = lane / LANES;
        left = p.n - n0 - c0;
        busy = n0 < p.n;
        base = p.base ? static_cast<const T*>(p.base) + row0 * p.base_stride + n0 + c0 : nullptr;
        y = static_cast<T*>(p.y) + row0 * p.y_stride + n0 + c0;
    }
    __device__ __forceinline__ void put(T* at, const V& v) const
    {
        if (left >= E) store_through(at, v);            // y is read by no one here (185 MB 107 us kept, 97 so)
        else
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e < left) at[e] = v[e];
    }
    // rows without an adapter
    __device__ __forceinline__ void copy(uint64_t none) const
    {
        if (!none || !busy || base == y) return;
        const int order = gathered(none, lane), rows = __builtin_popcountll(none);
        for (int n = r0; n < rows + r0; n += STEP) {
            const int row = __shfl(order, n & 63);
            if (n < rows) {
                V v = {};
                if (base) v = load_some(base + row * p.base_stride, left);
                put(y + row * p.y_stride, v);
            }
        }
    }
    __device__ __forceinline__ void load_b(int ad, int rank)
    {
        const int col = lane & 15, quarter = lane >> 4;
        const T* w = static_cast<const T*>(p.b) + (int64_t)ad * p.n * p.rank;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            int64_t n = n0 + 16 * j + col;
            n = n < p.n ? n : p.n - 1;                  // not written
#pragma unroll
            for (int c = 0; c < O::NC; ++c)
                b[c][j] = load_some(w + n * p.rank + O::rank0(c, quarter), rank - O::rank0(c, quarter));
        }
        scale = p.scales ? p.scales[ad] : 1.0f;
    }
    // base of N 16-row tiles from tile g on
    template <int N> __device__ __forceinline__ Base<T, N> request(int order, int rows, int g) const
    {
        Base<T, N> in;
        auto each = [&](auto from) {
#pragma unroll
            for (int u = 0; u < N; ++u)
#pragma unroll
                for (int i = 0; i < PIECES; ++i) {
                    const int n = 16 * (g + u) + i * STEP + r0;
                    in.row[u][i] = __shfl(order, n & 63);
                    in.v[u][i] = V{};
                    if (base && busy && n < rows) in.v[u][i] = from(base + in.row[u][i] * p.base_stride);
                }
        };
        // A base past half the last cache is not there from the projection before, and kept for no one
        // (185 MB 97.3 and 94.8 us; 16 MB 15.3 and 17.2)
        if (p.m * p.n * (int64_t)sizeof(T) >= (int64_t)128 << 20)
            each([&](const T* at) { return left >= E ? load_once(at) : load_some(at, left); });
        else each([&](const T* at) { return load_some(at, left); });
        return in;
    }
    template <int N>
    __device__ __forceinline__ void finish(const Base<T, N>& in, int rows, int g, const typename O::piece (*hf)[O::NH][64],
                                           const float* back, float (*turn)[68]) const
    {
        const int col = lane & 15, quarter = lane >> 4;
#pragma unroll
        for (int u = 0; u < N; ++u) {
            if (16 * (g + u) >= rows) break;
            f4_t acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < O::NH; ++c) {
                const typename O::piece h = hf[g + u][c][lane];
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] = product(b[c / O::PARTS][j], h, acc[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) *reinterpret_cast<f4_t*>(&turn[col][16 * j + 4 * quarter]) = acc[j];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const int at = i * STEP + r0, n = 16 * (g + u) + at;
                // h's power of two first: times the scale it may leave fp32's range, which times 0 or infinity is NaN
                const float up = sizeof(T) == 2 ? back[n] : 1.0f;
                V v;
#pragma unroll
                for (int q = 0; q < E / 4; ++q) {
                    const f4_t t = *reinterpret_cast<const f4_t*>(&turn[at][c0 + 4 * q]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[4 * q + e] = (T)__builtin_fmaf(t[e] * up, scale, (float)in.v[u][i][4 * q + e]);
                }
                if (n < rows) put(y + in.row[u][i] * p.y_stride, v);
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    }
};

// MORE: further blocks of 256 columns with the same h, for ranks whose h is long to read.
template <typename T, int RC, bool MORE>
__global__ __launch_bounds__(kUpWaves * 64, RC <= 1 ? 4 : 2) void adapters_up_kernel(Params p)
{
    typedef Up<T, RC> O;
    constexpr int TH = O::PITCH / 4;                    // lanes to a row of h
    constexpr int PRE = sizeof(T) == 4 ? (RC < 2 ? 2 : 1) : RC < 4 ? 4 : 2;   // 16-row tiles whose base is requested at once
    __shared__ __align__(16) typename O::piece hf[4][O::NH][64];    // h of four 16-row tiles, as operands
    __shared__ float back[64];
    __shared__ __align__(16) float turn[kUpWaves][16][68];

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const Place at = place_of(p);
    const int slot = at.slot;
    const int blocks = MORE ? p.blocks : 1;
    const int64_t n0 = ((int64_t)(at.rest % p.nblocks) * blocks * kUpWaves + wave) * 64;
    const int64_t row0 = (int64_t)(at.rest / p.nblocks) * p.tile;
    const Rows mine = rows_of(p, row0, lane);
    const uint64_t none = __builtin_amdgcn_ballot_w64(mine.adapter < 0 && mine.there);
    Columns<T, RC> w(p, row0, n0, lane);
    if (slot == 0) w.copy(none);
    if (MORE && slot == 0)
        for (int block = 1; block < blocks; ++block)
            Columns<T, RC>(p, row0, n0 + (int64_t)block * (64 * kUpWaves), lane).copy(none);
    for_adapters(mine, slot, p.slots, [&](int ad, int rank, uint64_t same) {
        const int order = gathered(same, lane), rows = __builtin_popcountll(same);
        // h: N times four ranks to a thread, some splits of each at once.  Where there is nothing to read the
        // first of h stands in, so that no load waits for a branch
        auto prepare = [&](auto count) {
            constexpr int N = decltype(count)::value, AT_ONCE = N >= 8 ? (sizeof(T) == 4 ? 1 : 2) : N >= 2 ? 4 : 8;
            const f4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
            f4_t v[N];
            const float* h[N];
            bool real[N];
            const int64_t step = p.m * p.pitch;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = threadIdx.x + i * kUpWaves * 64, n = at / TH, r = at % TH * 4;
                const int row = __shfl(order, n & 63);
                real[i] = n < rows && r < rank;
                h[i] = real[i] ? p.h + (row0 + row) * p.pitch + r : p.h;
                v[i] = zero;
            }
            int s = 0;
            for (; s + AT_ONCE <= p.splits; s += AT_ONCE) {
                f4_t q[AT_ONCE][N];
#pragma unroll
                for (int k = 0; k < AT_ONCE; ++k)
#pragma unroll
                    for (int i = 0; i < N; ++i) q[k][i] = *reinterpret_cast<const f4_t*>(h[i] + (s + k) * step);
#pragma unroll
                for (int k = 0; k < AT_ONCE; ++k)
#pragma unroll
                    for (int i = 0; i < N; ++i) v[i] += q[k][i];
            }
            for (; s < p.splits; ++s)
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] += *reinterpret_cast<const f4_t*>(h[i] + s * step);
            __syncthreads();                            // the last adapter's has been read
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int at = threadIdx.x + i * kUpWaves * 64, n = at / TH, r = at % TH * 4;
                if (n >= (rows + 15) / 16 * 16) break;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i][e] = real[i] && r + e < rank ? v[i][e] : 0.0f;
                const float f = O::put(v[i], n, r, hf);
                if (r == 0) back[n] = f;
            }
            __syncthreads();
        };
        auto columns = [&](Columns<T, RC>& w, bool first) {
            if (first || w.busy) w.load_b(ad, rank);
            if (rows <= 16) {
                // a few rows wait for their loads: base on its way beside h.  (More have no registers for it.)
                const auto in = w.template request<1>(order, rows, 0);
                if (first) prepare(std::integral_constant<int, TH < 16 ? 1 : TH / 16>());
                if (w.busy) w.finish(in, rows, 0, hf, back, turn[wave]);
            } else {
                if (first) prepare(std::integral_constant<int, TH / 4>());
                if (!w.busy) return;
#pragma unroll
                for (int g = 0; g < 4; g += PRE)
                    if (16 * g < rows) w.finish(w.template request<PRE>(order, rows, g), rows, g, hf, back, turn[wave]);
            }
        };
        // Where the registers are short the lanes' addresses are formed anew, from a lane's number that the compiler
        // cannot take for the last one, and not kept from block to block or beside h (rank 32, 8416 rows: 3 registers
        // in memory and 95.6 us with them kept, none and 91.3 so; rank 128, one token 10 and 11.4, none and 10.6, 64 rows
        // of 64 adapters 35.0 and 33.5.  Elsewhere none is in memory either way: 512 rows of 64 adapters of rank 64 75 and
        // 87, of rank 16 36.3 and 37.7)
        if constexpr (!MORE && RC != 1 && RC != 4) columns(w, true);
        else
            for (int block = 0; block < blocks; ++block) {
                int again = lane;
                asm volatile("" : "+v"(again));
                Columns<T, RC> next(p, row0, n0 + (int64_t)block * (64 * kUpWaves), again);
                columns(next, block == 0);
            }
    });
}

// Both products in one launch, for few rows: every workgroup forms the h of its slot's
// adapters, of a tile of 32 rows, by itself.
template <typename T, int RC> __global__ __launch_bounds__(kOneWaves * 64, 2) void adapters_one_kernel(Params p)
{
    typedef Up<T, RC> O;
    constexpr int RT = O::PITCH / 16, TH = O::PITCH / 4, KW = kOneWaves;
    __shared__ __align__(16) u4_t lds[KW * 16 * (2 + RT) * 8];
    static_assert(sizeof(lds) >= sizeof(float) * KW * 16 * 20 * (RT == 1 ? 2 : 4), "the sums fit");
    __shared__ __align__(16) float hs[32][O::PITCH];
    __shared__ __align__(16) typename O::piece hf[2][O::NH][64];
    __shared__ float back[32];
    float(*turn)[16][68] = reinterpret_cast<float(*)[16][68]>(lds);
    static_assert(sizeof(lds) >= sizeof(float) * KW * 16 * 68, "a tile of every wave fits");

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const Place at = place_near(p);
    const int slot = at.slot;
    if (slot >= p.slots) return;
    const int64_t n0 = ((int64_t)(at.rest % p.nblocks) * KW + wave) * 64;
    const int64_t row0 = (int64_t)(at.rest / p.nblocks) * p.tile;   // at most 32
    const Rows mine = rows_of(p, row0, lane);
    Columns<T, RC> w(p, row0, n0, lane);
    const uint64_t none = __builtin_amdgcn_ballot_w64(mine.adapter < 0 && mine.there);
    if (slot == 0) w.copy(none);
    for_adapters(mine, slot, p.slots, [&](int ad, int rank, uint64_t same) {
        const int order = gathered(same, lane), rows = __builtin_popcountll(same);
        w.load_b(ad, rank);
        const auto in = w.template request<1>(order, rows, 0);
        auto sink = [&](int n, int r, float sum, bool real) {
            if (real) hs[n][r] = sum;
        };
        if (rows > 16) down_rows<T, 2, RT, KW>(p, ad, 0, rank, order, rows, row0, 0, lds, sink);
        else down_rows<T, 1, RT, KW>(p, ad, 0, rank, order, rows, row0, 0, lds, sink);
        __syncthreads();
        for (int at = threadIdx.x; at < (rows + 15) / 16 * 16 * TH; at += KW * 64) {
            const int n = at / TH, r = at % TH * 4;
            f4_t v = *reinterpret_cast<const f4_t*>(&hs[n][r]);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = n < rows && r + i < rank ? v[i] : 0.0f;
            const float f = O::put(v, n, r, hf);
            if (r == 0) back[n] = f;
        }
        __syncthreads();
        if (w.busy) {
            w.finish(in, rows, 0, hf, back, turn[wave]);
            if (rows > 16) w.finish(w.template request<1>(order, rows, 1), rows, 1, hf, back, turn[wave]);
        }
    });
}

template <typename T> hipError_t launch_down(Params p, const Plan& c, hipStream_t s)
{
    p.slots = c.down_slots;
    p.tile = c.down_tile;
    p.rblocks = (p.rank + 16 * c.down_ranks - 1) / (16 * c.down_ranks);
    const dim3 grid((unsigned)(ceil_div(p.m, p.tile) * p.splits * p.slots * p.rblocks)), block(kDownWaves * 64);
    if (c.down_ranks == 1) adapters_down_kernel<T, 1><<<grid, block, 0, s>>>(p);
    else if (c.down_ranks == 2) adapters_down_kernel<T, 2><<<grid, block, 0, s>>>(p);
    else adapters_down_kernel<T, 4><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T> hipError_t launch_up(Params p, const Plan& c, hipStream_t s)
{
    p.slots = c.up_slots;
    p.tile = c.up_tile;
    p.blocks = c.up_blocks;
    p.nblocks = (int)ceil_div(p.n, 64 * kUpWaves * p.blocks);
    const dim3 grid((unsigned)(ceil_div(p.m, p.tile) * p.nblocks * p.slots)), block(kUpWaves * 64);
    if (p.rank <= 16) adapters_up_kernel<T, 0, false><<<grid, block, 0, s>>>(p);
    else if (p.rank <= 32) adapters_up_kernel<T, 1, false><<<grid, block, 0, s>>>(p);
    else if (p.rank <= 64 && p.blocks == 1) adapters_up_kernel<T, 2, false><<<grid, block, 0, s>>>(p);
    else if (p.rank <= 64) adapters_up_kernel<T, 2, true><<<grid, block, 0, s>>>(p);
    else if (p.blocks == 1) adapters_up_kernel<T, 4, false><<<grid, block, 0, s>>>(p);
    else adapters_up_kernel<T, 4, true><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T> hipError_t launch_one(Params p, const Plan& c, hipStream_t s)
{
    p.slots = c.one_slots;
    p.tile = 32;
    p.k_per = p.k;
    p.nblocks = (int)ceil_div(p.n, 64 * kOneWaves);
    const int slots = p.slots < 8 ? p.slots : (p.slots + 7) / 8 * 8;
    const dim3 grid((unsigned)(ceil_div(p.m, 32) * p.nblocks * slots)), block(kOneWaves * 64);
    if (p.rank <= 16) adapters_one_kernel<T, 0><<<grid, block, 0, s>>>(p);
    else adapters_one_kernel<T, 1><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T> hipError_t launch_both(const Params& p, const Plan& c, hipStream_t s)
{
    if (c.one) return launch_one<T>(p, c, s);
    const hipError_t e = launch_down<T>(p, c, s);
    return e != hipSuccess ? e : launch_up<T>(p, c, s);
}

}  // namespace

}  // namespace adapters

size_t adapters_workspace(int64_t m, int64_t n, int64_t k, int rank, int count, int f16)
{
    const adapters::Plan c = adapters::plan_of(m, n, k, rank, count, f16);
    return c.one ? 0 : (size_t)c.splits * m * c.pitch * 4;
}

hipError_t launch_adapters(const AdapterArgs& a, hipStream_t stream, const char** variant)
{
    const adapters::Plan c = adapters::plan_of(a.m, a.n, a.k, a.rank, a.count, a.f16);
    adapters::Params p = {};
    p.a = a.a;
    p.b = a.b;
    p.scales = a.scales;
    p.ranks = a.ranks;
    p.adapter = a.adapter;
    p.x = a.x;
    p.base = a.base;
    p.y = a.y;
    p.h = static_cast<float*>(a.workspace);
    p.m = a.m;
    p.n = a.n;
    p.k = a.k;
    p.x_stride = a.x_stride;
    p.base_stride = a.base_stride;
    p.y_stride = a.y_stride;
    p.k_per = c.k_per;
    p.rank = a.rank;
    p.count = a.count;
    p.splits = c.splits;
    p.pitch = c.pitch;
    *variant = c.one ? "adapters_one" : "adapters";
    return a.f16 ? adapters::launch_both<_Float16>(p, c, stream) : adapters::launch_both<float>(p, c, stream);
}

}  // namespace mnb
