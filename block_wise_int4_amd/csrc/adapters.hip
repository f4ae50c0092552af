// adapters.hip -- low-rank adapters of many requests beside one projection:
//
//   y[t] = base[t] + s_a B_a (A_a x[t]),   a = adapter[t],
//
// A_a [rank, k], B_a [n, rank]; rows of a call may have any adapters in any
// order.  Two kernels: h = A x in fp32, then y = base + s B h.
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
    int rank, count, splits, slots, pitch, rblocks, nblocks;
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

// The rows of a tile of 64, a lane each: adapter (-1: none, out of range or of rank 0) and its rank.
struct Rows {
    int adapter, rank;
};
__device__ __forceinline__ Rows rows_of(const Params& p, int64_t row)
{
    Rows r = {-1, p.rank};
    if (row < p.m) {
        const int a = p.adapter[row];
        if (a >= 0 && a < p.count) {
            if (p.ranks) r.rank = p.ranks[a] < p.rank ? p.ranks[a] : p.rank;
            r.adapter = r.rank > 0 ? a : -1;
        }
    }
    return r;
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

// Ranks rank0 .. of h = A x for up to 16 CU rows of one adapter, the waves sharing k.
template <typename T, int CU, int RT>
__device__ __forceinline__ void down_rows(const Params& p, int ad, int rank0, int rank, int order, int rows, int64_t row0,
                                          int split, float (*red)[64][20])
{
    constexpr int E = Vec<T>::E, STEP = 8 * E, KW = kDownWaves;
    constexpr int U = RT + CU <= 2 ? 4 : RT + CU <= 5 ? 2 : 1;   // steps requested at once
    constexpr int S = 4 < CU * RT ? 4 : CU * RT;        // 16 x 16 tiles that meet in LDS at once
    typedef typename Vec<T>::type V;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int64_t k0 = split * p.k_per, k1 = k0 + p.k_per < p.k ? k0 + p.k_per : p.k;
    const int full = (int)((k1 - k0) / STEP);
    const int left = (int)((k1 - k0) % STEP);

    const T* xp[CU];
#pragma unroll
    for (int u = 0; u < CU; ++u) {
        int n = 16 * u + col;
        n = n < rows ? n : rows - 1;                    // not written
        xp[u] = static_cast<const T*>(p.x) + (row0 + __shfl(order, n)) * p.x_stride + k0 + quarter * 2 * E;
    }
    const T* ap[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        int r = 16 * t + col;
        r = r < rank ? r : rank - 1;                    // not written
        ap[t] = static_cast<const T*>(p.a) + ((int64_t)ad * p.rank + rank0 + r) * p.k + k0 + quarter * 2 * E;
    }
    f4_t acc[CU][RT];
#pragma unroll
    for (int u = 0; u < CU; ++u)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[u][t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};

    int s = wave;
    for (; s + (U - 1) * KW < full; s += U * KW) {
        V xv[U][CU][2], av[U][RT][2];
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int64_t at = (int64_t)(s + i * KW) * STEP + e * E;
#pragma unroll
                for (int u = 0; u < CU; ++u) xv[i][u][e] = load(xp[u] + at);
#pragma unroll
                for (int t = 0; t < RT; ++t) av[i][t][e] = load(ap[t] + at);
            }
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int u = 0; u < CU; ++u) acc[u][t] = product(av[i][t][e], xv[i][u][e], acc[u][t]);
    }
    for (; s <= full; s += KW) {
        const int64_t at = (int64_t)s * STEP;
        const int valid = s < full ? STEP : left;
        if (valid == 0) break;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int here = valid - quarter * 2 * E - e * E;
            V xv[CU], av[RT];
#pragma unroll
            for (int u = 0; u < CU; ++u) xv[u] = load_some(xp[u] + at + e * E, here);
#pragma unroll
            for (int t = 0; t < RT; ++t) av[t] = load_some(ap[t] + at + e * E, here);
#pragma unroll
            for (int t = 0; t < RT; ++t)
#pragma unroll
                for (int u = 0; u < CU; ++u) acc[u][t] = product(av[t], xv[u], acc[u][t]);
        }
    }
    // the waves' sums meet in LDS
#pragma unroll
    for (int i0 = 0; i0 < CU * RT; i0 += S) {
        if (i0 / CU * 16 >= rank) break;
        __syncthreads();                                // the last ones have been read
#pragma unroll
        for (int i = 0; i < S; ++i)
            *reinterpret_cast<f4_t*>(&red[wave][16 * i + col][4 * quarter]) = acc[(i0 + i) % CU][(i0 + i) / CU];
        __syncthreads();
#pragma unroll
        for (int part = 0; part < (16 * S + 31) / 32; ++part) {
            const int at = (threadIdx.x >> 4) + 32 * part, r0 = threadIdx.x & 15;
            const int i = i0 + at / 16, n = 16 * (i % CU) + at % 16, r = 16 * (i / CU) + r0;
            const int row = __shfl(order, n & 63);
            if (at < 16 * S && n < rows && r < rank) {
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < KW; ++w) sum += red[w][at][r0];
                p.h[((int64_t)split * p.m + row0 + row) * p.pitch + rank0 + r] = sum;
            }
        }
    }
}

// h = A x for a tile of 64 rows, 16 RT ranks and the adapters of one slot.
template <typename T, int RT> __global__ __launch_bounds__(kDownWaves * 64, RT <= 2 ? 4 : 2) void adapters_down_kernel(Params p)
{
    __shared__ __align__(16) float red[kDownWaves][64][20];
    const int lane = threadIdx.x & 63;
    const int slot = blockIdx.x % p.slots, split = blockIdx.x / p.slots % p.splits;
    const int rank0 = blockIdx.x / p.slots / p.splits % p.rblocks * (16 * RT);
    const int64_t row0 = (int64_t)(blockIdx.x / p.slots / p.splits / p.rblocks) * 64;
    const Rows mine = rows_of(p, row0 + lane);
    for_adapters(mine, slot, p.slots, [&](int ad, int rank, uint64_t same) {
        const int order = gathered(same, lane), rows = __builtin_popcountll(same);
        const int here = rank - rank0 < 16 * RT ? rank - rank0 : 16 * RT;
        if (here <= 0) return;
        if (rows > 32) down_rows<T, 4, RT>(p, ad, rank0, here, order, rows, row0, split, red);
        else if (rows > 16) down_rows<T, 2, RT>(p, ad, rank0, here, order, rows, row0, split, red);
        else down_rows<T, 1, RT>(p, ad, rank0, here, order, rows, row0, split, red);
    });
}

// N ranks of h from rank r of a row on, the splits' sums added.
template <int N>
__device__ __forceinline__ void add_parts(const Params& p, int64_t row, int r, int rank, bool there, float* v)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    if (!there || r >= rank) return;
    const float* h = p.h + row * p.pitch + r;
    const int64_t step = p.m * p.pitch;
    int s = 0;
    for (; s + 4 <= p.splits; s += 4, h += 4 * step) {
        f4_t q[4][N / 4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < N / 4; ++i) q[k][i] = *reinterpret_cast<const f4_t*>(h + k * step + 4 * i);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += q[k][i / 4][i % 4];
    }
    for (; s < p.splits; ++s, h += step)
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const f4_t q = *reinterpret_cast<const f4_t*>(h + 4 * i);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * i + e] += q[e];
        }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = r + i < rank ? v[i] : 0.0f;
}

// The second product's operands.  RC: 32-rank chunks; 0: up to 16 ranks, both fp16 parts
// of h in one product.
template <typename T, int RC> struct Up;

template <int RC> struct Up<_Float16, RC> {
    static constexpr int NC = RC == 0 ? 1 : RC, PARTS = RC == 0 ? 1 : 2;
    typedef h8_t piece;
    // column of row i of tile j: a lane's results are 8 neighbours of the first 32
    // columns and 8 of the second
    static __device__ __forceinline__ int column(int j, int i) { return 32 * (j >> 1) + 8 * (i >> 2) + 4 * (j & 1) + (i & 3); }
    static __device__ __forceinline__ int rank0(int c, int quarter) { return RC == 0 ? 8 * (quarter & 1) : 32 * c + 8 * quarter; }
    // h as two fp16 parts, 22 bits, of the row scaled to below 2^15; the power of two taken out
    static __device__ __forceinline__ float load_h(const Params& p, int64_t row, int rank, bool there, int quarter, piece* out)
    {
        float v[NC][8], mx = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            add_parts<8>(p, row, rank0(c, quarter), rank, there, v[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(v[c][i]) < __builtin_inff() ? fabsf(v[c][i]) : 0.0f);
        }
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        int e = mx > 0.0f ? (int)(__builtin_bit_cast(uint32_t, mx) >> 23) - 127 - 14 : 0;
        e = e < -126 ? -126 : e;
        const float down = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            h8_t hi, lo;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = v[c][i] * down;
                hi[i] = (_Float16)s;
                lo[i] = fabsf(s) < __builtin_inff() ? (_Float16)(s - (float)hi[i]) : (_Float16)0.0f;
            }
            if constexpr (RC == 0) out[0] = quarter < 2 ? hi : lo;
            else {
                out[2 * c] = hi;
                out[2 * c + 1] = lo;
            }
        }
        return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
    }
};

template <int RC> struct Up<float, RC> {
    static constexpr int NC = RC == 0 ? 1 : 2 * RC, PARTS = 1;   // 16-rank chunks
    typedef f4_t piece;
    static __device__ __forceinline__ int column(int j, int i) { return 16 * j + i; }
    static __device__ __forceinline__ int rank0(int c, int quarter) { return 16 * c + 4 * quarter; }
    static __device__ __forceinline__ float load_h(const Params& p, int64_t row, int rank, bool there, int quarter, piece* out)
    {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float v[4];
            add_parts<4>(p, row, rank0(c, quarter), rank, there, v);
            out[c] = f4_t{v[0], v[1], v[2], v[3]};
        }
        return 1.0f;
    }
};

// A lane's elements of base in N 16-row tiles.
template <typename T, int NT> struct Base {
    static constexpr int N = NT;
    typename Vec<T>::type v[N][16 / Vec<T>::E];
    int row[N];
};

// y = base + s B h for 64 rows and 64 columns a wave.
template <typename T, int RC> __global__ __launch_bounds__(kUpWaves * 64, RC <= 1 ? 4 : 2) void adapters_up_kernel(Params p)
{
    typedef Up<T, RC> O;
    typedef typename Vec<T>::type V;
    constexpr int E = Vec<T>::E, PIECES = 16 / E;       // 16-byte pieces of a lane's 16 columns
    constexpr int NH = O::NC * O::PARTS;
    constexpr int PRE = sizeof(T) == 4 ? (RC < 2 ? 2 : 1) : RC < 4 ? 4 : 2;   // 16-row tiles whose base is requested at once
    __shared__ __align__(16) typename O::piece hf[4][NH][64];    // h of four 16-row tiles, as operands
    __shared__ float back[4][16];

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int slot = blockIdx.x % p.slots;
    const int64_t n0 = ((int64_t)(blockIdx.x / p.slots % p.nblocks) * kUpWaves + wave) * 64;
    const int64_t row0 = (int64_t)(blockIdx.x / p.slots / p.nblocks) * 64;
    const bool busy = n0 < p.n;                         // a wave past the columns only prepares h
    const Rows mine = rows_of(p, row0 + lane);
    auto at = [&](int i) { return O::column(i * E / 4, 4 * quarter); };   // column of piece i of the lane
    auto put = [&](T* y, int i, const V& v) {
        const int64_t left = p.n - n0 - at(i);
        if (left >= E) store(y + at(i), v);
        else
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e < left) y[at(i) + e] = v[e];
    };
    const T* base0 = p.base ? static_cast<const T*>(p.base) + row0 * p.base_stride + n0 : nullptr;
    T* y0 = static_cast<T*>(p.y) + row0 * p.y_stride + n0;

    // rows without an adapter
    const uint64_t none = __builtin_amdgcn_ballot_w64(mine.adapter < 0 && row0 + lane < p.m);
    if (none && slot == 0 && busy && base0 != y0) {
        const int order = gathered(none, lane), rows = __builtin_popcountll(none);
        for (int u = 0; 16 * u < rows; ++u) {
            const int row = __shfl(order, 16 * u + col);
            if (16 * u + col < rows) {
#pragma unroll
                for (int i = 0; i < PIECES; ++i) {
                    V v = {};
                    if (base0) v = load_some(base0 + row * p.base_stride + at(i), p.n - n0 - at(i));
                    put(y0 + row * p.y_stride, i, v);
                }
            }
        }
    }
    for_adapters(mine, slot, p.slots, [&](int ad, int rank, uint64_t same) {
        const int order = gathered(same, lane), rows = __builtin_popcountll(same);
        // B, of this wave's columns
        V b[O::NC][4];
        const T* w = static_cast<const T*>(p.b) + (int64_t)ad * p.n * p.rank;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            int64_t n = n0 + O::column(j, col);
            n = n < p.n ? n : p.n - 1;                  // not written
#pragma unroll
            for (int c = 0; c < O::NC; ++c)
                b[c][j] = load_some(w + n * p.rank + O::rank0(c, quarter), rank - O::rank0(c, quarter));
        }
        const float scale = p.scales ? p.scales[ad] : 1.0f;
        // N 16-row tiles of base from tile g on
        auto request = [&](auto in, int g) {
#pragma unroll
            for (int u = 0; u < decltype(in)::N; ++u) {
                in.row[u] = __shfl(order, 16 * (g + u) + col);
#pragma unroll
                for (int i = 0; i < PIECES; ++i) {
                    in.v[u][i] = V{};
                    if (base0 && busy && 16 * (g + u) + col < rows)
                        in.v[u][i] = load_some(base0 + in.row[u] * p.base_stride + at(i), p.n - n0 - at(i));
                }
            }
            return in;
        };
        auto finish = [&](const auto& in, int g) {
#pragma unroll
            for (int u = 0; u < std::decay<decltype(in)>::type::N; ++u) {
                if (16 * (g + u) >= rows) break;
                f4_t acc[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < NH; ++c) {
                    const typename O::piece h = hf[g + u][c][lane];
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[j] = product(b[c / O::PARTS][j], h, acc[j]);
                }
                const float factor = scale * back[g + u][col];
                if (16 * (g + u) + col < rows) {
#pragma unroll
                    for (int i = 0; i < PIECES; ++i) {
                        V v;
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            v[e] = (T)__builtin_fmaf(acc[(i * E + e) / 4][e & 3], factor, (float)in.v[u][i][e]);
                        put(y0 + in.row[u] * p.y_stride, i, v);
                    }
                }
            }
        };
        // h: a 16-row tile to a wave
        auto prepare = [&]() {
            __syncthreads();                            // the last adapter's has been read
            for (int u = wave; 16 * u < rows; u += kUpWaves) {
                typename O::piece h[NH];
                const int64_t from = row0 + __shfl(order, 16 * u + col);
                const float f = O::load_h(p, from, rank, 16 * u + col < rows, quarter, h);
#pragma unroll
                for (int c = 0; c < NH; ++c) hf[u][c][lane] = h[c];
                if (quarter == 0) back[u][col] = f;
            }
            __syncthreads();
        };
        if (rows <= 16) {
            // a few rows wait for their loads: base on its way beside h.  (More have no registers for it.)
            const auto in = request(Base<T, 1>(), 0);
            prepare();
            if (busy) finish(in, 0);
        } else {
            prepare();
            if (!busy) return;
#pragma unroll
            for (int g = 0; g < 4; g += PRE)
                if (16 * g < rows) finish(request(Base<T, PRE>(), g), g);
        }
    });
}

template <typename T> hipError_t launch_down(Params p, const Plan& c, hipStream_t s)
{
    p.slots = c.down_slots;
    p.rblocks = (p.rank + 63) / 64;
    const dim3 grid((unsigned)(ceil_div(p.m, 64) * p.splits * p.slots * p.rblocks)), block(kDownWaves * 64);
    if (p.rank <= 16) adapters_down_kernel<T, 1><<<grid, block, 0, s>>>(p);
    else if (p.rank <= 32) adapters_down_kernel<T, 2><<<grid, block, 0, s>>>(p);
    else adapters_down_kernel<T, 4><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T> hipError_t launch_up(Params p, const Plan& c, hipStream_t s)
{
    p.slots = c.up_slots;
    p.nblocks = (int)ceil_div(p.n, 64 * kUpWaves);
    const dim3 grid((unsigned)(ceil_div(p.m, 64) * p.nblocks * p.slots)), block(kUpWaves * 64);
    if (p.rank <= 16) adapters_up_kernel<T, 0><<<grid, block, 0, s>>>(p);
    else if (p.rank <= 32) adapters_up_kernel<T, 1><<<grid, block, 0, s>>>(p);
    else if (p.rank <= 64) adapters_up_kernel<T, 2><<<grid, block, 0, s>>>(p);
    else adapters_up_kernel<T, 4><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T> hipError_t launch_both(const Params& p, const Plan& c, hipStream_t s)
{
    const hipError_t e = launch_down<T>(p, c, s);
    return e != hipSuccess ? e : launch_up<T>(p, c, s);
}

}  // namespace

}  // namespace adapters

size_t adapters_workspace(int64_t m, int64_t n, int64_t k, int rank, int count, int f16)
{
    const adapters::Plan c = adapters::plan_of(m, n, k, rank, count, f16);
    return (size_t)c.splits * m * c.pitch * 4;
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
    *variant = "adapters";
    return a.f16 ? adapters::launch_both<_Float16>(p, c, stream) : adapters::launch_both<float>(p, c, stream);
}

}  // namespace mnb
