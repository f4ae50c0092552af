// adapters.hip -- low-rank adapters of many requests beside one projection:
//
//   y[t] = base[t] + s_a B_a (A_a x[t]),   a = adapter[t],
//
// A_a [rank, k], B_a [n, rank]; rows of a call may have any adapters in any
// order.  Two kernels: h = A x in fp32, then y = base + s B h.
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
    int rank, count, splits, slots, pitch, span, nblocks;
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

// The adapter of row `row`, or -1: none, out of range or of rank 0.
__device__ __forceinline__ int adapter_of(const Params& p, int64_t row, bool there)
{
    int a = -1;
    if (there && row < p.m) {
        a = p.adapter[row];
        a = a < 0 || a >= p.count ? -1 : a;
        if (a >= 0 && p.ranks && p.ranks[a] <= 0) a = -1;
    }
    return a;
}
__device__ __forceinline__ int rank_of(const Params& p, int a)
{
    const int r = p.ranks ? p.ranks[a] : p.rank;
    return uniform(r < p.rank ? r : p.rank);
}

// h = A x for a tile of 16 TT rows and the adapters of one slot: the waves share k.
template <typename T, int TT, int RT>
__global__ __launch_bounds__(kDownWaves * 64) void adapters_down_kernel(Params p)
{
    constexpr int E = Vec<T>::E, STEP = 8 * E, KW = kDownWaves, PITCH = 20;
    constexpr int U = RT * TT <= 2 ? 4 : RT * TT <= 4 ? 2 : 1;   // steps requested at once
    typedef typename Vec<T>::type V;
    __shared__ __align__(16) float red[KW][16 * TT][PITCH];

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int slot = blockIdx.x % p.slots, split = blockIdx.x / p.slots % p.splits;
    const int64_t row0 = (int64_t)(blockIdx.x / p.slots / p.splits) * (16 * TT);
    const int64_t k0 = split * p.k_per, k1 = k0 + p.k_per < p.k ? k0 + p.k_per : p.k;
    const int full = (int)((k1 - k0) / STEP);
    const int left = (int)((k1 - k0) % STEP);

    const T* xp[TT];
#pragma unroll
    for (int u = 0; u < TT; ++u) {
        int64_t row = row0 + 16 * u + col;
        row = row < p.m ? row : p.m - 1;
        xp[u] = static_cast<const T*>(p.x) + row * p.x_stride + k0 + quarter * 2 * E;
    }
    const int mine = adapter_of(p, row0 + lane, lane < 16 * TT);
    uint64_t todo = __builtin_amdgcn_ballot_w64(mine >= 0);
    int skip = slot;
    while (todo) {
        const int ad = __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo));
        const uint64_t same = __builtin_amdgcn_ballot_w64(mine == ad);
        todo &= ~same;
        if (skip > 0) {
            --skip;
            continue;
        }
        skip = p.slots - 1;
        const int rank = rank_of(p, ad);
        const T* ap[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            int r = 16 * t + col;
            r = r < rank ? r : rank - 1;                // not written
            ap[t] = static_cast<const T*>(p.a) + ((int64_t)ad * p.rank + r) * p.k + k0 + quarter * 2 * E;
        }
        f4_t acc[TT][RT];
#pragma unroll
        for (int u = 0; u < TT; ++u)
#pragma unroll
            for (int t = 0; t < RT; ++t) acc[u][t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};

        int s = wave;
        for (; s + (U - 1) * KW < full; s += U * KW) {
            V xv[U][TT][2], av[U][RT][2];
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int64_t at = (int64_t)(s + i * KW) * STEP + e * E;
#pragma unroll
                    for (int u = 0; u < TT; ++u) xv[i][u][e] = load(xp[u] + at);
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
                        for (int u = 0; u < TT; ++u) acc[u][t] = product(av[i][t][e], xv[i][u][e], acc[u][t]);
        }
        for (; s <= full; s += KW) {
            const int64_t at = (int64_t)s * STEP;
            const int valid = s < full ? STEP : left;
            if (valid == 0) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int here = valid - quarter * 2 * E - e * E;
                V xv[TT], av[RT];
#pragma unroll
                for (int u = 0; u < TT; ++u) xv[u] = load_some(xp[u] + at + e * E, here);
#pragma unroll
                for (int t = 0; t < RT; ++t) av[t] = load_some(ap[t] + at + e * E, here);
#pragma unroll
                for (int t = 0; t < RT; ++t)
#pragma unroll
                    for (int u = 0; u < TT; ++u) acc[u][t] = product(av[t], xv[u], acc[u][t]);
            }
        }
        // the waves' sums meet in LDS, 16 ranks at a time
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            if (16 * t >= rank) break;
#pragma unroll
            for (int u = 0; u < TT; ++u) *reinterpret_cast<f4_t*>(&red[wave][16 * u + col][4 * quarter]) = acc[u][t];
            __syncthreads();
            const int row = threadIdx.x >> 4, r = threadIdx.x & 15;
            if (row < 16 * TT && 16 * t + r < rank && (same >> row & 1)) {
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < KW; ++w) sum += red[w][row][r];
                p.h[((int64_t)split * p.m + row0 + row) * p.pitch + 16 * t + r] = sum;
            }
            __syncthreads();
        }
    }
}

// The second product's operand of a lane's row: ranks 8 quarter + 32 c ..  (fp32: 4
// quarter + 16 c ..), the splits' sums added.
__device__ __forceinline__ void add_parts(const Params& p, int64_t row, int r, int rank, bool there, float* v, int count)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < count) v[i] = 0.0f;
    if (!there || r >= rank) return;
    const float* h = p.h + row * p.pitch + r;
    for (int s = 0; s < p.splits; ++s, h += p.m * p.pitch) {
#pragma unroll
        for (int i = 0; i < 8; i += 4)
            if (i < count) {
                const f4_t q = *reinterpret_cast<const f4_t*>(h + i);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i + e] += q[e];
            }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < count && r + i >= rank) v[i] = 0.0f;
}

// RC: 32-rank chunks; 0: up to 16 ranks, both fp16 parts of h in one product.
template <typename T, int RC> struct Up;

template <int RC> struct Up<_Float16, RC> {
    static constexpr int NC = RC == 0 ? 1 : RC;
    h8_t b[NC][4], hi[NC], lo[NC];
    float back;                       // the power of two taken out of the row

    // column of row i of tile j: a lane's results are 8 neighbours of the first 32
    // columns and 8 of the second
    static __device__ __forceinline__ int column(int j, int i) { return 32 * (j >> 1) + 8 * (i >> 2) + 4 * (j & 1) + (i & 3); }
    static __device__ __forceinline__ int rank0(int c, int quarter) { return RC == 0 ? 8 * (quarter & 1) : 32 * c + 8 * quarter; }
    __device__ __forceinline__ void load_b(const Params& p, int ad, int rank, int64_t n0, int col, int quarter)
    {
        const _Float16* w = static_cast<const _Float16*>(p.b) + (int64_t)ad * p.n * p.rank;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            int64_t n = n0 + column(j, col);
            n = n < p.n ? n : p.n - 1;                  // not written
#pragma unroll
            for (int c = 0; c < NC; ++c) b[c][j] = load_some(w + n * p.rank + rank0(c, quarter), rank - rank0(c, quarter));
        }
    }
    // h as two fp16 parts, 22 bits, of the row scaled to below 2^15
    __device__ __forceinline__ void load_h(const Params& p, int64_t row, int rank, bool there, int quarter)
    {
        float v[NC][8], mx = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            add_parts(p, row, rank0(c, quarter), rank, there, v[c], 8);
#pragma unroll
            for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(v[c][i]) < __builtin_inff() ? fabsf(v[c][i]) : 0.0f);
        }
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        int e = mx > 0.0f ? (int)(__builtin_bit_cast(uint32_t, mx) >> 23) - 127 - 14 : 0;
        e = e < -126 ? -126 : e;
        const float down = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
        back = __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = v[c][i] * down;
                const _Float16 top = (_Float16)s;
                hi[c][i] = top;
                lo[c][i] = fabsf(s) < __builtin_inff() ? (_Float16)(s - (float)top) : (_Float16)0.0f;
            }
        if constexpr (RC == 0) hi[0] = quarter < 2 ? hi[0] : lo[0];
    }
    __device__ __forceinline__ void multiply(f4_t* acc) const
    {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[j] = mfma16(b[c][j], hi[c], acc[j]);
                if constexpr (RC > 0) acc[j] = mfma16(b[c][j], lo[c], acc[j]);
            }
    }
};

template <int RC> struct Up<float, RC> {
    static constexpr int NC = RC == 0 ? 1 : 2 * RC;     // 16-rank chunks
    f4_t b[NC][4], h[NC];
    static constexpr float back = 1.0f;

    static __device__ __forceinline__ int column(int j, int i) { return 16 * j + i; }
    __device__ __forceinline__ void load_b(const Params& p, int ad, int rank, int64_t n0, int col, int quarter)
    {
        const float* w = static_cast<const float*>(p.b) + (int64_t)ad * p.n * p.rank;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            int64_t n = n0 + column(j, col);
            n = n < p.n ? n : p.n - 1;                  // not written
#pragma unroll
            for (int c = 0; c < NC; ++c)
                b[c][j] = load_some(w + n * p.rank + 16 * c + 4 * quarter, rank - (16 * c + 4 * quarter));
        }
    }
    __device__ __forceinline__ void load_h(const Params& p, int64_t row, int rank, bool there, int quarter)
    {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float v[8];
            add_parts(p, row, 16 * c + 4 * quarter, rank, there, v, 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[c][i] = v[i];
        }
    }
    __device__ __forceinline__ void multiply(f4_t* acc) const
    {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = product(b[c][j], h[c], acc[j]);
    }
};

// y = base + s B h for 16 span rows and 64 columns a wave.
template <typename T, int RC>
__global__ __launch_bounds__(256) void adapters_up_kernel(Params p)
{
    constexpr int E = Vec<T>::E, PIECES = 16 / E;       // 16-byte pieces of a lane's 16 columns
    typedef typename Vec<T>::type V;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int slot = blockIdx.x % p.slots;
    const int64_t n0 = ((int64_t)(blockIdx.x / p.slots % p.nblocks) * (blockDim.x >> 6) + wave) * 64;
    const int64_t first = (int64_t)(blockIdx.x / p.slots / p.nblocks) * p.span;
    if (n0 >= p.n) return;
    Up<T, RC> up;
    int held = -1, rank = 0;
    float scale = 0.0f;
    for (int tile = 0; tile < p.span; ++tile) {
        const int64_t row = (first + tile) * 16 + col;
        if ((first + tile) * 16 >= p.m) break;
        const int mine = adapter_of(p, row, true);
        const T* base = p.base ? static_cast<const T*>(p.base) + row * p.base_stride + n0 : nullptr;
        T* y = static_cast<T*>(p.y) + row * p.y_stride + n0;
        // piece i of the lane: its column, and whether all of it is there
        auto at = [&](int i) { return Up<T, RC>::column(i * E / 4, 4 * quarter); };
        uint64_t todo = __builtin_amdgcn_ballot_w64(mine >= 0) & 0xFFFF;
        if (slot == 0 && mine < 0 && row < p.m && base != y) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const int64_t left = p.n - n0 - at(i);
                V v = {};
                if (base) v = load_some(base + at(i), left);
                if (left >= E) store(y + at(i), v);
                else
                    for (int e = 0; e < left; ++e) y[at(i) + e] = v[e];
            }
        }
        int skip = slot;
        while (todo) {
            const int ad = __builtin_amdgcn_readlane(mine, __builtin_ctzll(todo));
            todo &= ~__builtin_amdgcn_ballot_w64(mine == ad);
            if (skip > 0) {
                --skip;
                continue;
            }
            skip = p.slots - 1;
            const bool there = mine == ad;
            V in[PIECES];
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                in[i] = V{};
                if (base && there) in[i] = load_some(base + at(i), p.n - n0 - at(i));
            }
            if (ad != held) {
                held = ad;
                rank = rank_of(p, ad);
                scale = p.scales ? p.scales[ad] : 1.0f;
                up.load_b(p, ad, rank, n0, col, quarter);
            }
            up.load_h(p, row, rank, there, quarter);
            f4_t acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
            up.multiply(acc);
            const float factor = scale * up.back;
            if (there) {
#pragma unroll
                for (int i = 0; i < PIECES; ++i) {
                    V v;
#pragma unroll
                    for (int e = 0; e < E; ++e) v[e] = (T)__builtin_fmaf(acc[(i * E + e) / 4][e & 3], factor, (float)in[i][e]);
                    const int64_t left = p.n - n0 - at(i);
                    if (left >= E) store(y + at(i), v);
                    else
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            if (e < left) y[at(i) + e] = v[e];
                }
            }
        }
    }
}

template <typename T, int TT> hipError_t launch_down(const Params& p, const Plan& c, hipStream_t s)
{
    const dim3 grid((unsigned)(ceil_div(p.m, 16 * TT) * p.splits * p.slots)), block(kDownWaves * 64);
    if (p.rank <= 16) adapters_down_kernel<T, TT, 1><<<grid, block, 0, s>>>(p);
    else if (p.rank <= 32) adapters_down_kernel<T, TT, 2><<<grid, block, 0, s>>>(p);
    else if (p.rank <= 64) adapters_down_kernel<T, TT, 4><<<grid, block, 0, s>>>(p);
    else adapters_down_kernel<T, TT, 8><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T> hipError_t launch_both(Params p, const Plan& c, hipStream_t s)
{
    p.slots = c.down_slots;
    const hipError_t e = c.tiles16 == 2 ? launch_down<T, 2>(p, c, s) : launch_down<T, 1>(p, c, s);
    if (e != hipSuccess) return e;
    p.slots = c.up_slots;
    p.nblocks = (int)ceil_div(p.n, 64 * c.up_waves);
    const dim3 grid((unsigned)(ceil_div(ceil_div(p.m, 16), c.span) * p.nblocks * p.slots)), block(64 * c.up_waves);
    if (p.rank <= 16) adapters_up_kernel<T, 0><<<grid, block, 0, s>>>(p);
    else if (p.rank <= 32) adapters_up_kernel<T, 1><<<grid, block, 0, s>>>(p);
    else if (p.rank <= 64) adapters_up_kernel<T, 2><<<grid, block, 0, s>>>(p);
    else adapters_up_kernel<T, 4><<<grid, block, 0, s>>>(p);
    return hipGetLastError();
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
    p.span = c.span;
    *variant = c.tiles16 == 2 ? "adapters_prompt" : "adapters";
    return a.f16 ? adapters::launch_both<_Float16>(p, c, stream) : adapters::launch_both<float>(p, c, stream);
}

}  // namespace mnb
