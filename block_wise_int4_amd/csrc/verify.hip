// verify.hip -- drafted tokens against the target's probabilities, from given
// random numbers.
//
// A sequence's rows are those of its step: row 0 is the last sure token, row i the
// i-th draft, and row i's probabilities p judge the token of row i + 1.  Draft d with
// p(d), q(d) is accepted if u q(d) < p(d): with u uniform in [0, 1) that has
// probability min(1, p / q).  At the first refusal the token is drawn from
// max(p - q, 0), after the last draft from p: the lowest i whose sum of weights up to i
// passes pick times the sum of all.  So the tokens are distributed as if drawn from p.
//
// Products of two binary32 values are exact in 64 bits, and sums are kept in 64 bits:
// a token lies at the border of two sums, and 32 bits would give another for one draw
// in some hundred at 100000 tokens.
//
// A chunk of 1024 tokens a wave, of the one row that the draw needs (every workgroup
// finds that row for itself); then a wave takes the sequence's chunk and in it the token.
// Two launches, or one where a workgroup does for a sequence.  What is read bounds large calls,
// the row and its draft's once: 32 sequences of 128000 tokens in fp32, 32.8 MB, 12.1 us, the
// sums' kernel 7.8 of them (fp16 10.7 and 5.7).  Beside the loads it is work in 64 bits: per token a conversion and
// an addition, with drafts of a distribution five (512 certain fp16 rows of 128000: 47 us
// before the weights were chosen in 32 bits and a second sum taken only where it differs, 34 after
// in the same two launches).
// Small calls are latency: 7.3 us of one sequence in a graph are two launches, and the loads that wait
// for each other: rows, ids, a probability, the row; then the sums, the chunk.
#include "mnb_requests.hpp"
#include "mnb_vec.hpp"

namespace mnb {
namespace verify {

constexpr int kThreads = 256, kOneThreads = 1024, kChunk = kVerifyChunk;
constexpr int kOneChunks = 256;        // that one workgroup's LDS has room for

namespace {

typedef double d2_t __attribute__((ext_vector_type(2)));

struct Params {
    const void* target;
    const void* draft;
    int64_t target_stride, draft_stride;
    const int32_t* ids;
    const int32_t* q_start;
    const float* accept;
    const float* pick;
    int32_t* out;
    int32_t* accepted;
    double* sums;                     // [batch][chunks][2]: of max(p - q, 0), of p
    int batch, tokens, vocab, chunks;
};

struct Rows { int first, count; };
__device__ __forceinline__ Rows rows_of(const Params& p, int b)
{
    int first = b, end = b + 1;
    if (p.q_start) {
        first = p.q_start[b];
        end = p.q_start[b + 1];
    }
    first = first < 0 ? 0 : first;
    end = end > p.tokens ? p.tokens : end;
    return Rows{first, end > first ? end - first : 0};
}

// A weight: a positive finite probability, or 0.
template <typename T> __device__ __forceinline__ double weight(T x)
{
    const float f = (float)x;
    return (double)(__builtin_amdgcn_classf(f, 0x180) ? f : 0.0f);   // positive normal or denormal
}

// Drafts accepted before the first refusal; every lane of a wave calls it.
template <typename T> __device__ __forceinline__ int accepted_of(const Params& p, const Rows& r, int lane)
{
    const int n = r.count - 1;
    for (int i0 = 0; i0 < n; i0 += 64) {
        const int i = i0 + lane;
        bool good = true;
        if (i < n) {
            const int64_t row = r.first + i;
            const int d = p.ids[row + 1];
            good = d >= 0 && d < p.vocab;
            if (good) {
                const double t = weight(static_cast<const T*>(p.target)[row * p.target_stride + d]);
                const double q = p.draft ? weight(static_cast<const T*>(p.draft)[row * p.draft_stride + d]) : 1.0;
                good = (double)p.accept[row] * q < t;
            }
        }
        const uint64_t bad = __builtin_amdgcn_ballot_w64(!good);
        if (bad) return i0 + __builtin_ctzll(bad);
    }
    return n;
}

// What a token's weight is taken from.
template <typename T> struct Draw {
    const T* p;
    const T* q;                       // NULL: none
    int gone;                         // a certain draft that was refused, or -1
    __device__ __forceinline__ Draw(const Params& a, const Rows& r, int accepted)
    {
        const int64_t row = r.first + accepted;
        const bool refused = accepted < r.count - 1;
        p = static_cast<const T*>(a.target) + row * a.target_stride;
        q = refused && a.draft ? static_cast<const T*>(a.draft) + row * a.draft_stride : nullptr;
        gone = refused && !a.draft ? a.ids[row + 1] : -1;
    }
    __device__ __forceinline__ double rest(double w, double v, int i) const
    {
        return i == gone ? 0.0 : __builtin_fmax(w - v, 0.0);
    }
};

// x of another lane of the 16, 0 past their ends: a rotation (0x120 + n), a shift (0x110 + n).
template <int CTRL> __device__ __forceinline__ double moved(double x)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)u, CTRL, 0xF, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, 0xF, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_of(double x, int lane)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((int)u, lane), hi = __builtin_amdgcn_readlane((int)(u >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Sums of a wave's lanes, and of those before this one.  16 lanes by moves between lanes, not
// through LDS, whose latency a lone wave would wait for.
__device__ __forceinline__ double wave_sum(double x)
{
    x += moved<0x128>(x);
    x += moved<0x124>(x);
    x += moved<0x122>(x);
    x += moved<0x121>(x);
    return (lane_of(x, 0) + lane_of(x, 16)) + (lane_of(x, 32) + lane_of(x, 48));
}
__device__ __forceinline__ double before(double x, int lane, double& total)
{
    x += moved<0x111>(x);
    x += moved<0x112>(x);
    x += moved<0x114>(x);
    x += moved<0x118>(x);
    const double one = lane_of(x, 15), two = one + lane_of(x, 31), three = two + lane_of(x, 47);
    total = three + lane_of(x, 63);
    return (lane < 16 ? 0.0 : lane < 32 ? one : lane < 48 ? two : three) + moved<0x111>(x);
}

// A chunk's values of a wave's lanes, and its two sums, the same in every lane.
template <typename T> struct Chunk {
    static constexpr int E = Vec<T>::E, PIECES = kChunk / 64 / E;
    typename Vec<T>::type tv[PIECES], qv[PIECES];
    __device__ __forceinline__ void load(const Params& p, const Draw<T>& d, int chunk, int lane)
    {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int at = chunk * kChunk + (i * 64 + lane) * E;
            tv[i] = load_some(d.p + at, p.vocab - at);
            qv[i] = {};
            if (d.q) qv[i] = load_some(d.q + at, p.vocab - at);
        }
    }
    __device__ __forceinline__ d2_t sums(const Draw<T>& d, int chunk, int lane) const
    {
        double rest = 0.0, all = 0.0;
        // which of the sums differ, a wave's lanes agree
        const bool differ = d.q || (uint32_t)d.gone / kChunk == (uint32_t)chunk;
        auto each = [&](auto f) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) f(weight(tv[i][e]), qv[i][e], chunk * kChunk + (i * 64 + lane) * E + e);
        };
        if (d.q) {
            each([&](double w, T q, int) {
                all += w;
                rest += __builtin_fmax(w - weight(q), 0.0);
            });
        } else {
            each([&](double w, T, int) { all += w; });
            if (differ) each([&](double w, T, int at) { rest += at == d.gone ? 0.0 : w; });
        }
        all = wave_sum(all);
        return d2_t{differ ? wave_sum(rest) : all, all};
    }
};

// One wave: the chunk whose sums pass the border, then the token in it, then the sequence's rows.
// A lane holds neighbouring chunks, then neighbouring tokens.
template <typename T>
__device__ __forceinline__ void draw_token(const Params& p, const Rows& r, int b, int n, const d2_t* sums, int lane)
{
    constexpr int E = Vec<T>::E, PER = kChunk / 64;
    const int per = (p.chunks + 63) / 64, c0 = lane * per, c1 = c0 + per < p.chunks ? c0 + per : p.chunks;
    d2_t mine = {0.0, 0.0};
#pragma unroll 4
    for (int c = c0; c < c1; ++c) mine += sums[c];
    double rest, all;
    const double rest_before = before(mine[0], lane, rest), all_before = before(mine[1], lane, all);
    // nothing is left of p where q is no smaller anywhere: then p itself
    const bool left = n < r.count - 1 && rest > 0.0;
    // no sum passes a pick of 1 or more: sums of another order than the total's might end above it
    const float u = p.pick[b];
    const double border = u >= 1.0f ? __builtin_inf() : (u > 0.0f ? (double)u : 0.0) * (left ? rest : all);
    // the first chunk that passes the border, else the last with a weight
    double run = left ? rest_before : all_before, under = 0.0;
    int hit = -1, end = -1;
    for (int c = c0; c < c1; ++c) {
        const double s = left ? sums[c][0] : sums[c][1];
        if (hit < 0 && s > 0.0 && run + s > border) {
            hit = c;
            under = run;
        }
        if (s > 0.0) end = c;
        run += s;
    }
    const uint64_t hits = __builtin_amdgcn_ballot_w64(hit >= 0), ends = __builtin_amdgcn_ballot_w64(end >= 0);
    int token = -1;
    if (ends) {
        const int from = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(ends);
        const int chunk = __shfl(hits ? hit : end, from);
        run = __shfl(under, from);
        const Draw<T> d(p, r, n);
        double w[PER], own = 0.0;
        const int at = chunk * kChunk + lane * PER;
        typename Vec<T>::type tv[PER / E], qv[PER / E];
#pragma unroll
        for (int i = 0; i < PER / E; ++i) {
            tv[i] = load_some(d.p + at + i * E, p.vocab - at - i * E);
            qv[i] = {};
            if (d.q && left) qv[i] = load_some(d.q + at + i * E, p.vocab - at - i * E);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const double v = weight(tv[i / E][i % E]);
            w[i] = left ? d.rest(v, weight(qv[i / E][i % E]), at + i) : v;
            own += w[i];
        }
        run += before(own, lane, all);
        int first = -1, last = -1;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            run += w[i];
            if (w[i] > 0.0) {
                if (first < 0 && run > border) first = at + i;
                last = at + i;
            }
        }
        // sums of another order may end just below the border: then the chunk's last token
        const uint64_t firsts = __builtin_amdgcn_ballot_w64(first >= 0), lasts = __builtin_amdgcn_ballot_w64(last >= 0);
        token = hits && firsts ? __shfl(first, __builtin_ctzll(firsts)) : __shfl(last, 63 - __builtin_clzll(lasts));
    }
    for (int i = lane; i < r.count; i += 64)
        p.out[r.first + i] = i < n ? p.ids[r.first + i + 1] : i == n ? token : -1;
}

template <typename T> __global__ __launch_bounds__(kThreads) void verify_sums_kernel(Params p)
{
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int groups = (p.chunks + kThreads / 64 - 1) / (kThreads / 64);
    const int b = blockIdx.x / groups, chunk = blockIdx.x % groups * (kThreads / 64) + wave;
    const Rows r = rows_of(p, b);
    if (r.count == 0) return;
    const int n = uniform(accepted_of<T>(p, r, lane));
    if (chunk == 0 && lane == 0) p.accepted[b] = n;
    if (chunk >= p.chunks) return;
    const Draw<T> d(p, r, n);
    Chunk<T> c;
    c.load(p, d, chunk, lane);
    const d2_t sums = c.sums(d, chunk, lane);
    if (lane == 0) reinterpret_cast<d2_t*>(p.sums)[(int64_t)b * p.chunks + chunk] = sums;
}

template <typename T> __global__ __launch_bounds__(64) void verify_draw_kernel(Params p)
{
    const int b = blockIdx.x, lane = threadIdx.x;
    const Rows r = rows_of(p, b);
    if (r.count == 0) {
        if (lane == 0) p.accepted[b] = 0;
        return;
    }
    int n = p.accepted[b];
    n = n < 0 ? 0 : n >= r.count ? r.count - 1 : n;
    draw_token<T>(p, r, b, uniform(n), reinterpret_cast<const d2_t*>(p.sums) + (int64_t)b * p.chunks, lane);
}

// Both for small vocabularies: a workgroup a sequence, its sums in LDS.
template <typename T> __global__ __launch_bounds__(kOneThreads) void verify_one_kernel(Params p)
{
    __shared__ d2_t sums[kOneChunks];
    const int b = blockIdx.x, lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const Rows r = rows_of(p, b);
    if (r.count == 0) {
        if (threadIdx.x == 0) p.accepted[b] = 0;
        return;
    }
    const int n = uniform(accepted_of<T>(p, r, lane));
    const Draw<T> d(p, r, n);
    for (int chunk = wave; chunk < p.chunks; chunk += blockDim.x / 64) {
        Chunk<T> c;
        c.load(p, d, chunk, lane);
        const d2_t v = c.sums(d, chunk, lane);
        if (lane == 0) sums[chunk] = v;
    }
    __syncthreads();
    if (wave > 0) return;
    if (lane == 0) p.accepted[b] = n;
    draw_token<T>(p, r, b, n, sums, lane);
}

}  // namespace

}  // namespace verify

hipError_t launch_verify(const VerifyArgs& a, hipStream_t stream, const char** variant)
{
    verify::Params p;
    p.target = a.target;
    p.draft = a.draft;
    p.target_stride = a.target_stride;
    p.draft_stride = a.draft_stride;
    p.ids = a.ids;
    p.q_start = a.q_start;
    p.accept = a.accept;
    p.pick = a.pick;
    p.out = a.out;
    p.accepted = a.accepted;
    p.sums = static_cast<double*>(a.workspace);
    p.batch = (int)a.batch;
    p.tokens = (int)a.tokens;
    p.vocab = (int)a.vocab;
    p.chunks = (int)verify_chunks(a.vocab);
    const dim3 one((unsigned)a.batch);
    // One launch while a CU reads a sequence's row and draft quickly (one sequence in a graph, one launch and
    // two: 128 KB 5.9 and 6.6 us with 16 chunks, 6.5 and 6.5 with 32, where call by call an enqueue is spared; 256 KB
    // 8.2 and 7.1; 50 chunks 7.9 and 6.5 for 100 KB), or there are sequences for all CUs (256 of 50257 tokens,
    // fp16: 15 and 17; 512 certain ones of 128000: 27 and 34)
    const int64_t bytes = (int64_t)p.chunks * kVerifyChunk * (a.f16 ? 2 : 4) * (a.draft ? 2 : 1);
    if ((p.chunks <= 32 && bytes <= 128 * 1024) || (a.batch >= 256 && p.chunks <= verify::kOneChunks)) {
        *variant = "verify_one";
        // a wave a chunk at most, so the grid has 64 batch * chunks < 2^30 threads
        const int threads = 64 * p.chunks < verify::kOneThreads ? 64 * p.chunks : verify::kOneThreads;
        if (a.f16) verify::verify_one_kernel<_Float16><<<one, threads, 0, stream>>>(p);
        else verify::verify_one_kernel<float><<<one, threads, 0, stream>>>(p);
        return hipGetLastError();
    }
    *variant = "verify_drafts";
    const int64_t groups = (p.chunks + verify::kThreads / 64 - 1) / (verify::kThreads / 64);
    const dim3 grid((unsigned)(a.batch * groups)), block(verify::kThreads), wave(64);
    if (a.f16) verify::verify_sums_kernel<_Float16><<<grid, block, 0, stream>>>(p);
    else verify::verify_sums_kernel<float><<<grid, block, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.f16) verify::verify_draw_kernel<_Float16><<<one, wave, 0, stream>>>(p);
    else verify::verify_draw_kernel<float><<<one, wave, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace mnb
