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
// Two kernels: sums of chunks of the one row that the draw needs (every workgroup
// finds that row for itself), then per sequence the chunk and in it the token.
#include "mnb_requests.hpp"
#include "mnb_vec.hpp"

namespace mnb {
namespace verify {

constexpr int kThreads = 256, kChunk = kVerifyChunk;

namespace {

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
    return f > 0.0f && f < __builtin_inff() ? (double)f : 0.0;
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
        return i == gone ? 0.0 : w > v ? w - v : 0.0;
    }
};

__device__ __forceinline__ double wave_sum(double x)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
    return x;
}

// Sums of a wave's lanes before this one, and of all.
__device__ __forceinline__ double before(double x, int lane, double& total)
{
    double upto = x;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const double y = __shfl_up(upto, off);
        if (lane >= off) upto += y;
    }
    total = __shfl(upto, 63);
    const double own = __shfl_up(upto, 1);
    return lane > 0 ? own : 0.0;
}

template <typename T> __global__ __launch_bounds__(kThreads) void verify_sums_kernel(Params p)
{
    constexpr int E = Vec<T>::E, PIECES = kChunk / 64 / E;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int groups = (p.chunks + kThreads / 64 - 1) / (kThreads / 64);
    const int b = blockIdx.x / groups, chunk = blockIdx.x % groups * (kThreads / 64) + wave;
    const Rows r = rows_of(p, b);
    if (r.count == 0) return;
    const int n = uniform(accepted_of<T>(p, r, lane));
    if (chunk == 0 && lane == 0) p.accepted[b] = n;
    if (chunk >= p.chunks) return;
    const Draw<T> d(p, r, n);
    double rest = 0.0, all = 0.0;
    typename Vec<T>::type tv[PIECES], qv[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int at = chunk * kChunk + (i * 64 + lane) * E;
        tv[i] = load_some(d.p + at, p.vocab - at);
        qv[i] = {};
        if (d.q) qv[i] = load_some(d.q + at, p.vocab - at);
    }
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
        const int at = chunk * kChunk + (i * 64 + lane) * E;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const double w = weight(tv[i][e]);
            all += w;
            rest += d.rest(w, weight(qv[i][e]), at + e);
        }
    }
    all = wave_sum(all);
    rest = wave_sum(rest);
    if (lane == 0) {
        double* out = p.sums + ((int64_t)b * p.chunks + chunk) * 2;
        out[0] = rest;
        out[1] = all;
    }
}

// One wave: the chunk whose sums pass the border, then the token in it.  A lane holds
// neighbouring chunks, then neighbouring tokens.
template <typename T> __global__ __launch_bounds__(64) void verify_draw_kernel(Params p)
{
    constexpr int E = Vec<T>::E, PER = kChunk / 64;
    typedef double d2_t __attribute__((ext_vector_type(2)));
    const int b = blockIdx.x, lane = threadIdx.x;
    const Rows r = rows_of(p, b);
    if (r.count == 0) {
        if (lane == 0) p.accepted[b] = 0;
        return;
    }
    int n = p.accepted[b];
    n = n < 0 ? 0 : n >= r.count ? r.count - 1 : n;
    n = uniform(n);
    const d2_t* sums = reinterpret_cast<const d2_t*>(p.sums) + (int64_t)b * p.chunks;
    const int per = (p.chunks + 63) / 64, c0 = lane * per, c1 = c0 + per < p.chunks ? c0 + per : p.chunks;
    d2_t mine = {0.0, 0.0};
#pragma unroll 4
    for (int c = c0; c < c1; ++c) mine += sums[c];
    double rest, all;
    const double rest_before = before(mine[0], lane, rest), all_before = before(mine[1], lane, all);
    // nothing is left of p where q is no smaller anywhere: then p itself
    const bool left = n < r.count - 1 && rest > 0.0;
    const float u = p.pick[b];
    const double border = (u > 0.0f ? (double)u : 0.0) * (left ? rest : all);
    // the first chunk that passes the border; pick of 1 or more passes all: the last with a weight
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
    *variant = "verify_drafts";
    const int64_t groups = (p.chunks + verify::kThreads / 64 - 1) / (verify::kThreads / 64);
    const dim3 grid((unsigned)(a.batch * groups)), block(verify::kThreads), one((unsigned)a.batch), wave(64);
    if (a.f16) verify::verify_sums_kernel<_Float16><<<grid, block, 0, stream>>>(p);
    else verify::verify_sums_kernel<float><<<grid, block, 0, stream>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.f16) verify::verify_draw_kernel<_Float16><<<one, wave, 0, stream>>>(p);
    else verify::verify_draw_kernel<float><<<one, wave, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace mnb
