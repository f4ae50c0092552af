// rms_norm.hip -- RMS norm of the residual stream, one pass over the row.
//
//   h = x + r (rounded to the type), y = h * (mean(h^2) + eps)^-1/2 * w,
//
// written as values, or as 8-bit codes with one scale per row in the
// convention of the int8-activation products: s = max|y| / 127, q = y / s
// rounded half away from zero.  The norm's factor cancels from the codes,
//   q = 127 h w / max|h w|,
// so the sum of squares and the maximum are found together, by one reduction
// of the workgroup, and the codes do not depend on how the sum was rounded.
// h * w is exact in fp32 for fp16 operands and in fp64 for fp32 ones; the quotient is formed
// in fp64 and is off by at most 2^-45 at 127, so a code is off only where the exact quotient is
// a tie to within that.
//
// Bound by memory for many rows, by one round trip and the launch for few.  Measured:
// 8192 rows of 4096 with a residual, fp16, 45.8 us for 268 MB (5.9 TB/s; a large copy moves
// 5.15), fp32 92 us; 1023 rows of 11008 to fp16 codes, fp32, 32.7 us for 158 MB (4.8 TB/s), to
// int8 codes 33 us for 146; 1 row 2.3 us, 16 rows to codes 3.4 us.
//
// One workgroup holds one row in registers: every input byte is requested
// before the reduction's barrier and read once.  Loads and stores are 16 bytes
// whatever the row's alignment (unaligned access is native here); the last
// K mod 8 (4) elements go one to a thread.
#include <type_traits>

#include "mnb_device.hpp"
#include "mnb_kv4.hpp"

namespace mnb {

namespace {

struct NormParams {
    const void* x;
    const void* residual;
    const void* weight;
    void* out;
    float* scales;
    void* residual_out;
    int64_t x_stride, residual_stride;
    int k;
    float eps;
    float inv_k;
};

// 16 bytes of T at any element alignment
template <typename T> struct Vec;
template <> struct Vec<_Float16> {
    static constexpr int N = 8;
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2), may_alias));
};
template <> struct Vec<float> {
    static constexpr int N = 4;
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(4), may_alias));
};

template <typename T> __device__ __forceinline__ void unpack_vec(const u4_t& r, float* f)
{
    if constexpr (sizeof(T) == 2) {
        const h8_t h = __builtin_bit_cast(h8_t, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)h[i];
    } else {
        const f4_t h = __builtin_bit_cast(f4_t, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = h[i];
    }
}

template <typename T> __device__ __forceinline__ u4_t pack_vec(const float* f)
{
    if constexpr (sizeof(T) == 2) {
        h8_t h;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = (_Float16)f[i];
        return __builtin_bit_cast(u4_t, h);
    } else {
        f4_t h;
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = f[i];
        return __builtin_bit_cast(u4_t, h);
    }
}

// the larger one, or NaN if either is
template <typename P> __device__ __forceinline__ P max_of(P a, P b) { return __builtin_elementwise_maximum(a, b); }

// round half away from zero of 127 hw / max, as factor = 127 / max in fp64: at
// most 127 in magnitude, since no |hw| is above the row's largest
__device__ __forceinline__ int code_of(double hw, double factor)
{
    const double t = hw * factor;
    return (int)(t + __builtin_copysign(0.5, t));
}

template <typename T, int OUT, int NV>
__global__ __launch_bounds__(1024) void rms_norm_kernel(NormParams p)
{
    constexpr int VE = Vec<T>::N;
    typedef typename Vec<T>::raw raw_t;
    typedef typename std::conditional<sizeof(T) == 2, float, double>::type prod_t;   // holds h w exactly
    __shared__ float red[16];
    __shared__ prod_t red_mx[16];

    const int tid = threadIdx.x, nt = blockDim.x;
    const int64_t row = blockIdx.x;
    const int K = p.k;
    const int nv = K / VE;            // whole vectors
    const int tail = K - nv * VE;     // elements past them, one to a thread
    const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
    const T* r = p.residual ? static_cast<const T*>(p.residual) + row * p.residual_stride : nullptr;
    const T* w = static_cast<const T*>(p.weight);
    T* ro = p.residual_out ? static_cast<T*>(p.residual_out) + row * (int64_t)K : nullptr;

    auto load = [](const T* base, int v) -> u4_t { return *reinterpret_cast<const raw_t*>(base + (int64_t)v * VE); };
    // h of vector v from the raw operands, rounded to T where a residual is added
    auto sum_vec = [&](const u4_t& xv, const u4_t& rv, float* h) {
        unpack_vec<T>(xv, h);
        if (r) {
            float f[VE];
            unpack_vec<T>(rv, f);
#pragma unroll
            for (int i = 0; i < VE; ++i) h[i] = (float)(T)(h[i] + f[i]);
        }
    };

    u4_t xv[NV], rv[NV], wv[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int v = tid + u * nt;
        if (v < nv) {
            xv[u] = load(x, v);
            if (r) rv[u] = load(r, v);
            wv[u] = load(w, v);
        }
    }
    float ss = 0.0f;
    prod_t mx = 0;                    // largest |h w|
    float th = 0.0f, tw = 0.0f;       // the thread's element past the vectors
    const int te = nv * VE + tid;
    if (tid < tail) {
        th = (float)x[te];
        if (r) th = (float)(T)(th + (float)r[te]);
        tw = (float)w[te];
        ss = th * th;
        mx = __builtin_elementwise_abs((prod_t)th * tw);
    }
    auto add_vec = [&](const float* h, const u4_t& wr) {
#pragma unroll
        for (int i = 0; i < VE; ++i) ss = __builtin_fmaf(h[i], h[i], ss);
        if constexpr (OUT != kNormValues) {
            float f[VE];
            unpack_vec<T>(wr, f);
#pragma unroll
            for (int i = 0; i < VE; ++i) mx = max_of(mx, __builtin_elementwise_abs((prod_t)h[i] * f[i]));
        }
    };
    // the sums replace x in its registers, rounded as they are stored
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        if (tid + u * nt < nv) {
            float h[VE];
            sum_vec(xv[u], rv[u], h);
            xv[u] = pack_vec<T>(h);
            add_vec(h, wv[u]);
        }
    }
    // rows longer than the registers: read again below
    for (int v = tid + NV * nt; v < nv; v += nt) {
        float h[VE];
        sum_vec(load(x, v), r ? load(r, v) : u4_t{0, 0, 0, 0}, h);
        add_vec(h, load(w, v));
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        ss += __shfl_xor(ss, off);
        if constexpr (OUT != kNormValues) mx = max_of(mx, __shfl_xor(mx, off));
    }
    const int waves = nt >> 6;
    if (waves > 1) {
        if ((tid & 63) == 0) {
            red[tid >> 6] = ss;
            red_mx[tid >> 6] = mx;
        }
        __syncthreads();
        ss = 0.0f;
        mx = 0;
        for (int i = 0; i < waves; ++i) {
            ss += red[i];
            mx = max_of(mx, red_mx[i]);
        }
    }
    float var = __builtin_fmaf(ss, p.inv_k, p.eps), pre = 1.0f;
    if constexpr (sizeof(T) == 4) {
        // squares past either end of binary32 are summed again from elements scaled by a power of
        // two (the same choice in every thread: they hold the same sum)
        if (uniform(!(var <= 0x1p127f) || var < 0x1p-100f)) {
            pre = var < 1.0f ? 0x1p90f : 0x1p-90f;
            ss = tid < tail ? th * pre * (th * pre) : 0.0f;
            auto add = [&](const float* h) {
#pragma unroll
                for (int i = 0; i < VE; ++i) ss = __builtin_fmaf(h[i] * pre, h[i] * pre, ss);
            };
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                if (tid + u * nt < nv) {
                    float h[VE];
                    unpack_vec<T>(xv[u], h);
                    add(h);
                }
            }
            for (int v = tid + NV * nt; v < nv; v += nt) {
                float h[VE];
                sum_vec(load(x, v), r ? load(r, v) : u4_t{0, 0, 0, 0}, h);
                add(h);
            }
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) ss += __shfl_xor(ss, off);
            __shared__ float again[16];
            if ((tid & 63) == 0) again[tid >> 6] = ss;
            __syncthreads();
            ss = 0.0f;
            for (int i = 0; i < waves; ++i) ss += again[i];
            var = __builtin_fmaf(ss, p.inv_k, p.eps * pre * pre);
        }
    }
    const float rs = 1.0f / sqrtf(var);            // of pre h
    // no NaN and no infinity among the row's products (mx holds either)
    const bool fine = uniform(mx < (prod_t)__builtin_inff());
    const double factor = OUT != kNormValues && mx > 0 ? 127.0 / (double)mx : 0.0;

    auto store_vec = [&](int v, const float* h, const u4_t& wr) {
        if (ro) *reinterpret_cast<raw_t*>(ro + (int64_t)v * VE) = pack_vec<T>(h);
        float f[VE];
        unpack_vec<T>(wr, f);
        const int64_t e = row * K + (int64_t)v * VE;
        if constexpr (OUT == kNormValues) {
#pragma unroll
            for (int i = 0; i < VE; ++i) f[i] = h[i] * pre * rs * f[i];
            *reinterpret_cast<raw_t*>(static_cast<T*>(p.out) + e) = pack_vec<T>(f);
        } else {
            int q[VE];
#pragma unroll
            for (int i = 0; i < VE; ++i) q[i] = 0;
            if (fine) {
#pragma unroll
                for (int i = 0; i < VE; ++i) q[i] = code_of((prod_t)h[i] * f[i], factor);
            }
            if constexpr (OUT == kNormCodesF16) {
                typedef uint32_t out_t __attribute__((ext_vector_type(VE / 2), aligned(2), may_alias));
                out_t o;
#pragma unroll
                for (int i = 0; i < VE / 2; ++i)
                    o[i] = as_u32(h2_t{(_Float16)(float)q[2 * i], (_Float16)(float)q[2 * i + 1]});
                *reinterpret_cast<out_t*>(static_cast<_Float16*>(p.out) + e) = o;
            } else {
                typedef uint32_t out_t __attribute__((ext_vector_type(VE / 4), aligned(1), may_alias));
                out_t o;
#pragma unroll
                for (int i = 0; i < VE / 4; ++i)
                    o[i] = (uint32_t)(q[4 * i] & 255) | ((uint32_t)(q[4 * i + 1] & 255) << 8) |
                           ((uint32_t)(q[4 * i + 2] & 255) << 16) | ((uint32_t)q[4 * i + 3] << 24);
                *reinterpret_cast<out_t*>(static_cast<int8_t*>(p.out) + e) = o;
            }
        }
    };
    // the vectors past the registers first: they are read again, and residual_out
    // may be x or residual itself (a thread rewrites only what it has read)
    for (int v = tid + NV * nt; v < nv; v += nt) {
        float h[VE];
        sum_vec(load(x, v), r ? load(r, v) : u4_t{0, 0, 0, 0}, h);
        store_vec(v, h, load(w, v));
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const int v = tid + u * nt;
        if (v < nv) {
            float h[VE];
            unpack_vec<T>(xv[u], h);
            store_vec(v, h, wv[u]);
        }
    }
    if (tid < tail) {
        if (ro) ro[te] = (T)th;
        const int64_t e = row * K + te;
        if constexpr (OUT == kNormValues)
            static_cast<T*>(p.out)[e] = (T)(th * pre * rs * tw);
        else if constexpr (OUT == kNormCodesF16)
            static_cast<_Float16*>(p.out)[e] = (_Float16)(float)(fine ? code_of((prod_t)th * tw, factor) : 0);
        else
            static_cast<int8_t*>(p.out)[e] = (int8_t)(fine ? code_of((prod_t)th * tw, factor) : 0);
    }
    if (OUT != kNormValues && tid == 0)
        p.scales[row] = mx == 0 ? 0.0f : fine ? (float)(mx * pre * rs / 127) : __builtin_nanf("");
}

template <typename T, int OUT>
hipError_t launch_out(const NormArgs& a, NormParams p, hipStream_t s)
{
    // 16 bytes a thread of up to 512, of longer rows two or four times that; the registers
    // of four hold 16384 fp16 or 8192 fp32 elements, and what is left is read twice
    const int64_t nv = a.k / Vec<T>::N;
    const int threads = (int)(nv < 64 ? 64 : nv > 512 ? 512 : (nv + 63) / 64 * 64);
    constexpr int64_t kRows = 1 << 22;     // of a launch: a grid holds less than 2^32 threads
    const int64_t out_elem = OUT == kNormValues ? (int64_t)sizeof(T) : OUT == kNormCodesF16 ? 2 : 1;
    for (int64_t r0 = 0; r0 < a.m; r0 += kRows) {
        const dim3 grid((unsigned)(a.m - r0 < kRows ? a.m - r0 : kRows));
        if (nv <= 512)
            rms_norm_kernel<T, OUT, 1><<<grid, dim3(threads), 0, s>>>(p);
        else if (nv <= 1024)
            rms_norm_kernel<T, OUT, 2><<<grid, dim3(threads), 0, s>>>(p);
        else
            rms_norm_kernel<T, OUT, 4><<<grid, dim3(threads), 0, s>>>(p);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        p.x = static_cast<const T*>(p.x) + kRows * p.x_stride;
        if (p.residual) p.residual = static_cast<const T*>(p.residual) + kRows * p.residual_stride;
        if (p.residual_out) p.residual_out = static_cast<T*>(p.residual_out) + kRows * a.k;
        p.out = static_cast<unsigned char*>(p.out) + kRows * a.k * out_elem;
        if (p.scales) p.scales += kRows;
    }
    return hipSuccess;
}

template <typename T> hipError_t launch_type(const NormArgs& a, const NormParams& p, hipStream_t s)
{
    switch (a.out_kind) {
    case kNormValues: return launch_out<T, kNormValues>(a, p, s);
    case kNormCodesF16: return launch_out<T, kNormCodesF16>(a, p, s);
    default: return launch_out<T, kNormCodesI8>(a, p, s);
    }
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t stream, const char** variant)
{
    NormParams p;
    p.x = a.x;
    p.residual = a.residual;
    p.weight = a.weight;
    p.out = a.out;
    p.scales = a.scales;
    p.residual_out = a.residual_out;
    p.x_stride = a.x_stride;
    p.residual_stride = a.residual_stride;
    p.k = (int)a.k;
    p.eps = a.eps;
    p.inv_k = (float)(1.0 / (double)a.k);
    *variant = a.out_kind == kNormValues ? "rms_norm" : a.out_kind == kNormCodesF16 ? "rms_norm_codes_f16" : "rms_norm_codes_i8";
    return a.f16 ? launch_type<_Float16>(a, p, stream) : launch_type<float>(a, p, stream);
}

}  // namespace mnb
