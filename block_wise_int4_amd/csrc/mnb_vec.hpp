// mnb_vec.hpp -- 16-byte pieces of fp16 or fp32 rows that start at any element.
#pragma once

#include "mnb_device.hpp"

namespace mnb {

// 16 bytes of a row: 8 fp16 or 4 fp32 values, at any element.
template <typename T> struct Vec;
template <> struct Vec<_Float16> {
    static constexpr int E = 8;
    typedef h8_t type;
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(2), may_alias));
};
template <> struct Vec<float> {
    static constexpr int E = 4;
    typedef f4_t type;
    typedef uint32_t raw __attribute__((ext_vector_type(4), aligned(4), may_alias));
};
template <typename T> __device__ __forceinline__ typename Vec<T>::type load(const T* p)
{
    return __builtin_bit_cast(typename Vec<T>::type, (u4_t)*reinterpret_cast<const typename Vec<T>::raw*>(p));
}
template <typename T> __device__ __forceinline__ void store(T* p, const typename Vec<T>::type& v)
{
    *reinterpret_cast<typename Vec<T>::raw*>(p) = __builtin_bit_cast(u4_t, v);
}
// The same of memory that no one reads again soon: nothing is kept in the caches.
template <typename T> __device__ __forceinline__ typename Vec<T>::type load_once(const T* p)
{
    return __builtin_bit_cast(typename Vec<T>::type,
                              (u4_t)__builtin_nontemporal_load(reinterpret_cast<const typename Vec<T>::raw*>(p)));
}
template <typename T> __device__ __forceinline__ void store_through(T* p, const typename Vec<T>::type& v)
{
    __builtin_nontemporal_store((typename Vec<T>::raw)__builtin_bit_cast(u4_t, v),
                                reinterpret_cast<typename Vec<T>::raw*>(p));
}
// The first `valid` of them, zeros behind.
template <typename T> __device__ __forceinline__ typename Vec<T>::type load_some(const T* p, int64_t valid)
{
    typename Vec<T>::type v;
    if (valid >= Vec<T>::E) return load(p);
#pragma unroll
    for (int i = 0; i < Vec<T>::E; ++i) v[i] = i < valid ? p[i] : (T)0.0f;
    return v;
}

}  // namespace mnb
