// Types and wave reductions shared by the training operators' kernels.
#pragma once
#include <hip/hip_runtime.h>

#include "../train_params.h"

namespace trop {

using bf16 = __bf16;

// N consecutive elements at any element-aligned address.  The target's
// unaligned access mode serves these as single wide accesses, so one path
// covers every row stride and offset.
template <typename T, int N>
struct VecOf {
    typedef T raw __attribute__((ext_vector_type(N)));
    typedef raw type __attribute__((aligned(sizeof(T))));
};
template <int N>
using FloatVec = typename VecOf<float, N>::raw;

template <typename T, int N>
__device__ __forceinline__ typename VecOf<T, N>::raw load_vec(const T* p) {
    return *reinterpret_cast<const typename VecOf<T, N>::type*>(p);
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, typename VecOf<T, N>::raw v) {
    *reinterpret_cast<typename VecOf<T, N>::type*>(p) = v;
}
// The same for data that is read or written once: past the caches' reuse
// order (a 2 GiB read: 7.2 TB/s against 6.0).
template <typename T, int N>
__device__ __forceinline__ typename VecOf<T, N>::raw load_stream(const T* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const typename VecOf<T, N>::type*>(p));
}
template <typename T, int N>
__device__ __forceinline__ void store_stream(T* p, typename VecOf<T, N>::raw v) {
    __builtin_nontemporal_store(v, reinterpret_cast<typename VecOf<T, N>::type*>(p));
}
template <typename T, int N>
__device__ __forceinline__ FloatVec<N> to_float(typename VecOf<T, N>::raw v) {
    return __builtin_convertvector(v, FloatVec<N>);
}
template <typename T, int N>
__device__ __forceinline__ typename VecOf<T, N>::raw from_float(FloatVec<N> v) {
    return __builtin_convertvector(v, typename VecOf<T, N>::raw);
}

// Elements [c, c + N) of a row of n elements, zeros past its end.
template <typename T, int N>
__device__ __forceinline__ typename VecOf<T, N>::raw load_row(const T* row, int64_t c, int64_t n) {
    if (c + N <= n) return load_vec<T, N>(row + c);
    typename VecOf<T, N>::raw v = {};
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (c + e < n) v[e] = row[c + e];
    return v;
}
template <typename T, int N>
__device__ __forceinline__ typename VecOf<T, N>::raw load_row_stream(const T* row, int64_t c, int64_t n) {
    return c + N <= n ? load_stream<T, N>(row + c) : load_row<T, N>(row, c, n);
}
template <typename T, int N>
__device__ __forceinline__ void store_row(T* row, int64_t c, int64_t n, typename VecOf<T, N>::raw v) {
    if (c + N <= n) {
        store_vec<T, N>(row + c, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (c + e < n) row[c + e] = v[e];
}

template <typename T, int N>
__device__ __forceinline__ void store_row_stream(T* row, int64_t c, int64_t n, typename VecOf<T, N>::raw v) {
    if (c + N <= n)
        store_stream<T, N>(row + c, v);
    else
        store_row<T, N>(row, c, n, v);
}

// Maximum of the wave's 32-bit patterns as unsigned integers: for magnitudes
// (sign bit clear) the largest float, a NaN above infinity.  Six DPP steps
// (rows of 16 by shifts, then across rows); lane 63 ends with the result.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t x) {
    const uint32_t o = __builtin_amdgcn_update_dpp(0, x, CTRL, 0xf, 0xf, true);
    return o > x ? o : x;
}
// (lane 15 of each row of 16 ends with its row's)
__device__ __forceinline__ uint32_t row_umax(uint32_t x) {
    x = dpp_umax<0x111>(x);  // row_shr:1
    x = dpp_umax<0x112>(x);  // row_shr:2
    x = dpp_umax<0x114>(x);  // row_shr:4
    return dpp_umax<0x118>(x);  // row_shr:8
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t x) {
    x = row_umax(x);
    x = dpp_umax<0x142>(x);  // row_bcast:15
    x = dpp_umax<0x143>(x);  // row_bcast:31
    return __builtin_amdgcn_readlane(x, 63);
}

// Butterfly reductions: every lane ends with the wave's result, the same
// order of operations in every lane pair, so all lanes hold the same bits.
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
    return x;
}
// Maximum that keeps a NaN (fmaxf would drop it).
__device__ __forceinline__ float nan_max(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float wave_nan_max(float x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x = nan_max(x, __shfl_xor(x, o, 64));
    return x;
}

}  // namespace trop
