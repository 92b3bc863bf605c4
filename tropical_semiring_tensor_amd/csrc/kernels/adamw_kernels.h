// AdamW over many tensors in one launch.
//
// Per element a dozen operations on 28 bytes (32-bit state) or 16 (8-bit
// state): bound by HBM.  A launch's argument block lists up to 72 (56)
// tensors with the running count of their 4096-element chunks; a workgroup
// takes one chunk and finds its tensor by bisection over those counts
// (scalar loads of the argument block), so small and large tensors fill the
// device together.  316 million elements in 96 tensors: bfloat16 with master
// weights 1.58 ms (28 bytes an element, 5.6 TB/s), float32 with 8-bit states
// 1.10 ms (16 bytes, 4.6 TB/s) and their unpacking 0.68 (10 bytes, 4.7 TB/s); a
// large copy reaches 4.7.  25 float32 tensors of 65536 elements and fewer: 6.5
// us.  All arithmetic is one IEEE float32 operation at a time,
// in the order the header states.
#pragma once
#include <type_traits>

#include "train_common.h"

namespace trop {

template <typename PARAMS>
__device__ __forceinline__ int find_tensor(const PARAMS& p, uint32_t chunk) {
    int lo = 0, hi = p.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (chunk < p.chunk_end[mid])
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ void adamw_element(const TropAdamwScalars& s, float g, float& m, float& v, float& q) {
    m = m * s.beta1 + g * s.one_minus_beta1;
    v = v * s.beta2 + (g * g) * s.one_minus_beta2;
    q = q * s.keep - (m / (sqrtf(v) * s.root + s.eps)) * s.step_size;
}

// MASTER: q is the float32 master weight, param only receives its rounding.
template <typename T, bool MASTER>
__device__ __forceinline__ void adamw_body(const TropAdamwParams& p) {
    const int ti = find_tensor(p, blockIdx.x);
    const TropAdamwEntry& e = p.t[ti];
    const int64_t base = (int64_t)(blockIdx.x - (ti ? p.chunk_end[ti - 1] : 0u)) * TROP_ADAMW_CHUNK;
    constexpr int U = TROP_ADAMW_CHUNK / (256 * 4);
    FloatVec<4> q[U], m[U], v[U];
    typename VecOf<T, 4>::raw g[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = base + (u * 256 + threadIdx.x) * 4;
        g[u] = load_row_stream<T, 4>(static_cast<const T*>(e.grad), c, e.n);
        m[u] = load_row_stream<float, 4>(e.m, c, e.n);
        v[u] = load_row_stream<float, 4>(e.v, c, e.n);
        if constexpr (MASTER)
            q[u] = load_row_stream<float, 4>(e.master, c, e.n);
        else
            q[u] = to_float<T, 4>(load_row_stream<T, 4>(static_cast<const T*>(e.param), c, e.n));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = base + (u * 256 + threadIdx.x) * 4;
        const FloatVec<4> gf = to_float<T, 4>(g[u]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mm = m[u][i], vv = v[u][i], qq = q[u][i];
            adamw_element(p.s, gf[i], mm, vv, qq);
            m[u][i] = mm;
            v[u][i] = vv;
            q[u][i] = qq;
        }
        if (c < e.n) {
            store_row_stream<float, 4>(e.m, c, e.n, m[u]);
            store_row_stream<float, 4>(e.v, c, e.n, v[u]);
            if constexpr (MASTER) store_row_stream<float, 4>(e.master, c, e.n, q[u]);
            store_row_stream<T, 4>(static_cast<T*>(e.param), c, e.n, from_float<T, 4>(q[u]));
        }
    }
}

// Values of the 8-bit codes (t4: (c / 255)^4 by two squarings).
__device__ __forceinline__ float adamw8_m(float code, float a) {
    const float t = code * (1.0f / 127.0f);
    return (a * t) * fabsf(t);
}
__device__ __forceinline__ float adamw8_v(float code, float a) {
    const float t = code * (1.0f / 255.0f), t2 = t * t;
    return a * (t2 * t2);
}
// Codes of m and v in a block of scale a (0: every element is zero).  A block
// that holds a NaN or an infinity has a NaN scale, whatever its codes: an
// infinite one would stand for infinities where they are not zero.
__device__ __forceinline__ float adamw8_round_m(float m, float a) {
    return rintf(sqrtf(fabsf(m) / a) * 127.0f);
}
__device__ __forceinline__ float adamw8_round_v(float v, float a) {
    return rintf(sqrtf(sqrtf(v / a)) * 255.0f);
}
// The same through the reciprocal of a and the hardware root (1 ulp): the
// number that is rounded is off by 8 2^-24 of itself at most, below 1.3e-4.
// `sure` is cleared where a rounding boundary is within 2e-4, or nothing can
// be said (infinities, NaN).
__device__ __forceinline__ float adamw8_guess(float x, bool& sure) {
    const float c = rintf(x);
    sure &= fabsf(x - c) < 0.4998f;
    return c;
}
__device__ __forceinline__ int adamw8_code_m(float c, float m) {
    const int k = c <= 127.f ? (int)c : 0;
    return m < 0.f ? -k : k;
}
__device__ __forceinline__ int adamw8_code_v(float c, float v) {
    const int k = c <= 255.f ? (int)c : 0;
    return v > 0.f ? (k > 1 ? k : 1) : 0;
}

// One wave per block of 256 elements, four a lane: the block's scale is a
// wave reduction, no LDS.  Bound by the vector units before HBM when every
// code took its own division and roots (some 150 operations an element, 1.41
// ms for 316 million float32 elements); the guess leaves them to the one
// wave in twenty that holds an element next to a rounding boundary.
template <typename T, bool MASTER>
__device__ __forceinline__ void adamw8_body(const TropAdamw8Params& p) {
    const int ti = find_tensor(p, blockIdx.x);
    const TropAdamw8Entry& e = p.t[ti];
    const int64_t base = (int64_t)(blockIdx.x - (ti ? p.chunk_end[ti - 1] : 0u)) * TROP_ADAMW_CHUNK;
    constexpr int U = TROP_ADAMW_CHUNK / (256 * 4);
    FloatVec<4> q[U];
    typename VecOf<T, 4>::raw g[U];
    typename VecOf<int8_t, 4>::raw mc[U];
    typename VecOf<uint8_t, 4>::raw vc[U];
    float ma[U], va[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = base + (u * 256 + threadIdx.x) * 4;
        g[u] = load_row_stream<T, 4>(static_cast<const T*>(e.grad), c, e.n);
        mc[u] = load_row_stream<int8_t, 4>(e.m, c, e.n);
        vc[u] = load_row_stream<uint8_t, 4>(e.v, c, e.n);
        ma[u] = c < e.n ? e.m_scale[c / TROP_ADAMW_BLOCK_ELEMS] : 0.f;
        va[u] = c < e.n ? e.v_scale[c / TROP_ADAMW_BLOCK_ELEMS] : 0.f;
        if constexpr (MASTER)
            q[u] = load_row_stream<float, 4>(e.master, c, e.n);
        else
            q[u] = to_float<T, 4>(load_row_stream<T, 4>(static_cast<const T*>(e.param), c, e.n));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = base + (u * 256 + threadIdx.x) * 4;
        const FloatVec<4> gf = to_float<T, 4>(g[u]);
        float m[4], v[4];
        uint32_t am_bits = 0, av_bits = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = adamw8_m((float)mc[u][i], ma[u]);
            v[i] = adamw8_v((float)vc[u][i], va[u]);
            float qq = q[u][i];
            adamw_element(p.s, gf[i], m[i], v[i], qq);
            q[u][i] = qq;
            if (c + i >= e.n) m[i] = v[i] = 0.f;
            am_bits = max(am_bits, __builtin_bit_cast(uint32_t, m[i]) & 0x7fffffffu);
            av_bits = max(av_bits, __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);
        }
        float am = __builtin_bit_cast(float, wave_umax(am_bits));
        float av = __builtin_bit_cast(float, wave_umax(av_bits));
        am = am < INFINITY ? am : NAN;
        av = av < INFINITY ? av : NAN;
        const float dm = am > 0.f ? am : 1.f, dv = av > 0.f ? av : 1.f;
        const float rm = 1.0f / dm, rv = 1.0f / dv;
        float cm[4], cv[4];
        bool sure = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            cm[i] = adamw8_guess(__builtin_amdgcn_sqrtf(fabsf(m[i]) * rm) * 127.0f, sure);
            cv[i] = adamw8_guess(__builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf(v[i] * rv)) * 255.0f, sure);
        }
        if (__any(!sure)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                cm[i] = adamw8_round_m(m[i], dm);
                cv[i] = adamw8_round_v(v[i], dv);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mc[u][i] = (int8_t)adamw8_code_m(cm[i], m[i]);
            vc[u][i] = (uint8_t)adamw8_code_v(cv[i], v[i]);
        }
        if (c < e.n) {
            store_row_stream<int8_t, 4>(e.m, c, e.n, mc[u]);
            store_row_stream<uint8_t, 4>(e.v, c, e.n, vc[u]);
            if ((threadIdx.x & 63) == 0) {
                e.m_scale[c / TROP_ADAMW_BLOCK_ELEMS] = am;
                e.v_scale[c / TROP_ADAMW_BLOCK_ELEMS] = av;
            }
            if constexpr (MASTER) store_row_stream<float, 4>(e.master, c, e.n, q[u]);
            store_row_stream<T, 4>(static_cast<T*>(e.param), c, e.n, from_float<T, 4>(q[u]));
        }
    }
}

// The codes' values: m into `param`, v into `master` (either may be null).
__device__ __forceinline__ void adamw8_unpack_body(const TropAdamw8Params& p) {
    const int ti = find_tensor(p, blockIdx.x);
    const TropAdamw8Entry& e = p.t[ti];
    const int64_t base = (int64_t)(blockIdx.x - (ti ? p.chunk_end[ti - 1] : 0u)) * TROP_ADAMW_CHUNK;
    constexpr int U = TROP_ADAMW_CHUNK / (256 * 4);
    auto unpack = [&](const auto* codes, const float* scales, float* out, auto value) {
        using K = std::remove_cv_t<std::remove_pointer_t<decltype(codes)>>;
        typename VecOf<K, 4>::raw k[U];
        float a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = base + (u * 256 + threadIdx.x) * 4;
            k[u] = load_row_stream<K, 4>(codes, c, e.n);
            a[u] = c < e.n ? scales[c / TROP_ADAMW_BLOCK_ELEMS] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t c = base + (u * 256 + threadIdx.x) * 4;
            FloatVec<4> o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = value((float)k[u][i], a[u]);
            if (c < e.n) store_row_stream<float, 4>(out, c, e.n, o);
        }
    };
    if (e.param)
        unpack(e.m, e.m_scale, static_cast<float*>(e.param), [](float k, float a) { return adamw8_m(k, a); });
    if (e.master) unpack(e.v, e.v_scale, e.master, [](float k, float a) { return adamw8_v(k, a); });
}

}  // namespace trop
