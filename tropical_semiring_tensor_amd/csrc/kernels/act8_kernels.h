// Activations in 8 bits: rows packed to int8 codes with a power of two for
// each 32 elements, and unpacked.
//
//   a = max |x| of the block, e = floor(log2 a) - 6 + 127, one more where a
//   mantissa of 127.5 / 64 or more would round to 128, at least 1
//   c = rint(x 2^(127 - e)),  value c 2^(e - 127)
//
// (e is at most 248: magnitudes above 127 2^121 are taken as that.)
//
// A power of two as the block's step costs up to one of the 7 bits against a
// step of a / 127, and makes a value exact in bfloat16: the code's 7 bits and
// sign.  So unpacking rounds nothing, a matrix instruction takes the values as
// they are, and products with them are exact in float32.  32 elements to a
// step (a 32nd byte each) win back what the power of two costs.
//
// Bound by HBM: 16384 x 4096 bfloat16 (203 MB each way) packed in 33 us and
// unpacked in 31, 6.1 and 6.6 TB/s; 33 x 1000: 4 us each, latency.
#pragma once
#include "train_common.h"

namespace trop {

// The exponent for a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t act8_exponent(uint32_t bits) {
    if (bits >= 0x7f800000u) return 255;
    const int32_t e = (int32_t)((bits + 0x10000u) >> 23) - 6;  // (127.5 / 64 is mantissa 0x7f0000)
    return e < 1 ? 1 : e;
}
__device__ __forceinline__ float act8_step(uint32_t e) { return __builtin_bit_cast(float, e << 23); }

// Largest over the lanes that hold a block: 4 of 8 elements or 8 of 4.
template <int LANES>
__device__ __forceinline__ uint32_t act8_block_max(uint32_t m) {
    static_assert(LANES == 4 || LANES == 8, "lanes of a block");
    m = dpp_umax<0xb1>(m);  // quad_perm [1, 0, 3, 2]
    m = dpp_umax<0x4e>(m);  // quad_perm [2, 3, 0, 1]
    if constexpr (LANES == 8) m = dpp_umax<0x141>(m);  // row_half_mirror
    return m;
}

template <int VEC>
using Codes = typename VecOf<int8_t, VEC>::raw;

// Codes of a lane's VEC elements of a block and the block's exponent e.  All
// lanes of the block take part.
template <int VEC>
__device__ __forceinline__ Codes<VEC> act8_codes(FloatVec<VEC> v, uint32_t& e) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float x = v[i];  // (a bit cast of a vector's element itself takes element 0)
        const uint32_t b = __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
        m = b > m ? b : m;
    }
    e = act8_exponent(act8_block_max<TROP_ACT8_BLOCK_ELEMS / VEC>(m));
    if (__builtin_expect(e == 249, 0)) {  // 64 steps of 2^122 would be infinity
        e = 248;
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = fminf(fmaxf(v[i], -0x1.fcp+127f), 0x1.fcp+127f);
    }
    const float inv = __builtin_bit_cast(float, (254u - e) << 23);
    Codes<VEC> c;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        // the sum's last bit is worth 1: its low byte is rint(x inv)
        const uint32_t q = __builtin_bit_cast(uint32_t, __builtin_fmaf(v[i], inv, 12582912.0f));
        c[i] = e == 255 ? 0 : (int8_t)q;
    }
    return c;
}

// The same, stored: elements [c, c + VEC) of a row of n (c a multiple of VEC,
// lane 0 of the wave at the start of a block; elements past n are zero).
template <int VEC>
__device__ __forceinline__ void act8_store(int8_t* codes, uint8_t* exps, int64_t c, int64_t n, FloatVec<VEC> v) {
    uint32_t e;
    const Codes<VEC> q = act8_codes<VEC>(v, e);
    if (c < n) {
        store_row<int8_t, VEC>(codes, c, n, q);
        if (c % TROP_ACT8_BLOCK_ELEMS == 0) exps[c / TROP_ACT8_BLOCK_ELEMS] = (uint8_t)e;
    }
}

// Codes as 32-bit words, for a kernel to keep (as bytes each would take a
// register of its own).
template <int VEC>
using CodeWords = typename VecOf<uint32_t, VEC / 4>::raw;

// A lane's codes and exponent, to be turned into values later.
template <int VEC>
struct Act8Lane {
    Codes<VEC> codes;
    uint32_t e;
    __device__ __forceinline__ void load(const int8_t* codes_row, const uint8_t* exps_row, int64_t c, int64_t n) {
        codes = load_row_stream<int8_t, VEC>(codes_row, c, n);
        e = c < n ? exps_row[c / TROP_ACT8_BLOCK_ELEMS] : 1;
    }
    __device__ __forceinline__ FloatVec<VEC> values() const {
        const float step = act8_step(e);
        FloatVec<VEC> v = __builtin_convertvector(codes, FloatVec<VEC>);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] *= step;  // (e = 255: infinity times 0)
        return v;
    }
};

// Row and column of a chunk.
__device__ __forceinline__ void act8_chunk(const TropAct8Params& p, int64_t id, int64_t& row, int64_t& c) {
    if (p.rows_x == 1) {
        row = 0;
    } else if (((id | p.chunks) >> 32) == 0) {
        row = (uint32_t)id / (uint32_t)p.chunks;
    } else {
        row = id / p.chunks;
    }
    c = (id - row * p.chunks) * TROP_ACT8_CHUNK;
}
__device__ __forceinline__ int64_t act8_wave_id(int64_t group) {
    return group * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
}

// A wave takes a chunk of a row: 16 elements to a lane, in 16-byte vectors.
template <typename T>
__device__ __forceinline__ void act8_pack_body(const TropAct8Params& p) {
    constexpr int VEC = 16 / sizeof(T), NV = 16 / VEC;
    const int lane = threadIdx.x & 63;
    const int64_t id = act8_wave_id(blockIdx.x) + p.chunk0;
    if (id >= p.total) return;
    int64_t row, c0;
    act8_chunk(p, id, row, c0);
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    typename VecOf<T, VEC>::raw v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = load_row_stream<T, VEC>(x, c0 + (i * 64 + lane) * VEC, p.cols);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        act8_store<VEC>(p.codes + row * p.ldc, p.exps + row * p.lde, c0 + (i * 64 + lane) * VEC, p.cols,
                        to_float<T, VEC>(v[i]));
}

// Likewise back; rows and columns past the codes' are written as zeros.  Past
// the caches' reuse order in bfloat16, so that codes just written stay there
// (16384 x 4096 twice behind a forward: 202 us in all, then 184); not in float32,
// where rows are not whole lines as often (8192 x 4001: 69 us, 75 so).
template <typename T>
__device__ __forceinline__ void act8_unpack_chunk(const TropAct8Params& p, int64_t id) {
    constexpr int VEC = 8, NV = 2;
    const int lane = threadIdx.x & 63;
    int64_t row, c0;
    act8_chunk(p, id, row, c0);
    const int64_t n = row < p.rows ? p.cols : 0;
    Act8Lane<VEC> v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        v[i].load(p.codes + row * p.ldc, p.exps + row * p.lde, c0 + (i * 64 + lane) * VEC, n);
    T* out = static_cast<T*>(const_cast<void*>(p.x)) + row * p.ldx;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = c0 + (i * 64 + lane) * VEC;
        if (c >= p.cols_x) continue;
        const typename VecOf<T, VEC>::raw o = from_float<T, VEC>(v[i].values());
        if constexpr (sizeof(T) == 2)
            store_row_stream<T, VEC>(out, c, p.cols_x, o);
        else
            store_row<T, VEC>(out, c, p.cols_x, o);
    }
}
template <typename T>
__device__ __forceinline__ void act8_unpack_body(const TropAct8Params& p) {
    const int64_t id = act8_wave_id(blockIdx.x) + p.chunk0;
    if (id < p.total) act8_unpack_chunk<T>(p, id);
}

}  // namespace trop
