// Weight gradient of a linear layer from activations in 8 bits:
// grad_w[o][c] = sum_n dz[n][o] x[n][c].
//
// The values of x are exact in bfloat16, so one pass turns the codes into the
// product's operand (3 bytes an element moved) and the matrix cores do the
// rest.  Both operands lie along the product's rows ([token][column]), which
// the tile loop reads as they are.  float32 dz is taken apart into three
// bfloat16 values by cutting bits: 8, 8 and the last 8, whose sum is dz
// exactly; a tile of x meets the three of dz in turn.
//
// Measured (one MI355X): 8192 tokens x 4096 x 16384 bfloat16 841-871 us in all,
// 20-27 of them unpacking (1.26-1.31 PFLOP/s); on other values three calls in a
// row 1000-1030 and twenty 880-900, the library's product of unpacked bfloat16
// operands in turn with it 1060-1090 and 930.  Smaller ones are level with that
// product: 4096 x 4096 x 4096 135-145 us against 139-143, 2048 x 1024 x 1024
// 19.5-22 against 18-25.  One token x 8192 x 16384: 106 us, float32 215 (the
// output alone 54 and 108: 64 rows are unpacked, packed and multiplied, and a
// store writes 32 or 64 bytes of 16 rows).  4096 x 1024 x 4096
// float32 123-143 us: 27 to unpack and take apart (181 MB), 90 for three products
// (1.15 PFLOP/s, the matrix units busy half of the cycles: one round of 48 k
// tiles, with first loads and a last store that nothing hides), 13 to add four
// parts; the library's float32 product takes 258-290.  Two bfloat16 parts of dz
// would take two thirds of the product and lose its last 8 bits.
#pragma once
#include "act8_kernels.h"
#include "mfma_gemm.h"

namespace trop {

// Parts of dz: 1 (bfloat16) or 3 (float32).
template <typename T>
constexpr int grad_w_parts() {
    return sizeof(T) == 2 ? 1 : 3;
}

// dz's rows [0, tokens_p) x [0, outs_p) into [token / 64][part][64][outs_p],
// zeros past its end.  A wave takes 512 columns of a row.
template <typename T>
__device__ __forceinline__ void grad_w_pack_dz(const TropGradWParams& p, int64_t id) {
    constexpr int PARTS = grad_w_parts<T>();
    const int64_t chunks = (p.outs_p + 511) / 512;
    const int64_t n = id / chunks, o = (id - n * chunks) * 512 + (threadIdx.x & 63) * 8;
    if (n >= p.tokens_p || o >= p.outs_p) return;
    const int64_t have = n < p.tokens ? p.outs : 0;
    const T* row = static_cast<const T*>(p.dz) + n * p.lddz;
    bf16* out = static_cast<bf16*>(p.dzp) + ((n / 64 * PARTS) * 64 + n % 64) * p.outs_p + o;
    if constexpr (PARTS == 1) {
        *reinterpret_cast<VecOf<bf16, 8>::raw*>(out) = load_row<bf16, 8>(row, o, have);
    } else {
        VecOf<uint16_t, 8>::raw parts[3];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const FloatVec<4> v = load_row<float, 4>(row, o + q * 4, have);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float rest = v[i];
#pragma unroll
                for (int k = 0; k < 3; ++k) {  // (the third has no more than 8 bits left)
                    const uint32_t cut = __builtin_bit_cast(uint32_t, rest) & 0xffff0000u;
                    parts[k][q * 4 + i] = (uint16_t)(cut >> 16);
                    rest -= __builtin_bit_cast(float, cut);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<VecOf<uint16_t, 8>::raw*>(out + k * 64 * p.outs_p) = parts[k];
    }
}

// Both operands in one launch: the first x_groups workgroups unpack x.
template <typename T>
__device__ __forceinline__ void grad_w_pack_body(const TropGradWParams& p) {
    if (blockIdx.x < p.x_groups) {
        const int64_t id = act8_wave_id(blockIdx.x);
        if (id < p.x.total) act8_unpack_chunk<bf16>(p.x, id);
    } else {
        grad_w_pack_dz<T>(p, act8_wave_id(blockIdx.x - p.x_groups));
    }
}

// A tile of BM columns x BN output features, the sum over the tokens or over
// part `split` of them.  The columns are the product's rows, so a lane holds
// four consecutive ones of an output feature.
template <typename C, typename T>
__device__ __forceinline__ void grad_w_body(const TropGradWParams& p, char* lds) {
    constexpr int PARTS = grad_w_parts<T>();
    static_assert(C::REPEAT == PARTS && C::KT == 64, "k tiles");
    const int64_t tn = (p.cols + C::BM - 1) / C::BM;
    int64_t mi, q;
    if (!mg_tile(blockIdx.x, (p.outs + C::BN - 1) / C::BN, tn * p.splits, mi, q)) return;
    const int64_t ni = q % tn, split = q / tn;
    const int64_t ktiles = p.tokens_p / 64, per = (ktiles + p.splits - 1) / p.splits;
    const int64_t kt0 = min(split * per, ktiles), kt1 = min(kt0 + per, ktiles);
    MgOperand a, b;
    a.plane_bytes = b.plane_bytes = 0;
    a.exp = b.exp = 0;
    a.ld = p.cols_p;
    a.base = static_cast<const char*>(p.xp) + (kt0 * 64 * a.ld + ni * C::BM) * 2;
    a.k_bytes = 64 * a.ld * 2;
    a.last_row = (int32_t)((p.cols_p - ni * C::BM) / 8 - 1);
    a.last_k = 0x7fffffff;
    if (p.dzp) {
        b.ld = p.outs_p;
        b.base = static_cast<const char*>(p.dzp) + (kt0 * PARTS * 64 * b.ld + mi * C::BN) * 2;
        b.last_row = (int32_t)((p.outs_p - mi * C::BN) / 8 - 1);
        b.last_k = 0x7fffffff;
    } else {  // (bfloat16; past the last token x is zero)
        b.ld = p.lddz;
        b.base = static_cast<const char*>(p.dz) + (kt0 * 64 * b.ld + mi * C::BN) * 2;
        b.last_row = (int32_t)((p.outs - mi * C::BN) / 8 - 1);
        b.last_k = (int32_t)min(p.tokens - 1 - kt0 * 64, (int64_t)0x7fffffff);
    }
    b.k_bytes = 64 * b.ld * 2;
    const float scale[C::FN] = {};
    f32x4 acc[C::FM][C::FN];
    mg_walk<C>(acc, a, b, scale, (int)((kt1 - kt0) * PARTS), lds);
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int64_t c0 = ni * C::BM + (wave / C::WN) * (C::BM / C::WM) + 4 * (lane / 16);
    const int64_t o0 = mi * C::BN + (wave % C::WN) * (C::BN / C::WN) + (lane & 15);
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        const int64_t o = o0 + 16 * j;
        if (o >= p.outs) continue;
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            const int64_t c = c0 + 16 * i;
            if (c >= p.cols) continue;
            if (p.splits > 1)
                *reinterpret_cast<f32x4*>(p.part + (split * p.outs + o) * p.cols_p + c) = acc[i][j];
            else
                store_row<T, 4>(static_cast<T*>(p.grad_w) + o * p.ldgw, c, p.cols, from_float<T, 4>(acc[i][j]));
        }
    }
}

// The parts' sums in order; a workgroup takes 1024 columns of an output
// feature.  No parts: zeros.
template <typename T>
__device__ __forceinline__ void grad_w_finish_body(const TropGradWParams& p) {
    const int64_t id = p.id0 + blockIdx.x, blocks = (p.cols + 1023) / 1024;
    const int64_t o = id / blocks, c = (id - o * blocks) * 1024 + threadIdx.x * 4;
    if (c >= p.cols) return;
    FloatVec<4> s = FloatVec<4>(0.f);
    const float* q = p.part + o * p.cols_p + c;
#pragma unroll 8
    for (int k = 0; k < p.splits; ++k) {
        const FloatVec<4> v = load_vec<float, 4>(q + k * p.outs * p.cols_p);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += v[e];
    }
    store_row<T, 4>(static_cast<T*>(p.grad_w) + o * p.ldgw, c, p.cols, from_float<T, 4>(s));
}

}  // namespace trop
