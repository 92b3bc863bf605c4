// Matrix products on the matrix cores: C[i][j] = sum_k A(i, k) B(j, k) with
// 16-bit operands and float32 sums, the tile loop shared by the linear cross
// entropy's kernels.
//
// A workgroup of WM x WN waves computes a BM x BN tile; a wave computes
// (BM / WM) x (BN / WN) of it in 32 x 32 blocks (v_mfma_f32_32x32x16).  K is
// walked in tiles of 64.  A tile goes from global memory to LDS directly
// (16 bytes per lane, no registers in between) into one of two buffers while
// the other is multiplied.  Operands are read as they lie in memory, so
// nothing is transposed beforehand:
//   KM  element (i, k) at i ld + k           (rows along k)
//   MM  element (i, k) at k ld + i           (rows along i)
//   QK  element (i, k) at (k / 4) 4 ld + 4 i + k % 4    (quads along k)
//   QM  element (i, k) at (i / 4) 4 ld + 4 k + i % 4    (quads along i)
// A lane of the 32x32x16 instruction takes 8 consecutive k of one i: one
// 16-byte LDS read for KM, two 8-byte reads for QK, two transposing reads
// (ds_read_b64_tr_b16: 16 lanes exchange a 4 x 16 block) for MM and QM.  The
// LDS copies are swizzled in 16-byte chunks so that the lanes of a read
// meet distinct banks; since a direct load fills LDS in lane order, it is
// the lanes' global addresses that are permuted.
//
// PLANES = 1: bfloat16 values.  PLANES = 2: a float32 value scaled by a
// power of two, as the sum of two float16 values h + l (22 bits); the
// product is l h' + h l' + h h', three walks over K, smallest terms first.
#pragma once
#include "train_common.h"

namespace trop {

enum OperandKind { KM, MM, QK, QM };

constexpr int MG_BK = 64;  // k of one LDS tile

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// One operand of a tile's walk.
struct MgOperand {
    const char* base;     // tile row 0 at k = 0, plane 0
    int64_t ld;           // elements
    int64_t plane_bytes;  // from plane 0 to plane 1
    int64_t k_bytes;      // from one k tile to the next
    int32_t last_row;     // KM: last readable tile row; MM: last readable 8-element chunk of a row
    int32_t last_k;       // KM: last readable chunk of a row (counted from k = 0); MM: last readable k
};

#define MG_LDS __attribute__((address_space(3)))

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(MG_LDS const void*)p;
}

// 64 lanes x 16 bytes from base + voff to LDS at `lds` in lane order; not
// waited for.  No register is written, so nothing can be reused early.
__device__ __forceinline__ void load_to_lds(uint32_t lds, const char* base, uint32_t voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(voff), "s"(base)
                 : "memory");
}

// Every load to LDS of this wave has landed, every LDS read has returned,
// and so it is for all waves of the workgroup.
__device__ __forceinline__ void mg_sync() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <OperandKind KIND, int ROWS, int WAVES>
struct MgTile {
    static constexpr int BYTES = ROWS * MG_BK * 2;
    static constexpr int LOADS = ROWS / 8 / WAVES;  // per wave
    static_assert(LOADS >= 1 && ROWS % (8 * WAVES) == 0, "tile rows per wave");
    static constexpr int ROW_CHUNKS = KIND == KM ? 8 : KIND == MM ? ROWS / 8 : KIND == QK ? ROWS / 2 : 32;

    static __device__ __forceinline__ int swizzle(int line) {
        if constexpr (KIND == KM) return (line >> 1) & 7;
        if constexpr (KIND == MM) return ROWS >= 128 ? (line & 3) * 4 : ((line >> 1) & 1) * 4;
        if constexpr (KIND == QM) return (line & 7) * 2;
        return 0;
    }

    // This lane's byte offsets of its loads, from the tile's base.
    static __device__ __forceinline__ void offsets(const MgOperand& o, int wave, int lane, uint32_t (&off)[LOADS]) {
#pragma unroll
        for (int s = 0; s < LOADS; ++s) {
            const int c = (wave + WAVES * s) * 64 + lane;  // chunk of the tile
            const int line = c / ROW_CHUNKS, col = (c % ROW_CHUNKS) ^ swizzle(line);
            if constexpr (KIND == KM)
                off[s] = (uint32_t)((int64_t)min(line, o.last_row) * o.ld * 2 + col * 16);
            else if constexpr (KIND == MM)
                off[s] = (uint32_t)((int64_t)line * o.ld * 2 + min(col, o.last_row) * 16);
            else
                off[s] = (uint32_t)((int64_t)line * o.ld * 8 + col * 16);
        }
    }

    // Loads of k tile kt of a plane (base: that tile's) into `lds`.
    static __device__ __forceinline__ void load(const MgOperand& o, const char* base, int kt, uint32_t lds, int wave,
                                                int lane, const uint32_t (&off)[LOADS]) {
#pragma unroll
        for (int s = 0; s < LOADS; ++s) {
            uint32_t v = off[s];
            if constexpr (KIND == KM) {
                if ((kt + 1) * 8 - 1 > o.last_k) {  // the row ends inside this tile: its last chunk again
                    const int c = (wave + WAVES * s) * 64 + lane, col = (c % 8) ^ swizzle(c / 8);
                    v -= (uint32_t)max(0, kt * 8 + col - o.last_k) * 16;
                }
            }
            if constexpr (KIND == MM) {
                if ((kt + 1) * MG_BK - 1 > o.last_k) {
                    const int line = ((wave + WAVES * s) * 64 + lane) / ROW_CHUNKS;
                    v -= (uint32_t)((int64_t)max(0, kt * MG_BK + line - o.last_k) * o.ld * 2);
                }
            }
            load_to_lds(lds + (wave + WAVES * s) * 1024, base, v);
        }
    }

    // Fragment of rows [row, row + 32) and k [16 kk, 16 kk + 16) of a tile.
    static __device__ __forceinline__ s16x8 fragment(const char* tile, int row, int kk, int lane) {
        if constexpr (KIND == KM) {
            const int r = row + (lane & 31);
            return *reinterpret_cast<const s16x8*>(tile + r * 128 + (((kk * 2 + lane / 32) ^ swizzle(lane & 31)) * 16));
        } else if constexpr (KIND == QK) {
            const char* p = tile + (kk * 4 + (lane / 32) * 2) * (ROWS * 8) + (row + (lane & 31)) * 8;
            const s16x4 a = *reinterpret_cast<const s16x4*>(p);
            const s16x4 b = *reinterpret_cast<const s16x4*>(p + ROWS * 8);
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            const int g = lane / 16, i = lane & 15;
            s16x4 v[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int k = kk * 16 + (g / 2) * 8 + t * 4 + i / 4;
                const char* p;
                if constexpr (KIND == MM) {
                    const int chunk = row / 8 + (g & 1) * 2 + (i & 3) / 2;
                    p = tile + k * (ROWS * 2) + (chunk ^ swizzle(k)) * 16 + (i & 1) * 8;
                } else {
                    const int quad = row / 4 + (g & 1) * 4 + (i & 3);
                    p = tile + quad * 512 + ((k / 2) ^ swizzle(quad)) * 16 + (k & 1) * 8;
                }
                v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MG_LDS s16x4*)p);
            }
            return __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};

template <int PLANES>
__device__ __forceinline__ f32x16 mg_mfma(s16x8 a, s16x8 b, f32x16 c) {
    if constexpr (PLANES == 1)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

template <int BM_, int BN_, int WM_, int WN_, OperandKind KA_, OperandKind KB_, int PLANES_>
struct MgConfig {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, PLANES = PLANES_;
    static constexpr int WAVES = WM * WN, THREADS = WAVES * 64;
    static constexpr int FM = BM / WM / 32, FN = BN / WN / 32;  // 32 x 32 blocks of a wave
    static constexpr int PASSES = PLANES == 1 ? 1 : 3;
    using TA = MgTile<KA_, BM, WAVES>;
    using TB = MgTile<KB_, BN, WAVES>;
    static constexpr int STAGE = TA::BYTES + TB::BYTES;
    static constexpr int LDS_BYTES = 2 * STAGE;
};

// Walks k tiles [0, ktiles) of both operands.  The sums of row
// 32 fi + 8 (r / 4) + 4 (lane / 32) + r % 4 and column 32 fj + lane % 32 of
// the wave's part are acc[fi][fj][r].  `lds`: LDS_BYTES.
template <typename C>
__device__ __forceinline__ void mg_walk(f32x16 (&acc)[C::FM][C::FN], const MgOperand& a, const MgOperand& b,
                                        int ktiles, char* lds) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int arow = (wave / C::WN) * (C::BM / C::WM), brow = (wave % C::WN) * (C::BN / C::WN);
    uint32_t aoff[C::TA::LOADS], boff[C::TB::LOADS];
    C::TA::offsets(a, wave, lane, aoff);
    C::TB::offsets(b, wave, lane, boff);
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    const uint32_t lds0 = lds_offset(lds);
    const int total = ktiles * C::PASSES;
    // the next tile to load: its pass and its k tile
    int pass = 0, kt = 0;
    const char *pa = a.base, *pb = b.base;
    if constexpr (C::PASSES == 3) pa += a.plane_bytes;
    auto load_next = [&](int buf) {
        C::TA::load(a, pa, kt, lds0 + buf * C::STAGE, wave, lane, aoff);
        C::TB::load(b, pb, kt, lds0 + buf * C::STAGE + C::TA::BYTES, wave, lane, boff);
        pa += a.k_bytes;
        pb += b.k_bytes;
        if (++kt == ktiles) {
            kt = 0;
            ++pass;
            pa = a.base;
            pb = b.base + (C::PASSES == 3 && pass == 1 ? b.plane_bytes : 0);
        }
    };
    if (total > 0) load_next(0);
    mg_sync();
    for (int t = 0; t < total; ++t) {
        const int buf = t & 1;
        if (t + 1 < total) load_next(buf ^ 1);
        const char* ta = lds + buf * C::STAGE;
        const char* tb = ta + C::TA::BYTES;
#pragma unroll
        for (int kk = 0; kk < MG_BK / 16; ++kk) {
            s16x8 fa[C::FM], fb[C::FN];
#pragma unroll
            for (int j = 0; j < C::FN; ++j) fb[j] = C::TB::fragment(tb, brow + 32 * j, kk, lane);
#pragma unroll
            for (int i = 0; i < C::FM; ++i) fa[i] = C::TA::fragment(ta, arow + 32 * i, kk, lane);
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
#pragma unroll
                for (int j = 0; j < C::FN; ++j) acc[i][j] = mg_mfma<C::PLANES>(fa[i], fb[j], acc[i][j]);
        }
        mg_sync();
    }
}

}  // namespace trop
