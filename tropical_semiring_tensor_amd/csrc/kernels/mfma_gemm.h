// Matrix products on the matrix cores: C[i][j] = sum_k A(i, k) B(j, k) with
// 16-bit operands and float32 sums, the tile loop shared by the linear cross
// entropy's kernels and the weight gradient from 8-bit activations.
//
// A workgroup of WM x WN waves computes a BM x BN tile; a wave computes
// (BM / WM) x (BN / WN) of it in 16 x 16 blocks (v_mfma_f32_16x16x32).  K is
// walked in tiles of 64.  A tile goes from global memory to LDS directly
// (16 bytes per lane, no registers in between) into one of two buffers (or
// four, three tiles ahead) while another is multiplied.  Operands are read as they lie in
// memory, so nothing is transposed beforehand:
//   KM  element (i, k) at i ld + k           (rows along k)
//   MM  element (i, k) at k ld + i           (rows along i)
//   QK  element (i, k) at (k / 4) 4 ld + 4 i + k % 4    (quads along k)
//   QM  element (i, k) at (i / 4) 4 ld + 4 k + i % 4    (quads along i)
// A lane of the 16x16x32 instruction takes 8 consecutive k of one i: one
// 16-byte LDS read for KM, two 8-byte reads for QK, two transposing reads
// (ds_read_b64_tr_b16: 16 lanes exchange a 4 x 16 block) for MM and QM.  The
// LDS copies are swizzled in 16-byte chunks so that the lanes of a read
// meet distinct banks (no conflicts by the counters); since a direct load
// fills LDS in lane order, it is the lanes' global addresses that are
// permuted.
//
// PLANES = 1: bfloat16 values, k tiles of 64.  PLANES = 2: a float32 value
// scaled by a power of two, as the sum of two float16 values h + l (22
// bits); the product is l h' + h l' + h h'.  A k tile is 32 of both planes,
// as many bytes, so that every value is loaded and read once for its three
// products.  KM and MM have 32 consecutive elements' h, then their l (`ld`
// counts both).  QK and QM have the planes apart, and these hold the float32
// value's upper and lower 16 bits: the wave that reads a fragment joins them,
// scales the values and splits them.  The scale is one for each row of B, a
// column of the product, so that a column keeps its digits however small it
// is beside the others.  RKM and RMM are KM and MM in float32 as it lies in memory, scaled and split by the wave that reads it
// from LDS (16 bytes and 4 bytes a read): no copy beforehand, for matrices
// that one or two tiles read.
#pragma once
#include "train_common.h"

namespace trop {

enum OperandKind { KM, MM, QK, QM, RKM, RMM };

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// One operand of a tile's walk.
struct MgOperand {
    const char* base;     // tile row 0 at k = 0, plane 0
    int64_t ld;           // elements
    int64_t plane_bytes;  // QK, QM: from plane 0 to plane 1
    int64_t k_bytes;      // from one k tile to the next
    int32_t last_row;     // KM: last readable tile row; MM: last readable 16-byte chunk of a row
    int32_t last_k;       // KM: last readable chunk of a row (counted from k = 0); MM: last readable k
    int32_t exp;          // RKM, RMM: the scale's exponent
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
                 : "memory", "m0");
}

// This wave's LDS reads have returned (and, with LOADS, its loads to LDS have
// landed), and so it is for all waves of the workgroup.
template <bool LOADS>
__device__ __forceinline__ void mg_sync() {
    if constexpr (LOADS)
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}
__device__ __forceinline__ void mg_barrier() { asm volatile("s_barrier" ::: "memory"); }

template <OperandKind KIND, int ROWS, int PLANES, int WAVES>
struct MgTile {
    static constexpr bool RAW = KIND == RKM || KIND == RMM;
    static constexpr bool HALVES = PLANES == 2 && (KIND == QK || KIND == QM);
    static constexpr int BK = 64;       // 16-bit elements of a tile row, of both planes
    static_assert(!RAW || PLANES == 2, "float32");
    static constexpr int KT = BK / PLANES;  // its k
    static constexpr int BYTES = ROWS * BK * 2;
    static constexpr int LOADS = BYTES / 1024 / WAVES;  // per wave
    static_assert(LOADS >= 1 && BYTES % (1024 * WAVES) == 0, "tile rows per wave");
    // 16-byte chunks of a line of the LDS copy
    // (two planes: a line of MM holds both, as memory does; QK has the second
    // plane's lines after the first's, QM its chunks after the first's)
    static constexpr int ROW_CHUNKS = KIND == KM || KIND == RKM   ? BK / 8
                                      : KIND == MM || KIND == RMM ? PLANES * ROWS / 8
                                      : KIND == QK                ? ROWS / 2
                                                                  : BK / 2;

    // Chunk c of a line lies at c ^ swizzle(line).  LDS serves 256 bytes, 16
    // chunks, at a time, so the lanes of a read that are served together
    // must differ in their chunk modulo 16:
    //   KM  16 rows, one chunk each       MM, QM  4 lines x 2 chunks x 2 k groups
    //   QK  16 rows of 8 bytes in 2 lines    RMM  4 lines, 8 apart, x 4 chunks
    static __device__ __forceinline__ int swizzle(int line) {
        if constexpr (KIND == KM || KIND == RKM) return (line >> 1) & 7;
        if constexpr (KIND == RMM) return ((line >> 3) & 3) * 4;
        if constexpr (KIND == MM)
            return (PLANES * ROWS >= 128 ? (line & 3) * 4 : ((line >> 1) & 1) * 4) + ((line >> 3) & 1) * 2;
        if constexpr (KIND == QK) return ((line >> 1) & 1) * 8;
        if constexpr (KIND == QM) return (line & 1) * 2 + ((line >> 1) & 1) * 8;
        return 0;
    }

    // A wave's loads are STEP lines apart.  Where no line is clamped (all but
    // KM) those of equal swizzle then differ by a constant, kept out of the
    // vector registers: one offset serves all (two where MM's steps of 8
    // lines alternate in swizzle).  (Of two spilled registers, one was an
    // offset, whose reload waited for the loads before it: grad_w 970
    // against 830 us.)
    static constexpr int STEP = WAVES * 64 / ROW_CHUNKS;
    static constexpr int OFFSETS = KIND == KM || RAW ? LOADS : KIND == MM && STEP % 16 == 8 && LOADS > 1 ? 2 : 1;
    static_assert(KIND == KM || RAW || LOADS == 1 ||
                      (WAVES * 64 % ROW_CHUNKS == 0 && STEP % (KIND == MM ? 16 / OFFSETS : 4) == 0),
                  "equal swizzles OFFSETS STEP lines apart");
    static_assert(KIND != QK || PLANES == 1 || 8 % STEP == 0, "a load of QK within a plane");

    // This lane's byte offsets of its loads, from the tile's base.
    static __device__ __forceinline__ void offsets(const MgOperand& o, int wave, int lane, uint32_t (&off)[OFFSETS]) {
#pragma unroll
        for (int s = 0; s < OFFSETS; ++s) {
            const int c = (wave + WAVES * s) * 64 + lane;  // chunk of the tile
            const int line = c / ROW_CHUNKS, col = (c % ROW_CHUNKS) ^ swizzle(line);
            if constexpr (KIND == KM)
                off[s] = (uint32_t)((int64_t)min(line, o.last_row) * o.ld * 2 + col * 16);
            else if constexpr (KIND == MM)
                off[s] = (uint32_t)((int64_t)line * o.ld * 2 + min(col, o.last_row) * 16);
            else if constexpr (KIND == RKM)
                off[s] = (uint32_t)((int64_t)min(line, o.last_row) * o.ld * 4 + col * 16);
            else if constexpr (KIND == RMM)
                off[s] = (uint32_t)((int64_t)line * o.ld * 4 + min(col, o.last_row) * 16);
            else if constexpr (KIND == QM && PLANES == 2)
                off[s] = (uint32_t)((int64_t)line * o.ld * 8 + (col & 15) * 16 + (col >> 4) * o.plane_bytes);
            else
                off[s] = (uint32_t)((int64_t)line * o.ld * 8 + col * 16);
        }
    }

    // Loads of k tile kt (base: that tile's) into `lds`.
    static __device__ __forceinline__ void load(const MgOperand& o, const char* base, int kt, uint32_t lds, int wave,
                                                int lane, const uint32_t (&off)[OFFSETS]) {
        const int64_t step = STEP * o.ld * (KIND == MM ? 2 : 8);
        bool tail = false;  // the operand ends inside this tile
        if constexpr (KIND == KM && PLANES == 1) tail = (kt + 1) * (BK / 8) - 1 > o.last_k;
        if constexpr (KIND == MM && PLANES == 1) tail = (kt + 1) * BK - 1 > o.last_k;
        if constexpr (KIND == RKM) tail = (kt + 1) * (BK / 8) - 1 > o.last_k;
        if constexpr (KIND == RMM) tail = (kt + 1) * KT - 1 > o.last_k;
        if (__builtin_expect(tail, 0)) {
#pragma unroll
            for (int s = 0; s < LOADS; ++s) {
                const int c = (wave + WAVES * s) * 64 + lane, line = c / ROW_CHUNKS;
                uint32_t v;
                if constexpr (KIND == KM || KIND == RKM) {  // its last chunk again: x is zero there
                    const int col = (c % ROW_CHUNKS) ^ swizzle(line);
                    v = off[s] - (uint32_t)max(0, kt * (BK / 8) + col - o.last_k) * 16;
                } else if constexpr (KIND == RMM) {  // its last row again: G is zero there
                    v = off[s] - (uint32_t)((int64_t)max(0, kt * KT + line - o.last_k) * o.ld * 4);
                } else {
                    v = off[0] + (uint32_t)(s * step) - (uint32_t)((int64_t)max(0, kt * BK + line - o.last_k) * o.ld * 2);
                }
                load_to_lds(lds + (wave + WAVES * s) * 1024, base, v);
            }
        } else {
#pragma unroll
            for (int s = 0; s < LOADS; ++s) {
                if constexpr (KIND == KM || RAW)
                    load_to_lds(lds + (wave + WAVES * s) * 1024, base, off[s]);
                else if constexpr (KIND == QK && PLANES == 2)
                    load_to_lds(lds + (wave + WAVES * s) * 1024,
                                base + s * STEP / 8 * o.plane_bytes + s % (8 / STEP) * step, off[0]);
                else
                    load_to_lds(lds + (wave + WAVES * s) * 1024, base + s / OFFSETS * OFFSETS * step,
                                off[s % OFFSETS]);
            }
        }
    }

    // Fragment of rows [row, row + 16) of a tile: k [32 kk, 32 kk + 32), or
    // all 32 k of plane kk.
    static __device__ __forceinline__ s16x8 fragment(const char* tile, int row, int kk, int lane) {
        const int g = lane / 16, i = lane & 15;
        if constexpr (KIND == KM) {
            return *reinterpret_cast<const s16x8*>(tile + (row + i) * (BK * 2) + (((kk * 4 + g) ^ swizzle(i)) * 16));
        } else if constexpr (KIND == QK) {
            // (row is a multiple of 16 tokens, 8 chunks; i / 2 < 8)
            const int quad = kk * 8 + g * 2;
            const char* p = tile + quad * (ROWS * 8) + (((row + i) / 2) ^ swizzle(quad)) * 16 + (i & 1) * 8;
            const s16x4 a = *reinterpret_cast<const s16x4*>(p);
            const s16x4 b = *reinterpret_cast<const s16x4*>(p + ROWS * 8);
            return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            s16x4 v[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int k = kk * 32 + g * 8 + t * 4 + i / 4;
                const char* p;
                if constexpr (KIND == MM) {
                    const int chunk = row / 8 + (i & 3) / 2;
                    p = tile + k * (ROWS * 2) + (chunk ^ swizzle(k)) * 16 + (i & 1) * 8;
                } else {
                    const int quad = row / 4 + (i & 3);
                    p = tile + quad * (BK * 8) + ((k / 2) ^ swizzle(quad)) * 16 + (k & 1) * 8;
                }
                v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MG_LDS s16x4*)p);
            }
            return __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }

    // Two planes of MM, QK and QM: all of a lane's reads are at its `base` with
    // constant bits turned over or a constant added, so one register holds
    // their addresses (one each took 34 spilled ones in grad_w's 256 x 256
    // tile, beside HALVES' scales).  base: of the wave's rows from row0 on, a
    // multiple of their number; r: a multiple of 16 below that.
    static constexpr bool BASED = PLANES == 2 && (KIND == MM || KIND == QK || KIND == QM);
    static __device__ __forceinline__ uint32_t base(uint32_t tile, int row0, int lane) {
        const int g = lane / 16, i = lane & 15;
        if constexpr (KIND == MM) {
            const int line = g * 8 + i / 4;
            return tile + line * (ROWS * 4) + ((row0 / 4 + (i & 3) / 2) ^ swizzle(line)) * 16 + (i & 1) * 8;
        } else if constexpr (KIND == QK) {
            return tile + g * 2 * (ROWS * 8) + (((row0 + i) / 2) ^ swizzle(g * 2)) * 16 + (i & 1) * 8;
        } else {
            const int k = g * 8 + i / 4, quad = row0 / 4 + (i & 3);
            return tile + quad * (BK * 8) + ((k / 2) ^ swizzle(quad)) * 16 + (k & 1) * 8;
        }
    }
    static __device__ __forceinline__ s16x8 fragment_at(uint32_t base, int r, int kk) {
        s16x4 v[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if constexpr (KIND == MM) {
                const uint32_t p = (base ^ (r / 32 * 8 + kk * 4 + r % 32 / 8) * 16) + t * 4 * (ROWS * 4);
                v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MG_LDS s16x4*)p);
            } else if constexpr (KIND == QK) {
                const uint32_t p = (base ^ r / 2 * 16) + (kk * 8 + t) * (ROWS * 8);
                v[t] = *(MG_LDS const s16x4*)p;
            } else {
                const uint32_t p = (base ^ t * 2 * 16) + r / 4 * (BK * 8) + kk * 16 * 16;
                v[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MG_LDS s16x4*)p);
            }
        }
        return __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
    }

    // HALVES: the two fragments h and l hold become those of the float32 values
    // times `scale`, a power of two.
    static __device__ __forceinline__ void split(float scale, s16x8& h, s16x8& l) {
        const u32x4 u = __builtin_bit_cast(u32x4, h), d = __builtin_bit_cast(u32x4, l);
        f16x8 a, b;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const uint32_t bits = __builtin_amdgcn_perm(u[q / 2], d[q / 2], q & 1 ? 0x07060302u : 0x05040100u);
            const float v = __builtin_bit_cast(float, bits);
            a[q] = (_Float16)(v * scale);  // (the product is exact)
            b[q] = (_Float16)__builtin_fmaf(v, scale, -(float)a[q]);
        }
        h = __builtin_bit_cast(s16x8, a);
        l = __builtin_bit_cast(s16x8, b);
    }

    // Both fragments of rows [row0 + r, row0 + r + 16), from `tile` or from
    // `at`, the base.  RAW: of the values times 2^exp; HALVES: times `scale`.
    static __device__ __forceinline__ void fragments(const char* tile, uint32_t at, int row0, int r, int lane,
                                                     int32_t exp, float scale, s16x8& h, s16x8& l) {
        const int row = row0 + r;
        if constexpr (BASED) {
            h = fragment_at(at, r, 0);
            l = fragment_at(at, r, 1);
            if constexpr (HALVES) split(scale, h, l);
        } else if constexpr (!RAW) {
            h = fragment(tile, row, 0, lane);
            l = fragment(tile, row, 1, lane);
        } else {
            const int g = lane / 16, i = lane & 15;
            float v[8];
            if constexpr (KIND == RKM) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const f32x4 c = *reinterpret_cast<const f32x4*>(tile + (row + i) * (BK * 2) +
                                                                    (((2 * g + t) ^ swizzle(i)) * 16));
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[4 * t + q] = c[q];
                }
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    v[q] = *reinterpret_cast<const float*>(tile + (g * 8 + q) * (ROWS * 4) +
                                                           ((((row + i) / 4) ^ (g * 4)) * 16) + (i & 3) * 4);
            }
            f16x8 a, b;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float s = ldexpf(v[q], exp);
                a[q] = (_Float16)s;
                b[q] = (_Float16)(s - (float)a[q]);
            }
            h = __builtin_bit_cast(s16x8, a);
            l = __builtin_bit_cast(s16x8, b);
        }
    }
};

template <int PLANES>
__device__ __forceinline__ f32x4 mg_mfma(s16x8 a, s16x8 b, f32x4 c) {
    if constexpr (PLANES == 1)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0,
                                                      0, 0);
}

// A tile of eight waves alternates them in two groups (see mg_walk); four
// waves read and multiply in turn, with other workgroups' waves between.
// Measured at 256 x 256 (one MI355X, 8192 x 8192 x 4096 and 8192 x 4096 x
// 8192, float32 stored): KM KM 1241-1255 TFLOP/s, MM QK 1262-1288, MM QM
// 1260-1294; all eight waves in turn 1132-1151, 1242-1245, 1253-1257; in two
// groups with k tiles of 32 in four buffers 1199-1225, 1168-1201, 1224-1254
// (half-line requests for KM).  32 x 32 x 16 instructions, four waves of 128 x
// 128, more buffers, loads spread between the products: 1080-1290.  With the
// matrix units busy 60-65% of the cycles the clock settles at 1.85-2.05 GHz,
// lower where they are busier; with every load hitting the L1 (a timing copy)
// KM KM reaches 1500.  In 128 x 128, k tiles of 32 or three buffers are slower
// by up to a fifth.  Two planes: a third fewer loads and reads per product,
// and 1340 TFLOP/s of 16-bit products (logits of 4096 x 1024 x 32768, with their
// epilogue) against 1140 to 1250 in three walks, a plane pair each; the
// gradients, which also split float32's halves, 1160 to 1220 of them, the
// matrix units busy 62% of the cycles (1440 and 70% without the split).
// (A large library product on the same card: 1430-1470 in bfloat16, 153 in
// float32.)
// REPEAT: each k tile of A meets that many of B in turn (B's values in parts).
template <int BM_, int BN_, int WM_, int WN_, OperandKind KA_, OperandKind KB_, int PLANES_, int STAGES_ = 2,
          int REPEAT_ = 1>
struct MgConfig {
    static constexpr int REPEAT = REPEAT_;
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, PLANES = PLANES_;
    static constexpr int WAVES = WM * WN, THREADS = WAVES * 64;
    static constexpr int STAGES = STAGES_;  // buffers
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // 16 x 16 blocks of a wave
    using TA = MgTile<KA_, BM, PLANES, WAVES>;
    using TB = MgTile<KB_, BN, PLANES, WAVES>;
    static constexpr int KT = TA::KT;  // k of a tile
    static constexpr bool RAW = TA::RAW;
    static constexpr bool SCALED = TB::HALVES;  // B has a scale for each of its rows
    static constexpr int LOADS = TA::LOADS + TB::LOADS;  // of a wave for a tile
    static_assert(STAGES == 2 || (WAVES == 4 && (STAGES & (STAGES - 1)) == 0 && LOADS * (STAGES - 2) < 64), "the waits");
    static constexpr int STAGE = TA::BYTES + TB::BYTES;
    static constexpr int LDS_BYTES = STAGES * STAGE;
};

template <typename C>
__device__ __forceinline__ void mg_multiply(f32x4 (&acc)[C::FM][C::FN], const s16x8 (&a)[C::FM],
                                            const s16x8 (&b)[C::FN]) {
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = mg_mfma<C::PLANES>(a[i], b[j], acc[i][j]);
}

// Workgroup -> tile of an active tm x tn grid (false: none).  Each XCD (a
// workgroup's id modulo 8) takes a consecutive range of the tiles, which run
// down groups of 8 tile rows, so the tiles that an XCD works on at a time
// share operand panels in its L2.
__device__ __forceinline__ bool mg_tile(int64_t id, int64_t tm, int64_t tn, int64_t& mi, int64_t& ni) {
    const int64_t total = tm * tn, per = total / 8, rest = total % 8;
    const int64_t xcd = id % 8, k = id / 8;
    if (k >= per + (xcd < rest ? 1 : 0)) return false;
    const int64_t t = xcd * per + min(xcd, rest) + k;
    const int64_t group = t / (8 * tn), in = t - group * 8 * tn, rows = min((int64_t)8, tm - group * 8);
    mi = group * 8 + in % rows;
    ni = in / rows;
    return true;
}

// Walks the first `ktiles` k tiles of both operands, each of which starts
// at or before an operand's last_k.  `scale`: SCALED, of B's row 16 fj + lane %
// 16 of the wave's part.  The sum of row
// 16 fi + 4 (lane / 16) + r and column 16 fj + lane % 16 of the wave's part
// is acc[fi][fj][r].  `lds`: LDS_BYTES.
//
// Eight waves: the second four (one more wave on each SIMD) run half a turn
// behind the first, held by one extra barrier.  A turn is: read the tile's
// fragments; barrier; multiply; barrier.  So on each SIMD one wave
// multiplies while the other reads.  In the half turn in which the first
// group reads tile t and the second multiplies tile t - 1, both start their
// loads of tile t + 1 into the buffer that tile t - 1 left (the second group
// read it in the half turn before), and have until the end of the next half
// turn: the first group's multiplying, the second's reading.
template <typename C>
__device__ __forceinline__ void mg_walk(f32x4 (&acc)[C::FM][C::FN], const MgOperand& a, const MgOperand& b,
                                        const float (&scale)[C::FN], int ktiles, char* lds) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int arow = (wave / C::WN) * (C::BM / C::WM), brow = (wave % C::WN) * (C::BN / C::WN);
    uint32_t aoff[C::TA::OFFSETS], boff[C::TB::OFFSETS];
    C::TA::offsets(a, wave, lane, aoff);
    C::TB::offsets(b, wave, lane, boff);
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const uint32_t lds0 = lds_offset(lds);
    uint32_t abase = 0, bbase = 0;
    if constexpr (C::TA::BASED) abase = C::TA::base(lds0, arow, lane);
    if constexpr (C::TB::BASED) bbase = C::TB::base(lds0 + C::TA::BYTES, brow, lane);
    // the bases in a buffer, hidden from the compiler, which would make and
    // keep every read's address before the loop
    auto bases = [&](int buf, uint32_t& a_at, uint32_t& b_at) {
        a_at = abase + buf * C::STAGE;
        b_at = bbase + buf * C::STAGE;
        if constexpr (C::TA::BASED) asm volatile("" : "+v"(a_at));
        if constexpr (C::TB::BASED) asm volatile("" : "+v"(b_at));
    };
    if (ktiles <= 0) {
        mg_sync<true>();
        return;
    }
    int kt = 0;  // the next tile to load
    const char *pa = a.base, *pb = b.base;
    auto load_next = [&](int buf) {
        C::TA::load(a, pa, kt, lds0 + buf * C::STAGE, wave, lane, aoff);
        C::TB::load(b, pb, kt, lds0 + buf * C::STAGE + C::TA::BYTES, wave, lane, boff);
        ++kt;
        if (C::REPEAT == 1 || kt % C::REPEAT == 0) pa += a.k_bytes;
        pb += b.k_bytes;
    };
    if constexpr (C::WAVES == 8) {
        s16x8 fa[2][C::FM], fb[2][C::FN];
        auto read = [&](int buf) {
            const char* ta = lds + buf * C::STAGE;
            const char* tb = ta + C::TA::BYTES;
            uint32_t a_at, b_at;
            bases(buf, a_at, b_at);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                for (int j = 0; j < C::FN; ++j) {
                    if constexpr (C::TB::BASED)
                        fb[kk][j] = C::TB::fragment_at(b_at, 16 * j, kk);
                    else
                        fb[kk][j] = C::TB::fragment(tb, brow + 16 * j, kk, lane);
                }
#pragma unroll
                for (int i = 0; i < C::FM; ++i) {
                    if constexpr (C::TA::BASED)
                        fa[kk][i] = C::TA::fragment_at(a_at, 16 * i, kk);
                    else
                        fa[kk][i] = C::TA::fragment(ta, arow + 16 * i, kk, lane);
                }
            }
            if constexpr (C::SCALED) {
                // here, beside the other group's products: the compiler would
                // put it off past the barrier, before this group's own (8192 x
                // 2048 x 16384: a backward of 3.53 ms against 3.58)
#pragma unroll
                for (int j = 0; j < C::FN; ++j) {
                    C::TB::split(scale[j], fb[0][j], fb[1][j]);
                    asm volatile("" : "+v"(fb[0][j]), "+v"(fb[1][j]));
                }
            }
        };
        auto multiply = [&]() {
            if constexpr (C::PLANES == 1) {
                mg_multiply<C>(acc, fa[0], fb[0]);
                mg_multiply<C>(acc, fa[1], fb[1]);
            } else {
                mg_multiply<C>(acc, fa[1], fb[0]);
                mg_multiply<C>(acc, fa[0], fb[1]);
                mg_multiply<C>(acc, fa[0], fb[0]);
            }
        };
        load_next(0);
        mg_sync<true>();
        if (wave >= 4) {
            if (1 < ktiles) load_next(1);
            mg_barrier();
            for (int t = 0; t < ktiles; ++t) {
                read(t & 1);
                mg_sync<true>();
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_setprio(1);
                if (t + 2 < ktiles) load_next(t & 1);
                multiply();
                __builtin_amdgcn_s_setprio(0);
                __builtin_amdgcn_sched_barrier(0);
                mg_barrier();
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            for (int t = 0; t < ktiles; ++t) {
                if (t + 1 < ktiles) load_next((t + 1) & 1);
                read(t & 1);
                mg_sync<false>();
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_setprio(1);
                multiply();
                __builtin_amdgcn_s_setprio(0);
                __builtin_amdgcn_sched_barrier(0);
                mg_sync<true>();
                __builtin_amdgcn_sched_barrier(0);
            }
            mg_barrier();
        }
    } else {
        constexpr int S = C::STAGES;
        for (int t = 0; t < min(S - 1, ktiles); ++t) load_next(t);
        for (int t = 0; t < ktiles; ++t) {
            // tile t has landed (the S - 2 after it may be on their way);
            // tile t - 1 has been read
            if (S > 2 && t + S - 1 <= ktiles)
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * C::LOADS) : "memory");
            else
                mg_sync<true>();
            if (t + S - 1 < ktiles) load_next((t + S - 1) & (S - 1));
            const char* ta = lds + (t & (S - 1)) * C::STAGE;
            const char* tb = ta + C::TA::BYTES;
            s16x8 fa[2][C::FM], fb[2][C::FN];
            if constexpr (C::PLANES == 1) {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                    for (int j = 0; j < C::FN; ++j) fb[kk][j] = C::TB::fragment(tb, brow + 16 * j, kk, lane);
#pragma unroll
                    for (int i = 0; i < C::FM; ++i) fa[kk][i] = C::TA::fragment(ta, arow + 16 * i, kk, lane);
                    mg_multiply<C>(acc, fa[kk], fb[kk]);
                }
            } else {
                uint32_t a_at, b_at;
                bases(t & (S - 1), a_at, b_at);
#pragma unroll
                for (int j = 0; j < C::FN; ++j)
                    C::TB::fragments(tb, b_at, brow, 16 * j, lane, 0, scale[j], fb[0][j], fb[1][j]);
#pragma unroll
                for (int i = 0; i < C::FM; ++i)
                    C::TA::fragments(ta, a_at, arow, 16 * i, lane, a.exp, 1.f, fa[0][i], fa[1][i]);
                mg_multiply<C>(acc, fa[1], fb[0]);
                mg_multiply<C>(acc, fa[0], fb[1]);
                mg_multiply<C>(acc, fa[0], fb[0]);
            }
        }
    }
    mg_sync<true>();
}

}  // namespace trop
