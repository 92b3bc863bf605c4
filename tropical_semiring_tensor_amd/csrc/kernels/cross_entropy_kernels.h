// Softmax cross entropy of tokens over a large label set, from the hidden
// states x and the label matrix w, without keeping the logits l = x w^T.
//
//   lse_n = log sum_v exp l_nv           loss_n = lse_n - l_n,target
//   G_nv = g_n (exp(l_nv - lse_n) - [v = target_n])
//   grad_x = G w                         grad_w = G^T x
//
// Forward: the product's tiles end in their rows' maximum and sum of
// exponentials (8 bytes a token and tile); a merge joins them.  Backward:
// the label set is taken in pieces; a piece's logits are computed again and
// end as G in 16 bits, which two more products consume.  8 N V D operations
// in all, 2 more than with kept logits; the 4 N V bytes of logits are never
// written.  For many tokens the matrix cores bound it, for few the read of w.
// Measured, forward and backward: 8192 x 4096 x 65536 bfloat16 (7780 tokens
// count) 13.1 to 14.2 ms by the card's power, 1.18 to 1.27 PFLOP/s (logits
// 3.0, their gradient 3.3, both products of it 6.6 of 13.1 ms); 4096 x 1024 x
// 32768 float32 2.55 to 2.7 ms, 385 to 410 TFLOP/s (0.62, 0.67, 1.35 of 2.84
// under the profiler); 1000 x 1000 x 50001 bfloat16, a third ignored, 0.37 ms,
// bound by whole rounds of tiles; 256 x 512 x 8000 float32 88 to 91 us, by nine
// short launches.
//
// Tokens that do not count are left out: the kept ones are listed first
// (ordered, by one workgroup), and x is packed in that order, so masked
// tokens cost nothing and what they hold cannot reach a sum.  Packing also
// pads x with zeros to whole tiles and, for float32, splits it.
//
// float32 operands go through the matrix cores as two float16 planes of the
// value scaled by one power of two per matrix (largest magnitude in [2^14,
// 2^15)): 22 bits of every element above 2^-18 of its matrix's largest, an
// absolute 2^-39 of that largest below; three 16-bit products at 1/16 of the
// float32 units' cost each.  (A large w that few tokens meet is split by the
// tiles that read it, others beforehand.)  G is kept in float32 and split by
// the waves that read its fragments, with a scale of its own for every column of the
// product: a token's weight in grad_x, a label's largest |G| in grad_w.  So
// what the planes lose, 2^-39 of those, is nothing beside the column's own
// sum, whatever the other tokens' weights and the other labels'
// probabilities.  (With one scale for all of G a label of probability 1e-9
// had its row of grad_w to 2e-3, one of 1e-11 to a tenth.  The scales cost a
// backward of 4096 x 1024 x 32768 1.92 ms against 1.74.)
//
// G is stored in quads of labels ([label / 4][token][4]): four consecutive
// labels of a token are what a lane of the logits' product holds, so it
// stores 8 bytes next to its neighbours' without a transpose, and both
// products that follow read quads directly (along k, or across it with the
// transposing LDS read; float32's upper and lower 16 bits lie in two such
// planes for that).  It is scaled by grad_loss / max
// |grad_loss|, which the float32 sums get back at the end, so that with equal
// token weights only exp(l - lse) itself is rounded to bfloat16.
#pragma once
#include "mfma_gemm.h"

namespace trop {

constexpr float CE_LOG2E = 1.44269504088896340736f;

// exp of a logit less the maximum or lse.  The exponent's rounding makes it
// |x| 2^-24 of itself wrong, no more than the rounding of lse does.  (expf is
// a dozen operations more in the tiles' epilogues.)
__device__ __forceinline__ float ce_exp(float x) { return __builtin_amdgcn_exp2f(x * CE_LOG2E); }

__device__ __forceinline__ int64_t ce_target(const TropCeParams& p, int64_t n) {
    return p.target_bytes == 8 ? static_cast<const int64_t*>(p.target)[n]
                               : (int64_t)static_cast<const int32_t*>(p.target)[n];
}
__device__ __forceinline__ bool ce_counts(const TropCeParams& p, int64_t t) {
    return t != p.ignore_index && t >= 0 && t < p.vocab;
}

// ---- which tokens count ----------------------------------------------------
// One workgroup of 1024: each wave takes a run of consecutive tokens, 64 at a
// time, and counts by ballot; the waves' counts give each its first place.
__device__ __forceinline__ void ce_keep_body(const TropCeParams& p) {
    __shared__ int32_t wave_count[16];
    __shared__ float wave_max[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int64_t run = (p.tokens + 1023) / 1024 * 64;
    const int64_t n0 = min(wave * run, p.tokens), n1 = min(n0 + run, p.tokens);
    int32_t count = 0;
    float gmax = 0.f;
#pragma unroll 4
    for (int64_t b = n0; b < n1; b += 64) {
        const int64_t n = b + lane;
        const bool keep = n < n1 && ce_counts(p, ce_target(p, n));
        count += __popcll(__ballot(keep));
        if (p.backward && keep) {  // (of the finite ones: an infinite weight spoils its own token only)
            const float a = fabsf(p.grad_loss[n * p.grad_loss_stride]);
            gmax = a < INFINITY ? fmaxf(gmax, a) : gmax;
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) gmax = fmaxf(gmax, __shfl_xor(gmax, o, 64));
    if (lane == 0) {
        wave_count[wave] = count;
        wave_max[wave] = gmax;
    }
    __syncthreads();
    int32_t at = 0, total = 0;
    gmax = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        if (w < wave) at += wave_count[w];
        total += wave_count[w];
        gmax = fmaxf(gmax, wave_max[w]);
    }
    if (gmax == 0.f) gmax = 1.f;  // nothing to scale
#pragma unroll 4
    for (int64_t b = n0; b < n1; b += 64) {
        const int64_t n = b + lane;
        const int64_t t = n < n1 ? ce_target(p, n) : -1;
        const bool keep = n < n1 && ce_counts(p, t);
        const uint64_t mask = __ballot(keep);
        if (keep) {
            const int32_t i = at + __popcll(mask & (((uint64_t)1 << lane) - 1));
            p.slot[n] = i;
            p.rows[i] = (int32_t)n;
            p.kept_target[i] = (int32_t)t;
            if (p.backward) {
                p.kept_lse[i] = p.lse_in[n];
                p.kept_grad[i] = p.grad_loss[n * p.grad_loss_stride] / gmax;
            }
        } else if (n < n1) {
            p.slot[n] = -1;
            if (!p.backward) {
                p.loss[n] = 0.f;
                p.lse[n] = 0.f;
            }
        }
        at += __popcll(mask);
    }
    if (threadIdx.x == 0) {
        p.control->kept = total;
        p.control->grad_max = gmax;
    }
}

// ---- float32: the matrices' largest magnitudes -----------------------------
// Partial maxima over the finite elements of the rows of x that count and of
// w: workgroups 1 ... max_parts of the launch that lists the tokens.
__device__ __forceinline__ void ce_magnitude_body(const TropCeParams& p) {
    __shared__ float lds[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int64_t part = blockIdx.x - 1;
    for (int which = 0; which < 2; ++which) {
        const float* m = static_cast<const float*>(which ? p.w : p.x);
        const int64_t ld = which ? p.ldw : p.ldx, rows = which ? p.vocab : p.tokens;
        float best = 0.f;
        // a wave to a row
        for (int64_t r = part * 16 + wave; r < rows; r += (int64_t)p.max_parts * 16) {
            if (!which && !ce_counts(p, ce_target(p, r))) continue;
            const float* row = m + r * ld;
#pragma unroll 4
            for (int64_t c = lane * 4; c < p.width; c += 256) {
                const FloatVec<4> v = load_row_stream<float, 4>(row, c, p.width);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float a = fabsf(v[e]);
                    best = a < INFINITY ? fmaxf(best, a) : best;
                }
            }
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor(best, o, 64));
        if (lane == 0) lds[wave] = best;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < 16; ++w) best = fmaxf(best, lds[w]);
            p.magnitude[which * TROP_CE_MAX_PARTS + part] = best;
        }
        __syncthreads();
    }
}

// Exponent e with largest 2^e in [2^14, 2^15) (0 for a matrix of zeros).
__device__ __forceinline__ int32_t ce_scale_exp(float largest) {
    if (!(largest > 0.f)) return 0;
    return 15 - (__builtin_amdgcn_frexp_expf(largest));
}

// value 2^e as h + l, both float16.
__device__ __forceinline__ void ce_split(float scaled, _Float16& h, _Float16& l) {
    h = (_Float16)scaled;
    l = (_Float16)(scaled - (float)h);
}

// The exponent that a column of float32 G is scaled by: |v| 2^e in [2^14,
// 2^15) for its largest magnitude v, where 2^e is a float32 (a column below
// 2^-111 has fewer digits).
__device__ __forceinline__ int32_t ce_column_exp(float largest) { return min(ce_scale_exp(largest), 126); }
// The same for a token, from its weight (no G of it is larger, but for a rounding).
__device__ __forceinline__ int32_t ce_token_exp(float weight) {
    const float a = fabsf(weight);
    return ce_column_exp(a < INFINITY ? a : 0.f);
}

// m 2^e, where 2^e alone may be no float32.
struct CeScale {
    float m;
    int32_t e;
    __device__ __forceinline__ float operator()(float x) const { return ldexpf(x * m, e); }
};
// The sums' factor: max |grad_loss| / (2^own 2^other), own and other the
// exponents of G's column and of the other matrix (bfloat16: none).
template <int PLANES>
__device__ __forceinline__ CeScale ce_sum_scale(const TropCeParams& p, int32_t own, int32_t other) {
    const float g = p.control->grad_max;
    if constexpr (PLANES == 1) return {g, 0};
    return {__builtin_amdgcn_frexp_mantf(g), __builtin_amdgcn_frexp_expf(g) - own - other};
}

// ---- packing ---------------------------------------------------------------
// 8 elements of a row [c, c + 8), zeros past its end, into the packed row
// (float32: 32 elements' h, then their l).
template <int PLANES>
__device__ __forceinline__ void ce_pack8(const void* row, int64_t c, int64_t width, int32_t e, char* out) {
    if constexpr (PLANES == 1) {
        *reinterpret_cast<VecOf<bf16, 8>::raw*>(out + c * 2) = load_row<bf16, 8>(static_cast<const bf16*>(row), c, width);
    } else {
        f16x8 h, l;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const FloatVec<4> v = load_row<float, 4>(static_cast<const float*>(row), c + q * 4, width);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                _Float16 a, b;
                ce_split(ldexpf(v[i], e), a, b);
                h[q * 4 + i] = a;
                l[q * 4 + i] = b;
            }
        }
        out += c / 32 * 128 + c % 32 * 2;
        *reinterpret_cast<f16x8*>(out) = h;
        *reinterpret_cast<f16x8*>(out + 64) = l;
    }
}

// Kept rows of x, in order, and zero rows up to a whole tile (the first
// pack_x workgroups), then rows [v0, v0 + piece) of w (its last row again past
// the vocabulary).  A wave takes a row; for float32 each workgroup reduces
// the partial maxima, and the first leaves the exponents for the kernels after.
template <int PLANES>
__device__ __forceinline__ void ce_pack_body(const TropCeParams& p) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const bool is_w = blockIdx.x >= p.pack_x;
    const int64_t i = ((int64_t)blockIdx.x - (is_w ? p.pack_x : 0)) * 4 + wave;
    __shared__ float lds[2][4];
    int32_t e = 0;
    if constexpr (PLANES == 2) {
        int32_t exps[2];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float b = (int)threadIdx.x < p.max_parts ? p.magnitude[which * TROP_CE_MAX_PARTS + threadIdx.x] : 0.f;
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) b = fmaxf(b, __shfl_xor(b, o, 64));
            if (lane == 0) lds[which][wave] = b;
        }
        __syncthreads();
#pragma unroll
        for (int which = 0; which < 2; ++which)
            exps[which] = ce_scale_exp(fmaxf(fmaxf(lds[which][0], lds[which][1]), fmaxf(lds[which][2], lds[which][3])));
        e = is_w ? exps[1] : exps[0];
        if (!is_w && blockIdx.x == 0 && threadIdx.x == 0) {
            p.control->x_exp = exps[0];
            p.control->w_exp = exps[1];
        }
    }
    const size_t eb = PLANES == 1 ? 2 : 4;
    const char* row;
    char* out;
    if (is_w) {
        if (i >= p.piece) return;
        row = static_cast<const char*>(p.w) + min(p.v0 + i, p.vocab - 1) * p.ldw * eb;
        out = static_cast<char*>(p.wp) + i * p.width_p * 2 * PLANES;
    } else {
        const int64_t kept = p.control->kept;
        if (i >= (kept + 255) / 256 * 256) return;
        row = i < kept ? static_cast<const char*>(p.x) + (int64_t)p.rows[i] * p.ldx * eb : nullptr;
        out = static_cast<char*>(p.xp) + i * p.width_p * 2 * PLANES;
    }
#pragma unroll 2
    for (int64_t c = lane * 8; c < p.width_p; c += 64 * 8)
        ce_pack8<PLANES>(row, c, row ? p.width : 0, e, out);
}

// ---- tiles -----------------------------------------------------------------
// Workgroup -> tile of an active tm x tn grid (false: none).  Each XCD (a
// workgroup's id modulo 8) takes a consecutive range of the tiles, which run
// down groups of 8 tile rows, so the tiles that an XCD works on at a time
// share operand panels in its L2.
__device__ __forceinline__ bool ce_tile(int64_t id, int64_t tm, int64_t tn, int64_t& mi, int64_t& ni) {
    const int64_t total = tm * tn, per = total / 8, rest = total % 8;
    const int64_t xcd = id % 8, k = id / 8;
    if (k >= per + (xcd < rest ? 1 : 0)) return false;
    const int64_t t = xcd * per + min(xcd, rest) + k;
    const int64_t group = t / (8 * tn), in = t - group * 8 * tn, rows = min((int64_t)8, tm - group * 8);
    mi = group * 8 + in % rows;
    ni = in / rows;
    return true;
}

// The label matrix's rows from piece row r0 on as a KM operand (along the width).
template <typename C>
__device__ __forceinline__ MgOperand ce_w_rows(const TropCeParams& p, int64_t r0) {
    MgOperand o;
    o.k_bytes = 128;
    o.plane_bytes = 0;
    o.exp = 0;
    if constexpr (C::RAW) {
        o.base = static_cast<const char*>(p.w) + (p.v0 + r0) * p.ldw * 4;
        o.ld = p.ldw;
        o.last_row = (int32_t)min(p.vocab - 1 - (p.v0 + r0), (int64_t)0x7fffffff);
        o.last_k = (int32_t)(p.width / 4 - 1);
        o.exp = p.control->w_exp;
    } else if (C::PLANES == 2 || p.w_packed) {
        o.ld = p.width_p * C::PLANES;
        o.base = static_cast<const char*>(p.wp) + r0 * o.ld * 2;
        o.last_row = 0x7fffffff;
        o.last_k = 0x7fffffff;
    } else {
        o.base = static_cast<const char*>(p.w) + (p.v0 + r0) * p.ldw * 2;
        o.ld = p.ldw;
        o.last_row = (int32_t)min(p.vocab - 1 - (p.v0 + r0), (int64_t)0x7fffffff);
        o.last_k = (int32_t)(p.width / 8 - 1);
    }
    return o;
}

enum CeEpilogue { CE_STATS, CE_GRAD };

// Logits of a BM-label x BN-token tile, and their row statistics or G.
template <typename C, CeEpilogue EPI>
__device__ __forceinline__ void ce_logits_body(const TropCeParams& p, char* lds) {
    const int64_t kept = p.control->kept;
    int64_t mi, ni;
    if (!ce_tile(blockIdx.x, p.piece / C::BM, (kept + C::BN - 1) / C::BN, mi, ni)) return;
    MgOperand b;
    b.ld = p.width_p * C::PLANES;
    b.base = static_cast<const char*>(p.xp) + ni * C::BN * b.ld * 2;
    b.plane_bytes = 0;
    b.k_bytes = 128;
    b.last_row = b.last_k = 0x7fffffff;
    f32x4 acc[C::FM][C::FN];
    // (only tiles that hold a column: the loads clamp to a row's last chunk
    // within a tile, not from a tile past it)
    const float none[C::FN] = {};
    mg_walk<C>(acc, ce_w_rows<C>(p, mi * C::BM), b, none, (int)((p.width + C::KT - 1) / C::KT), lds);

    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int64_t v_wave = p.v0 + mi * C::BM + (wave / C::WN) * (C::BM / C::WM);  // label of the wave's row 0
    const int n_wave = (wave % C::WN) * (C::BN / C::WN);                          // token of its column 0 in the tile
    if constexpr (C::PLANES == 2) {
        const int32_t e = -(p.control->x_exp + p.control->w_exp);
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = ldexpf(acc[i][j][r], e);
    }
    // labels past the vocabulary (the last tile only)
    const bool ragged = v_wave + C::BM / C::WM > p.vocab;
    if (ragged) {
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t v = v_wave + 16 * i + 4 * (lane / 16) + r;
#pragma unroll
                for (int j = 0; j < C::FN; ++j) acc[i][j][r] = v < p.vocab ? acc[i][j][r] : -INFINITY;
            }
    }
    // the target's row of the wave's part, where this lane holds it
    // (register r of block i: row 16 i + 4 (lane / 16) + r), else -1
    int64_t n[C::FN];
    int32_t trow[C::FN];
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        n[j] = ni * C::BN + n_wave + 16 * j + (lane & 15);
        const int64_t d = n[j] < kept ? p.kept_target[n[j]] - v_wave : -1;
        trow[j] = d >= 0 && d < C::BM / C::WM && ((d >> 2) & 3) == lane / 16 ? (int32_t)d : -1;
    }
    if constexpr (EPI == CE_STATS) {
        float2* part = reinterpret_cast<float2*>(lds);  // [WM][BN]
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            if (__any(trow[j] >= 0)) {
                float l = 0.f;
#pragma unroll
                for (int i = 0; i < C::FM; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) l = trow[j] == 16 * i + 4 * (lane / 16) + r ? acc[i][j][r] : l;
                if (trow[j] >= 0) p.target_logit[n[j]] = l;
            }
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) m = nan_max(m, acc[i][j][r]);
            m = nan_max(m, __shfl_xor(m, 16, 64));
            m = nan_max(m, __shfl_xor(m, 32, 64));
            // (a block of -inf has nothing to sum; its logits minus 0 stay -inf)
            const float base = m == -INFINITY ? 0.f : m;
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) s += ce_exp(acc[i][j][r] - base);
            s += __shfl_xor(s, 16, 64);
            s += __shfl_xor(s, 32, 64);
            if (lane < 16) part[(wave / C::WN) * C::BN + n_wave + 16 * j + lane] = make_float2(m, s);
        }
        __syncthreads();
        if (threadIdx.x < C::BN) {
            const int64_t tok = ni * C::BN + threadIdx.x;
            float2 a = part[threadIdx.x];
#pragma unroll
            for (int q = 1; q < C::WM; ++q) {
                const float2 o = part[q * C::BN + threadIdx.x];
                const float m = nan_max(a.x, o.x), base = m == -INFINITY ? 0.f : m;
                a.y = a.y * ce_exp(a.x - base) + o.y * ce_exp(o.x - base);
                a.x = m;
            }
            if (tok < kept) reinterpret_cast<float2*>(p.stats)[tok * p.tiles + p.tile0 + mi] = a;
        }
    } else {
        const int64_t plane = p.piece * p.padded * 2;  // bytes
        uint32_t top[C::FM][4] = {};  // float32: the lane's largest finite |G| of its labels, as bits
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            const bool on = n[j] < kept;
            const float lse = on ? p.kept_lse[n[j]] : 0.f, weight = on ? p.kept_grad[n[j]] : 0.f;
#pragma unroll
            for (int i = 0; i < C::FM; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = ce_exp(acc[i][j][r] - lse);
            if (__any(trow[j] >= 0)) {
#pragma unroll
                for (int i = 0; i < C::FM; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[i][j][r] -= trow[j] == 16 * i + 4 * (lane / 16) + r ? 1.f : 0.f;
            }
            char* out = static_cast<char*>(p.g) + (((v_wave - p.v0) / 4 + lane / 16) * p.padded + n[j]) * 8;
#pragma unroll
            for (int i = 0; i < C::FM; ++i) {
                FloatVec<4> g;
#pragma unroll
                for (int r = 0; r < 4; ++r) g[r] = on ? acc[i][j][r] * weight : 0.f;
                char* o = out + (int64_t)(4 * i) * p.padded * 8;
                if constexpr (C::PLANES == 1) {
                    *reinterpret_cast<VecOf<bf16, 4>::raw*>(o) = from_float<bf16, 4>(g);
                } else {
                    const u32x4 u = __builtin_bit_cast(u32x4, g);
                    *reinterpret_cast<uint2*>(o) = make_uint2(__builtin_amdgcn_perm(u[1], u[0], 0x07060302u),
                                                              __builtin_amdgcn_perm(u[3], u[2], 0x07060302u));
                    *reinterpret_cast<uint2*>(o + plane) = make_uint2(__builtin_amdgcn_perm(u[1], u[0], 0x05040100u),
                                                                      __builtin_amdgcn_perm(u[3], u[2], 0x05040100u));
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t a = u[r] & 0x7fffffffu;
                        top[i][r] = max(top[i][r], a < 0x7f800000u ? a : 0u);
                    }
                }
            }
        }
        if constexpr (C::PLANES == 2) {
            // the tile's tokens' largest for each label: 16 lanes, then the waves
            float* part = reinterpret_cast<float*>(lds);  // [WN][BM]
#pragma unroll
            for (int i = 0; i < C::FM; ++i) {
                f32x4 m;
#pragma unroll
                for (int r = 0; r < 4; ++r) m[r] = __builtin_bit_cast(float, row_umax(top[i][r]));
                if ((lane & 15) == 15)
                    *reinterpret_cast<f32x4*>(part + (wave % C::WN) * C::BM + (wave / C::WN) * (C::BM / C::WM) + 16 * i +
                                              4 * (lane / 16)) = m;
            }
            __syncthreads();
            if (threadIdx.x < C::BM) {
                float m = part[threadIdx.x];
#pragma unroll
                for (int q = 1; q < C::WN; ++q) m = fmaxf(m, part[q * C::BM + threadIdx.x]);
                p.label_max[ni * p.piece + mi * C::BM + threadIdx.x] = m;
            }
        }
    }
}

// Tile `id` of grad_x: BM columns x BN tokens over part `split` of the piece's
// labels, into (or added to) the part's float32 sums.  The columns are the
// product's rows, so a lane holds four consecutive ones of a token.
template <typename C>
__device__ __forceinline__ void ce_grad_x_body(const TropCeParams& p, int64_t id, char* lds) {
    const int64_t kept = p.control->kept;
    const int64_t tm = (kept + C::BN - 1) / C::BN, tn = (p.width + C::BM - 1) / C::BM;
    int64_t mi, q;
    if (!ce_tile(id, tm, tn * p.splits, mi, q)) return;
    const int64_t ni = q % tn, split = q / tn;
    // (k tiles that hold a label: a part past them is empty, its sums zero)
    const int64_t ktiles = (min(p.piece, p.vocab - p.v0) + C::KT - 1) / C::KT;
    const int64_t kt0 = min(split * p.split_tiles, ktiles), kt1 = min(kt0 + p.split_tiles, ktiles);
    const int64_t k0 = kt0 * C::KT;
    MgOperand a, b;
    a.plane_bytes = 0;
    a.exp = 0;
    if constexpr (C::RAW) {
        a.base = static_cast<const char*>(p.w) + ((p.v0 + k0) * p.ldw + ni * C::BM) * 4;
        a.ld = p.ldw;
        a.last_row = (int32_t)((p.width - ni * C::BM) / 4 - 1);
        a.last_k = (int32_t)min(p.vocab - 1 - (p.v0 + k0), (int64_t)0x7fffffff);
        a.exp = p.control->w_exp;
    } else if (C::PLANES == 2 || p.w_packed) {
        a.ld = p.width_p * C::PLANES;
        a.base = static_cast<const char*>(p.wp) + (k0 * a.ld + ni * C::BM * C::PLANES) * 2;
        a.last_row = (int32_t)((p.width_p - ni * C::BM) * C::PLANES / 8 - 1);
        a.last_k = 0x7fffffff;
    } else {
        a.base = static_cast<const char*>(p.w) + ((p.v0 + k0) * p.ldw + ni * C::BM) * 2;
        a.ld = p.ldw;
        a.last_row = (int32_t)((p.width - ni * C::BM) / 8 - 1);
        a.last_k = (int32_t)min(p.vocab - 1 - (p.v0 + k0), (int64_t)0x7fffffff);
    }
    a.k_bytes = C::KT * a.ld * (C::RAW ? 4 : 2);
    b.base = static_cast<const char*>(p.g) + (k0 / 4 * p.padded + mi * C::BN) * 8;
    b.ld = p.padded;
    b.plane_bytes = p.piece * p.padded * 2;
    b.k_bytes = (C::KT / 4) * p.padded * 8;
    b.last_row = b.last_k = 0;
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int64_t c0 = ni * C::BM + (wave / C::WN) * (C::BM / C::WM) + 4 * (lane / 16);
    const int64_t n0 = mi * C::BN + (wave % C::WN) * (C::BN / C::WN) + (lane & 15);
    float scale[C::FN] = {};
    if constexpr (C::SCALED) {
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
            scale[j] = n0 + 16 * j < kept ? ldexpf(1.f, ce_token_exp(p.kept_grad[n0 + 16 * j])) : 0.f;
    }
    f32x4 acc[C::FM][C::FN];
    mg_walk<C>(acc, a, b, scale, (int)(kt1 - kt0), lds);
    float* out = p.gx_part + (split * p.padded + n0) * p.width_p + c0;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
        if (c0 + 16 * i >= p.width_p) continue;
#pragma unroll
        for (int j = 0; j < C::FN; ++j) {
            f32x4* o = reinterpret_cast<f32x4*>(out + (int64_t)(16 * j) * p.width_p + 16 * i);
            f32x4 v = acc[i][j];
            if (p.accumulate) {
                const f32x4 before = *o;
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] += before[r];
            }
            *o = v;
        }
    }
}

// The scales' exponents of a grad_w tile's labels (piece rows r0 + 16 j + lane
// % 16 of the wave's part): from the largest |G| that the logits' tiles left,
// by the whole workgroup.
template <typename C>
__device__ __forceinline__ void ce_label_exps(const TropCeParams& p, int64_t tile_row, int64_t kept, char* lds,
                                              int32_t (&e)[C::FN]) {
    float* part = reinterpret_cast<float*>(lds);  // [THREADS / BN][BN]
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int64_t row = tile_row + threadIdx.x % C::BN, tiles = (kept + p.logits_edge - 1) / p.logits_edge;
    float m = 0.f;
    if (row < p.piece) {
#pragma unroll 8
        for (int64_t t = threadIdx.x / C::BN; t < tiles; t += C::THREADS / C::BN)
            m = fmaxf(m, p.label_max[t * p.piece + row]);
    }
    part[threadIdx.x] = m;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        const int label = (wave % C::WN) * (C::BN / C::WN) + 16 * j + (lane & 15);
        m = part[label];
#pragma unroll
        for (int q = 1; q < C::THREADS / C::BN; ++q) m = fmaxf(m, part[q * C::BN + label]);
        e[j] = ce_column_exp(m);
    }
    __syncthreads();  // the walk's loads go to the same LDS
}

// Tile `id` of grad_w: BM columns x BN labels, the sum over the kept tokens, or
// over part `split` of them into the part's float32 sums (few tiles).
template <typename C, typename T>
__device__ __forceinline__ void ce_grad_w_body(const TropCeParams& p, int64_t id, char* lds) {
    const int64_t kept = p.control->kept;
    const int64_t tn = (p.width + C::BM - 1) / C::BM;
    int64_t mi, q;
    if (!ce_tile(id, (min(p.piece, p.vocab - p.v0) + C::BN - 1) / C::BN, tn * p.gw_splits, mi, q)) return;
    const int64_t ni = q % tn, split = q / tn;
    const int64_t ktiles = (kept + C::KT - 1) / C::KT, per = (ktiles + p.gw_splits - 1) / p.gw_splits;
    const int64_t kt0 = min(split * per, ktiles), kt1 = min(kt0 + per, ktiles), k0 = kt0 * C::KT;
    MgOperand a, b;
    a.ld = p.width_p * C::PLANES;
    a.base = static_cast<const char*>(p.xp) + (k0 * a.ld + ni * C::BM * C::PLANES) * 2;
    a.plane_bytes = 0;
    a.exp = 0;
    a.k_bytes = C::KT * a.ld * 2;
    a.last_row = (int32_t)((p.width_p - ni * C::BM) * C::PLANES / 8 - 1);
    a.last_k = 0x7fffffff;
    b.base = static_cast<const char*>(p.g) + (mi * (C::BN / 4) * p.padded + k0) * 8;
    b.ld = p.padded;
    b.plane_bytes = p.piece * p.padded * 2;
    b.k_bytes = C::KT * 8;
    b.last_row = b.last_k = 0;
    int32_t e[C::FN] = {};
    float scale[C::FN] = {};
    if constexpr (C::SCALED) {
        ce_label_exps<C>(p, mi * C::BN, kept, lds, e);
#pragma unroll
        for (int j = 0; j < C::FN; ++j) scale[j] = ldexpf(1.f, e[j]);
    }
    f32x4 acc[C::FM][C::FN];
    mg_walk<C>(acc, a, b, scale, (int)(kt1 - kt0), lds);
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int64_t c0 = ni * C::BM + (wave / C::WN) * (C::BM / C::WM) + 4 * (lane / 16);
    const int64_t v0 = p.v0 + mi * C::BN + (wave % C::WN) * (C::BN / C::WN) + (lane & 15);
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
        const int64_t v = v0 + 16 * j;
        if (v >= p.vocab) continue;
        const CeScale sum = ce_sum_scale<C::PLANES>(p, e[j], p.control->x_exp);
        if (C::SCALED && p.gw_splits > 1 && ni == 0 && split == 0 && wave / C::WN == 0 && lane < 16)
            p.label_exp[v - p.v0] = e[j];
        T* out = static_cast<T*>(p.grad_w) + v * p.ldgw;
        float* part = p.gw_part + (split * p.piece + (v - p.v0)) * p.width_p;
#pragma unroll
        for (int i = 0; i < C::FM; ++i) {
            if (c0 + 16 * i >= p.width) continue;
            if (p.gw_splits > 1) {
                *reinterpret_cast<f32x4*>(part + c0 + 16 * i) = acc[i][j];
            } else {
                FloatVec<4> g;
#pragma unroll
                for (int r = 0; r < 4; ++r) g[r] = sum(acc[i][j][r]);
                store_row<T, 4>(out, c0 + 16 * i, p.width, from_float<T, 4>(g));
            }
        }
    }
}

// Both gradients of a piece in one launch: neither reads what the other
// writes, and their tiles fill one another's last round of workgroups.
// Two launches against one: 256 x 512 x 8000 float32 36 and 25 us, 655 x 733 x
// 46669 float32 354 and 337, 8192 x 4096 x 65536 bfloat16 6.91 and 6.83 ms.
template <typename CX, typename CW, typename T>
__device__ __forceinline__ void ce_gradients_body(const TropCeParams& p, char* lds) {
    static_assert(CX::THREADS == CW::THREADS && CX::LDS_BYTES == CW::LDS_BYTES, "one launch");
    if (blockIdx.x < p.gx_groups)
        ce_grad_x_body<CX>(p, blockIdx.x, lds);
    else
        ce_grad_w_body<CW, T>(p, blockIdx.x - p.gx_groups, lds);
}

// Columns [c, c + 4) of a row summed over `splits` parts, `step` floats apart.
__device__ __forceinline__ FloatVec<4> ce_sum_parts(const float* q, int splits, int64_t step, CeScale scale) {
    FloatVec<4> s = load_vec<float, 4>(q);
#pragma unroll 8
    for (int k = 1; k < splits; ++k) {
        const FloatVec<4> o = load_vec<float, 4>(q + k * step);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] += o[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = scale(s[e]);
    return s;
}

// grad_x: the parts' sums in order, scaled; zeros for tokens that do not
// count.  A workgroup takes 1024 columns of a row (blockIdx.x = (row - row0)
// blocks + block).
template <typename T, int PLANES>
__device__ __forceinline__ void ce_finish_body(const TropCeParams& p) {
    const int64_t blocks = (p.width + 1023) / 1024;
    const int64_t n = p.row0 + blockIdx.x / blocks, c = (blockIdx.x % blocks) * 1024 + threadIdx.x * 4;
    if (c >= p.width) return;
    int64_t i = n;
    CeScale scale = {1.f, 0};
    if (p.identity) {
        if (!ce_counts(p, ce_target(p, n))) i = -1;
    } else {
        i = p.slot[n];
        const int32_t e = PLANES == 2 && i >= 0 ? ce_token_exp(p.kept_grad[i]) : 0;
        scale = ce_sum_scale<PLANES>(p, e, p.control->w_exp);
    }
    FloatVec<4> s = {0.f, 0.f, 0.f, 0.f};
    if (i >= 0) s = ce_sum_parts(p.gx_part + i * p.width_p + c, p.splits, p.padded * p.width_p, scale);
    store_row<T, 4>(static_cast<T*>(p.grad_x) + n * p.ldgx, c, p.width, from_float<T, 4>(s));
}

// grad_w of a piece from its parts, likewise.
template <typename T, int PLANES>
__device__ __forceinline__ void ce_finish_w_body(const TropCeParams& p) {
    const int64_t blocks = (p.width + 1023) / 1024;
    const int64_t r = blockIdx.x / blocks, c = (blockIdx.x % blocks) * 1024 + threadIdx.x * 4;
    if (c >= p.width) return;
    const CeScale scale = ce_sum_scale<PLANES>(p, PLANES == 2 ? p.label_exp[r] : 0, p.control->x_exp);
    const FloatVec<4> s = ce_sum_parts(p.gw_part + r * p.width_p + c, p.gw_splits, p.piece * p.width_p, scale);
    store_row<T, 4>(static_cast<T*>(p.grad_w) + (p.v0 + r) * p.ldgw, c, p.width, from_float<T, 4>(s));
}

// ---- few tokens ------------------------------------------------------------
// Up to 64 tokens (32 in bfloat16's backward and where w is large): w is
// streamed from HBM straight into the matrix instructions' registers, with no
// LDS copy and no packing.  The logits' pass reads it once; the backward reads
// it twice and writes grad_w.  They want many loads in flight: the four waves
// of a workgroup share its rows and split the sum.  One token is bound by w's
// bytes (4096 x 65536 bfloat16: 96 us, 5.6 TB/s); 16 tokens take 152 us on the
// same w, since every workgroup of 32 labels reads all of x too, 268 MB through
// the caches beside w's 537.  From 17 on the float32 matrix instructions take
// as long as the reads (26 tokens x 2560 x 58817 float32: logits 206 us, grad_x
// 135, grad_w 175, where w's bytes take 100 to 125).
//
// Logits: a workgroup takes 16 RF labels and all tokens (16 to a block
// column).  A lane reads 16 bytes of row lane % 16 at k chunk lane / 16, so
// a row's four lanes read 64 consecutive bytes.  float32 stays float32 (four
// 16x16x4 instructions per 16 k; the order of k within them is the same for
// both operands and otherwise free).  G is kept in float32, [label][16 NB].
template <typename T, int RF, int NB, CeEpilogue EPI>
__device__ __forceinline__ void ce_few_body(const TropCeParams& p) {
    constexpr int VEC = 16 / sizeof(T), KSTEP = 4 * VEC;
    // One unit of U steps is loaded while the one before is multiplied, where
    // the registers of both leave enough waves: 16 tokens x 4096 x 65536
    // bfloat16 193 -> 152 us, 30 x 2560 x 58817 bfloat16 100 -> 92; but 26 x
    // 2560 x 58817 float32 204 -> 225.
    constexpr bool AHEAD = NB == 1 || (NB == 2 && sizeof(T) == 2);
    constexpr int U = RF == 4 ? 2 : 4;
    using V = typename VecOf<T, VEC>::raw;
    __shared__ f32x4 sums[3][RF * NB][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int64_t v0 = p.v0 + (int64_t)blockIdx.x * 16 * RF;
    const T* wr[RF];
    const T* xr[NB];
#pragma unroll
    for (int i = 0; i < RF; ++i)
        wr[i] = static_cast<const T*>(p.w) + min(v0 + 16 * i + (lane & 15), p.vocab - 1) * p.ldw;
#pragma unroll
    for (int j = 0; j < NB; ++j)
        xr[j] = static_cast<const T*>(p.x) + min((int64_t)(16 * j + (lane & 15)), p.tokens - 1) * p.ldx;
    f32x4 acc[RF][NB] = {};
    auto step = [&](const V (&a)[RF], const V (&b)[NB]) {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < RF; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
        } else {  // (the sums in turn: an instruction waits for the one before it on its sum)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < RF; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i][e], b[j][e], acc[i][j], 0, 0, 0);
        }
    };
    const int kl = (lane / 16) * VEC;
    // Each workgroup starts its walk along the rows one unit (256 bytes)
    // after the one before it: rows are often a multiple of 8 KiB apart, and
    // workgroups in step would ask the same few memory channels (512 MiB of
    // 8 KiB rows: 93 us against 127).
    const int64_t units = p.width / (U * KSTEP), first = units ? blockIdx.x % units : 0;
    V a[AHEAD ? 2 : 1][U][RF], b[AHEAD ? 2 : 1][U][NB];
    auto load = [&](int buf, int64_t unit) {
        const int64_t at = unit + first < units ? unit + first : unit + first - units;
        const int64_t k = at * U * KSTEP + kl;
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < RF; ++i) a[buf][u][i] = load_vec<T, VEC>(wr[i] + k + u * KSTEP);
#pragma unroll
            for (int j = 0; j < NB; ++j) b[buf][u][j] = load_vec<T, VEC>(xr[j] + k + u * KSTEP);
        }
    };
    auto multiply = [&](int buf) {
#pragma unroll
        for (int u = 0; u < U; ++u) step(a[buf][u], b[buf][u]);
    };
    if constexpr (AHEAD) {
        // (the last unit again past the end; the scheduler would put the
        // loads off to save registers)
        const int64_t last = units - 1 - (units - 1 - wave) % 4;
        if (wave < units) load(0, wave);
        for (int64_t unit = wave; unit < units; unit += 8) {
            load(1, min(unit + 4, last));
            __builtin_amdgcn_sched_barrier(0);
            multiply(0);
            __builtin_amdgcn_sched_barrier(0);
            load(0, min(unit + 8, last));
            __builtin_amdgcn_sched_barrier(0);
            if (unit + 4 < units) multiply(1);
            __builtin_amdgcn_sched_barrier(0);
        }
    } else {
        for (int64_t unit = wave; unit < units; unit += 4) {
            load(0, unit);
            multiply(0);
        }
    }
    for (int64_t k = units * U * KSTEP + wave * KSTEP; k < p.width; k += 4 * KSTEP) {
        V a[RF], b[NB];
#pragma unroll
        for (int i = 0; i < RF; ++i) a[i] = load_row<T, VEC>(wr[i], k + kl, p.width);
#pragma unroll
        for (int j = 0; j < NB; ++j) b[j] = load_row<T, VEC>(xr[j], k + kl, p.width);
        step(a, b);
    }
    // the waves' sums, added in wave order by the first
    if (wave > 0) {
#pragma unroll
        for (int i = 0; i < RF; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) sums[wave - 1][i * NB + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int i = 0; i < RF; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const f32x4 o = sums[q][i * NB + j][lane];
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] += o[r];
            }
    // row 16 i + 4 (lane / 16) + r, column 16 j + lane % 16
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int64_t n = 16 * j + (lane & 15);
        const int64_t t = n < p.tokens ? ce_target(p, n) : -1;
        if constexpr (EPI == CE_STATS) {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < RF; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int64_t v = v0 + 16 * i + 4 * (lane / 16) + r;
                    if (v == t && v < p.vocab) p.target_logit[n] = acc[i][j][r];
                    if (v >= p.vocab) acc[i][j][r] = -INFINITY;
                    m = nan_max(m, acc[i][j][r]);
                }
            m = nan_max(m, __shfl_xor(m, 16, 64));
            m = nan_max(m, __shfl_xor(m, 32, 64));
            const float base = m == -INFINITY ? 0.f : m;
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < RF; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) s += ce_exp(acc[i][j][r] - base);
            s += __shfl_xor(s, 16, 64);
            s += __shfl_xor(s, 32, 64);
            if (lane < 16 && n < p.tokens)
                reinterpret_cast<float2*>(p.stats)[n * p.tiles + p.tile0 + blockIdx.x] = make_float2(m, s);
        } else {
            const bool on = n < p.tokens && ce_counts(p, t);
            const float lse = on ? p.lse_in[n] : 0.f;
            const float weight = on ? p.grad_loss[n * p.grad_loss_stride] : 0.f;
            float* out = static_cast<float*>(p.g) + (v0 - p.v0) * (16 * NB) + n;
#pragma unroll
            for (int i = 0; i < RF; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * i + 4 * (lane / 16) + r;
                    const float g = ce_exp(acc[i][j][r] - lse) - (v0 + row == t ? 1.f : 0.f);
                    out[(int64_t)row * (16 * NB)] = on && v0 + row < p.vocab ? g * weight : 0.f;
                }
        }
    }
}

// grad_x of all tokens, 16 DV columns to a workgroup, over part
// blockIdx.x / column blocks of the piece's labels: 16x16x4 float32
// instructions with k = label, so that a lane reads DV consecutive columns
// (16 bytes) of label lane / 16 and instruction j takes columns DV m + j as
// its rows m.  bfloat16 w is widened: the product is exact.  The four waves
// take 4 U labels in turn; their sums are added in wave order.
template <typename T, int NB>
__device__ __forceinline__ void ce_few_grad_x_body(const TropCeParams& p) {
    constexpr int DV = 16 / sizeof(T), U = 4, NP = 16 * NB;
    using V = typename VecOf<T, DV>::raw;
    __shared__ f32x4 sums[DV * NB][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int64_t blocks = (p.width + 16 * DV - 1) / (16 * DV);
    const int64_t split = blockIdx.x / blocks;
    const int64_t c = (blockIdx.x % blocks) * 16 * DV + (lane & 15) * DV;
    const int64_t labels = min(p.piece, p.vocab - p.v0), per = (int64_t)p.split_tiles * 4 * U * 4;
    const int64_t r0 = split * per, r1 = min(r0 + per, labels);
    const float* g = static_cast<const float*>(p.g) + (lane & 15);
    f32x4 acc[DV][NB] = {};
    // One round is loaded while another is multiplied (the scheduler kept from
    // putting that off): waves that all load and then all multiply add the two
    // times.  26, 60 tokens x 2560 x 58817 float32: 197 -> 136, 267 -> 206 us.
    auto walk = [&](auto whole) {
        V w[2][U];
        float b[2][U][NB];
        auto load = [&](int buf, int64_t r) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t row = min(r + 4 * u + lane / 16, labels - 1);
                const T* at = static_cast<const T*>(p.w) + (p.v0 + row) * p.ldw;
                if constexpr (decltype(whole)::value)
                    w[buf][u] = load_vec<T, DV>(at + c);
                else
                    w[buf][u] = load_row<T, DV>(at, c, p.width);
#pragma unroll
                for (int j = 0; j < NB; ++j) b[buf][u][j] = g[row * NP + 16 * j];
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        auto multiply = [&](int buf, int64_t r) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const FloatVec<DV> f = to_float<T, DV>(w[buf][u]);
                const bool on = r + 4 * u + lane / 16 < r1;  // a label past the part's end: its G taken as 0
#pragma unroll
                for (int d = 0; d < DV; ++d)
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        acc[d][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[d], on ? b[buf][u][j] : 0.f, acc[d][j], 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        constexpr int STEP = 4 * 4 * U;
        int64_t r = r0 + wave * 4 * U;
        if (r >= r1) return;
        load(0, r);
        for (; r < r1; r += 2 * STEP) {
            load(1, r + STEP);
            multiply(0, r);
            load(0, r + 2 * STEP);
            if (r + STEP < r1) multiply(1, r + STEP);
        }
    };
    if ((blockIdx.x % blocks + 1) * 16 * DV <= p.width)
        walk(std::true_type());
    else
        walk(std::false_type());
    for (int q = 1; q < 4; ++q) {
        __syncthreads();
        if (wave == q) {
#pragma unroll
            for (int d = 0; d < DV; ++d)
#pragma unroll
                for (int j = 0; j < NB; ++j) sums[d * NB + j][lane] = acc[d][j];
        }
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int d = 0; d < DV; ++d)
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const f32x4 o = sums[d * NB + j][lane];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[d][j][e] += o[e];
                }
        }
    }
    if (wave > 0) return;
    // instruction d, row 4 (lane / 16) + e, column lane % 16: columns
    // DV (4 (lane / 16) + e) + d of token 16 j + lane % 16
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int64_t n = 16 * j + (lane & 15);
        if (n >= p.tokens) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t col = (blockIdx.x % blocks) * 16 * DV + DV * (4 * (lane / 16) + e);
            if (col >= p.width_p) continue;
#pragma unroll
            for (int h = 0; h < DV; h += 4) {
                f32x4 v = {acc[h][j][e], acc[h + 1][j][e], acc[h + 2][j][e], acc[h + 3][j][e]};
                f32x4* o = reinterpret_cast<f32x4*>(p.gx_part + (split * p.padded + n) * p.width_p + col + h);
                if (p.accumulate) {
                    const f32x4 before = *o;
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] += before[q];
                }
                *o = v;
            }
        }
    }
}

// grad_w: a wave takes 16 VB labels and every (column parts)-th block of
// 16 DV columns; k = token, G stays in registers, x comes from the caches.
// Instruction d takes column d of chunk (m % 4) 4 + m / 4 (of DV columns) as
// its row m: a lane ends with chunk 4 e + lane / 16 in register e, so that a
// label's four lanes store 64 consecutive bytes.
template <typename T, int NB>
__device__ __forceinline__ void ce_few_grad_w_body(const TropCeParams& p) {
    constexpr int DV = 16 / sizeof(T), VB = 2, NP = 16 * NB;
    using V = typename VecOf<T, DV>::raw;
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int64_t labels = min(p.piece, p.vocab - p.v0);
    const int64_t groups = (labels + 64 * VB - 1) / (64 * VB);
    const int64_t part = blockIdx.x / groups, parts = gridDim.x / groups;
    const int64_t r0 = ((blockIdx.x % groups) * 4 + wave) * 16 * VB;
    if (r0 >= labels) return;
    const float* g = static_cast<const float*>(p.g);
    float b[VB][4 * NB];
    bool on[4 * NB];  // token lane / 16 + 4 s counts
    const int chunk = (lane & 3) * 4 + (lane & 15) / 4;
#pragma unroll
    for (int s = 0; s < 4 * NB; ++s) {
        const int64_t n = 4 * s + lane / 16;
        on[s] = n < p.tokens && ce_counts(p, ce_target(p, n));
#pragma unroll
        for (int i = 0; i < VB; ++i) {
            const int64_t row = r0 + 16 * i + (lane & 15);
            b[i][s] = row < labels ? g[row * NP + n] : 0.f;
        }
    }
    // (workgroups start at different columns, as in the logits' pass)
    const int64_t blocks = (p.width + 16 * DV - 1) / (16 * DV), mine = (blocks - part + parts - 1) / parts;
    for (int64_t k = 0; k < mine; ++k) {
        const int64_t c0 = (part + (k + blockIdx.x % groups) % mine * parts) * 16 * DV;
        f32x4 acc[DV][VB] = {};
#pragma unroll
        for (int s = 0; s < 4 * NB; ++s) {
            V x = {};
            if (on[s])
                x = load_row<T, DV>(static_cast<const T*>(p.x) + (4 * s + lane / 16) * p.ldx, c0 + chunk * DV, p.width);
            const FloatVec<DV> f = to_float<T, DV>(x);
#pragma unroll
            for (int d = 0; d < DV; ++d)
#pragma unroll
                for (int i = 0; i < VB; ++i)
                    acc[d][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[d], b[i][s], acc[d][i], 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < VB; ++i) {
            const int64_t row = r0 + 16 * i + (lane & 15);
            if (row >= labels) continue;
            T* out = static_cast<T*>(p.grad_w) + (p.v0 + row) * p.ldgw;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t col = c0 + DV * (4 * e + lane / 16);
                FloatVec<DV> v;
#pragma unroll
                for (int d = 0; d < DV; ++d) v[d] = acc[d][i][e];
                if (col < p.width) store_row<T, DV>(out, col, p.width, from_float<T, DV>(v));
            }
        }
    }
}

// ---- statistics joined -----------------------------------------------------
// A workgroup takes a token: its tiles' maxima and sums, then loss and lse.
__device__ __forceinline__ void ce_merge_body(const TropCeParams& p) {
    __shared__ float2 lds[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const int64_t i = blockIdx.x;
    const int64_t kept = p.identity ? p.tokens : (int64_t)p.control->kept;
    if (i >= kept) return;
    const int64_t n = p.identity ? i : (int64_t)p.rows[i];
    if (p.identity && !ce_counts(p, ce_target(p, n))) {
        if (threadIdx.x == 0) p.loss[n] = p.lse[n] = 0.f;
        return;
    }
    const float2* q = reinterpret_cast<const float2*>(p.stats) + i * p.tiles;
    float m = -INFINITY, s = 0.f;
#pragma unroll 4
    for (int64_t t = threadIdx.x; t < p.tiles; t += 256) {
        const float2 a = q[t];
        const float top = nan_max(m, a.x), base = top == -INFINITY ? 0.f : top;
        s = s * ce_exp(m - base) + a.y * ce_exp(a.x - base);
        m = top;
    }
    float top = wave_nan_max(m), base = top == -INFINITY ? 0.f : top;
    s = wave_sum(s * ce_exp(m - base));
    if (lane == 0) lds[wave] = make_float2(top, s);
    __syncthreads();
    if (threadIdx.x == 0) {
        m = nan_max(nan_max(lds[0].x, lds[1].x), nan_max(lds[2].x, lds[3].x));
        base = m == -INFINITY ? 0.f : m;
        s = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) s += lds[w].y * ce_exp(lds[w].x - base);
        const float lse = m + logf(s);
        p.lse[n] = lse;
        p.loss[n] = lse - p.target_logit[i];
    }
}

}  // namespace trop
