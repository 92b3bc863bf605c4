// Between two residual blocks: the norm after a block, its gate, the residual
// sum and the norm before the next block, forward and backward.
//
//   v = post norm of u,  h = residual_scale r + (branch_scale gate) v,
//   y = pre norm of h
//
// Apart, these are four passes that move 13 elements for every one of h; fused
// they move the 4 (forward: r, u, h, y) or 6 (backward: dy, dh, h, u, dr, du)
// that they cannot do without, and are bound by HBM.  A row stays in registers
// between its reductions: forward at most four in turn (both means, both sums
// of squares about them), backward two of two sums each.
//
// Backward, for a row: with x^ = (h - mean) rstd and w = dy gamma,
//   H = dh + rstd (w - mean(w) - x^ mean(w x^)),  dr = residual_scale H
//   dv = branch_scale gate H, and the same through the post norm to du.
// The sums over rows (gradients of both norms' weights, of the gate) are kept
// by the thread that holds the column, for the rows of its workgroup's part: a
// run of rows inside one gate row, or several whole gate rows, whose gradient
// it then writes by itself.  The parts' sums are added in order by a second
// kernel: no atomics, the same bits every time.
//
// Measured (one MI355X; a large copy moves 5.0 TB/s): 16384 x 4096 bfloat16, u
// and h kept in 8 bits, 675 MB each way: forward with a gate and a pre norm
// 119-124 us (5.5-5.7 TB/s), backward with a post norm as well 131-135 us
// (5.0-5.2) and 6 us for the parts' sums.  1537 x 1001 float32: forward 9 us (25
// MB), backward 16 + 6 us (28 MB; 406 parts of four rows, latency).  One row of
// 4096: 4 us, the way from the load through two norms' reductions to the store.
//
// Row groups: forward 16 elements to a thread, which reaches the copy's rate;
// backward 8 (float32 rows of 512 to 2048 columns 4), since a thread holds dy,
// dh, h and u of its next row besides its columns' sums: bfloat16 rows then fit
// 128 registers, four waves to a SIMD (16384 x 4096: 152 us, with three waves
// 186, before later steps).
#pragma once
#include "act8_kernels.h"
#include "layer_norm_kernels.h"

namespace trop {

enum { RN_NONE = 0, RN_LAYER = 1, RN_RMS = 2 };  // trop_norm

// Sum over the wave (every lane gets it), by DPP steps: rows of 16 by
// shifts, then across the rows.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
    return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float wave_total(float x) {
    x = dpp_add<0x111>(x);  // row_shr:1
    x = dpp_add<0x112>(x);  // row_shr:2
    x = dpp_add<0x114>(x);  // row_shr:4
    x = dpp_add<0x118>(x);  // row_shr:8
    x = dpp_add<0x142>(x);  // row_bcast:15
    x = dpp_add<0x143>(x);  // row_bcast:31
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

// Sums over the TPR threads of a row, by way of an LDS slot of their own when
// the row has several waves: each wave then reads one wave's sum to a lane and
// adds them across its lanes, so the sums end in scalar registers.  A slot is
// written again only after another reduction's barrier.
template <int TPR, int NVAL>
struct RowSums {
    float lds[NVAL][TPR > 64 ? TPR / 64 : 1];
};
template <int TPR, int NVAL>
__device__ __forceinline__ void row_sums(float (&v)[NVAL], RowSums<TPR, NVAL>& s) {
#pragma unroll
    for (int i = 0; i < NVAL; ++i) v[i] = wave_total(v[i]);
    if constexpr (TPR > 64) {
        constexpr int WAVES = TPR / 64;
        static_assert(WAVES == 2 || WAVES == 4 || WAVES == 8 || WAVES == 16, "steps below");
        const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < NVAL; ++i) s.lds[i][wave] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NVAL; ++i) {
            float x = dpp_add<0x111>(s.lds[i][lane & (WAVES - 1)]);  // row_shr:1
            if constexpr (WAVES > 2) x = dpp_add<0x112>(x);          // row_shr:2
            if constexpr (WAVES > 4) x = dpp_add<0x114>(x);          // row_shr:4
            if constexpr (WAVES > 8) x = dpp_add<0x118>(x);          // row_shr:8
            v[i] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), WAVES - 1));
        }
    }
}

__device__ __forceinline__ int64_t rn_divide(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
__device__ __forceinline__ int64_t rn_gate_row(const TropResidualParams& p, int64_t r) {
    return p.gate_group >= p.rows ? 0 : rn_divide(r, p.gate_group);
}
// branch_scale gate, elements [c, c + VEC) of a gate row.
template <typename T, int VEC>
__device__ __forceinline__ FloatVec<VEC> rn_gate(const TropResidualParams& p, int64_t row, int64_t c) {
    FloatVec<VEC> g;
    if (!p.gate)
        g = FloatVec<VEC>(1.f);
    else if (sizeof(T) == 4 || p.gate_f32)
        g = load_row<float, VEC>(static_cast<const float*>(p.gate) + row * p.ldgate, c, p.cols);
    else
        g = to_float<T, VEC>(load_row<T, VEC>(static_cast<const T*>(p.gate) + row * p.ldgate, c, p.cols));
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] *= p.branch_scale;
    return g;
}

// Row r of a matrix, a uniform pointer in scalar registers, and element c of
// it, by a 32-bit byte offset that the load takes as it is.  Both are hidden
// from the compiler, which would rather add each lane's column to the base
// before the loop over the rows and keep 64-bit lane addresses (60 registers
// of a backward's 190).
template <typename T>
__device__ __forceinline__ T* rn_row(T* base, int64_t r, int64_t ld) {
    auto row = (__attribute__((address_space(1))) T*)(base + r * ld);
    asm("" : "+s"(row));
    return (T*)row;
}
// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ float rn_scalar(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}
template <typename T>
__device__ __forceinline__ T* rn_at(T* row, uint32_t c) {
    uint32_t offset = c * (uint32_t)sizeof(T);
    asm volatile("" : "+v"(offset));
    return (T*)((__attribute__((address_space(1))) char*)(__attribute__((address_space(1))) T*)row + offset);
}
// The same, and norm weights, where the whole vector is inside the row.
template <typename T, int VEC>
__device__ __forceinline__ FloatVec<VEC> rn_gate_full(const TropResidualParams& p, int64_t row, uint32_t c) {
    FloatVec<VEC> g;
    if (!p.gate)
        g = FloatVec<VEC>(1.f);
    else if (sizeof(T) == 4 || p.gate_f32)
        g = load_vec<float, VEC>(rn_at(rn_row(static_cast<const float*>(p.gate), row, p.ldgate), c));
    else
        g = to_float<T, VEC>(load_vec<T, VEC>(rn_at(rn_row(static_cast<const T*>(p.gate), row, p.ldgate), c)));
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] *= p.branch_scale;
    return g;
}
template <int VEC>
__device__ __forceinline__ FloatVec<VEC> rn_weight(const TropResidualParams& p, const void* w, uint32_t c, float other) {
    if (!w) return FloatVec<VEC>(other);
    if (p.weight_f32) return load_vec<float, VEC>(rn_at(rn_row(static_cast<const float*>(w), 0, 0), c));
    return to_float<bf16, VEC>(load_vec<bf16, VEC>(rn_at(rn_row(static_cast<const bf16*>(w), 0, 0), c)));
}

// A row's statistics: mean (0 for RMS) and rstd of x, whose elements past the
// row's end are zero.  The sum of squares is taken about the mean.
template <int TPR, int VEC, int NV>
__device__ __forceinline__ void rn_statistics(const TropResidualParams& p, const FloatVec<VEC> (&x)[NV], int t,
                                              bool layer, float eps, float& mean, float& rstd,
                                              RowSums<TPR, 1> (&sums)[2]) {
    float s[1] = {0.f};
    mean = 0.f;
    if (layer) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[0] += x[i][e];
        row_sums<TPR, 1>(s, sums[0]);
        mean = s[0] * p.inv_cols;
        s[0] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t)(i * TPR + t) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float d = c + e < p.cols ? x[i][e] - mean : 0.f;
            s[0] = __builtin_fmaf(d, d, s[0]);
        }
    }
    row_sums<TPR, 1>(s, sums[1]);
    rstd = 1.0f / sqrtf(s[0] * p.inv_cols + eps);
}

// Rows are read and written past the caches' reuse order: 16384 x 4096 bfloat16
// with u and h left in 8 bits 137 us otherwise, so 124.  What reads y next may
// find less of it in the caches.  Streaming stores of h and y against ordinary
// ones, us, pairs in a graph; alone, then with an elementwise reader of y behind
// it, then with a product by a square matrix (bfloat16 but for the last):
//   16384 x 4096, 8 bits left   130 136   184 186   555 558
//   16384 x 4096                102 100   143 137   529 526
//   4096 x 4096, 8 bits left     40  39    51  49   149 148
//   4096 x 4096                  30  31    43  41   141 139
//   1 x 4096                    3.8 3.8   5.7 5.4    20  20
//   1537 x 1001 float32         8.0 8.1  11.5 12.5   44  45
// Ahead where 8-bit rows are left of a large batch and in float32, a few percent
// behind elsewhere; one form serves all.
template <typename T, typename P, int TPR>
__device__ __forceinline__ void residual_norm_forward_body(const TropResidualParams& p) {
    constexpr int VEC = ln_vec<T>(), NV = 16 / VEC, RPB = TPR == 64 ? 4 : 1;
    __shared__ RowSums<TPR, 1> sums[4];
    const int t = threadIdx.x % TPR;
    const int64_t r = p.row0 + (int64_t)blockIdx.x * RPB + __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
    if (r >= p.rows) return;  // whole waves, and only where no barrier follows (TPR = 64)
    typename VecOf<T, VEC>::raw raw[NV];
    FloatVec<VEC> x[NV], gate[NV];
    const T* u = static_cast<const T*>(p.u) + r * p.ldu;
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = to_float<T, VEC>(load_row_stream<T, VEC>(u, (int64_t)(i * TPR + t) * VEC, p.cols));
    if (p.r) {
        const T* res = static_cast<const T*>(p.r) + r * p.ldr;
#pragma unroll
        for (int i = 0; i < NV; ++i) raw[i] = load_row_stream<T, VEC>(res, (int64_t)(i * TPR + t) * VEC, p.cols);
    }
    const int64_t gate_row = rn_gate_row(p, r);
#pragma unroll
    for (int i = 0; i < NV; ++i) gate[i] = rn_gate<T, VEC>(p, gate_row, (int64_t)(i * TPR + t) * VEC);
    if (p.u_codes) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            act8_store<VEC>(p.u_codes + r * p.ldu_codes, p.u_exps + r * p.ldu_exps, (int64_t)(i * TPR + t) * VEC, p.cols,
                            x[i]);
    }
    float mean, rstd;
    if (p.post) {
        rn_statistics<TPR, VEC, NV>(p, x, t, p.post == RN_LAYER, p.post_eps, mean, rstd,
                                    reinterpret_cast<RowSums<TPR, 1>(&)[2]>(sums[0]));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * TPR + t) * VEC;
            const FloatVec<VEC> g = load_param<P, VEC>(p.post_gamma, c, p.cols, 1.f);
            const FloatVec<VEC> b = load_param<P, VEC>(p.post_beta, c, p.cols, 0.f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[i][e] = __builtin_fmaf((x[i][e] - mean) * rstd, g[e], b[e]);
        }
        if (t == 0) {
            if (p.post_mean && p.post == RN_LAYER) p.post_mean[r] = mean;
            if (p.post_rstd) p.post_rstd[r] = rstd;
        }
    }
    // (products and sum apart: without a post norm h then depends on nothing
    // but the inputs' bits, and h8 with it)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t)(i * TPR + t) * VEC;
        const FloatVec<VEC> res = to_float<T, VEC>(raw[i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float h = gate[i][e] * x[i][e];
            if (p.r) h = res[e] * p.residual_scale + h;
            x[i][e] = c + e < p.cols ? h : 0.f;
        }
    }
    if (p.h_codes) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            act8_store<VEC>(p.h_codes + r * p.ldh_codes, p.h_exps + r * p.ldh_exps, (int64_t)(i * TPR + t) * VEC, p.cols,
                            x[i]);
    }
    if (p.h) {
        T* h = static_cast<T*>(p.h) + r * p.ldh;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * TPR + t) * VEC;
            if (c < p.cols) store_row_stream<T, VEC>(h, c, p.cols, from_float<T, VEC>(x[i]));
        }
    }
    if (!p.pre) return;
    rn_statistics<TPR, VEC, NV>(p, x, t, p.pre == RN_LAYER, p.pre_eps, mean, rstd,
                                reinterpret_cast<RowSums<TPR, 1>(&)[2]>(sums[2]));
    if (t == 0) {
        if (p.pre_mean && p.pre == RN_LAYER) p.pre_mean[r] = mean;
        if (p.pre_rstd) p.pre_rstd[r] = rstd;
    }
    if (!p.y) return;
    T* y = static_cast<T*>(p.y) + r * p.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t)(i * TPR + t) * VEC;
        if (c < p.cols) {
            const FloatVec<VEC> g = load_param<P, VEC>(p.pre_gamma, c, p.cols, 1.f);
            const FloatVec<VEC> b = load_param<P, VEC>(p.pre_beta, c, p.cols, 0.f);
            FloatVec<VEC> o;
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = __builtin_fmaf((x[i][e] - mean) * rstd, g[e], b[e]);
            store_row_stream<T, VEC>(y, c, p.cols, from_float<T, VEC>(o));
        }
    }
}

// Rows wider than the registers: a walk for each statistic and one that
// writes; h is made again from r and u in each (the row stays in the XCD's L2),
// and r is last read where h is written, so h may be r.
template <typename T, typename P>
__device__ __forceinline__ void residual_norm_forward_loop_body(const TropResidualParams& p) {
    constexpr int VEC = ln_vec<T>(), TPR = 1024;
    __shared__ RowSums<TPR, 1> sums[4];
    const int64_t r = p.row0 + blockIdx.x, gate_row = rn_gate_row(p, r);
    const T* u = static_cast<const T*>(p.u) + r * p.ldu;
    float mean[2] = {0.f, 0.f}, rstd[2] = {1.f, 1.f};  // post, pre
    auto load_u = [&](int64_t c) { return to_float<T, VEC>(load_row<T, VEC>(u, c, p.cols)); };
    auto load_h = [&](int64_t c) {
        FloatVec<VEC> x = load_u(c);
        if (p.post) {
            const FloatVec<VEC> g = load_param<P, VEC>(p.post_gamma, c, p.cols, 1.f);
            const FloatVec<VEC> b = load_param<P, VEC>(p.post_beta, c, p.cols, 0.f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[e] = __builtin_fmaf((x[e] - mean[0]) * rstd[0], g[e], b[e]);
        }
        const FloatVec<VEC> gate = rn_gate<T, VEC>(p, gate_row, c);
        FloatVec<VEC> res = FloatVec<VEC>(0.f);
        if (p.r) res = to_float<T, VEC>(load_row<T, VEC>(static_cast<const T*>(p.r) + r * p.ldr, c, p.cols));
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float h = gate[e] * x[e];
            if (p.r) h = res[e] * p.residual_scale + h;
            x[e] = c + e < p.cols ? h : 0.f;
        }
        return x;
    };
    // (every lane walks to the same end: blocks of 8-bit codes span lanes)
    auto statistics = [&](auto load, bool layer, float eps, int which) {
        float s[1] = {0.f};
        if (layer) {
            for (int64_t at = 0; at < p.cols; at += TPR * VEC) {
                const FloatVec<VEC> x = load(at + (int64_t)threadIdx.x * VEC);
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[0] += x[e];
            }
            row_sums<TPR, 1>(s, sums[2 * which]);
            mean[which] = s[0] * p.inv_cols;
            s[0] = 0.f;
        }
        for (int64_t at = 0; at < p.cols; at += TPR * VEC) {
            const int64_t c = at + (int64_t)threadIdx.x * VEC;
            const FloatVec<VEC> x = load(c);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = c + e < p.cols ? x[e] - mean[which] : 0.f;
                s[0] = __builtin_fmaf(d, d, s[0]);
            }
        }
        row_sums<TPR, 1>(s, sums[2 * which + 1]);
        rstd[which] = 1.0f / sqrtf(s[0] * p.inv_cols + eps);
    };
    if (p.post) statistics(load_u, p.post == RN_LAYER, p.post_eps, 0);
    if (p.pre) statistics(load_h, p.pre == RN_LAYER, p.pre_eps, 1);
    if (threadIdx.x == 0) {
        if (p.post_mean && p.post == RN_LAYER) p.post_mean[r] = mean[0];
        if (p.post_rstd && p.post) p.post_rstd[r] = rstd[0];
        if (p.pre_mean && p.pre == RN_LAYER) p.pre_mean[r] = mean[1];
        if (p.pre_rstd && p.pre) p.pre_rstd[r] = rstd[1];
    }
    for (int64_t at = 0; at < p.cols; at += TPR * VEC) {
        const int64_t c = at + (int64_t)threadIdx.x * VEC;
        if (p.u_codes)
            act8_store<VEC>(p.u_codes + r * p.ldu_codes, p.u_exps + r * p.ldu_exps, c, p.cols, load_u(c));
        const FloatVec<VEC> h = load_h(c);
        if (p.h_codes) act8_store<VEC>(p.h_codes + r * p.ldh_codes, p.h_exps + r * p.ldh_exps, c, p.cols, h);
        if (c >= p.cols) continue;
        if (p.h) store_row<T, VEC>(static_cast<T*>(p.h) + r * p.ldh, c, p.cols, from_float<T, VEC>(h));
        if (p.y) {
            const FloatVec<VEC> g = load_param<P, VEC>(p.pre_gamma, c, p.cols, 1.f);
            const FloatVec<VEC> b = load_param<P, VEC>(p.pre_beta, c, p.cols, 0.f);
            FloatVec<VEC> o;
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = __builtin_fmaf((h[e] - mean[1]) * rstd[1], g[e], b[e]);
            store_row<T, VEC>(static_cast<T*>(p.y) + r * p.ldy, c, p.cols, from_float<T, VEC>(o));
        }
    }
}

// ---- backward ----------------------------------------------------------------

// What a lane holds of u or h: elements as they are, or 8-bit codes.
template <typename T, int VEC, bool HELD>
struct RnKept {
    typename VecOf<T, VEC>::raw v;
    __device__ __forceinline__ void load(const void* m, int64_t ld, const int8_t*, int64_t, const uint8_t*, int64_t,
                                         int64_t r, uint32_t c, bool) {
        v = load_stream<T, VEC>(rn_at(rn_row(static_cast<const T*>(m), r, ld), c));
    }
    // the values less `mean`
    __device__ __forceinline__ FloatVec<VEC> about(float mean, uint32_t, bool) const {
        FloatVec<VEC> x = to_float<T, VEC>(v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] -= mean;
        return x;
    }
};
template <typename T, int VEC>
struct RnKept<T, VEC, true> {
    CodeWords<VEC> codes;
    // Exponents of the first element and, in rows that end inside a vector
    // (`ragged`: the last vectors may lie across two blocks), of the last.  Kept
    // as the bytes they are: put together, or widened, they would be waited
    // for where they are loaded, a row ahead of their use (16384 x 1024
    // bfloat16 57 us against 49).
    uint8_t first, last;
    __device__ __forceinline__ void load(const void*, int64_t, const int8_t* m, int64_t ldc, const uint8_t* e,
                                         int64_t lde, int64_t r, uint32_t c, bool ragged) {
        codes = __builtin_bit_cast(CodeWords<VEC>, load_stream<int8_t, VEC>(rn_at(rn_row(m, r, ldc), c)));
        const uint8_t* row = rn_row(e, r, lde);
        first = *rn_at(row, c / TROP_ACT8_BLOCK_ELEMS);
        if (ragged) last = *rn_at(row, (c + VEC - 1) / TROP_ACT8_BLOCK_ELEMS);
    }
    __device__ __forceinline__ FloatVec<VEC> about(float mean, uint32_t c, bool ragged) const {
        const float step = act8_step(first);
        const FloatVec<VEC> q = __builtin_convertvector(__builtin_bit_cast(Codes<VEC>, codes), FloatVec<VEC>);
        FloatVec<VEC> x;
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] = __builtin_fmaf(q[e], step, -mean);  // (the product is exact)
        if (ragged) {
            int split = TROP_ACT8_BLOCK_ELEMS - (int)(c % TROP_ACT8_BLOCK_ELEMS);
            asm volatile("" : "+v"(split));  // (the comparisons are not to be kept over the rows)
            if (split < VEC) {  // a block ends inside the vector
                const float other = act8_step(last);
                CodeWords<VEC> again;  // (converted anew: no registers for it elsewhere)
#pragma unroll
                for (int i = 0; i < VEC / 4; ++i) {
                    uint32_t word = codes[i];
                    asm volatile("" : "+v"(word));
                    again[i] = word;
                }
                const FloatVec<VEC> q1 = __builtin_convertvector(__builtin_bit_cast(Codes<VEC>, again), FloatVec<VEC>);
#pragma unroll
                for (int e = 1; e < VEC; ++e)
                    if (e >= split) x[e] = __builtin_fmaf(q1[e], other, -mean);
            }
        }
        return x;
    }
};

// What a kernel does with its rows: everything; for rows too wide to keep their
// sums in registers, the rows' gradients (and the pre norm's two means, left for
// the sums); their sums, each workgroup TPR EPT columns of a part's rows.
enum RnWork { RN_ALL, RN_ROWS, RN_COLUMNS };

// The rows of part blockIdx.x, TPR threads to a row, EPT elements to a thread
// in vectors of 16 bytes.  A part inside a gate row: rows one by one, to the
// workgroup's row groups in turn (four waves, or one group).  A part of whole
// gate rows: those in turn, their rows one by one.
//
// A vector that would pass the row's end lies at the end instead: its first
// elements, which the lane before holds too, come to the same bits in both and
// are stored twice; only the row's sums leave them out.  So no load or store
// is taken apart.  Lanes past the end repeat the last vector and store nothing.
//
// Within a gate row the gate, gamma and beta are constants of a column, so two
// sums serve three gradients: with A = sum H x^ and B = sum H,
//   dgamma = gate A,  dbeta = gate B,  dgate = gamma A + beta B
// (all but the scales).  A part of whole gate rows adds up the first two in
// LDS, a slot to each thread, whenever a gate row ends.
template <typename T, int TPR, int EPT, bool HELD, bool PRE, bool POST, RnWork WORK>
__device__ __forceinline__ void residual_norm_backward_body(const TropResidualParams& p) {
    constexpr int VEC = ln_vec<T>(), NV = EPT / VEC, RPB = TPR == 64 ? 4 : 1, THREADS = TPR * RPB;
    using V = typename VecOf<T, VEC>::raw;
    __shared__ RowSums<TPR, 2> sums[2][2];
    constexpr bool SUMS = WORK != RN_ROWS, ROWS = WORK != RN_COLUMNS;
    // Weights and gate stay in registers where there are enough: not with 16
    // elements to a thread, nor in float32 with 1024 threads (128 registers each;
    // 4096 x 8192: 183 us kept and spilled, 156 read again for each row).
    constexpr bool KEEP = EPT <= 8 && !(TPR == 1024 && sizeof(T) == 4);
    __shared__ float post_lds[POST && SUMS ? 2 : 1][POST && SUMS ? EPT : 1][THREADS];
    __shared__ float cols_lds[TPR == 64 ? 4 : 1][TPR == 64 ? TPR * EPT : 1];
    const int t = threadIdx.x % TPR, group = RPB == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
    const int cols = (int)p.cols;
    int part = blockIdx.x, col0 = 0;
    if constexpr (!ROWS) {
        const int block = (int)p.col0 + part / p.parts;
        part %= p.parts;
        col0 = block * (TPR * EPT);
    }
    uint32_t at[NV];
    int dup[NV];  // first column; elements of the vector that the lane before holds
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = col0 + (i * TPR + t) * VEC;
        at[i] = min(c, cols - VEC);
        dup[i] = c - (int)at[i];
    }
    // sums of dy x^ and dy; A and B
    float pg[SUMS ? EPT : 1] = {}, pb[SUMS ? EPT : 1] = {}, sa[SUMS ? EPT : 1] = {}, sb[SUMS ? EPT : 1] = {};
    V dyv[NV], dhv[NV] = {};
    RnKept<T, VEC, HELD> hv[NV], uv[NV];
    float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f, c1_row = 0.f, c2_row = 0.f;
    const bool need_u = POST || (SUMS && p.need_v);
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (PRE) {
                dyv[i] = load_stream<T, VEC>(rn_at(rn_row(static_cast<const T*>(p.dy), r, p.lddy), at[i]));
                hv[i].load(p.h, p.ldh, p.h_codes, p.ldh_codes, p.h_exps, p.ldh_exps, r, at[i], p.ragged);
            }
            if (!PRE || p.dh) dhv[i] = load_stream<T, VEC>(rn_at(rn_row(static_cast<const T*>(p.dh), r, p.lddh), at[i]));
            if (need_u) uv[i].load(p.u, p.ldu, p.u_codes, p.ldu_codes, p.u_exps, p.ldu_exps, r, at[i], p.ragged);
        }
        if constexpr (PRE) {
            if (p.pre_mean) mean1 = p.pre_mean[r];
            rstd1 = p.pre_rstd[r];
            if (!ROWS && p.row_sums) {  // (not there where no sum needs H)
                c1_row = p.row_sums[2 * r];
                c2_row = p.row_sums[2 * r + 1];
            }
        }
        if constexpr (POST) {
            if (p.post_mean) mean2 = p.post_mean[r];
            rstd2 = p.post_rstd[r];
        }
    };
    FloatVec<VEC> pre_g[NV], gg[NV];  // gamma of the pre norm; branch_scale gate, times gamma of the post norm
    auto weights = [&](bool pre, bool post, int64_t gate_row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (pre && PRE) pre_g[i] = rn_weight<VEC>(p, p.pre_gamma, at[i], 1.f);
            if (!post) continue;
            gg[i] = rn_gate_full<T, VEC>(p, gate_row, at[i]);
            if constexpr (POST) {
                const FloatVec<VEC> g = rn_weight<VEC>(p, p.post_gamma, at[i], 1.f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) gg[i][e] *= g[e];
            }
        }
    };
    // this row group's rows: units of unit_rows, RPB units apart
    const bool whole = p.group_parts == 0;
    const int64_t unit_rows = whole ? p.gate_group : 1;
    int64_t first, end, gate_row;  // rows of the part
    if (whole) {
        first = part * p.part_rows;
        end = min(first + p.part_rows, p.rows);
        gate_row = 0;
    } else {
        gate_row = rn_divide(part, p.group_parts);
        const int64_t q = part - gate_row * p.group_parts, last = min((gate_row + 1) * p.gate_group, p.rows);
        first = min(gate_row * p.gate_group + q * p.part_rows, last);
        end = min(first + p.part_rows, last);
    }
    int64_t unit = first + group * unit_rows, r = unit, unit_end = min(unit + unit_rows, end);
    if (whole && r < end) gate_row = rn_divide(r, p.gate_group);
    if (KEEP && r < end) weights(true, false, 0);
    if (r < end) fetch(r);
    if (whole) {
        if constexpr (POST && SUMS) {
#pragma unroll
            for (int e = 0; e < EPT; ++e) post_lds[0][e][threadIdx.x] = post_lds[1][e][threadIdx.x] = 0.f;
        }
    }
    // Sums of w and w x over the row, without the elements held twice.
    auto add = [&](float (&s)[2], const FloatVec<VEC>& w, const FloatVec<VEC>& x, int d) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            a += w[e];
            b = __builtin_fmaf(w[e], x[e], b);
        }
        if (cols < TPR * EPT) {
            asm volatile("" : "+v"(d));  // (the comparisons are not to be kept over the rows)
            if (d > 0) {
                a = b = 0.f;
#pragma unroll
                for (int e = 1; e < VEC; ++e)
                    if (e >= d) {
                        a += w[e];
                        b = __builtin_fmaf(w[e], x[e], b);
                    }
            }
        }
        s[0] += a;
        s[1] += b;
    };
    int slot = 0;
    bool new_gate = true;
    while (r < end) {  // the groups of a workgroup share barriers only when RPB = 1
        if (KEEP && new_gate) {
            weights(false, true, gate_row);
            new_gate = false;
        }
        const int64_t row = r;
        bool flush = false;
        if (++r == unit_end) {  // the row after this one
            flush = whole;
            unit += RPB * unit_rows;
            r = unit;
            unit_end = min(unit + unit_rows, end);
        }
        FloatVec<VEC> H[NV], x[NV], w[NV], u[NV];
        RnKept<T, VEC, HELD> uraw[NV];
        float s[2] = {0.f, 0.f};
        const float mu1 = rn_scalar(mean1), rs1 = rn_scalar(rstd1), mu2 = rn_scalar(mean2), rs2 = rn_scalar(rstd2);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            H[i] = to_float<T, VEC>(dhv[i]);
            if constexpr (PRE) {
                const FloatVec<VEC> dy = to_float<T, VEC>(dyv[i]);
                x[i] = hv[i].about(mu1, at[i], p.ragged);
                if constexpr (!KEEP) pre_g[i] = rn_weight<VEC>(p, p.pre_gamma, at[i], 1.f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    x[i][e] *= rs1;
                    w[i][e] = dy[e] * pre_g[i][e];
                    if constexpr (SUMS) {
                        pg[i * VEC + e] = __builtin_fmaf(dy[e], x[i][e], pg[i * VEC + e]);
                        pb[i * VEC + e] += dy[e];
                    }
                }
                if constexpr (ROWS) add(s, w[i], x[i], dup[i]);
            }
            uraw[i] = uv[i];
        }
        float c1 = rn_scalar(c1_row), c2 = rn_scalar(c2_row);
        if (r < end) fetch(r);
        if constexpr (PRE) {
            if constexpr (ROWS) {
                row_sums<TPR, 2>(s, sums[slot][0]);
                c1 = p.pre == RN_LAYER ? s[0] * p.inv_cols : 0.f;
                c2 = s[1] * p.inv_cols;
                if (WORK == RN_ROWS && p.row_sums && t == 0) {
                    p.row_sums[2 * row] = c1;
                    p.row_sums[2 * row + 1] = c2;
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    H[i][e] = __builtin_fmaf(__builtin_fmaf(-c2, x[i][e], w[i][e] - c1), rs1, H[i][e]);
        }
        if (ROWS && p.dr) {
            T* dr = rn_row(static_cast<T*>(p.dr), row, p.lddr);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                FloatVec<VEC> o;
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = H[i][e] * p.residual_scale;
                if (dup[i] < VEC) store_stream<T, VEC>(rn_at(dr, at[i]), from_float<T, VEC>(o));
            }
        }
        if (need_u) {
#pragma unroll
            for (int i = 0; i < NV; ++i) u[i] = uraw[i].about(mu2, at[i], p.ragged);
            if constexpr (POST) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) u[i][e] *= rs2;
            }
            if constexpr (SUMS) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) sa[i * VEC + e] = __builtin_fmaf(H[i][e], u[i][e], sa[i * VEC + e]);
            }
        }
        if constexpr (!KEEP) weights(false, true, gate_row);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                if constexpr (POST && SUMS) sb[i * VEC + e] += H[i][e];
                if constexpr (ROWS) w[i][e] = H[i][e] * gg[i][e];
            }
        if constexpr (POST && ROWS) {
            s[0] = s[1] = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) add(s, w[i], u[i], dup[i]);
            row_sums<TPR, 2>(s, sums[slot][1]);
            c1 = p.post == RN_LAYER ? s[0] * p.inv_cols : 0.f;
            c2 = s[1] * p.inv_cols;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) w[i][e] = __builtin_fmaf(-c2, u[i][e], w[i][e] - c1) * rs2;
        }
        slot ^= 1;
        if (ROWS && p.du) {
            T* du = rn_row(static_cast<T*>(p.du), row, p.lddu);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (dup[i] < VEC) store_stream<T, VEC>(rn_at(du, at[i]), from_float<T, VEC>(w[i]));
        }
        if (flush) {
            if constexpr (SUMS) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const FloatVec<VEC> gs = rn_gate_full<T, VEC>(p, gate_row, at[i]);
                    const FloatVec<VEC> g = rn_weight<VEC>(p, p.post_gamma, at[i], 1.f);
                    const FloatVec<VEC> b = rn_weight<VEC>(p, p.post_beta, at[i], 0.f);
                    FloatVec<VEC> o;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int k = i * VEC + e;
                        o[e] = (g[e] * sa[k] + b[e] * sb[k]) * p.branch_scale;
                        if constexpr (POST) {
                            post_lds[0][k][threadIdx.x] += gs[e] * sa[k];
                            post_lds[1][k][threadIdx.x] += gs[e] * sb[k];
                        }
                        sa[k] = sb[k] = 0.f;
                    }
                    if (p.dgate && dup[i] < VEC) {
                        if (sizeof(T) == 4 || p.gate_f32)
                            store_vec<float, VEC>(rn_at(rn_row(static_cast<float*>(p.dgate), gate_row, p.lddgate), at[i]), o);
                        else
                            store_vec<T, VEC>(rn_at(rn_row(static_cast<T*>(p.dgate), gate_row, p.lddgate), at[i]),
                                              from_float<T, VEC>(o));
                    }
                }
            }
            gate_row += RPB;
            new_gate = true;
        }
    }
    if constexpr (SUMS) {
        // this part's sums
        auto leave = [&](float* out, const float (&v)[EPT]) {
            if (!out) return;
            out += (int64_t)part * cols;
            if constexpr (TPR == 64) {  // the four waves' sums, added in wave order
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    FloatVec<VEC> o;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o[e] = v[i * VEC + e];
                    if (dup[i] < VEC) store_vec<float, VEC>(&cols_lds[group][at[i]], o);
                }
                __syncthreads();
                for (int c = threadIdx.x; c < cols; c += 256)
                    out[c] = cols_lds[0][c] + cols_lds[1][c] + cols_lds[2][c] + cols_lds[3][c];
                __syncthreads();
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    FloatVec<VEC> o;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o[e] = v[i * VEC + e];
                    if (dup[i] < VEC) store_vec<float, VEC>(rn_at(out, at[i]), o);
                }
            }
        };
        if constexpr (PRE) {
            leave(p.part[TROP_RN_PRE_GAMMA], pg);
            leave(p.part[TROP_RN_PRE_BETA], pb);
        }
        if (!p.part[TROP_RN_POST_GAMMA] && !p.part[TROP_RN_POST_BETA] && !p.part[TROP_RN_GATE]) return;
        if (whole) {
            if constexpr (POST) {
#pragma unroll
                for (int e = 0; e < EPT; ++e) {
                    sa[e] = post_lds[0][e][threadIdx.x];
                    sb[e] = post_lds[1][e][threadIdx.x];
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const FloatVec<VEC> gs = rn_gate_full<T, VEC>(p, gate_row, at[i]);
                const FloatVec<VEC> g = rn_weight<VEC>(p, p.post_gamma, at[i], 1.f);
                const FloatVec<VEC> b = rn_weight<VEC>(p, p.post_beta, at[i], 0.f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int k = i * VEC + e;
                    pg[k] = g[e] * sa[k] + b[e] * sb[k];
                    sa[k] *= gs[e];
                    sb[k] *= gs[e];
                }
            }
            leave(p.part[TROP_RN_GATE], pg);
        }
        if constexpr (POST) {
            leave(p.part[TROP_RN_POST_GAMMA], sa);
            leave(p.part[TROP_RN_POST_BETA], sb);
        }
    }
}

// u or h of a row, elements [c, c + VEC) (VEC 1 or c a multiple of it) as
// values, zeros past its end.
template <typename T, int VEC, bool HELD>
__device__ __forceinline__ FloatVec<VEC> rn_kept(const void* m, int64_t ld, const int8_t* codes, int64_t ldc,
                                                 const uint8_t* exps, int64_t lde, int64_t r, int64_t c, int64_t n) {
    if constexpr (HELD) {
        Act8Lane<VEC> k;
        k.load(codes + r * ldc, exps + r * lde, c, n);
        return k.values();
    } else {
        return to_float<T, VEC>(load_row<T, VEC>(static_cast<const T*>(m) + r * ld, c, n));
    }
}

// Rows wider than that, narrower than a vector, or without a norm: a walk for
// the pre norm's means, kept for the column sums; one for the post norm's,
// which writes dr (and du without a post norm); one for du.
template <typename T, typename P, bool HELD>
__device__ __forceinline__ void residual_norm_backward_loop_body(const TropResidualParams& p) {
    constexpr int VEC = ln_vec<T>(), TPR = 1024;
    __shared__ RowSums<TPR, 2> sums[2];
    const int64_t r = p.row0 + blockIdx.x, gate_row = rn_gate_row(p, r);
    float mean1 = 0.f, rstd1 = 1.f, mean2 = 0.f, rstd2 = 1.f, c1 = 0.f, c2 = 0.f;
    const T* dy = static_cast<const T*>(p.dy) + r * p.lddy;
    const T* dh = static_cast<const T*>(p.dh) + r * p.lddh;
    auto load_x = [&](int64_t c) {
        FloatVec<VEC> x = rn_kept<T, VEC, HELD>(p.h, p.ldh, p.h_codes, p.ldh_codes, p.h_exps, p.ldh_exps, r, c, p.cols);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] = c + e < p.cols ? (x[e] - mean1) * rstd1 : 0.f;
        return x;
    };
    auto load_w = [&](int64_t c) {
        FloatVec<VEC> w = to_float<T, VEC>(load_row<T, VEC>(dy, c, p.cols));
        const FloatVec<VEC> g = load_param<P, VEC>(p.pre_gamma, c, p.cols, 1.f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = c + e < p.cols ? w[e] * g[e] : 0.f;
        return w;
    };
    if (p.pre) {
        if (p.pre == RN_LAYER) mean1 = p.pre_mean[r];
        rstd1 = p.pre_rstd[r];
        float s[2] = {0.f, 0.f};
        for (int64_t c = (int64_t)threadIdx.x * VEC; c < p.cols; c += TPR * VEC) {
            const FloatVec<VEC> x = load_x(c), w = load_w(c);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s[0] += w[e];
                s[1] = __builtin_fmaf(w[e], x[e], s[1]);
            }
        }
        row_sums<TPR, 2>(s, sums[0]);
        c1 = p.pre == RN_LAYER ? s[0] * p.inv_cols : 0.f;
        c2 = s[1] * p.inv_cols;
        if (threadIdx.x == 0 && p.row_sums) {
            p.row_sums[2 * r] = c1;
            p.row_sums[2 * r + 1] = c2;
        }
    }
    if (!p.dr && !p.du) return;
    auto load_H = [&](int64_t c) {
        FloatVec<VEC> H = FloatVec<VEC>(0.f);
        if (p.dh) H = to_float<T, VEC>(load_row<T, VEC>(dh, c, p.cols));
        if (p.pre) {
            const FloatVec<VEC> x = load_x(c), w = load_w(c);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                H[e] = __builtin_fmaf(__builtin_fmaf(-c2, x[e], w[e] - c1), rstd1, H[e]);
        }
        return H;
    };
    if (p.post && p.du) {
        if (p.post == RN_LAYER) mean2 = p.post_mean[r];
        rstd2 = p.post_rstd[r];
    }
    auto load_u = [&](int64_t c) {
        FloatVec<VEC> x = rn_kept<T, VEC, HELD>(p.u, p.ldu, p.u_codes, p.ldu_codes, p.u_exps, p.ldu_exps, r, c, p.cols);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] = c + e < p.cols ? (x[e] - mean2) * rstd2 : 0.f;
        return x;
    };
    float s[2] = {0.f, 0.f};
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < p.cols; c += TPR * VEC) {
        const FloatVec<VEC> H = load_H(c);
        FloatVec<VEC> o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = H[e] * p.residual_scale;
        if (p.dr) store_row<T, VEC>(static_cast<T*>(p.dr) + r * p.lddr, c, p.cols, from_float<T, VEC>(o));
        if (!p.du) continue;
        const FloatVec<VEC> gate = rn_gate<T, VEC>(p, gate_row, c);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = H[e] * gate[e];
        if (!p.post) {
            store_row<T, VEC>(static_cast<T*>(p.du) + r * p.lddu, c, p.cols, from_float<T, VEC>(o));
            continue;
        }
        const FloatVec<VEC> g = load_param<P, VEC>(p.post_gamma, c, p.cols, 1.f), x = load_u(c);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float w = c + e < p.cols ? o[e] * g[e] : 0.f;
            s[0] += w;
            s[1] = __builtin_fmaf(w, x[e], s[1]);
        }
    }
    if (!p.post || !p.du) return;
    row_sums<TPR, 2>(s, sums[1]);
    const float d1 = p.post == RN_LAYER ? s[0] * p.inv_cols : 0.f, d2 = s[1] * p.inv_cols;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < p.cols; c += TPR * VEC) {
        const FloatVec<VEC> H = load_H(c), gate = rn_gate<T, VEC>(p, gate_row, c), x = load_u(c);
        const FloatVec<VEC> g = load_param<P, VEC>(p.post_gamma, c, p.cols, 1.f);
        FloatVec<VEC> o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = __builtin_fmaf(-d2, x[e], H[e] * gate[e] * g[e] - d1) * rstd2;
        store_row<T, VEC>(static_cast<T*>(p.du) + r * p.lddu, c, p.cols, from_float<T, VEC>(o));
    }
}

// Column sums of wide rows, after their rows: a thread keeps a column for the
// rows of a part.  blockIdx.x = part + parts * (256-column block, from col0 on).
template <typename T, typename P, bool HELD>
__device__ __forceinline__ void residual_norm_columns_body(const TropResidualParams& p) {
    const int64_t block = rn_divide(blockIdx.x, p.parts), part = blockIdx.x - block * p.parts;
    const int64_t c = p.col0 + block * 256 + threadIdx.x;
    if (c >= p.cols) return;
    const bool whole = p.group_parts == 0;
    int64_t first, end, gate_row;
    if (whole) {
        first = part * p.part_rows;
        end = min(first + p.part_rows, p.rows);
        gate_row = rn_divide(first, p.gate_group);
    } else {
        gate_row = rn_divide(part, p.group_parts);
        const int64_t q = part - gate_row * p.group_parts, last = min((gate_row + 1) * p.gate_group, p.rows);
        first = min(gate_row * p.gate_group + q * p.part_rows, last);
        end = min(first + p.part_rows, last);
    }
    const float pre_g = load_param<P, 1>(p.pre_gamma, c, p.cols, 1.f)[0];
    const float post_g = load_param<P, 1>(p.post_gamma, c, p.cols, 1.f)[0];
    const float post_b = load_param<P, 1>(p.post_beta, c, p.cols, 0.f)[0];
    float acc[TROP_RN_SUMS] = {};
    float gate = 0.f;
    int64_t gate_end = first;  // (the first row reads its gate)
    const bool need_u = p.need_v || p.need_post;
    for (int64_t r = first; r < end; ++r) {
        if (r == gate_end || r == first) {
            gate = rn_gate<T, 1>(p, gate_row, c)[0];
            gate_end = whole ? min(r + p.gate_group, end) : end;
        }
        float H = p.dh ? (float)static_cast<const T*>(p.dh)[r * p.lddh + c] : 0.f;
        if (p.pre) {
            const float dy = (float)static_cast<const T*>(p.dy)[r * p.lddy + c], rstd = p.pre_rstd[r];
            const float h =
                rn_kept<T, 1, HELD>(p.h, p.ldh, p.h_codes, p.ldh_codes, p.h_exps, p.ldh_exps, r, c, p.cols)[0];
            const float x = (h - (p.pre == RN_LAYER ? p.pre_mean[r] : 0.f)) * rstd;
            acc[TROP_RN_PRE_GAMMA] = __builtin_fmaf(dy, x, acc[TROP_RN_PRE_GAMMA]);
            acc[TROP_RN_PRE_BETA] += dy;
            if (need_u)
                H = __builtin_fmaf(__builtin_fmaf(-p.row_sums[2 * r + 1], x, dy * pre_g - p.row_sums[2 * r]), rstd, H);
        }
        if (need_u) {
            float u = rn_kept<T, 1, HELD>(p.u, p.ldu, p.u_codes, p.ldu_codes, p.u_exps, p.ldu_exps, r, c, p.cols)[0];
            if (p.post) {
                const float x = (u - (p.post == RN_LAYER ? p.post_mean[r] : 0.f)) * p.post_rstd[r], dv = H * gate;
                acc[TROP_RN_POST_GAMMA] = __builtin_fmaf(dv, x, acc[TROP_RN_POST_GAMMA]);
                acc[TROP_RN_POST_BETA] += dv;
                u = __builtin_fmaf(x, post_g, post_b);
            }
            acc[TROP_RN_GATE] = __builtin_fmaf(H, u, acc[TROP_RN_GATE]);
        }
        if (whole && r + 1 == gate_end) {
            if (p.dgate) {
                const float o = acc[TROP_RN_GATE] * p.branch_scale;
                if (sizeof(T) == 4 || p.gate_f32)
                    static_cast<float*>(p.dgate)[gate_row * p.lddgate + c] = o;
                else
                    static_cast<T*>(p.dgate)[gate_row * p.lddgate + c] = (T)o;
            }
            acc[TROP_RN_GATE] = 0.f;
            ++gate_row;
        }
    }
#pragma unroll
    for (int k = 0; k < TROP_RN_SUMS; ++k)
        if (p.part[k]) p.part[k][part * p.cols + c] = acc[k];
}

// Sums of parts.  A workgroup takes 2^column_bits columns of an output row and
// shares the parts out among its 1024 / 2^column_bits groups of threads (group g
// adds parts g, g + groups, ...), whose sums are added pairwise: few columns
// where there are many parts, so that no thread has many loads in a row.
template <typename T>
__device__ __forceinline__ void part_sums_body(const TropRowSumsParams& p) {
    __shared__ float lds[1024];
    const uint32_t id = (uint32_t)p.id0 + blockIdx.x;
    int k = 0;
    while (k + 1 < p.count && id >= p.e[k].blocks) ++k;
    const TropRowSumsEntry& e = p.e[k];
    const int bits = e.column_bits, width = 1 << bits, groups = 1024 >> bits;
    const uint32_t at = id - (k ? p.e[k - 1].blocks : 0), columns = (uint32_t)((p.cols + width - 1) >> bits);
    const int64_t row = at / columns, c = ((int64_t)(at % columns) << bits) + (threadIdx.x & (width - 1));
    float s = 0.f;
    if (c < p.cols) {
        const float* q = e.src + row * e.parts * p.cols + c;
#pragma unroll 8
        for (int64_t i = threadIdx.x >> bits; i < e.parts; i += groups) s += q[i * p.cols];
    }
    lds[threadIdx.x] = s;
    for (int n = 512; n >= width; n >>= 1) {
        __syncthreads();
        if ((int)threadIdx.x < n) lds[threadIdx.x] = s = s + lds[threadIdx.x + n];
    }
    if ((int)threadIdx.x < width && c < p.cols) {
        s *= e.scale;
        if (e.f32)
            static_cast<float*>(e.dst)[row * e.ldd + c] = s;
        else
            static_cast<T*>(e.dst)[row * e.ldd + c] = (T)s;
    }
}

}  // namespace trop
