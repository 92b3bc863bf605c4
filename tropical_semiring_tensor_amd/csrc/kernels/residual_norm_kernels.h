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
// the row has several waves.  A slot is written again only after another
// reduction's barrier.
template <int TPR, int NVAL>
struct RowSums {
    float lds[TPR > 64 ? TPR / 64 : 1][NVAL];
};
template <int TPR, int NVAL>
__device__ __forceinline__ void row_sums(float (&v)[NVAL], RowSums<TPR, NVAL>& s) {
#pragma unroll
    for (int i = 0; i < NVAL; ++i) v[i] = wave_total(v[i]);
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x / 64;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < NVAL; ++i) s.lds[wave][i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NVAL; ++i) {
            v[i] = s.lds[0][i];
#pragma unroll
            for (int w = 1; w < TPR / 64; ++w) v[i] += s.lds[w][i];
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
    for (int i = 0; i < NV; ++i) x[i] = to_float<T, VEC>(load_row<T, VEC>(u, (int64_t)(i * TPR + t) * VEC, p.cols));
    if (p.r) {
        const T* res = static_cast<const T*>(p.r) + r * p.ldr;
#pragma unroll
        for (int i = 0; i < NV; ++i) raw[i] = load_row<T, VEC>(res, (int64_t)(i * TPR + t) * VEC, p.cols);
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
            if (c < p.cols) store_row<T, VEC>(h, c, p.cols, from_float<T, VEC>(x[i]));
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
            store_row<T, VEC>(y, c, p.cols, from_float<T, VEC>(o));
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
                                         int64_t r, int64_t c, int64_t n) {
        v = load_row_stream<T, VEC>(static_cast<const T*>(m) + r * ld, c, n);
    }
    __device__ __forceinline__ FloatVec<VEC> values() const { return to_float<T, VEC>(v); }
};
template <typename T, int VEC>
struct RnKept<T, VEC, true> {
    Act8Lane<VEC> v;
    __device__ __forceinline__ void load(const void*, int64_t, const int8_t* codes, int64_t ldc, const uint8_t* exps,
                                         int64_t lde, int64_t r, int64_t c, int64_t n) {
        v.load(codes + r * ldc, exps + r * lde, c, n);
    }
    __device__ __forceinline__ FloatVec<VEC> values() const { return v.values(); }
};

// The rows of part blockIdx.x, TPR threads to a row, 8 elements to a thread.
// A part inside a gate row: rows one by one, to the workgroup's row groups in
// turn (four waves, or one group).  A part of whole gate rows: those in turn,
// their rows one by one.
template <typename T, typename P, int TPR, bool HELD>
__device__ __forceinline__ void residual_norm_backward_body(const TropResidualParams& p) {
    constexpr int VEC = ln_vec<T>(), NV = 8 / VEC, RPB = TPR == 64 ? 4 : 1;
    // the weights' registers, where there are enough
    constexpr bool KEEP = TPR < 1024;
    __shared__ RowSums<TPR, 2> sums[2][2];
    __shared__ float cols_lds[TPR == 64 ? TROP_RN_COLS_WAVE : 1];
    const int t = threadIdx.x % TPR, group = RPB == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / TPR);
    float acc[TROP_RN_SUMS][NV * VEC] = {};
    typename VecOf<T, VEC>::raw dyv[NV], dhv[NV];
    RnKept<T, VEC, HELD> hv[NV], uv[NV];
    float pre_mean = 0.f, pre_rstd = 1.f, post_mean = 0.f, post_rstd = 1.f;
    const bool need_u = p.need_v || p.need_post;
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * TPR + t) * VEC;
            if (p.pre) {
                dyv[i] = load_row_stream<T, VEC>(static_cast<const T*>(p.dy) + r * p.lddy, c, p.cols);
                hv[i].load(p.h, p.ldh, p.h_codes, p.ldh_codes, p.h_exps, p.ldh_exps, r, c, p.cols);
            }
            if (p.dh) dhv[i] = load_row_stream<T, VEC>(static_cast<const T*>(p.dh) + r * p.lddh, c, p.cols);
            if (need_u) uv[i].load(p.u, p.ldu, p.u_codes, p.ldu_codes, p.u_exps, p.ldu_exps, r, c, p.cols);
        }
        if (p.pre) {
            if (p.pre == RN_LAYER) pre_mean = p.pre_mean[r];
            pre_rstd = p.pre_rstd[r];
        }
        if (p.post && need_u) {
            if (p.post == RN_LAYER) post_mean = p.post_mean[r];
            post_rstd = p.post_rstd[r];
        }
    };
    FloatVec<VEC> pre_g[NV], post_g[NV], post_b[NV], gate[NV];
    auto weights = [&](bool pre) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * TPR + t) * VEC;
            if (pre) {
                pre_g[i] = load_param<P, VEC>(p.pre_gamma, c, p.cols, 1.f);
            } else {
                post_g[i] = load_param<P, VEC>(p.post_gamma, c, p.cols, 1.f);
                post_b[i] = load_param<P, VEC>(p.post_beta, c, p.cols, 0.f);
            }
        }
    };
    if constexpr (KEEP) {
        weights(true);
        weights(false);
    }
    // this row group's rows: `units` of unit_rows, `stride` units apart
    const bool whole = p.group_parts == 0;
    const int64_t unit_rows = whole ? p.gate_group : 1;
    int64_t first, end, gate_row;  // rows of the part
    if (whole) {
        first = blockIdx.x * p.part_rows;
        end = min(first + p.part_rows, p.rows);
        gate_row = 0;
    } else {
        gate_row = rn_divide(blockIdx.x, p.group_parts);
        const int64_t q = blockIdx.x - gate_row * p.group_parts, last = min((gate_row + 1) * p.gate_group, p.rows);
        first = min(gate_row * p.gate_group + q * p.part_rows, last);
        end = min(first + p.part_rows, last);
    }
    int slot = 0;
    int64_t unit = first + group * unit_rows, r = unit, unit_end = min(unit + unit_rows, end);
    bool new_gate = true;
    if (whole && r < end) gate_row = rn_divide(r, p.gate_group);
    if (r < end) fetch(r);
    while (r < end) {  // the groups of a workgroup share barriers only when RPB = 1
        if (new_gate) {
#pragma unroll
            for (int i = 0; i < NV; ++i) gate[i] = rn_gate<T, VEC>(p, gate_row, (int64_t)(i * TPR + t) * VEC);
            new_gate = false;
        }
        const int64_t row = r;
        // the row after this one
        bool flush = false;
        int64_t next_gate = gate_row;
        if (++r == unit_end) {
            flush = whole;
            unit += RPB * unit_rows;
            r = unit;
            unit_end = min(unit + unit_rows, end);
            if (whole) next_gate = gate_row + RPB;
        }
        FloatVec<VEC> H[NV], x[NV], w[NV];
        float s[2] = {0.f, 0.f};
        const float mean1 = pre_mean, rstd1 = pre_rstd, mean2 = post_mean, rstd2 = post_rstd;
        if constexpr (!KEEP) weights(true);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * TPR + t) * VEC;
            if (p.dh)
                H[i] = to_float<T, VEC>(dhv[i]);
            else
                H[i] = FloatVec<VEC>(0.f);
            if (p.pre) {
                const FloatVec<VEC> h = hv[i].values(), dy = to_float<T, VEC>(dyv[i]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    // past the row's end everything is held to zero, so that a
                    // non-finite statistic or weight adds nothing there
                    const float xx = c + e < p.cols ? (h[e] - mean1) * rstd1 : 0.f;
                    const float ww = c + e < p.cols ? dy[e] * pre_g[i][e] : 0.f;
                    x[i][e] = xx;
                    w[i][e] = ww;
                    acc[TROP_RN_PRE_GAMMA][i * VEC + e] = __builtin_fmaf(dy[e], xx, acc[TROP_RN_PRE_GAMMA][i * VEC + e]);
                    acc[TROP_RN_PRE_BETA][i * VEC + e] += dy[e];
                    s[0] += ww;
                    s[1] = __builtin_fmaf(ww, xx, s[1]);
                }
            }
        }
        FloatVec<VEC> u[NV];
        if (need_u) {
#pragma unroll
            for (int i = 0; i < NV; ++i) u[i] = uv[i].values();
        }
        if (r < end) fetch(r);
        if (p.pre) {
            row_sums<TPR, 2>(s, sums[slot][0]);
            const float c1 = p.pre == RN_LAYER ? s[0] * p.inv_cols : 0.f, c2 = s[1] * p.inv_cols;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * TPR + t) * VEC;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float d = __builtin_fmaf(__builtin_fmaf(-c2, x[i][e], w[i][e] - c1), rstd1, H[i][e]);
                    H[i][e] = c + e < p.cols ? d : 0.f;
                }
            }
        }
        if (p.dr) {
            T* dr = static_cast<T*>(p.dr) + row * p.lddr;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * TPR + t) * VEC;
                FloatVec<VEC> o;
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = H[i][e] * p.residual_scale;
                if (c < p.cols) store_row_stream<T, VEC>(dr, c, p.cols, from_float<T, VEC>(o));
            }
        }
        if constexpr (!KEEP) {
            if (p.post) weights(false);
        }
        if (need_u && p.post) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * TPR + t) * VEC;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    x[i][e] = c + e < p.cols ? (u[i][e] - mean2) * rstd2 : 0.f;
                    u[i][e] = c + e < p.cols ? __builtin_fmaf(x[i][e], post_g[i][e], post_b[i][e]) : 0.f;
                }
            }
        }
        if (p.need_v) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    acc[TROP_RN_GATE][i * VEC + e] = __builtin_fmaf(H[i][e], u[i][e], acc[TROP_RN_GATE][i * VEC + e]);
        }
        float c1 = 0.f, c2 = 0.f;
        if (p.need_post) {
            s[0] = s[1] = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * TPR + t) * VEC;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float dv = c + e < p.cols ? H[i][e] * gate[i][e] : 0.f;
                    const float ww = c + e < p.cols ? dv * post_g[i][e] : 0.f;
                    w[i][e] = ww;
                    acc[TROP_RN_POST_GAMMA][i * VEC + e] =
                        __builtin_fmaf(dv, x[i][e], acc[TROP_RN_POST_GAMMA][i * VEC + e]);
                    acc[TROP_RN_POST_BETA][i * VEC + e] += dv;
                    s[0] += ww;
                    s[1] = __builtin_fmaf(ww, x[i][e], s[1]);
                }
            }
            row_sums<TPR, 2>(s, sums[slot][1]);
            c1 = p.post == RN_LAYER ? s[0] * p.inv_cols : 0.f;
            c2 = s[1] * p.inv_cols;
        }
        slot ^= 1;
        if (p.du) {
            T* du = static_cast<T*>(p.du) + row * p.lddu;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * TPR + t) * VEC;
                FloatVec<VEC> o;
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    o[e] = p.post ? __builtin_fmaf(-c2, x[i][e], w[i][e] - c1) * rstd2 : H[i][e] * gate[i][e];
                if (c < p.cols) store_row_stream<T, VEC>(du, c, p.cols, from_float<T, VEC>(o));
            }
        }
        if (flush) {
            if (p.dgate) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int64_t c = (int64_t)(i * TPR + t) * VEC;
                    FloatVec<VEC> o;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        o[e] = acc[TROP_RN_GATE][i * VEC + e] * p.branch_scale;
                        acc[TROP_RN_GATE][i * VEC + e] = 0.f;
                    }
                    if (c >= p.cols) continue;
                    if (sizeof(T) == 4 || p.gate_f32)
                        store_row_stream<float, VEC>(static_cast<float*>(p.dgate) + gate_row * p.lddgate, c, p.cols, o);
                    else
                        store_row_stream<T, VEC>(static_cast<T*>(p.dgate) + gate_row * p.lddgate, c, p.cols,
                                                 from_float<T, VEC>(o));
                }
            }
            gate_row = next_gate;
            new_gate = true;
        }
    }
#pragma unroll
    for (int k = 0; k < TROP_RN_SUMS; ++k) {
        if (!p.part[k]) continue;
        float* out = p.part[k] + (int64_t)blockIdx.x * p.cols;
        if constexpr (TPR == 64) {  // the four waves' sums, added in wave order
            for (int wv = 0; wv < 4; ++wv) {
                if (group == wv) {
#pragma unroll
                    for (int i = 0; i < NV; ++i)
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            const int c = (i * TPR + t) * VEC + e;
                            cols_lds[c] = wv ? cols_lds[c] + acc[k][i * VEC + e] : acc[k][i * VEC + e];
                        }
                }
                __syncthreads();
            }
            for (int c = threadIdx.x; c < p.cols; c += 256) out[c] = cols_lds[c];
            __syncthreads();
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * TPR + t) * VEC;
                FloatVec<VEC> o;
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = acc[k][i * VEC + e];
                if (c < p.cols) store_row<float, VEC>(out, c, p.cols, o);
            }
        }
    }
}

// u or h of a row, elements [c, c + VEC) as values.
template <typename T, int VEC, bool HELD>
__device__ __forceinline__ FloatVec<VEC> rn_kept(const void* m, int64_t ld, const int8_t* codes, int64_t ldc,
                                                 const uint8_t* exps, int64_t lde, int64_t r, int64_t c, int64_t n) {
    RnKept<T, VEC, HELD> k;
    k.load(m, ld, codes, ldc, exps, lde, r, c, n);
    return k.values();
}

// Rows wider than the registers: a walk for the pre norm's means, kept for the
// column sums; one for the post norm's, which writes dr (and du without a post
// norm); one for du.
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

// Sums of parts.  A workgroup takes 64 columns of an output row, 16 waves the
// parts wave, wave + 16, ...; the waves' sums are added in wave order.
template <typename T>
__device__ __forceinline__ void part_sums_body(const TropRowSumsParams& p) {
    __shared__ float lds[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const uint32_t id = (uint32_t)p.id0 + blockIdx.x;
    int k = 0;
    while (k + 1 < p.count && id >= p.e[k].blocks) ++k;
    const TropRowSumsEntry& e = p.e[k];
    const uint32_t at = id - (k ? p.e[k - 1].blocks : 0), columns = (uint32_t)((p.cols + 63) / 64);
    const int64_t row = at / columns, c = (int64_t)(at % columns) * 64 + lane;
    float s = 0.f;
    if (c < p.cols) {
        const float* q = e.src + row * e.parts * p.cols + c;
#pragma unroll 4
        for (int64_t i = wave; i < e.parts; i += 16) s += q[i * p.cols];
    }
    lds[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < p.cols) {
        float a = lds[0][lane];
#pragma unroll
        for (int w = 1; w < 16; ++w) a += lds[w][lane];
        a *= e.scale;
        if (e.f32)
            static_cast<float*>(e.dst)[row * e.ldd + c] = a;
        else
            static_cast<T*>(e.dst)[row * e.ldd + c] = (T)a;
    }
}

}  // namespace trop
