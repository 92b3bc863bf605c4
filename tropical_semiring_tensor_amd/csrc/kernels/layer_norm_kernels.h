// Layer norm forward and backward.
//
// Both passes move each element once and do a few operations on it, so they
// are bound by HBM; the design keeps a row in registers between its
// reductions and its output (one read of x, one write of y), and keeps
// enough rows in flight per CU to cover the memory latency.
//
//   forward   mean, then the variance about the mean from the registers (no
//             cancellation), then y
//   backward  with h = (x - mean) rstd, w = dy gamma:
//             dx = rstd (w - mean(w) - h mean(w h));
//             dgamma = sum_r dy h, dbeta = sum_r dy
//
// A group of TPR threads takes a row, 16 elements per thread in 16-byte
// vectors: a wave up to 1024 columns (four rows per workgroup, no barrier),
// 256 threads up to 4096, 1024 threads up to 16384.  Wider rows are read
// once per pass by the looping forms.  In the backward a thread keeps its
// columns for every row its workgroup takes, so dgamma and dbeta are summed
// in its registers; the workgroups' partial sums ([2][parts][cols]) are
// added in order by a second kernel: no atomics, the same bits every time.
// The backward streams x, dy and dx past the caches (forward and backward of
// 16384 x 4096 bfloat16 in turn: 48 + 72 us against 51 + 78); the forward
// does not gain from it, and its y is read next.  Those 48 and 72 us move 268
// and 403 MB at 5.6 TB/s, the partial sums' merge takes 4.5 us more; a large
// copy reaches 4.7 TB/s, a read 6.  1537 x 1001 float32 (a wave to a row): 5.7,
// 8.8 and 4.0 us; one row of 4096 bfloat16 3.2 us, all of it latency.
#pragma once
#include "train_common.h"

namespace trop {

// Sum over the TPR threads of a row group (every thread gets it).  TPR > 64:
// two LDS slots per value taken in turn (`slot`), so that one barrier per
// reduction is enough: a wave can be at most one reduction ahead of another.
template <int TPR, int NVAL>
__device__ __forceinline__ void group_sum(float (&v)[NVAL], float (*lds)[NVAL][TPR > 64 ? TPR / 64 : 1], int slot) {
#pragma unroll
    for (int i = 0; i < NVAL; ++i) v[i] = wave_sum(v[i]);
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x / 64, lane = threadIdx.x & 63;
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < NVAL; ++i) lds[slot][i][wave] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NVAL; ++i) {
            float s = lds[slot][i][0];
#pragma unroll
            for (int w = 1; w < TPR / 64; ++w) s += lds[slot][i][w];
            v[i] = s;
        }
    }
}

template <typename T>
constexpr int ln_vec() {
    return 16 / sizeof(T);
}

template <typename P, int N>
__device__ __forceinline__ FloatVec<N> load_param(const void* p, int64_t c, int64_t n, float other) {
    if (!p) return FloatVec<N>(other);
    return to_float<P, N>(load_row<P, N>(static_cast<const P*>(p), c, n));
}

template <typename T, typename P, int TPR>
__device__ __forceinline__ void layer_norm_forward_body(const TropLayerNormParams& p) {
    constexpr int VEC = ln_vec<T>(), NV = 16 / VEC, RPB = TPR == 64 ? 4 : 1;
    __shared__ float red[2][1][TPR > 64 ? TPR / 64 : 1];
    const int t = threadIdx.x % TPR;
    const int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    if (r >= p.rows) return;  // whole waves, and only where no barrier follows (TPR = 64)
    const T* x = static_cast<const T*>(p.x) + r * p.ldx;
    FloatVec<VEC> v[NV];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        v[i] = to_float<T, VEC>(load_row<T, VEC>(x, (int64_t)(i * TPR + t) * VEC, p.cols));
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[0] += v[i][e];
    }
    group_sum<TPR, 1>(s, red, 0);
    const float mean = s[0] * p.inv_cols;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t)(i * TPR + t) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float d = c + e < p.cols ? v[i][e] - mean : 0.f;
            s[0] = __builtin_fmaf(d, d, s[0]);
        }
    }
    group_sum<TPR, 1>(s, red, 1);
    const float rstd = 1.0f / sqrtf(s[0] * p.inv_cols + p.eps);
    T* y = static_cast<T*>(p.y) + r * p.ldy;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = (int64_t)(i * TPR + t) * VEC;
        if (c < p.cols) {
            const FloatVec<VEC> g = load_param<P, VEC>(p.gamma, c, p.cols, 1.f);
            const FloatVec<VEC> b = load_param<P, VEC>(p.beta, c, p.cols, 0.f);
            FloatVec<VEC> o;
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = __builtin_fmaf((v[i][e] - mean) * rstd, g[e], b[e]);
            store_row<T, VEC>(y, c, p.cols, from_float<T, VEC>(o));
        }
    }
    if (t == 0) {
        if (p.mean) p.mean[r] = mean;
        if (p.rstd) p.rstd[r] = rstd;
    }
}

// Rows wider than the registers of 1024 threads: three walks over the row
// (it stays in the XCD's L2 between them).
template <typename T, typename P>
__device__ __forceinline__ void layer_norm_forward_loop_body(const TropLayerNormParams& p) {
    constexpr int VEC = ln_vec<T>(), TPR = 1024;
    __shared__ float red[2][1][TPR / 64];
    const int64_t r = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + r * p.ldx;
    float s[1] = {0.f};
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < p.cols; c += TPR * VEC) {
        const FloatVec<VEC> v = to_float<T, VEC>(load_row<T, VEC>(x, c, p.cols));
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[0] += v[e];
    }
    group_sum<TPR, 1>(s, red, 0);
    const float mean = s[0] * p.inv_cols;
    s[0] = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < p.cols; c += TPR * VEC) {
        const FloatVec<VEC> v = to_float<T, VEC>(load_row<T, VEC>(x, c, p.cols));
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float d = c + e < p.cols ? v[e] - mean : 0.f;
            s[0] = __builtin_fmaf(d, d, s[0]);
        }
    }
    group_sum<TPR, 1>(s, red, 1);
    const float rstd = 1.0f / sqrtf(s[0] * p.inv_cols + p.eps);
    T* y = static_cast<T*>(p.y) + r * p.ldy;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < p.cols; c += TPR * VEC) {
        const FloatVec<VEC> v = to_float<T, VEC>(load_row<T, VEC>(x, c, p.cols));
        const FloatVec<VEC> g = load_param<P, VEC>(p.gamma, c, p.cols, 1.f);
        const FloatVec<VEC> b = load_param<P, VEC>(p.beta, c, p.cols, 0.f);
        FloatVec<VEC> o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = __builtin_fmaf((v[e] - mean) * rstd, g[e], b[e]);
        store_row<T, VEC>(y, c, p.cols, from_float<T, VEC>(o));
    }
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[r] = mean;
        if (p.rstd) p.rstd[r] = rstd;
    }
}

// Rows blockIdx.x RPB + group, then every parts RPB further; the next row's
// x and dy are loaded before the current one is reduced (not with 1024
// threads, whose 128 registers would spill).
template <typename T, typename P, int TPR>
__device__ __forceinline__ void layer_norm_backward_body(const TropLayerNormParams& p) {
    constexpr int VEC = ln_vec<T>(), NV = 16 / VEC, RPB = TPR == 64 ? 4 : 1;
    using V = typename VecOf<T, VEC>::raw;
    __shared__ float red[2][2][TPR > 64 ? TPR / 64 : 1];
    __shared__ float cols_lds[TPR == 64 ? 2 * TROP_LN_COLS_WAVE : 1];
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int64_t step = (int64_t)p.parts * RPB;
    float dg[NV * VEC] = {}, db[NV * VEC] = {};
    V xv[NV], yv[NV];
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](int64_t r) {
        const T* x = static_cast<const T*>(p.x) + r * p.ldx;
        const T* dy = static_cast<const T*>(p.dy) + r * p.lddy;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * TPR + t) * VEC;
            xv[i] = load_row_stream<T, VEC>(x, c, p.cols);
            yv[i] = load_row_stream<T, VEC>(dy, c, p.cols);
        }
        mean = p.mean[r];
        rstd = p.rstd[r];
    };
    int64_t r = (int64_t)blockIdx.x * RPB + group;
    if (TPR < 1024 && r < p.rows) fetch(r);
    int slot = 0;
    for (; r < p.rows; r += step) {  // the groups of a workgroup share barriers only when RPB = 1
        if constexpr (TPR == 1024) fetch(r);
        FloatVec<VEC> h[NV], w[NV];
        const float rs = rstd;
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * TPR + t) * VEC;
            const FloatVec<VEC> x = to_float<T, VEC>(xv[i]), dy = to_float<T, VEC>(yv[i]);
            const FloatVec<VEC> g = load_param<P, VEC>(p.gamma, c, p.cols, 1.f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                // past the row's end dy is zero; h is held to zero too, so
                // that a non-finite statistic adds nothing there
                const float hh = c + e < p.cols ? (x[e] - mean) * rs : 0.f;
                h[i][e] = hh;
                w[i][e] = c + e < p.cols ? dy[e] * g[e] : 0.f;
                dg[i * VEC + e] = __builtin_fmaf(dy[e], hh, dg[i * VEC + e]);
                db[i * VEC + e] += dy[e];
                s[0] += w[i][e];
                s[1] = __builtin_fmaf(w[i][e], hh, s[1]);
            }
        }
        if (TPR < 1024 && r + step < p.rows) fetch(r + step);
        group_sum<TPR, 2>(s, red, slot);
        slot ^= 1;
        if (p.y) {
            const float c1 = s[0] * p.inv_cols, c2 = s[1] * p.inv_cols;
            T* dx = static_cast<T*>(p.y) + r * p.ldy;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(i * TPR + t) * VEC;
                FloatVec<VEC> o;
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = __builtin_fmaf(-c2, h[i][e], w[i][e] - c1) * rs;
                if (c < p.cols) store_row_stream<T, VEC>(dx, c, p.cols, from_float<T, VEC>(o));
            }
        }
    }
    if (!p.part) return;
    float* pg = p.part + (int64_t)blockIdx.x * p.cols;
    float* pb = pg + (int64_t)p.parts * p.cols;
    if constexpr (TPR == 64) {  // the four waves' sums, added in wave order
        for (int wv = 0; wv < 4; ++wv) {
            if (group == wv) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int c = (i * TPR + t) * VEC + e;
                        cols_lds[c] = wv ? cols_lds[c] + dg[i * VEC + e] : dg[i * VEC + e];
                        cols_lds[TROP_LN_COLS_WAVE + c] =
                            wv ? cols_lds[TROP_LN_COLS_WAVE + c] + db[i * VEC + e] : db[i * VEC + e];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < p.cols; c += 256) {
            pg[c] = cols_lds[c];
            pb[c] = cols_lds[TROP_LN_COLS_WAVE + c];
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(i * TPR + t) * VEC;
            FloatVec<VEC> a, b;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                a[e] = dg[i * VEC + e];
                b[e] = db[i * VEC + e];
            }
            if (c < p.cols) {
                store_row<float, VEC>(pg, c, p.cols, a);
                store_row<float, VEC>(pb, c, p.cols, b);
            }
        }
    }
}

// Rows wider than the registers: dx by two walks over the row ...
template <typename T, typename P>
__device__ __forceinline__ void layer_norm_backward_loop_body(const TropLayerNormParams& p) {
    constexpr int VEC = ln_vec<T>(), TPR = 1024;
    __shared__ float red[2][2][TPR / 64];
    const int64_t r = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + r * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + r * p.lddy;
    const float mean = p.mean[r], rstd = p.rstd[r];
    float s[2] = {0.f, 0.f};
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < p.cols; c += TPR * VEC) {
        const FloatVec<VEC> a = to_float<T, VEC>(load_row<T, VEC>(x, c, p.cols));
        const FloatVec<VEC> b = to_float<T, VEC>(load_row<T, VEC>(dy, c, p.cols));
        const FloatVec<VEC> g = load_param<P, VEC>(p.gamma, c, p.cols, 1.f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float h = c + e < p.cols ? (a[e] - mean) * rstd : 0.f;
            const float w = c + e < p.cols ? b[e] * g[e] : 0.f;
            s[0] += w;
            s[1] = __builtin_fmaf(w, h, s[1]);
        }
    }
    group_sum<TPR, 2>(s, red, 0);
    const float c1 = s[0] * p.inv_cols, c2 = s[1] * p.inv_cols;
    T* dx = static_cast<T*>(p.y) + r * p.ldy;
    for (int64_t c = (int64_t)threadIdx.x * VEC; c < p.cols; c += TPR * VEC) {
        const FloatVec<VEC> a = to_float<T, VEC>(load_row<T, VEC>(x, c, p.cols));
        const FloatVec<VEC> b = to_float<T, VEC>(load_row<T, VEC>(dy, c, p.cols));
        const FloatVec<VEC> g = load_param<P, VEC>(p.gamma, c, p.cols, 1.f);
        FloatVec<VEC> o;
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = __builtin_fmaf(-c2, (a[e] - mean) * rstd, b[e] * g[e] - c1) * rstd;
        store_row<T, VEC>(dx, c, p.cols, from_float<T, VEC>(o));
    }
}

// ... and the partial column sums by threads that keep a column each:
// blockIdx.x = part + parts * (256-column block, from col0 on); part q sums
// rows q, q + parts, ...  Runs before the dx walk, which may overwrite dy.
template <typename T>
__device__ __forceinline__ void layer_norm_columns_body(const TropLayerNormParams& p) {
    const int64_t part = blockIdx.x % p.parts, c = p.col0 + (int64_t)(blockIdx.x / p.parts) * 256 + threadIdx.x;
    if (c >= p.cols) return;
    float dg = 0.f, db = 0.f;
    for (int64_t r = part; r < p.rows; r += p.parts) {
        const float x = (float)static_cast<const T*>(p.x)[r * p.ldx + c];
        const float dy = (float)static_cast<const T*>(p.dy)[r * p.lddy + c];
        dg = __builtin_fmaf(dy, (x - p.mean[r]) * p.rstd[r], dg);
        db += dy;
    }
    p.part[part * p.cols + c] = dg;
    p.part[(p.parts + part) * p.cols + c] = db;
}

// Sum of the partial column sums.  A workgroup takes 64 columns of dgamma or
// (the second half of them) dbeta, 16 waves the parts wave, wave + 16, ...; the waves' sums are added
// in wave order.
template <typename P>
__device__ __forceinline__ void layer_norm_merge_body(const TropLayerNormMergeParams& p) {
    __shared__ float lds[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
    const uint32_t blocks = gridDim.x / 2;
    const bool beta = blockIdx.x >= blocks;
    const int64_t c = p.col0 + (int64_t)(blockIdx.x - (beta ? blocks : 0)) * 64 + lane;
    P* out = static_cast<P*>(beta ? p.dbeta : p.dgamma);
    if (!out) return;
    float s = 0.f;
    if (c < p.cols) {
        const float* q = p.part + (beta ? (int64_t)p.parts * p.cols : 0) + c;
#pragma unroll 4
        for (int i = wave; i < p.parts; i += 16) s += q[(int64_t)i * p.cols];
    }
    lds[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && c < p.cols) {
        float a = lds[0][lane];
#pragma unroll
        for (int w = 1; w < 16; ++w) a += lds[w][lane];
        out[c] = (P)a;
    }
}

}  // namespace trop
