// Layer norm: argument checks and the choice of the row group (see
// layer_norm_kernels.h).
#include <cmath>
#include <string>

#include "train.h"

namespace trop {
namespace {

trop_status check_types(trop_dtype dt, trop_dtype pdt, int64_t rows, int64_t cols) {
    if (dt != TROP_F32 && dt != TROP_BF16)
        return fail(TROP_ERR_INVALID_ARGUMENT, "layer norm takes float32 or bfloat16, got dtype " + std::to_string((int)dt));
    if (ln_index(dt, pdt) < 0)
        return fail(TROP_ERR_INVALID_ARGUMENT, "layer norm weights are float32 or of the rows' type");
    if (rows < 0 || cols < 0) return fail(TROP_ERR_INVALID_ARGUMENT, "negative size");
    return TROP_OK;
}

// Row group by the columns 16 elements per thread cover.
int group_of(int64_t cols) {
    return cols <= TROP_LN_COLS_WAVE ? 0 : cols <= TROP_LN_COLS_BLOCK ? 1 : cols <= TROP_LN_COLS_WIDE ? 2 : 3;
}

// Workgroups of the backward, each making one partial sum: one row group
// per row while they are few.
int64_t backward_parts(int64_t rows, int64_t cols) {
    const int64_t rpb = group_of(cols) == 0 ? 4 : 1;
    const int64_t n = (rows + rpb - 1) / rpb;
    return n < TROP_LN_MAX_PARTS ? n : TROP_LN_MAX_PARTS;
}

trop_status part_bytes(int64_t rows, int64_t cols, size_t* bytes) {
    int64_t b;
    if (__builtin_mul_overflow(backward_parts(rows, cols) * 8, cols, &b))
        return fail(TROP_ERR_INVALID_ARGUMENT, "layer norm workspace size overflows");
    *bytes = (size_t)b;
    return TROP_OK;
}

// A kernel with a row group to a row: as many launches as its rows need.
// `rpg`: rows of a workgroup; eb: bytes of an element.
trop_status launch_rows(int dev, TrainKernelId id, trop_train_family fam, TropLayerNormParams p, int64_t rpg,
                        uint32_t block, size_t eb, hipStream_t s) {
    const int64_t rows = p.rows, most = max_groups(block) * rpg;
    for (int64_t r0 = 0; r0 < rows; r0 += most) {
        p.rows = rows - r0 < most ? rows - r0 : most;
        const trop_status st = train_launch(dev, id, fam, (p.rows + rpg - 1) / rpg, block, &p, s);
        if (st != TROP_OK) return st;
        p.x = static_cast<const char*>(p.x) + (size_t)most * p.ldx * eb;
        if (p.dy) p.dy = static_cast<const char*>(p.dy) + (size_t)most * p.lddy * eb;
        p.y = static_cast<char*>(p.y) + (size_t)most * p.ldy * eb;
        if (p.mean) p.mean += most;
        if (p.rstd) p.rstd += most;
    }
    return TROP_OK;
}

trop_status forward(trop_dtype dt, trop_dtype pdt, const void* x, int64_t ldx, const void* gamma, const void* beta,
                    float eps, void* y, int64_t ldy, float* mean, float* rstd, int64_t rows, int64_t cols,
                    void* stream) {
    trop_status st = check_types(dt, pdt, rows, cols);
    if (st != TROP_OK) return st;
    if (!(eps >= 0.f) || std::isinf(eps)) return fail(TROP_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
    if (rows == 0 || cols == 0) return ok();
    int dev = -1;
    if ((st = train_device(&dev)) != TROP_OK) return st;
    const size_t eb = elem_size(dt), pb = elem_size(pdt);
    SpanChecker checker(dev);
    if ((st = checker.matrix(x, rows, cols, ldx, eb, "x")) != TROP_OK) return st;
    if ((st = checker.matrix(y, rows, cols, ldy, eb, "y")) != TROP_OK) return st;
    if (x == y && ldx != ldy) return fail(TROP_ERR_INVALID_ARGUMENT, "y is x but its row stride is another");
    if (gamma && (st = checker.span(gamma, cols, pb, "gamma")) != TROP_OK) return st;
    if (beta && (st = checker.span(beta, cols, pb, "beta")) != TROP_OK) return st;
    if (mean && (st = checker.span(mean, rows, 4, "mean")) != TROP_OK) return st;
    if (rstd && (st = checker.span(rstd, rows, 4, "rstd")) != TROP_OK) return st;
    TropLayerNormParams p = {};
    p.x = x;
    p.gamma = gamma;
    p.beta = beta;
    p.y = y;
    p.mean = mean;
    p.rstd = rstd;
    p.ldx = ldx;
    p.ldy = ldy;
    p.rows = rows;
    p.cols = cols;
    p.eps = eps;
    p.inv_cols = (float)(1.0 / (double)cols);
    static const TrainKernelId ids[] = {TK_LN_FWD_WAVE, TK_LN_FWD_BLOCK, TK_LN_FWD_WIDE, TK_LN_FWD_LOOP};
    const int g = group_of(cols);
    st = launch_rows(dev, (TrainKernelId)(ids[g] + ln_index(dt, pdt)), TROP_T_LAYER_NORM_FORWARD, p, g == 0 ? 4 : 1,
                     g < 2 ? 256 : 1024, eb, static_cast<hipStream_t>(stream));
    return st == TROP_OK ? ok() : st;
}

trop_status backward(trop_dtype dt, trop_dtype pdt, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                     const float* mean, const float* rstd, const void* gamma, void* dx, int64_t lddx, void* dgamma,
                     void* dbeta, int64_t rows, int64_t cols, void* workspace, size_t workspace_bytes, void* stream) {
    trop_status st = check_types(dt, pdt, rows, cols);
    if (st != TROP_OK) return st;
    if (cols == 0 || (!dgamma && !dbeta && (!dx || rows == 0))) return ok();
    int dev = -1;
    if ((st = train_device(&dev)) != TROP_OK) return st;
    const size_t eb = elem_size(dt), pb = elem_size(pdt);
    SpanChecker checker(dev);
    if (rows > 0) {
        if ((st = checker.matrix(dy, rows, cols, lddy, eb, "dy")) != TROP_OK) return st;
        if ((st = checker.matrix(x, rows, cols, ldx, eb, "x")) != TROP_OK) return st;
        if ((st = checker.span(mean, rows, 4, "mean")) != TROP_OK) return st;
        if ((st = checker.span(rstd, rows, 4, "rstd")) != TROP_OK) return st;
        if (dx && (st = checker.matrix(dx, rows, cols, lddx, eb, "dx")) != TROP_OK) return st;
        if (dx && dx == dy && lddx != lddy)
            return fail(TROP_ERR_INVALID_ARGUMENT, "dx is dy but its row stride is another");
    }
    if (gamma && (st = checker.span(gamma, cols, pb, "gamma")) != TROP_OK) return st;
    if (dgamma && (st = checker.span(dgamma, cols, pb, "dgamma")) != TROP_OK) return st;
    if (dbeta && (st = checker.span(dbeta, cols, pb, "dbeta")) != TROP_OK) return st;
    const bool params = dgamma || dbeta;
    size_t need = 0;
    if (params && (st = part_bytes(rows, cols, &need)) != TROP_OK) return st;
    if (need) {
        if (!workspace || workspace_bytes < need)
            return fail(TROP_ERR_WORKSPACE_TOO_SMALL, "layer norm backward needs " + std::to_string(need) +
                                                          " workspace bytes, got " +
                                                          std::to_string(workspace ? workspace_bytes : 0));
        if ((st = checker.span(workspace, (int64_t)(need / 4), 4, "workspace")) != TROP_OK)
            return st;
    }
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t parts = backward_parts(rows, cols);
    TropLayerNormParams p = {};
    p.x = x;
    p.dy = dy;
    p.gamma = gamma;
    p.y = dx;
    p.mean = const_cast<float*>(mean);
    p.rstd = const_cast<float*>(rstd);
    p.part = params ? static_cast<float*>(workspace) : nullptr;
    p.ldx = ldx;
    p.lddy = lddy;
    p.ldy = lddx;
    p.rows = rows;
    p.cols = cols;
    p.inv_cols = (float)(1.0 / (double)cols);
    p.parts = (int32_t)parts;
    const int g = group_of(cols);
    if (rows > 0) {
        const int idx = ln_index(dt, pdt);
        if (g < 3) {
            static const TrainKernelId ids[] = {TK_LN_BWD_WAVE, TK_LN_BWD_BLOCK, TK_LN_BWD_WIDE};
            st = train_launch(dev, (TrainKernelId)(ids[g] + idx), TROP_T_LAYER_NORM_BACKWARD, parts,
                              g < 2 ? 256 : 1024, &p, s);
            if (st != TROP_OK) return st;
        } else {
            if (params) {  // before dx, which may be dy's own buffer
                const int64_t most = max_groups(256) / parts * 256;
                for (; p.col0 < cols; p.col0 += most) {
                    const int64_t n = cols - p.col0 < most ? cols - p.col0 : most;
                    st = train_launch(dev, (TrainKernelId)(TK_LN_COLUMNS + (dt == TROP_BF16)),
                                      TROP_T_LAYER_NORM_BACKWARD, parts * ((n + 255) / 256), 256, &p, s);
                    if (st != TROP_OK) return st;
                }
            }
            if (dx) {
                st = launch_rows(dev, (TrainKernelId)(TK_LN_BWD_LOOP + idx), TROP_T_LAYER_NORM_BACKWARD, p, 1, 1024, eb,
                                 s);
                if (st != TROP_OK) return st;
            }
        }
    }
    if (params) {
        TropLayerNormMergeParams q = {};
        q.part = static_cast<const float*>(workspace);
        q.dgamma = dgamma;
        q.dbeta = dbeta;
        q.cols = cols;
        q.parts = (int32_t)parts;
        const int64_t most = max_groups(1024) / 2 * 64;
        for (; q.col0 < cols; q.col0 += most) {
            const int64_t n = cols - q.col0 < most ? cols - q.col0 : most;
            st = train_launch(dev, (TrainKernelId)(TK_LN_MERGE + (pdt == TROP_BF16)), TROP_T_LAYER_NORM_BACKWARD,
                              2 * ((n + 63) / 64), 1024, &q, s);
            if (st != TROP_OK) return st;
        }
    }
    return ok();
}

}  // namespace
}  // namespace trop

extern "C" trop_status tropical_layer_norm_forward(trop_dtype dtype, trop_dtype param_dtype, const void* x,
                                                   int64_t ldx, const void* gamma, const void* beta, float eps,
                                                   void* y, int64_t ldy, float* mean, float* rstd, int64_t rows,
                                                   int64_t cols, void* stream) {
    return trop::guarded("tropical_layer_norm_forward", [&] {
        return trop::forward(dtype, param_dtype, x, ldx, gamma, beta, eps, y, ldy, mean, rstd, rows, cols, stream);
    });
}

extern "C" trop_status tropical_layer_norm_backward_workspace_size(int64_t rows, int64_t cols, int with_params,
                                                                   size_t* bytes) {
    return trop::guarded("tropical_layer_norm_backward_workspace_size", [&]() -> trop_status {
        if (!bytes) return trop::fail(TROP_ERR_INVALID_ARGUMENT, "bytes is NULL");
        if (rows < 0 || cols < 0) return trop::fail(TROP_ERR_INVALID_ARGUMENT, "negative size");
        *bytes = 0;
        if (with_params) {
            const trop_status st = trop::part_bytes(rows, cols, bytes);
            if (st != TROP_OK) return st;
        }
        return trop::ok();
    });
}

extern "C" trop_status tropical_layer_norm_backward(trop_dtype dtype, trop_dtype param_dtype, const void* dy,
                                                    int64_t lddy, const void* x, int64_t ldx, const float* mean,
                                                    const float* rstd, const void* gamma, void* dx, int64_t lddx,
                                                    void* dgamma, void* dbeta, int64_t rows, int64_t cols,
                                                    void* workspace, size_t workspace_bytes, void* stream) {
    return trop::guarded("tropical_layer_norm_backward", [&] {
        return trop::backward(dtype, param_dtype, dy, lddy, x, ldx, mean, rstd, gamma, dx, lddx, dgamma, dbeta, rows,
                              cols, workspace, workspace_bytes, stream);
    });
}
