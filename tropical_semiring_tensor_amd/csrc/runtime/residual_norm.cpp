// Between two residual blocks: argument checks, the parts of the backward's
// column sums and the launches (see residual_norm_kernels.h).
#include <algorithm>
#include <cmath>
#include <string>

#include "product_tiles.h"
#include "train.h"

namespace trop {
namespace {

trop_status invalid(const std::string& what) { return fail(TROP_ERR_INVALID_ARGUMENT, what); }

trop_status check_norms(const trop_residual_norm& op) {
    if (op.dtype != TROP_F32 && op.dtype != TROP_BF16)
        return invalid("residual norms take float32 or bfloat16, got dtype " + std::to_string((int)op.dtype));
    for (const trop_norm n : {op.post, op.pre})
        if (n != TROP_NORM_NONE && n != TROP_NORM_LAYER && n != TROP_NORM_RMS)
            return invalid("no norm " + std::to_string((int)n));
    if (op.rows < 0 || op.cols < 0) return invalid("negative size");
    if (op.gate && op.gate_group < 1) return invalid("gate_group must be at least 1");
    return TROP_OK;
}

trop_status check_op(const trop_residual_norm& op) {
    const trop_status st = check_norms(op);
    if (st != TROP_OK) return st;
    if (ln_index(op.dtype, op.param_dtype) < 0) return invalid("norm weights are float32 or of the rows' type");
    if (op.gate && ln_index(op.dtype, op.gate_dtype) < 0) return invalid("the gate is float32 or of the rows' type");
    for (const float f : {op.residual_scale, op.branch_scale})
        if (!std::isfinite(f)) return invalid("the scales must be finite");
    for (const float f : {op.post_eps, op.pre_eps})
        if (!(f >= 0.f) || std::isinf(f)) return invalid("eps must be finite and >= 0");
    return TROP_OK;
}

// Rows of a gate row, and gate rows (one for all rows without a gate).
int64_t gate_group(const trop_residual_norm& op) {
    return op.gate ? std::min(op.gate_group, std::max<int64_t>(op.rows, 1)) : std::max<int64_t>(op.rows, 1);
}
int64_t gate_rows(const trop_residual_norm& op) { return ceil_div(op.rows, gate_group(op)); }

// Row group of the backward: 0 to 4 a wave, 128, 256, 512 and 1024 threads of 8
// columns (float32 1 and 2: twice the threads, 4 columns); kWide: rows too wide
// to keep their sums as well; kNarrow: narrower than a vector; kPlain: without
// a norm.
enum { kRegisters = 5, kWide = 5, kNarrow = 6, kPlain = 7 };
int backward_group(const trop_residual_norm& op) {
    if (op.cols < 8) return kNarrow;
    if (op.pre == TROP_NORM_NONE && op.post == TROP_NORM_NONE) return kPlain;
    int group = 0;
    while (group < kRegisters && op.cols > (TROP_RN_COLS_ALL >> 4) << group) ++group;
    return group;
}

// Parts a backward makes at most, by row group: more keep more loads in flight,
// but each leaves its sums for a second kernel to add.  Rows and sums in 512,
// 768, 1024 and 2048 parts: 16384 x 1024 bfloat16 68, 56, 48 and 50 us (two
// waves to a row); 8192 x 2048 bfloat16 48, 49, 50 and 62 (four); 16384 x 512 26,
// 27, 28 and 35 (one); 16384 x 1001 float32 in 512 and 1024 78 and 87 (four).
// 1024 threads to a row fill a CU.  Where the sums have a kernel of their own
// its blocks of columns make more workgroups.
int64_t most_parts(const trop_residual_norm& op) {
    const int group = backward_group(op);
    if (group < kRegisters) return group == 4 ? 256 : group == 1 && op.dtype == TROP_BF16 ? 1024 : 512;
    return std::max<int64_t>(128, 1024 / ceil_div(std::max<int64_t>(op.cols, 1), TROP_RN_COLS_SUMS));
}

// The backward's parts: each inside one gate row (group_parts to one), so
// that the gate's gradient is summed as the weights' are; with more gate rows
// than parts, several whole gate rows (group_parts 0), whose gradients the
// part writes itself.
struct Parts {
    int64_t parts, part_rows, group_parts;
};
Parts parts_of(const trop_residual_norm& op, int64_t limit) {
    if (op.rows == 0) return {0, 1, 1};
    // (four rows at least, a wave each or one after another: 1537 x 1001 with 29
    // gate rows in 783 parts of two 20 + 9 us, in 406 of four 20 + 5)
    const int64_t group = gate_group(op), gates = gate_rows(op);
    if (gates <= limit) {
        const int64_t most = std::min(limit / gates, ceil_div(group, 4));
        const int64_t rows = ceil_div(group, most), per = ceil_div(group, rows);
        return {gates * per, rows, per};
    }
    const int64_t whole = ceil_div(gates, limit);
    return {ceil_div(gates, whole), whole * group, 0};
}

// Workspace: partial sums of every gradient that op can have, and of wide
// rows the pre norm's two means.
struct Layout {
    Parts parts;
    int64_t at[TROP_RN_SUMS];  // in floats
    int64_t row_sums;
    size_t bytes;
};
trop_status plan(const trop_residual_norm& op, Layout* l) {
    l->parts = parts_of(op, most_parts(op));
    const bool has[TROP_RN_SUMS] = {op.pre != TROP_NORM_NONE, op.pre != TROP_NORM_NONE, op.post != TROP_NORM_NONE,
                                    op.post != TROP_NORM_NONE, op.gate && l->parts.group_parts > 0};
    int64_t one, total = 0;
    if (__builtin_mul_overflow(l->parts.parts * 4, op.cols, &one) || one > ((int64_t)1 << 58))
        return invalid("workspace size overflows");
    for (int i = 0; i < TROP_RN_SUMS; ++i) {
        l->at[i] = total / 4;
        if (has[i]) total += one;
    }
    l->row_sums = total / 4;
    if (backward_group(op) >= kRegisters && op.pre != TROP_NORM_NONE) {
        int64_t more;
        if (__builtin_mul_overflow(op.rows, (int64_t)8, &more) || __builtin_add_overflow(total, more, &total))
            return invalid("workspace size overflows");
    }
    l->bytes = (size_t)total;
    return TROP_OK;
}

trop_status check_matrix(SpanChecker& checker, const trop_matrix& m, const trop_residual_norm& op, const char* what) {
    if (!m.data) return fail(TROP_ERR_NOT_DEVICE_MEMORY, std::string(what) + " is NULL");
    return checker.matrix(m.data, op.rows, op.cols, m.ld, elem_size(op.dtype), what);
}

// What both directions' kernels get.
trop_status common(const trop_residual_norm& op, SpanChecker& checker, TropResidualParams& p) {
    trop_status st = TROP_OK;
    const size_t pb = elem_size(op.param_dtype);
    if (op.gate) {
        st = checker.matrix(op.gate, gate_rows(op), op.cols, op.ldgate, elem_size(op.gate_dtype), "gate");
        if (st != TROP_OK) return st;
        p.gate = op.gate;
        p.ldgate = op.ldgate;
    }
    p.gate_f32 = op.gate_dtype == TROP_F32;
    p.weight_f32 = op.param_dtype == TROP_F32;
    p.gate_group = gate_group(op);
    auto weight = [&](bool there, const void* w, const char* what) -> const void* {
        if (!there || !w || st != TROP_OK) return nullptr;
        st = checker.span(w, op.cols, pb, what);
        return w;
    };
    p.post_gamma = weight(op.post != TROP_NORM_NONE, op.post_gamma, "post_gamma");
    p.post_beta = weight(op.post != TROP_NORM_NONE, op.post_beta, "post_beta");
    p.pre_gamma = weight(op.pre != TROP_NORM_NONE, op.pre_gamma, "pre_gamma");
    p.pre_beta = weight(op.pre != TROP_NORM_NONE, op.pre_beta, "pre_beta");
    p.post = op.post;
    p.pre = op.pre;
    p.residual_scale = op.residual_scale;
    p.branch_scale = op.branch_scale;
    p.post_eps = op.post_eps;
    p.pre_eps = op.pre_eps;
    p.rows = op.rows;
    p.cols = op.cols;
    p.inv_cols = op.cols ? (float)(1.0 / (double)op.cols) : 0.f;
    return st;
}

// A kernel with a row group to a row: as many launches as its rows need.
trop_status launch_rows(int dev, int id, trop_train_family fam, TropResidualParams p, int64_t rpg, uint32_t block,
                        hipStream_t s) {
    const int64_t most = max_groups(block) * rpg;
    trop_status st = TROP_OK;
    for (; st == TROP_OK && p.row0 < p.rows; p.row0 += most)
        st = train_launch(dev, (TrainKernelId)id, fam, ceil_div(std::min(p.rows - p.row0, most), rpg), block, &p, s);
    return st;
}

trop_status forward(const trop_residual_norm* opp, const trop_residual_norm_rows* io, void* stream) {
    if (!opp || !io) return invalid("NULL structure");
    const trop_matrix &r = io->r, &u = io->u, &h = io->h, &y = io->y;
    const trop_act8 *u8 = io->u8, *h8 = io->h8;
    const trop_residual_norm& op = *opp;
    trop_status st = check_op(op);
    if (st != TROP_OK) return st;
    if (y.data && op.pre == TROP_NORM_NONE) return invalid("y without a norm before the next block");
    if (op.rows == 0 || op.cols == 0) return ok();
    int dev = -1;
    if ((st = block_device(&dev)) != TROP_OK) return st;
    SpanChecker checker(dev);
    TropResidualParams p = {};
    if ((st = common(op, checker, p)) != TROP_OK) return st;
    auto matrix = [&](const trop_matrix& m, const char* what) {
        return check_matrix(checker, m, op, what);
    };
    if ((st = matrix(u, "u")) != TROP_OK) return st;
    if (r.data && (st = matrix(r, "r")) != TROP_OK) return st;
    if (h.data && (st = matrix(h, "h")) != TROP_OK) return st;
    if (h.data && h.data == r.data && h.ld != r.ld) return invalid("h is r but its row stride is another");
    if (y.data && (st = matrix(y, "y")) != TROP_OK) return st;
    auto rows = [&](bool there, float* v, const char* what) -> float* {
        if (!there || !v || st != TROP_OK) return nullptr;
        st = checker.span(v, op.rows, 4, what);
        return v;
    };
    p.post_mean = rows(op.post == TROP_NORM_LAYER, io->post_mean, "post_mean");
    p.post_rstd = rows(op.post != TROP_NORM_NONE, io->post_rstd, "post_rstd");
    p.pre_mean = rows(op.pre == TROP_NORM_LAYER, io->pre_mean, "pre_mean");
    p.pre_rstd = rows(op.pre != TROP_NORM_NONE, io->pre_rstd, "pre_rstd");
    if (st != TROP_OK) return st;
    if (u8) {
        if ((st = check_act8(checker, *u8, op.rows, op.cols, "u8's")) != TROP_OK) return st;
        p.u_codes = u8->codes;
        p.u_exps = u8->exponents;
        p.ldu_codes = u8->ld;
        p.ldu_exps = u8->ld_exponents;
    }
    if (h8) {
        if ((st = check_act8(checker, *h8, op.rows, op.cols, "h8's")) != TROP_OK) return st;
        p.h_codes = h8->codes;
        p.h_exps = h8->exponents;
        p.ldh_codes = h8->ld;
        p.ldh_exps = h8->ld_exponents;
    }
    p.r = r.data;
    p.u = u.data;
    p.h = h.data;
    p.y = y.data;
    p.ldr = r.ld;
    p.ldu = u.ld;
    p.ldh = h.ld;
    p.ldy = y.ld;
    // 16 elements to a thread
    static const TrainKernelId ids[] = {TK_RN_FWD_WAVE, TK_RN_FWD_BLOCK, TK_RN_FWD_HALF, TK_RN_FWD_WIDE, TK_RN_FWD_LOOP};
    static const uint32_t threads[] = {256, 256, 512, 1024, 1024};
    const int g = op.cols <= 64 * 16 ? 0 : op.cols <= 256 * 16 ? 1 : op.cols <= 512 * 16 ? 2 : op.cols <= 1024 * 16 ? 3 : 4;
    st = launch_rows(dev, ids[g] + ln_index(op.dtype, op.param_dtype), TROP_T_RESIDUAL_FORWARD, p, g == 0 ? 4 : 1,
                     threads[g], static_cast<hipStream_t>(stream));
    return st == TROP_OK ? ok() : st;
}

// The sums of the parts into the gradients that were asked for.
trop_status sum_parts(int dev, const trop_residual_norm& op, const trop_residual_norm_grads& g, const Layout& l,
                      const float* workspace, hipStream_t s) {
    TropRowSumsParams q = {};
    q.cols = op.cols;
    int64_t blocks = 0;
    auto entry = [&](int i, void* dst, int64_t ldd, int64_t rows, int64_t parts, float scale, trop_dtype dt) {
        if (!dst) return;
        TropRowSumsEntry& e = q.e[q.count++];
        e.src = workspace ? workspace + l.at[i] : nullptr;
        e.dst = dst;
        e.ldd = ldd;
        e.rows = rows;
        e.parts = parts;
        e.scale = scale;
        e.f32 = dt == TROP_F32;
        e.column_bits = parts <= 16 ? 8 : parts <= 64 || rows * op.cols >= 4096 ? 6 : 4;
        blocks += rows * ceil_div(op.cols, (int64_t)1 << e.column_bits);
        e.blocks = (uint32_t)blocks;
    };
    const int64_t parts = l.parts.parts;
    entry(TROP_RN_PRE_GAMMA, g.dpre_gamma, op.cols, 1, parts, 1.f, op.param_dtype);
    entry(TROP_RN_PRE_BETA, g.dpre_beta, op.cols, 1, parts, 1.f, op.param_dtype);
    entry(TROP_RN_POST_GAMMA, g.dpost_gamma, op.cols, 1, parts, 1.f, op.param_dtype);
    entry(TROP_RN_POST_BETA, g.dpost_beta, op.cols, 1, parts, 1.f, op.param_dtype);
    if (l.parts.group_parts && op.rows)
        entry(TROP_RN_GATE, g.dgate.data, g.dgate.ld, gate_rows(op), l.parts.group_parts, op.branch_scale, op.gate_dtype);
    if (blocks >= (int64_t)1 << 32) return invalid("too many columns");
    trop_status st = TROP_OK;
    const int64_t most = max_groups(1024);
    for (; st == TROP_OK && q.id0 < blocks; q.id0 += most)
        st = train_launch(dev, (TrainKernelId)(TK_PART_SUMS + (op.dtype == TROP_BF16)), TROP_T_RESIDUAL_BACKWARD,
                          std::min(blocks - q.id0, most), 1024, &q, s);
    return st;
}

trop_status backward(const trop_residual_norm* opp, const trop_residual_norm_kept* kp, const trop_residual_norm_grads* gp,
                     void* workspace, size_t workspace_bytes, void* stream) {
    if (!opp || !kp || !gp) return invalid("NULL structure");
    const trop_residual_norm& op = *opp;
    const trop_residual_norm_kept& k = *kp;
    const trop_residual_norm_grads& g = *gp;
    trop_status st = check_op(op);
    if (st != TROP_OK) return st;
    const bool pre = op.pre != TROP_NORM_NONE, post = op.post != TROP_NORM_NONE;
    if ((g.dpre_gamma || g.dpre_beta) && !pre) return invalid("no norm before the next block to have gradients");
    if ((g.dpost_gamma || g.dpost_beta) && !post) return invalid("no norm after the block to have gradients");
    if (g.dgate.data && !op.gate) return invalid("no gate to have a gradient");
    if (k.dy.data && !pre) return invalid("dy without a norm before the next block");
    if ((k.u8 && k.u.data) || (k.h8 && k.h.data)) return invalid("u and h are given in one form");
    const bool params = g.dpre_gamma || g.dpre_beta || g.dpost_gamma || g.dpost_beta;
    if (op.cols == 0 || (!params && (op.rows == 0 || (!g.dr.data && !g.du.data && !g.dgate.data)))) return ok();
    int dev = -1;
    if ((st = block_device(&dev)) != TROP_OK) return st;
    const size_t pb = elem_size(op.param_dtype);
    SpanChecker checker(dev);
    TropResidualParams p = {};
    Layout l = {};
    if ((st = plan(op, &l)) != TROP_OK) return st;
    // what the sums alone need, and what the rows' gradients need besides
    const bool sum_post = g.dpost_gamma || g.dpost_beta, sums = params || g.dgate.data;
    const bool through_post = post && (g.du.data || sum_post), need_u = through_post || g.dgate.data;
    const bool held = k.u8 || k.h8;
    auto weight = [&](void* w, const char* what) {
        if (w && st == TROP_OK) st = checker.span(w, op.cols, pb, what);
    };
    weight(g.dpre_gamma, "dpre_gamma");
    weight(g.dpre_beta, "dpre_beta");
    weight(g.dpost_gamma, "dpost_gamma");
    weight(g.dpost_beta, "dpost_beta");
    if (st != TROP_OK) return st;
    if (op.rows > 0) {
        if ((st = common(op, checker, p)) != TROP_OK) return st;
        auto matrix = [&](const trop_matrix& m, const char* what) {
            return check_matrix(checker, m, op, what);
        };
        auto statistic = [&](bool there, const float* v, const char* what) -> float* {
            if (!there || st != TROP_OK) return nullptr;
            st = checker.span(v, op.rows, 4, what);
            return const_cast<float*>(v);
        };
        if (pre) {
            if ((st = matrix(k.dy, "dy")) != TROP_OK) return st;
            if (k.h8) {
                if ((st = check_act8(checker, *k.h8, op.rows, op.cols, "h8's")) != TROP_OK) return st;
                p.h_codes = k.h8->codes;
                p.h_exps = k.h8->exponents;
                p.ldh_codes = k.h8->ld;
                p.ldh_exps = k.h8->ld_exponents;
            } else if (held) {
                return invalid("h is needed in 8 bits, as u is");
            } else if ((st = matrix(k.h, "h")) != TROP_OK) {
                return st;
            }
        }
        if (!pre || k.dh.data) {
            if ((st = matrix(k.dh, "dh")) != TROP_OK) return st;
        }
        if (need_u) {
            if (k.u8) {
                if ((st = check_act8(checker, *k.u8, op.rows, op.cols, "u8's")) != TROP_OK) return st;
                p.u_codes = k.u8->codes;
                p.u_exps = k.u8->exponents;
                p.ldu_codes = k.u8->ld;
                p.ldu_exps = k.u8->ld_exponents;
            } else if (held) {
                return invalid("u is needed in 8 bits, as h is");
            } else if ((st = matrix(k.u, "u")) != TROP_OK) {
                return st;
            }
        }
        p.pre_mean = statistic(op.pre == TROP_NORM_LAYER, k.pre_mean, "pre_mean");
        p.pre_rstd = statistic(pre, k.pre_rstd, "pre_rstd");
        p.post_mean = statistic(need_u && op.post == TROP_NORM_LAYER, k.post_mean, "post_mean");
        p.post_rstd = statistic(need_u && post, k.post_rstd, "post_rstd");
        if (st != TROP_OK) return st;
        if (g.dr.data && (st = matrix(g.dr, "dr")) != TROP_OK) return st;
        if (g.du.data && (st = matrix(g.du, "du")) != TROP_OK) return st;
        if (g.dgate.data) {
            st = checker.matrix(g.dgate.data, gate_rows(op), op.cols, g.dgate.ld, elem_size(op.gate_dtype), "dgate");
            if (st != TROP_OK) return st;
        }
    }
    if (sums && l.bytes) {
        if (!workspace || workspace_bytes < l.bytes)
            return fail(TROP_ERR_WORKSPACE_TOO_SMALL, "the residual norm's backward needs " + std::to_string(l.bytes) +
                                                          " workspace bytes, got " +
                                                          std::to_string(workspace ? workspace_bytes : 0));
        if ((st = checker.span(workspace, (int64_t)(l.bytes / 4), 4, "workspace")) != TROP_OK) return st;
    }
    float* ws = static_cast<float*>(workspace);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (op.rows > 0) {
        p.dy = k.dy.data;
        p.dh = k.dh.data;
        p.h = k.h.data;
        p.u = k.u.data;
        p.dr = g.dr.data;
        p.du = g.du.data;
        p.lddy = k.dy.ld;
        p.lddh = k.dh.ld;
        p.ldh = k.h.ld;
        p.ldu = k.u.ld;
        p.lddr = g.dr.ld;
        p.lddu = g.du.ld;
        p.lddgate = g.dgate.ld;
        p.parts = (int32_t)l.parts.parts;
        p.part_rows = l.parts.part_rows;
        p.group_parts = l.parts.group_parts;
        p.dgate = l.parts.group_parts ? nullptr : g.dgate.data;
        const void* asked[TROP_RN_SUMS] = {g.dpre_gamma, g.dpre_beta, g.dpost_gamma, g.dpost_beta,
                                           l.parts.group_parts ? g.dgate.data : nullptr};
        for (int i = 0; i < TROP_RN_SUMS; ++i) p.part[i] = asked[i] ? ws + l.at[i] : nullptr;
        p.need_v = g.dgate.data != nullptr;
        p.need_post = through_post;
        p.ragged = op.cols % (16 / (int64_t)elem_size(op.dtype)) != 0;
        const int kind = backward_group(op), variant = 2 * held + (op.dtype == TROP_BF16);
        const int loop = ln_index(op.dtype, op.param_dtype) + (held ? 3 : 0);
        // norms of the rows' gradients, and of the sums: 0 pre, 1 post, 2 both, 3 none
        const int norms = pre ? (post && need_u ? 2 : 0) : post && need_u ? 1 : 3;
        if (kind < kRegisters && norms < 3) {
            static const uint32_t threads[] = {256, 128, 256, 512, 1024};
            const uint32_t more = op.dtype == TROP_F32 && (kind == 1 || kind == 2) ? 2 : 1;
            st = train_launch(dev, (TrainKernelId)(TK_RN_BWD + 12 * kind + 4 * norms + variant), TROP_T_RESIDUAL_BACKWARD,
                              l.parts.parts, threads[kind] * more, &p, s);
        } else {
            p.row_sums = pre && (sum_post || g.dgate.data) ? ws + l.row_sums : nullptr;
            if (g.dr.data || g.du.data || p.row_sums) {
                if (kind == kWide && op.cols <= TROP_RN_COLS_ROWS && norms < 3) {
                    TropResidualParams q = p;
                    const Parts rows = parts_of(op, 256);
                    q.part_rows = rows.part_rows;
                    q.group_parts = rows.group_parts;
                    st = train_launch(dev, (TrainKernelId)(TK_RN_BWD_ROWS + 4 * norms + variant),
                                      TROP_T_RESIDUAL_BACKWARD, rows.parts, 1024, &q, s);
                } else {
                    st = launch_rows(dev, TK_RN_BWD_LOOP + loop, TROP_T_RESIDUAL_BACKWARD, p, 1, 1024, s);
                }
            }
            if (st == TROP_OK && sums) {
                p.need_post = sum_post;
                // (the vectors' kernel counts bytes of a row in 32 bits)
                const bool vectors = kind != kNarrow && op.cols <= (int64_t)1 << 29;
                const int64_t width = vectors ? TROP_RN_COLS_SUMS : 256, blocks = ceil_div(op.cols, width);
                const int64_t most = max_groups(256) / l.parts.parts;
                for (int64_t b = 0; st == TROP_OK && b < blocks; b += most) {
                    p.col0 = vectors ? b : b * width;
                    st = train_launch(dev, (TrainKernelId)(vectors ? TK_RN_BWD_SUMS + 4 * norms + variant : TK_RN_COLUMNS + loop),
                                      TROP_T_RESIDUAL_BACKWARD, l.parts.parts * std::min(blocks - b, most), 256, &p, s);
                }
            }
        }
    }
    if (st == TROP_OK && sums) st = sum_parts(dev, op, g, l, ws, s);
    return st == TROP_OK ? ok() : st;
}

}  // namespace
}  // namespace trop

extern "C" trop_status tropical_residual_norm_forward(const trop_residual_norm* op, const trop_residual_norm_rows* rows,
                                                      void* stream) {
    return trop::guarded("tropical_residual_norm_forward", [&] { return trop::forward(op, rows, stream); });
}

extern "C" trop_status tropical_residual_norm_backward(const trop_residual_norm* op, const trop_residual_norm_kept* kept,
                                                       const trop_residual_norm_grads* grads, void* workspace,
                                                       size_t workspace_bytes, void* stream) {
    return trop::guarded("tropical_residual_norm_backward",
                         [&] { return trop::backward(op, kept, grads, workspace, workspace_bytes, stream); });
}

extern "C" trop_status tropical_residual_norm_backward_workspace_size(const trop_residual_norm* op, size_t* bytes) {
    return trop::guarded("tropical_residual_norm_backward_workspace_size", [&]() -> trop_status {
        if (!op || !bytes) return trop::invalid("NULL argument");
        *bytes = 0;
        trop_status st = trop::check_norms(*op);
        if (st != TROP_OK) return st;
        trop::Layout l = {};
        if ((st = trop::plan(*op, &l)) != TROP_OK) return st;
        *bytes = l.bytes;
        return trop::ok();
    });
}
