// AdamW: argument checks, the scalars, and the launches that carry the
// tensor table in their argument block (see adamw_kernels.h).
#include <cmath>
#include <string>

#include "train.h"

namespace trop {
namespace {

// Workgroups of 256 threads that one launch may have.
constexpr int64_t kMaxChunks = 0xffffff;

trop_status scalars(const trop_adamw_hyper* h, TropAdamwScalars* s) {
    if (!h) return fail(TROP_ERR_INVALID_ARGUMENT, "hyper is NULL");
    if (h->step < 1) return fail(TROP_ERR_INVALID_ARGUMENT, "step counts from 1");
    if (!(h->beta1 >= 0 && h->beta1 < 1) || !(h->beta2 >= 0 && h->beta2 < 1))
        return fail(TROP_ERR_INVALID_ARGUMENT, "betas must lie in [0, 1)");
    if (!(h->lr >= 0 && std::isfinite(h->lr)) || !(h->eps >= 0 && std::isfinite(h->eps)) ||
        !(h->weight_decay >= 0 && std::isfinite(h->weight_decay)))
        return fail(TROP_ERR_INVALID_ARGUMENT, "lr, eps and weight_decay must be finite and >= 0");
    s->beta1 = (float)h->beta1;
    s->one_minus_beta1 = (float)(1 - h->beta1);
    s->beta2 = (float)h->beta2;
    s->one_minus_beta2 = (float)(1 - h->beta2);
    s->keep = (float)(1 - h->lr * h->weight_decay);
    s->step_size = (float)(h->lr / (1 - std::pow(h->beta1, (double)h->step)));
    s->root = (float)(1 / std::sqrt(1 - std::pow(h->beta2, (double)h->step)));
    s->eps = (float)h->eps;
    return TROP_OK;
}

trop_status check_table(const void* tensors, int64_t count) {
    if (count < 0) return fail(TROP_ERR_INVALID_ARGUMENT, "negative count");
    if (count > 0 && !tensors) return fail(TROP_ERR_INVALID_ARGUMENT, "tensors is NULL");
    return TROP_OK;
}

trop_status check_elements(int64_t n, int64_t i) {
    // one tensor's chunks fit one launch
    if (n < 0 || n > kMaxChunks * TROP_ADAMW_CHUNK)
        return fail(TROP_ERR_INVALID_ARGUMENT, "elements of tensor " + std::to_string(i) + " out of range");
    return TROP_OK;
}

// Walks the entries with elements, at most `cap` tensors and kMaxChunks
// chunks to a launch: `put(e, i)` fills entry e from tensor i.
template <typename PARAMS, typename ENTRY, typename PUT>
trop_status launch_table(int dev, TrainKernelId id, PARAMS& p, const ENTRY* tensors, int64_t count, int cap, PUT&& put,
                         hipStream_t stream) {
    uint64_t chunks = 0;
    p.count = 0;
    for (int64_t i = 0; i <= count; ++i) {
        const uint64_t c = i < count ? ((uint64_t)tensors[i].elements + TROP_ADAMW_CHUNK - 1) / TROP_ADAMW_CHUNK : 0;
        if (p.count && (i == count || p.count == cap || chunks + c > (uint64_t)kMaxChunks)) {
            const trop_status st = train_launch(dev, id, TROP_T_ADAMW, (int64_t)chunks, 256, &p, stream);
            if (st != TROP_OK) return st;
            p.count = 0;
            chunks = 0;
        }
        if (i == count || c == 0) continue;
        chunks += c;
        put(p.t[p.count], i);
        p.chunk_end[p.count] = (uint32_t)chunks;
        ++p.count;
    }
    return ok();
}

trop_status step32(trop_dtype dt, const trop_adamw_tensor* t, int64_t count, const trop_adamw_hyper* hyper,
                   void* stream) {
    if (dt != TROP_F32 && dt != TROP_BF16)
        return fail(TROP_ERR_INVALID_ARGUMENT, "AdamW takes float32 or bfloat16, got dtype " + std::to_string((int)dt));
    TropAdamwParams p;
    trop_status st = scalars(hyper, &p.s);
    if (st == TROP_OK) st = check_table(t, count);
    if (st != TROP_OK) return st;
    bool any = false;
    for (int64_t i = 0; i < count; ++i) {
        if ((st = check_elements(t[i].elements, i)) != TROP_OK) return st;
        any |= t[i].elements > 0;
    }
    if (!any) return ok();
    int dev = -1;
    if ((st = train_device(&dev)) != TROP_OK) return st;
    SpanChecker checker(dev);
    int masters = 0, with = 0;
    for (int64_t i = 0; i < count; ++i) {
        const int64_t n = t[i].elements;
        if (n == 0) continue;
        ++with;
        if ((st = checker.span(t[i].param, n, elem_size(dt), "param", i)) != TROP_OK) return st;
        if ((st = checker.span(t[i].grad, n, elem_size(dt), "grad", i)) != TROP_OK) return st;
        if ((st = checker.span(t[i].exp_avg, n, 4, "exp_avg", i)) != TROP_OK) return st;
        if ((st = checker.span(t[i].exp_avg_sq, n, 4, "exp_avg_sq", i)) != TROP_OK) return st;
        if (t[i].master) {
            ++masters;
            if ((st = checker.span(t[i].master, n, 4, "master", i)) != TROP_OK) return st;
        }
    }
    if (masters && masters != with)
        return fail(TROP_ERR_INVALID_ARGUMENT, "master weights are given for some tensors and not for others");
    const TrainKernelId id = (TrainKernelId)(TK_ADAMW + (dt == TROP_BF16 ? 2 : 0) + (masters ? 1 : 0));
    return launch_table(
        dev, id, p, t, count, TROP_ADAMW_TENSORS,
        [&](TropAdamwEntry& e, int64_t i) {
            e = {t[i].param, t[i].grad, t[i].exp_avg, t[i].exp_avg_sq, t[i].master, t[i].elements};
        },
        static_cast<hipStream_t>(stream));
}

trop_status step8(trop_dtype dt, const trop_adamw8_tensor* t, int64_t count, const trop_adamw_hyper* hyper,
                  void* stream) {
    if (dt != TROP_F32 && dt != TROP_BF16)
        return fail(TROP_ERR_INVALID_ARGUMENT, "AdamW takes float32 or bfloat16, got dtype " + std::to_string((int)dt));
    TropAdamw8Params p;
    trop_status st = scalars(hyper, &p.s);
    if (st == TROP_OK) st = check_table(t, count);
    if (st != TROP_OK) return st;
    bool any = false;
    for (int64_t i = 0; i < count; ++i) {
        if ((st = check_elements(t[i].elements, i)) != TROP_OK) return st;
        any |= t[i].elements > 0;
    }
    if (!any) return ok();
    int dev = -1;
    if ((st = train_device(&dev)) != TROP_OK) return st;
    SpanChecker checker(dev);
    int masters = 0, with = 0;
    for (int64_t i = 0; i < count; ++i) {
        const int64_t n = t[i].elements, nb = (n + TROP_ADAMW_BLOCK - 1) / TROP_ADAMW_BLOCK;
        if (n == 0) continue;
        ++with;
        if ((st = checker.span(t[i].param, n, elem_size(dt), "param", i)) != TROP_OK) return st;
        if ((st = checker.span(t[i].grad, n, elem_size(dt), "grad", i)) != TROP_OK) return st;
        if ((st = checker.span(t[i].exp_avg, n, 1, "exp_avg", i)) != TROP_OK) return st;
        if ((st = checker.span(t[i].exp_avg_scale, nb, 4, "exp_avg_scale", i)) != TROP_OK) return st;
        if ((st = checker.span(t[i].exp_avg_sq, n, 1, "exp_avg_sq", i)) != TROP_OK) return st;
        if ((st = checker.span(t[i].exp_avg_sq_scale, nb, 4, "exp_avg_sq_scale", i)) != TROP_OK) return st;
        if (t[i].master) {
            ++masters;
            if ((st = checker.span(t[i].master, n, 4, "master", i)) != TROP_OK) return st;
        }
    }
    if (masters && masters != with)
        return fail(TROP_ERR_INVALID_ARGUMENT, "master weights are given for some tensors and not for others");
    const TrainKernelId id = (TrainKernelId)(TK_ADAMW8 + (dt == TROP_BF16 ? 2 : 0) + (masters ? 1 : 0));
    return launch_table(
        dev, id, p, t, count, TROP_ADAMW8_TENSORS,
        [&](TropAdamw8Entry& e, int64_t i) {
            e = {t[i].param,         t[i].grad,   t[i].exp_avg, t[i].exp_avg_scale, t[i].exp_avg_sq,
                 t[i].exp_avg_sq_scale, t[i].master, t[i].elements};
        },
        static_cast<hipStream_t>(stream));
}

trop_status unpack8(const trop_adamw8_tensor* t, int64_t count, float* const* mv, float* const* vv, void* stream) {
    trop_status st = check_table(t, count);
    if (st != TROP_OK) return st;
    bool any = false;
    for (int64_t i = 0; i < count; ++i) {
        if ((st = check_elements(t[i].elements, i)) != TROP_OK) return st;
        any |= t[i].elements > 0;
    }
    if (!any || (!mv && !vv)) return ok();
    int dev = -1;
    if ((st = train_device(&dev)) != TROP_OK) return st;
    SpanChecker checker(dev);
    for (int64_t i = 0; i < count; ++i) {
        const int64_t n = t[i].elements, nb = (n + TROP_ADAMW_BLOCK - 1) / TROP_ADAMW_BLOCK;
        if (n == 0) continue;
        if (mv && mv[i]) {
            if ((st = checker.span(t[i].exp_avg, n, 1, "exp_avg", i)) != TROP_OK) return st;
            if ((st = checker.span(t[i].exp_avg_scale, nb, 4, "exp_avg_scale", i)) != TROP_OK) return st;
            if ((st = checker.span(mv[i], n, 4, "exp_avg_values", i)) != TROP_OK) return st;
        }
        if (vv && vv[i]) {
            if ((st = checker.span(t[i].exp_avg_sq, n, 1, "exp_avg_sq", i)) != TROP_OK) return st;
            if ((st = checker.span(t[i].exp_avg_sq_scale, nb, 4, "exp_avg_sq_scale", i)) != TROP_OK) return st;
            if ((st = checker.span(vv[i], n, 4, "exp_avg_sq_values", i)) != TROP_OK) return st;
        }
    }
    TropAdamw8Params p = {};
    return launch_table(
        dev, TK_ADAMW8_UNPACK, p, t, count, TROP_ADAMW8_TENSORS,
        [&](TropAdamw8Entry& e, int64_t i) {
            e = {mv ? mv[i] : nullptr,  nullptr,
                 t[i].exp_avg,          t[i].exp_avg_scale,
                 t[i].exp_avg_sq,       t[i].exp_avg_sq_scale,
                 vv ? vv[i] : nullptr,  t[i].elements};
        },
        static_cast<hipStream_t>(stream));
}

}  // namespace
}  // namespace trop

extern "C" trop_status tropical_adamw_step(trop_dtype dtype, const trop_adamw_tensor* tensors, int64_t count,
                                           const trop_adamw_hyper* hyper, void* stream) {
    return trop::guarded("tropical_adamw_step", [&] { return trop::step32(dtype, tensors, count, hyper, stream); });
}

extern "C" trop_status tropical_adamw8_step(trop_dtype dtype, const trop_adamw8_tensor* tensors, int64_t count,
                                            const trop_adamw_hyper* hyper, void* stream) {
    return trop::guarded("tropical_adamw8_step", [&] { return trop::step8(dtype, tensors, count, hyper, stream); });
}

extern "C" trop_status tropical_adamw8_unpack(const trop_adamw8_tensor* tensors, int64_t count,
                                              float* const* exp_avg_values, float* const* exp_avg_sq_values,
                                              void* stream) {
    return trop::guarded("tropical_adamw8_unpack",
                         [&] { return trop::unpack8(tensors, count, exp_avg_values, exp_avg_sq_values, stream); });
}
