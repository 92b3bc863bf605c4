// The training operators' code objects: each loaded once per process and device
// by the first call of its operators, apart from the contraction's, so that
// programs that only contract never load them.  Launches and loads are counted
// here.
#include <atomic>
#include <cstring>
#include <mutex>
#include <string>

#include "train.h"

// Embedded code objects (co_blob.S): kernels below TK_ACT8_PACK, and from it on.
extern "C" const unsigned char trop_train_code_object[];
extern "C" const unsigned char trop_block_code_object[];

namespace trop {
namespace {

constexpr int kMaxDevices = 64;

const char* const kNames[] = {
    "trop_ln_fwd_wave_f32_f32",   "trop_ln_fwd_wave_bf16_bf16",  "trop_ln_fwd_wave_bf16_f32",
    "trop_ln_fwd_block_f32_f32",  "trop_ln_fwd_block_bf16_bf16", "trop_ln_fwd_block_bf16_f32",
    "trop_ln_fwd_wide_f32_f32",   "trop_ln_fwd_wide_bf16_bf16",  "trop_ln_fwd_wide_bf16_f32",
    "trop_ln_fwd_loop_f32_f32",   "trop_ln_fwd_loop_bf16_bf16",  "trop_ln_fwd_loop_bf16_f32",
    "trop_ln_bwd_wave_f32_f32",   "trop_ln_bwd_wave_bf16_bf16",  "trop_ln_bwd_wave_bf16_f32",
    "trop_ln_bwd_block_f32_f32",  "trop_ln_bwd_block_bf16_bf16", "trop_ln_bwd_block_bf16_f32",
    "trop_ln_bwd_wide_f32_f32",   "trop_ln_bwd_wide_bf16_bf16",  "trop_ln_bwd_wide_bf16_f32",
    "trop_ln_bwd_loop_f32_f32",   "trop_ln_bwd_loop_bf16_bf16",  "trop_ln_bwd_loop_bf16_f32",
    "trop_ln_columns_f32",        "trop_ln_columns_bf16",
    "trop_ln_merge_f32",          "trop_ln_merge_bf16",
    "trop_adamw_f32",             "trop_adamw_f32_master",
    "trop_adamw_bf16",            "trop_adamw_bf16_master",
    "trop_adamw8_f32",            "trop_adamw8_f32_master",
    "trop_adamw8_bf16",           "trop_adamw8_bf16_master",
    "trop_adamw8_unpack",
    "trop_ce_keep",               "trop_ce_merge",
    "trop_ce_pack_f32", "trop_ce_pack_bf16",
    "trop_ce_finish_f32", "trop_ce_finish_bf16",
    "trop_ce_finish_w_f32", "trop_ce_finish_w_bf16",
    "trop_ce_stats256_f32", "trop_ce_stats256_bf16",
    "trop_ce_stats128_f32", "trop_ce_stats128_bf16",
    "trop_ce_stats64_f32", "trop_ce_stats64_bf16",
    "trop_ce_stats128d_f32", "trop_ce_stats128d_bf16",
    "trop_ce_grad256_f32", "trop_ce_grad256_bf16",
    "trop_ce_grad128_f32", "trop_ce_grad128_bf16",
    "trop_ce_grad64_f32", "trop_ce_grad64_bf16",
    "trop_ce_grad128d_f32", "trop_ce_grad128d_bf16",
    "trop_ce_gradients256_f32", "trop_ce_gradients256_bf16",
    "trop_ce_gradients128_f32", "trop_ce_gradients128_bf16",
    "trop_ce_gradients64_f32", "trop_ce_gradients64_bf16",
    "trop_ce_stats128_raw", "trop_ce_stats64_raw", "trop_ce_stats128d_raw",
    "trop_ce_grad128_raw", "trop_ce_grad64_raw", "trop_ce_grad128d_raw",
    "trop_ce_gradients128_raw", "trop_ce_gradients64_raw",
    "trop_ce_few1_n1_f32", "trop_ce_few1_n1_bf16",
    "trop_ce_few1_n2_f32", "trop_ce_few1_n2_bf16",
    "trop_ce_few1_n4_f32", "trop_ce_few1_n4_bf16",
    "trop_ce_few2_n1_f32", "trop_ce_few2_n1_bf16",
    "trop_ce_few2_n2_f32", "trop_ce_few2_n2_bf16",
    "trop_ce_few2_n4_f32", "trop_ce_few2_n4_bf16",
    "trop_ce_few_grad1_n1_f32", "trop_ce_few_grad1_n1_bf16", "trop_ce_few_grad1_n2_f32",
    "trop_ce_few_grad1_n2_bf16", "trop_ce_few_grad1_n4_f32",
    "trop_ce_few_grad2_n1_f32", "trop_ce_few_grad2_n1_bf16", "trop_ce_few_grad2_n2_f32",
    "trop_ce_few_grad2_n2_bf16", "trop_ce_few_grad2_n4_f32",
    "trop_ce_few_gx_n1_f32", "trop_ce_few_gx_n1_bf16", "trop_ce_few_gx_n2_f32",
    "trop_ce_few_gx_n2_bf16", "trop_ce_few_gx_n4_f32",
    "trop_ce_few_gw_n1_f32", "trop_ce_few_gw_n1_bf16", "trop_ce_few_gw_n2_f32",
    "trop_ce_few_gw_n2_bf16", "trop_ce_few_gw_n4_f32",
    "trop_act8_pack_f32", "trop_act8_pack_bf16",
    "trop_act8_unpack_f32", "trop_act8_unpack_bf16",
    "trop_grad_w_pack_f32", "trop_grad_w_pack_bf16",
    "trop_grad_w_finish_f32", "trop_grad_w_finish_bf16",
    "trop_part_sums_f32", "trop_part_sums_bf16",
    "trop_grad_w256_f32", "trop_grad_w256_bf16",
    "trop_grad_w128_f32", "trop_grad_w128_bf16",
    "trop_grad_w64_f32", "trop_grad_w64_bf16",
    "trop_grad_w64d_f32", "trop_grad_w64d_bf16",
#define TROP_RN_TYPES(KERNEL, HELD) \
    "trop_rn_" KERNEL "_f32_f32" HELD, "trop_rn_" KERNEL "_bf16_bf16" HELD, "trop_rn_" KERNEL "_bf16_f32" HELD,
    TROP_RN_TYPES("fwd_wave", "") TROP_RN_TYPES("fwd_block", "")
    TROP_RN_TYPES("fwd_half", "") TROP_RN_TYPES("fwd_wide", "") TROP_RN_TYPES("fwd_loop", "")
#define TROP_RN_NORMS(KERNEL)                                                              \
    TROP_RN_KEPT(KERNEL "_pre") TROP_RN_KEPT(KERNEL "_post") TROP_RN_KEPT(KERNEL "_both")
#define TROP_RN_KEPT(KERNEL) \
    "trop_rn_bwd_" KERNEL "_f32", "trop_rn_bwd_" KERNEL "_bf16", "trop_rn_bwd_" KERNEL "_f32_held8", \
    "trop_rn_bwd_" KERNEL "_bf16_held8",
    TROP_RN_NORMS("c512") TROP_RN_NORMS("c1k") TROP_RN_NORMS("c2k") TROP_RN_NORMS("c4k") TROP_RN_NORMS("c8k")
    TROP_RN_NORMS("rows") TROP_RN_NORMS("sums") TROP_RN_KEPT("sums_none")
    TROP_RN_TYPES("bwd_loop", "") TROP_RN_TYPES("bwd_loop", "_held8")
    TROP_RN_TYPES("columns", "") TROP_RN_TYPES("columns", "_held8")
#undef TROP_RN_KEPT
#undef TROP_RN_NORMS
#undef TROP_RN_TYPES
};
static_assert(sizeof(kNames) / sizeof(kNames[0]) == TK_COUNT, "training kernels");

struct TrainModule {
    std::atomic<bool> loaded[2] = {};
    hipFunction_t fn[TK_COUNT] = {};  // of the objects that are loaded
};

std::mutex g_mu;
std::atomic<TrainModule*> g_dev[kMaxDevices];
std::atomic<uint64_t> g_loads{0}, g_total{0};
std::atomic<uint64_t> g_launches[TROP_T_FAMILIES];

// Object 0: kernels below TK_ACT8_PACK, 1: from it on.
trop_status load(int dev, int object) {
    if (dev < 0 || dev >= kMaxDevices) return fail(TROP_ERR_INVALID_ARGUMENT, "device index out of range");
    TrainModule* m = g_dev[dev].load(std::memory_order_acquire);
    if (m && m->loaded[object].load(std::memory_order_acquire)) return TROP_OK;
    std::lock_guard<std::mutex> lock(g_mu);
    m = g_dev[dev].load(std::memory_order_acquire);
    if (!m) {
        m = new TrainModule;
        g_dev[dev].store(m, std::memory_order_release);
    }
    if (m->loaded[object].load(std::memory_order_acquire)) return TROP_OK;
    hipModule_t module = nullptr;
    hipError_t e = hipModuleLoadData(&module, object ? trop_block_code_object : trop_train_code_object);
    if (e != hipSuccess) return hip_fail(e, "hipModuleLoadData (training code object)");
    g_loads.fetch_add(1);
    for (int i = object ? TK_ACT8_PACK : 0; i < (object ? TK_COUNT : TK_ACT8_PACK); ++i) {
        e = hipModuleGetFunction(&m->fn[i], module, kNames[i]);
        if (e != hipSuccess) {
            (void)hipModuleUnload(module);
            return hip_fail(e, kNames[i]);
        }
    }
    m->loaded[object].store(true, std::memory_order_release);
    return TROP_OK;
}

trop_status device(int* dev, int object) {
    hipError_t e = hipGetDevice(dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    return load(*dev, object);
}

}  // namespace

trop_status train_device(int* dev) { return device(dev, 0); }
trop_status block_device(int* dev) { return device(dev, 1); }

trop_status train_launch(int dev, TrainKernelId id, trop_train_family fam, int64_t grid, uint32_t block,
                         const void* params, hipStream_t stream) {
    TrainModule* m = g_dev[dev].load(std::memory_order_acquire);
    if (!m || !m->loaded[id >= TK_ACT8_PACK].load(std::memory_order_acquire))
        return fail(TROP_ERR_HIP, "training code object not loaded on this device");
    if (grid <= 0) return TROP_OK;
    if (grid > max_groups(block))
        return fail(TROP_ERR_INVALID_ARGUMENT, std::string(kNames[id]) + ": too many workgroups");
    void* args[] = {const_cast<void*>(params)};
    hipError_t e = hipModuleLaunchKernel(m->fn[id], (uint32_t)grid, 1, 1, block, 1, 1, 0, stream, args, nullptr);
    if (e != hipSuccess) return hip_fail(e, kNames[id]);
    g_total.fetch_add(1, std::memory_order_relaxed);
    g_launches[fam].fetch_add(1, std::memory_order_relaxed);
    return TROP_OK;
}

void reset_train_launches() {
    g_total.store(0);
    for (auto& n : g_launches) n.store(0);
}

trop_status SpanChecker::span(const void* p, int64_t elems, size_t elem_bytes, const char* what, int64_t index) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    const int known = found_ < kRanges ? found_ : kRanges;
    for (int i = known - 1; i >= 0; --i)
        if (a >= lo_[i] && a < hi_[i] && a % elem_bytes == 0 && (unsigned __int128)elems * elem_bytes <= hi_[i] - a)
            return TROP_OK;
    const std::string name = index < 0 ? what : std::string(what) + " of tensor " + std::to_string(index);
    if (a % elem_bytes) return fail(TROP_ERR_INVALID_ARGUMENT, name + " is not aligned to its elements");
    const trop_status st = check_device_span(p, dev_, elems, elem_bytes, name.c_str());
    if (st != TROP_OK) return st;
    hipDeviceptr_t base = nullptr;
    size_t size = 0;
    if (hipMemGetAddressRange(&base, &size, const_cast<void*>(p)) == hipSuccess) {
        const int at = found_++ % kRanges;
        lo_[at] = reinterpret_cast<uintptr_t>(base);
        hi_[at] = lo_[at] + size;
    } else {
        (void)hipGetLastError();
    }
    return TROP_OK;
}

trop_status SpanChecker::matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t elem_bytes,
                                const char* what) {
    if (ld < cols) return fail(TROP_ERR_INVALID_ARGUMENT, std::string(what) + ": row stride below the row's length");
    int64_t elems = 0;
    if (__builtin_mul_overflow(rows - 1, ld, &elems) || __builtin_add_overflow(elems, cols, &elems))
        return fail(TROP_ERR_INVALID_ARGUMENT, std::string(what) + " extent overflows");
    return span(p, elems, elem_bytes, what);
}

}  // namespace trop

extern "C" trop_status tropical_train_init(int device) {
    using namespace trop;
    return guarded("tropical_train_init", [&]() -> trop_status {
        int n = 0, cur = -1;
        hipError_t e = hipGetDeviceCount(&n);
        if (e != hipSuccess) return hip_fail(e, "hipGetDeviceCount");
        if (device < 0 || device >= n)
            return fail(TROP_ERR_INVALID_ARGUMENT, "tropical_train_init: no device " + std::to_string(device));
        e = hipGetDevice(&cur);
        if (e == hipSuccess && cur != device) e = hipSetDevice(device);
        if (e != hipSuccess) return hip_fail(e, "hipSetDevice");
        trop_status st = load(device, 0);
        if (st == TROP_OK) st = load(device, 1);
        if (cur != device) (void)hipSetDevice(cur);
        return st == TROP_OK ? ok() : st;
    });
}

extern "C" trop_status tropical_get_train_stats(trop_train_stats* out) {
    using namespace trop;
    if (!out) return fail(TROP_ERR_INVALID_ARGUMENT, "tropical_get_train_stats: out is NULL");
    std::memset(out, 0, sizeof(*out));
    out->module_loads = g_loads.load();
    out->launches_total = g_total.load();
    for (int i = 0; i < TROP_T_FAMILIES; ++i) out->launches[i] = g_launches[i].load();
    return ok();
}
