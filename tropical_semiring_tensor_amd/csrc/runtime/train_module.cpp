// The training operators' code object: loaded once per process and device by
// the first training call, apart from the contraction's, so that programs
// that only contract never load it.  Launches and loads are counted here.
#include <atomic>
#include <cstring>
#include <mutex>
#include <string>

#include "train.h"

// Embedded code object (co_blob.S).
extern "C" const unsigned char trop_train_code_object[];

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
};
static_assert(sizeof(kNames) / sizeof(kNames[0]) == TK_COUNT, "training kernels");

struct TrainModule {
    hipModule_t module = nullptr;
    hipFunction_t fn[TK_COUNT] = {};
};

std::mutex g_mu;
std::atomic<TrainModule*> g_dev[kMaxDevices];
std::atomic<uint64_t> g_loads{0}, g_total{0};
std::atomic<uint64_t> g_launches[TROP_T_FAMILIES];

trop_status load(int dev) {
    if (dev < 0 || dev >= kMaxDevices) return fail(TROP_ERR_INVALID_ARGUMENT, "device index out of range");
    if (g_dev[dev].load(std::memory_order_acquire)) return TROP_OK;
    std::lock_guard<std::mutex> lock(g_mu);
    if (g_dev[dev].load(std::memory_order_acquire)) return TROP_OK;
    TrainModule* m = new TrainModule;
    hipError_t e = hipModuleLoadData(&m->module, trop_train_code_object);
    trop_status st = e == hipSuccess ? TROP_OK : hip_fail(e, "hipModuleLoadData (training code object)");
    if (st == TROP_OK) {
        g_loads.fetch_add(1);
        for (int i = 0; i < TK_COUNT && st == TROP_OK; ++i) {
            e = hipModuleGetFunction(&m->fn[i], m->module, kNames[i]);
            if (e != hipSuccess) st = hip_fail(e, kNames[i]);
        }
        if (st != TROP_OK) (void)hipModuleUnload(m->module);
    }
    if (st != TROP_OK) {
        delete m;
        return st;
    }
    g_dev[dev].store(m, std::memory_order_release);
    return TROP_OK;
}

}  // namespace

trop_status train_device(int* dev) {
    hipError_t e = hipGetDevice(dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    return load(*dev);
}

trop_status train_launch(int dev, TrainKernelId id, trop_train_family fam, int64_t grid, uint32_t block,
                         const void* params, hipStream_t stream) {
    TrainModule* m = g_dev[dev].load(std::memory_order_acquire);
    if (!m) return fail(TROP_ERR_HIP, "training code object not loaded on this device");
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
    if (a >= lo_ && a < hi_ && a % elem_bytes == 0 && (unsigned __int128)elems * elem_bytes <= hi_ - a) return TROP_OK;
    const std::string name = index < 0 ? what : std::string(what) + " of tensor " + std::to_string(index);
    if (a % elem_bytes) return fail(TROP_ERR_INVALID_ARGUMENT, name + " is not aligned to its elements");
    const trop_status st = check_device_span(p, dev_, elems, elem_bytes, name.c_str());
    if (st != TROP_OK) return st;
    hipDeviceptr_t base = nullptr;
    size_t size = 0;
    if (hipMemGetAddressRange(&base, &size, const_cast<void*>(p)) == hipSuccess) {
        lo_ = reinterpret_cast<uintptr_t>(base);
        hi_ = lo_ + size;
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
        const trop_status st = load(device);
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
