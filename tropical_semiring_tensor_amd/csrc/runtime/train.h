// Internal interfaces of the training operators' host runtime.
#pragma once
#include <exception>
#include <string>

#include "../train_params.h"
#include "internal.h"

namespace trop {

// Kernels of the training code object.  A family has one entry point per
// (element type, weights' type), in ln_index / ce_index order.
enum TrainKernelId : int {
    TK_LN_FWD_WAVE = 0,  // + ln_index: f32 f32, bf16 bf16, bf16 f32
    TK_LN_FWD_BLOCK = TK_LN_FWD_WAVE + 3,
    TK_LN_FWD_WIDE = TK_LN_FWD_BLOCK + 3,
    TK_LN_FWD_LOOP = TK_LN_FWD_WIDE + 3,
    TK_LN_BWD_WAVE = TK_LN_FWD_LOOP + 3,
    TK_LN_BWD_BLOCK = TK_LN_BWD_WAVE + 3,
    TK_LN_BWD_WIDE = TK_LN_BWD_BLOCK + 3,
    TK_LN_BWD_LOOP = TK_LN_BWD_WIDE + 3,
    TK_LN_COLUMNS = TK_LN_BWD_LOOP + 3,  // + (bf16 ? 1 : 0)
    TK_LN_MERGE = TK_LN_COLUMNS + 2,
    TK_ADAMW = TK_LN_MERGE + 2,  // + 2 (bf16) + (master ? 1 : 0)
    TK_ADAMW8 = TK_ADAMW + 4,
    TK_ADAMW8_UNPACK = TK_ADAMW8 + 4,
    TK_CE_KEEP,
    TK_CE_MERGE,
    TK_CE_PACK,  // every family from here on: + (bf16 ? 1 : 0)
    TK_CE_FINISH = TK_CE_PACK + 2,
    TK_CE_FINISH_W = TK_CE_FINISH + 2,
    TK_CE_STATS = TK_CE_FINISH_W + 2,  // + 2 tile (256, 128, 64, 128 with four buffers)
    TK_CE_GRAD = TK_CE_STATS + 8,      // likewise
    TK_CE_GRADIENTS = TK_CE_GRAD + 8,  // + 2 tile (256, 128, 64)
    // float32 w as it lies: tiles 128, 64, 128 with four buffers (gradients: 128, 64)
    TK_CE_STATS_RAW = TK_CE_GRADIENTS + 6,
    TK_CE_GRAD_RAW = TK_CE_STATS_RAW + 3,
    TK_CE_GRADIENTS_RAW = TK_CE_GRAD_RAW + 3,
    // few tokens: + (bf16 ? 1 : 0) + 2 log2(blocks of 16 tokens: 1, 2, 4) + 6 (5) where a
    // workgroup takes several blocks of labels (trop_ce_few_rows)
    TK_CE_FEW = TK_CE_GRADIENTS_RAW + 2,  // statistics
    TK_CE_FEW_GRAD = TK_CE_FEW + 12,   // G; likewise, without bf16 for 4 blocks
    TK_CE_FEW_GX = TK_CE_FEW_GRAD + 10,  // the gradients: without label blocks
    TK_CE_FEW_GW = TK_CE_FEW_GX + 5,
    TK_COUNT = TK_CE_FEW_GW + 5
};

// Current device with the training code object loaded on it.
trop_status train_device(int* dev);
trop_status train_launch(int dev, TrainKernelId id, trop_train_family fam, int64_t grid, uint32_t block,
                         const void* params, hipStream_t stream);
// Workgroups of `block` threads that one launch may have.
inline int64_t max_groups(uint32_t block) { return 0xffffffffLL / block; }
void reset_train_launches();

inline size_t elem_size(trop_dtype dt) { return dt == TROP_BF16 ? 2 : 4; }

// Extents and allocations of one call's pointers.  One inside the allocation
// that the call checked last needs no further query (small tensors share the
// allocator's segments, a call's own are often neighbours).
class SpanChecker {
   public:
    explicit SpanChecker(int dev) : dev_(dev) {}
    // `elems` elements from p on, aligned to their size
    trop_status span(const void* p, int64_t elems, size_t elem_bytes, const char* what, int64_t index = -1);
    // a row-major rows x cols matrix of row stride ld (rows, cols >= 1)
    trop_status matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t elem_bytes, const char* what);

   private:
    int dev_;
    uintptr_t lo_ = 1, hi_ = 0;
};

// A C entry point's body: no C++ exception leaves the library.
template <typename F>
trop_status guarded(const char* what, F&& body) {
    try {
        return body();
    } catch (const std::exception& e) {
        try {
            return fail(TROP_ERR_HIP, std::string(what) + ": " + e.what());
        } catch (...) {
            return TROP_ERR_HIP;
        }
    }
}

}  // namespace trop
