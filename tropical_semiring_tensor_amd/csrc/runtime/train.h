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
    TK_ACT8_PACK = TK_CE_FEW_GW + 5,  // + (bf16 ? 1 : 0), to TK_GRAD_W
    TK_ACT8_UNPACK = TK_ACT8_PACK + 2,
    TK_GRAD_W_PACK = TK_ACT8_UNPACK + 2,
    TK_GRAD_W_FINISH = TK_GRAD_W_PACK + 2,
    TK_PART_SUMS = TK_GRAD_W_FINISH + 2,
    TK_GRAD_W = TK_PART_SUMS + 2,      // + 2 tile (256, 128, 64, 64 with four buffers)
    TK_RN_FWD_WAVE = TK_GRAD_W + 8,    // + ln_index
    TK_RN_FWD_BLOCK = TK_RN_FWD_WAVE + 3,
    TK_RN_FWD_HALF = TK_RN_FWD_BLOCK + 3,
    TK_RN_FWD_WIDE = TK_RN_FWD_HALF + 3,
    TK_RN_FWD_LOOP = TK_RN_FWD_WIDE + 3,
    TK_RN_BWD = TK_RN_FWD_LOOP + 3,  // + 12 row group + 4 (norms: pre, post, both) + 2 (8 bits) + (bf16 ? 1 : 0)
    TK_RN_BWD_ROWS = TK_RN_BWD + 60,   // likewise, without row groups
    TK_RN_BWD_SUMS = TK_RN_BWD_ROWS + 12,  // + 4 (norms: pre, post, both, none) + 2 (8 bits) + (bf16 ? 1 : 0)
    TK_RN_BWD_LOOP = TK_RN_BWD_SUMS + 16,  // + ln_index + 3 (u and h in 8 bits)
    TK_RN_COLUMNS = TK_RN_BWD_LOOP + 6,
    TK_COUNT = TK_RN_COLUMNS + 6
};

// Current device with the code object of layer norm, cross entropy and AdamW
// loaded on it, or that of the kernels from TK_ACT8_PACK on.
trop_status train_device(int* dev);
trop_status block_device(int* dev);
trop_status train_launch(int dev, TrainKernelId id, trop_train_family fam, int64_t grid, uint32_t block,
                         const void* params, hipStream_t stream);
// Workgroups of `block` threads that one launch may have.
inline int64_t max_groups(uint32_t block) { return 0xffffffffLL / block; }
void reset_train_launches();

// A norm's kernels by the rows' and the weights' type: 0: f32 f32, 1: bf16
// bf16, 2: bf16 f32, -1: none
inline int ln_index(trop_dtype dt, trop_dtype pdt) {
    if (dt == TROP_F32 && pdt == TROP_F32) return 0;
    if (dt == TROP_BF16 && pdt == TROP_BF16) return 1;
    if (dt == TROP_BF16 && pdt == TROP_F32) return 2;
    return -1;
}

inline size_t elem_size(trop_dtype dt) { return dt == TROP_BF16 ? 2 : 4; }

// Extents and allocations of one call's pointers.  One inside an allocation
// that the call looked up before needs no further query (small tensors share the
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
    static constexpr int kRanges = 8;
    int found_ = 0;  // ranges looked up, the last kRanges of them kept
    uintptr_t lo_[kRanges], hi_[kRanges];
};

// Both buffers of an 8-bit rows x cols matrix.
trop_status check_act8(SpanChecker& checker, const trop_act8& a, int64_t rows, int64_t cols, const char* what);

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
