// The gfx950 code object of the training operators: every kernel entry
// point.  Built with hipcc --genco and embedded in the library beside the
// contraction's; loaded once per device by the first training call.
#include "adamw_kernels.h"
#include "layer_norm_kernels.h"

using namespace trop;

// suffix: element type, then the weights' type
#define TROP_LN_ENTRIES(NAME, T, P)                                                                    \
    extern "C" __global__ __launch_bounds__(256) void trop_ln_fwd_wave_##NAME(TropLayerNormParams p) {  \
        layer_norm_forward_body<T, P, 64>(p);                                                           \
    }                                                                                                   \
    extern "C" __global__ __launch_bounds__(256) void trop_ln_fwd_block_##NAME(TropLayerNormParams p) { \
        layer_norm_forward_body<T, P, 256>(p);                                                          \
    }                                                                                                   \
    extern "C" __global__ __launch_bounds__(1024) void trop_ln_fwd_wide_##NAME(TropLayerNormParams p) { \
        layer_norm_forward_body<T, P, 1024>(p);                                                         \
    }                                                                                                   \
    extern "C" __global__ __launch_bounds__(1024) void trop_ln_fwd_loop_##NAME(TropLayerNormParams p) { \
        layer_norm_forward_loop_body<T, P>(p);                                                          \
    }                                                                                                   \
    extern "C" __global__ __launch_bounds__(256) void trop_ln_bwd_wave_##NAME(TropLayerNormParams p) {  \
        layer_norm_backward_body<T, P, 64>(p);                                                          \
    }                                                                                                   \
    extern "C" __global__ __launch_bounds__(256) void trop_ln_bwd_block_##NAME(TropLayerNormParams p) { \
        layer_norm_backward_body<T, P, 256>(p);                                                         \
    }                                                                                                   \
    extern "C" __global__ __launch_bounds__(1024) void trop_ln_bwd_wide_##NAME(TropLayerNormParams p) { \
        layer_norm_backward_body<T, P, 1024>(p);                                                        \
    }                                                                                                   \
    extern "C" __global__ __launch_bounds__(1024) void trop_ln_bwd_loop_##NAME(TropLayerNormParams p) { \
        layer_norm_backward_loop_body<T, P>(p);                                                         \
    }
TROP_LN_ENTRIES(f32_f32, float, float)
TROP_LN_ENTRIES(bf16_bf16, bf16, bf16)
TROP_LN_ENTRIES(bf16_f32, bf16, float)

#define TROP_LN_COLUMNS(NAME, T)                                                                       \
    extern "C" __global__ __launch_bounds__(256) void trop_ln_columns_##NAME(TropLayerNormParams p) {   \
        layer_norm_columns_body<T>(p);                                                                  \
    }                                                                                                   \
    extern "C" __global__ __launch_bounds__(1024) void trop_ln_merge_##NAME(TropLayerNormMergeParams p) { \
        layer_norm_merge_body<T>(p);                                                                    \
    }
TROP_LN_COLUMNS(f32, float)
TROP_LN_COLUMNS(bf16, bf16)

#define TROP_ADAMW_ENTRIES(NAME, T, MASTER)                                                            \
    extern "C" __global__ __launch_bounds__(256) void trop_adamw_##NAME(TropAdamwParams p) {            \
        adamw_body<T, MASTER>(p);                                                                       \
    }                                                                                                   \
    extern "C" __global__ __launch_bounds__(256) void trop_adamw8_##NAME(TropAdamw8Params p) {          \
        adamw8_body<T, MASTER>(p);                                                                      \
    }
TROP_ADAMW_ENTRIES(f32, float, false)
TROP_ADAMW_ENTRIES(f32_master, float, true)
TROP_ADAMW_ENTRIES(bf16, bf16, false)
TROP_ADAMW_ENTRIES(bf16_master, bf16, true)

extern "C" __global__ __launch_bounds__(256) void trop_adamw8_unpack(TropAdamw8Params p) { adamw8_unpack_body(p); }
