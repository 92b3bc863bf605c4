// The gfx950 code object of the operators around a residual block: activations
// in 8 bits, the weight gradient from them, and the norms, gate and sum
// between two blocks.  Built and loaded beside train_kernels.hip's.
#include "act8_grad_w_kernels.h"
#include "residual_norm_kernels.h"

using namespace trop;

#define TROP_ACT8_ENTRIES(NAME, T)                                                                          \
    extern "C" __global__ __launch_bounds__(256) void trop_act8_pack_##NAME(TropAct8Params p) {              \
        act8_pack_body<T>(p);                                                                                \
    }                                                                                                        \
    extern "C" __global__ __launch_bounds__(256) void trop_act8_unpack_##NAME(TropAct8Params p) {            \
        act8_unpack_body<T>(p);                                                                              \
    }                                                                                                        \
    extern "C" __global__ __launch_bounds__(256) void trop_grad_w_pack_##NAME(TropGradWParams p) {           \
        grad_w_pack_body<T>(p);                                                                              \
    }                                                                                                        \
    extern "C" __global__ __launch_bounds__(256) void trop_grad_w_finish_##NAME(TropGradWParams p) {         \
        grad_w_finish_body<T>(p);                                                                            \
    }                                                                                                        \
    extern "C" __global__ __launch_bounds__(1024) void trop_part_sums_##NAME(TropRowSumsParams p) {          \
        part_sums_body<T>(p);                                                                                \
    }
#define TROP_GRAD_W_TILE(NAME, T, TILE, EDGE, WM, WN, BUFFERS)                                               \
    using GradW8_##TILE##_##NAME = MgConfig<EDGE, EDGE, WM, WN, MM, MM, 1, BUFFERS, grad_w_parts<T>()>;      \
    extern "C" __global__ __launch_bounds__(GradW8_##TILE##_##NAME::THREADS) void                            \
        trop_grad_w##TILE##_##NAME(TropGradWParams p) {                                                      \
        __shared__ __align__(1024) char lds[GradW8_##TILE##_##NAME::LDS_BYTES];                              \
        grad_w_body<GradW8_##TILE##_##NAME, T>(p, lds);                                                      \
    }
#define TROP_GRAD_W_TILES(NAME, T)                                                                           \
    TROP_GRAD_W_TILE(NAME, T, 256, 256, 2, 4, 2)                                                             \
    TROP_GRAD_W_TILE(NAME, T, 128, 128, 2, 2, 2)                                                             \
    TROP_GRAD_W_TILE(NAME, T, 64, 64, 2, 2, 2)                                                               \
    TROP_GRAD_W_TILE(NAME, T, 64d, 64, 2, 2, 4)
TROP_ACT8_ENTRIES(f32, float)
TROP_ACT8_ENTRIES(bf16, bf16)
TROP_GRAD_W_TILES(f32, float)
TROP_GRAD_W_TILES(bf16, bf16)

// suffix: element type, the weights' type; backward: u and h as they are, or in 8 bits
#define TROP_RN_ENTRY(KERNEL, THREADS, BODY) TROP_RN_ENTRY_WAVES(KERNEL, THREADS, 1, BODY)
// WAVES: at least so many to a SIMD
#define TROP_RN_ENTRY_WAVES(KERNEL, THREADS, WAVES, BODY)                                                    \
    extern "C" __global__ __launch_bounds__(THREADS, WAVES) void trop_rn_##KERNEL(TropResidualParams p) { BODY(p); }
#define TROP_RN_WIDE(NAME, T, P, HELD)                                                                       \
    TROP_RN_ENTRY(bwd_loop_##NAME, 1024, (residual_norm_backward_loop_body<T, P, HELD>))                     \
    TROP_RN_ENTRY(columns_##NAME, 256, (residual_norm_columns_body<T, P, HELD>))
#define TROP_RN_ENTRIES(NAME, T, P)                                                                          \
    TROP_RN_ENTRY(fwd_wave_##NAME, 256, (residual_norm_forward_body<T, P, 64>))                              \
    TROP_RN_ENTRY(fwd_block_##NAME, 256, (residual_norm_forward_body<T, P, 256>))                            \
    TROP_RN_ENTRY_WAVES(fwd_half_##NAME, 512, 4, (residual_norm_forward_body<T, P, 512>))                    \
    TROP_RN_ENTRY(fwd_wide_##NAME, 1024, (residual_norm_forward_body<T, P, 1024>))                           \
    TROP_RN_ENTRY(fwd_loop_##NAME, 1024, (residual_norm_forward_loop_body<T, P>))                            \
    TROP_RN_WIDE(NAME, T, P, false)                                                                          \
    TROP_RN_WIDE(NAME##_held8, T, P, true)
TROP_RN_ENTRIES(f32_f32, float, float)
TROP_RN_ENTRIES(bf16_bf16, bf16, bf16)
TROP_RN_ENTRIES(bf16_f32, bf16, float)
// rows in registers: which norms there are, element type (at least four waves
// to a SIMD in bfloat16)
#define TROP_RN_ROWS(KERNEL, NAME, THREADS, T, TPR, EPT, HELD, PRE, POST, WORK)                              \
    TROP_RN_ENTRY_WAVES(bwd_##KERNEL##_##NAME, THREADS, sizeof(T) == 2 ? 4 : 1,                              \
                        (residual_norm_backward_body<T, TPR, EPT, HELD, PRE, POST, WORK>))
// c512 ... c8k: by the widest row.  float32 rows of 512 to 2048 columns have twice
// the threads, 4 elements (one vector, as in bfloat16) to each: a row's way from
// load to store is shorter and 5 waves fit a SIMD instead of 3 (1537 x 1001 16
// us against 20, 16384 x 1001 78 against 84, x 2000 alike; 16384 x 500, with two
// waves to a row for one, 46 against 40).
#define RN_MORE(T) (sizeof(T) / 2)
#define TROP_RN_BACKWARD(NAME, T, HELD, PRE, POST)                                                           \
    TROP_RN_ROWS(c512, NAME, 256, T, 64, 8, HELD, PRE, POST, RN_ALL)                                        \
    TROP_RN_ROWS(c1k, NAME, 128 * RN_MORE(T), T, 128 * RN_MORE(T), 8 / RN_MORE(T), HELD, PRE, POST, RN_ALL) \
    TROP_RN_ROWS(c2k, NAME, 256 * RN_MORE(T), T, 256 * RN_MORE(T), 8 / RN_MORE(T), HELD, PRE, POST, RN_ALL) \
    TROP_RN_ROWS(c4k, NAME, 512, T, 512, 8, HELD, PRE, POST, RN_ALL)                                        \
    TROP_RN_ROWS(c8k, NAME, 1024, T, 1024, 8, HELD, PRE, POST, RN_ALL)                                      \
    TROP_RN_ROWS(rows, NAME, 1024, T, 1024, 16, HELD, PRE, POST, RN_ROWS)                                    \
    TROP_RN_ROWS(sums, NAME, 256, T, 256, 8, HELD, PRE, POST, RN_COLUMNS)
#define TROP_RN_NORMS(NAME, T, HELD)                                                                         \
    TROP_RN_BACKWARD(pre_##NAME, T, HELD, true, false)                                                       \
    TROP_RN_BACKWARD(post_##NAME, T, HELD, false, true)                                                      \
    TROP_RN_BACKWARD(both_##NAME, T, HELD, true, true)                                                       \
    TROP_RN_ROWS(sums, none_##NAME, 256, T, 256, 8, HELD, false, false, RN_COLUMNS)
TROP_RN_NORMS(f32, float, false)
TROP_RN_NORMS(bf16, bf16, false)
TROP_RN_NORMS(f32_held8, float, true)
TROP_RN_NORMS(bf16_held8, bf16, true)
