// The gfx950 code object of the training operators: every kernel entry
// point.  Built with hipcc --genco and embedded in the library beside the
// contraction's; loaded once per device by the first training call.
#include "adamw_kernels.h"
#include "cross_entropy_kernels.h"
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

extern "C" __global__ __launch_bounds__(1024) void trop_ce_keep(TropCeParams p) {
    if (blockIdx.x == 0)
        ce_keep_body(p);
    else
        ce_magnitude_body(p);
}
extern "C" __global__ __launch_bounds__(256) void trop_ce_merge(TropCeParams p) { ce_merge_body(p); }

// one product tile: its LDS and the body's workgroup
#define TROP_CE_TILE(NAME, CONFIG, BODY)                                                          \
    extern "C" __global__ __launch_bounds__(CONFIG::THREADS) void trop_ce_##NAME(TropCeParams p) { \
        __shared__ __align__(1024) char lds[CONFIG::LDS_BYTES];                                    \
        BODY(p, lds);                                                                              \
    }
#define TROP_CE_ENTRIES(NAME, T, PLANES)                                                               \
    extern "C" __global__ __launch_bounds__(256) void trop_ce_pack_##NAME(TropCeParams p) {             \
        ce_pack_body<PLANES>(p);                                                                        \
    }                                                                                                   \
    extern "C" __global__ __launch_bounds__(256) void trop_ce_finish_##NAME(TropCeParams p) {           \
        ce_finish_body<T, PLANES>(p);                                                                   \
    }                                                                                                   \
    extern "C" __global__ __launch_bounds__(256) void trop_ce_finish_w_##NAME(TropCeParams p) {         \
        ce_finish_w_body<T, PLANES>(p);                                                                 \
    }                                                                                                   \
    using Logits256_##NAME = MgConfig<256, 256, 2, 4, KM, KM, PLANES>;                                  \
    using Logits128_##NAME = MgConfig<128, 128, 2, 2, KM, KM, PLANES>;                                  \
    using Logits128d_##NAME = MgConfig<128, 128, 2, 2, KM, KM, PLANES, 4>;                              \
    using Logits64_##NAME = MgConfig<64, 64, 2, 2, KM, KM, PLANES, 4>;                                  \
    using GradX64_##NAME = MgConfig<64, 64, 2, 2, MM, QK, PLANES>;                                      \
    using GradW64_##NAME = MgConfig<64, 64, 2, 2, MM, QM, PLANES>;                                      \
    using GradX256_##NAME = MgConfig<256, 256, 2, 4, MM, QK, PLANES>;                                   \
    using GradX128_##NAME = MgConfig<128, 128, 2, 2, MM, QK, PLANES>;                                   \
    using GradW256_##NAME = MgConfig<256, 256, 2, 4, MM, QM, PLANES>;                                   \
    using GradW128_##NAME = MgConfig<128, 128, 2, 2, MM, QM, PLANES>;                                   \
    TROP_CE_TILE(stats256_##NAME, Logits256_##NAME, (ce_logits_body<Logits256_##NAME, CE_STATS>))       \
    TROP_CE_TILE(stats128_##NAME, Logits128_##NAME, (ce_logits_body<Logits128_##NAME, CE_STATS>))       \
    TROP_CE_TILE(stats128d_##NAME, Logits128d_##NAME, (ce_logits_body<Logits128d_##NAME, CE_STATS>))    \
    TROP_CE_TILE(grad128d_##NAME, Logits128d_##NAME, (ce_logits_body<Logits128d_##NAME, CE_GRAD>))      \
    TROP_CE_TILE(stats64_##NAME, Logits64_##NAME, (ce_logits_body<Logits64_##NAME, CE_STATS>))          \
    TROP_CE_TILE(grad64_##NAME, Logits64_##NAME, (ce_logits_body<Logits64_##NAME, CE_GRAD>))            \
    TROP_CE_TILE(gradients64_##NAME, GradX64_##NAME,                                              \
                 (ce_gradients_body<GradX64_##NAME, GradW64_##NAME, T>))                               \
    TROP_CE_TILE(grad256_##NAME, Logits256_##NAME, (ce_logits_body<Logits256_##NAME, CE_GRAD>))         \
    TROP_CE_TILE(grad128_##NAME, Logits128_##NAME, (ce_logits_body<Logits128_##NAME, CE_GRAD>))         \
    TROP_CE_TILE(gradients256_##NAME, GradX256_##NAME,                                            \
                 (ce_gradients_body<GradX256_##NAME, GradW256_##NAME, T>))                             \
    TROP_CE_TILE(gradients128_##NAME, GradX128_##NAME,                                            \
                 (ce_gradients_body<GradX128_##NAME, GradW128_##NAME, T>))                             \
    TROP_CE_FEW(NAME, T, 1)                                                                             \
    TROP_CE_FEW(NAME, T, 2)                                                                             \
    TROP_CE_FEW(NAME, T, 4)                                                                             \
    TROP_CE_FEW_GRAD(NAME, T, 1)                                                                        \
    TROP_CE_FEW_GRAD(NAME, T, 2)
// few tokens: NB blocks of 16; one or several blocks of 16 labels a workgroup
#define TROP_CE_FEW(NAME, T, NB)                                                                          \
    extern "C" __global__ __launch_bounds__(256) void trop_ce_few1_n##NB##_##NAME(TropCeParams p) {        \
        ce_few_body<T, 1, NB, CE_STATS>(p);                                                                \
    }                                                                                                      \
    extern "C" __global__ __launch_bounds__(256, 2) void trop_ce_few2_n##NB##_##NAME(TropCeParams p) {        \
        ce_few_body<T, trop_ce_few_rows(NB, sizeof(T)), NB, CE_STATS>(p);                                                                \
    }
#define TROP_CE_FEW_GRAD(NAME, T, NB)                                                                     \
    extern "C" __global__ __launch_bounds__(256) void trop_ce_few_grad1_n##NB##_##NAME(TropCeParams p) {   \
        ce_few_body<T, 1, NB, CE_GRAD>(p);                                                                 \
    }                                                                                                      \
    extern "C" __global__ __launch_bounds__(256) void trop_ce_few_grad2_n##NB##_##NAME(TropCeParams p) {   \
        ce_few_body<T, trop_ce_few_rows(NB, sizeof(T)), NB, CE_GRAD>(p);                                                                 \
    }                                                                                                      \
    extern "C" __global__ __launch_bounds__(256) void trop_ce_few_gx_n##NB##_##NAME(TropCeParams p) {      \
        ce_few_grad_x_body<T, NB>(p);                                                                      \
    }                                                                                                      \
    extern "C" __global__ __launch_bounds__(256) void trop_ce_few_gw_n##NB##_##NAME(TropCeParams p) {      \
        ce_few_grad_w_body<T, NB>(p);                                                                      \
    }
// float32 w read as it lies, for one or two tiles of tokens
using Raw128 = MgConfig<128, 128, 2, 2, RKM, KM, 2>;
using Raw128d = MgConfig<128, 128, 2, 2, RKM, KM, 2, 4>;
using Raw64 = MgConfig<64, 64, 2, 2, RKM, KM, 2, 4>;
using RawX128 = MgConfig<128, 128, 2, 2, RMM, QK, 2>;
using RawX64 = MgConfig<64, 64, 2, 2, RMM, QK, 2>;
TROP_CE_ENTRIES(f32, float, 2)
TROP_CE_ENTRIES(bf16, bf16, 1)
TROP_CE_FEW_GRAD(f32, float, 4)
TROP_CE_TILE(stats128_raw, Raw128, (ce_logits_body<Raw128, CE_STATS>))
TROP_CE_TILE(stats64_raw, Raw64, (ce_logits_body<Raw64, CE_STATS>))
TROP_CE_TILE(stats128d_raw, Raw128d, (ce_logits_body<Raw128d, CE_STATS>))
TROP_CE_TILE(grad128_raw, Raw128, (ce_logits_body<Raw128, CE_GRAD>))
TROP_CE_TILE(grad64_raw, Raw64, (ce_logits_body<Raw64, CE_GRAD>))
TROP_CE_TILE(grad128d_raw, Raw128d, (ce_logits_body<Raw128d, CE_GRAD>))
TROP_CE_TILE(gradients128_raw, RawX128, (ce_gradients_body<RawX128, GradW128_f32, float>))
TROP_CE_TILE(gradients64_raw, RawX64, (ce_gradients_body<RawX64, GradW64_f32, float>))
