// Argument blocks of the training operators' kernels, passed by value to
// every launch (host runtime and device code agree on the layout; no pointer
// in them is kept after a call returns).
#pragma once
#include <stdint.h>

// ---- layer norm ------------------------------------------------------------
// Partial column sums (dgamma, dbeta) a backward call makes at most.
#define TROP_LN_MAX_PARTS 512
// Columns a wave / 256 threads / 1024 threads hold in registers (16 each).
#define TROP_LN_COLS_WAVE 1024
#define TROP_LN_COLS_BLOCK 4096
#define TROP_LN_COLS_WIDE 16384

struct TropLayerNormParams {
    const void* x;
    const void* dy;     // backward
    const void* gamma;  // may be null
    const void* beta;   // forward, may be null
    void* y;            // forward: y; backward: dx (may be null)
    float* mean;        // forward: written, may be null; backward: read
    float* rstd;
    float* part;        // backward: [2][parts][cols], null without dgamma and dbeta
    int64_t ldx, lddy, ldy;
    int64_t rows, cols;
    int64_t col0;       // partial column sums of wide rows: the launch's first column
    float eps, inv_cols;
    int32_t parts;      // workgroups of the backward
    int32_t pad_;
};

struct TropLayerNormMergeParams {
    const float* part;
    void* dgamma;  // may be null
    void* dbeta;   // may be null
    int64_t cols, col0;  // col0: the launch's first column
    int32_t parts;
    int32_t pad_;
};

// ---- AdamW -----------------------------------------------------------------
// Elements of one workgroup's chunk of a tensor, and of a scale's block.
#define TROP_ADAMW_CHUNK 4096
#define TROP_ADAMW_BLOCK_ELEMS 256
// Tensors of one launch (a 4 KiB argument block).
#define TROP_ADAMW_TENSORS 72
#define TROP_ADAMW8_TENSORS 56

struct TropAdamwScalars {
    float beta1, one_minus_beta1, beta2, one_minus_beta2;
    float keep;       // 1 - lr weight_decay
    float step_size;  // lr / (1 - beta1^step)
    float root;       // 1 / sqrt(1 - beta2^step)
    float eps;
};

struct TropAdamwEntry {
    void* param;
    const void* grad;
    float* m;
    float* v;
    float* master;
    int64_t n;
};

struct TropAdamwParams {
    TropAdamwScalars s;
    int32_t count, pad_;
    uint32_t chunk_end[TROP_ADAMW_TENSORS];  // chunks of this tensor and all before it
    TropAdamwEntry t[TROP_ADAMW_TENSORS];
};

struct TropAdamw8Entry {
    void* param;        // unpack: float values of m (may be null)
    const void* grad;
    int8_t* m;
    float* m_scale;
    uint8_t* v;
    float* v_scale;
    float* master;      // unpack: float values of v (may be null)
    int64_t n;
};

struct TropAdamw8Params {
    TropAdamwScalars s;
    int32_t count, pad_;
    uint32_t chunk_end[TROP_ADAMW8_TENSORS];
    TropAdamw8Entry t[TROP_ADAMW8_TENSORS];
};

// ---- linear cross entropy --------------------------------------------------
// Tokens up to this many may take the streaming kernels (no packing).
#define TROP_CE_FEW 64
// Blocks of 16 labels that a workgroup of its logits takes when there are
// plenty, for nb blocks of 16 tokens: they share the tokens' loads, as far as
// the registers go.  Two blocks and four, 26 tokens x 2560 x 58817: float32's
// G 189 and 171 us; 60 tokens: bfloat16 137 and 97, but float32 300 and 326.
constexpr int trop_ce_few_rows(int nb, int elem_bytes) {
    return nb == 2 || (nb == 4 && elem_bytes == 2) ? 4 : 2;
}
// Workgroups of the magnitude pass, each leaving two partial maxima.
#define TROP_CE_MAX_PARTS 256

// Scalars that the first kernels of a call leave for the later ones.
struct TropCeControl {
    int32_t kept;      // tokens that count
    float grad_max;    // largest finite |grad_loss| of a kept token (1 when that is 0)
    int32_t x_exp;     // float32 operands: x 2^x_exp and w 2^w_exp are split
    int32_t w_exp;     // into float16 planes
};

struct TropCeParams {
    const void* x;
    const void* w;
    const void* target;
    const float* lse_in;      // backward
    const float* grad_loss;   // backward
    float* loss;              // forward
    float* lse;               // forward
    void* grad_x;
    void* grad_w;
    int64_t ldx, ldw, ldgx, ldgw, grad_loss_stride, ignore_index;
    int64_t tokens, width, vocab;
    // workspace
    TropCeControl* control;
    int32_t* rows;            // kept index -> token
    int32_t* slot;            // token -> kept index or -1
    int32_t* kept_target;     // per kept token
    float* kept_lse;
    float* kept_grad;         // grad_loss / grad_max
    float* magnitude;         // [2][TROP_CE_MAX_PARTS]
    float* stats;             // forward: [token][tiles][2] maximum and sum of exponentials
    float* target_logit;      // per kept token (per token in the streaming kernel)
    void* xp;                 // packed x: [padded][width_p], float32 [padded][width_p / 32][2][32]
    void* wp;                 // packed piece of w: [piece] rows likewise
    void* g;                  // piece of the logits' gradient: [planes][piece / 4][padded][4]; float32: upper, lower 16 bits
    float* label_max;         // float32: its largest finite magnitudes, [tokens / logits_edge][piece]
    int32_t* label_exp;       // float32: the exponents of grad_w's scales, when gw_splits > 1
    float* gx_part;           // [splits][padded][width_p]
    float* gw_part;           // [gw_splits][piece][width_p], when gw_splits > 1
    int64_t padded, width_p;
    int64_t logits_edge;      // tokens of a logits tile
    int64_t v0, piece;        // this launch's labels: [v0, v0 + piece), piece a multiple of the tile
    int64_t tile0;            // first statistics tile of this launch
    int64_t row0;             // finishing grad_x: the launch's first token
    int64_t tiles;            // statistics tiles in all
    int32_t target_bytes;
    int32_t w_packed;         // the piece is read from wp (else from w itself)
    int32_t splits, split_tiles;  // gx: parts along the labels and k tiles of each
    int32_t gw_splits;        // gw: parts along the tokens
    uint32_t gx_groups;       // workgroups of grad_x, before grad_w's (a multiple of 8)
    int32_t accumulate;       // gx: add to what the piece before left
    int32_t max_parts;        // workgroups of the magnitude pass
    int32_t pack_x;           // packing: workgroups that take rows of x
    int32_t identity;         // merge: kept index = token (streaming kernel)
    int32_t backward;
};

static_assert(sizeof(TropAdamwParams) <= 4096 && sizeof(TropAdamw8Params) <= 4096, "kernel argument block");
