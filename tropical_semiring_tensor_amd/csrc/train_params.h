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

// ---- activations in 8 bits --------------------------------------------------
// Elements of a row that share an exponent; elements of a wave's chunk of a row.
#define TROP_ACT8_BLOCK_ELEMS 32
#define TROP_ACT8_CHUNK 1024

struct TropAct8Params {
    const void* x;        // packing: the rows; unpacking: written
    int8_t* codes;
    uint8_t* exps;
    int64_t ldx, ldc, lde;
    int64_t rows, cols;   // of the codes
    int64_t rows_x, cols_x;  // unpacking: of the rows (zeros past the codes)
    int64_t chunks;       // of a row
    int64_t chunk0;       // the launch's first chunk
    int64_t total;        // chunks in all
};

// Operands of the weight gradient, then its product: piece [c0, c0 + cols) x
// [o0, o0 + outs) of the gradient.
struct TropGradWParams {
    TropAct8Params x;     // unpacked into xp
    const void* dz;       // at the piece's first output feature
    void* grad_w;         // at the piece's first element
    void* xp;             // [tokens_p][cols_p] bfloat16
    void* dzp;            // packed dz: [tokens_p / 64][parts][64][outs_p] bfloat16, or null: dz as it lies
    float* part;          // [splits][outs][cols_p], when splits > 1
    int64_t lddz, ldgw;
    int64_t tokens, tokens_p, cols, cols_p, outs, outs_p;
    int64_t id0;          // finishing: the launch's first workgroup
    uint32_t x_groups;    // packing: workgroups that unpack x, before those that pack dz
    int32_t splits;
};

// ---- between two residual blocks ---------------------------------------------
// Widest row whose sums the backward keeps in registers, and the widest of its
// rows' gradients alone (1024 threads of 8 and of 16 columns).
#define TROP_RN_COLS_ALL 8192
#define TROP_RN_COLS_ROWS 16384
// Columns of a workgroup of wide rows' sums.
#define TROP_RN_COLS_SUMS 2048
// Column sums: gradients of the pre norm's weights, the post norm's, the gate.
enum { TROP_RN_PRE_GAMMA, TROP_RN_PRE_BETA, TROP_RN_POST_GAMMA, TROP_RN_POST_BETA, TROP_RN_GATE, TROP_RN_SUMS };

struct TropResidualParams {
    const void* r;          // forward, may be null
    const void* u;
    const void* gate;       // may be null
    const void* post_gamma; // may be null
    const void* post_beta;
    const void* pre_gamma;
    const void* pre_beta;
    const void* dy;         // backward
    const void* dh;
    void* h;                // forward: written, may be null; backward: read
    void* y;
    void* dr;
    void* du;
    void* dgate;            // gate rows that a part takes whole are written here
    float* post_mean;
    float* post_rstd;
    float* pre_mean;
    float* pre_rstd;
    int8_t* u_codes;        // forward: written, may be null; backward: read
    uint8_t* u_exps;
    int8_t* h_codes;
    uint8_t* h_exps;
    float* part[TROP_RN_SUMS];  // backward: [parts][cols] each, null where not asked for
    float* row_sums;        // backward of wide rows: [rows][2], the pre norm's two means
    int64_t ldr, ldu, ldgate, lddy, lddh, ldh, ldy, lddr, lddu, lddgate, ldu_codes, ldu_exps, ldh_codes, ldh_exps;
    int64_t rows, cols;
    int64_t row0;           // the launch's first row
    int64_t col0;           // wide rows' sums: the launch's first block of columns (narrow ones': column)
    int64_t gate_group;     // rows of a gate row (rows or more: one gate row)
    int64_t part_rows;      // backward: rows of a part
    int64_t group_parts;    // backward: parts of a gate row, or 0: a part takes whole gate rows
    float residual_scale, branch_scale, post_eps, pre_eps, inv_cols;
    int32_t post, pre;      // trop_norm
    int32_t gate_f32, weight_f32;
    int32_t parts;
    int32_t need_v, need_post;  // backward: the gate's gradient; the post norm's gradients or du through it
    int32_t ragged;         // backward: rows that end inside a 16-byte vector
    int32_t pad_;
};

// Partial sums of up to TROP_RN_SUMS column sums: entry i has `rows[i]` output
// rows, each the sum of `parts` consecutive rows of src.
struct TropRowSumsEntry {
    const float* src;
    void* dst;
    int64_t ldd, rows, parts;
    uint32_t blocks;        // workgroups of this entry and all before it
    int32_t f32;
    float scale;
    int32_t column_bits;    // log2 of a workgroup's columns
};
struct TropRowSumsParams {
    TropRowSumsEntry e[TROP_RN_SUMS];
    int64_t cols, id0;      // id0: the launch's first workgroup
    int32_t count, pad_;
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
