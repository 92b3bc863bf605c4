// Activations in 8 bits and the weight gradient from them: argument checks,
// the gradient's plan and the launches (see act8_kernels.h and
// act8_grad_w_kernels.h).
#include <algorithm>
#include <string>

#include "product_tiles.h"
#include "train.h"

namespace trop {

trop_status check_act8(SpanChecker& checker, const trop_act8& a, int64_t rows, int64_t cols, const char* what) {
    const trop_status st = checker.matrix(a.codes, rows, cols, a.ld, 1, (std::string(what) + " codes").c_str());
    if (st != TROP_OK) return st;
    return checker.matrix(a.exponents, rows, ceil_div(cols, TROP_ACT8_BLOCK_ELEMS), a.ld_exponents, 1,
                          (std::string(what) + " exponents").c_str());
}

namespace {

static_assert(TROP_ACT8_BLOCK == TROP_ACT8_BLOCK_ELEMS, "the format's block");

constexpr int64_t kPieceBytes = 256 << 20;  // of x as bfloat16, of packed dz
constexpr int64_t kMaxSize = 1 << 22;       // 32-bit offsets within a tile

// Chunks of rows_x x cols_x rows.
void set_chunks(TropAct8Params& p) {
    p.chunks = ceil_div(p.cols_x, TROP_ACT8_CHUNK);
    p.total = p.rows_x * p.chunks;
}

trop_status pack_or_unpack(bool pack, trop_dtype dt, const void* x, int64_t ldx, const trop_act8* a, int64_t rows,
                           int64_t cols, void* stream) {
    if (dt != TROP_F32 && dt != TROP_BF16)
        return fail(TROP_ERR_INVALID_ARGUMENT,
                    "activations are float32 or bfloat16, got dtype " + std::to_string((int)dt));
    if (!a) return fail(TROP_ERR_INVALID_ARGUMENT, "trop_act8 is NULL");
    if (rows < 0 || cols < 0) return fail(TROP_ERR_INVALID_ARGUMENT, "negative size");
    if (rows == 0 || cols == 0) return ok();
    int dev = -1;
    trop_status st = block_device(&dev);
    if (st != TROP_OK) return st;
    SpanChecker checker(dev);
    if ((st = checker.matrix(x, rows, cols, ldx, elem_size(dt), pack ? "x" : "out")) != TROP_OK) return st;
    if ((st = check_act8(checker, *a, rows, cols, "8-bit")) != TROP_OK) return st;
    TropAct8Params p = {};
    p.x = x;
    p.codes = a->codes;
    p.exps = a->exponents;
    p.ldx = ldx;
    p.ldc = a->ld;
    p.lde = a->ld_exponents;
    p.rows = rows;
    p.cols = cols;
    // rows of whole blocks that follow one another are one long row
    if (cols % TROP_ACT8_BLOCK == 0 && ldx == cols && a->ld == cols && a->ld_exponents == cols / TROP_ACT8_BLOCK) {
        p.rows = 1;
        p.cols = rows * cols;
    }
    p.rows_x = p.rows;
    p.cols_x = p.cols;
    set_chunks(p);
    const int id = (pack ? TK_ACT8_PACK : TK_ACT8_UNPACK) + (dt == TROP_BF16);
    const int64_t most = max_groups(256) * 4;
    for (; st == TROP_OK && p.chunk0 < p.total; p.chunk0 += most)
        st = train_launch(dev, (TrainKernelId)id, TROP_T_ACT8, ceil_div(std::min(p.total - p.chunk0, most), 4), 256, &p,
                          static_cast<hipStream_t>(stream));
    return st == TROP_OK ? ok() : st;
}

// ---- weight gradient ---------------------------------------------------------

// Tiles of the product: 0: 256 x 256, 1: 128 x 128, 2: 64 x 64, 3: 64 x 64 with
// four buffers, for few tiles: alone on a CU, or beside one other, a tile waits
// for its loads (1000 tokens x 1001 x 777 bfloat16, 208 tiles: 11.1 us with two
// buffers, 8.1 with four; 512 x 1024 x 1024 float32, 256: 15.0 and 11.0; but 64 x
// 2048 x 2048 bfloat16, 1024: 7.3 and 8.2; and 128 x 128 gain nothing: 26 and 27
// us for 2048 x 2048 x 2048).
constexpr int kTiles = 4;
int64_t grad_w_edge(int tile) { return tile == 3 ? 64 : tile_edge(tile); }
double grad_w_time(int tile, int64_t tiles, double k) {
    if (tile == 3) return tiles <= 256 ? k * 0.27 + 4.0 : (double)ceil_div(tiles, 512) * (k * 0.41 + 4.0);
    return tile_time(tile, tiles, k);
}

struct GradWPlan {
    int64_t parts;             // of dz's values
    int64_t tokens_p;
    int64_t cols, outs;        // of a piece, multiples of 256 where there are several
    int tile;
    int64_t splits;
    size_t xp, dzp, part, bytes;
};

// A piece's columns when a column takes `bytes` of a kPieceBytes buffer: equal
// pieces, multiples of 256.
int64_t piece_columns(int64_t n, int64_t bytes) {
    const int64_t most = std::max<int64_t>(kPieceBytes / bytes / 256 * 256, 256);
    return n <= most ? n : round_up(ceil_div(n, ceil_div(n, most)), 256);
}

// Sizes in range and at least 1.  packed: dz goes through the workspace.
void plan_grad_w(trop_dtype dt, bool packed, int64_t tokens, int64_t cols, int64_t outs, GradWPlan* c) {
    c->parts = dt == TROP_BF16 ? 1 : 3;
    c->tokens_p = round_up(tokens, 64);
    c->cols = piece_columns(cols, c->tokens_p * 2);
    c->outs = packed ? piece_columns(outs, c->tokens_p * 2 * c->parts) : outs;
    const int64_t ktiles = c->tokens_p / 64, cols_p = round_up(c->cols, 64);
    // tile and parts along the tokens with the least time; the parts' sums
    // are written and read again at 4 TB/s, by one more launch
    double least = -1;
    for (int kind = 0; kind < kTiles; ++kind) {
        const int64_t edge = grad_w_edge(kind), tiles = ceil_div(c->cols, edge) * ceil_div(c->outs, edge);
        for (int64_t n = 1; n <= 32 && (n == 1 || (ktiles >= 2 * n && tiles * n <= 2048)); ++n) {
            const double extra = n == 1 ? 0.0 : 4.0 + (double)(2 * n * c->outs * cols_p * 4) / 4e6;
            const double t = grad_w_time(kind, tiles * n, (double)(ceil_div(ktiles, n) * c->parts)) + extra;
            if (least < 0 || t < least) {
                least = t;
                c->tile = kind;
                c->splits = n;
            }
        }
    }
    // a piece's tiles in one launch
    const int64_t edge = grad_w_edge(c->tile);
    const int64_t most = max_groups(tile_threads(c->tile)) / (ceil_div(c->cols, edge) * c->splits) * edge / 256 * 256;
    if (c->outs > most) c->outs = most;
    c->bytes = 256;  // room to align the caller's pointer
    auto take = [&](size_t* at, int64_t bytes) {
        *at = c->bytes;
        c->bytes += (size_t)round_up(bytes, 256);
    };
    take(&c->xp, c->tokens_p * cols_p * 2);
    if (packed) take(&c->dzp, c->tokens_p * round_up(c->outs, 64) * 2 * c->parts);
    if (c->splits > 1) take(&c->part, c->splits * c->outs * cols_p * 4);
}

trop_status check_grad_w(trop_dtype dt, int64_t tokens, int64_t cols, int64_t outs) {
    if (dt != TROP_F32 && dt != TROP_BF16)
        return fail(TROP_ERR_INVALID_ARGUMENT, "the weight gradient is float32 or bfloat16, got dtype " +
                                                   std::to_string((int)dt));
    if (tokens < 0 || cols < 0 || outs < 0) return fail(TROP_ERR_INVALID_ARGUMENT, "negative size");
    if (tokens > kMaxSize || cols > kMaxSize || outs > kMaxSize)
        return fail(TROP_ERR_UNSUPPORTED, "more than 2^22 tokens, columns or output features");
    return TROP_OK;
}

// Can the product read dz where it lies?  16-byte chunks of rows.
bool direct_dz(trop_dtype dt, const void* dz, int64_t lddz, int64_t outs) {
    return dt == TROP_BF16 && outs % 8 == 0 && lddz % 8 == 0 && lddz <= kMaxSize &&
           reinterpret_cast<uintptr_t>(dz) % 16 == 0;
}

trop_status finish(int dev, trop_dtype dt, TropGradWParams p, hipStream_t s) {
    const int64_t total = p.outs * ceil_div(p.cols, 1024), most = max_groups(256);
    trop_status st = TROP_OK;
    for (; st == TROP_OK && p.id0 < total; p.id0 += most)
        st = train_launch(dev, (TrainKernelId)(TK_GRAD_W_FINISH + (dt == TROP_BF16)), TROP_T_ACT8_GRAD_W,
                          std::min(total - p.id0, most), 256, &p, s);
    return st;
}

trop_status grad_w(trop_dtype dt, const void* dz, int64_t lddz, const trop_act8* x, void* grad_w, int64_t ldgw,
                   int64_t tokens, int64_t cols, int64_t outs, void* workspace, size_t workspace_bytes, void* stream) {
    trop_status st = check_grad_w(dt, tokens, cols, outs);
    if (st != TROP_OK) return st;
    if (!x) return fail(TROP_ERR_INVALID_ARGUMENT, "trop_act8 is NULL");
    if (cols == 0 || outs == 0) return ok();
    int dev = -1;
    if ((st = block_device(&dev)) != TROP_OK) return st;
    const size_t eb = elem_size(dt);
    SpanChecker checker(dev);
    if (tokens > 0) {
        if ((st = checker.matrix(dz, tokens, outs, lddz, eb, "dz")) != TROP_OK) return st;
        if ((st = check_act8(checker, *x, tokens, cols, "x's")) != TROP_OK) return st;
    }
    if ((st = checker.matrix(grad_w, outs, cols, ldgw, eb, "grad_w")) != TROP_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    TropGradWParams p = {};
    p.lddz = lddz;
    p.ldgw = ldgw;
    p.tokens = tokens;
    if (tokens == 0) {
        p.grad_w = grad_w;
        p.cols = cols;
        p.outs = outs;
        st = finish(dev, dt, p, s);
        return st == TROP_OK ? ok() : st;
    }
    const bool packed = !direct_dz(dt, dz, lddz, outs);
    GradWPlan c = {};
    plan_grad_w(dt, packed, tokens, cols, outs, &c);
    if (!workspace || workspace_bytes < c.bytes)
        return fail(TROP_ERR_WORKSPACE_TOO_SMALL, "the weight gradient needs " + std::to_string(c.bytes) +
                                                      " workspace bytes, got " +
                                                      std::to_string(workspace ? workspace_bytes : 0));
    if ((st = checker.span(workspace, (int64_t)c.bytes, 1, "workspace")) != TROP_OK) return st;
    // (offsets start after the room for alignment)
    char* ws = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(workspace) + 255) / 256 * 256) - 256;
    p.tokens_p = c.tokens_p;
    p.splits = (int32_t)c.splits;
    p.xp = ws + c.xp;
    p.dzp = packed ? ws + c.dzp : nullptr;
    p.part = reinterpret_cast<float*>(ws + c.part);
    const int64_t edge = grad_w_edge(c.tile);
    for (int64_t c0 = 0; st == TROP_OK && c0 < cols; c0 += c.cols) {
        p.cols = std::min(c.cols, cols - c0);
        p.cols_p = round_up(p.cols, 64);
        p.x = {};
        p.x.x = p.xp;
        p.x.codes = x->codes + c0;
        p.x.exps = x->exponents + c0 / TROP_ACT8_BLOCK;
        p.x.ldx = p.x.cols_x = p.cols_p;
        p.x.ldc = x->ld;
        p.x.lde = x->ld_exponents;
        p.x.rows = tokens;
        p.x.cols = p.cols;
        p.x.rows_x = c.tokens_p;
        set_chunks(p.x);
        for (int64_t o0 = 0; st == TROP_OK && o0 < outs; o0 += c.outs) {
            p.outs = std::min(c.outs, outs - o0);
            p.outs_p = round_up(p.outs, 64);
            p.dz = static_cast<const char*>(dz) + o0 * eb;
            p.grad_w = static_cast<char*>(grad_w) + (o0 * ldgw + c0) * eb;
            p.x_groups = o0 == 0 ? (uint32_t)ceil_div(p.x.total, 4) : 0;
            const int64_t dz_groups = packed ? ceil_div(c.tokens_p * ceil_div(p.outs_p, 512), 4) : 0;
            st = train_launch(dev, (TrainKernelId)(TK_GRAD_W_PACK + (dt == TROP_BF16)), TROP_T_ACT8_GRAD_W,
                              p.x_groups + dz_groups, 256, &p, s);
            if (st == TROP_OK)
                st = train_launch(dev, (TrainKernelId)(TK_GRAD_W + 2 * c.tile + (dt == TROP_BF16)), TROP_T_ACT8_GRAD_W,
                                  ceil_div(p.cols, edge) * ceil_div(p.outs, edge) * c.splits, tile_threads(c.tile), &p,
                                  s);
            if (st == TROP_OK && c.splits > 1) st = finish(dev, dt, p, s);
        }
    }
    return st == TROP_OK ? ok() : st;
}

}  // namespace
}  // namespace trop

extern "C" trop_status tropical_act8_pack(trop_dtype dtype, const void* x, int64_t ldx, const trop_act8* out,
                                          int64_t rows, int64_t cols, void* stream) {
    return trop::guarded("tropical_act8_pack",
                         [&] { return trop::pack_or_unpack(true, dtype, x, ldx, out, rows, cols, stream); });
}

extern "C" trop_status tropical_act8_unpack(const trop_act8* in, trop_dtype dtype, void* out, int64_t ldo, int64_t rows,
                                            int64_t cols, void* stream) {
    return trop::guarded("tropical_act8_unpack",
                         [&] { return trop::pack_or_unpack(false, dtype, out, ldo, in, rows, cols, stream); });
}

extern "C" trop_status tropical_act8_linear_grad_w(trop_dtype dtype, const void* dz, int64_t lddz, const trop_act8* x,
                                                   void* grad_w, int64_t ldgw, int64_t tokens, int64_t cols,
                                                   int64_t out_features, void* workspace, size_t workspace_bytes,
                                                   void* stream) {
    return trop::guarded("tropical_act8_linear_grad_w", [&] {
        return trop::grad_w(dtype, dz, lddz, x, grad_w, ldgw, tokens, cols, out_features, workspace, workspace_bytes,
                            stream);
    });
}

extern "C" trop_status tropical_act8_linear_grad_w_workspace_size(trop_dtype dtype, int64_t tokens, int64_t cols,
                                                                  int64_t out_features, size_t* bytes) {
    using namespace trop;
    return guarded("tropical_act8_linear_grad_w_workspace_size", [&]() -> trop_status {
        if (!bytes) return fail(TROP_ERR_INVALID_ARGUMENT, "bytes is NULL");
        *bytes = 0;
        const trop_status st = check_grad_w(dtype, tokens, cols, out_features);
        if (st != TROP_OK) return st;
        if (tokens == 0 || cols == 0 || out_features == 0) return ok();
        for (const bool packed : {true, false}) {
            GradWPlan c = {};
            plan_grad_w(dtype, packed, tokens, cols, out_features, &c);
            *bytes = std::max(*bytes, c.bytes);
        }
        return ok();
    });
}
