// Linear cross entropy: argument checks, the plan of a call (tiles, pieces
// of the label set, workspace layout) and its launches (see
// cross_entropy_kernels.h).
#include <algorithm>
#include <string>

#include "product_tiles.h"
#include "train.h"

namespace trop {
namespace {

constexpr int64_t kBK = 64;               // k of a product's tile
constexpr int64_t kPieceBytes = 256 << 20;  // of a piece of G, and of packed w
constexpr int64_t kMaxTokens = 1 << 22, kMaxWidth = 1 << 22;  // 32-bit offsets within a tile
constexpr int64_t kLargeElements = 10 << 20;  // of a w that few tokens' tiles read as it lies
constexpr int64_t kTileElements = 16 << 20;  // of a bfloat16 w for 33 to 64 tokens' logits in tiles
constexpr int64_t kMaxVocab = ((int64_t)1 << 31) - 512;       // label indices are 32-bit

// A piece's labels when a label takes `bytes` of a kPieceBytes buffer: equal
// pieces, multiples of 256.
int64_t piece_labels(int64_t vocab, int64_t bytes) {
    int64_t most = kPieceBytes / bytes / 256 * 256;
    if (most < 256) most = 256;
    return round_up(ceil_div(vocab, ceil_div(vocab, most)), 256);
}

// Time of `tx` tiles over kx, then `tw` over kw in one launch: a slot that
// the first leave takes the second's.
double pair_time(int kind, int64_t tx, double kx, int64_t tw, double kw) {
    const TileRate x = tile_rate(kind, tx + tw, kx), w = tile_rate(kind, tx + tw, kw);
    // after `full` rounds of the first, `late` slots have one more of them
    const int64_t full = tx / x.slots, late = tx % x.slots, free = x.slots - late;
    const double lag = x.us / w.us;
    // rounds of the second when it ends in the free slots, or in the late ones
    const int64_t whole = (int64_t)lag;
    int64_t i = std::min(ceil_div(tw, free), (tw + late * whole) / x.slots);
    int64_t j = std::max<int64_t>(0, (tw - free * (whole + 1)) / x.slots);
    while (free * i + late * std::max<int64_t>(0, (int64_t)((double)i - lag)) < tw) ++i;
    while (free * (int64_t)((double)j + lag) + late * j < tw) ++j;
    return full * x.us + std::max(late ? x.us : 0.0, std::min(i * w.us, x.us + j * w.us));
}

// The logits' product: the 64 x 64 tiles have four buffers, and so do the 128 x
// 128 (kind 3) where a CU has no more than one of them: with no other workgroup
// beside it a tile waits for its loads (66 tokens x 1856 x 25495 float32, 200
// tiles of 128: 77 us with two buffers, 61 with four; 110 x 3392 x 7405, 232
// tiles of 64: 63 and 41; but 303 x 1856 x 16810, 396 of 128: 84 and 106).  A 64
// x 64 one takes 0.27 us a k tile alone on a CU, 0.41 beside another.
double logits_time(int kind, int64_t tiles, double k) {
    if (kind == 2) return tiles <= 256 ? k * 0.27 + 4.0 : (double)ceil_div(tiles, 512) * (k * 0.41 + 4.0);
    if (kind == 3) return (double)ceil_div(tiles, 256) * (k * 0.77 + 5.0);
    if (kind == 1) return (double)ceil_div(tiles, 512) * (k * 1.15 + 5.0);
    return tile_time(kind, tiles, k);
}

// The gradients of `tokens` x `labels` of G: tile and parts along k with the
// least time.  kx, kw: k tiles (`unit` of a tile_rate's each).  A part's sums
// are written and read again at 4 TB/s; grad_w's parts take one more launch.
// How many tokens count is not known here, and a part of grad_x that is right
// for all of them can outlast the rest when some are left out (1000 x 1000 x
// 50001, bfloat16, a third ignored: 197 us in 7 parts, 164 in 10): the time
// is the mean over all and half of them.
struct GradTiles {
    int tile;
    int64_t splits, gw_splits;
};
GradTiles choose_grad_tiles(bool raw, int64_t tokens, int64_t labels, int64_t width, int64_t kx, int64_t kw, double unit,
                            int64_t gx_bytes, int64_t gw_bytes) {
    GradTiles best = {0, 1, 1};
    double least = -1;
    for (int kind = raw ? 1 : 0; kind < 3; ++kind) {
        const int64_t edge = tile_edge(kind), columns = ceil_div(width, edge);
        const int64_t tx = ceil_div(tokens, edge) * columns, tw = ceil_div(labels, edge) * columns;
        const int64_t tx_half = ceil_div((tokens + 1) / 2, edge) * columns;
        int64_t m = 1;
        double wtime = tile_time(kind, tw, (double)kw * unit), wextra = 0;
        for (int64_t n = 2; n <= 16 && kw / n >= 8 && tw * n <= 1024; ++n) {
            const double extra = 4.0 + (double)(2 * n * gw_bytes) / 4e6;
            const double t = tile_time(kind, tw * n, (double)ceil_div(kw, n) * unit) + extra;
            if (t < wtime) {
                wtime = t;
                wextra = extra;
                m = n;
            }
        }
        const double ww = (double)ceil_div(kw, m) * unit, ww_half = (double)ceil_div((kw + 1) / 2, m) * unit;
        for (int64_t n = 1; n <= 32 && (n == 1 || kx / n >= 8); n += 1 + n / 8) {
            if (tx * n + tw * m + 8 > max_groups(tile_threads(kind))) break;  // one launch
            const double wx = (double)ceil_div(kx, n) * unit;
            const double t = wextra + (double)(2 * n * gx_bytes) / 4e6 +
                             (pair_time(kind, tx * n, wx, tw * m, ww) + pair_time(kind, tx_half * n, wx, tw * m, ww_half)) / 2;
            if (least < 0 || t < least) {
                least = t;
                best = {kind, n, m};
            }
        }
    }
    return best;
}

struct CePlan {
    int64_t planes, padded, width_p;
    bool few;           // few tokens: streaming kernels, no packing
    bool packed;        // w is read from packed pieces
    bool raw;           // float32 w is read as it lies
    int64_t piece;      // labels of a piece (a multiple of 256; forward unpacked: all, but for a launch's limit)
    int logits_tile, grad_tile;  // 0: 256, 1: 128, 2: 64, 3: 128 with four buffers
    int few_blocks;     // streaming kernels: log2 of the blocks of 16 tokens
    int few_rows;       // and blocks of 16 labels of a logits workgroup
    int64_t tiles;      // statistics per token
    int64_t splits, gw_splits;
    int64_t split_tiles;  // streaming grad_x: rounds of a part
    int64_t max_parts;
    // workspace offsets
    size_t control, rows, slot, kept_target, kept_lse, kept_grad, magnitude, stats, target_logit, xp, wp, g, label_max,
        label_exp, gx_part, gw_part;
    size_t bytes;
};

bool take(CePlan* c, size_t* at, int64_t bytes) {
    *at = c->bytes;
    int64_t next;
    if (__builtin_add_overflow((int64_t)c->bytes, bytes, &next) || next > ((int64_t)1 << 62)) return false;
    c->bytes = (size_t)round_up(next, 256);
    return true;
}

// Workgroups of the streaming gradients that run at once on 256 CUs, by their
// registers (for 1, 2, 4 blocks of tokens: grad_x 112, 152, 232 in float32,
// 152, 220 in bfloat16; grad_w 100, 112, 144 and 152, 168).
int64_t few_slots(trop_dtype dt, int few_blocks, bool grad_x) {
    static constexpr int x[2][3] = {{4, 3, 2}, {3, 2, 2}}, w[2][3] = {{4, 4, 3}, {3, 3, 3}};
    return 256 * (grad_x ? x : w)[dt == TROP_BF16][few_blocks];
}

// Streaming kernels (at most TROP_CE_FEW tokens).
bool plan_few(trop_dtype dt, int64_t tokens, int64_t width, int64_t vocab, bool backward, CePlan* c) {
    c->few = true;
    c->few_blocks = tokens <= 16 ? 0 : tokens <= 32 ? 1 : 2;
    const int64_t np = (int64_t)16 << c->few_blocks;
    // (one block of labels where more would leave fewer than four workgroups
    // of two for each CU)
    c->few_rows = vocab >= 1024 * 32 ? trop_ce_few_rows(1 << c->few_blocks, (int)elem_size(dt)) : 1;
    bool ok = true;
    if (!backward) {
        c->piece = vocab;
        c->tiles = ceil_div(vocab, 16 * c->few_rows);
        ok &= take(c, &c->stats, tokens * c->tiles * 8);
        ok &= take(c, &c->target_logit, tokens * 4);
        return ok;
    }
    c->piece = piece_labels(vocab, np * 4);
    ok &= take(c, &c->g, (c->piece + 64) * np * 4);
    // grad_x: parts along the labels that the device holds at once, each of
    // at least two rounds of the labels that its four waves take at a time
    const int64_t round = 64;
    const int64_t blocks = ceil_div(width, dt == TROP_BF16 ? 128 : 64), rounds = ceil_div(c->piece, round);
    int64_t n = few_slots(dt, c->few_blocks, true) / blocks;
    if (n > ceil_div(rounds, 2)) n = ceil_div(rounds, 2);
    if (n > 64) n = 64;
    if (n < 1) n = 1;
    c->split_tiles = ceil_div(rounds, n);
    c->splits = ceil_div(rounds, c->split_tiles);
    ok &= take(c, &c->gx_part, c->splits * c->padded * c->width_p * 4);
    return ok;
}

// tokens, width, vocab in range (check_sizes), vocab and width >= 1.
bool plan(trop_dtype dt, int64_t tokens, int64_t width, int64_t vocab, bool backward, bool packed, CePlan* c) {
    *c = CePlan();
    c->planes = dt == TROP_BF16 ? 1 : 2;
    c->width_p = round_up(width, kBK);
    c->bytes = 256;  // room to align the caller's pointer
    c->splits = c->gw_splits = 1;
    // Few tokens take the streaming kernels.  Beyond 32 the tiles are faster
    // where they need no packed copy of a large w, and always in bfloat16's
    // backward, whose streaming form sums widened values (both directions, in
    // tiles and streaming: 65 and 64 tokens x 2560 x 58817 float32 887 and 1085
    // us, 4096 x 8000 288 and 278; forward, bfloat16, 60 tokens: 4096 x 16100 36 and
    // 80, 4096 x 5000 37 and 43, 1024 x 12000 24 and 22, 4096 x 2600 36 and 27).
    const bool large = !packed && vocab * width >= (backward ? kLargeElements : kTileElements);
    const bool tiles = backward ? dt == TROP_BF16 || large : dt == TROP_BF16 && large;
    if (tokens > 0 && tokens <= (tiles ? TROP_CE_FEW / 2 : TROP_CE_FEW)) {
        c->padded = TROP_CE_FEW;
        return plan_few(dt, tokens, width, vocab, backward, c);
    }
    c->padded = round_up(tokens > 0 ? tokens : 1, 256);
    // float32 w as it lies, split by the tiles that read it, saves its packed
    // copy where two tiles of tokens at most read it, but has them wait for
    // the split: forward and backward, packed and as it lies, 66 tokens x 1856
    // x 25495: 467 and 364 us; 250 x 1856 x 16810: 420 and 359; 183 x 320 x
    // 33477 (11 million elements): 171 and 161; 232 x 2560 x 3457 (9 million):
    // 160 and 174; 150 x 1024 x 259: 62 and 75.
    c->raw = dt == TROP_F32 && !packed && tokens <= 256 && vocab * width >= kLargeElements;
    c->packed = packed || (dt == TROP_F32 && !c->raw);
    bool ok = true;
    const int64_t w_row = c->width_p * 2 * c->planes, g_label = c->padded * 2 * c->planes;
    const int64_t count = tokens > 0 ? tokens : 1, kt = kBK / c->planes;
    const double unit = c->planes == 1 ? 1.0 : 1.25;
    const bool whole = !backward && !c->packed;  // one launch over all labels
    c->piece = round_up(vocab, 256);
    if (!whole) {
        int64_t bytes = c->packed ? w_row : 0;
        if (backward && g_label > bytes) bytes = g_label;
        c->piece = piece_labels(vocab, bytes);
    }
    const int64_t labels = c->piece < vocab ? c->piece : vocab;
    const double wtiles = (double)ceil_div(width, kt) * unit;
    double best = -1;
    for (int kind = c->raw ? 1 : 0; kind < 4; ++kind) {
        const int64_t edge = tile_edge(kind);
        const double t = logits_time(kind, ceil_div(labels, edge) * ceil_div(count, edge), wtiles);
        if (best < 0 || t < best) {
            best = t;
            c->logits_tile = kind;
        }
    }
    // a piece's logits in one launch
    const int64_t edge = tile_edge(c->logits_tile);
    const int64_t most = max_groups(tile_threads(c->logits_tile)) / ceil_div(count, edge) * edge / 256 * 256;
    if (c->piece > most) c->piece = most;
    ok &= take(c, &c->control, sizeof(TropCeControl));
    ok &= take(c, &c->rows, c->padded * 4);
    ok &= take(c, &c->slot, c->padded * 4);
    ok &= take(c, &c->kept_target, c->padded * 4);
    if (c->planes == 2) {
        c->max_parts = TROP_CE_MAX_PARTS;
        ok &= take(c, &c->magnitude, 2 * TROP_CE_MAX_PARTS * 4);
    }
    ok &= take(c, &c->xp, c->padded * c->width_p * 2 * c->planes);
    if (c->packed) ok &= take(c, &c->wp, c->piece * w_row);
    if (!backward) {
        c->tiles = ceil_div(vocab, tile_edge(c->logits_tile));
        ok &= take(c, &c->stats, tokens * c->tiles * 8);
        ok &= take(c, &c->target_logit, c->padded * 4);
        return ok;
    }
    ok &= take(c, &c->kept_lse, c->padded * 4);
    ok &= take(c, &c->kept_grad, c->padded * 4);
    // (the weight's 256-label tiles may read past a piece that ends at 128)
    ok &= take(c, &c->g, (c->piece + 256) * g_label);
    if (c->planes == 2) {
        ok &= take(c, &c->label_max, ceil_div(count, tile_edge(c->logits_tile)) * c->piece * 4);
        ok &= take(c, &c->label_exp, c->piece * 4);
    }
    const int64_t part = c->padded * c->width_p * 4;
    const GradTiles t = choose_grad_tiles(c->raw, count, labels, width, ceil_div(labels, kt), ceil_div(count, kt), unit, part,
                                          labels * c->width_p * 4);
    c->grad_tile = t.tile;
    c->splits = t.splits;
    c->gw_splits = t.gw_splits;
    ok &= take(c, &c->gx_part, c->splits * part);
    if (c->gw_splits > 1) ok &= take(c, &c->gw_part, c->gw_splits * c->piece * c->width_p * 4);
    return ok;
}

trop_status check_sizes(trop_dtype dt, int64_t tokens, int64_t width, int64_t vocab) {
    if (dt != TROP_F32 && dt != TROP_BF16)
        return fail(TROP_ERR_INVALID_ARGUMENT,
                    "linear cross entropy takes float32 or bfloat16, got dtype " + std::to_string((int)dt));
    if (tokens < 0 || width < 0 || vocab < 0) return fail(TROP_ERR_INVALID_ARGUMENT, "negative size");
    if (tokens > 0 && (width < 1 || vocab < 1))
        return fail(TROP_ERR_INVALID_ARGUMENT, "tokens need a width and a vocabulary of at least 1");
    if (tokens > kMaxTokens || width > kMaxWidth || vocab > kMaxVocab)
        return fail(TROP_ERR_UNSUPPORTED, "more than 2^22 tokens, a width above 2^22 or 2^31 labels");
    return TROP_OK;
}

// Can the products read w where it lies?  16-byte rows, and row offsets
// within a tile that fit 32 bits.
bool direct_w(trop_dtype dt, const void* w, int64_t ldw, int64_t width) {
    const int64_t chunk = dt == TROP_BF16 ? 8 : 4;
    return width % chunk == 0 && ldw % chunk == 0 && ldw <= kMaxWidth && reinterpret_cast<uintptr_t>(w) % 16 == 0;
}

struct CeCall {
    trop_dtype dt;
    const void *x, *w, *target;
    int64_t ldx, ldw;
    int target_bytes;
    int64_t ignore_index;
    int64_t tokens, width, vocab;
    void* workspace;
    size_t workspace_bytes;
    void* stream;
};

trop_status check_inputs(const CeCall& a, SpanChecker& checker) {
    const size_t eb = elem_size(a.dt);
    trop_status st;
    if (a.tokens > 0) {
        if ((st = checker.matrix(a.x, a.tokens, a.width, a.ldx, eb, "x")) != TROP_OK) return st;
        if ((st = checker.span(a.target, a.tokens, a.target_bytes, "target")) != TROP_OK) return st;
    }
    return checker.matrix(a.w, a.vocab, a.width, a.ldw, eb, "w");
}

trop_status check_workspace(const CeCall& a, const CePlan& c, SpanChecker& checker, char** base) {
    if (!a.workspace || a.workspace_bytes < c.bytes)
        return fail(TROP_ERR_WORKSPACE_TOO_SMALL,
                    "linear cross entropy needs " + std::to_string(c.bytes) + " workspace bytes, got " +
                        std::to_string(a.workspace ? a.workspace_bytes : 0));
    const trop_status st = checker.span(a.workspace, (int64_t)c.bytes, 1, "workspace");
    *base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(a.workspace) + 255) / 256 * 256);
    return st;
}

TropCeParams params(const CeCall& a, const CePlan& c, char* ws) {
    TropCeParams p = {};
    p.x = a.x;
    p.w = a.w;
    p.target = a.target;
    p.ldx = a.ldx;
    p.ldw = a.ldw;
    p.target_bytes = a.target_bytes;
    p.ignore_index = a.ignore_index;
    p.tokens = a.tokens;
    p.width = a.width;
    p.vocab = a.vocab;
    ws -= 256;  // (offsets start after the room for alignment)
    p.control = reinterpret_cast<TropCeControl*>(ws + c.control);
    p.rows = reinterpret_cast<int32_t*>(ws + c.rows);
    p.slot = reinterpret_cast<int32_t*>(ws + c.slot);
    p.kept_target = reinterpret_cast<int32_t*>(ws + c.kept_target);
    p.kept_lse = reinterpret_cast<float*>(ws + c.kept_lse);
    p.kept_grad = reinterpret_cast<float*>(ws + c.kept_grad);
    p.magnitude = reinterpret_cast<float*>(ws + c.magnitude);
    p.stats = reinterpret_cast<float*>(ws + c.stats);
    p.target_logit = reinterpret_cast<float*>(ws + c.target_logit);
    p.xp = ws + c.xp;
    p.wp = ws + c.wp;
    p.g = ws + c.g;
    p.label_max = reinterpret_cast<float*>(ws + c.label_max);
    p.label_exp = reinterpret_cast<int32_t*>(ws + c.label_exp);
    p.gx_part = reinterpret_cast<float*>(ws + c.gx_part);
    p.gw_part = reinterpret_cast<float*>(ws + c.gw_part);
    p.padded = c.padded;
    p.width_p = c.width_p;
    p.logits_edge = tile_edge(c.logits_tile);
    p.tiles = c.tiles;
    p.w_packed = c.packed;
    p.splits = (int32_t)c.splits;
    p.gw_splits = (int32_t)c.gw_splits;
    p.identity = c.few;
    p.max_parts = (int32_t)c.max_parts;
    return p;
}

TrainKernelId typed(int id, trop_dtype dt) { return (TrainKernelId)(id + (dt == TROP_BF16 ? 1 : 0)); }

// List the kept tokens (and, for float32, look for the largest magnitudes).
trop_status list_tokens(int dev, const CePlan& c, const TropCeParams& p, hipStream_t s) {
    return train_launch(dev, TK_CE_KEEP, TROP_T_CE_PACK, 1 + c.max_parts, 1024, &p, s);
}

// This piece's labels into p; x packed with the first, and w if it has to be.
trop_status prepare_piece(int dev, const CeCall& a, const CePlan& c, int64_t v0, TropCeParams& p, hipStream_t s) {
    const int64_t labels = a.vocab - v0 < c.piece ? a.vocab - v0 : c.piece;
    p.v0 = v0;
    p.piece = round_up(labels, tile_edge(c.logits_tile));
    p.tile0 = v0 / tile_edge(c.logits_tile);
    p.pack_x = v0 == 0 ? (int32_t)(c.padded / 4) : 0;
    const int64_t groups = p.pack_x + (c.packed ? ceil_div(p.piece, 4) : 0);
    return train_launch(dev, typed(TK_CE_PACK, a.dt), TROP_T_CE_PACK, groups, 256, &p, s);
}

TrainKernelId logits_kernel(int id, int raw_id, const CePlan& c, trop_dtype dt) {
    return c.raw ? (TrainKernelId)(raw_id + c.logits_tile - 1) : typed(id + 2 * c.logits_tile, dt);
}

// A streaming kernel of the family at `id` (`per`: its kernels for one label block).
TrainKernelId few_kernel(int id, int per, const CePlan& c, trop_dtype dt) {
    return typed(id + per * (c.few_rows > 1) + 2 * c.few_blocks, dt);
}

// The backward's pieces with the streaming kernels.
trop_status few_pieces(int dev, const CeCall& a, const CePlan& c, TropCeParams& p, hipStream_t s) {
    trop_status st = TROP_OK;
    const bool bf = a.dt == TROP_BF16;
    for (int64_t v0 = 0; st == TROP_OK && v0 < a.vocab; v0 += c.piece) {
        const int64_t labels = a.vocab - v0 < c.piece ? a.vocab - v0 : c.piece;
        p.v0 = v0;
        p.piece = labels;
        p.accumulate = v0 > 0;
        p.split_tiles = (int32_t)c.split_tiles;
        st = train_launch(dev, few_kernel(TK_CE_FEW_GRAD, 5, c, a.dt), TROP_T_CE_LOGITS,
                          ceil_div(labels, 16 * c.few_rows), 256, &p, s);
        if (st == TROP_OK && p.grad_x)
            st = train_launch(dev, few_kernel(TK_CE_FEW_GX, 0, c, a.dt), TROP_T_CE_GRAD,
                              ceil_div(a.width, bf ? 128 : 64) * c.splits, 256, &p, s);
        if (st == TROP_OK && p.grad_w) {
            // a workgroup's labels; the columns in as many parts as make the
            // rounds of workgroups shortest
            const int64_t groups = ceil_div(labels, 128), slots = few_slots(a.dt, c.few_blocks, false);
            const int64_t most = std::min(ceil_div(a.width, bf ? 128 : 64), std::max<int64_t>(4, slots / groups));
            int64_t parts = 1;
            for (int64_t n = 2; n <= most; ++n)
                if (ceil_div(groups * n, slots) * parts < ceil_div(groups * parts, slots) * n) parts = n;
            st = train_launch(dev, few_kernel(TK_CE_FEW_GW, 0, c, a.dt), TROP_T_CE_GRAD, groups * parts, 256, &p, s);
        }
    }
    return st;
}

// The backward's pieces with the products' tiles.
trop_status tile_pieces(int dev, const CeCall& a, const CePlan& c, TropCeParams& p, hipStream_t s) {
    const int64_t tokens = a.tokens > 0 ? a.tokens : 1;
    trop_status st = list_tokens(dev, c, p, s);
    for (int64_t v0 = 0; st == TROP_OK && v0 < a.vocab; v0 += c.piece) {
        const int64_t labels = a.vocab - v0 < c.piece ? a.vocab - v0 : c.piece;
        st = prepare_piece(dev, a, c, v0, p, s);
        if (st == TROP_OK && a.tokens > 0) {
            const int64_t edge = tile_edge(c.logits_tile);
            st = train_launch(dev, logits_kernel(TK_CE_GRAD, TK_CE_GRAD_RAW, c, a.dt), TROP_T_CE_LOGITS,
                              p.piece / edge * ceil_div(tokens, edge), tile_threads(c.logits_tile), &p, s);
        }
        if (st == TROP_OK) {
            const int64_t edge = tile_edge(c.grad_tile), columns = ceil_div(a.width, edge);
            const int64_t gx = p.grad_x ? round_up(ceil_div(tokens, edge) * columns * c.splits, 8) : 0;
            const int64_t gw = p.grad_w ? ceil_div(labels, edge) * columns * c.gw_splits : 0;
            p.split_tiles = (int32_t)ceil_div(ceil_div(labels, kBK / c.planes), c.splits);
            p.accumulate = v0 > 0;
            p.gx_groups = (uint32_t)gx;
            st = train_launch(dev,
                              c.raw ? (TrainKernelId)(TK_CE_GRADIENTS_RAW + c.grad_tile - 1)
                                    : typed(TK_CE_GRADIENTS + 2 * c.grad_tile, a.dt),
                              TROP_T_CE_GRAD, gx + gw, tile_threads(c.grad_tile), &p, s);
            if (st == TROP_OK && p.grad_w && c.gw_splits > 1)
                st = train_launch(dev, typed(TK_CE_FINISH_W, a.dt), TROP_T_CE_MERGE,
                                  labels * ceil_div(a.width, 1024), 256, &p, s);
        }
    }
    return st;
}

trop_status ce_forward(const CeCall& a, float* loss, float* lse) {
    trop_status st = check_sizes(a.dt, a.tokens, a.width, a.vocab);
    if (st != TROP_OK) return st;
    if (a.target_bytes != 4 && a.target_bytes != 8)
        return fail(TROP_ERR_INVALID_ARGUMENT, "targets have 4 or 8 bytes");
    if (a.tokens == 0) return ok();
    int dev = -1;
    if ((st = train_device(&dev)) != TROP_OK) return st;
    SpanChecker checker(dev);
    if ((st = check_inputs(a, checker)) != TROP_OK) return st;
    if ((st = checker.span(loss, a.tokens, 4, "loss")) != TROP_OK) return st;
    if ((st = checker.span(lse, a.tokens, 4, "lse")) != TROP_OK) return st;
    CePlan c;
    if (!plan(a.dt, a.tokens, a.width, a.vocab, false, !direct_w(a.dt, a.w, a.ldw, a.width), &c))
        return fail(TROP_ERR_UNSUPPORTED, "workspace size overflows");
    char* ws = nullptr;
    if ((st = check_workspace(a, c, checker, &ws)) != TROP_OK) return st;
    TropCeParams p = params(a, c, ws);
    p.loss = loss;
    p.lse = lse;
    const hipStream_t s = static_cast<hipStream_t>(a.stream);
    if (c.few) {
        const int64_t most = max_groups(256);
        for (; st == TROP_OK && p.tile0 < c.tiles; p.tile0 += most) {
            p.v0 = p.tile0 * 16 * c.few_rows;
            st = train_launch(dev, few_kernel(TK_CE_FEW, 6, c, a.dt), TROP_T_CE_LOGITS, std::min(c.tiles - p.tile0, most),
                              256, &p, s);
        }
    } else {
        st = list_tokens(dev, c, p, s);
        for (int64_t v0 = 0; st == TROP_OK && v0 < a.vocab; v0 += c.piece) {
            st = prepare_piece(dev, a, c, v0, p, s);
            const int64_t edge = tile_edge(c.logits_tile);
            if (st == TROP_OK)
                st = train_launch(dev, logits_kernel(TK_CE_STATS, TK_CE_STATS_RAW, c, a.dt), TROP_T_CE_LOGITS,
                                  p.piece / edge * ceil_div(a.tokens, edge), tile_threads(c.logits_tile), &p, s);
        }
    }
    if (st == TROP_OK) st = train_launch(dev, TK_CE_MERGE, TROP_T_CE_MERGE, a.tokens, 256, &p, s);
    return st == TROP_OK ? ok() : st;
}

trop_status ce_backward(const CeCall& a, const float* lse, const float* grad_loss, int64_t grad_loss_stride,
                        void* grad_x, int64_t ldgx, void* grad_w, int64_t ldgw) {
    trop_status st = check_sizes(a.dt, a.tokens, a.width, a.vocab);
    if (st != TROP_OK) return st;
    if (a.target_bytes != 4 && a.target_bytes != 8)
        return fail(TROP_ERR_INVALID_ARGUMENT, "targets have 4 or 8 bytes");
    if (grad_loss_stride < 0) return fail(TROP_ERR_INVALID_ARGUMENT, "negative stride for grad_loss");
    if (a.tokens == 0) grad_x = nullptr;
    if (a.width == 0 || a.vocab == 0 || (!grad_x && !grad_w)) return ok();
    int dev = -1;
    if ((st = train_device(&dev)) != TROP_OK) return st;
    const size_t eb = elem_size(a.dt);
    SpanChecker checker(dev);
    if ((st = check_inputs(a, checker)) != TROP_OK) return st;
    if (a.tokens > 0) {
        if ((st = checker.span(lse, a.tokens, 4, "lse")) != TROP_OK) return st;
        // one element every grad_loss_stride
        int64_t reach = 0;
        if (__builtin_mul_overflow(a.tokens - 1, grad_loss_stride, &reach))
            return fail(TROP_ERR_INVALID_ARGUMENT, "grad_loss extent overflows");
        if ((st = checker.span(grad_loss, reach + 1, 4, "grad_loss")) != TROP_OK) return st;
    }
    if (grad_x && (st = checker.matrix(grad_x, a.tokens, a.width, ldgx, eb, "grad_x")) != TROP_OK) return st;
    if (grad_w && (st = checker.matrix(grad_w, a.vocab, a.width, ldgw, eb, "grad_w")) != TROP_OK) return st;
    CePlan c;
    if (!plan(a.dt, a.tokens, a.width, a.vocab, true, !direct_w(a.dt, a.w, a.ldw, a.width), &c))
        return fail(TROP_ERR_UNSUPPORTED, "workspace size overflows");
    char* ws = nullptr;
    if ((st = check_workspace(a, c, checker, &ws)) != TROP_OK) return st;
    TropCeParams p = params(a, c, ws);
    p.backward = 1;
    p.lse_in = lse;
    p.grad_loss = grad_loss;
    p.grad_loss_stride = grad_loss_stride;
    p.grad_x = grad_x;
    p.grad_w = grad_w;
    p.ldgx = ldgx;
    p.ldgw = ldgw;
    const hipStream_t s = static_cast<hipStream_t>(a.stream);
    st = c.few ? few_pieces(dev, a, c, p, s) : tile_pieces(dev, a, c, p, s);
    if (grad_x) {
        const int64_t blocks = ceil_div(a.width, 1024), most = max_groups(256) / blocks;
        for (; st == TROP_OK && p.row0 < a.tokens; p.row0 += most)
            st = train_launch(dev, typed(TK_CE_FINISH, a.dt), TROP_T_CE_MERGE, std::min(a.tokens - p.row0, most) * blocks,
                              256, &p, s);
    }
    return st == TROP_OK ? ok() : st;
}

}  // namespace
}  // namespace trop

extern "C" trop_status tropical_linear_cross_entropy_forward(trop_dtype dtype, const void* x, int64_t ldx,
                                                             const void* w, int64_t ldw, const void* target,
                                                             int target_bytes, int64_t ignore_index, float* loss,
                                                             float* lse, int64_t tokens, int64_t width, int64_t vocab,
                                                             void* workspace, size_t workspace_bytes, void* stream) {
    return trop::guarded("tropical_linear_cross_entropy_forward", [&] {
        return trop::ce_forward({dtype, x, w, target, ldx, ldw, target_bytes, ignore_index, tokens, width, vocab,
                                 workspace, workspace_bytes, stream},
                                loss, lse);
    });
}

extern "C" trop_status tropical_linear_cross_entropy_workspace_size(trop_dtype dtype, int64_t tokens, int64_t width,
                                                                    int64_t vocab, int backward, size_t* bytes) {
    using namespace trop;
    return guarded("tropical_linear_cross_entropy_workspace_size", [&]() -> trop_status {
        if (!bytes) return fail(TROP_ERR_INVALID_ARGUMENT, "bytes is NULL");
        *bytes = 0;
        const trop_status st = check_sizes(dtype, tokens, width, vocab);
        if (st != TROP_OK) return st;
        if (width == 0 || vocab == 0 || (tokens == 0 && !backward)) return ok();
        for (const bool packed : {true, false}) {
            CePlan c;
            if (!plan(dtype, tokens, width, vocab, backward != 0, packed, &c))
                return fail(TROP_ERR_UNSUPPORTED, "workspace size overflows");
            if (c.bytes > *bytes) *bytes = c.bytes;
        }
        return ok();
    });
}

extern "C" trop_status tropical_linear_cross_entropy_backward(
    trop_dtype dtype, const void* x, int64_t ldx, const void* w, int64_t ldw, const void* target, int target_bytes,
    int64_t ignore_index, const float* lse, const float* grad_loss, int64_t grad_loss_stride, void* grad_x,
    int64_t ldgx, void* grad_w, int64_t ldgw, int64_t tokens, int64_t width, int64_t vocab, void* workspace,
    size_t workspace_bytes, void* stream) {
    return trop::guarded("tropical_linear_cross_entropy_backward", [&] {
        return trop::ce_backward({dtype, x, w, target, ldx, ldw, target_bytes, ignore_index, tokens, width, vocab,
                                  workspace, workspace_bytes, stream},
                                 lse, grad_loss, grad_loss_stride, grad_x, ldgx, grad_w, ldgw);
    });
}
