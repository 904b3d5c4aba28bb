// C ABI of the operators around the losses (declared in
// include/rl_post_loss.h): the vocabulary cross
// entropy, layer norm, RMS norm, the AdamW step and the gradients' norm.
//
// As in abi.cpp, arguments are validated on the host before any HIP call,
// nothing is allocated and nothing synchronises; kernels go to the caller's
// stream.
#include "train_abi.h"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <new>
#include <numeric>

#include "adamw_kernels.h"
#include "ce_kernels.h"
#include "grad_kernels.h"
#include "norm_kernels.h"
#include "rms_kernels.h"

namespace {

using namespace rlpl;

constexpr int64_t kMaxRows = int64_t(1) << 31;

// Whether device dev is set up for the kernels.
bool set_up(int dev) {
    if (!is_gfx950(dev)) return false;
    // the contractions take their LDS ring beyond the default limit
    for (int dt : {RLPL_F16, RLPL_BF16})
        for (bool small : {false, true})
            for (const void* k :
                 {pick_ce_gemm(dt, small, kCeLogits), pick_ce_gemm(dt, small, kCeDlogits), pick_ce_grads(dt, small)})
                if (hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize,
                                        small ? kCeSmall.lds : kCeLarge.lds) != hipSuccess)
                    return false;
    for (int dt : {RLPL_F16, RLPL_BF16})
        if (hipFuncSetAttribute(pick_ce_deep_logits(dt), hipFuncAttributeMaxDynamicSharedMemorySize, kCeDeepLds) != hipSuccess)
            return false;
    return true;
}

Devices<set_up> g_devices;
int device() { return g_devices.current(); }

// ----------------------------------------------------------------------------- vocabulary cross entropy

constexpr int64_t kCeMaxVocab = int64_t(1) << 22;     // a 256-row panel is addressed with 32-bit offsets
constexpr int64_t kCeMaxHidden = 65536;
// Tiles of one product (x 512 lanes < 2^31).  The launch of both gradient products has the hidden product's and the
// weight's, vocabulary by hidden tiles, which with at most 2^14 and 2^8 of those reach 2^22 only where the rows are
// fewer than 2^8 tiles: the two together stay below 2^23.
constexpr int64_t kCeMaxTiles = int64_t(1) << 22;
// A piece of the vocabulary: kCePieceElements of dz (256 MiB), at least kCePieceCols columns, so that
// adding a piece's hidden gradient to the float32 planes stays small beside its product.  Where that least number
// does not make it larger, the loss's pass leaves the logits of the first columns, as many as a piece of all rows has
// (512 MiB), and their dz is a pass over them (1024 x 4096 x 128256 bf16: 150 us, where forming them again took 957;
// 3.64 -> 2.92 ms for the call; 16 rows: 868 -> 735 us).  Where rows do not count, more columns fit (6001 x 2048 x
// 50021, half of the rows: 135 us less).
constexpr int64_t kCePieceElements = int64_t(1) << 27;
constexpr int64_t kCePieceCols = 8192;

// The time of a launch's tiles in microseconds, to choose between their shapes: a tile of `steps` K steps takes
// fixed + step * steps alone, and a chip full of them fill + pace * steps each on one of its 256 compute units
// (fitted to both shapes' times at 19 sizes between 128 x 512 x 32000 and 3000 x 1024 x 6000; 128 x 512 x 32000 takes
// 59 us with the small shape and 107 with the large one, 2048 x 2048 x 8192 logits 122 and 76).
struct CePace {
    double fixed, step, fill, pace;
};
constexpr CePace kPaceLarge{13.0, 1.1, 13.0, 1.1}, kPaceSmall{5.0, 0.35, 1.0, 0.17};
double ce_time(const CePace& p, double tiles, double tile_steps, double longest) {
    const double one = p.fixed + p.step * longest, all = (p.fill * tiles + p.pace * tile_steps) / 256.0;
    return all > one ? all + 0.5 * one : one + 0.2 * all;
}
double ce_logits_time(const CeShape& s, const CePace& p, int64_t n, int64_t h, int64_t vocab) {
    const double tiles = double(div_up(n, s.tile)) * double(div_up(vocab, s.tile)), steps = double(div_up(h, kGemmBK));
    return ce_time(p, tiles, tiles * steps, steps);
}
double ce_grads_time(const CeShape& s, const CePace& p, int64_t n, int64_t h, int64_t vocab) {
    const double tiles_h = double(div_up(h, s.tile)), tiles_r = double(div_up(n, s.tile)), tiles_v = double(div_up(vocab, s.tile));
    const double steps_v = double(div_up(vocab, kGemmBK)), steps_r = double(div_up(n, kGemmBK));
    double splits = s.at_once / (tiles_r * tiles_h);         // of the hidden product
    if (splits > kCeMaxSplits) splits = kCeMaxSplits;
    if (splits < 1.0) splits = 1.0;
    const double longest = steps_v / splits > steps_r ? steps_v / splits : steps_r;
    return ce_time(p, tiles_h * (tiles_v + tiles_r * splits), tiles_h * (tiles_r * steps_v + tiles_v * steps_r), longest);
}

bool ce_shape_ok(int64_t n, int64_t h, int64_t vocab) {
    const int64_t tile = kCeLarge.tile;
    return n >= 1 && n <= kCeMaxRows && h >= 8 && h <= kCeMaxHidden && h % 8 == 0 && vocab >= 1 && vocab < kCeMaxVocab &&
           div_up(n, tile) * div_up(vocab, tile) < kCeMaxTiles &&
           div_up(n, tile) * div_up(h, tile) < kCeMaxTiles;
}

// Workspace of a call, sized for every row: what the compaction leaves and the kept hidden states, then
// the loss's tile partials, whose place the gradient's dz, planes and column sums take afterwards.
struct CeLayout {
    bool small_z, small_g;             // the shapes of the logits' products and of the gradients'
    CeShape z, g;
    int64_t piece, tiles_m, tiles_n, splits, plane_rows;   // tiles of the logits
    bool keep;                         // the first piece's logits
    size_t row, place, target, lse, row_loss, target_logit, hidden, kept, part, dz, planes, cols, total;   // offsets
};
CeLayout ce_layout(int64_t n, int64_t h, int64_t vocab, bool grads) {
    CeLayout L{};
    size_t at = 256;   // CeState
    const auto take = [&at](size_t bytes) {
        const size_t o = at;
        at += up256(bytes);
        return o;
    };
    const int64_t large = kCeLarge.tile;
    L.small_z = ce_logits_time(kCeSmall, kPaceSmall, n, h, vocab) < ce_logits_time(kCeLarge, kPaceLarge, n, h, vocab) &&
                div_up(n, kCeSmall.tile) * div_up(vocab, kCeSmall.tile) < kCeMaxTiles;
    L.small_g = ce_grads_time(kCeSmall, kPaceSmall, n, h, vocab) < ce_grads_time(kCeLarge, kPaceLarge, n, h, vocab) &&
                div_up(vocab > n ? vocab : n, kCeSmall.tile) * div_up(h, kCeSmall.tile) < kCeMaxTiles;
    L.z = L.small_z ? kCeSmall : kCeLarge;
    L.g = L.small_g ? kCeSmall : kCeLarge;
    L.tiles_m = div_up(n, L.z.tile);
    L.tiles_n = div_up(vocab, L.z.tile);
    for (size_t* p : {&L.row, &L.place, &L.target, &L.lse, &L.row_loss, &L.target_logit}) *p = take(size_t(n) * 4);
    L.hidden = take(size_t(n) * size_t(h) * 2);
    if (grads) {
        const int64_t rows16 = div_up(n, 16) * 16;
        int64_t piece = kCePieceElements / rows16 / large * large;
        if (piece < kCePieceCols) piece = kCePieceCols;
        // whole rounds of 256 tiles where a piece has several (6001 x 2048 x 50021 with half of the rows ignored: ten
        // rounds of logits instead of twelve)
        const int64_t row_tiles = div_up(n, large), rounds = piece / large * row_tiles / 256;
        if (rounds > 0) piece = rounds * 256 / row_tiles * large;
        const int64_t all = div_up(vocab, large) * large;
        L.piece = piece < all ? piece : all;
        L.keep = rows16 * L.piece <= kCePieceElements;
        L.kept = take(L.keep ? size_t(rows16) * size_t(L.piece) * sizeof(float) : 0);
    }
    L.part = at;
    const size_t after_loss = at + up256(size_t(n) * size_t(L.tiles_n) * 8);
    if (grads) {
        // planes for up to kCeMaxSplits splits of K, and no more than twice the workgroups that run at once
        const int64_t tiles_h = div_up(h, L.g.tile), tiles_r = div_up(n, L.g.tile), most = L.piece / large * 2;
        L.splits = most < kCeMaxSplits ? most : kCeMaxSplits;
        L.plane_rows = div_up(2 * L.g.at_once, tiles_h);
        if (L.plane_rows > tiles_r * L.splits) L.plane_rows = tiles_r * L.splits;
        if (L.plane_rows < tiles_r) L.plane_rows = tiles_r;
        const int64_t rows = L.plane_rows * L.g.tile < n * L.splits ? L.plane_rows * L.g.tile : n * L.splits;
        L.dz = take(size_t(n) * size_t(L.piece) * 2);
        L.planes = take(size_t(rows < n ? n : rows) * size_t(h) * sizeof(float));
        L.cols = take(size_t(L.tiles_m) * size_t(vocab) * sizeof(float));
    }
    L.total = at > after_loss ? at : after_loss;
    return L;
}

unsigned capped(int64_t grid, int64_t cap) { return unsigned(grid < cap ? grid : cap); }

struct CeCall {
    const void *hidden, *weight, *bias;
    const int64_t* targets;
    int64_t n, h, vocab;
    int dtype;
    int64_t ignore_index;
    float z_loss;
    int reduction;
    float* loss;
    void *grad_hidden, *grad_weight, *grad_bias;
    int weight_grad_dtype, accumulate;
    void* workspace;
    size_t workspace_bytes;
    uint32_t flags = 0;
};

int ce_check(const CeCall& c, bool grads) {
    if (!c.hidden || !c.weight || !c.targets || !c.loss) return RLPL_ERR_NULL;
    if (!ce_shape_ok(c.n, c.h, c.vocab)) return RLPL_ERR_SHAPE;
    if (c.dtype != RLPL_F16 && c.dtype != RLPL_BF16) return RLPL_ERR_DTYPE;
    if (grads && c.weight_grad_dtype != RLPL_F32 && c.weight_grad_dtype != c.dtype) return RLPL_ERR_DTYPE;
    if (!std::isfinite(c.z_loss) || c.z_loss < 0.0f || c.z_loss > 1.0f) return RLPL_ERR_PARAM;
    if (c.reduction != RLPL_REDUCE_MEAN && c.reduction != RLPL_REDUCE_SUM) return RLPL_ERR_PARAM;
    if (c.flags & ~uint32_t(RLPL_CE_HIDDEN_F32)) return RLPL_ERR_PARAM;
    if (grads && c.accumulate && c.weight_grad_dtype != RLPL_F32) return RLPL_ERR_PARAM;
    const size_t we = grads ? dtype_bytes(c.weight_grad_dtype) : 1;
    if (!is_aligned(c.hidden, 16) || !is_aligned(c.weight, 16) || !is_aligned(c.bias, 2) || !is_aligned(c.targets, 8) ||
        !is_aligned(c.loss, 4) || !is_aligned(c.grad_hidden, 16) || !is_aligned(c.grad_weight, 16) ||
        !is_aligned(c.grad_bias, we))
        return RLPL_ERR_ALIGN;
    if (!c.workspace || c.workspace_bytes < ce_layout(c.n, c.h, c.vocab, grads).total) return RLPL_ERR_WORKSPACE;
    return is_aligned(c.workspace, 256) ? RLPL_OK : RLPL_ERR_ALIGN;
}

int ce_run(const CeCall& c, bool grads, hipStream_t stream) {
    int st = ce_check(c, grads);
    if (st != RLPL_OK) return st;
    if ((st = device()) != RLPL_OK) return st;
    const CeLayout L = ce_layout(c.n, c.h, c.vocab, grads);
    char* ws = static_cast<char*>(c.workspace);
    auto* state = reinterpret_cast<CeState*>(ws);
    const auto ints = [ws](size_t at) { return reinterpret_cast<int32_t*>(ws + at); };
    const auto floats = [ws](size_t at) { return reinterpret_cast<float*>(ws + at); };

    const CePrepareArgs prepare{c.targets,      c.ignore_index, c.vocab,  int32_t(c.n),    ints(L.row),
                                ints(L.place),  ints(L.target), state,    c.hidden,        ws + L.hidden,
                                int32_t(c.h)};
    if (c.n <= kCePrepareRows) {
        st = enqueue(ce_prepare_kernel(), prepare, dim3(unsigned(c.n)), kCeThreads, stream);
    } else {
        st = enqueue(ce_compact_kernel(), prepare, dim3(1), kCeCompactThreads, stream);
        if (st == RLPL_OK) st = enqueue(ce_gather_kernel(), prepare, dim3(capped(c.n, 1 << 16)), kCeThreads, stream);
    }
    if (st != RLPL_OK) return st;

    CeGemmArgs z{};                    // logits of the whole vocabulary, then of its pieces
    z.a = ws + L.hidden;
    z.b = c.weight;
    z.lda = z.ldb = c.h;
    z.M = int32_t(c.n);
    z.N = int32_t(c.vocab);
    z.K = int32_t(c.h);
    z.tiles_m = uint32_t(L.tiles_m);
    z.tiles_n = uint32_t(L.tiles_n);
    z.state = state;
    z.bias = c.bias;
    z.target = ints(L.target);
    z.part = floats(L.part);
    z.target_logit = floats(L.target_logit);
    z.dz_scale = ce_dz_scale(c.dtype, c.z_loss);
    const auto product = [&](const void* kernel, const CeShape& shape, const auto& args, uint32_t blocks) {
        return enqueue(kernel, args, dim3(blocks), shape.threads, stream, size_t(shape.lds));
    };
    const bool any = grads && (c.grad_hidden || c.grad_weight || c.grad_bias);
    if (any && L.keep) {
        z.kept = floats(L.kept);
        z.kept_room = uint32_t(div_up(c.n, 16) * (L.piece / 256));
    }
    const uint32_t tiles_z = z.tiles_m * z.tiles_n;
    st = L.small_z && tiles_z <= kCeDeepTiles
             ? enqueue(pick_ce_deep_logits(c.dtype), z, dim3(tiles_z), L.z.threads, stream, size_t(kCeDeepLds))
             : product(pick_ce_gemm(c.dtype, L.small_z, kCeLogits), L.z, z, tiles_z);
    if (st != RLPL_OK) return st;
    const uint32_t tiles_h = uint32_t(div_up(c.h, L.g.tile));
    const CeRowArgs rows{floats(L.part), floats(L.target_logit), ints(L.target), state, floats(L.lse), floats(L.row_loss),
                         c.loss, c.z_loss, 1.0f / z.dz_scale, int32_t(L.tiles_n),
                         c.reduction == RLPL_REDUCE_MEAN ? 1 : 0, int32_t(L.piece), grads ? int32_t(L.splits) : 1,
                         uint32_t(L.plane_rows), tiles_h,
                         c.grad_weight ? uint32_t(div_up(L.piece < c.vocab ? L.piece : c.vocab, L.g.tile)) * tiles_h : 0,
                         L.small_g ? 1 : 0};
    if ((st = enqueue(ce_row_kernel(), rows, dim3(capped(div_up(c.n, kCeThreads / 64), kCeRowGrid)), kCeThreads, stream)) != RLPL_OK) return st;
    if (!any) return RLPL_OK;

    const size_t we = dtype_bytes(c.weight_grad_dtype);
    const int f32 = c.weight_grad_dtype == RLPL_F32 ? 1 : 0;
    const uint32_t tiles_r = uint32_t(div_up(c.n, L.g.tile));
    for (int64_t v0 = 0; v0 < c.vocab; v0 += L.piece) {
        const int64_t cols = c.vocab - v0 < L.piece ? c.vocab - v0 : L.piece;
        const char* weight = static_cast<const char*>(c.weight) + size_t(v0) * size_t(c.h) * 2;
        z.b = weight;
        z.N = int32_t(cols);
        z.tiles_n = uint32_t(div_up(cols, L.z.tile));
        z.bias = c.bias ? static_cast<const char*>(c.bias) + size_t(v0) * 2 : nullptr;
        z.first = int32_t(v0);
        z.lse = floats(L.lse);
        z.z_loss2 = 2.0f * c.z_loss;
        z.c = ws + L.dz;
        z.ldc = L.piece;
        z.col_part = c.grad_bias ? floats(L.cols) + v0 : nullptr;
        z.col_ld = c.vocab;
        const uint32_t tiles = z.tiles_m * z.tiles_n;
        // Kept logits reach beyond the first piece where rows do not count: both kernels pass over the other's tiles.
        if (L.keep) st = enqueue(pick_ce_dz(c.dtype, L.small_z), z, dim3(tiles), L.z.threads, stream);
        if (st == RLPL_OK && (v0 > 0 || !L.keep)) st = product(pick_ce_gemm(c.dtype, L.small_z, kCeDlogits), L.z, z, tiles);
        if (st != RLPL_OK) return st;
        CeGradArgs g{};
        CeGemmArgs& hg = g.hidden;
        hg.a = ws + L.dz;
        hg.b = weight;
        hg.lda = L.piece;
        hg.ldb = hg.ldc = c.h;
        hg.M = int32_t(c.n);
        hg.N = int32_t(c.h);
        hg.K = int32_t(cols);
        hg.split_k = int32_t(L.piece);
        hg.tiles_m = tiles_r;
        hg.tiles_n = tiles_h;
        hg.state = state;
        hg.c = ws + L.planes;
        hg.accumulate = v0 > 0 ? 1 : 0;
        if (c.grad_hidden) g.hidden_blocks = uint32_t(div_up(L.plane_rows * tiles_h, 8) * 8);
        CeGemmArgs& wg = g.weight;
        wg.a = ws + L.dz;
        wg.b = ws + L.hidden;
        wg.lda = L.piece;
        wg.ldb = wg.ldc = c.h;
        wg.M = int32_t(cols);
        wg.N = int32_t(c.h);
        wg.K = int32_t(c.n);
        wg.tiles_m = uint32_t(div_up(cols, L.g.tile));
        wg.tiles_n = tiles_h;
        wg.state = state;
        if (c.grad_weight) wg.c = static_cast<char*>(c.grad_weight) + size_t(v0) * size_t(c.h) * we;
        wg.out_f32 = f32;
        wg.accumulate = c.accumulate ? 1 : 0;
        const uint32_t blocks = g.hidden_blocks + (c.grad_weight ? wg.tiles_m * tiles_h : 0);
        if (blocks > 0 && (st = product(pick_ce_grads(c.dtype, L.small_g), L.g, g, blocks)) != RLPL_OK) return st;
    }
    const CeFinishArgs f{floats(L.planes), ints(L.place), state, c.grad_hidden, int32_t(c.n), int32_t(c.h),
                         c.grad_hidden ? capped(c.n, 1 << 16) : 0, c.flags & RLPL_CE_HIDDEN_F32 ? 1 : 0, floats(L.cols),
                         c.grad_bias, int32_t(c.vocab), f32, c.accumulate ? 1 : 0, L.z.tile};
    const unsigned bias_blocks = c.grad_bias ? unsigned(div_up(c.vocab, kCeThreads)) : 0;
    if (f.row_blocks + bias_blocks == 0) return RLPL_OK;
    return enqueue(pick_ce_finish(c.dtype), f, dim3(f.row_blocks + bias_blocks), kCeThreads, stream);
}

// ----------------------------------------------------------------------------- layer norm

bool norm_types_ok(int dtype, int wdtype) {
    return known_dtype(dtype) && known_dtype(wdtype) && (wdtype == dtype || wdtype == RLPL_F32);
}

bool norm_shape_ok(int64_t rows, int64_t cols) {
    return rows >= 1 && rows < kMaxRows && cols >= 1 && cols <= kNormMaxCols;
}

// Slabs of rows of the backward pass of long rows: about 2048 workgroups, at least 16 rows each (four a wavefront).
int64_t norm_slabs(int64_t rows, int64_t col_tiles) {
    int64_t slabs = 2048 / col_tiles;
    const int64_t most = div_up(rows, 16);
    if (slabs > most) slabs = most;
    if (slabs < 1) slabs = 1;
    const int64_t slab_rows = div_up(rows, slabs);
    return div_up(rows, slab_rows);
}

unsigned row_grid(int64_t rows, int per_group) {
    const int64_t g = div_up(rows, per_group);
    return unsigned(g < kNormMaxGrid ? g : kNormMaxGrid);
}

// Workgroups of the backward kernel that holds rows: four rows at least for each row a workgroup has at a time, so
// that a row's loads overlap another's sums and the partials stay few (of a short batch fewer, up to kNormHeldFew
// workgroups: 100 x 768 bf16 8.4 -> 6.6 us, 17 x 8192 17.5 -> 13.4), and more of them the shorter a row is
// (shorter rows take fewer registers).
int64_t norm_held_grid(int64_t rows, int64_t cols, int rows_per_group) {
    const int64_t each = div_up(rows, rows_per_group), few = each < kNormHeldFew ? each : kNormHeldFew;
    int64_t g = div_up(rows, 4 * rows_per_group);
    if (g < few) g = few;
    int64_t most = kNormHeldElements / cols;
    if (most > kNormHeldGrid) most = kNormHeldGrid;
    if (most < kNormHeldLeast) most = kNormHeldLeast;
    return g < most ? g : most;
}

struct NormLayout {
    size_t sums, part, total;
};
NormLayout norm_layout(int64_t rows, int64_t cols) {
    NormLayout L{};
    int64_t parts;
    if (cols <= kNormHeldCols) {
        parts = norm_held_grid(rows, cols, 1);                    // the most a kernel's shape asks for
    } else {
        L.sums = up256(size_t(rows) * sizeof(float2));
        parts = norm_slabs(rows, div_up(cols, norm_col_tile(RLPL_F16)));   // so does the widest column tile
    }
    L.part = up256(size_t(parts) * 2 * size_t(cols) * sizeof(float));
    L.total = L.sums + L.part;
    return L;
}

// ----------------------------------------------------------------------------- RMS norm

bool rms_shape_ok(int64_t rows, int64_t cols) {
    return rows >= 1 && rows < kMaxRows && cols >= 1 && cols <= kRmsMaxCols;
}

// Room for one plane of column sums of each workgroup (and of a second one, as the joining kernel counts them).
size_t rms_bytes(int64_t rows, int64_t cols) {
    return up256(size_t(norm_held_grid(rows, cols, 1)) * 2 * size_t(cols) * sizeof(float));
}

struct RmsCall {
    const void *x, *weight, *residual;
    int64_t rows, cols;
    int dtype, weight_dtype, stream_dtype;
    float eps;
    void* y;
    float* scale;
    float* rstd;
    void* stream_out;
};

int rms_forward(const RmsCall& c, bool fp8, hipStream_t stream) {
    if (!c.x || !c.y || (fp8 && !c.scale) || (c.residual && !c.stream_out)) return RLPL_ERR_NULL;
    if (!rms_shape_ok(c.rows, c.cols)) return RLPL_ERR_SHAPE;
    if (!norm_types_ok(c.dtype, c.weight_dtype) || !norm_types_ok(c.dtype, c.stream_dtype)) return RLPL_ERR_DTYPE;
    if (!std::isfinite(c.eps) || c.eps < 0.0f) return RLPL_ERR_PARAM;
    const size_t e = dtype_bytes(c.dtype), re = dtype_bytes(c.stream_dtype);
    if (!is_aligned(c.x, e) || !is_aligned(c.y, fp8 ? 1 : e) || !is_aligned(c.weight, dtype_bytes(c.weight_dtype)) ||
        !is_aligned(c.residual, re) || !is_aligned(c.stream_out, re) || !is_aligned(c.rstd, 4) || !is_aligned(c.scale, 4))
        return RLPL_ERR_ALIGN;
    const int st = device();
    if (st != RLPL_OK) return st;
    const NormRowKernel k = pick_rms_fwd(c.dtype, c.residual ? c.stream_dtype : c.dtype, fp8, c.cols);
    if (!k.kernel) return RLPL_ERR_DTYPE;
    const RmsFwdArgs a{c.x, c.residual, c.weight, c.residual ? c.stream_out : nullptr, c.y, c.scale, c.rstd, c.rows,
                       int32_t(c.cols), int32_t(div_up(c.cols, kFp8Group)), c.weight_dtype == RLPL_F32 ? 1 : 0, c.eps};
    return enqueue(k.kernel, a, dim3(row_grid(c.rows, k.rows_per_group)), k.threads, stream);
}

// ----------------------------------------------------------------------------- gradients' norm

constexpr int64_t kGradMaxTensors = int64_t(1) << 24;
constexpr int64_t kGradMaxElements = int64_t(1) << 40;
constexpr int64_t kGradMaxChunks = int64_t(1) << 31;        // of a launch

int grad_check(void* const* grads, const int64_t* sizes, const int32_t* dtypes, int64_t count) {
    if (!grads || !sizes || !dtypes) return RLPL_ERR_NULL;
    if (count < 1 || count > kGradMaxTensors) return RLPL_ERR_SHAPE;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] < 0 || sizes[i] > kGradMaxElements) return RLPL_ERR_SHAPE;
        if (!known_dtype(dtypes[i])) return RLPL_ERR_DTYPE;
        if (sizes[i] == 0) continue;
        if (!grads[i]) return RLPL_ERR_NULL;
        if (!is_aligned(grads[i], dtype_bytes(dtypes[i]))) return RLPL_ERR_ALIGN;
    }
    return RLPL_OK;
}

// Windows of the list that fit a launch's arguments: calls f(chunks) with each in `list`, until one fails.
template <typename F>
int grad_windows(GradList& list, void* const* grads, const int64_t* sizes, const int32_t* dtypes, int64_t count, F f) {
    list.count = 0;
    int64_t chunks = 0;
    const auto close = [&]() {
        list.first[list.count] = uint32_t(chunks);
        const int st = list.count ? f(chunks) : int(RLPL_OK);
        list.count = 0;
        chunks = 0;
        return st;
    };
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] == 0) continue;
        const int64_t here = div_up(sizes[i], kGradChunk);
        if (list.count == kGradWindow || chunks + here >= kGradMaxChunks) {
            const int st = close();
            if (st != RLPL_OK) return st;
        }
        list.p[list.count] = grads[i];
        list.n[list.count] = sizes[i] * 4 + dtypes[i];
        list.first[list.count++] = uint32_t(chunks);
        chunks += here;
    }
    return close();
}

// The launches that grad_windows makes of a list, or -1 where its sizes cannot be taken.
int64_t grad_launches(const int64_t* sizes, int64_t count) {
    if (!sizes || count < 1 || count > kGradMaxTensors) return -1;
    int64_t launches = 0, tensors = 0, chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] < 0 || sizes[i] > kGradMaxElements) return -1;
        if (sizes[i] == 0) continue;
        const int64_t here = div_up(sizes[i], kGradChunk);
        if (tensors == kGradWindow || chunks + here >= kGradMaxChunks) {
            ++launches;
            tensors = chunks = 0;
        }
        ++tensors;
        chunks += here;
    }
    return launches + (tensors > 0);
}
size_t grad_bytes(int64_t launches) { return up256(size_t(launches > 0 ? launches : 1) * kGradGrid * sizeof(double)); }

// Whether two of the tensors share memory; false too where there is no host memory to find out.
bool grads_apart(void* const* grads, const int64_t* sizes, const int32_t* dtypes, int64_t count) {
    const auto begin = [&](int64_t i) { return reinterpret_cast<uintptr_t>(grads[i]); };
    const auto end = [&](int64_t i) { return begin(i) + uintptr_t(sizes[i]) * dtype_bytes(dtypes[i]); };
    const auto ordered = [&](auto at) {
        int64_t before = -1;
        for (int64_t k = 0; k < count; ++k) {
            const int64_t i = at(k);
            if (sizes[i] == 0) continue;
            if (before >= 0 && begin(i) < end(before)) return false;
            before = i;
        }
        return true;
    };
    if (ordered([](int64_t k) { return k; })) return true;
    const std::unique_ptr<int64_t[]> order(new (std::nothrow) int64_t[size_t(count)]);
    if (!order) return false;
    std::iota(order.get(), order.get() + count, int64_t(0));
    std::sort(order.get(), order.get() + count, [&](int64_t a, int64_t b) { return begin(a) < begin(b); });
    return ordered([&](int64_t k) { return order[size_t(k)]; });
}

unsigned grad_grid(int64_t chunks) { return unsigned(chunks < kGradGrid ? chunks : kGradGrid); }

// ----------------------------------------------------------------------------- AdamW

constexpr int64_t kAdamMaxTensors = int64_t(1) << 24;
constexpr int64_t kAdamMaxElements = int64_t(1) << 40;      // of one tensor
constexpr int64_t kAdamMaxChunks = int64_t(1) << 31;
constexpr int64_t kAdamLaunchChunks = int64_t(1) << 23;     // workgroups of one launch (x 256 lanes < 2^32)

// Chunks of a list of tensors, or -1 where its sizes cannot be taken.
int64_t adam_chunks(const int64_t* sizes, int64_t count) {
    if (!sizes || count < 1 || count > kAdamMaxTensors) return -1;
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] < 0 || sizes[i] > kAdamMaxElements) return -1;
        chunks += div_up(sizes[i], kAdamChunk);
        if (chunks >= kAdamMaxChunks) return -1;
    }
    return chunks;
}

size_t adam_bytes(int64_t count, int64_t chunks) {
    return sizeof(AdamPlan) + size_t(count) * sizeof(AdamTensor) + size_t(chunks) * sizeof(AdamChunk);
}

// The murmur3 finalizer, as the kernels' mix32.
uint32_t mix(uint32_t h) {
    h ^= h >> 16;
    h *= 0x85ebca6bu;
    h ^= h >> 13;
    h *= 0xc2b2ae35u;
    return h ^ (h >> 16);
}

}  // namespace

extern "C" {

size_t linear_cross_entropy_workspace_bytes(int64_t n, int64_t hidden_size, int64_t vocab, int gradients) {
    return ce_shape_ok(n, hidden_size, vocab) ? ce_layout(n, hidden_size, vocab, gradients != 0).total : 0;
}

int linear_cross_entropy_fwd(const void* hidden, const void* weight, const void* bias, const int64_t* targets, int64_t n,
                             int64_t hidden_size, int64_t vocab, int dtype, int64_t ignore_index, float z_loss,
                             int reduction, float* loss_out, void* workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    const CeCall c{hidden, weight, bias, targets, n, hidden_size, vocab, dtype, ignore_index, z_loss, reduction, loss_out,
                   nullptr, nullptr, nullptr, RLPL_F32, 0, workspace, workspace_bytes};
    return ce_run(c, false, stream);
}

int linear_cross_entropy(const void* hidden, const void* weight, const void* bias, const int64_t* targets, int64_t n,
                         int64_t hidden_size, int64_t vocab, int dtype, int64_t ignore_index, float z_loss, int reduction,
                         float* loss_out, void* grad_hidden, void* grad_weight, void* grad_bias, int weight_grad_dtype,
                         int accumulate, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    return rlpl_linear_cross_entropy(0, hidden, weight, bias, targets, n, hidden_size, vocab, dtype, ignore_index, z_loss,
                                     reduction, loss_out, grad_hidden, grad_weight, grad_bias, weight_grad_dtype,
                                     accumulate, workspace, workspace_bytes, stream);
}

int rlpl_linear_cross_entropy(uint32_t flags, const void* hidden, const void* weight, const void* bias,
                              const int64_t* targets, int64_t n, int64_t hidden_size, int64_t vocab, int dtype,
                              int64_t ignore_index, float z_loss, int reduction, float* loss_out, void* grad_hidden,
                              void* grad_weight, void* grad_bias, int weight_grad_dtype, int accumulate, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
    const CeCall c{hidden, weight, bias, targets, n, hidden_size, vocab, dtype, ignore_index, z_loss, reduction, loss_out,
                   grad_hidden, grad_weight, grad_bias, weight_grad_dtype, accumulate, workspace, workspace_bytes, flags};
    return ce_run(c, true, stream);
}

size_t rlpl_adamw_plan_bytes(const int64_t* sizes, int64_t count) {
    const int64_t chunks = adam_chunks(sizes, count);
    return chunks < 0 ? 0 : adam_bytes(count, chunks);
}

int rlpl_adamw_plan_build(void* plan, size_t plan_bytes, const int64_t* sizes, int64_t count, void* const* params,
                          int param_dtype, void* const* copies, int copy_dtype, void* const* exp_avg,
                          void* const* exp_avg_sq, float* const* exp_avg_scale, float* const* exp_avg_sq_scale,
                          int state_bits, const double* weight_decay) {
    if (!plan || !sizes || !params || !exp_avg || !exp_avg_sq || !weight_decay) return RLPL_ERR_NULL;
    if (state_bits != 32 && state_bits != 8) return RLPL_ERR_DTYPE;
    const bool eight = state_bits == 8;
    if (eight && (!exp_avg_scale || !exp_avg_sq_scale)) return RLPL_ERR_NULL;
    const int64_t chunks = adam_chunks(sizes, count);
    if (chunks < 0) return RLPL_ERR_SHAPE;
    if (!known_dtype(param_dtype)) return RLPL_ERR_DTYPE;
    if (copies && (param_dtype != RLPL_F32 || (copy_dtype != RLPL_F16 && copy_dtype != RLPL_BF16))) return RLPL_ERR_DTYPE;
    if (!is_aligned(plan, 8)) return RLPL_ERR_ALIGN;
    if (plan_bytes < adam_bytes(count, chunks)) return RLPL_ERR_WORKSPACE;
    for (int64_t i = 0; i < count; ++i) {
        if (!std::isfinite(weight_decay[i]) || weight_decay[i] < 0.0) return RLPL_ERR_PARAM;
        if (sizes[i] == 0) continue;
        if (!params[i] || !exp_avg[i] || !exp_avg_sq[i] || (copies && !copies[i]) ||
            (eight && (!exp_avg_scale[i] || !exp_avg_sq_scale[i])))
            return RLPL_ERR_NULL;
        const uintptr_t state = eight ? 1 : 4;
        if (!is_aligned(params[i], dtype_bytes(param_dtype)) || (copies && !is_aligned(copies[i], 2)) ||
            !is_aligned(exp_avg[i], state) || !is_aligned(exp_avg_sq[i], state) ||
            (eight && (!is_aligned(exp_avg_scale[i], 4) || !is_aligned(exp_avg_sq_scale[i], 4))))
            return RLPL_ERR_ALIGN;
    }
    AdamPlan h{};
    h.magic = kAdamMagic;
    h.count = count;
    h.chunks = chunks;
    h.param_dtype = param_dtype;
    h.copy_dtype = copies ? copy_dtype : -1;
    h.state_bits = state_bits;
    h.tensors_at = sizeof(AdamPlan);
    h.chunks_at = h.tensors_at + uint64_t(count) * sizeof(AdamTensor);
    h.bytes = adam_bytes(count, chunks);
    char* out = static_cast<char*>(plan);
    std::memcpy(out, &h, sizeof(h));
    auto* tensors = reinterpret_cast<AdamTensor*>(out + h.tensors_at);
    auto* chunk = reinterpret_cast<AdamChunk*>(out + h.chunks_at);
    for (int64_t i = 0; i < count; ++i) {
        AdamTensor t{};
        t.param = params[i];
        t.copy = copies ? copies[i] : nullptr;
        t.m = exp_avg[i];
        t.v = exp_avg_sq[i];
        t.m_scale = eight ? exp_avg_scale[i] : nullptr;
        t.v_scale = eight ? exp_avg_sq_scale[i] : nullptr;
        t.n = sizes[i];
        t.weight_decay = weight_decay[i];
        t.aligned = is_aligned(t.param, 16) && is_aligned(t.copy, 16) && is_aligned(t.m, 16) && is_aligned(t.v, 16);
        tensors[i] = t;
        for (int64_t c = 0; c < div_up(sizes[i], kAdamChunk); ++c) *chunk++ = AdamChunk{uint32_t(i), uint32_t(c)};
    }
    return RLPL_OK;
}

int rlpl_adamw_step(const void* plan, const void* plan_device, const void* const* grads, int grad_dtype, double lr,
                    const float* lr_device, double beta1, double beta2, double eps, int64_t step,
                    const int64_t* step_device, const float* grad_scale, uint32_t seed, hipStream_t stream) {
    if (!plan || !plan_device || !grads) return RLPL_ERR_NULL;
    if (!known_dtype(grad_dtype)) return RLPL_ERR_DTYPE;
    if (!is_aligned(plan, 8) || !is_aligned(plan_device, 8) || !is_aligned(lr_device, 4) || !is_aligned(step_device, 8) ||
        !is_aligned(grad_scale, 4))
        return RLPL_ERR_ALIGN;
    if (!std::isfinite(lr) || lr < 0.0 || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) ||
        !std::isfinite(eps) || eps < 0.0 || (!step_device && step < 1))
        return RLPL_ERR_PARAM;
    AdamPlan h;
    std::memcpy(&h, plan, sizeof(h));
    if (h.magic != kAdamMagic) return RLPL_ERR_PARAM;
    const auto* tensors = reinterpret_cast<const AdamTensor*>(static_cast<const char*>(plan) + h.tensors_at);
    for (int64_t i = 0; i < h.count; ++i)
        if (!is_aligned(grads[i], dtype_bytes(grad_dtype))) return RLPL_ERR_ALIGN;
    const int st = device();
    if (st != RLPL_OK) return st;
    const char* dev = static_cast<const char*>(plan_device);
    AdamArgs a{};
    a.tensors = reinterpret_cast<const AdamTensor*>(dev + h.tensors_at);
    a.grad_scale = grad_scale;
    a.lr_at = lr_device;
    a.step_at = step_device;
    a.lr = lr;
    const double t = step_device ? 1.0 : double(step);
    a.correction1 = 1.0 - std::pow(beta1, t);
    a.log_beta1 = std::log(beta1);
    a.log_beta2 = std::log(beta2);
    a.root = float(1.0 / std::sqrt(1.0 - std::pow(beta2, t)));
    a.beta1 = float(beta1);
    a.beta2 = float(beta2);
    a.one_minus_beta1 = float(1.0 - beta1);
    a.one_minus_beta2 = float(1.0 - beta2);
    a.eps = float(eps);
    a.seed = mix(seed);
    a.step = uint32_t(step);
    a.copy_dtype = h.copy_dtype;
    const void* kernel = pick_adamw(h.param_dtype, grad_dtype, h.state_bits);
    // Windows of tensors whose gradients' pointers fit the kernel arguments, and within one at
    // most kAdamLaunchChunks workgroups a launch.
    const auto* chunk0 = reinterpret_cast<const AdamChunk*>(dev + h.chunks_at);
    int64_t done = 0;
    for (int64_t first = 0; first < h.count; first += kAdamWindow) {
        const int64_t last = first + kAdamWindow < h.count ? first + kAdamWindow : h.count;
        int64_t chunks = 0;
        for (int64_t i = first; i < last; ++i) {
            a.grads[i - first] = grads[i];
            chunks += div_up(tensors[i].n, kAdamChunk);
        }
        a.first = uint32_t(first);
        while (chunks > 0) {
            const int64_t now = chunks < kAdamLaunchChunks ? chunks : kAdamLaunchChunks;
            a.chunks = chunk0 + done;
            const int s = enqueue(kernel, a, dim3(unsigned(now)), kAdamThreads, stream);
            if (s != RLPL_OK) return s;
            done += now;
            chunks -= now;
        }
    }
    return RLPL_OK;
}

int layer_norm_fwd(const void* x, const void* weight, const void* bias, int64_t rows, int64_t cols, int dtype,
                   int weight_dtype, float eps, void* y, float* mean_out, float* rstd_out, hipStream_t stream) {
    if (!x || !y) return RLPL_ERR_NULL;
    if (!norm_shape_ok(rows, cols)) return RLPL_ERR_SHAPE;
    if (!norm_types_ok(dtype, weight_dtype)) return RLPL_ERR_DTYPE;
    if (!std::isfinite(eps) || eps < 0.0f) return RLPL_ERR_PARAM;
    const size_t e = dtype_bytes(dtype), we = dtype_bytes(weight_dtype);
    if (!is_aligned(x, e) || !is_aligned(y, e) || !is_aligned(weight, we) || !is_aligned(bias, we) ||
        !is_aligned(mean_out, 4) || !is_aligned(rstd_out, 4))
        return RLPL_ERR_ALIGN;
    const int st = device();
    if (st != RLPL_OK) return st;
    const NormRowKernel k = pick_norm_fwd(dtype, weight_dtype, cols);
    if (!k.kernel) return RLPL_ERR_DTYPE;
    const NormFwdArgs a{x, weight, bias, y, mean_out, rstd_out, rows, int32_t(cols), eps};
    return enqueue(k.kernel, a, dim3(row_grid(rows, k.rows_per_group)), k.threads, stream);
}

size_t layer_norm_workspace_bytes(int64_t rows, int64_t cols) {
    return norm_shape_ok(rows, cols) ? norm_layout(rows, cols).total : 0;
}

int layer_norm_bwd(const void* grad_y, const void* x, const void* weight, const float* mean, const float* rstd,
                   int64_t rows, int64_t cols, int dtype, int weight_dtype, void* grad_x, void* grad_weight,
                   void* grad_bias, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!grad_y || !x || !mean || !rstd) return RLPL_ERR_NULL;
    if (!norm_shape_ok(rows, cols)) return RLPL_ERR_SHAPE;
    if (!norm_types_ok(dtype, weight_dtype)) return RLPL_ERR_DTYPE;
    const size_t e = dtype_bytes(dtype), we = dtype_bytes(weight_dtype);
    if (!is_aligned(grad_y, e) || !is_aligned(x, e) || !is_aligned(grad_x, e) || !is_aligned(weight, we) ||
        !is_aligned(grad_weight, we) || !is_aligned(grad_bias, we) || !is_aligned(mean, 4) || !is_aligned(rstd, 4))
        return RLPL_ERR_ALIGN;
    const NormLayout L = norm_layout(rows, cols);
    if (!workspace || workspace_bytes < L.total) return RLPL_ERR_WORKSPACE;
    if (!is_aligned(workspace, 256)) return RLPL_ERR_ALIGN;
    int st = device();
    if (st != RLPL_OK) return st;
    const bool sums = grad_weight || grad_bias;
    if (!grad_x && !sums) return RLPL_OK;
    NormBwdArgs a{};
    a.dy = grad_y;
    a.x = x;
    a.w = weight;
    a.mean = mean;
    a.rstd = rstd;
    a.dx = grad_x;
    a.row_sums = static_cast<float2*>(workspace);
    a.part = sums ? reinterpret_cast<float*>(static_cast<char*>(workspace) + L.sums) : nullptr;
    a.rows = rows;
    a.cols = int32_t(cols);
    int64_t slabs;
    if (cols <= kNormHeldCols) {
        const NormRowKernel k = pick_norm_bwd_held(dtype, weight_dtype, cols);
        slabs = norm_held_grid(rows, cols, k.rows_per_group);
        st = enqueue(k.kernel, a, dim3(unsigned(slabs)), k.threads, stream);
    } else {
        const int64_t col_tiles = div_up(cols, norm_col_tile(dtype));
        slabs = norm_slabs(rows, col_tiles);
        a.slab_rows = div_up(rows, slabs);
        if (grad_x) {
            st = enqueue(pick_norm_row_sums(dtype, weight_dtype, cols), a, dim3(row_grid(rows, kNormThreads / 64)), kNormThreads,
                         stream);
            if (st != RLPL_OK) return st;
        }
        st = enqueue(pick_norm_bwd(dtype, weight_dtype, cols), a, dim3(unsigned(col_tiles), unsigned(slabs)), kNormThreads, stream);
    }
    if (st != RLPL_OK || !sums) return st;
    const NormReduceArgs r{a.part, grad_weight, grad_bias, int32_t(slabs), int32_t(cols)};
    return enqueue(pick_norm_reduce(weight_dtype), r, dim3(unsigned(div_up(cols, kNormReduceCols)), 2), kNormReduceThreads,
                   stream);
}

int rms_norm_fwd(const void* x, const void* weight, const void* residual, int64_t rows, int64_t cols, int dtype,
                 int weight_dtype, int stream_dtype, float eps, void* y, float* rstd_out, void* stream_out,
                 hipStream_t stream) {
    return rms_forward({x, weight, residual, rows, cols, dtype, weight_dtype, stream_dtype, eps, y, nullptr, rstd_out,
                        stream_out}, false, stream);
}

int rms_norm_fp8(const void* x, const void* weight, const void* residual, int64_t rows, int64_t cols, int dtype,
                 int weight_dtype, int stream_dtype, float eps, void* q, float* scale, float* rstd_out, void* stream_out,
                 hipStream_t stream) {
    return rms_forward({x, weight, residual, rows, cols, dtype, weight_dtype, stream_dtype, eps, q, scale, rstd_out,
                        stream_out}, true, stream);
}

size_t rms_norm_workspace_bytes(int64_t rows, int64_t cols) { return rms_shape_ok(rows, cols) ? rms_bytes(rows, cols) : 0; }

int rms_norm_bwd(const void* grad_y, const void* h, const void* weight, const float* rstd, const void* grad_stream,
                 int64_t rows, int64_t cols, int dtype, int weight_dtype, int stream_dtype, void* grad_h, void* grad_weight,
                 void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!grad_y || !h || !rstd) return RLPL_ERR_NULL;
    if (!rms_shape_ok(rows, cols)) return RLPL_ERR_SHAPE;
    if (!norm_types_ok(dtype, weight_dtype) || !norm_types_ok(dtype, stream_dtype)) return RLPL_ERR_DTYPE;
    const size_t re = dtype_bytes(stream_dtype), we = dtype_bytes(weight_dtype);
    if (!is_aligned(grad_y, dtype_bytes(dtype)) || !is_aligned(h, re) || !is_aligned(weight, we) || !is_aligned(rstd, 4) ||
        !is_aligned(grad_stream, re) || !is_aligned(grad_h, re) || !is_aligned(grad_weight, we))
        return RLPL_ERR_ALIGN;
    if (!workspace || workspace_bytes < rms_bytes(rows, cols)) return RLPL_ERR_WORKSPACE;
    if (!is_aligned(workspace, 256)) return RLPL_ERR_ALIGN;
    int st = device();
    if (st != RLPL_OK) return st;
    if (!grad_h && !grad_weight) return RLPL_OK;
    const NormRowKernel k = pick_rms_bwd(dtype, stream_dtype, cols);
    if (!k.kernel) return RLPL_ERR_DTYPE;
    const int64_t groups = norm_held_grid(rows, cols, k.rows_per_group);
    const RmsBwdArgs a{grad_y, h, weight, rstd, grad_stream, grad_h, grad_weight ? static_cast<float*>(workspace) : nullptr,
                       rows, int32_t(cols), weight_dtype == RLPL_F32 ? 1 : 0};
    st = enqueue(k.kernel, a, dim3(unsigned(groups)), k.threads, stream);
    if (st != RLPL_OK || !grad_weight) return st;
    const NormReduceArgs r{a.part, grad_weight, nullptr, int32_t(groups), int32_t(cols)};
    return enqueue(pick_norm_reduce(weight_dtype), r, dim3(unsigned(div_up(cols, kNormReduceCols)), 1), kNormReduceThreads,
                   stream);
}

size_t rlpl_grad_norm_workspace_bytes(const int64_t* sizes, int64_t count) {
    const int64_t launches = grad_launches(sizes, count);
    return launches < 0 ? 0 : grad_bytes(launches);
}

int rlpl_grad_norm(const void* const* grads, const int64_t* sizes, const int32_t* dtypes, int64_t count, int norm_kind,
                   const float* grad_scale, float max_norm, float eps, float* norm_out, float* scale_out, void* workspace,
                   size_t workspace_bytes, hipStream_t stream) {
    void* const* list = const_cast<void* const*>(grads);
    int st = grad_check(list, sizes, dtypes, count);
    if (st != RLPL_OK) return st;
    if (!norm_out) return RLPL_ERR_NULL;
    if (norm_kind != RLPL_NORM_2 && norm_kind != RLPL_NORM_INF) return RLPL_ERR_PARAM;
    if (scale_out && (!std::isfinite(max_norm) || max_norm < 0.0f || !std::isfinite(eps) || eps < 0.0f)) return RLPL_ERR_PARAM;
    if (!is_aligned(grad_scale, 4) || !is_aligned(norm_out, 4) || !is_aligned(scale_out, 4)) return RLPL_ERR_ALIGN;
    if (!workspace || workspace_bytes < grad_bytes(grad_launches(sizes, count))) return RLPL_ERR_WORKSPACE;
    if (!is_aligned(workspace, 256)) return RLPL_ERR_ALIGN;
    if ((st = device()) != RLPL_OK) return st;
    const bool inf = norm_kind == RLPL_NORM_INF;
    int64_t chunks = 0, tensors = 0;
    for (int64_t i = 0; i < count && chunks <= kGradAloneChunks; ++i) {
        chunks += div_up(sizes[i], kGradChunk);
        tensors += sizes[i] > 0;
    }
    GradNormArgs a;
    a.part = static_cast<double*>(workspace);
    a.finish = GradFinish{a.part, norm_out, scale_out, grad_scale, max_norm, eps, 0, inf ? 1 : 0};
    if (chunks <= kGradAloneChunks && tensors <= kGradWindow && tensors > 0)
        return grad_windows(a.list, list, sizes, dtypes, count,
                            [&](int64_t) { return enqueue(pick_grad_alone(inf), a, dim3(1), kGradAloneThreads, stream); });
    st = grad_windows(a.list, list, sizes, dtypes, count, [&](int64_t here) {
        const unsigned grid = grad_grid(here);
        const int s = enqueue(pick_grad_norm(inf), a, dim3(grid), kGradThreads, stream);
        a.part += grid;
        a.finish.parts += int32_t(grid);
        return s;
    });
    return st != RLPL_OK ? st : enqueue(grad_finish_kernel(), a.finish, dim3(1), kGradAloneThreads, stream);
}

int rlpl_grad_scale(void* const* grads, const int64_t* sizes, const int32_t* dtypes, int64_t count, const float* scale,
                    hipStream_t stream) {
    int st = grad_check(grads, sizes, dtypes, count);
    if (st != RLPL_OK) return st;
    if (!scale) return RLPL_ERR_NULL;
    if (!is_aligned(scale, 4)) return RLPL_ERR_ALIGN;
    if (!grads_apart(grads, sizes, dtypes, count)) return RLPL_ERR_PARAM;
    if ((st = device()) != RLPL_OK) return st;
    GradScaleArgs a;
    a.scale = scale;
    return grad_windows(a.list, grads, sizes, dtypes, count, [&](int64_t here) {
        return enqueue(grad_scale_kernel(), a, dim3(grad_grid(here)), kGradThreads, stream);
    });
}

}  // extern "C"
