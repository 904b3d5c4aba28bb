// C ABI of the operators that score tokens (declared in
// include/rl_post_loss.h): log-probabilities over logit rows, and products of
// 8-bit operands with the quantisation of those.
//
// As in abi.cpp, arguments are validated on the host before any HIP call,
// nothing is allocated and nothing synchronises; kernels go to the caller's
// stream.
#include "train_abi.h"

#include <cmath>

#include "fp8_kernels.h"
#include "token_kernels.h"

namespace {

using namespace rlpl;

constexpr int64_t kMaxRows = int64_t(1) << 31;
constexpr int64_t kMaxVocab = (int64_t(1) << 31) - 65536;   // columns are counted in 32 bits, a step of lanes past the end
constexpr int64_t kMaxTopVocab = int64_t(1) << 22;          // 32 pieces of 131,072 with 64 alternatives
constexpr int64_t kMaxElements = int64_t(1) << 62;

// The tiles' ring is beyond the default limit of LDS.
bool set_up(int dev) {
    if (!is_gfx950(dev)) return false;
    for (int dt : {RLPL_F32, RLPL_F16, RLPL_BF16})
        for (int kind = 0; kind < kFp8Kinds; ++kind) {
            const void* k = pick_fp8_tile(dt, kind);
            if (k && hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, kFp8Shapes[kind].lds) != hipSuccess)
                return false;
        }
    return true;
}

Devices<set_up> g_devices;
int device() { return g_devices.current(); }

unsigned capped(int64_t grid, int64_t cap) { return unsigned(grid < cap ? grid : cap); }

// ----------------------------------------------------------------------------- token log-probabilities

bool token_shape_ok(int64_t rows, int64_t vocab, int64_t top_k) {
    return rows >= 1 && rows < kMaxRows && vocab >= 1 && vocab <= (top_k > 0 ? kMaxTopVocab : kMaxVocab) && top_k >= 0 &&
           top_k <= kTokenMaxTop && top_k <= vocab;
}
// Rows r at group_stride (r / inner) + row_stride (r % inner), all of them within 2^62 elements.
bool token_strides_ok(int64_t rows, int64_t inner, int64_t group_stride, int64_t row_stride) {
    if (inner < 1 || inner > rows || group_stride < 0 || row_stride < 0) return false;
    const __int128 last = __int128((rows - 1) / inner) * group_stride + __int128(inner - 1) * row_stride;
    return last < kMaxElements;
}
float token_scale(float t) { return float(1.4426950408889634 / double(t)); }
// T such that log2(e) / T is a float.
bool token_temperature_ok(float t) { return std::isfinite(t) && t > 0.0f && std::isfinite(token_scale(t)); }
int token_vector(int dtype) { return 16 / int(dtype_bytes(dtype)); }
int64_t token_vectors(int64_t vocab, int dtype) { return vocab / token_vector(dtype); }

// The pieces depend on the elements' size through their vectors: workspaces are sized for the most of them.
size_t token_bytes(int64_t rows, int64_t vocab, int64_t top_k) {
    const int64_t pieces = token_fwd_pieces(rows, token_vectors(vocab, RLPL_F32), token_vector(RLPL_F32), int(top_k));
    if (pieces == 1 || vocab <= kTokenShort) return 256;
    return up256(size_t(rows) * size_t(pieces) * sizeof(TokenPart)) +
           up256(size_t(rows) * size_t(pieces) * size_t(top_k) * sizeof(uint64_t));
}

// ----------------------------------------------------------------------------- 8-bit products

constexpr int64_t kFp8MaxRows = int64_t(1) << 20;
constexpr int64_t kFp8MaxHidden = 65536;
constexpr int64_t kFp8MaxVocab = int64_t(1) << 22;
constexpr int64_t kFp8MaxTiles = int64_t(1) << 24;          // of the small shape (x 256 lanes < 2^32)

bool fp8_shape_ok(int64_t n, int64_t h, int64_t vocab) {
    return n >= 1 && n <= kFp8MaxRows && h >= 16 && h <= kFp8MaxHidden && h % 16 == 0 && vocab >= 1 && vocab < kFp8MaxVocab &&
           div_up(n, kFp8Shapes[kFp8Small].tokens) * div_up(vocab, kFp8Shapes[kFp8Small].vocab) < kFp8MaxTiles;
}

// The time of a product's tiles in microseconds, to choose between their shapes: a tile of `steps` blocks of K takes
// fixed + step * steps alone, and a chip full of them fill + pace * steps each on one of its 256 compute units; a
// projection that the last cache does not hold arrives at `rate` GB a millisecond, once a row of tiles.  Fitted to 219 sizes drawn
// from 17 to 4096 rows, H from 64 to 8192 and 1000 to 131072 entries, where the choice is 1 to 2 % behind the best shape's time:
// 333 x 2048 x 5003 takes 11 us with the small shape, 18 and 38 with the middle and the large one; 2048 x 4096 x 4096 66, 46 and
// 58; small, narrow and middle 64 x 4096 x 32000 24, 31 and 39, 64 x 4096 x 128256 126, 117 and 123, 128 x 4096 x 32000 37, 32
// and 42; 128 x 4096 x 128256 182, 166, 136 and the large one 139; 2048 x 4096 x 128256 1969 with the small one, 1533 with the
// middle and 1026 with the large one.
struct Fp8Pace {
    double fixed, step, fill, pace, rate;
};
constexpr Fp8Pace kFp8Paces[] = {{2.8, 0.51, 0.30, 0.236, 6.0}, {1.0, 0.685, 0.79, 0.44, 6.4}, {3.7, 0.89, 1.37, 0.633, 4.5},
                                 {9.2, 1.02, 7.5, 1.53, 3.6}};
// float32 outputs take twice the matrix instructions, and conversions (1024 x 4096 x 4096 46 and 51 us with the small shape
// and the middle one, 2048 x 4096 x 4096 86 and 69, 8192^3 1257 and 974).
constexpr Fp8Pace kFp8WidePaces[] = {{0.0, 0.82, 0.65, 0.30, 5.4}, {0.7, 0.86, 1.44, 0.566, 5.4}, {2.9, 1.19, 2.57, 0.90, 3.6}};
constexpr double kFp8Cached = 268435456.0;
double fp8_time(int kind, int64_t n, int64_t blocks, int64_t vocab, bool wide) {
    const Fp8TileShape& s = kFp8Shapes[kind];
    const Fp8Pace& p = wide ? kFp8WidePaces[kind] : kFp8Paces[kind];
    const double rows = double(div_up(n, s.tokens)), tiles = double(div_up(vocab, s.vocab)) * rows;
    // few workgroups a compute unit leave part of the last round idle
    const double rounds = kind == kFp8Small ? tiles / 256.0 : 0.5 * (tiles / 256.0 + std::ceil(tiles / 256.0));
    const double one = p.fixed + p.step * double(blocks), all = rounds * (p.fill + p.pace * double(blocks));
    const double bytes = double(vocab) * double(blocks) * kFp8Group, stream = bytes > kFp8Cached ? bytes * rows / p.rate * 1e-6 : 0.0;
    const double busy = all > one ? all + 0.3 * one : one + 0.3 * all;
    return busy > stream ? busy : stream;
}
int fp8_kind(int64_t n, int64_t blocks, int64_t vocab, int out_dtype) {
    // One small tile for each compute unit at most, or two: four groups of wavefronts share K, or two (33 x 8192 x 4096, 64
    // tiles: 40, 27 and 21 us with one, two and four; 64 x 8192 x 8192, 128 tiles: 41, 29 and 24; 128 x 8192 x 12000, 376 tiles:
    // 43, 35 and 46; 64 x 4096 x 32000, 500 tiles: 24.5, 22.7 and 29.7; 700 x 4096 x 3000, 517 tiles: 25, 31 and 37).
    const Fp8TileShape& small = kFp8Shapes[kFp8Small];
    const int64_t tiles = div_up(vocab, small.vocab) * div_up(n, small.tokens);
    if (blocks >= 8 && tiles <= 512) return tiles <= 256 ? kFp8Deep : kFp8Twice;
    const bool wide = out_dtype == RLPL_F32;
    int best = kFp8Small;
    for (int kind = kFp8Narrow; kind <= (wide ? kFp8Middle : kFp8Large); ++kind)
        if (fp8_time(kind, n, blocks, vocab, wide) < fp8_time(best, n, blocks, vocab, wide)) best = kind;
    return best;
}

// Entries a workgroup of few rows takes: fewer where there would be few workgroups (one compute unit streams 64 of 8192 in
// 19 us), more where x is read often (1 x 8192 x 512 takes 11.2, 11.6 and 19.0 us with 16, 32 and 64; 1 x 4096 x 16384 12.8,
// 12.5 and 14.8; 16 x 4096 x 128256 150, 117 and 105).
int fp8_few_entries(int64_t vocab) { return vocab <= 8192 ? 16 : vocab <= 24576 ? 32 : 64; }

// For the large shape, the scales of the rows, one block of K after the other: a lane's tokens are then neighbours
// (2048 x 4096 x 128256: 1113 us with the scales where they lie, a cache line a token and step; 1026 with 3 us to turn
// them).
int64_t fp8_scale_ld(int64_t n) { return div_up(n, kTurnRows) * kTurnRows; }
size_t fp8_bytes(int64_t n, int64_t h) { return up256(size_t(fp8_scale_ld(n)) * size_t(div_up(h, kFp8Group)) * sizeof(float)); }

}  // namespace

extern "C" {

size_t token_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int64_t top_k) {
    return token_shape_ok(rows, vocab, top_k) ? token_bytes(rows, vocab, top_k) : 0;
}

int token_logprobs_fwd(const void* logits, const int64_t* targets, const void* mask, int64_t rows, int64_t vocab,
                       int64_t inner, int64_t group_stride, int64_t row_stride, int dtype, float temperature, int64_t top_k,
                       float* logp_out, float* lse_out, float* entropy_out, float* top_logp_out, int64_t* top_index_out,
                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
    if (!logits || !targets || !logp_out || !lse_out || (top_k > 0 && (!top_logp_out || !top_index_out))) return RLPL_ERR_NULL;
    if (!token_shape_ok(rows, vocab, top_k) || !token_strides_ok(rows, inner, group_stride, row_stride)) return RLPL_ERR_SHAPE;
    if (!known_dtype(dtype)) return RLPL_ERR_DTYPE;
    if (!token_temperature_ok(temperature)) return RLPL_ERR_PARAM;
    if (!is_aligned(logits, dtype_bytes(dtype)) || !is_aligned(targets, 8) || !is_aligned(logp_out, 4) ||
        !is_aligned(lse_out, 4) || !is_aligned(entropy_out, 4) || !is_aligned(top_logp_out, 4) || !is_aligned(top_index_out, 8))
        return RLPL_ERR_ALIGN;
    if (!workspace || workspace_bytes < token_bytes(rows, vocab, top_k)) return RLPL_ERR_WORKSPACE;
    if (!is_aligned(workspace, 256)) return RLPL_ERR_ALIGN;
    int st = device();
    if (st != RLPL_OK) return st;
    const int64_t vectors = token_vectors(vocab, dtype);
    TokenFwdArgs a{};
    a.in = TokenRows{logits, static_cast<const uint8_t*>(mask), rows, inner, group_stride, row_stride, vocab};
    a.targets = targets;
    a.logp = logp_out;
    a.lse = lse_out;
    a.entropy = entropy_out;
    a.top_logp = top_logp_out;
    a.top_index = top_index_out;
    a.pieces = vocab <= kTokenShort ? 1 : int32_t(token_fwd_pieces(rows, vectors, token_vector(dtype), int(top_k)));
    a.piece_vectors = div_up(vectors > 0 ? vectors : 1, a.pieces);
    a.top_k = int32_t(top_k);
    a.scale = token_scale(temperature);
    a.part = static_cast<TokenPart*>(workspace);
    a.part_top = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) +
                                             up256(size_t(rows) * size_t(a.pieces) * sizeof(TokenPart)));
    const int64_t groups = vocab <= kTokenShort ? div_up(rows, kTokenThreads / 64) : rows * a.pieces;
    st = enqueue(pick_token_fwd(dtype, top_k > 0, vocab), a, dim3(capped(groups, kTokenMaxGrid)), kTokenThreads, stream);
    if (st != RLPL_OK || a.pieces == 1) return st;
    return enqueue(pick_token_join(dtype), a, dim3(capped(rows, kTokenMaxGrid)), kTokenThreads, stream);
}

int token_logprobs_bwd(const void* logits, const int64_t* targets, const void* mask, const float* lse, const float* entropy,
                       const float* grad_logp, const float* grad_entropy, int64_t rows, int64_t vocab, int64_t inner,
                       int64_t group_stride, int64_t row_stride, int dtype, float temperature, void* grad_logits,
                       hipStream_t stream) {
    if (!logits || !targets || !lse || !grad_logits || (grad_entropy && !entropy)) return RLPL_ERR_NULL;
    if (!token_shape_ok(rows, vocab, 0) || !token_strides_ok(rows, inner, group_stride, row_stride)) return RLPL_ERR_SHAPE;
    if (!known_dtype(dtype)) return RLPL_ERR_DTYPE;
    if (!token_temperature_ok(temperature)) return RLPL_ERR_PARAM;
    const size_t e = dtype_bytes(dtype);
    if (!is_aligned(logits, e) || !is_aligned(targets, 8) || !is_aligned(lse, 4) || !is_aligned(entropy, 4) ||
        !is_aligned(grad_logp, 4) || !is_aligned(grad_entropy, 4) || !is_aligned(grad_logits, e))
        return RLPL_ERR_ALIGN;
    const int st = device();
    if (st != RLPL_OK) return st;
    const int64_t vectors = token_vectors(vocab, dtype);
    TokenBwdArgs a{};
    a.in = TokenRows{logits, static_cast<const uint8_t*>(mask), rows, inner, group_stride, row_stride, vocab};
    a.targets = targets;
    a.lse = lse;
    a.entropy = entropy;
    a.grad_logp = grad_logp;
    a.grad_entropy = grad_entropy;
    a.grad = grad_logits;
    // pieces of 8 vectors a lane
    const int lanes = vocab <= kTokenShortBwd ? 64 : kTokenThreads;
    a.pieces = int32_t(div_up(vectors > 0 ? vectors : 1, 8 * lanes));
    a.piece_vectors = div_up(vectors > 0 ? vectors : 1, a.pieces);
    a.inv_t = float(1.0 / double(temperature));
    a.scale = token_scale(temperature);
    return enqueue(pick_token_bwd(dtype, vocab), a, dim3(capped(div_up(rows * a.pieces, kTokenThreads / lanes), kTokenMaxGrid)),
                   kTokenThreads, stream);
}

int rlpl_fp8_quantize(const void* x, int64_t rows, int64_t cols, int64_t row_stride, int dtype, int block_rows, void* q,
                      float* scale, hipStream_t stream) {
    if (!x || !q || !scale) return RLPL_ERR_NULL;
    if (rows < 1 || rows >= kMaxRows || cols < 1 || cols > kMaxVocab || row_stride < 0 ||
        __int128(rows - 1) * row_stride >= kMaxElements)
        return RLPL_ERR_SHAPE;
    if (!known_dtype(dtype)) return RLPL_ERR_DTYPE;
    if (block_rows != 1 && block_rows != kFp8Group) return RLPL_ERR_PARAM;
    if (!is_aligned(x, dtype_bytes(dtype)) || !is_aligned(scale, 4)) return RLPL_ERR_ALIGN;
    const int st = device();
    if (st != RLPL_OK) return st;
    const int64_t groups = div_up(cols, kFp8Group);
    const QuantiseArgs a{x, static_cast<uint8_t*>(q), scale, rows, row_stride, int32_t(cols), int32_t(groups)};
    const int64_t work = block_rows == 1 ? div_up(rows * groups, 16) : div_up(rows, kFp8Group) * groups;
    return enqueue(pick_quantise(dtype, block_rows != 1), a, dim3(capped(work, kFp8MaxGrid)), kFp8Threads, stream);
}

size_t fp8_linear_workspace_bytes(int64_t n, int64_t hidden_size, int64_t vocab) {
    return fp8_shape_ok(n, hidden_size, vocab) ? fp8_bytes(n, hidden_size) : 0;
}

int fp8_linear(const void* x, const float* x_scale, const void* weight, const float* weight_scale, const void* bias, int64_t n,
               int64_t hidden_size, int64_t vocab, int out_dtype, void* out, void* workspace, size_t workspace_bytes,
               hipStream_t stream) {
    if (!x || !x_scale || !weight || !weight_scale || !out) return RLPL_ERR_NULL;
    if (!fp8_shape_ok(n, hidden_size, vocab)) return RLPL_ERR_SHAPE;
    if (!known_dtype(out_dtype)) return RLPL_ERR_DTYPE;
    const size_t e = dtype_bytes(out_dtype);
    if (!is_aligned(x, 16) || !is_aligned(weight, 16) || !is_aligned(x_scale, 4) || !is_aligned(weight_scale, 4) ||
        !is_aligned(bias, e) || !is_aligned(out, e))
        return RLPL_ERR_ALIGN;
    if (!workspace || workspace_bytes < fp8_bytes(n, hidden_size)) return RLPL_ERR_WORKSPACE;
    if (!is_aligned(workspace, 256)) return RLPL_ERR_ALIGN;
    const int st = device();
    if (st != RLPL_OK) return st;
    Fp8LinearArgs a{static_cast<const uint8_t*>(x), x_scale, static_cast<const uint8_t*>(weight), weight_scale, bias, out,
                    int32_t(n), int32_t(hidden_size), int32_t(vocab), int32_t(div_up(hidden_size, kFp8Group)), 0, 0};
    if (n <= kFp8FewRows) {
        const int entries = fp8_few_entries(vocab);
        return enqueue(pick_fp8_few(out_dtype, entries), a, dim3(unsigned(div_up(vocab, entries))), kFp8Threads, stream);
    }
    const int kind = fp8_kind(n, a.blocks, vocab, out_dtype);
    const Fp8TileShape& s = kFp8Shapes[kind];
    a.tiles_v = uint32_t(div_up(vocab, s.vocab));
    a.tiles_t = uint32_t(div_up(n, s.tokens));
    if (kind == kFp8Large) {
        a.scale_ld = int32_t(fp8_scale_ld(n));
        const TurnArgs t{x_scale, static_cast<float*>(workspace), a.n, a.blocks, a.scale_ld};
        const int turned = enqueue(turn_kernel(), t, dim3(unsigned(div_up(n, kTurnRows)), unsigned(div_up(a.blocks, kTurnCols))),
                                   kTurnRows, stream);
        if (turned != RLPL_OK) return turned;
        a.x_scale = t.to;
    }
    return enqueue(pick_fp8_tile(out_dtype, kind), a, dim3(a.tiles_v * a.tiles_t), s.threads, stream, size_t(s.lds));
}

}  // extern "C"
