// Internal interface between the C ABI layer (train_abi.cpp) and the
// vocabulary cross-entropy kernels (ce_kernels.hip).  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "logprob_kernels.h"

namespace rlpl {

constexpr int kCeThreads = 256;            // workgroups of the row and column kernels
constexpr int kCeCompactThreads = 1024;
// The shapes of the products' tiles: `tile` rows by columns, workgroups of `threads` with a ring of `lds` bytes.  For
// the splits of K: how many run at once, and, in quarters of a K step, what a workgroup's first copies and epilogue
// cost (of the hidden product, of the weight's), what a plane's sum at the end does, and how many of a plane's
// tiles take one more (their bytes).
struct CeShape {
    int tile, threads, lds, at_once, extra, weight_extra, plane, plane_tiles;
};
constexpr CeShape kCeLarge{256, 512, 160 * 1024, 256, 48, 28, 1, 3};
constexpr CeShape kCeSmall{64, 256, 32 * 1024, 1280, 24, 24, 3, 32};
// The small tile's ring for the loss's logits where its tiles are few: four slots of each operand, two workgroups a
// compute unit, up to kCeDeepTiles of them (64 x 4096 x 8000: loss 43.6 -> 32.6 us, 200 x 2048 x 4000 27.8 -> 23.4).
constexpr int kCeDeepLds = 64 * 1024;
constexpr int64_t kCeDeepTiles = 512;
constexpr int64_t kCeMaxRows = int64_t(1) << 24;
constexpr int kCeMaxSplits = 64;

// What the compaction leaves on the device: the number of rows that count, (after the loss) the
// factor of the gradients: 1 / max(count, 1) or 1, over the scale dz is held at, and the splits of the
// hidden product's K; and how many workgroups of ce_row are done with their rows.
struct CeState {
    int32_t count;
    float scale;
    uint32_t splits;
    uint32_t done;
};

// The rows whose target is not ignore_index, in order, and their hidden states side by side.
struct CePrepareArgs {
    const int64_t* targets;    // (n)
    int64_t ignore_index, vocab;
    int32_t n;
    int32_t* row;              // (n): row of the k-th kept one
    int32_t* place;            // (n): place of a row among the kept ones, or -1
    int32_t* target;           // (n): target of the k-th kept row, -1 where it is outside [0, vocab)
    CeState* state;
    const void* hidden;        // (n, cols) 2-byte elements, cols a multiple of 8
    void* out;                 // (kept rows, cols)
    int32_t cols;
};
// Up to kCePrepareRows rows in one kernel, a workgroup a row, each counting the kept rows before its own; more in
// two: one workgroup's scan, then the copy.  The one kernel's counting grows with n^2: 200 rows of 512 take 2.8 us,
// 1024 of 4096 7.6 and 2048 of 4096 10.7; the two kernels take 10.8 + 7.4 for 6001 rows of 2048, half of them kept.
constexpr int64_t kCePrepareRows = 2048;
const void* ce_prepare_kernel();
const void* ce_compact_kernel();
const void* ce_gather_kernel();

// One of the step's four products (the kernel's template argument):
//   kCeLogits   per row and tile of columns (max, sum exp(z - max)), and the target's logit
//   kCeDlogits  dz of a piece of the vocabulary, in the operand dtype, scaled by dz_scale
//   kCeHidden   dz . weight of a piece, into (or added to) float32 planes, one a split of K
//   kCeWeight   dz^T . hidden of a piece, scaled, in the gradient's dtype
// with z = hidden . weight^T + bias.  A (M x K) and B (K x N) as in GemmArgs.
enum { kCeLogits = 0, kCeDlogits = 1, kCeHidden = 2, kCeWeight = 3 };

struct CeGemmArgs {
    const void* a;
    const void* b;
    int64_t lda, ldb;
    int32_t M, N, K;           // kCeWeight: K, else M, is at most state->count
    int32_t split_k;           // the longest piece's K (kCeHidden)
    uint32_t tiles_m, tiles_n; // of the launch (tiles past the kept rows end at once)
    const CeState* state;
    void* c;
    int64_t ldc;
    int32_t accumulate;        // add to c (kCeHidden, and kCeWeight with a float32 c)
    int32_t out_f32;           // kCeWeight: c is float32, else the operand dtype
    const void* bias;          // (N) or NULL
    const int32_t* target;     // (kept rows)
    int32_t first;             // vocabulary index of column 0
    const float* lse;          // (kept rows) (kCeDlogits)
    float z_loss2;             // 2 z_loss (kCeDlogits)
    float dz_scale;            // (kCeDlogits)
    float* part;               // (kept rows, tiles_n, 2) (kCeLogits)
    float* target_logit;       // (kept rows) (kCeLogits)
    float* col_part;           // (tiles_m, col_ld) from column 0 on: sums of dz over a tile's rows, or NULL (kCeDlogits)
    int64_t col_ld;
    float* kept;               // room for the first columns' logits, kept_room blocks of 16 rows by 256 columns, written by
    uint32_t kept_room;        // kCeLogits; or NULL
};
const void* pick_ce_gemm(int dtype, bool small, int product);   // kCeLogits or kCeDlogits
const void* pick_ce_deep_logits(int dtype);                     // kCeLogits, small, with kCeDeepLds
const void* pick_ce_dz(int dtype, bool small);                  // kCeDlogits of the tiles with kept logits (kCeDlogits of
                                                                // a piece that has `kept` forms the others')

// The two products that take dz, in one launch: the first hidden_blocks workgroups (a multiple of 8, or 0) are the
// hidden product's, the others the weight's.  Their tiles share the chip, so neither ends with idle compute units.
struct CeGradArgs {
    CeGemmArgs hidden, weight;
    uint32_t hidden_blocks;
};
const void* pick_ce_grads(int dtype, bool small);

// dz is held at this scale (the onehot's 1), so that small probabilities stay
// above fp16's subnormals; bf16 has float32's range.  A penalty's factor
// 1 + 2 z_loss lse takes room above: the scale is the largest of 256, 128 and
// 64 (z_loss <= 1) that holds it for |lse| up to 500.
inline float ce_dz_scale(int dtype, float z_loss) {
    if (dtype != 1) return 1.0f;
    float scale = 256.0f;
    while (scale * (1.0f + 1000.0f * z_loss) > 65504.0f) scale *= 0.5f;
    return scale;
}

// A kept row's log-sum-exp and loss; the workgroup that is done last sums the rows' losses.
struct CeRowArgs {
    const float* part;
    const float* target_logit;
    const int32_t* target;
    CeState* state;
    float* lse;                // (kept rows)
    float* row_loss;           // (kept rows)
    float* loss;
    float z_loss, inv_dz_scale;
    int32_t tiles, mean;
    int32_t split_k, most;     // of the hidden product that follows: the longest piece's K, the most splits (1 where none
    uint32_t plane_rows;       // follows), the rows of tiles that the planes have room for, its tiles along the hidden
    uint32_t tiles_h;          // size, the weight product's tiles beside it, their shape
    uint32_t weight_tiles;
    int32_t small;
};
constexpr int64_t kCeRowGrid = 512;
const void* ce_row_kernel();

// The hidden gradient: the splits' planes of a kept row summed in order and scaled, zeros in an ignored row; and, by
// the workgroups after the first row_blocks, the bias's gradient: the row tiles' column sums, likewise.
struct CeFinishArgs {
    const float* part;
    const int32_t* place;
    const CeState* state;
    void* out;                 // (n, cols) operand dtype or float32
    int32_t n, cols;
    uint32_t row_blocks;       // 0: no hidden gradient
    int32_t hidden_f32;
    const float* col_part;     // (tiles of col_tile rows, vocab)
    void* bias;                // (vocab) operand dtype or float32
    int32_t vocab, out_f32, accumulate;
    int32_t col_tile;          // rows of a tile of dz
};
const void* pick_ce_finish(int dtype);

}  // namespace rlpl
