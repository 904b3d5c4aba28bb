// Internal interface between the C ABI layer (score_abi.cpp) and the kernels
// of the token log-probabilities over logit rows (token_kernels.hip).  Not
// part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace rlpl {

constexpr int kTokenThreads = 256;
constexpr int kTokenMaxTop = 64;           // alternatives a row can give: no more than a wavefront's lanes
constexpr int kTokenMaxPieces = 64;        // pieces of a row
constexpr int kTokenMaxKeys = 2048;        // pieces times alternatives
constexpr int kTokenBlocks = 16;           // blocks of 32 elements that a lane has of a piece with alternatives, at most
// Rows of up to this many elements go to a wavefront each (20480 rows of bf16, a workgroup a row in brackets: 333 elements
// 12.5 (35.7) us and with 20 alternatives 23.6 (101), 4001 elements 35.9 (54.6) and 69 (122); backward 333 elements 11.8
// (26.1), 2048 27 (36), 4001 59 (52)).
constexpr int64_t kTokenShort = 4096;
constexpr int64_t kTokenShortBwd = 2048;
// From this |lse| on, its rounding to float32 is half a step of a float16 gradient (2^-11), and the backward pass does without it.
constexpr float kTokenFar = 8192.0f;
// Such a row is shared by this many workgroups at most, since each of them reads all of it (a row of 2^31 elements has 262,144
// pieces otherwise).
constexpr int kTokenFarPieces = 1024;
constexpr int64_t kTokenMaxGrid = 1 << 20; // workgroups of a launch (they stride over the rest)

// Where the rows lie: row r at group_stride (r / inner) + row_stride (r % inner) elements.
struct TokenRows {
    const void* logits;
    const uint8_t* mask;       // (rows) bytes, zero: the row is not read; or NULL
    int64_t rows, inner, group_stride, row_stride;
    int64_t vocab;             // < 2^31
};

// What a piece of a row leaves: its largest logit, and the sums over its elements that count from it.
struct TokenPart {
    float top, sum, weighted, pad;
};

struct TokenFwdArgs {
    TokenRows in;
    const int64_t* targets;    // (rows)
    float* logp;               // (rows)
    float* lse;                // (rows)
    float* entropy;            // (rows) or NULL
    float* top_logp;           // (rows, top_k)
    int64_t* top_index;        // (rows, top_k)
    TokenPart* part;           // (rows, pieces), pieces > 1
    uint64_t* part_top;        // (rows, pieces, top_k) keys, the largest first
    int64_t piece_vectors;     // 16-byte vectors of a piece
    int32_t pieces, top_k;
    float scale;               // log2(e) / temperature
};

struct TokenBwdArgs {
    TokenRows in;
    const int64_t* targets;
    const float* lse;
    const float* entropy;      // (rows), read with grad_entropy only
    const float* grad_logp;    // (rows) or NULL
    const float* grad_entropy; // (rows) or NULL
    void* grad;                // (rows, vocab), dense
    int64_t piece_vectors;
    int32_t pieces;
    float inv_t;               // 1 / temperature
    float scale;               // log2(e) / temperature
};

// Pieces a row is cut into by the forward, so that few long rows still fill the chip: 1024 workgroups in all, each with a
// vector for every lane at least; with alternatives pieces of 131,072 elements at most (32 of them take 2^22 elements).
// Rows of up to 32 vectors a lane stay whole, since a second launch takes longer than what pieces save (8 rows of bf16
// with 20 alternatives, whole and in pieces: 32000 elements 15.3 and 17.4 us, 65536 15.4 and 17.5, 128256 18.0 and 18.3; 300
// rows of 65536 17.2 and 21.7).
inline int64_t token_fwd_pieces(int64_t rows, int64_t vectors, int vector, int top_k) {
    const int64_t most = (vectors + kTokenThreads - 1) / kTokenThreads;
    if (most <= 32) return 1;
    int64_t p = 1024 / rows;
    if (p > most) p = most;
    if (p > kTokenMaxPieces) p = kTokenMaxPieces;
    if (top_k > 0) {
        if (p > kTokenMaxKeys / top_k) p = kTokenMaxKeys / top_k;
        const int64_t room = int64_t(kTokenBlocks) * 32 / vector * kTokenThreads;   // vectors
        const int64_t least = (vectors + room - 1) / room;
        if (p < least) p = least;
    }
    return p < 1 ? 1 : p;
}

const void* pick_token_fwd(int dtype, bool top, int64_t vocab);
const void* pick_token_join(int dtype);
const void* pick_token_bwd(int dtype, int64_t vocab);

}  // namespace rlpl
