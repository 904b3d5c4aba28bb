// Internal interface between the C ABI layer (score_abi.cpp) and the kernels
// of 8-bit operands (fp8_kernels.hip).  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "rms_kernels.h"

namespace rlpl {

constexpr int kFp8Threads = 256;
constexpr int64_t kFp8MaxGrid = 1 << 20;

struct QuantiseArgs {
    const void* x;             // (rows, cols) dtype, rows ld elements apart
    uint8_t* q;                // (rows, cols) e4m3, dense
    float* scale;              // (row blocks, groups)
    int64_t rows, ld;
    int32_t cols, groups;
};
const void* pick_quantise(int dtype, bool square);   // groups of 1 x 128, or 128 x 128

struct Fp8LinearArgs {
    const uint8_t* x;          // (n, K) e4m3
    const float* x_scale;      // (n, blocks)
    const uint8_t* w;          // (vocab, K) e4m3
    const float* w_scale;      // (vocab / 128, blocks)
    const void* bias;          // (vocab) of the output's type, or NULL
    void* out;                 // (n, vocab)
    int32_t n, K, vocab, blocks;
    uint32_t tiles_v, tiles_t; // of fp8_tile
    int32_t scale_ld;          // kFp8Large: x_scale is (blocks, scale_ld)
};
// (rows, cols) to (cols, ld).
struct TurnArgs {
    const float* from;
    float* to;
    int32_t rows, cols, ld;
};
const void* turn_kernel();
constexpr int kTurnRows = 64, kTurnCols = 4;   // of a workgroup

// Tiles of entries by tokens (fp8_gemm.hip).
struct Fp8TileShape {
    int vocab, tokens, threads, lds;
};
enum { kFp8Small = 0, kFp8Narrow = 1, kFp8Middle = 2, kFp8Large = 3, kFp8Deep = 4, kFp8Twice = 5, kFp8Kinds = 6 };   // no large float32 one
constexpr Fp8TileShape kFp8Shapes[] = {{64, 64, 256, 32 * 1024}, {128, 64, 256, 72 * 1024}, {128, 128, 256, 80 * 1024},
                                       {256, 256, 512, 160 * 1024}, {64, 64, 1024, 128 * 1024}, {64, 64, 512, 64 * 1024}};
const void* pick_fp8_tile(int out_dtype, int kind);

// Up to 16 rows: a workgroup takes 64 vocabulary entries, or 32 or 16, its four wavefronts every fourth block of K each.
constexpr int kFp8FewRows = 16;
const void* pick_fp8_few(int out_dtype, int entries);

}  // namespace rlpl
