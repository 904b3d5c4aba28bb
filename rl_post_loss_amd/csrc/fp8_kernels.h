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
};

// Few rows: a workgroup takes 64 vocabulary entries and `tokens` rows, its four wavefronts every fourth block of K each.
constexpr int kFp8SmallVocab = 64;
const void* pick_fp8_small(int out_dtype, int tokens);   // 16, 32 or 64 rows

}  // namespace rlpl
