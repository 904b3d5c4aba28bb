// Internal interface between the C ABI layer (train_abi.cpp) and the RMS norm
// kernels (rms_kernels.hip).  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "norm_kernels.h"

namespace rlpl {

constexpr int64_t kRmsMaxCols = 16384;
constexpr int kFp8Group = 128;             // columns that share a scale

struct RmsFwdArgs {
    const void* x;             // (rows, cols) dtype
    const void* residual;      // (rows, cols) stream dtype, or NULL
    const void* w;             // (cols) dtype or float32, or NULL (ones)
    void* stream;              // (rows, cols) stream dtype: x + residual, with a residual
    void* y;                   // (rows, cols) dtype, or e4m3
    float* scale;              // (rows, groups) with e4m3
    float* rstd;               // (rows) or NULL
    int64_t rows;
    int32_t cols, groups;
    int32_t w_f32;
    float eps;
};
NormRowKernel pick_rms_fwd(int dtype, int stream_dtype, bool fp8, int64_t cols);

struct RmsBwdArgs {
    const void* dy;            // (rows, cols) dtype
    const void* h;             // (rows, cols) stream dtype
    const void* w;             // (cols) dtype or float32, or NULL (ones)
    const float* rstd;         // (rows)
    const void* dstream;       // (rows, cols) stream dtype, or NULL
    void* dh;                  // (rows, cols) stream dtype, or NULL
    float* part;               // (workgroups, 2, cols): column sums of dy h rstd (the second plane is not used), or NULL
    int64_t rows;
    int32_t cols;
    int32_t w_f32;
};
NormRowKernel pick_rms_bwd(int dtype, int stream_dtype, int64_t cols);

}  // namespace rlpl
