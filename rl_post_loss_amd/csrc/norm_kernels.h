// Internal interface between the C ABI layer (train_abi.cpp) and the layer
// norm kernels (norm_kernels.hip).  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace rlpl {

constexpr int64_t kNormMaxCols = 65536;
// Workgroups a launch over rows has at most (the kernels stride over the rest): grids times lanes stay below 2^32.
constexpr int64_t kNormMaxGrid = 1 << 20;
constexpr int kNormThreads = 256;          // workgroups of the kernels that do not hold rows

struct NormFwdArgs {
    const void* x;             // (rows, cols) dtype
    const void* w;             // (cols) weight dtype, or NULL (ones)
    const void* b;             // (cols) weight dtype, or NULL (zeros)
    void* y;                   // (rows, cols) dtype
    float* mean;               // (rows) or NULL
    float* rstd;               // (rows) or NULL
    int64_t rows;
    int32_t cols;
    float eps;
};

// A kernel whose workgroups of `threads` lanes hold rows_per_group rows at a time.
struct NormRowKernel {
    const void* kernel;
    int threads, rows_per_group;
};
NormRowKernel pick_norm_fwd(int dtype, int wdtype, int64_t cols);

constexpr int64_t kNormHeldCols = 16384;   // longest row of the backward kernel that holds rows
constexpr int64_t kNormHeldElements = 1 << 21;   // its workgroups times columns at most,
constexpr int64_t kNormHeldGrid = 1024;          // and its workgroups, which may be one a compute unit
constexpr int64_t kNormHeldLeast = 256;
constexpr int64_t kNormHeldFew = 128;

struct NormBwdArgs {
    const void* dy;            // (rows, cols) dtype
    const void* x;             // (rows, cols) dtype
    const void* w;             // (cols) weight dtype, or NULL (ones)
    const float* mean;         // (rows)
    const float* rstd;         // (rows)
    void* dx;                  // (rows, cols) dtype, or NULL
    float2* row_sums;          // (rows), rows longer than kNormHeldCols: mean over the columns of (dy w, dy w xhat)
    float* part;               // (slabs or workgroups, 2, cols): column sums of dy xhat and dy over their rows, or NULL
    int64_t rows;
    int64_t slab_rows;         // rows per slab
    int32_t cols;
};
NormRowKernel pick_norm_bwd_held(int dtype, int wdtype, int64_t cols);
const void* pick_norm_row_sums(int dtype, int wdtype, int64_t cols);
const void* pick_norm_bwd(int dtype, int wdtype, int64_t cols);

// Sums the slabs' partials in slab order into the weight's and bias's gradients.
struct NormReduceArgs {
    const float* part;
    void* dw;                  // (cols) weight dtype, or NULL
    void* db;                  // (cols) weight dtype, or NULL
    int32_t slabs, cols;
};
constexpr int kNormReduceCols = 32;        // columns per workgroup
constexpr int kNormReduceThreads = 1024;
const void* pick_norm_reduce(int wdtype);

// Columns a workgroup of norm_bwd covers.
inline int64_t norm_col_tile(int dtype) { return 64 * (dtype == 0 ? 4 : 8); }

}  // namespace rlpl
