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

// A forward kernel: `threads` lanes per row (64: four rows per workgroup of
// 256), each holding up to `chunks` vectors of `vec` elements.
struct NormFwdKernel {
    const void* kernel;
    int threads, rows_per_group;
};
NormFwdKernel pick_norm_fwd(int dtype, int wdtype, bool vector, int64_t cols);

struct NormBwdArgs {
    const void* dy;            // (rows, cols) dtype
    const void* x;             // (rows, cols) dtype
    const void* w;             // (cols) weight dtype, or NULL (ones)
    const float* mean;         // (rows)
    const float* rstd;         // (rows)
    void* dx;                  // (rows, cols) dtype, or NULL
    float2* row_sums;          // (rows): mean over the columns of (dy w, dy w xhat)
    float* part;               // (slabs, 2, cols): column sums of dy xhat and dy over a slab's rows, or NULL
    int64_t rows;
    int64_t slab_rows;         // rows per slab
    int32_t cols;
};
const void* pick_norm_row_sums(int dtype, int wdtype, bool vector);
const void* pick_norm_bwd(int dtype, int wdtype, bool vector);

// Sums the slabs' partials in slab order into the weight's and bias's gradients.
struct NormReduceArgs {
    const float* part;
    void* dw;                  // (cols) weight dtype, or NULL
    void* db;                  // (cols) weight dtype, or NULL
    int32_t slabs, cols;
};
constexpr int kNormReduceCols = 32;        // columns per workgroup
const void* pick_norm_reduce(int wdtype);

// Columns a workgroup of the column kernel covers, and how many slabs of rows
// a (rows, cols) problem is split into (shared by the workspace's size and the launch).
inline int64_t norm_col_tile(int dtype, bool vector) { return 64 * (vector ? (dtype == 0 ? 4 : 8) : 1); }

}  // namespace rlpl
