// Internal interface between the C ABI layer (train_abi.cpp) and the kernels
// of the gradient norm and of scaling gradients (grad_kernels.hip).  Not part
// of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace rlpl {

constexpr int kGradThreads = 256;
constexpr int kGradAloneThreads = 1024;
constexpr int kGradChunk = 4096;           // elements of one tensor
constexpr int kGradWindow = 190;           // tensors one launch covers
constexpr int kGradGrid = 2048;            // workgroups of a launch at most: eight a compute unit
constexpr int64_t kGradAloneChunks = 16;   // a list of so few chunks is one workgroup's

// The tensors of a launch.
struct GradList {
    void* p[kGradWindow];
    int64_t n[kGradWindow];                // elements, times 4, plus the type
    uint32_t first[kGradWindow + 1];       // each tensor's first chunk; all chunks
    uint32_t count;
};

struct GradFinish {
    const double* part;                    // the launches' partial sums
    float* norm;
    float* scale;                          // or NULL
    const float* grad_scale;               // what the gradients are multiplied by, or NULL (1)
    float max_norm, eps;
    int32_t parts, inf;
};
struct GradNormArgs {
    GradList list;
    double* part;                          // this launch's, one a workgroup
    GradFinish finish;                     // of the launch of one workgroup
};
struct GradScaleArgs {
    GradList list;
    const float* scale;
};
static_assert(sizeof(GradNormArgs) <= 4096 && sizeof(GradScaleArgs) <= 4096, "kernel arguments");

const void* pick_grad_norm(bool inf);      // partial sums
const void* pick_grad_alone(bool inf);     // one workgroup, with the results
const void* grad_finish_kernel();
const void* grad_scale_kernel();

}  // namespace rlpl
