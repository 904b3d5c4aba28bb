// Internal interface between the C ABI layer (train_abi.cpp) and the AdamW
// kernels (adamw_kernels.hip).  Not part of the public ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace rlpl {

constexpr int kAdamThreads = 256;
constexpr int kAdamBlock = 256;            // values of an 8-bit state that share one scale
constexpr int kAdamChunk = 4096;           // elements of one tensor a workgroup updates
constexpr int kAdamWindow = 440;           // tensors one launch covers (their gradients' pointers are kernel arguments)

// One tensor of a plan: pointers into device memory, fixed for the plan's life.
struct AdamTensor {
    void* param;
    void* copy;                // 16-bit copy of the parameter, or NULL
    void* m;                   // first moment: float32 or e4m3
    void* v;                   // second moment: float32, or its root in e4m3
    float* m_scale;            // one per 256 elements (8-bit states)
    float* v_scale;
    int64_t n;
    double weight_decay;
    uint64_t aligned;          // parameter, copy and states allow 16-byte accesses
};

// A plan, in host memory and, byte for byte, in device memory: this header, the
// tensors, then one entry per chunk (the tensor, and the chunk's place in it).
struct AdamChunk {
    uint32_t tensor, place;
};
struct AdamPlan {
    uint64_t magic;
    int64_t count, chunks;
    int32_t param_dtype, copy_dtype, state_bits, pad;
    uint64_t tensors_at, chunks_at, bytes;   // offsets from the plan's start, its size
};
constexpr uint64_t kAdamMagic = 0x726c706c41646d57ull;

struct AdamArgs {
    const AdamTensor* tensors;         // of the whole plan (device memory)
    const AdamChunk* chunks;           // of this launch's window
    const float* grad_scale;           // device scalar the gradients are multiplied by, or NULL
    const float* lr_at;                // device scalars that take the place of lr and of the step t, or NULL
    const int64_t* step_at;
    double lr, correction1;            // lr, 1 - beta1^t
    double log_beta1, log_beta2;       // for a step read on the device
    float root;                        // 1 / sqrt(1 - beta2^t)
    float beta1, beta2, one_minus_beta1, one_minus_beta2, eps;
    uint32_t seed, step;               // of the rounding's random numbers (8-bit states): hashed seed, low word of t
    uint32_t first;                    // the window's first tensor
    int32_t copy_dtype;
    const void* grads[kAdamWindow];
};
static_assert(sizeof(AdamArgs) <= 4096, "kernel arguments");

const void* pick_adamw(int param_dtype, int grad_dtype, int state_bits);

}  // namespace rlpl
