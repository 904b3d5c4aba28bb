// Host-side pieces shared by the entry points of train_abi.cpp.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "rl_post_loss.h"

namespace rlpl {

inline bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t up256(size_t b) { return (b + 255) & ~size_t(255); }
inline bool known_dtype(int d) { return d == RLPL_F32 || d == RLPL_F16 || d == RLPL_BF16; }
inline size_t dtype_bytes(int d) { return d == RLPL_F32 ? 4 : 2; }

// One launch on the caller's stream; the sticky error of a failed one is cleared.
template <typename A>
int enqueue(const void* kernel, const A& a, dim3 grid, int threads, hipStream_t stream, size_t dyn_lds = 0) {
    if (!kernel) return RLPL_ERR_DTYPE;
    void* params[] = {const_cast<A*>(&a)};
    if (hipLaunchKernel(kernel, grid, dim3(unsigned(threads)), params, dyn_lds, stream) != hipSuccess) {
        (void)hipGetLastError();
        return RLPL_ERR_LAUNCH;
    }
    return RLPL_OK;
}

}  // namespace rlpl
