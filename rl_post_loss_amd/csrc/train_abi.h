// Host-side pieces shared by the entry points of train_abi.cpp and score_abi.cpp.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "rl_post_loss.h"

namespace rlpl {

inline bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t up256(size_t b) { return (b + 255) & ~size_t(255); }
inline bool known_dtype(int d) { return d == RLPL_F32 || d == RLPL_F16 || d == RLPL_BF16; }
inline size_t dtype_bytes(int d) { return d == RLPL_F32 ? 4 : 2; }

// Whether device dev is a gfx950 with a known number of compute units.
inline bool is_gfx950(int dev) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess || std::strncmp(prop.gcnArchName, "gfx950", 6) != 0) return false;
    int cus = 0;
    return hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && cus >= 1;
}

// Devices that SET_UP(dev) has set up, each once.
template <bool (*SET_UP)(int)>
class Devices {
public:
    // The current device, set up.  A failure is not kept: the next call tries again.
    int current() {
        int dev = -1;
        if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMost) {
            (void)hipGetLastError();
            return RLPL_ERR_DEVICE;
        }
        One& d = all_[dev];
        if (d.ready.load(std::memory_order_acquire)) return RLPL_OK;
        const std::lock_guard<std::mutex> hold(d.lock);
        if (d.ready.load(std::memory_order_relaxed)) return RLPL_OK;
        if (!SET_UP(dev)) {
            (void)hipGetLastError();
            return RLPL_ERR_DEVICE;
        }
        d.ready.store(true, std::memory_order_release);
        return RLPL_OK;
    }

private:
    static constexpr int kMost = 64;
    struct One {
        std::mutex lock;
        std::atomic<bool> ready{false};
    };
    One all_[kMost];
};

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
