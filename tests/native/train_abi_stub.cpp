// train_abi.cpp with a HIP runtime of this file's own: calls of the device queries can be made to fail, and launches
// are written down instead of made.  Prints "ok <checks> checks".
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstring>
#include <map>

#include "rl_post_loss.h"

static int g_fail_properties = 0, g_fail_attribute = 0, g_fail_function = 0, g_queries = 0;
static int g_launches = 0;
static uint64_t g_lanes = 0;               // the most lanes of a launch

extern "C" {
hipError_t hipGetDevice(int* dev) {
    *dev = 0;
    return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* prop, int) {
    ++g_queries;
    if (g_fail_properties > 0 && g_fail_properties--) return hipErrorUnknown;
    std::memset(prop, 0, sizeof(*prop));
    std::strcpy(prop->gcnArchName, "gfx950:sramecc+:xnack-");
    return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
    if (g_fail_attribute > 0 && g_fail_attribute--) return hipErrorUnknown;
    *v = 256;
    return hipSuccess;
}
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) {
    return g_fail_function > 0 && g_fail_function-- ? hipErrorUnknown : hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
    ++g_launches;
    const uint64_t lanes = uint64_t(grid.x) * grid.y * grid.z * block.x * block.y * block.z;
    if (lanes > g_lanes) g_lanes = lanes;
    return hipSuccess;
}
}

static long g_checks = 0;
#define CHECK(cond)                                                             \
    do {                                                                        \
        ++g_checks;                                                             \
        if (!(cond)) {                                                          \
            std::printf("FAILED line %d: %s\n", __LINE__, #cond);               \
            return 1;                                                           \
        }                                                                       \
    } while (0)

static void* at(uintptr_t p) { return reinterpret_cast<void*>(p); }
static const uintptr_t A = 0x7F0000000000;

static int norm() {
    return layer_norm_fwd(at(A), nullptr, nullptr, 10, 64, RLPL_BF16, RLPL_BF16, 1e-5f, at(A + 4096), nullptr, nullptr,
                          nullptr);
}

// A query that fails is asked again by the next call; one that worked is not asked twice.
static int device_failures() {
    for (int* fail : {&g_fail_properties, &g_fail_attribute, &g_fail_function}) {
        *fail = 1;
        CHECK(norm() == RLPL_ERR_DEVICE && g_launches == 0 && *fail == 0);
    }
    CHECK(norm() == RLPL_OK && g_launches == 1);
    const int asked = g_queries;
    g_fail_properties = g_fail_attribute = g_fail_function = 1;
    CHECK(norm() == RLPL_OK && g_launches == 2 && g_queries == asked);
    return 0;
}

int main() {
    if (device_failures()) return 1;
    std::printf("ok %ld checks\n", g_checks);
    return 0;
}
