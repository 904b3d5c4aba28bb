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

// The header's bounds are the code's, and every launch of a shape within them has fewer than 2^32 lanes, the joint
// launch of both gradient products among them.
static int cross_entropy_shapes() {
    const int64_t rows[] = {1, 15, 16, 255, 256, 257, 2048, 2049, 8191, 16384, 65536, 1 << 20, (1 << 22) - 1, 1 << 22, 1 << 24};
    const int64_t hiddens[] = {8, 64, 256, 264, 4096, 16128, 16136, 16384, 32768, 65280, 65536};
    const int64_t vocabs[] = {1, 255, 256, 257, 8192, 65535, 65536, 128256, 1 << 20, (1 << 22) - 256, (1 << 22) - 1};
    const auto tiles = [](int64_t v) { return (v + 255) / 256; };
    long taken = 0;
    for (int64_t n : rows)
        for (int64_t h : hiddens)
            for (int64_t v : vocabs) {
                const bool within = tiles(n) * tiles(v) < (1 << 22) && tiles(n) * tiles(h) < (1 << 22);
                for (int grads = 0; grads < 2; ++grads) {
                    const size_t bytes = linear_cross_entropy_workspace_bytes(n, h, v, grads);
                    CHECK((bytes > 0) == within);
                    if (!within) continue;
                    if (grads) {           // what the header says that it holds: dz, planes, column sums
                        CHECK(bytes >= size_t(n) * 2 * size_t(v < 8192 ? v : 8192) + size_t(n) * 4 * size_t(h));
                        CHECK(bytes >= size_t(tiles(n)) * size_t(v) * 4);
                    }
                    g_lanes = 0;
                    const auto targets = static_cast<int64_t*>(at(A));
                    const auto loss = static_cast<float*>(at(A));
                    CHECK((grads ? linear_cross_entropy(at(A), at(A), at(A), targets, n, h, v, RLPL_BF16, -100, 0.0f, 0, loss,
                                                        at(A), at(A), at(A), RLPL_BF16, 0, at(A), bytes, nullptr)
                                 : linear_cross_entropy_fwd(at(A), at(A), at(A), targets, n, h, v, RLPL_BF16, -100, 0.0f, 0,
                                                            loss, at(A), bytes, nullptr)) == RLPL_OK);
                    CHECK(g_lanes > 0 && g_lanes < (uint64_t(1) << 32));
                    ++taken;
                }
            }
    CHECK(taken > 1000);
    CHECK(linear_cross_entropy_workspace_bytes(int64_t(1) << 24, 16384, 100, 1) == 0);   // 2^22 tiles of rows by hidden values
    CHECK(linear_cross_entropy_workspace_bytes(int64_t(1) << 24, 16128, 100, 1) > 0);
    return 0;
}

int main() {
    if (device_failures() || cross_entropy_shapes()) return 1;
    std::printf("ok %ld checks\n", g_checks);
    return 0;
}
