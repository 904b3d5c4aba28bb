// Drives the host side of train_abi.cpp under the sanitizers, with no GPU visible: rejected and extreme arguments of
// every entry point, valid ones up to the device lookup, and AdamW plans built in buffers of their exact size.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "adamw_kernels.h"
#include "rl_post_loss.h"

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

static int cross_entropy() {
    const int64_t ns[] = {INT64_MIN, -1, 0, 1, 17, 2048, 2049, 65536, 1 << 24, (1 << 24) + 1, INT64_MAX};
    const int64_t hs[] = {-8, 0, 7, 8, 64, 4096, 65536, 65544, INT64_MAX};
    const int64_t vs[] = {-1, 0, 1, 255, 256, 8192, 128256, (1 << 22) - 1, 1 << 22, INT64_MAX};
    for (int64_t n : ns)
        for (int64_t h : hs)
            for (int64_t v : vs)
                for (int grads = 0; grads < 2; ++grads) {
                    const size_t bytes = linear_cross_entropy_workspace_bytes(n, h, v, grads);
                    auto call = [&](size_t have) {
                        return grads ? linear_cross_entropy(at(A), at(A), at(A), static_cast<int64_t*>(at(A)), n, h, v, 2, -100,
                                                            0.0f, 0, static_cast<float*>(at(A)), at(A), at(A), at(A), 2, 0,
                                                            at(A), have, nullptr)
                                     : linear_cross_entropy_fwd(at(A), at(A), nullptr, static_cast<int64_t*>(at(A)), n, h, v, 1,
                                                                INT64_MIN, 1.0f, 1, static_cast<float*>(at(A)), at(A), have,
                                                                nullptr);
                    };
                    if (bytes == 0) {
                        CHECK(call(SIZE_MAX) == RLPL_ERR_SHAPE);
                        continue;
                    }
                    CHECK(bytes % 256 == 0);
                    CHECK(call(bytes - 1) == RLPL_ERR_WORKSPACE);
                    CHECK(call(bytes) == RLPL_ERR_DEVICE);
                }
    return 0;
}

static int layer_norm() {
    const int64_t rows[] = {INT64_MIN, -1, 0, 1, 3, 1000, (int64_t(1) << 31) - 1, int64_t(1) << 31, INT64_MAX};
    const int64_t cols[] = {-1, 0, 1, 7, 8, 2048, 8192, 16384, 16385, 65536, 65537, INT64_MAX};
    for (int64_t r : rows)
        for (int64_t c : cols) {
            const size_t bytes = layer_norm_workspace_bytes(r, c);
            const bool ok = r >= 1 && r < (int64_t(1) << 31) && c >= 1 && c <= 65536;
            CHECK((bytes > 0) == ok);
            const int want = ok ? RLPL_ERR_DEVICE : RLPL_ERR_SHAPE;
            CHECK(layer_norm_fwd(at(A), nullptr, nullptr, r, c, 0, 0, 1e-5f, at(A), nullptr, nullptr, nullptr) == want);
            CHECK(layer_norm_bwd(at(A), at(A), at(A), static_cast<float*>(at(A)), static_cast<float*>(at(A)), r, c, 2, 0, at(A),
                                 at(A), at(A), at(A), bytes, nullptr) == want);
            if (ok)
                CHECK(layer_norm_bwd(at(A), at(A), at(A), static_cast<float*>(at(A)), static_cast<float*>(at(A)), r, c, 2, 0,
                                     at(A), at(A), at(A), at(A), bytes - 1, nullptr) == RLPL_ERR_WORKSPACE);
        }
    return 0;
}

static int adamw() {
    const std::vector<std::vector<int64_t>> lists = {
        {0}, {1}, {4095}, {4096}, {4097}, {0, 0, 5, 0}, {1, 2, 3, 100000}, std::vector<int64_t>(439, 3),
        std::vector<int64_t>(440, 3), std::vector<int64_t>(441, 5000), std::vector<int64_t>(2000, 17)};
    for (const auto& sizes : lists)
        for (int bits : {32, 8}) {
            const int64_t count = int64_t(sizes.size());
            // every list at its exact length
            int64_t* s = static_cast<int64_t*>(std::malloc(size_t(count) * 8));
            void** p = static_cast<void**>(std::malloc(size_t(count) * sizeof(void*)));
            float** f = static_cast<float**>(std::malloc(size_t(count) * sizeof(float*)));
            double* d = static_cast<double*>(std::malloc(size_t(count) * 8));
            for (int64_t i = 0; i < count; ++i) {
                s[i] = sizes[size_t(i)];
                p[i] = sizes[size_t(i)] ? at(A + 4096 * uintptr_t(i)) : nullptr;
                f[i] = static_cast<float*>(p[i]);
                d[i] = 0.01 * double(i % 3);
            }
            const size_t bytes = rlpl_adamw_plan_bytes(s, count);
            CHECK(bytes > 0);
            void* plan = std::malloc(bytes);
            CHECK(rlpl_adamw_plan_build(plan, bytes - 1, s, count, p, 0, nullptr, 0, p, p, f, f, bits, d) == RLPL_ERR_WORKSPACE);
            CHECK(rlpl_adamw_plan_build(plan, bytes, s, count, p, 0, p, 2, p, p, f, f, bits, d) == RLPL_OK);
            const auto* h = static_cast<const rlpl::AdamPlan*>(plan);
            const auto* t = reinterpret_cast<const rlpl::AdamTensor*>(static_cast<const char*>(plan) + h->tensors_at);
            const auto* c = reinterpret_cast<const rlpl::AdamChunk*>(static_cast<const char*>(plan) + h->chunks_at);
            CHECK(h->bytes == bytes && h->count == count);
            int64_t k = 0;                 // the chunks are the tensors' in order, each within its tensor
            for (int64_t i = 0; i < count; ++i)
                for (int64_t o = 0; o < sizes[size_t(i)]; o += rlpl::kAdamChunk, ++k)
                    CHECK(c[k].tensor == uint32_t(i) && int64_t(c[k].place) * rlpl::kAdamChunk == o && t[i].n == sizes[size_t(i)]);
            CHECK(k == h->chunks);
            CHECK(rlpl_adamw_step(plan, at(A), p, 2, 1e-3, nullptr, 0.9, 0.999, 1e-8, 1, nullptr, nullptr, 0, nullptr) ==
                  RLPL_ERR_DEVICE);
            std::free(plan);
            std::free(s);
            std::free(p);
            std::free(f);
            std::free(d);
        }
    const int64_t bad[][2] = {{-1, 5}, {(int64_t(1) << 40) + 1, 1}, {INT64_MAX, INT64_MAX}, {INT64_MIN, 0}};
    for (const auto& s : bad) CHECK(rlpl_adamw_plan_bytes(s, 2) == 0);
    const int64_t many = 5;
    CHECK(rlpl_adamw_plan_bytes(&many, INT64_MAX) == 0 && rlpl_adamw_plan_bytes(&many, -1) == 0);
    return 0;
}

int main() {
    if (cross_entropy() || layer_norm() || adamw()) return 1;
    std::printf("ok %ld checks\n", g_checks);
    return 0;
}
