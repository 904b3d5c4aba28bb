// score_abi.cpp and train_abi.cpp (its RMS norm and gradient norm) with a HIP runtime of this file's own: launches are
// looked at instead of made.  Extreme and rejected arguments of every entry point; of those taken, that the launches
// cover their work, stay within the workspace and the launch limits.  Prints "ok <checks> checks".
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <vector>

#include "fp8_kernels.h"
#include "grad_kernels.h"
#include "norm_kernels.h"
#include "rl_post_loss.h"
#include "rms_kernels.h"
#include "token_kernels.h"

using namespace rlpl;

struct Launch {
    const void* kernel;
    uint64_t groups, threads;
    size_t lds;
    const void* args;                      // during the call only
};
static std::function<void(const Launch&)> g_look;
static int g_launches = 0;
static bool g_within = true;               // every launch has lanes, fewer than 2^32

extern "C" {
hipError_t hipGetDevice(int* dev) {
    *dev = 0;
    return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* prop, int) {
    std::memset(prop, 0, sizeof(*prop));
    std::strcpy(prop->gcnArchName, "gfx950:sramecc+:xnack-");
    return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
    *v = 256;
    return hipSuccess;
}
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) { return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipLaunchKernel(const void* kernel, dim3 grid, dim3 block, void** args, size_t lds, hipStream_t) {
    const Launch l{kernel, uint64_t(grid.x) * grid.y * grid.z, block.x, lds, args[0]};
    const uint64_t lanes = l.groups * l.threads;
    g_within = g_within && lanes > 0 && lanes < (uint64_t(1) << 32) && l.threads <= 1024 && l.lds <= 160 * 1024;
    if (g_look) g_look(l);
    ++g_launches;
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
template <typename T>
static T* as(uintptr_t p) { return reinterpret_cast<T*>(p); }
static uintptr_t address(const void* p) { return reinterpret_cast<uintptr_t>(p); }
static const uintptr_t A = 0x7F0000000000;

static int token_logprobs() {
    const int64_t rows[] = {INT64_MIN, -1, 0, 1, 2, 7, 100, 1023, 1024, 1025, 100000, (int64_t(1) << 31) - 1, int64_t(1) << 31, INT64_MAX};
    const int64_t vocabs[] = {INT64_MIN, 0, 1, 3, 64, 2048, 2049, 4096, 4097, 8192, 50021, 131072, 1000003, int64_t(1) << 22,
                              (int64_t(1) << 22) + 1, (int64_t(1) << 31) - 65536, (int64_t(1) << 31) - 65535, INT64_MAX};
    const int64_t tops[] = {INT64_MIN, -1, 0, 1, 3, 20, 63, 64, 65, INT64_MAX};
    long taken = 0;
    for (int64_t r : rows)
        for (int64_t v : vocabs) {
            for (int64_t k : tops) {
                const bool ok = r >= 1 && r < (int64_t(1) << 31) && v >= 1 && v <= (k > 0 ? int64_t(1) << 22 : (int64_t(1) << 31) - 65536) &&
                                k >= 0 && k <= 64 && k <= v;
                const size_t bytes = token_logprobs_workspace_bytes(r, v, k);
                CHECK((bytes > 0) == ok && bytes % 256 == 0);
                for (int dt = 0; dt < 3; ++dt) {
                    const int64_t vec = dt == RLPL_F32 ? 4 : 8;
                    std::vector<TokenFwdArgs> seen;
                    g_look = [&](const Launch& l) { seen.push_back(*static_cast<const TokenFwdArgs*>(l.args)); };
                    const auto call = [&](size_t have) {
                        return token_logprobs_fwd(at(A), as<int64_t>(A), nullptr, r, v, r > 0 ? r : 1, 0, v > 0 && v < INT64_MAX / 4 ? 0 : 1, dt, 1.0f, k,
                                                  as<float>(A), as<float>(A), nullptr, as<float>(A), as<int64_t>(A), at(A), have, nullptr);
                    };
                    if (!ok) {
                        CHECK(call(SIZE_MAX) == RLPL_ERR_SHAPE && seen.empty());
                        continue;
                    }
                    CHECK(call(bytes - 1) == RLPL_ERR_WORKSPACE && seen.empty());
                    CHECK(call(bytes) == RLPL_OK);
                    const TokenFwdArgs& a = seen[0];
                    CHECK(seen.size() == (a.pieces > 1 ? 2u : 1u) && a.pieces >= 1 && a.pieces <= kTokenMaxPieces);
                    CHECK(a.pieces == 1 || v > kTokenShort);
                    const int64_t vectors = v / vec;
                    CHECK(a.pieces * a.piece_vectors >= vectors && (a.pieces - 1) * a.piece_vectors <= INT32_MAX);
                    if (k > 0) {
                        CHECK(a.pieces * k <= kTokenMaxKeys);
                        CHECK(a.piece_vectors <= int64_t(kTokenBlocks) * 32 / vec * kTokenThreads);
                    }
                    if (a.pieces > 1) {
                        CHECK(address(a.part) == A && address(a.part_top) >= A + size_t(r) * size_t(a.pieces) * sizeof(TokenPart));
                        CHECK(address(a.part_top) + size_t(r) * size_t(a.pieces) * size_t(k) * 8 <= A + bytes);
                    }
                    ++taken;
                }
            }
            std::vector<TokenBwdArgs> seen;
            std::vector<uint64_t> groups;
            g_look = [&](const Launch& l) {
                seen.push_back(*static_cast<const TokenBwdArgs*>(l.args));
                groups.push_back(l.groups);
            };
            const bool ok = r >= 1 && r < (int64_t(1) << 31) && v >= 1 && v <= (int64_t(1) << 31) - 65536;
            CHECK(token_logprobs_bwd(at(A), as<int64_t>(A), nullptr, as<float>(A), as<float>(A), as<float>(A), as<float>(A), r, v, 1, 0, 0,
                                     RLPL_BF16, 1.0f, at(A), nullptr) == (ok ? RLPL_OK : RLPL_ERR_SHAPE));
            CHECK(seen.size() == (ok ? 1u : 0u));
            if (ok) {
                CHECK(seen[0].pieces * seen[0].piece_vectors >= v / 8);
                CHECK((seen[0].pieces - 1) * seen[0].piece_vectors <= INT32_MAX);
            }
        }
    g_look = nullptr;
    CHECK(taken > 1000);
    // strides
    const int64_t big = int64_t(1) << 61;
    const struct { int64_t rows, inner, group, row; bool ok; } strides[] = {
        {4, 4, 0, 100, true}, {4, 2, 1000, 100, true}, {4, 0, 0, 100, false}, {4, 5, 0, 100, false}, {4, 4, -1, 100, false}, {4, 4, 0, -1, false},
        {2, 2, 0, big, true}, {3, 3, 0, big, false}, {3, 1, big, 0, false}, {1, 1, INT64_MAX, INT64_MAX, true},
        {(int64_t(1) << 31) - 1, 1, INT64_MAX, INT64_MAX, false}};
    for (const auto& s : strides) {
        const size_t bytes = token_logprobs_workspace_bytes(s.rows, 100, 0);
        CHECK(token_logprobs_fwd(at(A), as<int64_t>(A), nullptr, s.rows, 100, s.inner, s.group, s.row, RLPL_BF16, 1.0f, 0, as<float>(A),
                                 as<float>(A), nullptr, nullptr, nullptr, at(A), bytes, nullptr) == (s.ok ? RLPL_OK : RLPL_ERR_SHAPE));
        CHECK(token_logprobs_bwd(at(A), as<int64_t>(A), nullptr, as<float>(A), nullptr, nullptr, nullptr, s.rows, 100, s.inner, s.group, s.row,
                                 RLPL_BF16, 1.0f, at(A), nullptr) == (s.ok ? RLPL_OK : RLPL_ERR_SHAPE));
    }
    const float temperatures[] = {0.0f, -0.0f, -1.0f, INFINITY, NAN, 1e-40f};
    for (float t : temperatures)
        CHECK(token_logprobs_fwd(at(A), as<int64_t>(A), nullptr, 1, 100, 1, 0, 0, RLPL_BF16, t, 0, as<float>(A), as<float>(A), nullptr, nullptr,
                                 nullptr, at(A), 256, nullptr) == RLPL_ERR_PARAM);
    return 0;
}

static int fp8() {
    const int64_t ns[] = {INT64_MIN, 0, 1, 16, 17, 64, 65, 333, 2048, 4096, 65536, 1 << 20, (1 << 20) + 1, INT64_MAX};
    const int64_t hs[] = {INT64_MIN, 0, 8, 16, 24, 128, 2048, 4096, 8208, 65536, 65552, INT64_MAX};
    const int64_t vs[] = {INT64_MIN, 0, 1, 64, 512, 5003, 20000, 128256, 1 << 20, (1 << 22) - 1, 1 << 22, INT64_MAX};
    long taken = 0, kinds[kFp8Kinds] = {};
    for (int64_t n : ns)
        for (int64_t h : hs)
            for (int64_t v : vs) {
                const bool limits = n >= 1 && n <= (1 << 20) && h >= 16 && h <= 65536 && h % 16 == 0 && v >= 1 && v < (1 << 22);
                const bool ok = limits && (n + 63) / 64 * ((v + 63) / 64) < (int64_t(1) << 24);
                const size_t bytes = fp8_linear_workspace_bytes(n, h, v);
                CHECK((bytes > 0) == ok && bytes % 256 == 0);
                for (int dt = 0; dt < 3; ++dt) {
                    std::vector<Launch> seen;
                    Fp8LinearArgs last{};
                    TurnArgs turned{};
                    g_look = [&](const Launch& l) {
                        seen.push_back(l);
                        if (l.kernel == turn_kernel()) turned = *static_cast<const TurnArgs*>(l.args);
                        else last = *static_cast<const Fp8LinearArgs*>(l.args);
                    };
                    const auto call = [&](size_t have) {
                        return fp8_linear(at(A), as<float>(A + 4), at(A), as<float>(A), nullptr, n, h, v, dt, at(A), at(A + 256), have, nullptr);
                    };
                    if (!ok) {
                        CHECK(call(SIZE_MAX) == RLPL_ERR_SHAPE && seen.empty());
                        continue;
                    }
                    CHECK(call(bytes - 1) == RLPL_ERR_WORKSPACE && seen.empty());
                    CHECK(call(bytes) == RLPL_OK && !seen.empty());
                    const Launch& l = seen.back();
                    ++taken;
                    CHECK(last.n == n && last.K == h && last.vocab == v && last.blocks == (h + 127) / 128);
                    if (n <= kFp8FewRows) {
                        CHECK(seen.size() == 1 && last.x_scale == as<float>(A + 4));
                        CHECK(l.groups == uint64_t((v + 15) / 16) || l.groups == uint64_t((v + 31) / 32) || l.groups == uint64_t((v + 63) / 64));
                        continue;
                    }
                    int kind = -1;
                    for (int i = 0; i < kFp8Kinds; ++i)
                        if (l.kernel == pick_fp8_tile(dt, i)) kind = i;
                    CHECK(kind >= 0);
                    ++kinds[kind];
                    const Fp8TileShape& s = kFp8Shapes[kind];
                    CHECK(l.threads == uint64_t(s.threads) && l.lds == size_t(s.lds) && l.groups == uint64_t(last.tiles_v) * last.tiles_t);
                    CHECK(int64_t(last.tiles_v) * s.vocab >= v && int64_t(last.tiles_t) * s.tokens >= n);
                    CHECK((seen.size() == 2) == (kind == kFp8Large));
                    if (kind == kFp8Large) {
                        CHECK(turned.from == as<float>(A + 4) && last.x_scale == turned.to && address(turned.to) == A + 256);
                        CHECK(turned.ld >= n && turned.ld == last.scale_ld && turned.rows == n && turned.cols == last.blocks);
                        CHECK(size_t(turned.ld) * size_t(turned.cols) * 4 <= bytes);
                        CHECK(seen[0].groups * kTurnRows * kTurnCols >= uint64_t(n) * uint64_t(last.blocks));
                    }
                }
            }
    g_look = nullptr;
    CHECK(taken > 500);
    for (long k : kinds) CHECK(k > 0);
    const int64_t dims[] = {INT64_MIN, -1, 0, 1, 100, 4096, (int64_t(1) << 31) - 65536, (int64_t(1) << 31) - 1, INT64_MAX};
    for (int64_t r : dims)
        for (int64_t c : dims)
            for (int64_t ld : {INT64_MIN, int64_t(0), int64_t(4096), int64_t(1) << 31, INT64_MAX}) {
                const bool ok = r >= 1 && r < (int64_t(1) << 31) && c >= 1 && c <= (int64_t(1) << 31) - 65536 && ld >= 0 &&
                                __int128(r - 1) * ld < (int64_t(1) << 62);
                for (int block : {1, 128})
                    CHECK(rlpl_fp8_quantize(at(A), r, c, ld, RLPL_BF16, block, at(A), as<float>(A), nullptr) == (ok ? RLPL_OK : RLPL_ERR_SHAPE));
            }
    CHECK(rlpl_fp8_quantize(at(A), 1, 1, 1, RLPL_BF16, 64, at(A), as<float>(A), nullptr) == RLPL_ERR_PARAM);
    return 0;
}

static int rms() {
    const int64_t rows[] = {INT64_MIN, -1, 0, 1, 3, 1000, 100000, (int64_t(1) << 31) - 1, int64_t(1) << 31, INT64_MAX};
    const int64_t cols[] = {-1, 0, 1, 7, 8, 9, 128, 129, 512, 513, 1024, 2048, 4001, 8192, 16384, 16385, INT64_MAX};
    for (int64_t r : rows)
        for (int64_t c : cols) {
            const bool ok = r >= 1 && r < (int64_t(1) << 31) && c >= 1 && c <= 16384;
            const size_t bytes = rms_norm_workspace_bytes(r, c);
            CHECK((bytes > 0) == ok);
            const int want = ok ? RLPL_OK : RLPL_ERR_SHAPE;
            for (int dt = 0; dt < 3; ++dt) {
                CHECK(rms_norm_fwd(at(A), nullptr, nullptr, r, c, dt, 0, dt, 1e-6f, at(A), nullptr, nullptr, nullptr) == want);
                CHECK(rms_norm_fp8(at(A), at(A), at(A), r, c, dt, dt, 0, 1e-6f, at(A), as<float>(A), as<float>(A), at(A), nullptr) == want);
                uint64_t groups = 0;
                RmsBwdArgs a{};
                g_look = [&](const Launch& l) {
                    if (!groups) {
                        groups = l.groups;
                        a = *static_cast<const RmsBwdArgs*>(l.args);
                    }
                };
                const auto call = [&](size_t have) {
                    return rms_norm_bwd(at(A), at(A), at(A), as<float>(A), nullptr, r, c, dt, dt, 0, at(A), at(A), at(A), have, nullptr);
                };
                if (ok) CHECK(call(bytes - 1) == RLPL_ERR_WORKSPACE);
                CHECK(call(bytes) == want);
                if (ok) CHECK(address(a.part) == A && groups * 2 * uint64_t(c) * 4 <= bytes);
                g_look = nullptr;
            }
        }
    return 0;
}

// Every chunk of every tensor in one launch, the partial sums side by side in the workspace.
static int gradients() {
    const std::vector<std::vector<int64_t>> lists = {
        {0}, {1}, {0, 0}, {4095}, {4096}, {4097}, {65536}, {65537}, {0, 0, 5, 0}, {1, 2, 3, 100000}, std::vector<int64_t>(189, 3),
        std::vector<int64_t>(190, 3), std::vector<int64_t>(191, 3), std::vector<int64_t>(380, 5000), std::vector<int64_t>(2000, 17),
        {int64_t(1) << 40, 1, int64_t(1) << 40}, std::vector<int64_t>(9, int64_t(1) << 40)};
    for (const auto& sizes : lists) {
        const int64_t count = int64_t(sizes.size());
        std::vector<void*> p;
        std::vector<int32_t> types;
        for (int64_t i = 0; i < count; ++i) {
            p.push_back(sizes[size_t(i)] ? at(A + (uintptr_t(i) << 43)) : nullptr);
            types.push_back(int32_t(i % 3));
        }
        const size_t bytes = rlpl_grad_norm_workspace_bytes(sizes.data(), count);
        CHECK(bytes > 0 && bytes % 256 == 0);
        std::vector<GradList> windows;
        std::vector<std::pair<uintptr_t, uint64_t>> parts;
        GradFinish finish{};
        bool finished = false, alone = false;
        g_look = [&](const Launch& l) {
            if (l.kernel == grad_finish_kernel()) {
                finish = *static_cast<const GradFinish*>(l.args);
                finished = true;
                return;
            }
            const auto* a = static_cast<const GradNormArgs*>(l.args);
            alone = alone || l.kernel == pick_grad_alone(false);
            windows.push_back(a->list);
            parts.emplace_back(address(a->part), l.groups);
        };
        const auto call = [&](size_t have) {
            return rlpl_grad_norm(p.data(), sizes.data(), types.data(), count, RLPL_NORM_2, nullptr, 1.0f, 1e-6f, as<float>(A), as<float>(A),
                                  at(A), have, nullptr);
        };
        CHECK(call(bytes - 1) == RLPL_ERR_WORKSPACE && windows.empty());
        CHECK(call(bytes) == RLPL_OK);
        CHECK(finished != alone && (!alone || windows.size() == 1));
        const auto covered = [&]() {
            size_t next = 0;               // the tensor after those seen
            for (const GradList& l : windows) {
                CHECK(l.count >= 1 && l.count <= uint32_t(kGradWindow) && l.first[0] == 0);
                for (uint32_t j = 0; j < l.count; ++j) {
                    while (next < sizes.size() && sizes[next] == 0) ++next;
                    CHECK(next < sizes.size() && l.p[j] == p[next] && l.n[j] == sizes[next] * 4 + types[next]);
                    CHECK(int64_t(l.first[j + 1]) - int64_t(l.first[j]) == (sizes[next] + kGradChunk - 1) / kGradChunk);
                    ++next;
                }
            }
            while (next < sizes.size() && sizes[next] == 0) ++next;
            CHECK(next == sizes.size());
            return 0;
        };
        if (covered()) return 1;
        if (finished) {
            uintptr_t end = A;
            for (const auto& part : parts) {
                CHECK(part.first == end && part.second <= uint64_t(kGradGrid));
                end += part.second * 8;
            }
            CHECK(end <= A + bytes && finish.part == as<double>(A) && uintptr_t(finish.parts) * 8 == end - A);
        }
        windows.clear();
        g_look = [&](const Launch& l) { windows.push_back(static_cast<const GradScaleArgs*>(l.args)->list); };
        CHECK(rlpl_grad_scale(p.data(), sizes.data(), types.data(), count, as<float>(A), nullptr) == RLPL_OK);
        if (covered()) return 1;
        g_look = nullptr;
    }
    const int64_t bad[][2] = {{-1, 5}, {(int64_t(1) << 40) + 1, 1}, {INT64_MAX, INT64_MAX}, {INT64_MIN, 0}};
    void* p[2] = {at(A), at(A + (uintptr_t(1) << 42))};
    const int32_t types[2] = {0, 0};
    for (const auto& s : bad) {
        CHECK(rlpl_grad_norm_workspace_bytes(s, 2) == 0);
        CHECK(rlpl_grad_norm(p, s, types, 2, RLPL_NORM_2, nullptr, 1.0f, 0.0f, as<float>(A), nullptr, at(A), SIZE_MAX, nullptr) == RLPL_ERR_SHAPE);
        CHECK(rlpl_grad_scale(p, s, types, 2, as<float>(A), nullptr) == RLPL_ERR_SHAPE);
    }
    const int64_t many = 5;
    CHECK(rlpl_grad_norm_workspace_bytes(&many, INT64_MAX) == 0 && rlpl_grad_norm_workspace_bytes(&many, -1) == 0);
    const int64_t two[2] = {100, 100};
    void* over[2] = {at(A), at(A + 396)};
    CHECK(rlpl_grad_scale(over, two, types, 2, as<float>(A), nullptr) == RLPL_ERR_PARAM);
    void* side[2] = {at(A + 400), at(A)};
    CHECK(rlpl_grad_scale(side, two, types, 2, as<float>(A), nullptr) == RLPL_OK);
    return 0;
}

int main() {
    if (token_logprobs() || fp8() || rms() || gradients()) return 1;
    CHECK(g_within && g_launches > 1000);
    std::printf("ok %ld checks\n", g_checks);
    return 0;
}
