// Layer norm on gfx950: forward, backward, and the reduction of the weight's
// and bias's gradients.
//
//   y = (x - mean) rstd w + b,   mean and var over a row's columns, rstd = 1 / sqrt(var + eps)
//   xhat = (x - mean) rstd,  g = dy w
//   dx = rstd (g - avg(g) - xhat avg(g xhat)),   dw = sum_rows dy xhat,   db = sum_rows dy
//
// All of it is bound by memory traffic: the forward reads x and writes y once
// (a row is held in registers between the mean, the squared deviations and
// the output, so that the variance is a true second pass without a second
// read).  Statistics and sums are float32; each output is rounded once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "loss_kernels.h"
#include "norm_kernels.h"
#include "row_io.h"

namespace rlpl {

namespace {

// The sum over a row's THREADS lanes, in every one of them (lane tree, then
// wavefronts in order).  red: THREADS / 64 floats of LDS (unused for one wavefront).
template <int THREADS>
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = wave_sum(v);
    if constexpr (THREADS == 64) return v;
    __syncthreads();                       // red may still be read by a previous sum
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = red[0];
#pragma unroll
    for (int i = 1; i < THREADS / 64; ++i) t += red[i];
    return t;
}

template <int VEC, typename TW>
__device__ __forceinline__ void load_affine(const TW* p, int col, float (&v)[VEC], float none) {
    if (p) {
        load_row<VEC>(p + col, v);
    } else {
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = none;
    }
}

template <typename T, typename TW, int VEC, int THREADS, int NC>
__global__ void __launch_bounds__(THREADS < 256 ? 256 : THREADS) norm_fwd(const NormFwdArgs a) {
    __shared__ float red[THREADS / 64];
    constexpr int kRows = THREADS == 64 ? 4 : 1;
    const int lane = threadIdx.x & (THREADS - 1);
    const float inv = 1.0f / float(a.cols);
    // a row a wavefront (four a workgroup), or a row a workgroup
    for (int64_t row = int64_t(blockIdx.x) * kRows + (THREADS == 64 ? threadIdx.x >> 6 : 0); row < a.rows;
         row += int64_t(gridDim.x) * kRows) {
        const T* x = static_cast<const T*>(a.x) + row * a.cols;
        float v[NC][VEC];
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = (c * THREADS + lane) * VEC;
            if (col < a.cols) {
                load_row<VEC>(x + col, v[c]);
            } else {
#pragma unroll
                for (int k = 0; k < VEC; ++k) v[c][k] = 0.0f;
            }
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int k = 0; k < VEC; ++k) s += v[c][k];
        const float mean = row_sum<THREADS>(s, red) * inv;
        float q = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const bool in = (c * THREADS + lane) * VEC < a.cols;
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                v[c][k] -= mean;
                q += in ? v[c][k] * v[c][k] : 0.0f;
            }
        }
        const float var = row_sum<THREADS>(q, red) * inv;
        const float rstd = 1.0f / sqrtf(var + a.eps);
        if (lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        T* y = static_cast<T*>(a.y) + row * a.cols;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = (c * THREADS + lane) * VEC;
            if (col >= a.cols) continue;
            float w[VEC], b[VEC];
            load_affine<VEC>(static_cast<const TW*>(a.w), col, w, 1.0f);
            load_affine<VEC>(static_cast<const TW*>(a.b), col, b, 0.0f);
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[c][k] = fmaf(v[c][k] * rstd, w[k], b[k]);
            store_row<VEC>(y + col, v[c]);
        }
    }
}

// Per row, the averages over its columns of g = dy w and of g xhat: one wavefront a row.
template <typename T, typename TW, int VEC>
__global__ void __launch_bounds__(kNormThreads) norm_row_sums(const NormBwdArgs a) {
    const int lane = threadIdx.x & 63;
    const float inv = 1.0f / float(a.cols);
    for (int64_t row = int64_t(blockIdx.x) * (kNormThreads / 64) + (threadIdx.x >> 6); row < a.rows;
         row += int64_t(gridDim.x) * (kNormThreads / 64)) {
        const T* x = static_cast<const T*>(a.x) + row * a.cols;
        const T* dy = static_cast<const T*>(a.dy) + row * a.cols;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s = 0.0f, t = 0.0f;
        for (int col = lane * VEC; col < a.cols; col += 64 * VEC) {
            float xv[VEC], gv[VEC], w[VEC];
            load_row<VEC>(x + col, xv);
            load_row<VEC>(dy + col, gv);
            load_affine<VEC>(static_cast<const TW*>(a.w), col, w, 1.0f);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float g = gv[k] * w[k];
                s += g;
                t += g * ((xv[k] - mean) * rstd);
            }
        }
        s = wave_sum(s);
        t = wave_sum(t);
        if (lane == 0) a.row_sums[row] = make_float2(s * inv, t * inv);
    }
}

// The input's gradient and a slab's column sums: a workgroup takes 64 * VEC
// columns of a slab's rows, its four wavefronts every fourth row each.
template <typename T, typename TW, int VEC>
__global__ void __launch_bounds__(kNormThreads) norm_bwd(const NormBwdArgs a) {
    __shared__ float sums[2][3][64 * VEC];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = (int(blockIdx.x) * 64 + lane) * VEC;
    const int64_t first = int64_t(blockIdx.y) * a.slab_rows;
    const int64_t last = first + a.slab_rows < a.rows ? first + a.slab_rows : a.rows;
    const bool in = col < a.cols;
    float w[VEC], dw[VEC] = {}, db[VEC] = {};
    if (in) load_affine<VEC>(static_cast<const TW*>(a.w), col, w, 1.0f);
    for (int64_t row = first + wave; row < last && in; row += kNormThreads / 64) {
        float xv[VEC], gv[VEC];
        load_row<VEC>(static_cast<const T*>(a.x) + row * a.cols + col, xv);
        load_row<VEC>(static_cast<const T*>(a.dy) + row * a.cols + col, gv);
        const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            xv[k] = (xv[k] - mean) * rstd;
            dw[k] += gv[k] * xv[k];
            db[k] += gv[k];
        }
        if (a.dx) {
            const float2 c = a.row_sums[row];
#pragma unroll
            for (int k = 0; k < VEC; ++k) gv[k] = rstd * (gv[k] * w[k] - c.x - xv[k] * c.y);
            store_row<VEC>(static_cast<T*>(a.dx) + row * a.cols + col, gv);
        }
    }
    if (!a.part) return;
    if (wave > 0) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            sums[0][wave - 1][lane * VEC + k] = dw[k];
            sums[1][wave - 1][lane * VEC + k] = db[k];
        }
    }
    __syncthreads();
    if (wave == 0 && in) {
        float* part = a.part + int64_t(blockIdx.y) * 2 * a.cols + col;
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            float p = dw[k], q = db[k];
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                p += sums[0][i][lane * VEC + k];
                q += sums[1][i][lane * VEC + k];
            }
            part[k] = p;
            part[a.cols + k] = q;
        }
    }
}

// A workgroup sums 32 columns of the slabs' partials: eight groups of lanes
// take every eighth slab, then their sums are added in group order.
// blockIdx.y: 0 the weight's gradient, 1 the bias's.
template <typename TW>
__global__ void __launch_bounds__(kNormThreads) norm_reduce(const NormReduceArgs a) {
    __shared__ float sums[8][kNormReduceCols];
    TW* out = static_cast<TW*>(blockIdx.y ? a.db : a.dw);
    if (!out) return;
    const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
    const int col = int(blockIdx.x) * kNormReduceCols + lane;
    float s = 0.0f;
    if (col < a.cols)
        for (int i = group; i < a.slabs; i += 8) s += a.part[(int64_t(i) * 2 + blockIdx.y) * a.cols + col];
    sums[group][lane] = s;
    __syncthreads();
    if (group == 0 && col < a.cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sums[i][lane];
        out[col] = TW(s);
    }
}

// ----------------------------------------------------------------------------- host-side tables

template <typename T, typename TW, int VEC, int THREADS, int NC>
bool fits(int64_t cols, NormFwdKernel* out) {
    if (cols > int64_t(THREADS) * NC * VEC) return false;
    *out = {reinterpret_cast<const void*>(&norm_fwd<T, TW, VEC, THREADS, NC>), THREADS < 256 ? 256 : THREADS,
            THREADS == 64 ? 4 : 1};
    return true;
}

// The smallest shape that holds a row: a wavefront up to 2048 vector elements
// (no barrier), then workgroups of 256 and 1024 lanes.
template <typename T, typename TW>
NormFwdKernel fwd_for(bool vector, int64_t cols) {
    NormFwdKernel k{nullptr, 0, 0};
    constexpr int V = kVec16<T>;
    if (!vector) {
        (void)(fits<T, TW, 1, 64, 4>(cols, &k) || fits<T, TW, 1, 64, 16>(cols, &k) ||
               fits<T, TW, 1, 256, 16>(cols, &k) || fits<T, TW, 1, 1024, 16>(cols, &k) ||
               fits<T, TW, 1, 1024, 64>(cols, &k));
    } else {
        (void)(fits<T, TW, V, 64, 1>(cols, &k) || fits<T, TW, V, 64, 2>(cols, &k) || fits<T, TW, V, 64, 4>(cols, &k) ||
               fits<T, TW, V, 256, 2>(cols, &k) || fits<T, TW, V, 256, 4>(cols, &k) ||
               fits<T, TW, V, 1024, 2>(cols, &k) || fits<T, TW, V, 1024, 8>(cols, &k) ||
               fits<T, TW, V, 1024, 16>(cols, &k));
    }
    return k;
}

template <typename F>
auto by_types(int dtype, int wdtype, F f) -> decltype(f(float(), float())) {
    if (dtype == kF32 && wdtype == kF32) return f(float(), float());
    if (dtype == kF16 && wdtype == kF16) return f(_Float16(), _Float16());
    if (dtype == kF16 && wdtype == kF32) return f(_Float16(), float());
    if (dtype == kBF16 && wdtype == kBF16) return f(__bf16(), __bf16());
    if (dtype == kBF16 && wdtype == kF32) return f(__bf16(), float());
    return {};
}

}  // namespace

NormFwdKernel pick_norm_fwd(int dtype, int wdtype, bool vector, int64_t cols) {
    return by_types(dtype, wdtype, [&](auto t, auto tw) { return fwd_for<decltype(t), decltype(tw)>(vector, cols); });
}

const void* pick_norm_row_sums(int dtype, int wdtype, bool vector) {
    return by_types(dtype, wdtype, [&](auto t, auto tw) -> const void* {
        using T = decltype(t);
        using TW = decltype(tw);
        return vector ? reinterpret_cast<const void*>(&norm_row_sums<T, TW, kVec16<T>>)
                      : reinterpret_cast<const void*>(&norm_row_sums<T, TW, 1>);
    });
}

const void* pick_norm_bwd(int dtype, int wdtype, bool vector) {
    return by_types(dtype, wdtype, [&](auto t, auto tw) -> const void* {
        using T = decltype(t);
        using TW = decltype(tw);
        return vector ? reinterpret_cast<const void*>(&norm_bwd<T, TW, kVec16<T>>)
                      : reinterpret_cast<const void*>(&norm_bwd<T, TW, 1>);
    });
}

const void* pick_norm_reduce(int wdtype) {
    switch (wdtype) {
    case kF32: return reinterpret_cast<const void*>(&norm_reduce<float>);
    case kF16: return reinterpret_cast<const void*>(&norm_reduce<_Float16>);
    case kBF16: return reinterpret_cast<const void*>(&norm_reduce<__bf16>);
    }
    return nullptr;
}

}  // namespace rlpl
