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
// read); the backward reads dy and x and writes dx once, for rows up to 16384
// columns (longer ones are read twice).  Statistics and sums are float32; each
// output is rounded once.  Measured, launch included: forward 65536 x 4096
// bf16 186 us (5.8 TB/s of its 1.07 GB), backward 32768 x 4096 bf16 154 us
// (5.2 TB/s of 0.81 GB; 280 us when the two averages over a row were a kernel of their own).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "loss_kernels.h"
#include "norm_kernels.h"
#include "row_io.h"

namespace rlpl {

namespace {

// The sum over a row's THREADS lanes, in every one of them (lane tree, then
// wavefronts in order).  red: THREADS / 64 floats of LDS (unused up to one wavefront).
template <int THREADS>
__device__ __forceinline__ float row_sum(float v, float* red) {
    if constexpr (THREADS == 16) {         // a row of lanes: the first four steps of wave_sum
        const auto add = [&v](uint32_t other) { v += __uint_as_float(other); };
        add(dpp_move<0xB1>(__float_as_uint(v)));
        add(dpp_move<0x4E>(__float_as_uint(v)));
        add(dpp_move<0x141>(__float_as_uint(v)));
        add(dpp_move<0x140>(__float_as_uint(v)));
        return v;
    }
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

// Rows a workgroup holds at a time, with THREADS lanes each.
template <int THREADS> constexpr int kRowsAtOnce = THREADS < kNormThreads ? kNormThreads / THREADS : 1;

template <typename T, typename TW, int MODE, int THREADS, int NC>
__global__ void __launch_bounds__(THREADS < 256 ? 256 : THREADS) norm_fwd(const NormFwdArgs a) {
    constexpr int V = kVec16<T>;
    using Piece = RowPiece<T, MODE>;
    __shared__ float red[THREADS < 64 ? 1 : THREADS / 64];
    constexpr int kRows = kRowsAtOnce<THREADS>;
    const int lane = threadIdx.x & (THREADS - 1);
    const float inv = 1.0f / float(a.cols);
    for (int64_t row = int64_t(blockIdx.x) * kRows + (kRows > 1 ? threadIdx.x / THREADS : 0); row < a.rows;
         row += int64_t(gridDim.x) * kRows) {
        const T* x = static_cast<const T*>(a.x) + row * a.cols;
        float v[NC][V];
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Piece p(c * THREADS + lane, a.cols);
            u32x4 raw{0, 0, 0, 0};
            if (p.any()) raw = p.load(x);
            widen_raw<T>(raw, v[c]);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Piece p(c * THREADS + lane, a.cols);
#pragma unroll
            for (int k = 0; k < V; ++k) s += p.own(k) ? v[c][k] : 0.0f;
        }
        const float mean = row_sum<THREADS>(s, red) * inv;
        float q = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Piece p(c * THREADS + lane, a.cols);
            const bool any = p.any();
#pragma unroll
            for (int k = 0; k < V; ++k) {
                v[c][k] -= mean;
                q += any && p.own(k) ? v[c][k] * v[c][k] : 0.0f;
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
            const Piece p(c * THREADS + lane, a.cols);
            if (!p.any()) continue;
            float w[V], b[V];
            p.vector(static_cast<const TW*>(a.w), 1.0f, w);
            p.vector(static_cast<const TW*>(a.b), 0.0f, b);
#pragma unroll
            for (int k = 0; k < V; ++k) v[c][k] = fmaf(v[c][k] * rstd, w[k], b[k]);
            p.store(y, v[c]);
        }
    }
}

// Backward of rows that a group of lanes or a workgroup holds: each row is read once, its two averages
// are joined while the next row's loads are in flight, and the column sums of the rows a workgroup takes stay
// in registers until its end.
template <typename T, typename TW, int MODE, int THREADS, int NC>
__global__ void __launch_bounds__(THREADS < kNormThreads ? kNormThreads : THREADS) norm_bwd_held(const NormBwdArgs a) {
    constexpr int V = kVec16<T>;
    using Piece = RowPiece<T, MODE>;
    constexpr int kRows = kRowsAtOnce<THREADS>;
    constexpr int kWavesHere = (THREADS < kNormThreads ? kNormThreads : THREADS) / 64;
    __shared__ float red[2][kWavesHere];
    __shared__ float joined[THREADS < kNormThreads ? 2 * THREADS * NC * V : 1];
    const int lane = threadIdx.x & (THREADS - 1), wave = threadIdx.x >> 6;
    const float inv = 1.0f / float(a.cols);
    float w[NC][V], dw[NC][V] = {}, db[NC][V] = {};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const Piece p(c * THREADS + lane, a.cols);
#pragma unroll
        for (int k = 0; k < V; ++k) w[c][k] = 0.0f;
        if (p.any()) p.vector(static_cast<const TW*>(a.w), 1.0f, w[c]);
    }
    u32x4 xr[NC], gr[NC];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Piece p(c * THREADS + lane, a.cols);
            xr[c] = gr[c] = u32x4{0, 0, 0, 0};
            if (p.any()) {
                xr[c] = p.load(static_cast<const T*>(a.x) + row * a.cols);
                gr[c] = p.load(static_cast<const T*>(a.dy) + row * a.cols);
            }
        }
    };
    int64_t row = int64_t(blockIdx.x) * kRows + (kRows > 1 ? threadIdx.x / THREADS : 0);
    const int64_t step = int64_t(gridDim.x) * kRows;
    if (row < a.rows) load(row);
    for (; row < a.rows; row += step) {
        float h[NC][V], g[NC][V];
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s = 0.0f, t = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Piece p(c * THREADS + lane, a.cols);
            widen_raw<T>(xr[c], h[c]);
            widen_raw<T>(gr[c], g[c]);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                h[c][k] = (h[c][k] - mean) * rstd;         // past the row's end meets a gradient of zero
                dw[c][k] += g[c][k] * h[c][k];
                db[c][k] += g[c][k];
                g[c][k] *= w[c][k];
                s += p.own(k) ? g[c][k] : 0.0f;
                t += p.own(k) ? g[c][k] * h[c][k] : 0.0f;
            }
        }
        if (row + step < a.rows) load(row + step);
        if (!a.dx) continue;
        if constexpr (THREADS <= 64) {
            s = row_sum<THREADS>(s, nullptr);
            t = row_sum<THREADS>(t, nullptr);
        } else {
            s = wave_sum(s);
            t = wave_sum(t);
            __syncthreads();               // red may still be read
            if ((threadIdx.x & 63) == 0) {
                red[0][wave] = s;
                red[1][wave] = t;
            }
            __syncthreads();
            s = red[0][0];
            t = red[1][0];
#pragma unroll
            for (int i = 1; i < kWavesHere; ++i) {
                s += red[0][i];
                t += red[1][i];
            }
        }
        s *= inv;
        t *= inv;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Piece p(c * THREADS + lane, a.cols);
            if (!p.any()) continue;
#pragma unroll
            for (int k = 0; k < V; ++k) g[c][k] = rstd * (g[c][k] - s - h[c][k] * t);
            p.store(static_cast<T*>(a.dx) + row * a.cols, g[c]);
        }
    }
    if (!a.part) return;
    float* part = a.part + int64_t(blockIdx.x) * 2 * a.cols;
    if constexpr (THREADS < kNormThreads) {
        // a wavefront's groups of lanes, then the four wavefronts one after the other
#pragma unroll
        for (int off = THREADS; off < 64; off <<= 1)
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    dw[c][k] += __shfl_xor(dw[c][k], off, 64);
                    db[c][k] += __shfl_xor(db[c][k], off, 64);
                }
        for (int turn = 0; turn < kNormThreads / 64; ++turn) {
            if (wave == turn && int(threadIdx.x & 63) < THREADS) {
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        float* at = joined + 2 * ((c * V + k) * THREADS + lane);
                        at[0] = turn ? at[0] + dw[c][k] : dw[c][k];
                        at[1] = turn ? at[1] + db[c][k] : db[c][k];
                    }
            }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < THREADS * NC * V; i += kNormThreads) {
            const Piece p(i / (THREADS * V) * THREADS + i % THREADS, a.cols);
            const int k = i / THREADS % V;
            if (p.any() && p.own(k)) {
                part[p.at + k] = joined[2 * i];
                part[a.cols + p.at + k] = joined[2 * i + 1];
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Piece p(c * THREADS + lane, a.cols);
            if (!p.any()) continue;
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (p.own(k)) {
                    part[p.at + k] = dw[c][k];
                    part[a.cols + p.at + k] = db[c][k];
                }
        }
    }
}

// Longer rows, in two kernels.  Per row, the averages over its columns of g = dy w and of g xhat: a wavefront a row.
template <typename T, typename TW, int MODE>
__global__ void __launch_bounds__(kNormThreads) norm_row_sums(const NormBwdArgs a) {
    constexpr int V = kVec16<T>;
    const int lane = threadIdx.x & 63, pieces = (a.cols + V - 1) / V;
    const float inv = 1.0f / float(a.cols);
    for (int64_t row = int64_t(blockIdx.x) * (kNormThreads / 64) + (threadIdx.x >> 6); row < a.rows;
         row += int64_t(gridDim.x) * (kNormThreads / 64)) {
        const T* x = static_cast<const T*>(a.x) + row * a.cols;
        const T* dy = static_cast<const T*>(a.dy) + row * a.cols;
        const float mean = a.mean[row], rstd = a.rstd[row];
        float s = 0.0f, t = 0.0f;
#pragma unroll 4
        for (int i = lane; i < pieces; i += 64) {
            const RowPiece<T, MODE> p(i, a.cols);
            float xv[V], gv[V], w[V];
            widen_raw<T>(p.load(x), xv);
            widen_raw<T>(p.load(dy), gv);
            p.vector(static_cast<const TW*>(a.w), 1.0f, w);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float g = p.own(k) ? gv[k] * w[k] : 0.0f;
                s += g;
                t += g * ((xv[k] - mean) * rstd);
            }
        }
        s = wave_sum(s);
        t = wave_sum(t);
        if (lane == 0) a.row_sums[row] = make_float2(s * inv, t * inv);
    }
}

// The input's gradient and a slab's column sums: a workgroup takes 64 pieces of
// columns of a slab's rows, its four wavefronts every fourth row each.
template <typename T, typename TW, int MODE>
__global__ void __launch_bounds__(kNormThreads) norm_bwd(const NormBwdArgs a) {
    constexpr int V = kVec16<T>;
    __shared__ float sums[2][3][64 * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const RowPiece<T, MODE> p(int(blockIdx.x) * 64 + lane, a.cols);
    const int64_t first = int64_t(blockIdx.y) * a.slab_rows;
    const int64_t last = first + a.slab_rows < a.rows ? first + a.slab_rows : a.rows;
    float w[V], dw[V] = {}, db[V] = {};
    if (p.any()) p.vector(static_cast<const TW*>(a.w), 1.0f, w);
#pragma unroll 2
    for (int64_t row = first + wave; row < last && p.any(); row += kNormThreads / 64) {
        float xv[V], gv[V];
        widen_raw<T>(p.load(static_cast<const T*>(a.x) + row * a.cols), xv);
        widen_raw<T>(p.load(static_cast<const T*>(a.dy) + row * a.cols), gv);
        const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            xv[k] = (xv[k] - mean) * rstd;
            dw[k] += gv[k] * xv[k];
            db[k] += gv[k];
        }
        if (a.dx) {
            const float2 c = a.row_sums[row];
#pragma unroll
            for (int k = 0; k < V; ++k) gv[k] = rstd * (gv[k] * w[k] - c.x - xv[k] * c.y);
            p.store(static_cast<T*>(a.dx) + row * a.cols, gv);
        }
    }
    if (!a.part) return;
    if (wave > 0) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            sums[0][wave - 1][lane * V + k] = dw[k];
            sums[1][wave - 1][lane * V + k] = db[k];
        }
    }
    __syncthreads();
    if (wave == 0 && p.any()) {
        float* part = a.part + int64_t(blockIdx.y) * 2 * a.cols + p.at;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (!p.own(k)) continue;
            float dwk = dw[k], dbk = db[k];
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                dwk += sums[0][i][lane * V + k];
                dbk += sums[1][i][lane * V + k];
            }
            part[k] = dwk;
            part[a.cols + k] = dbk;
        }
    }
}

// A workgroup sums 32 columns of the slabs' partials: 32 groups of lanes
// take every 32nd slab, then their sums are added in group order.
// blockIdx.y: 0 the weight's gradient, 1 the bias's.
template <typename TW>
__global__ void __launch_bounds__(kNormReduceThreads) norm_reduce(const NormReduceArgs a) {
    constexpr int kGroups = kNormReduceThreads / kNormReduceCols;
    __shared__ float sums[kGroups][kNormReduceCols];
    TW* out = static_cast<TW*>(blockIdx.y ? a.db : a.dw);
    if (!out) return;
    const int lane = threadIdx.x % kNormReduceCols, group = threadIdx.x / kNormReduceCols;
    const int col = int(blockIdx.x) * kNormReduceCols + lane;
    float s = 0.0f;
    if (col < a.cols) {
#pragma unroll 8
        for (int i = group; i < a.slabs; i += kGroups) s += a.part[(int64_t(i) * 2 + blockIdx.y) * a.cols + col];
    }
    sums[group][lane] = s;
    __syncthreads();
    if (group == 0 && col < a.cols) {
#pragma unroll
        for (int i = 1; i < kGroups; ++i) s += sums[i][lane];
        out[col] = TW(s);
    }
}

// ----------------------------------------------------------------------------- host-side tables

// Shapes: THREADS lanes a row, E columns a lane.
template <typename T, typename TW, int MODE, int THREADS, int E>
bool fits(int64_t cols, NormRowKernel* out) {
    if (cols > int64_t(THREADS) * E) return false;
    *out = {reinterpret_cast<const void*>(&norm_fwd<T, TW, MODE, THREADS, E / kVec16<T>>), THREADS < 256 ? 256 : THREADS,
            kRowsAtOnce<THREADS>};
    return true;
}
template <typename T, typename TW, int MODE, int THREADS, int E>
bool fits_bwd(int64_t cols, NormRowKernel* out) {
    if (cols > int64_t(THREADS) * E) return false;
    *out = {reinterpret_cast<const void*>(&norm_bwd_held<T, TW, MODE, THREADS, E / kVec16<T>>),
            THREADS < kNormThreads ? kNormThreads : THREADS, kRowsAtOnce<THREADS>};
    return true;
}

// The smallest shape that holds a row: 16 lanes (four rows a wavefront), a
// wavefront (no barrier), then workgroups of 256 and 1024 lanes.
template <typename T, typename TW>
NormRowKernel fwd_for(int64_t cols) {
    NormRowKernel k{nullptr, 0, 0};
    switch (row_mode(cols, kVec16<T>)) {
    case kRowShort: (void)fits<T, TW, kRowShort, 16, 8>(cols, &k); break;
    case kRowExact:
        (void)(fits<T, TW, kRowExact, 16, 8>(cols, &k) || fits<T, TW, kRowExact, 64, 8>(cols, &k) ||
               fits<T, TW, kRowExact, 64, 16>(cols, &k) || fits<T, TW, kRowExact, 64, 32>(cols, &k) ||
               fits<T, TW, kRowExact, 256, 16>(cols, &k) || fits<T, TW, kRowExact, 256, 32>(cols, &k) ||
               fits<T, TW, kRowExact, 1024, 16>(cols, &k) || fits<T, TW, kRowExact, 1024, 64>(cols, &k));
        break;
    case kRowOverlap:
        (void)(fits<T, TW, kRowOverlap, 16, 8>(cols, &k) || fits<T, TW, kRowOverlap, 64, 8>(cols, &k) ||
               fits<T, TW, kRowOverlap, 64, 16>(cols, &k) || fits<T, TW, kRowOverlap, 64, 32>(cols, &k) ||
               fits<T, TW, kRowOverlap, 256, 16>(cols, &k) || fits<T, TW, kRowOverlap, 256, 32>(cols, &k) ||
               fits<T, TW, kRowOverlap, 1024, 16>(cols, &k) || fits<T, TW, kRowOverlap, 1024, 64>(cols, &k));
    }
    return k;
}
template <typename T, typename TW>
NormRowKernel bwd_for(int64_t cols) {
    NormRowKernel k{nullptr, 0, 0};
    switch (row_mode(cols, kVec16<T>)) {
    case kRowShort: (void)fits_bwd<T, TW, kRowShort, 16, 8>(cols, &k); break;
    case kRowExact:
        (void)(fits_bwd<T, TW, kRowExact, 16, 8>(cols, &k) || fits_bwd<T, TW, kRowExact, 64, 8>(cols, &k) ||
               fits_bwd<T, TW, kRowExact, 64, 16>(cols, &k) || fits_bwd<T, TW, kRowExact, 256, 8>(cols, &k) ||
               fits_bwd<T, TW, kRowExact, 256, 16>(cols, &k) || fits_bwd<T, TW, kRowExact, 256, 32>(cols, &k) ||
               fits_bwd<T, TW, kRowExact, 512, 32>(cols, &k));
        break;
    case kRowOverlap:
        (void)(fits_bwd<T, TW, kRowOverlap, 16, 8>(cols, &k) || fits_bwd<T, TW, kRowOverlap, 64, 8>(cols, &k) ||
               fits_bwd<T, TW, kRowOverlap, 64, 16>(cols, &k) || fits_bwd<T, TW, kRowOverlap, 256, 8>(cols, &k) ||
               fits_bwd<T, TW, kRowOverlap, 256, 16>(cols, &k) || fits_bwd<T, TW, kRowOverlap, 256, 32>(cols, &k) ||
               fits_bwd<T, TW, kRowOverlap, 512, 32>(cols, &k));
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

NormRowKernel pick_norm_fwd(int dtype, int wdtype, int64_t cols) {
    return by_types(dtype, wdtype, [&](auto t, auto tw) { return fwd_for<decltype(t), decltype(tw)>(cols); });
}

NormRowKernel pick_norm_bwd_held(int dtype, int wdtype, int64_t cols) {
    return by_types(dtype, wdtype, [&](auto t, auto tw) { return bwd_for<decltype(t), decltype(tw)>(cols); });
}

const void* pick_norm_row_sums(int dtype, int wdtype, int64_t cols) {
    return by_types(dtype, wdtype, [&](auto t, auto tw) {
        using T = decltype(t);
        using TW = decltype(tw);
        return cols % kVec16<T> ? reinterpret_cast<const void*>(&norm_row_sums<T, TW, kRowOverlap>)
                                : reinterpret_cast<const void*>(&norm_row_sums<T, TW, kRowExact>);
    });
}

const void* pick_norm_bwd(int dtype, int wdtype, int64_t cols) {
    return by_types(dtype, wdtype, [&](auto t, auto tw) {
        using T = decltype(t);
        using TW = decltype(tw);
        return cols % kVec16<T> ? reinterpret_cast<const void*>(&norm_bwd<T, TW, kRowOverlap>)
                                : reinterpret_cast<const void*>(&norm_bwd<T, TW, kRowExact>);
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
