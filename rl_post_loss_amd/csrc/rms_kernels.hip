// RMS norm on gfx950, with the addition of a residual and an output in 8 bits
// with scales, and its backward pass.
//
//   h = x + r (rounded to the stream's type),  rstd = 1 / sqrt(avg h^2 + eps),  y = h rstd w
//   q = e4m3(y 448 / top), scale = top / 448 for the largest magnitude `top` of 128 columns
//   xhat = h rstd,  g = dy w,  dh = rstd (g - xhat avg(g xhat)) + dstream,  dw = sum_rows dy xhat
//
// Bound by memory traffic: a row is read once and held in registers until its
// mean square is known; the 16 lanes that hold a group of 128 columns join
// its largest magnitude by lane moves.  The norm is that of h as it is stored,
// which is what the backward pass reads.  Statistics and sums are float32;
// each output is rounded once.
//
// With a residual, in 8 bits, 32768 x 4096 bf16 take 160 us (5.9 TB/s of 0.94 GB);
// backward 16384 x 4096 96 us (5.6 TB/s of 0.54 GB with the stream's gradient) and 4.5 for the sum over
// workgroups.  Rows whose elements start between two dwords (16-bit types, odd
// lengths) take 1.2 to 1.4 times as long as those of even ones (30000 x 4001: forward 105 us, 4002: 87; backward 218 and 162,
// 296 and 233 with the stream's gradient; float32 rows of 4001, whose accesses start at dwords, backward 332, of 4000 322).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "fp8_convert.h"
#include "loss_kernels.h"
#include "rms_kernels.h"
#include "row_io.h"

namespace rlpl {

namespace {

// Eight columns of a row: whole ones (cols a multiple of 8), with the last piece of a row moved back to end with it
// (its first columns, `twice` of them, are then the piece before's, and not stored again), or a short one (cols < 8).
template <int MODE>
struct Piece8 {
    int at, twice, n;
    __device__ __forceinline__ Piece8(int piece, int cols) {
        const int col = piece * 8;
        at = MODE == kRowOverlap && col + 8 > cols ? cols - 8 : col;
        twice = MODE == kRowOverlap && col < cols ? col - at : 0;
        n = MODE == kRowShort ? (cols - col < 8 ? cols - col : 8) : (col < cols ? 8 : 0);
    }
    __device__ __forceinline__ bool any() const { return n > 0; }
    __device__ __forceinline__ bool own(int k) const {
        return (MODE == kRowExact || k >= twice) && (MODE != kRowShort || k < n);
    }
    __device__ __forceinline__ bool whole() const { return MODE == kRowExact || (MODE == kRowOverlap && twice == 0); }
};

// A piece as it lies in memory.
template <typename T>
struct Raw8 {
    u32x4 d[sizeof(T) / 2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (auto& v : d) v = u32x4{0, 0, 0, 0};
    }
    template <int MODE>
    __device__ __forceinline__ void load(const T* row, const Piece8<MODE>& p) {
        if constexpr (MODE == kRowShort) {
            uint32_t w[2 * sizeof(T)] = {};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < p.n) {
                    if constexpr (sizeof(T) == 4) w[k] = reinterpret_cast<const uint32_t*>(row + p.at)[k];
                    else w[k >> 1] |= uint32_t(reinterpret_cast<const uint16_t*>(row + p.at)[k]) << (16 * (k & 1));
                }
#pragma unroll
            for (int i = 0; i < int(sizeof(T)) / 2; ++i) d[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < int(sizeof(T)) / 2; ++i)
                d[i] = reinterpret_cast<const typename Unaligned16<T>::type*>(row + p.at)[i];
        }
    }
    __device__ __forceinline__ void widen(float (&v)[8]) const {
        constexpr int V = kVec16<T>;
#pragma unroll
        for (int i = 0; i < 8 / V; ++i) {
            float part[V];
            widen_raw<T>(d[i], part);
#pragma unroll
            for (int k = 0; k < V; ++k) v[i * V + k] = part[k];
        }
    }
};

template <typename T, int MODE>
__device__ __forceinline__ void store8(T* row, const Piece8<MODE>& p, const float (&v)[8]) {
    constexpr int V = kVec16<T>;
    if (p.whole()) {
#pragma unroll
        for (int i = 0; i < 8 / V; ++i) {
            float part[V];
#pragma unroll
            for (int k = 0; k < V; ++k) part[k] = v[i * V + k];
            reinterpret_cast<typename Unaligned16<T>::type*>(row + p.at)[i] = narrow_raw<T>(part);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (p.own(k)) row[p.at + k] = T(v[k]);
    }
}

// The columns' weights: ones without a vector.
template <typename T, int MODE>
__device__ __forceinline__ void weights(const void* w, int w_f32, const Piece8<MODE>& p, float (&v)[8]) {
    if (!w) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 1.0f;
    } else if (w_f32) {
        Raw8<float> raw;
        raw.load(static_cast<const float*>(w), p);
        raw.widen(v);
    } else {
        Raw8<T> raw;
        raw.load(static_cast<const T*>(w), p);
        raw.widen(v);
    }
}

// The sum over a row's THREADS lanes, in every one of them (lane tree, then wavefronts in order).
template <int THREADS>
__device__ __forceinline__ float row_sum(float v, float* red) {
    if constexpr (THREADS <= 32) {
        const auto add = [&v](uint32_t other) { v += __uint_as_float(other); };
        add(dpp_move<0xB1>(__float_as_uint(v)));
        add(dpp_move<0x4E>(__float_as_uint(v)));
        add(dpp_move<0x141>(__float_as_uint(v)));
        add(dpp_move<0x140>(__float_as_uint(v)));
        if constexpr (THREADS == 32) v += __shfl_xor(v, 16, 64);
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

template <typename T, typename R, bool FP8, int MODE, int THREADS, int NC>
__global__ void __launch_bounds__(THREADS < kNormThreads ? kNormThreads : THREADS) rms_fwd(const RmsFwdArgs a) {
    using Piece = Piece8<MODE>;
    __shared__ float red[THREADS < 64 ? 1 : THREADS / 64];
    constexpr int kRows = kRowsAtOnce<THREADS>;
    const int lane = threadIdx.x & (THREADS - 1);
    const float inv = 1.0f / float(a.cols);
    for (int64_t row = int64_t(blockIdx.x) * kRows + (kRows > 1 ? threadIdx.x / THREADS : 0); row < a.rows;
         row += int64_t(gridDim.x) * kRows) {
        float h[NC][8];
        Raw8<T> x[NC];
        Raw8<R> r[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Piece p(c * THREADS + lane, a.cols);
            x[c].clear();
            r[c].clear();
            if (p.any()) {
                x[c].load(static_cast<const T*>(a.x) + row * a.cols, p);
                if (a.residual) r[c].load(static_cast<const R*>(a.residual) + row * a.cols, p);
            }
        }
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Piece p(c * THREADS + lane, a.cols);
            x[c].widen(h[c]);
            if (a.residual) {
                float rv[8];
                r[c].widen(rv);
#pragma unroll
                for (int k = 0; k < 8; ++k) h[c][k] = float(R(h[c][k] + rv[k]));
                if (p.any()) store8(static_cast<R*>(a.stream) + row * a.cols, p, h[c]);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) s += p.any() && p.own(k) ? h[c][k] * h[c][k] : 0.0f;
        }
        const float rstd = 1.0f / sqrtf(row_sum<THREADS>(s, red) * inv + a.eps);
        if (lane == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int piece = c * THREADS + lane;
            const Piece p(piece, a.cols);
            float w[8];
            if (p.any()) {
                weights<T>(a.w, a.w_f32, p, w);
#pragma unroll
                for (int k = 0; k < 8; ++k) h[c][k] = h[c][k] * rstd * w[k];
            }
            if constexpr (FP8) {
                float top = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, p.any() && p.own(k) ? finite_abs(h[c][k]) : 0.0f);
                const Fp8Scale f(row16_max(top));
                if (!p.any()) continue;
                if ((piece & 15) == 0) a.scale[row * a.groups + (piece >> 4)] = f.scale;
                uint8_t* y = static_cast<uint8_t*>(a.y) + row * a.cols + p.at;
                const float lo[4] = {h[c][0], h[c][1], h[c][2], h[c][3]}, hi[4] = {h[c][4], h[c][5], h[c][6], h[c][7]};
                const uint32_t q[2] = {fp8_pack(lo, f.inv), fp8_pack(hi, f.inv)};
                if (p.whole()) {
                    typedef u32x2 bytes8 __attribute__((aligned(1)));
                    *reinterpret_cast<bytes8*>(y) = u32x2{q[0], q[1]};
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (p.own(k)) y[k] = uint8_t(q[k >> 2] >> (8 * (k & 3)));
                }
            } else {
                if (p.any()) store8(static_cast<T*>(a.y) + row * a.cols, p, h[c]);
            }
        }
    }
}

// Backward of rows that a group of lanes or a workgroup holds: each row is read once, its average is joined
// while the next row's loads are in flight, and the column sums of the rows a workgroup takes stay in registers until
// its end.
template <typename T, typename R, int MODE, int THREADS, int NC>
__global__ void __launch_bounds__(THREADS < kNormThreads ? kNormThreads : THREADS) rms_bwd(const RmsBwdArgs a) {
    using Piece = Piece8<MODE>;
    constexpr int kRows = kRowsAtOnce<THREADS>;
    constexpr int kWavesHere = (THREADS < kNormThreads ? kNormThreads : THREADS) / 64;
    __shared__ float red[kWavesHere];
    __shared__ float joined[THREADS < kNormThreads ? THREADS * NC * 8 : 1];
    const int lane = threadIdx.x & (THREADS - 1), wave = threadIdx.x >> 6;
    const float inv = 1.0f / float(a.cols);
    float w[NC][8], dw[NC][8] = {};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const Piece p(c * THREADS + lane, a.cols);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[c][k] = 0.0f;
        if (p.any()) weights<T>(a.w, a.w_f32, p, w[c]);
    }
    Raw8<R> hr[NC], sr[NC];
    Raw8<T> gr[NC];
    auto load = [&](int64_t row) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Piece p(c * THREADS + lane, a.cols);
            hr[c].clear();
            gr[c].clear();
            sr[c].clear();
            if (p.any()) {
                hr[c].load(static_cast<const R*>(a.h) + row * a.cols, p);
                gr[c].load(static_cast<const T*>(a.dy) + row * a.cols, p);
                if (a.dstream) sr[c].load(static_cast<const R*>(a.dstream) + row * a.cols, p);
            }
        }
    };
    int64_t row = int64_t(blockIdx.x) * kRows + (kRows > 1 ? threadIdx.x / THREADS : 0);
    const int64_t step = int64_t(gridDim.x) * kRows;
    if (row < a.rows) load(row);
    for (; row < a.rows; row += step) {
        float h[NC][8], g[NC][8];
        const float rstd = a.rstd[row];
        float t = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Piece p(c * THREADS + lane, a.cols);
            hr[c].widen(h[c]);
            gr[c].widen(g[c]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                h[c][k] *= rstd;
                dw[c][k] += g[c][k] * h[c][k];             // past the row's end both are zero
                g[c][k] *= w[c][k];
                t += p.own(k) ? g[c][k] * h[c][k] : 0.0f;
            }
        }
        if (a.dh) {
            if constexpr (THREADS <= 64) {
                t = row_sum<THREADS>(t, nullptr);
            } else {
                t = row_sum<THREADS>(t, red);
            }
            t *= inv;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const Piece p(c * THREADS + lane, a.cols);
                if (!p.any()) continue;
                float add[8];
                sr[c].widen(add);
#pragma unroll
                for (int k = 0; k < 8; ++k) g[c][k] = fmaf(rstd, g[c][k] - h[c][k] * t, add[k]);
                store8(static_cast<R*>(a.dh) + row * a.cols, p, g[c]);
            }
        }
        if (row + step < a.rows) load(row + step);
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
                for (int k = 0; k < 8; ++k) dw[c][k] += __shfl_xor(dw[c][k], off, 64);
        for (int turn = 0; turn < kNormThreads / 64; ++turn) {
            if (wave == turn && int(threadIdx.x & 63) < THREADS) {
#pragma unroll
                for (int c = 0; c < NC; ++c)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float* at = joined + (c * 8 + k) * THREADS + lane;
                        *at = turn ? *at + dw[c][k] : dw[c][k];
                    }
            }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < THREADS * NC * 8; i += kNormThreads) {
            const Piece p(i / (THREADS * 8) * THREADS + i % THREADS, a.cols);
            const int k = i / THREADS % 8;
            if (p.any() && p.own(k)) part[p.at + k] = joined[i];
        }
    } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const Piece p(c * THREADS + lane, a.cols);
            if (!p.any()) continue;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (p.own(k)) part[p.at + k] = dw[c][k];
        }
    }
}

// ----------------------------------------------------------------------------- host-side tables

// The smallest shape that holds a row, THREADS lanes of NC pieces each.  Idle lanes cost: rows of 256 in 8 bits take 68 us
// with 32 lanes and 90 with 64 (200000 of them), rows of 4100 backward 154 with 256 x 3 and 239 with 256 x 4 (30000), of 6001
// 171 and 269 (20000).
template <typename T, typename R, bool FP8, int MODE, int THREADS, int NC>
bool fits(int64_t cols, NormRowKernel* out) {
    if (cols > int64_t(THREADS) * NC * 8) return false;
    *out = {reinterpret_cast<const void*>(&rms_fwd<T, R, FP8, MODE, THREADS, NC>),
            THREADS < kNormThreads ? kNormThreads : THREADS, kRowsAtOnce<THREADS>};
    return true;
}
template <typename T, typename R, int MODE, int THREADS, int NC>
bool fits_bwd(int64_t cols, NormRowKernel* out) {
    if (cols > int64_t(THREADS) * NC * 8) return false;
    *out = {reinterpret_cast<const void*>(&rms_bwd<T, R, MODE, THREADS, NC>),
            THREADS < kNormThreads ? kNormThreads : THREADS, kRowsAtOnce<THREADS>};
    return true;
}

template <typename T, typename R, bool FP8, int MODE>
bool fwd_mode(int64_t cols, NormRowKernel* k) {
    return fits<T, R, FP8, MODE, 16, 1>(cols, k) || fits<T, R, FP8, MODE, 32, 1>(cols, k) || fits<T, R, FP8, MODE, 64, 1>(cols, k) ||
           fits<T, R, FP8, MODE, 64, 2>(cols, k) || fits<T, R, FP8, MODE, 64, 4>(cols, k) ||
           fits<T, R, FP8, MODE, 256, 2>(cols, k) || fits<T, R, FP8, MODE, 256, 3>(cols, k) || fits<T, R, FP8, MODE, 256, 4>(cols, k) ||
           fits<T, R, FP8, MODE, 1024, 2>(cols, k);
}
template <typename T, typename R, bool FP8>
NormRowKernel fwd_for(int64_t cols) {
    NormRowKernel k{nullptr, 0, 0};
    switch (row_mode(cols, 8)) {
    case kRowShort: (void)fits<T, R, FP8, kRowShort, 16, 1>(cols, &k); break;
    case kRowExact: (void)fwd_mode<T, R, FP8, kRowExact>(cols, &k); break;
    case kRowOverlap: (void)fwd_mode<T, R, FP8, kRowOverlap>(cols, &k); break;
    }
    return k;
}
template <typename T, typename R, int MODE>
bool bwd_mode(int64_t cols, NormRowKernel* k) {
    return fits_bwd<T, R, MODE, 16, 1>(cols, k) || fits_bwd<T, R, MODE, 32, 1>(cols, k) || fits_bwd<T, R, MODE, 64, 1>(cols, k) ||
           fits_bwd<T, R, MODE, 64, 2>(cols, k) || fits_bwd<T, R, MODE, 256, 1>(cols, k) ||
           fits_bwd<T, R, MODE, 256, 2>(cols, k) || fits_bwd<T, R, MODE, 256, 3>(cols, k) || fits_bwd<T, R, MODE, 256, 4>(cols, k) ||
           fits_bwd<T, R, MODE, 1024, 2>(cols, k);
}
template <typename T, typename R>
NormRowKernel bwd_for(int64_t cols) {
    NormRowKernel k{nullptr, 0, 0};
    switch (row_mode(cols, 8)) {
    case kRowShort: (void)fits_bwd<T, R, kRowShort, 16, 1>(cols, &k); break;
    case kRowExact: (void)bwd_mode<T, R, kRowExact>(cols, &k); break;
    case kRowOverlap: (void)bwd_mode<T, R, kRowOverlap>(cols, &k); break;
    }
    return k;
}

template <typename F>
NormRowKernel by_types(int dtype, int stream_dtype, F f) {
    if (dtype == kF32 && stream_dtype == kF32) return f(float(), float());
    if (dtype == kF16 && stream_dtype == kF16) return f(_Float16(), _Float16());
    if (dtype == kF16 && stream_dtype == kF32) return f(_Float16(), float());
    if (dtype == kBF16 && stream_dtype == kBF16) return f(__bf16(), __bf16());
    if (dtype == kBF16 && stream_dtype == kF32) return f(__bf16(), float());
    return {nullptr, 0, 0};
}

}  // namespace

NormRowKernel pick_rms_fwd(int dtype, int stream_dtype, bool fp8, int64_t cols) {
    return by_types(dtype, stream_dtype, [&](auto t, auto r) {
        return fp8 ? fwd_for<decltype(t), decltype(r), true>(cols) : fwd_for<decltype(t), decltype(r), false>(cols);
    });
}

NormRowKernel pick_rms_bwd(int dtype, int stream_dtype, int64_t cols) {
    return by_types(dtype, stream_dtype, [&](auto t, auto r) { return bwd_for<decltype(t), decltype(r)>(cols); });
}

}  // namespace rlpl
