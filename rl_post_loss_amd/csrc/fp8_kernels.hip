// Products of 8-bit operands (e4m3) with a float32 scale for each block of 128
// on gfx950, and the quantisation of their operands.
//
//   out[i][v] = sum_b sx[i][b] sw[v / 128][b] sum_{k in block b} x[i][k] w[v][k]  (+ bias[v])
//
// A block of K is one matrix instruction deep (v_mfma_f32_16x16x128_f8f6f4):
// each starts from zero and its result is added to the accumulators times the
// block's two scales.  The projection takes the instruction's rows and the
// tokens its columns, so that a lane's four results share both scales and
// lie side by side in the output.  Sums are float32; the output is rounded once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "fp8_convert.h"
#include "fp8_kernels.h"
#include "loss_kernels.h"
#include "row_io.h"

namespace rlpl {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// A 16 x 16 tile of one block of K: element (i, j) = sum_k a[i][k] b[j][k].  Lane l holds 32 consecutive K bytes from
// 32 (l / 16) of row l % 16 of each operand, and rows 4 (l / 16) .. + 3 of column l % 16 of the result.
__device__ __forceinline__ f32x4 product(v8i a, v8i b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

// 32 bytes of a row from byte k on, zeros past K (a multiple of 16).
__device__ __forceinline__ v8i load32(const uint8_t* row, int32_t k, int32_t K) {
    u32x4 lo{0, 0, 0, 0}, hi{0, 0, 0, 0};
    if (k < K) lo = *reinterpret_cast<const u32x4*>(row + k);
    if (k + 16 < K) hi = *reinterpret_cast<const u32x4*>(row + k + 16);
    return v8i{int(lo.x), int(lo.y), int(lo.z), int(lo.w), int(hi.x), int(hi.y), int(hi.z), int(hi.w)};
}

template <typename T, int NT>
__global__ void __launch_bounds__(kFp8Threads) fp8_small(const Fp8LinearArgs a) {
    constexpr int F = kFp8SmallVocab / 16;
    __shared__ f32x4 part[3][F * NT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, quarter = lane >> 4;
    const int32_t v0 = int32_t(blockIdx.x) * kFp8SmallVocab, t0 = int32_t(blockIdx.y) * (16 * NT);
    f32x4 acc[F][NT] = {};
    const uint8_t* w[F];
    const uint8_t* x[NT];
    const float* sx[NT];
#pragma unroll
    for (int f = 0; f < F; ++f) {          // rows past the end read the last one: their results are not stored
        const int32_t v = v0 + 16 * f + row < a.vocab ? v0 + 16 * f + row : a.vocab - 1;
        w[f] = a.w + int64_t(v) * a.K;
    }
#pragma unroll
    for (int g = 0; g < NT; ++g) {
        const int32_t t = t0 + 16 * g + row < a.n ? t0 + 16 * g + row : a.n - 1;
        x[g] = a.x + int64_t(t) * a.K;
        sx[g] = a.x_scale + int64_t(t) * a.blocks;
    }
    const float* sw = a.w_scale + int64_t(v0 / kFp8Group) * a.blocks;
    for (int32_t b = wave; b < a.blocks; b += kFp8Threads / 64) {
        const int32_t k = b * kFp8Group + 32 * quarter;
        v8i wf[F], xf[NT];
#pragma unroll
        for (int f = 0; f < F; ++f) wf[f] = load32(w[f], k, a.K);
#pragma unroll
        for (int g = 0; g < NT; ++g) xf[g] = load32(x[g], k, a.K);
#pragma unroll
        for (int g = 0; g < NT; ++g) {
            const float s = sx[g][b] * sw[b];
#pragma unroll
            for (int f = 0; f < F; ++f) acc[f][g] += s * product(wf[f], xf[g]);
        }
    }
    // the wavefronts' shares, in their order
    if (wave > 0) {
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int g = 0; g < NT; ++g) part[wave - 1][f * NT + g][lane] = acc[f][g];
    }
    __syncthreads();
    if (wave > 0) return;
    T* out = static_cast<T*>(a.out);
    const T* bias = static_cast<const T*>(a.bias);
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int g = 0; g < NT; ++g) {
            f32x4 s = acc[f][g];
#pragma unroll
            for (int i = 0; i < 3; ++i) s += part[i][f * NT + g][lane];
            const int32_t t = t0 + 16 * g + row, v = v0 + 16 * f + 4 * quarter;
            if (t >= a.n) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (v + i < a.vocab) out[int64_t(t) * a.vocab + v + i] = T(bias ? s[i] + widen(bias[v + i]) : s[i]);
        }
}

// A lane's piece of 8 columns: where it lies and how many are there.
struct Eight {
    int32_t at, n;
};
template <typename T>
__device__ __forceinline__ void load8(const T* row, Eight p, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
    if (p.n == 8) {
        constexpr int V = kVec16<T>;
#pragma unroll
        for (int i = 0; i < 8 / V; ++i) {
            float part[V];
            widen_raw<T>(reinterpret_cast<const typename Unaligned16<T>::type*>(row + p.at)[i], part);
#pragma unroll
            for (int k = 0; k < V; ++k) v[i * V + k] = part[k];
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < p.n) v[k] = widen(row[p.at + k]);
    }
}
__device__ __forceinline__ void store8(uint8_t* row, Eight p, const float (&v)[8], float inv) {
    const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
    const uint32_t q[2] = {fp8_pack(lo, inv), fp8_pack(hi, inv)};
    if (p.n == 8) {
        typedef u32x2 bytes8 __attribute__((aligned(1)));
        *reinterpret_cast<bytes8*>(row + p.at) = u32x2{q[0], q[1]};
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < p.n) row[p.at + k] = uint8_t(q[k >> 2] >> (8 * (k & 3)));
    }
}
__device__ __forceinline__ float top8(const float (&v)[8]) {
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, finite_abs(v[k]));
    return top;
}

// 16 lanes a group of 128 columns.  A workgroup takes 16 groups of a row, or (SQUARE) 16 rows of one group at a time, 8
// times.
template <typename T, bool SQUARE>
__global__ void __launch_bounds__(kFp8Threads) quantise(const QuantiseArgs a) {
    __shared__ float tops[kFp8Threads / 64];
    const int lane = threadIdx.x & 15, team = threadIdx.x >> 4;
    const T* x = static_cast<const T*>(a.x);
    if constexpr (!SQUARE) {
        const int64_t all = a.rows * a.groups;
        for (int64_t item = int64_t(blockIdx.x) * 16 + team; item < all; item += int64_t(gridDim.x) * 16) {
            const int64_t row = item / a.groups;
            const int32_t group = int32_t(item % a.groups), at = group * kFp8Group + 8 * lane, left = a.cols - at;
            const Eight p{at, left < 0 ? 0 : left < 8 ? left : 8};
            float v[8];
            load8(x + row * a.ld, p, v);
            const Fp8Scale f(row16_max(top8(v)));
            store8(a.q + row * a.cols, p, v, f.inv);
            if (lane == 0) a.scale[item] = f.scale;
        }
    } else {
        constexpr int kSteps = kFp8Group / 16;
        const int64_t all = (a.rows + kFp8Group - 1) / kFp8Group * a.groups;
        for (int64_t item = blockIdx.x; item < all; item += gridDim.x) {
            const int64_t row0 = item / a.groups * kFp8Group + team;
            const int32_t at = int32_t(item % a.groups) * kFp8Group + 8 * lane, left = a.cols - at;
            const Eight p{at, left < 0 ? 0 : left < 8 ? left : 8};
            float v[kSteps][8], top = 0.0f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int64_t row = row0 + 16 * s;
                load8(x + row * a.ld, row < a.rows ? p : Eight{0, 0}, v[s]);
                top = fmaxf(top, top8(v[s]));
            }
            top = wave_max(top);
            __syncthreads();
            if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kFp8Threads / 64; ++i) top = fmaxf(top, tops[i]);
            const Fp8Scale f(top);
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int64_t row = row0 + 16 * s;
                if (row < a.rows) store8(a.q + row * a.cols, p, v[s], f.inv);
            }
            if (threadIdx.x == 0) a.scale[item] = f.scale;
        }
    }
}

template <typename T>
const void* small_of(int tokens) {
    switch (tokens) {
    case 16: return reinterpret_cast<const void*>(&fp8_small<T, 1>);
    case 32: return reinterpret_cast<const void*>(&fp8_small<T, 2>);
    case 64: return reinterpret_cast<const void*>(&fp8_small<T, 4>);
    }
    return nullptr;
}
template <bool SQUARE>
const void* quantise_of(int dtype) {
    switch (dtype) {
    case kF32: return reinterpret_cast<const void*>(&quantise<float, SQUARE>);
    case kF16: return reinterpret_cast<const void*>(&quantise<_Float16, SQUARE>);
    case kBF16: return reinterpret_cast<const void*>(&quantise<__bf16, SQUARE>);
    }
    return nullptr;
}

}  // namespace

const void* pick_fp8_small(int out_dtype, int tokens) {
    switch (out_dtype) {
    case kF32: return small_of<float>(tokens);
    case kF16: return small_of<_Float16>(tokens);
    case kBF16: return small_of<__bf16>(tokens);
    }
    return nullptr;
}
const void* pick_quantise(int dtype, bool square) { return square ? quantise_of<true>(dtype) : quantise_of<false>(dtype); }

}  // namespace rlpl
