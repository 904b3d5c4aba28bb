// Products of 8-bit operands (e4m3) with a float32 scale for each block of 128
// on gfx950, and the quantisation of their operands.
//
//   out[i][v] = sum_b sx[i][b] sw[v / 128][b] sum_{k in block b} x[i][k] w[v][k]  (+ bias[v])
//
// A block of K starts from zero on the matrix cores (fp8_mfma.h), and its result is added to the
// accumulators times the block's two scales.  The projection takes the instructions' rows and the
// tokens their columns, so that a lane's four results share both scales and
// lie side by side in the output.  Sums are float32; the output is rounded once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "fp8_convert.h"
#include "fp8_kernels.h"
#include "fp8_mfma.h"
#include "loss_kernels.h"
#include "row_io.h"

namespace rlpl {

namespace {

// The rows of an operand from `first` on as a buffer: what lies past the last one reads as zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_from(const uint8_t* x, int32_t first, int32_t rows, int32_t K) {
    const int64_t bytes = int64_t(rows - first) * K;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(x) + int64_t(first) * K, 0,
                                             int(bytes < 0x7FFFFFF0 ? bytes : 0x7FFFFFF0), 0x00020000);
}
// 32 bytes from `offset` (32 bytes of one row, `left` of them, or fewer, before its end; a multiple of 16), zeros past that.
__device__ __forceinline__ v8i load32(__amdgpu_buffer_rsrc_t from, uint32_t offset, int32_t left) {
    constexpr uint32_t kPast = 0xFFFFFFF0u;
    const auto lo = __builtin_amdgcn_raw_buffer_load_b128(from, int(left > 0 ? offset : kPast), 0, 0);
    const auto hi = __builtin_amdgcn_raw_buffer_load_b128(from, int(left > 16 ? offset + 16u : kPast), 0, 0);
    return __builtin_bit_cast(v8i, __builtin_shufflevector(__builtin_bit_cast(u32x4, lo), __builtin_bit_cast(u32x4, hi), 0, 1, 2, 3,
                                                           4, 5, 6, 7));
}

// Up to 16 rows: the projection goes from memory to registers, each byte once; the next block's 64 x 128 bytes are on
// their way while a block's are multiplied.  1 x 4096 x 128256: 94 us, 5.6 TB/s.  For 32 or 64 rows two or four fragments of
// tokens a wavefront were slower than the tiles of fp8_gemm.hip (64 x 4096 x 128256 175 us instead of 125): each workgroup reads
// all tokens again.
template <typename T, int F>
__global__ void __launch_bounds__(kFp8Threads) fp8_few(const Fp8LinearArgs a) {
    constexpr int kStep = kFp8Threads / 64;
    using Frag = Fragment<sizeof(T) == 4>;
    __shared__ f32x4 part[kStep - 1][F][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row = lane & 15, quarter = lane >> 4;
    const int32_t v0 = int32_t(blockIdx.x) * (16 * F);
    f32x4 acc[F] = {};
    const __amdgpu_buffer_rsrc_t from_w = rows_from(a.w, v0, a.vocab, a.K), from_x = rows_from(a.x, 0, a.n, a.K);
    const float* sx = a.x_scale + int64_t(row < a.n ? row : a.n - 1) * a.blocks;
    const float* sw = a.w_scale + int64_t(v0 / kFp8Group) * a.blocks;
    v8i wf[F], xf;
    float s_x = 0.0f, s_w = 0.0f;
    const auto load = [&](int32_t b) {
        const int32_t k = b * kFp8Group + 32 * quarter;
#pragma unroll
        for (int f = 0; f < F; ++f) wf[f] = load32(from_w, uint32_t(16 * f + row) * uint32_t(a.K) + uint32_t(k), a.K - k);
        xf = load32(from_x, uint32_t(row) * uint32_t(a.K) + uint32_t(k), a.K - k);
        s_x = sx[b];
        s_w = sw[b];
    };
    if (wave < a.blocks) load(wave);
    for (int32_t b = wave; b < a.blocks; b += kStep) {
        Frag wb[F];
        const Frag xb(xf);
        const float sb = s_x * s_w;
#pragma unroll
        for (int f = 0; f < F; ++f) wb[f] = Frag(wf[f]);
        if (b + kStep < a.blocks) load(b + kStep);
#pragma unroll
        for (int f = 0; f < F; ++f) acc[f] += sb * block_product(wb[f], xb);
    }
    // the wavefronts' shares, in their order
    if (wave > 0) {
#pragma unroll
        for (int f = 0; f < F; ++f) part[wave - 1][f][lane] = acc[f];
    }
    __syncthreads();
    if (wave > 0 || row >= a.n) return;
    T* out = static_cast<T*>(a.out) + int64_t(row) * a.vocab;
    const T* bias = static_cast<const T*>(a.bias);
#pragma unroll
    for (int f = 0; f < F; ++f) {
        f32x4 sum = acc[f];
#pragma unroll
        for (int i = 0; i < kStep - 1; ++i) sum += part[i][f][lane];
        const int32_t v = v0 + 16 * f + 4 * quarter;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (v + i < a.vocab) out[v + i] = T(bias ? sum[i] + widen(bias[v + i]) : sum[i]);
    }
}

// Scales turned over: a wavefront takes four columns of 64 rows, a lane a row.
__global__ void __launch_bounds__(64) turn(const TurnArgs a) {
    const int64_t r = int64_t(blockIdx.x) * kTurnRows + threadIdx.x;
    const int32_t c0 = int32_t(blockIdx.y) * kTurnCols;
    if (r >= a.rows) return;
    float v[kTurnCols];
#pragma unroll
    for (int k = 0; k < kTurnCols; ++k) v[k] = a.from[r * a.cols + (c0 + k < a.cols ? c0 + k : c0)];
#pragma unroll
    for (int k = 0; k < kTurnCols; ++k)
        if (c0 + k < a.cols) a.to[int64_t(c0 + k) * a.ld + r] = v[k];
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

// 128256 x 4096 bf16: 281 us by rows, 284 by squares (5.6 TB/s).  16 lanes a group of 128 columns.  A workgroup takes 16 groups of a row, or (SQUARE) 16 rows of one group at a time, 8
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

template <int F>
const void* few_of(int out_dtype) {
    switch (out_dtype) {
    case kF32: return reinterpret_cast<const void*>(&fp8_few<float, F>);
    case kF16: return reinterpret_cast<const void*>(&fp8_few<_Float16, F>);
    case kBF16: return reinterpret_cast<const void*>(&fp8_few<__bf16, F>);
    }
    return nullptr;
}
const void* pick_fp8_few(int out_dtype, int entries) {
    switch (entries) {
    case 16: return few_of<1>(out_dtype);
    case 32: return few_of<2>(out_dtype);
    case 64: return few_of<4>(out_dtype);
    }
    return nullptr;
}
const void* turn_kernel() { return reinterpret_cast<const void*>(&turn); }
const void* pick_quantise(int dtype, bool square) { return square ? quantise_of<true>(dtype) : quantise_of<false>(dtype); }

}  // namespace rlpl
