// The norm over a list of gradients, the factor that clips it, and gradients
// multiplied by a factor in place, on gfx950.
//
//   norm = sqrt(sum g^2) or max |g|,  scale = min(1, max_norm / (norm + eps))
//
// One launch covers up to 190 tensors of any float types, whose chunks of 4096
// elements its workgroups take in runs of equal length, across the tensors'
// ends.  Squares are summed in float64, in which no float32 value overflows
// or vanishes: a lane's serially, then lanes, wavefronts and
// workgroups in a fixed order (no atomics), so equal calls give equal bits.
// Bound by reading the gradients once: 150 M elements in 300 tensors take 61 us in bf16
// and 106 in float32 (4.9 and 5.7 TB/s), scaled in place 200 in float32 (6 TB/s both ways).  A short list is one
// workgroup's, in one launch (6 us for 24,000 elements; two launches take 4.6 more).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "grad_kernels.h"
#include "loss_kernels.h"
#include "row_io.h"

namespace rlpl {

namespace {

// NaN stays one.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

template <bool INF>
struct Total;
template <>
struct Total<false> {
    double v = 0.0;
    __device__ __forceinline__ void add(float x) { v = fma(double(x), double(x), v); }
    __device__ __forceinline__ void join(double o) { v += o; }
    __device__ __forceinline__ double value() const { return v; }
};
template <>
struct Total<true> {
    float v = 0.0f;
    __device__ __forceinline__ void add(float x) { v = larger(v, fabsf(x)); }
    __device__ __forceinline__ void join(double o) { v = larger(v, float(o)); }
    __device__ __forceinline__ double value() const { return double(v); }
};

// Calls f(pointer to T, first element, elements) for each part of one tensor that lies in chunks [lo, hi) of the list.
template <typename F>
__device__ __forceinline__ void walk(const GradList& l, uint32_t lo, uint32_t hi, F f) {
    if (lo >= hi) return;
    uint32_t a = 0, b = l.count;           // the tensor of chunk lo: the last one whose first chunk is not past it
    while (b - a > 1) {
        const uint32_t m = (a + b) / 2;
        if (l.first[m] <= lo) a = m;
        else b = m;
    }
    for (; a < l.count && l.first[a] < hi; ++a) {
        const uint32_t from = l.first[a] > lo ? l.first[a] : lo, to = l.first[a + 1] < hi ? l.first[a + 1] : hi;
        if (from >= to) continue;          // an empty tensor
        const int64_t n = l.n[a] >> 2, begin = int64_t(from - l.first[a]) * kGradChunk;
        int64_t end = int64_t(to - l.first[a]) * kGradChunk;
        if (end > n) end = n;
        switch (int(l.n[a] & 3)) {
        case kF32: f(static_cast<float*>(l.p[a]) + begin, end - begin); break;
        case kF16: f(static_cast<_Float16*>(l.p[a]) + begin, end - begin); break;
        default: f(static_cast<__bf16*>(l.p[a]) + begin, end - begin); break;
        }
    }
}

// Elements before p is aligned to 16 bytes.
template <typename T>
__device__ __forceinline__ int64_t head_of(const T* p, int64_t n) {
    const int64_t head = int64_t((-reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    return head < n ? head : n;
}

template <bool INF, int THREADS>
__device__ __forceinline__ double sum_chunks(const GradList& l, uint32_t lo, uint32_t hi) {
    constexpr int U = 4;
    Total<INF> t;
    walk(l, lo, hi, [&t](auto* p, int64_t n) {
        using T = std::remove_pointer_t<decltype(p)>;
        constexpr int V = kVec16<T>;
        const int64_t head = head_of(p, n), vectors = (n - head) / V, rest = n - head - vectors * V;
        const int tid = threadIdx.x;
        if (tid < head) t.add(widen(load_word<T, true>(p + tid)));
        if (tid < rest) t.add(widen(load_word<T, true>(p + n - rest + tid)));
        const T* q = p + head;
        int64_t i = tid;
        for (; i + (U - 1) * THREADS < vectors; i += U * THREADS) {
            u32x4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) raw[u] = load_word<u32x4, true>(q + (i + u * THREADS) * V);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[V];
                widen_raw<T>(raw[u], x);
#pragma unroll
                for (int k = 0; k < V; ++k) t.add(x[k]);
            }
        }
        for (; i < vectors; i += THREADS) {
            float x[V];
            widen_raw<T>(load_word<u32x4, true>(q + i * V), x);
#pragma unroll
            for (int k = 0; k < V; ++k) t.add(x[k]);
        }
    });
    return t.value();
}

// The workgroup's total in every lane: lanes by a tree, then wavefronts in order.
template <bool INF, int THREADS>
__device__ __forceinline__ double join_all(double v, double* red) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        Total<INF> t;
        t.v = v;
        t.join(__shfl_xor(v, off, 64));
        v = t.value();
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    Total<INF> t;
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) t.join(red[i]);
    return t.value();
}

__device__ __forceinline__ void write_norm(const GradFinish& f, double total) {
    const float g = f.grad_scale ? *f.grad_scale : 1.0f;
    const float norm = float((f.inf ? total : sqrt(total)) * fabs(double(g)));
    *f.norm = norm;
    if (f.scale) {
        const float clip = f.max_norm / (norm + f.eps);
        *f.scale = g * (clip < 1.0f ? clip : norm == norm ? 1.0f : clip);    // a norm of NaN gives NaN
    }
}

template <bool INF>
__global__ void __launch_bounds__(kGradThreads) grad_norm(const GradNormArgs a) {
    __shared__ double red[kGradThreads / 64];
    const uint64_t chunks = a.list.first[a.list.count];
    const uint32_t lo = uint32_t(chunks * blockIdx.x / gridDim.x), hi = uint32_t(chunks * (blockIdx.x + 1) / gridDim.x);
    const double t = join_all<INF, kGradThreads>(sum_chunks<INF, kGradThreads>(a.list, lo, hi), red);
    if (threadIdx.x == 0) a.part[blockIdx.x] = t;
}

template <bool INF>
__global__ void __launch_bounds__(kGradAloneThreads) grad_alone(const GradNormArgs a) {
    __shared__ double red[kGradAloneThreads / 64];
    const double t = join_all<INF, kGradAloneThreads>(sum_chunks<INF, kGradAloneThreads>(a.list, 0, a.list.first[a.list.count]), red);
    if (threadIdx.x == 0) write_norm(a.finish, t);
}

template <bool INF>
__device__ __forceinline__ double all_parts(const GradFinish& f, double* red) {
    Total<INF> t;
    for (int i = threadIdx.x; i < f.parts; i += kGradAloneThreads) t.join(f.part[i]);
    return join_all<INF, kGradAloneThreads>(t.value(), red);
}
__global__ void __launch_bounds__(kGradAloneThreads) grad_finish(const GradFinish f) {
    __shared__ double red[kGradAloneThreads / 64];
    const double t = f.inf ? all_parts<true>(f, red) : all_parts<false>(f, red);
    if (threadIdx.x == 0) write_norm(f, t);
}

// The tensors' elements times *scale, each rounded once.  A factor of one writes nothing.
__global__ void __launch_bounds__(kGradThreads) grad_scale(const GradScaleArgs a) {
    const float s = *a.scale;
    if (s == 1.0f) return;
    const uint64_t chunks = a.list.first[a.list.count];
    const uint32_t lo = uint32_t(chunks * blockIdx.x / gridDim.x), hi = uint32_t(chunks * (blockIdx.x + 1) / gridDim.x);
    walk(a.list, lo, hi, [s](auto* p, int64_t n) {
        using T = std::remove_pointer_t<decltype(p)>;
        constexpr int V = kVec16<T>, U = 4;
        const int64_t head = head_of(p, n), vectors = (n - head) / V, rest = n - head - vectors * V;
        const int tid = threadIdx.x;
        if (tid < head) store_word<true>(p + tid, T(widen(load_word<T, true>(p + tid)) * s));
        if (tid < rest) store_word<true>(p + n - rest + tid, T(widen(load_word<T, true>(p + n - rest + tid)) * s));
        T* q = p + head;
        int64_t i = tid;
        for (; i + (U - 1) * kGradThreads < vectors; i += U * kGradThreads) {
            u32x4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) raw[u] = load_word<u32x4, true>(q + (i + u * kGradThreads) * V);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[V];
                widen_raw<T>(raw[u], x);
#pragma unroll
                for (int k = 0; k < V; ++k) x[k] *= s;
                store_word<true>(q + (i + u * kGradThreads) * V, narrow_raw<T>(x));
            }
        }
        for (; i < vectors; i += kGradThreads) {
            float x[V];
            widen_raw<T>(load_word<u32x4, true>(q + i * V), x);
#pragma unroll
            for (int k = 0; k < V; ++k) x[k] *= s;
            store_word<true>(q + i * V, narrow_raw<T>(x));
        }
    });
}

}  // namespace

const void* pick_grad_norm(bool inf) {
    return inf ? reinterpret_cast<const void*>(&grad_norm<true>) : reinterpret_cast<const void*>(&grad_norm<false>);
}
const void* pick_grad_alone(bool inf) {
    return inf ? reinterpret_cast<const void*>(&grad_alone<true>) : reinterpret_cast<const void*>(&grad_alone<false>);
}
const void* grad_finish_kernel() { return reinterpret_cast<const void*>(&grad_finish); }
const void* grad_scale_kernel() { return reinterpret_cast<const void*>(&grad_scale); }

}  // namespace rlpl
