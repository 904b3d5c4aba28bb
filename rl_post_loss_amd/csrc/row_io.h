// Element loads and stores of the kernels that walk rows or tensors: VEC
// consecutive elements as floats, 16 bytes at a time (VEC = 8 or 4) or one by
// one.  Included by the .hip sources only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace rlpl {

template <typename T> constexpr int kVec16 = 16 / int(sizeof(T));   // elements in 16 bytes

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(_Float16 x) { return float(x); }
__device__ __forceinline__ float widen(__bf16 x) { return float(x); }

// VEC elements at p as floats.  VEC > 1 needs p aligned to VEC * sizeof(T) bytes.
template <int VEC, typename T>
__device__ __forceinline__ void load_row(const T* p, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = widen(*p);
    } else if constexpr (VEC * sizeof(T) == 16) {
        const u32x4 d = *reinterpret_cast<const u32x4*>(p);
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = Elem<T>::get(w, k);
    } else if constexpr (VEC * sizeof(T) == 8) {
        const u32x2 d = *reinterpret_cast<const u32x2*>(p);
        const uint32_t w[2] = {d.x, d.y};
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = Elem<T>::get(w, k);
    } else {
        static_assert(VEC * sizeof(T) == 32, "32-, 16- or 8-byte vectors");
        float lo[VEC / 2], hi[VEC / 2];
        load_row<VEC / 2>(p, lo);
        load_row<VEC / 2>(p + VEC / 2, hi);
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = k < VEC / 2 ? lo[k] : hi[k - VEC / 2];
    }
}

// VEC floats rounded to T (nearest even) at p.
template <int VEC, typename T>
__device__ __forceinline__ void store_row(T* p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        *p = T(v[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < VEC; k += 4)
            *reinterpret_cast<u32x4*>(p + k) = u32x4{__float_as_uint(v[k]), __float_as_uint(v[k + 1]),
                                                     __float_as_uint(v[k + 2]), __float_as_uint(v[k + 3])};
    } else if constexpr (VEC == 8) {
        *reinterpret_cast<u32x4*>(p) = u32x4{Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]),
                                             Elem<T>::pack(v[4], v[5]), Elem<T>::pack(v[6], v[7])};
    } else {
        static_assert(VEC == 4, "vectors of 8 or 4");
        *reinterpret_cast<u32x2*>(p) = u32x2{Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3])};
    }
}

}  // namespace rlpl
