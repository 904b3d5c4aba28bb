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

// A word of memory at p.  GLOBAL: p is known to be no LDS address (one that was itself read from memory; the
// compiler sees that of kernel arguments, and would make a flat access of this one).
template <typename W, bool GLOBAL>
__device__ __forceinline__ W load_word(const void* p) {
    if constexpr (GLOBAL) return *(const __attribute__((address_space(1))) W*)p;
    else return *static_cast<const W*>(p);
}
template <bool GLOBAL, typename W>
__device__ __forceinline__ void store_word(void* p, W w) {
    if constexpr (GLOBAL) *(__attribute__((address_space(1))) W*)p = w;
    else *static_cast<W*>(p) = w;
}

// VEC elements at p as floats.  VEC > 1 needs p aligned to VEC * sizeof(T) bytes, 16 at most.
template <int VEC, bool GLOBAL = false, typename T>
__device__ __forceinline__ void load_row(const T* p, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = widen(load_word<T, GLOBAL>(p));
    } else if constexpr (VEC * sizeof(T) == 16) {
        const u32x4 d = load_word<u32x4, GLOBAL>(p);
        const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = Elem<T>::get(w, k);
    } else if constexpr (VEC * sizeof(T) == 8) {
        const u32x2 d = load_word<u32x2, GLOBAL>(p);
        const uint32_t w[2] = {d.x, d.y};
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = Elem<T>::get(w, k);
    } else {
        static_assert(VEC * sizeof(T) == 32, "32-, 16- or 8-byte vectors");
        float lo[VEC / 2], hi[VEC / 2];
        load_row<VEC / 2, GLOBAL>(p, lo);
        load_row<VEC / 2, GLOBAL>(p + VEC / 2, hi);
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = k < VEC / 2 ? lo[k] : hi[k - VEC / 2];
    }
}

// VEC floats rounded to T (nearest even) at p.
template <int VEC, bool GLOBAL = false, typename T>
__device__ __forceinline__ void store_row(T* p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        store_word<GLOBAL>(p, T(v[0]));
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < VEC; k += 4)
            store_word<GLOBAL>(p + k, u32x4{__float_as_uint(v[k]), __float_as_uint(v[k + 1]), __float_as_uint(v[k + 2]),
                                            __float_as_uint(v[k + 3])});
    } else if constexpr (VEC == 8) {
        store_word<GLOBAL>(p, u32x4{Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]), Elem<T>::pack(v[4], v[5]),
                                    Elem<T>::pack(v[6], v[7])});
    } else {
        static_assert(VEC == 4, "vectors of 8 or 4");
        store_word<GLOBAL>(p, u32x2{Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3])});
    }
}

// 16 bytes of a row that may start at any element (the memory system takes such accesses whole).
template <typename T> struct Unaligned16;
template <> struct Unaligned16<float> { typedef u32x4 type __attribute__((aligned(4))); };
template <> struct Unaligned16<_Float16> { typedef u32x4 type __attribute__((aligned(2))); };
template <> struct Unaligned16<__bf16> { typedef u32x4 type __attribute__((aligned(2))); };

template <typename T>
__device__ __forceinline__ void widen_raw(u32x4 d, float (&v)[kVec16<T>]) {
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int k = 0; k < kVec16<T>; ++k) v[k] = Elem<T>::get(w, k);
}
template <typename T>
__device__ __forceinline__ u32x4 narrow_raw(const float (&v)[kVec16<T>]) {
    if constexpr (sizeof(T) == 4)
        return u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    else
        return u32x4{Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]), Elem<T>::pack(v[4], v[5]),
                     Elem<T>::pack(v[6], v[7])};
}

// How a row's columns are cut into pieces of V = kVec16<T>: exactly (cols a multiple of V); with the last piece
// moved back to end with the row, so that its first columns are the piece before's too (cols >= V); or
// with a short last piece (any cols).
enum { kRowExact = 0, kRowOverlap = 1, kRowShort = 2 };
inline int row_mode(int64_t cols, int v) { return cols % v == 0 ? kRowExact : cols >= v ? kRowOverlap : kRowShort; }

// A piece of a row: its first column, how many of its columns belong to the piece before, and how many there are.
template <typename T, int MODE>
struct RowPiece {
    static constexpr int V = kVec16<T>;
    int at, twice, n;
    __device__ __forceinline__ RowPiece(int piece, int cols) {
        const int col = piece * V;
        at = MODE == kRowOverlap && col + V > cols ? cols - V : col;
        twice = MODE == kRowOverlap && col < cols ? col - at : 0;
        n = MODE == kRowShort ? (cols - col < V ? cols - col : V) : (col < cols ? V : 0);
    }
    __device__ __forceinline__ bool any() const { return n > 0; }
    // Whether column k of the piece is this piece's own.
    __device__ __forceinline__ bool own(int k) const {
        return (MODE == kRowExact || k >= twice) && (MODE != kRowShort || k < n);
    }
    // The piece as it lies (zeros past a short one's end).
    __device__ __forceinline__ u32x4 load(const T* row) const {
        if constexpr (MODE == kRowShort) {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (k < n) {
                    if constexpr (sizeof(T) == 4) w[k] = reinterpret_cast<const uint32_t*>(row + at)[k];
                    else w[k >> 1] |= uint32_t(reinterpret_cast<const uint16_t*>(row + at)[k]) << (16 * (k & 1));
                }
            return u32x4{w[0], w[1], w[2], w[3]};
        } else {
            return *reinterpret_cast<const typename Unaligned16<T>::type*>(row + at);
        }
    }
    __device__ __forceinline__ void store(T* row, const float (&v)[V]) const {
        if constexpr (MODE == kRowShort) {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (k < n) row[at + k] = T(v[k]);
        } else {
            *reinterpret_cast<typename Unaligned16<T>::type*>(row + at) = narrow_raw<T>(v);
        }
    }
    // The columns' values of a vector of TW, `none` where there is no vector.
    template <typename TW>
    __device__ __forceinline__ void vector(const TW* p, float none, float (&v)[V]) const {
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = none;
        if (!p) return;
        if constexpr (MODE == kRowShort) {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (k < n) v[k] = widen(p[at + k]);
        } else {
            constexpr int W = kVec16<TW>;
#pragma unroll
            for (int c = 0; c < V; c += W) {
                float x[W];
                widen_raw<TW>(*reinterpret_cast<const typename Unaligned16<TW>::type*>(p + at + c), x);
#pragma unroll
                for (int k = 0; k < W; ++k) v[c + k] = x[k];
            }
        }
    }
};

}  // namespace rlpl
