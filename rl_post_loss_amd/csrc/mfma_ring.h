// Rings of operand stages in LDS: fragments of a K-contiguous stage tile, and the
// waits between the copies that fill a ring and the wavefronts that read it.
// The stages are those of mfma_tile.h, rows of 128 bytes.  Included by the .hip sources only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "mfma_tile.h"

namespace rlpl {

namespace {

// The fragments are read by asm statements that wait for their own reads: for a load or a builtin the compiler
// would add a wait for every copy into LDS in flight.

// Fragments of a K-contiguous stage tile: lane l's eight K values 32 half + 8 (l / 16) .. + 8 of row l % 16 of
// 16-row tiles, 2048 bytes apart.  k_base is the lane's place for the first of them.
__device__ __forceinline__ uint32_t lds_address(const char* p) {
    return uint32_t(uintptr_t((const __attribute__((address_space(3))) char*)p));
}
__device__ __forceinline__ uint32_t k_base(const char* t, int first, int half, int lane) {
    return lds_address(t + Stage<kGemmBK>::kc_offset(first + (lane & 15), half * 4 + (lane >> 4)));
}
// Four tiles from each of two places, as 16-byte pieces.
__device__ __forceinline__ void read_k(uint32_t at0, uint32_t at1, u32x4 (&v)[8]) {
    asm volatile(
        "ds_read_b128 %0, %8\n\tds_read_b128 %1, %8 offset:2048\n\t"
        "ds_read_b128 %2, %8 offset:4096\n\tds_read_b128 %3, %8 offset:6144\n\t"
        "ds_read_b128 %4, %9\n\tds_read_b128 %5, %9 offset:2048\n\t"
        "ds_read_b128 %6, %9 offset:4096\n\tds_read_b128 %7, %9 offset:6144\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
        : "v"(at0), "v"(at1)
        : "memory");
}
__device__ __forceinline__ void fragments_k(uint32_t at0, uint32_t at1, uint4 (&x)[4], uint4 (&y)[4]) {
    u32x4 v[8];
    read_k(at0, at1, v);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        x[c] = __builtin_bit_cast(uint4, v[c]);
        y[c] = __builtin_bit_cast(uint4, v[4 + c]);
    }
}
// From each of four places.
__device__ __forceinline__ void read_k(uint32_t at0, uint32_t at1, uint32_t at2, uint32_t at3, u32x4 (&v)[16]) {
    asm volatile(
        "ds_read_b128 %0, %16\n\tds_read_b128 %1, %16 offset:2048\n\t"
        "ds_read_b128 %2, %16 offset:4096\n\tds_read_b128 %3, %16 offset:6144\n\t"
        "ds_read_b128 %4, %17\n\tds_read_b128 %5, %17 offset:2048\n\t"
        "ds_read_b128 %6, %17 offset:4096\n\tds_read_b128 %7, %17 offset:6144\n\t"
        "ds_read_b128 %8, %18\n\tds_read_b128 %9, %18 offset:2048\n\t"
        "ds_read_b128 %10, %18 offset:4096\n\tds_read_b128 %11, %18 offset:6144\n\t"
        "ds_read_b128 %12, %19\n\tds_read_b128 %13, %19 offset:2048\n\t"
        "ds_read_b128 %14, %19 offset:4096\n\tds_read_b128 %15, %19 offset:6144\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7]),
          "=&v"(v[8]), "=&v"(v[9]), "=&v"(v[10]), "=&v"(v[11]), "=&v"(v[12]), "=&v"(v[13]), "=&v"(v[14]), "=&v"(v[15])
        : "v"(at0), "v"(at1), "v"(at2), "v"(at3)
        : "memory");
}
__device__ __forceinline__ void fragments_k(uint32_t at0, uint32_t at1, uint32_t at2, uint32_t at3, uint4 (&x)[4],
                                            uint4 (&y)[4], uint4 (&z)[4], uint4 (&w)[4]) {
    u32x4 v[16];
    read_k(at0, at1, at2, at3, v);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        x[c] = __builtin_bit_cast(uint4, v[c]);
        y[c] = __builtin_bit_cast(uint4, v[4 + c]);
        z[c] = __builtin_bit_cast(uint4, v[8 + c]);
        w[c] = __builtin_bit_cast(uint4, v[12 + c]);
    }
}

// Two tiles from each of two places.
__device__ __forceinline__ void read_k2(uint32_t at0, uint32_t at1, u32x4 (&v)[4]) {
    asm volatile(
        "ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:2048\n\t"
        "ds_read_b128 %2, %5\n\tds_read_b128 %3, %5 offset:2048\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
        : "v"(at0), "v"(at1)
        : "memory");
}
__device__ __forceinline__ void fragments_k2(uint32_t at0, uint32_t at1, uint4 (&x)[2], uint4 (&y)[2]) {
    u32x4 v[4];
    read_k2(at0, at1, v);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        x[c] = __builtin_bit_cast(uint4, v[c]);
        y[c] = __builtin_bit_cast(uint4, v[2 + c]);
    }
}
// Waits for a wavefront's copies into LDS, the last PENDING excepted.
template <int PENDING>
__device__ __forceinline__ void wait_copies() {
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(PENDING));
    asm volatile("" ::: "memory");
}
// The workgroup's barrier, with nothing moved across it.
__device__ __forceinline__ void meet() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

}  // namespace

}  // namespace rlpl
