// Values held in e4m3 with a float32 scale for a group of them: scale = (the
// largest finite magnitude) / 448, or 0 where that is below 2^-118, and each
// value x 448 / largest rounded to nearest even.  A value that is not finite
// becomes NaN and leaves its group's others as they are.  Included by the
// .hip sources only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace rlpl {

constexpr float kFp8Top = 448.0f;
constexpr float kFp8InvTop = 1.0f / 448.0f;
constexpr float kFp8Tiny = 0x1p-118f;

struct Fp8Scale {
    float scale, inv;
    __device__ __forceinline__ explicit Fp8Scale(float top) {
        const bool live = top >= kFp8Tiny;
        scale = live ? top * kFp8InvTop : 0.0f;
        inv = live ? kFp8Top / top : 0.0f;
    }
};

// The magnitude where it is finite, else 0.
__device__ __forceinline__ float finite_abs(float x) {
    const float m = fabsf(x);
    return m < __builtin_inff() ? m : 0.0f;
}

// The largest over 16 lanes side by side, in each of them, and over a wavefront; values >= 0.
__device__ __forceinline__ float row16_max(float v) {
    const auto more = [&v](uint32_t other) { v = fmaxf(v, __uint_as_float(other)); };
    more(dpp_move<0xB1>(__float_as_uint(v)));     // quad_perm [1, 0, 3, 2]
    more(dpp_move<0x4E>(__float_as_uint(v)));     // quad_perm [2, 3, 0, 1]
    more(dpp_move<0x141>(__float_as_uint(v)));    // row_half_mirror
    more(dpp_move<0x140>(__float_as_uint(v)));    // row_mirror
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
    v = row16_max(v);
    v = fmaxf(v, __uint_as_float(dpp_move<0x142, 0xA>(__float_as_uint(v))));    // row_bcast:15
    v = fmaxf(v, __uint_as_float(dpp_move<0x143, 0xC>(__float_as_uint(v))));    // row_bcast:31
    return __uint_as_float(uint32_t(__builtin_amdgcn_readlane(int(__float_as_uint(v)), 63)));
}

// Four values to four e4m3 bytes.  The largest one times inv may round to just over 448, which the conversion takes to
// 448 again; what was not finite is NaN times anything (inf times 0 included) or stays infinite, and becomes NaN.
__device__ __forceinline__ uint32_t fp8_pack(const float (&x)[4], float inv) {
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        q[k] = x[k] * inv;
        q[k] = fabsf(q[k]) < __builtin_inff() ? q[k] : __builtin_nanf("");
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
    return uint32_t(w);
}

}  // namespace rlpl
