// AdamW over a list of tensors on gfx950, moments in float32 or in 8 bits.
//
//   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
//   p = p (1 - lr wd) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// One launch covers up to 440 tensors: a workgroup takes one chunk of 4096
// elements of one tensor, found through the plan's table.  Each element's
// state is read and written once, which bounds it: 150 M parameters in 300
// tensors with float32 moments, 16-bit gradients and copies take 0.81 to 0.92 ms
// (kernel trace; 4.9 to 5.6 TB/s of 4.5 GB), 525 M with 8-bit moments 1.71 ms (4.9
// TB/s of 8.4 GB; 1.84 ms while an element's rounding took 125 vector instructions
// instead of 100).
//
// 8-bit moments: 256 consecutive elements of a tensor share a float32 scale,
// their largest magnitude / 448, and are held as e4m3 values of x / scale.
// The second moment is held by its root, which halves its range of exponents.
// With three bits of mantissa a step of 1 - beta changes no value when it is
// rounded to nearest, so each rounding goes up with the probability of the
// part it drops, by 16 random bits made from (seed, step, tensor, element): the
// first moment and the second one's root are then right on average after each
// step.  The root's square is not: a step adds the rounding's variance, at most
// (the step's move) x (the distance of neighbours, an eighth of a normal value
// at most), which over the 1 / (1 - beta2) steps that a moment remembers comes to
// an eighth of it at most.  Gaussian gradients leave the second moment 5 %
// above the exact one on average (beta2 0.999, from 1000 steps on), so updates
// 2.5 % smaller.  A root above zero is never rounded
// to zero, since the next update divides by it.  An element that is not
// finite is held as NaN and leaves the rest of its block as it is.
//
// Every operation here is one IEEE float32 operation in the order written
// (no contraction), so that equal inputs give equal bits on any layout.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "adamw_kernels.h"
#include "device_common.h"
#include "loss_kernels.h"
#include "row_io.h"

namespace rlpl {

namespace {

#pragma clang fp contract(off)

constexpr float kE4m3Max = 448.0f;
constexpr float kInvE4m3Max = 1.0f / 448.0f;
constexpr float kTinyBlock = 0x1p-118f;    // a block with no value from here on is held as zeros

struct Hyper {
    float beta1, beta2, c1, c2, eps, step_size, root, decay;
};

// The new parameter from the new first moment and the root of the new second one.
__device__ __forceinline__ float updated(float p, float m, float root_v, const Hyper& h) {
    const float denom = root_v * h.root + h.eps;
    const float u = (m / denom) * h.step_size;
    return p * h.decay - u;
}

__device__ __forceinline__ float new_first(float m, float g, const Hyper& h) { return m * h.beta1 + g * h.c1; }
__device__ __forceinline__ float new_second(float v, float g, const Hyper& h) { return v * h.beta2 + (g * h.c2) * g; }

// The largest of a wavefront's words, in every lane, by DPP lane moves (0 where no lane is the source).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    const auto more = [&v](uint32_t other) { v = other > v ? other : v; };
    more(dpp_move<0xB1>(v));               // quad_perm [1, 0, 3, 2]
    more(dpp_move<0x4E>(v));               // quad_perm [2, 3, 0, 1]
    more(dpp_move<0x141>(v));              // row_half_mirror
    more(dpp_move<0x140>(v));              // row_mirror
    more(dpp_move<0x142, 0xA>(v));         // row_bcast:15
    more(dpp_move<0x143, 0xC>(v));         // row_bcast:31
    return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}

constexpr uint32_t kInfBits = 0x7F800000u;

// a = |x| / scale (finite, at most about 448) to an e4m3 value, up where the part below the last place plus
// u16 / 2^16 reaches one.  Normal values: a carry in the bits.  Below 2^-6 the last place is 2^-9.
__device__ __forceinline__ float e4m3_round(float a, uint32_t u16) {
    const float normal = __uint_as_float((__float_as_uint(a) + (u16 << 4)) & 0xFFF00000u);
    const float small = floorf(fmaf(a, 0x1p9f, float(u16) * 0x1p-16f)) * 0x1p-9f;   // a * 2^9 is exact
    const float q = a < 0x1p-6f ? small : normal;
    return q > kE4m3Max ? kE4m3Max : q;
}

// A block's four values a lane (all >= 0 where ROOT) to four e4m3 bytes and the block's scale, with 16 random bits each.
template <bool ROOT>
__device__ __forceinline__ uint32_t quantise(const float (&x)[4], const uint32_t (&u16)[4], float* scale, int lane) {
    uint32_t top_bits = 0, all = 0;        // of the finite magnitudes, and of all
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t m = __float_as_uint(x[k]) & 0x7FFFFFFFu;
        all = m > all ? m : all;
        top_bits = m > top_bits && m < kInfBits ? m : top_bits;
    }
    const bool bad = __any(all >= kInfBits);
    const float top = __uint_as_float(wave_max(top_bits));
    const bool live = top >= kTinyBlock;
    const float inv = live ? kE4m3Max / top : 0.0f;
    if (lane == 0) store_word<true>(scale, live ? top * kInvE4m3Max : 0.0f);
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        q[k] = e4m3_round(fabsf(x[k]) * inv, u16[k]);
        if (ROOT) q[k] = x[k] > 0.0f ? fmaxf(q[k], 0x1p-9f) : q[k];
        else q[k] = copysignf(q[k], x[k]);
    }
    if (bad) {                             // some value of the wavefront's block is not finite
#pragma unroll
        for (int k = 0; k < 4; ++k)
            q[k] = (__float_as_uint(x[k]) & 0x7FFFFFFFu) >= kInfBits ? __builtin_nanf("") : q[k];
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
    return uint32_t(w);
}

__device__ __forceinline__ void widen_e4m3(uint32_t w, float scale, float (&v)[4]) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(w), true);
    v[0] = lo[0] * scale;
    v[1] = lo[1] * scale;
    v[2] = hi[0] * scale;
    v[3] = hi[1] * scale;
}

template <int VEC>
__device__ __forceinline__ void store_copy(void* copy, int dtype, int64_t i, const float (&p)[VEC]) {
    if (!copy) return;
    if (dtype == kBF16) store_row<VEC, true>(static_cast<__bf16*>(copy) + i, p);
    else store_row<VEC, true>(static_cast<_Float16*>(copy) + i, p);
}

// VEC consecutive elements with moments in float32.
template <typename P, typename G, int VEC>
__device__ __forceinline__ void step32(const AdamTensor& t, const G* g, float scale, int64_t i, int copy_dtype,
                                       const Hyper& h) {
    float p[VEC], gv[VEC], m[VEC], v[VEC];
    load_row<VEC, true>(static_cast<const P*>(t.param) + i, p);
    load_row<VEC, true>(g + i, gv);
    load_row<VEC, true>(static_cast<const float*>(t.m) + i, m);
    load_row<VEC, true>(static_cast<const float*>(t.v) + i, v);
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
        const float gk = gv[k] * scale;
        m[k] = new_first(m[k], gk, h);
        v[k] = new_second(v[k], gk, h);
        p[k] = updated(p[k], m[k], sqrtf(v[k]), h);
    }
    store_row<VEC, true>(static_cast<P*>(t.param) + i, p);
    store_row<VEC, true>(static_cast<float*>(t.m) + i, m);
    store_row<VEC, true>(static_cast<float*>(t.v) + i, v);
    store_copy<VEC>(t.copy, copy_dtype, i, p);
}

// A block of 256 elements from i0 on (n in the tensor) with moments in 8 bits: four consecutive ones a lane.
template <typename P, typename G, bool VECTOR>
__device__ __forceinline__ void step8(const AdamTensor& t, const G* g, float scale, int64_t i0, int copy_dtype,
                                      const Hyper& h, uint32_t key) {
    const int lane = threadIdx.x & 63;
    const int64_t i = i0 + 4 * lane, block = i0 / kAdamBlock;
    float p[4] = {}, gv[4] = {}, m[4], r[4];
    uint32_t um[4], ur[4];
    uint32_t mq = 0, rq = 0;
    const bool whole = VECTOR && i + 4 <= t.n;
    const int here = i >= t.n ? 0 : t.n - i < 4 ? int(t.n - i) : 4;
    if (whole) {
        load_row<4, true>(static_cast<const P*>(t.param) + i, p);
        load_row<4, true>(g + i, gv);
        mq = load_word<uint32_t, true>(static_cast<const uint8_t*>(t.m) + i);
        rq = load_word<uint32_t, true>(static_cast<const uint8_t*>(t.v) + i);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k >= here) continue;
            p[k] = widen(load_word<P, true>(static_cast<const P*>(t.param) + i + k));
            gv[k] = widen(load_word<G, true>(g + i + k));
            mq |= uint32_t(load_word<uint8_t, true>(static_cast<const uint8_t*>(t.m) + i + k)) << (8 * k);
            rq |= uint32_t(load_word<uint8_t, true>(static_cast<const uint8_t*>(t.v) + i + k)) << (8 * k);
        }
    }
    widen_e4m3(mq, load_word<float, true>(t.m_scale + block), m);
    widen_e4m3(rq, load_word<float, true>(t.v_scale + block), r);
    const uint32_t mine = mix32(key + uint32_t(uint64_t(i) >> 32));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float gk = gv[k] * scale;
        m[k] = new_first(m[k], gk, h);
        r[k] = sqrtf(new_second(r[k] * r[k], gk, h));
        p[k] = updated(p[k], m[k], r[k], h);
        const uint32_t word = mix32(uint32_t(i + k) ^ mine);
        um[k] = word & 0xFFFFu;
        ur[k] = word >> 16;
        if (k >= here) m[k] = r[k] = 0.0f;   // past the tensor's end: nothing that the block's scale sees
    }
    mq = quantise<false>(m, um, t.m_scale + block, lane);
    rq = quantise<true>(r, ur, t.v_scale + block, lane);
    if (whole) {
        store_row<4, true>(static_cast<P*>(t.param) + i, p);
        store_word<true>(static_cast<uint8_t*>(t.m) + i, mq);
        store_word<true>(static_cast<uint8_t*>(t.v) + i, rq);
        store_copy<4>(t.copy, copy_dtype, i, p);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (k >= here) continue;
            store_word<true>(static_cast<P*>(t.param) + i + k, P(p[k]));
            store_word<true>(static_cast<uint8_t*>(t.m) + i + k, uint8_t(mq >> (8 * k)));
            store_word<true>(static_cast<uint8_t*>(t.v) + i + k, uint8_t(rq >> (8 * k)));
            const float one[1] = {p[k]};
            store_copy<1>(t.copy, copy_dtype, i + k, one);
        }
    }
}

template <typename P, typename G, int BITS>
__global__ void __launch_bounds__(kAdamThreads) adamw(const AdamArgs a) {
    const AdamChunk c = a.chunks[blockIdx.x];
    const AdamTensor t = a.tensors[c.tensor];
    const G* g = static_cast<const G*>(a.grads[c.tensor - a.first]);
    if (!g) return;                        // no gradient: the tensor stays as it is
    const float scale = a.grad_scale ? *a.grad_scale : 1.0f;
    const double lr = a.lr_at ? double(*a.lr_at) : a.lr;
    double correction1 = a.correction1;
    float root = a.root;
    uint32_t step = a.step;
    if (a.step_at) {
        const int64_t s = *a.step_at;
        correction1 = -expm1(double(s) * a.log_beta1);
        root = float(1.0 / sqrt(-expm1(double(s) * a.log_beta2)));
        step = uint32_t(s);
    }
    const Hyper h{a.beta1, a.beta2, a.one_minus_beta1, a.one_minus_beta2, a.eps, float(lr / correction1), root,
                  float(1.0 - lr * t.weight_decay)};
    const int64_t first = int64_t(c.place) * kAdamChunk;
    const int64_t last = first + kAdamChunk < t.n ? first + kAdamChunk : t.n;
    const bool vector = t.aligned && (reinterpret_cast<uintptr_t>(g) & 15) == 0;
    if constexpr (BITS == 32) {
        const int64_t vlast = vector ? first + (last - first) / 4 * 4 : first;
        for (int64_t i = first + 4 * int64_t(threadIdx.x); i < vlast; i += 4 * kAdamThreads)
            step32<P, G, 4>(t, g, scale, i, a.copy_dtype, h);
        for (int64_t i = vlast + threadIdx.x; i < last; i += kAdamThreads)
            step32<P, G, 1>(t, g, scale, i, a.copy_dtype, h);
    } else {
        const uint32_t key = mix32(mix32(a.seed ^ step) ^ c.tensor);
        for (int64_t i0 = first + int64_t(threadIdx.x >> 6) * kAdamBlock; i0 < last; i0 += (kAdamThreads / 64) * kAdamBlock) {
            if (vector) step8<P, G, true>(t, g, scale, i0, a.copy_dtype, h, key);
            else step8<P, G, false>(t, g, scale, i0, a.copy_dtype, h, key);
        }
    }
}

template <typename P, typename G>
const void* for_bits(int bits) {
    return bits == 32 ? reinterpret_cast<const void*>(&adamw<P, G, 32>) : reinterpret_cast<const void*>(&adamw<P, G, 8>);
}
template <typename P>
const void* for_grad(int grad, int bits) {
    switch (grad) {
    case kF32: return for_bits<P, float>(bits);
    case kF16: return for_bits<P, _Float16>(bits);
    case kBF16: return for_bits<P, __bf16>(bits);
    }
    return nullptr;
}

}  // namespace

const void* pick_adamw(int param_dtype, int grad_dtype, int state_bits) {
    switch (param_dtype) {
    case kF32: return for_grad<float>(grad_dtype, state_bits);
    case kF16: return for_grad<_Float16>(grad_dtype, state_bits);
    case kBF16: return for_grad<__bf16>(grad_dtype, state_bits);
    }
    return nullptr;
}

}  // namespace rlpl
