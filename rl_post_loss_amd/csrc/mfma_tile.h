// Tiles of a matrix-core contraction on gfx950: operand stages in LDS filled
// by buffer-to-LDS copies, their bank layouts, fragments for
// v_mfma_f32_32x32x16, and the order of tiles over the XCDs.  The tile
// constants are those of logprob_kernels.h.  Included by the .hip sources only.
#pragma once

#include <hip/hip_runtime.h>
#include <float.h>
#include <stdint.h>

#include "device_common.h"
#include "logprob_kernels.h"

namespace rlpl {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float floatx16 __attribute__((ext_vector_type(16)));

// One v_mfma_f32_32x32x16 of the operand type (tag argument selects bf16 or fp16).
template <typename U> struct Mfma {
    static __device__ __forceinline__ floatx16 run(uint4 a, uint4 b, floatx16 c, __bf16) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
    }
    static __device__ __forceinline__ floatx16 run(uint4 a, uint4 b, floatx16 c, _Float16) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b),
                                                      c, 0, 0, 0);
    }
};

template <typename T> __device__ __forceinline__ float to_f(T x) { return float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x) { return T(x); }

constexpr int kGemmWaves = kGemmWavesM * kGemmWavesN;
constexpr int kWaveM = kGemmBM / kGemmWavesM;   // rows of C per wavefront
constexpr int kWaveN = kGemmBN / kGemmWavesN;   // columns of C per wavefront
constexpr int kFragM = kWaveM / 32;      // 32 x 32 MFMA tiles per wavefront, rows
constexpr int kFragN = kWaveN / 32;      // and columns
constexpr float kLog2eG = 1.4426950408889634f;

static_assert(kWaveM % 32 == 0 && kWaveN % 32 == 0, "32 x 32 matrix tiles");
static_assert(kGemmBN == 256 && kGemmBM <= kGemmThreads && kGemmBN <= kGemmThreads,
              "the epilogues use one thread per tile column / row");
static_assert(kWaveM == 64 || kWaveM == 128, "log-sum-exp partial layout");

// LDS layout of one R x BK operand tile (R = kGemmBM or kGemmBN rows, BK the stage depth),
// filled by 16-byte global->LDS copies (each wavefront copy writes 1 KB
// contiguously: lane l's 16 bytes at +16*l), with an XOR swizzle of 16-byte
// chunks that keeps the matrix-core fragment reads free of bank conflicts.
// A 16-byte read serves 16 lanes per pass over all 64 banks (256 bytes), so
// the 16 rows a pass reads must spread over distinct 16-byte bank groups.
//
// K-contiguous operand (element (r, k) at x[r*ld + k]): row r is 2 BK bytes,
// kC = BK / 8 chunks; chunk c (elements 8c..8c+7) sits in slot
// c ^ swizzle(r).  64-byte rows (BK = 32): rows four apart share banks,
// swizzle (r >> 2) & 3 (measured free of bank conflicts on gfx950; (r >> 1) & 3
// had 2-way conflicts).  128-byte rows (BK = 64): rows two apart share
// banks, swizzle (r >> 1) & 7.  Fragment reads are one 16-byte read per lane;
// a copy covers 1024 / (2 BK) whole rows, so it reads full 64- or 128-byte
// row segments (the 128-byte ones copy about 1.5x faster from cache,
// measured).
//
// MN-contiguous operand (element (r, k) at x[k*ld + r]): blocks of 64 r by
// BK K rows; in a block, K row k is 128 bytes and its chunk c (r = 8c..8c+7 of
// the block) sits in slot c ^ (4 ((k >> 1) & 1)), so that a copy brings 8 K
// rows of 128 bytes.  Fragment reads are two transposing 8-byte reads per
// lane (ds_read_b64_tr_b16); a pass of 32 lanes reads 4 K rows of 32 r, and
// the swizzle puts K rows two apart on the other half of the banks.
// The stages of depth BK: sizes, copy counts and LDS layouts.
template <int BK>
struct Stage {
    static constexpr int kBytesA = kGemmBM * BK * 2;   // A tile of one stage
    static constexpr int kBytesB = kGemmBN * BK * 2;   // B tile of one stage
    static constexpr int kBytes = kBytesA + kBytesB;
    static constexpr int kCount = kGemmDynLds / kBytes;   // ring slots
    static constexpr int kDmaA = kBytesA / 1024 / kGemmWaves;   // 1 KB copies per wavefront for the A tile
    static constexpr int kDmaB = kBytesB / 1024 / kGemmWaves;   // and for the B tile
    static constexpr int kC = BK / 8;                 // 16-byte chunks per K-contiguous row
    static constexpr int kRowsPerCopy = 1024 / (2 * BK);
    static_assert(kC == 4 || kC == 8, "32- or 64-deep stages");
    static_assert(kCount >= 2 && kCount * kBytes == kGemmDynLds, "LDS ring");
    static_assert(kDmaA * kGemmWaves * 1024 == kBytesA && kDmaB * kGemmWaves * 1024 == kBytesB, "whole copies");
    static __device__ __forceinline__ int kc_swizzle(int r) { return kC == 4 ? (r >> 2) & 3 : (r >> 1) & 7; }
    static __device__ __forceinline__ int kc_offset(int r, int c) { return r * (2 * BK) + 16 * (c ^ kc_swizzle(r)); }
    static __device__ __forceinline__ int mn_swizzle(int k) { return ((k >> 1) & 1) << 2; }
    static __device__ __forceinline__ int mn_offset(int k, int r) {
        return (r >> 6) * (128 * BK) + k * 128 + 16 * (((r & 63) >> 3) ^ mn_swizzle(k)) + 2 * (r & 7);
    }
};

// Per-lane source of the wavefront's 1 KB copies of one operand tile: copy q
// (0 .. R * BK / 512 - 1; each wavefront issues 1/kGemmWaves of them) of
// the tile whose first element is (r0, k0).  Returns the byte offset of the
// lane's 16 bytes from that element (the copy goes through a buffer descriptor
// based there), or kOutOfRange for a chunk of rows past R or of K at or past
// ke, which the buffer unit reads as zeros.  A chunk that starts before ke is
// read whole: the caller guarantees that the elements past ke in it are zeros
// or that ke is a multiple of 8.  Offsets stay below 2 * (BK + 256 * ld)
// bytes.
constexpr uint32_t kOutOfRange = 0xFFFFFFF0u;
constexpr int kBufferRecords = 0x7FFFFFF0;

template <bool KCONTIG, int BK, typename St = Stage<BK>>
__device__ __forceinline__ uint32_t dma_source(int q, int lane, uint32_t ld, int R, int ke, int r0, int k0) {
    if constexpr (KCONTIG) {
        const int r = St::kRowsPerCopy * q + lane / St::kC;
        const int c = (lane % St::kC) ^ St::kc_swizzle(r);
        const bool ok = r0 + r < R && k0 + 8 * c < ke;
        return ok ? 2u * (uint32_t(r) * ld + uint32_t(8 * c)) : kOutOfRange;
    } else {
        const int cb = q / (BK / 8), k = 8 * (q % (BK / 8)) + (lane >> 3);
        const int c = (lane & 7) ^ St::mn_swizzle(k);
        const int rr = 64 * cb + 8 * c;
        const bool ok = r0 + rr < R && k0 + k < ke;
        return ok ? 2u * (uint32_t(k) * ld + uint32_t(rr)) : kOutOfRange;
    }
}

// One 16-byte copy per lane from a buffer (offset `off`) into LDS at lds + 16 * lane.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t src, uint32_t off, void* lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (__attribute__((address_space(3))) void*)lds, 16, int(off), 0, 0, 0);
}

// Raw buffer descriptor over the memory from p on (gfx9 raw-buffer flags).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, kBufferRecords, 0x00020000);
}

// s_waitcnt immediate that waits for vmcnt <= v (expcnt and lgkmcnt left at their maxima).
constexpr int vmcnt_imm(int v) { return 0x0F70 | (v & 15) | ((v >> 4) << 14); }

// Wait until at most `pending` (compile-time) stages of this wavefront's copies
// (kDmaA + kDmaB of Stage<BK> per stage) are in flight, then meet the other
// wavefronts.
template <int PENDING, int BK>
__device__ __forceinline__ void wait_stages() {
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(PENDING * (Stage<BK>::kDmaA + Stage<BK>::kDmaB)));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Matrix-core fragments of stage tile t for wavefront row/column block wb (of
// WT rows), 32-row tile f, K step kk (16 K): the eight K values lane l needs
// for row/column wb*WT + f*32 + l%32, K 8*(l/32) .. +8.
template <bool KCONTIG, int WT, int BK>
__device__ __forceinline__ uint4 fragment(const uint16_t* __restrict__ t, int wb, int f, int kk, int lane) {
    if constexpr (KCONTIG) {
        const int r = wb * WT + f * 32 + (lane & 31);
        return *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(t) + Stage<BK>::kc_offset(r, kk * 2 + (lane >> 5)));
    } else {
        // 16-lane group G: columns 16*(G%2) .. +16 of the 32-wide tile, K base 8*(G/2).
        // Input lane q = 4j + t of the group points at K row kbase + j, columns 4t .. 4t+3;
        // output lane i then holds K rows kbase .. kbase+3 of column i.
        const int G = lane >> 4, q = lane & 15;
        const int r = wb * WT + f * 32 + 16 * (G & 1) + 4 * (q & 3);
        const int k = kk * 16 + 8 * (G >> 1) + (q >> 2);
        typedef short v4s __attribute__((ext_vector_type(4)));
        const char* base = reinterpret_cast<const char*>(t);
        const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) v4s*)(base + Stage<BK>::mn_offset(k, r)));
        const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) v4s*)(base + Stage<BK>::mn_offset(k + 4, r)));
        const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
        return make_uint4(a.x, a.y, b.x, b.y);
    }
}

// Column of partial p's row in the log-sum-exp partial layout: rows XOR p % 32
// (32 writing lanes, one row: distinct banks), and the four 32-partial shares
// of a row, read at once by the row's four merging threads, moved apart by
// 4 (p / 32) (16 lanes of four rows: distinct banks).
__device__ __forceinline__ int part_swizzle(int p) { return (p & 31) ^ ((p >> 5) << 2); }

// The value of the neighbouring lane (lane ^ 1), by a DPP quad permute [1, 0, 3, 2].
__device__ __forceinline__ float swap_pair(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));
}

// The value of lane ^ X within a quad (X = 1: permute [1, 0, 3, 2]; X = 2: [2, 3, 0, 1]).
template <int X>
__device__ __forceinline__ float quad_xor(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), X == 1 ? 0xB1 : 0x4E, 0xF, 0xF, false));
}

// What a sum of exponentials counts from, given its largest term (by fmaxf, which passes over NaN): that term, or 0
// where it is -inf, so that terms of -inf add 0 and a NaN among them stays one.
__device__ __forceinline__ float sum_from(float top) { return top == -__builtin_inff() ? 0.0f : top; }

// XCD-aware tile order: consecutive block indices go to different XCDs, so
// XCD x (block % 8) takes a contiguous run of the (split, tile) pairs, split
// slowest (a split-K product gives each split's tiles to whole XCDs).
// Within the run, tiles come in groups of kTileGroupM M tiles by all N
// tiles, M varying fastest inside a group: the 32 tiles an XCD runs at once
// form a 4 x 8 block that shares 4 A panels and 8 B panels in its L2 (M
// fastest over the whole range would, for a tall product, put 32 A panels
// beside one B panel).  b is the linear block index over splits blocks of
// tiles_m * tiles_n.
constexpr uint32_t kTileGroupM = 4;
__device__ __forceinline__ void tile_of(uint32_t b, uint32_t tiles_m, uint32_t tiles_n, uint32_t splits, uint32_t& tm,
                                        uint32_t& tn, uint32_t& split) {
    const uint32_t T = tiles_m * tiles_n, all = T * splits;
    const uint32_t x = b & 7u, idx = b >> 3;
    const uint32_t q = all >> 3, r = all & 7u;
    const uint32_t v = (x < r ? x * (q + 1u) : r * (q + 1u) + (x - r) * q) + idx;
    split = v / T;
    const uint32_t t = v % T;
    const uint32_t group = t / (kTileGroupM * tiles_n), in = t % (kTileGroupM * tiles_n);
    const uint32_t m_first = group * kTileGroupM;
    const uint32_t rows = tiles_m - m_first < kTileGroupM ? tiles_m - m_first : kTileGroupM;
    tm = m_first + in % rows;
    tn = in / rows;
}

}  // namespace

}  // namespace rlpl
