// Softmax cross entropy of an output projection over a large vocabulary on
// gfx950, with its gradients, in pieces of the vocabulary: up to 2^27 logits are
// held in float32, one piece's worth.  For the rows i whose target y_i is not ignored (N of them),
//
//   z_i = hidden_i . weight^T + bias,   lse_i = log sum_v exp(z_iv)
//   loss = s sum_i (lse_i - z_i[y_i] + c lse_i^2),   s = 1 / max(N, 1) or 1
//   dz_iv = s ((1 + 2 c lse_i) exp(z_iv - lse_i) - [v == y_i])
//   d hidden = dz . weight,  d weight = dz^T . hidden,  d bias = sum_i dz_i
//
// Rows that are ignored cost nothing: a scan lists the others and their hidden
// states are copied side by side, the number N stays on the device, and tiles
// past it end at once.
//
// Loss: each 256 x 256 tile of logits is reduced in registers to its rows'
// (max, sum exp) and target logit; one kernel joins a row's tiles.  Gradient,
// per piece of the vocabulary: dz goes to the workspace in the operand dtype,
// from the float32 logits that the loss's pass left of the first columns, or from logits
// formed again (n x V of them would take 4 bytes each), and two products take
// it from there.  The weight's gradient of a piece comes out whole, so it is rounded once and written once;
// the hidden states' is summed over the pieces in float32.
//
// dz is formed without s and, in fp16, held at a scale that z_loss alone decides
// (ce_kernels.h; without a penalty its largest value is about 1): s would push a
// long batch's small probabilities under fp16's range.  Both factors are applied
// to the float32 results.
//
// What bounds it: the products, 6 n H V operations (8 where logits are formed
// again), where n is large.  In them a tile's ends: its ring leaves a compute
// unit no second workgroup to cover its first copies and its epilogue, 13 us by
// the fit of train_abi.cpp beside 1.1 a step of K (the weight's product over 1024
// rows has 16 steps).  Within the steps the port of LDS: a step of 64 of K over a
// 256 x 256 tile has 2048 cycles of matrix instructions; its fragment reads take
// 1573 alone and its copies 1863, both 2575 together, the step 2860 (8192^3, 1.37
// PFLOP/s, where the library's product by tiles of this size reaches 1.61; 1.22
// at 1024 x 4096 x 128256).  Few rows are bound by the weight's bytes: 16 rows of
// 4096 x 128256 read it at 4.4 to 5.5 TB/s (logits 190 to 237 us), and write its
// gradient beside (483 to 525).
//
// The contraction and its tiles are those of mfma_tile.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ce_kernels.h"
#include "device_common.h"
#include "loss_kernels.h"
#include "mfma_tile.h"
#include "row_io.h"

namespace rlpl {

namespace {

// A wavefront's 128 x 64 block as 8 x 4 tiles of v_mfma_f32_16x16x32: at random operands, which hold the
// chip to its power, it reaches 2.04 PFLOP/s from registers against 1.82 for 32x32x16 (a loop of
// matrix instructions alone), at 2.05 against 1.80 GHz.
typedef float floatx4 __attribute__((ext_vector_type(4)));

template <typename T>
__device__ __forceinline__ floatx4 mfma16(uint4 a, uint4 b, floatx4 c) {
    if constexpr (sizeof(T) == 2 && std::is_same_v<T, __bf16>)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                       0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Stages as in mfma_tile.h, but for the MN-contiguous operand's swizzle: a pass of 32 lanes reads 16
// columns of K rows k .. k + 3 and k + 8 .. k + 11, which bits 1 and 3 of k spread over all banks.
struct CeStage : Stage<kGemmBK> {
    static __device__ __forceinline__ int mn_swizzle(int k) { return (((k >> 1) & 1) << 2) | (((k >> 3) & 1) << 1); }
    static __device__ __forceinline__ int mn_offset(int k, int r) {
        return (r >> 6) * (128 * kGemmBK) + k * 128 + 16 * (((r & 63) >> 3) ^ mn_swizzle(k)) + 2 * (r & 7);
    }
};

// The fragments are read by asm statements that wait for their own reads: for a load or a builtin the compiler
// would add a wait for every copy into LDS in flight.

// Fragments of a K-contiguous stage tile: lane l's eight K values 32 half + 8 (l / 16) .. + 8 of row l % 16 of
// 16-row tiles, 2048 bytes apart.  k_base is the lane's place for the first of them.
__device__ __forceinline__ uint32_t lds_address(const char* p) {
    return uint32_t(uintptr_t((const __attribute__((address_space(3))) char*)p));
}
__device__ __forceinline__ uint32_t k_base(const char* t, int first, int half, int lane) {
    return lds_address(t + CeStage::kc_offset(first + (lane & 15), half * 4 + (lane >> 4)));
}
// Four tiles from each of two places.
__device__ __forceinline__ void fragments_k(uint32_t at0, uint32_t at1, uint4 (&x)[4], uint4 (&y)[4]) {
    u32x4 v[8];
    asm volatile(
        "ds_read_b128 %0, %8\n\tds_read_b128 %1, %8 offset:2048\n\t"
        "ds_read_b128 %2, %8 offset:4096\n\tds_read_b128 %3, %8 offset:6144\n\t"
        "ds_read_b128 %4, %9\n\tds_read_b128 %5, %9 offset:2048\n\t"
        "ds_read_b128 %6, %9 offset:4096\n\tds_read_b128 %7, %9 offset:6144\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
        : "v"(at0), "v"(at1)
        : "memory");
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        x[c] = __builtin_bit_cast(uint4, v[c]);
        y[c] = __builtin_bit_cast(uint4, v[4 + c]);
    }
}
// From each of four places.
__device__ __forceinline__ void fragments_k(uint32_t at0, uint32_t at1, uint32_t at2, uint32_t at3, uint4 (&x)[4],
                                            uint4 (&y)[4], uint4 (&z)[4], uint4 (&w)[4]) {
    u32x4 v[16];
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
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        x[c] = __builtin_bit_cast(uint4, v[c]);
        y[c] = __builtin_bit_cast(uint4, v[4 + c]);
        z[c] = __builtin_bit_cast(uint4, v[8 + c]);
        w[c] = __builtin_bit_cast(uint4, v[12 + c]);
    }
}

// Fragments of an MN-contiguous stage tile, by transposing reads: in a group of 16 lanes, lane q = 4j + c
// points at K row j, columns 4c .. 4c + 3, and lane i gets the four K rows of column i.  `mn_base` is the
// lane's place for the 16 columns 16 c (c < 4) of a block of 64; the eight fragments are those columns at
// byte offsets FIRST and SECOND (blocks are 8192 bytes apart, halves of K 4096).
__device__ __forceinline__ uint32_t mn_base(const char* t, int c, int lane) {
    const int q = lane & 15, r = 16 * c + 4 * (q & 3), k = 8 * (lane >> 4) + (q >> 2);
    return lds_address(t + CeStage::mn_offset(k, r));
}
template <int FIRST, int SECOND>
__device__ __forceinline__ void fragments_mn(const uint32_t (&at)[4], uint4 (&first)[4], uint4 (&second)[4]) {
    uint2 v[16];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %16 offset:%20\n\tds_read_b64_tr_b16 %1, %16 offset:%21\n\t"
        "ds_read_b64_tr_b16 %2, %17 offset:%20\n\tds_read_b64_tr_b16 %3, %17 offset:%21\n\t"
        "ds_read_b64_tr_b16 %4, %18 offset:%20\n\tds_read_b64_tr_b16 %5, %18 offset:%21\n\t"
        "ds_read_b64_tr_b16 %6, %19 offset:%20\n\tds_read_b64_tr_b16 %7, %19 offset:%21\n\t"
        "ds_read_b64_tr_b16 %8, %16 offset:%22\n\tds_read_b64_tr_b16 %9, %16 offset:%23\n\t"
        "ds_read_b64_tr_b16 %10, %17 offset:%22\n\tds_read_b64_tr_b16 %11, %17 offset:%23\n\t"
        "ds_read_b64_tr_b16 %12, %18 offset:%22\n\tds_read_b64_tr_b16 %13, %18 offset:%23\n\t"
        "ds_read_b64_tr_b16 %14, %19 offset:%22\n\tds_read_b64_tr_b16 %15, %19 offset:%23\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7]),
          "=&v"(v[8]), "=&v"(v[9]), "=&v"(v[10]), "=&v"(v[11]), "=&v"(v[12]), "=&v"(v[13]), "=&v"(v[14]), "=&v"(v[15])
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(FIRST), "n"(FIRST + 512), "n"(SECOND), "n"(SECOND + 512)
        : "memory");
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        first[c] = make_uint4(v[2 * c].x, v[2 * c].y, v[2 * c + 1].x, v[2 * c + 1].y);
        second[c] = make_uint4(v[8 + 2 * c].x, v[8 + 2 * c].y, v[9 + 2 * c].x, v[9 + 2 * c].y);
    }
}

// The same from half a block of 64 columns, and from two 16-row tiles, for the small tile: both halves of K.
__device__ __forceinline__ void fragments_k2(uint32_t at0, uint32_t at1, uint4 (&x)[2], uint4 (&y)[2]) {
    u32x4 v[4];
    asm volatile(
        "ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:2048\n\t"
        "ds_read_b128 %2, %5\n\tds_read_b128 %3, %5 offset:2048\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3])
        : "v"(at0), "v"(at1)
        : "memory");
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        x[c] = __builtin_bit_cast(uint4, v[c]);
        y[c] = __builtin_bit_cast(uint4, v[2 + c]);
    }
}
__device__ __forceinline__ void fragments_mn2(uint32_t at0, uint32_t at1, uint4 (&x)[2], uint4 (&y)[2]) {
    uint2 v[8];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8\n\tds_read_b64_tr_b16 %1, %8 offset:512\n\t"
        "ds_read_b64_tr_b16 %2, %9\n\tds_read_b64_tr_b16 %3, %9 offset:512\n\t"
        "ds_read_b64_tr_b16 %4, %8 offset:4096\n\tds_read_b64_tr_b16 %5, %8 offset:4608\n\t"
        "ds_read_b64_tr_b16 %6, %9 offset:4096\n\tds_read_b64_tr_b16 %7, %9 offset:4608\n\ts_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
        : "v"(at0), "v"(at1)
        : "memory");
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        x[c] = make_uint4(v[2 * c].x, v[2 * c].y, v[2 * c + 1].x, v[2 * c + 1].y);
        y[c] = make_uint4(v[4 + 2 * c].x, v[4 + 2 * c].y, v[5 + 2 * c].x, v[5 + 2 * c].y);
    }
}

// The shapes of a tile (ce_kernels.h says which a launch takes), as wavefronts along M and N, and their rings:
// three slots of the A operand's stages and two of the B operand's, all of a compute unit's LDS; or two of both, so that
// five workgroups fit one (16 rows of 4096 x 128256, all products by this tile and the logits formed twice: 905 us,
// against 1001 with three slots and 1110 with four); or four, where a launch has no more workgroups than those.
template <int BM_, int BN_, int WAVES_M, int WAVES_N, int SLOTS_A, int SLOTS_B>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, kWavesM = WAVES_M, kWavesN = WAVES_N;
    static constexpr int kWaves = WAVES_M * WAVES_N, kThreads = 64 * kWaves;
    static constexpr int kWaveM = BM / WAVES_M, kWaveN = BN / WAVES_N;
    static constexpr int kRowTiles = kWaveM / 16, kColTiles = kWaveN / 16;
    static constexpr int kBytesA = BM * kGemmBK * 2, kBytesB = BN * kGemmBK * 2;   // of a stage
    static constexpr int kSlotsA = SLOTS_A, kSlotsB = SLOTS_B;
    static constexpr int kLds = kSlotsA * kBytesA + kSlotsB * kBytesB;
    static constexpr int kCopies = kBytesA / 1024 / kWaves;   // 1 KB copies of a wavefront per operand and stage
    static_assert(BM == BN && kCopies * kWaves * 1024 == kBytesA, "whole copies, alike for both operands");
};
using Large = Shape<256, 256, 2, 4, 3, 2>;
using Small = Shape<64, 64, 2, 2, 2, 2>;
using Deep = Shape<64, 64, 2, 2, 4, 4>;
static_assert(Deep::kLds == kCeDeepLds, "as launched");
static_assert(Large::BM == kCeLarge.tile && Large::kThreads == kCeLarge.threads && Large::kLds == kCeLarge.lds, "as launched");
static_assert(Small::BM == kCeSmall.tile && Small::kThreads == kCeSmall.threads && Small::kLds == kCeSmall.lds, "as launched");
static_assert(Large::kWaveM == 128 && Large::kWaveN == 64 && Small::kWaveM == 32 && Small::kWaveN == 32 && kGemmBK == 64,
              "the places that the fragments are read at");

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

// A tile of 16-bit results in LDS: rows whose 32-byte pieces are swizzled by bits 0, 2 and 3 of the row (a
// wavefront writes such a piece of eight rows at once).
template <typename S> constexpr int kTileBytes = S::BM * S::BN * 2;
template <typename S>
__device__ __forceinline__ int tile_at(int row, int byte) {
    return row * (2 * S::BN) + (byte ^ ((((row & 1) | ((row >> 1) & 6)) << 5) & (2 * S::BN - 1)));
}

// The accumulators, rounded, into the tile: lanes 2c and 2c + 1 (adjacent columns) swap one value, so that
// each writes two adjacent columns of one row as 32 bits.
template <typename T, typename S, typename Row, typename Col, typename Value>
__device__ __forceinline__ void stage_tile(char* tile, int lane, Row row_of, Col col_of, Value value) {
    const int odd = lane & 1;
#pragma unroll
    for (int i = 0; i < S::kRowTiles; ++i)
#pragma unroll
        for (int e = 0; e < 4; e += 2)
#pragma unroll
            for (int j = 0; j < S::kColTiles; ++j) {
                const float a = value(i, j, e), b = value(i, j, e + 1);
                const float got = swap_pair(odd ? a : b);
                *reinterpret_cast<uint32_t*>(tile + tile_at<S>(row_of(i) + e + odd, 2 * (col_of(j) - odd))) =
                    Elem<T>::pack(odd ? got : a, odd ? b : got);
            }
}

// The tile's rows below M and columns below N (a multiple of 8) to memory, 16 bytes a lane.
template <typename T, typename S>
__device__ __forceinline__ void store_tile(const char* tile, T* out, int64_t ld, int m0, int M, int n0, int N) {
    constexpr int kLanes = S::BN / 8;      // lanes a row
    const int c = threadIdx.x % kLanes, col = n0 + 8 * c;
#pragma unroll 4
    for (int r = threadIdx.x / kLanes; r < S::BM; r += S::kThreads / kLanes)
        if (m0 + r < M && col < N)
            *reinterpret_cast<u32x4*>(out + int64_t(m0 + r) * ld + col) =
                *reinterpret_cast<const u32x4*>(tile + tile_at<S>(r, 16 * c));
}

}  // namespace

__device__ __forceinline__ void keep_row(const CePrepareArgs& a, int64_t row, int place, int64_t target) {
    a.row[place] = int(row);
    a.target[place] = target >= 0 && target < a.vocab ? int(target) : -1;
}
__device__ __forceinline__ void copy_row(const CePrepareArgs& a, int64_t row, int place) {
    const int words = a.cols / 8;
    const u32x4* from = reinterpret_cast<const u32x4*>(a.hidden) + row * words;
    u32x4* to = reinterpret_cast<u32x4*>(a.out) + int64_t(place) * words;
    for (int i = threadIdx.x; i < words; i += kCeThreads) to[i] = from[i];
}

// A workgroup a row: its place is the number of kept rows before it.
__global__ void __launch_bounds__(kCeThreads) ce_prepare(const CePrepareArgs a) {
    __shared__ uint32_t red[kCeThreads / 64];
    const int row = blockIdx.x;
    uint32_t before = 0;
    for (int i = threadIdx.x; i < row; i += kCeThreads) before += a.targets[i] != a.ignore_index;
    const int place = int(block_sum(before, red));
    const int64_t target = a.targets[row];
    const bool kept = target != a.ignore_index;
    if (threadIdx.x == 0) {
        a.place[row] = kept ? place : -1;
        if (kept) keep_row(a, row, place, target);
        if (row == a.n - 1) *a.state = CeState{place + (kept ? 1 : 0), 0.0f, 1u, 0u};
    }
    if (kept) copy_row(a, row, place);
}

// One workgroup scans the targets, eight consecutive ones a lane.
__global__ void __launch_bounds__(kCeCompactThreads) ce_compact(const CePrepareArgs a) {
    __shared__ int sums[kCeCompactThreads / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int base = 0;
    for (int64_t i0 = 0; i0 < a.n; i0 += 8 * kCeCompactThreads) {
        const int64_t i = i0 + 8 * int64_t(threadIdx.x);
        int64_t t[8];
        int mine = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            t[k] = i + k < a.n ? a.targets[i + k] : a.ignore_index;
            mine += t[k] != a.ignore_index;
        }
        int before = mine;                 // inclusive scan over the wavefront
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(before, off, 64);
            before += lane >= off ? v : 0;
        }
        __syncthreads();                   // sums may still be read
        if (lane == 63) sums[wave] = before;
        __syncthreads();
        int total = 0, waves_before = 0;
#pragma unroll
        for (int w = 0; w < kCeCompactThreads / 64; ++w) {
            waves_before += w < wave ? sums[w] : 0;
            total += sums[w];
        }
        int k0 = base + waves_before + before - mine;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (i + k >= a.n) continue;
            const bool kept = t[k] != a.ignore_index;
            a.place[i + k] = kept ? k0 : -1;
            if (kept) keep_row(a, i + k, k0++, t[k]);
        }
        base += total;
    }
    if (threadIdx.x == 0) *a.state = CeState{base, 0.0f, 1u, 0u};
}

__global__ void __launch_bounds__(kCeThreads) ce_gather(const CePrepareArgs a) {
    const int count = a.state->count;
    for (int k = blockIdx.x; k < count; k += gridDim.x) copy_row(a, a.row[k], k);
}

// The first columns' logits are kept as the lanes hold them: 16 x 16 blocks of 64 lanes' four values, a wavefront's
// columns side by side, rows in blocks of 16 after one another, for as many columns as there is room for with M rows.
// col: of the tile, from the vocabulary's start.
template <typename S>
__device__ __forceinline__ bool is_kept(const CeGemmArgs& g, int M, int col) {
    return g.kept && col + S::BN <= int(min(g.kept_room / uint32_t((M + 15) / 16), 1u << 14)) * 256;
}
template <typename S>
__device__ __forceinline__ float* kept_at(const CeGemmArgs& g, int M, int m0, int col, int wm, int wn, int i, int lane) {
    const int64_t rows = int64_t(col / S::kWaveN + wn) * ((M + 15) / 16) + (m0 + wm * S::kWaveM) / 16 + i;
    return g.kept + rows * (S::kColTiles * 256) + 4 * lane;
}

__device__ __forceinline__ int32_t ce_k_split(int32_t split_k, uint32_t splits) {
    const int32_t steps = (split_k + kGemmBK - 1) / kGemmBK;
    return (steps + int32_t(splits) - 1) / int32_t(splits) * kGemmBK;
}

// One tile of a product: workgroup `block` of those the launch has for it.  A_KCONTIG, B_KCONTIG: the operands'
// layouts (mfma_tile.h).
template <typename T, typename S, int PRODUCT, bool A_KCONTIG, bool B_KCONTIG>
__device__ __forceinline__ void ce_tile(const CeGemmArgs& g, const uint32_t block) {
    extern __shared__ __attribute__((aligned(1024))) char ring[];
    constexpr int BK = kGemmBK;

    const int count = g.state->count;
    const int M = PRODUCT == kCeWeight ? g.M : min(g.M, count);
    const int K = PRODUCT == kCeWeight ? min(g.K, count) : g.K;
    const uint32_t tiles_m = uint32_t(M + S::BM - 1) / uint32_t(S::BM);
    const uint32_t splits = PRODUCT == kCeHidden ? g.state->splits : 1u;
    if (block >= tiles_m * g.tiles_n * splits) return;     // the launch was sized for every row
    uint32_t tm, tn, split;
    tile_of(block, tiles_m, g.tiles_n, splits, tm, tn, split);
    const int m0 = int(tm) * S::BM, n0 = int(tn) * S::BN;
    if (PRODUCT == kCeDlogits && is_kept<S>(g, M, g.first + n0)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / S::kWavesN, wn = wave % S::kWavesN;
    const int k_split = PRODUCT == kCeHidden ? ce_k_split(g.split_k, splits) : K;
    const int kb = int(split) * k_split, ke = min(K, kb + k_split);
    if (PRODUCT == kCeHidden && g.accumulate && kb >= ke) return;   // a short last piece adds nothing to this plane
    const uint16_t* __restrict__ A = static_cast<const uint16_t*>(g.a);
    const uint16_t* __restrict__ B = static_cast<const uint16_t*>(g.b);

    // Accumulator element e of tile (i, j) is the workgroup tile's row row_of(i) + e and column col_of(j).
    auto row_of = [&](int i) { return wm * S::kWaveM + i * 16 + 4 * (lane >> 4); };
    auto col_of = [&](int j) { return wn * S::kWaveN + j * 16 + (lane & 15); };

    floatx4 acc[S::kRowTiles][S::kColTiles];
#pragma unroll
    for (int i = 0; i < S::kRowTiles; ++i)
#pragma unroll
        for (int j = 0; j < S::kColTiles; ++j) acc[i][j] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    const int nst = kb < ke ? (ke - kb + BK - 1) / BK : 0;
    // Byte offsets of this lane's 16-byte pieces of the wavefront's copies, from an operand's tile at any stage.
    uint32_t off_a[S::kCopies], off_b[S::kCopies];
#pragma unroll
    for (int u = 0; u < S::kCopies; ++u) {
        off_a[u] = dma_source<A_KCONTIG, BK, CeStage>(wave * S::kCopies + u, lane, uint32_t(g.lda), M, INT32_MAX, m0, 0);
        off_b[u] = dma_source<B_KCONTIG, BK, CeStage>(wave * S::kCopies + u, lane, uint32_t(g.ldb), g.N, INT32_MAX, n0, 0);
    }
    // The wavefront's copies of an operand's stage s into its ring; the last stage's K past ke read as zeros.
    auto issue = [&](auto kcontig, const uint16_t* x, int64_t ld, int first, int R, const uint32_t (&off)[S::kCopies], int s,
                     char* to) {
        const int k0 = kb + s * BK;
        const __amdgpu_buffer_rsrc_t from =
            buffer_at(x + (kcontig ? int64_t(first) * ld + k0 : int64_t(k0) * ld + first));
#pragma unroll
        for (int u = 0; u < S::kCopies; ++u) {
            const int q = wave * S::kCopies + u;
            const uint32_t o =
                k0 + BK <= ke ? off[u] : dma_source<kcontig, BK, CeStage>(q, lane, uint32_t(ld), R, ke, first, k0);
            dma16(from, o, to + q * 1024);
        }
    };
    char* const ring_b = ring + S::kSlotsA * S::kBytesA;
    auto issue_a = [&](int s) {
        if (s < nst)
            issue(std::integral_constant<bool, A_KCONTIG>(), A, g.lda, m0, M, off_a, s, ring + s % S::kSlotsA * S::kBytesA);
    };
    auto issue_b = [&](int s) {
        if (s < nst)
            issue(std::integral_constant<bool, B_KCONTIG>(), B, g.ldb, n0, g.N, off_b, s, ring_b + s % S::kSlotsB * S::kBytesB);
    };
    auto stage_a = [&](int s) { return ring + s % S::kSlotsA * S::kBytesA; };
    auto stage_b = [&](int s) { return ring_b + s % S::kSlotsB * S::kBytesB; };
    if constexpr (S::BM == 64) {
        // One barrier a step: once stage s has landed and every wavefront is done with s - 1, the stage that is
        // kAhead further goes to that one's slot.
        constexpr int kAhead = S::kSlotsA - 1;
        static_assert(S::kSlotsA == S::kSlotsB && kAhead >= 1 && kAhead <= 3, "the waits below");
        uint4 af[2][2], bf[2][2];          // [half of K][tile]
        for (int s = 0; s < kAhead; ++s) {
            issue_a(s);
            issue_b(s);
        }
        for (int s = 0; s < nst; ++s) {
            if (kAhead >= 3 && s + 2 < nst) wait_copies<4 * S::kCopies>();
            else if (kAhead >= 2 && s + 1 < nst) wait_copies<2 * S::kCopies>();
            else wait_copies<0>();
            meet();
            issue_a(s + kAhead);
            issue_b(s + kAhead);
            if constexpr (A_KCONTIG)
                fragments_k2(k_base(stage_a(s), wm * S::kWaveM, 0, lane), k_base(stage_a(s), wm * S::kWaveM, 1, lane), af[0],
                             af[1]);
            else
                fragments_mn2(mn_base(stage_a(s), 2 * wm, lane), mn_base(stage_a(s), 2 * wm + 1, lane), af[0], af[1]);
            if constexpr (B_KCONTIG)
                fragments_k2(k_base(stage_b(s), wn * S::kWaveN, 0, lane), k_base(stage_b(s), wn * S::kWaveN, 1, lane), bf[0],
                             bf[1]);
            else
                fragments_mn2(mn_base(stage_b(s), 2 * wn, lane), mn_base(stage_b(s), 2 * wn + 1, lane), bf[0], bf[1]);
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) acc[i][j] = mfma16<T>(af[half][i], bf[half][j], acc[i][j]);
        }
    } else {
        uint4 af[2][S::kRowTiles / 2], bf[2][S::kColTiles];
        auto read_a = [&](int s, auto half) {  // the fragments of 32 of stage s's K
            if constexpr (A_KCONTIG) {
                const uint32_t at = k_base(stage_a(s), wm * S::kWaveM, half, lane);
                fragments_k(at, at + 8192, af[0], af[1]);
            } else {
                uint32_t at[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) at[c] = mn_base(stage_a(s) + wm * 2 * 8192, c, lane);
                fragments_mn<4096 * half, 8192 + 4096 * half>(at, af[0], af[1]);
            }
        };
        auto read_b = [&](int s) {             // of all of it
            if constexpr (B_KCONTIG) {
                fragments_k(k_base(stage_b(s), wn * S::kWaveN, 0, lane), k_base(stage_b(s), wn * S::kWaveN, 1, lane), bf[0], bf[1]);
            } else {
                uint32_t at[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) at[c] = mn_base(stage_b(s) + wn * 8192, c, lane);
                fragments_mn<0, 4096>(at, bf[0], bf[1]);
            }
        };
        auto multiply = [&](auto half) {
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int i = 0; i < S::kRowTiles; ++i)
#pragma unroll
                for (int j = 0; j < S::kColTiles; ++j) acc[i][j] = mfma16<T>(af[i / 4][i % 4], bf[half][j], acc[i][j]);
            __builtin_amdgcn_s_setprio(0);
        };
        const std::integral_constant<int, 0> lower{};
        const std::integral_constant<int, 1> upper{};
        // Stage s has landed once only the copies of stage s + 1 are in flight.
        auto wait_stage = [&](int s) {
            if (s + 1 < nst) wait_copies<2 * S::kCopies>();
            else wait_copies<0>();
        };
        // A step in four turns, each ended by the workgroup's barrier: fragments of half a stage, their matrix
        // instructions, and the same for the other half.  The wavefronts of the tile's lower half (one on
        // each SIMD, as those of the upper) run one turn behind, so that one group reads LDS while the other
        // multiplies.  Copies run two stages ahead: stage s + 2 of A goes to the slot that stage s - 1 left,
        // that of B to stage s's own, whose fragments are all in registers after the step's first two turns.
        if (nst > 0) {
            issue_a(0);
            issue_b(0);
            issue_a(1);
            issue_b(1);
            wait_stage(0);
            meet();
            if (wm == 1) meet();
            for (int s = 0; s < nst; ++s) {
                issue_a(s + 2);
                if constexpr (A_KCONTIG && B_KCONTIG) {
                    const uint32_t at = k_base(stage_a(s), wm * S::kWaveM, 0, lane);
                    fragments_k(at, at + 8192, k_base(stage_b(s), wn * S::kWaveN, 0, lane),
                                k_base(stage_b(s), wn * S::kWaveN, 1, lane), af[0], af[1], bf[0], bf[1]);
                } else {
                    read_b(s);
                    read_a(s, lower);
                }
                meet();
                multiply(lower);
                meet();
                issue_b(s + 2);
                read_a(s, upper);
                if (wm == 1) wait_stage(s + 1);
                meet();
                multiply(upper);
                if (wm == 0) wait_stage(s + 1);
                meet();
            }
            if (wm == 0) meet();
        }
    }
    __syncthreads();                       // the ring is free

    if constexpr (PRODUCT == kCeHidden || PRODUCT == kCeWeight) {
        const bool f32 = PRODUCT == kCeHidden || g.out_f32;
        const float scale = PRODUCT == kCeHidden ? 1.0f : g.state->scale;
        if (f32) {
            float* __restrict__ C = static_cast<float*>(g.c);
            if (PRODUCT == kCeHidden) C += int64_t(split) * g.N * M;
            // Up to 128 of the tile's rows at a time through LDS, so that every access is 16 bytes of whole rows.
            constexpr int kRows = S::BM < 128 ? S::BM : 128, kLanes = S::BN / 4;
            const auto at = [](int r, int byte) { return r * (4 * S::BN) + (byte ^ (((r >> 2) & 3) << 6)); };
            for (int r0 = 0; r0 < S::BM; r0 += kRows) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < S::kRowTiles; ++i) {
                    const int r = row_of(i) - r0;
                    if (r < 0 || r >= kRows) continue;
#pragma unroll
                    for (int j = 0; j < S::kColTiles; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<float*>(ring + at(r + e, 4 * col_of(j))) = acc[i][j][e] * scale;
                }
                __syncthreads();
                const int c = threadIdx.x % kLanes, col = n0 + 4 * c;
                for (int r = threadIdx.x / kLanes; r < kRows; r += S::kThreads / kLanes) {
                    const int row = m0 + r0 + r;
                    if (row >= M || col >= g.N) continue;
                    float v[4];
                    load_row<4>(reinterpret_cast<const float*>(ring + at(r, 16 * c)), v);
                    float* to = C + int64_t(row) * g.ldc + col;
                    if (g.accumulate) {
                        float old[4];
                        load_row<4>(static_cast<const float*>(to), old);
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] += old[k];
                    }
                    store_row<4>(to, v);
                }
            }
            return;
        }
        stage_tile<T, S>(ring, lane, row_of, col_of, [&](int i, int j, int e) { return acc[i][j][e] * scale; });
        __syncthreads();
        store_tile<T, S>(ring, static_cast<T*>(g.c), g.ldc, m0, M, n0, g.N);
        return;
    }

    // Logits: z = acc + bias; columns past N are -inf.
    const T* __restrict__ bias = static_cast<const T*>(g.bias);
#pragma unroll
    for (int j = 0; j < S::kColTiles; ++j) {
        const int col = n0 + col_of(j);
        const float b = col < g.N ? (bias ? to_f<T>(bias[col]) : 0.0f) : -__builtin_inff();
#pragma unroll
        for (int i = 0; i < S::kRowTiles; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] += b;
    }

    if (PRODUCT == kCeLogits && is_kept<S>(g, M, n0)) {
#pragma unroll
        for (int i = 0; i < S::kRowTiles; ++i) {
            if (m0 + wm * S::kWaveM + i * 16 >= M) break;
            float* to = kept_at<S>(g, M, m0, n0, wm, wn, i, lane);
#pragma unroll
            for (int j = 0; j < S::kColTiles; ++j) *reinterpret_cast<floatx4*>(to + 256 * j) = acc[i][j];
        }
    }

    if constexpr (PRODUCT == kCeDlogits) {
        float* row_lse = reinterpret_cast<float*>(ring + kTileBytes<S>);
        float* row_f = row_lse + S::BM;
        int* tgt_col = reinterpret_cast<int*>(row_f + S::BM);
        float(*sums)[S::BN] = reinterpret_cast<float(*)[S::BN]>(tgt_col + S::BM);
        if (int(threadIdx.x) < S::BM) {
            const int row = m0 + int(threadIdx.x);
            const float lse = row < M ? g.lse[row] : 0.0f;
            const int t = row < M ? g.target[row] - g.first - n0 : -1;
            row_lse[threadIdx.x] = lse;
            row_f[threadIdx.x] = row < M ? g.dz_scale * (1.0f + g.z_loss2 * lse) : 0.0f;
            tgt_col[threadIdx.x] = t >= 0 && t < S::BN && n0 + t < g.N ? t : -1;
        }
        __syncthreads();
        // rows past M have a factor of 0 and no target, columns past N a logit of -inf: exact zeros
#pragma unroll
        for (int i = 0; i < S::kRowTiles; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = row_of(i) + e;
                const float l = row_lse[r], f = row_f[r];
                const int tc = tgt_col[r];
#pragma unroll
                for (int j = 0; j < S::kColTiles; ++j) {
                    const float p = __builtin_amdgcn_exp2f((acc[i][j][e] - l) * kLog2eG);
                    acc[i][j][e] = (f != 0.0f ? f * p : 0.0f) - (col_of(j) == tc ? g.dz_scale : 0.0f);
                }
            }
        if (g.col_part) {
#pragma unroll
            for (int j = 0; j < S::kColTiles; ++j) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < S::kRowTiles; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s += acc[i][j][e];
                s += __shfl_xor(s, 16, 64);
                s += __shfl_xor(s, 32, 64);
                if (lane < 16) sums[wm][col_of(j)] = s;
            }
        }
        stage_tile<T, S>(ring, lane, row_of, col_of, [&](int i, int j, int e) { return acc[i][j][e]; });
        __syncthreads();
        // the piece's columns past N too: their zeros are the hidden product's K tail
        store_tile<T, S>(ring, static_cast<T*>(g.c), g.ldc, m0, M, n0, int(g.ldc));
        const int col = n0 + int(threadIdx.x);
        if (g.col_part && threadIdx.x < S::BN && col < g.N)
            g.col_part[int64_t(tm) * g.col_ld + col] = sums[0][threadIdx.x] + sums[1][threadIdx.x];
        return;
    }

    // kCeLogits: a lane reduces its columns of a row; the 16 partials a wavefront has of a row meet the others' in LDS,
    // laid out [partial][row ^ part_row(partial)] (writes and reads free of bank conflicts), and neighbouring lanes
    // merge a row.
    constexpr int kParts = S::kWavesN * 16;
    constexpr int kMerge = S::kThreads / S::BM;            // lanes that merge a row
    constexpr int kShare = kParts / kMerge;
    static_assert((kMerge == 2 || kMerge == 4) && kParts * S::BM * 8 + S::BM * 4 <= S::kLds, "the partials fit");
    const auto part_row = [](int p) { return ((p & 3) | ((p & 12) << 1)) ^ ((p >> 5) << 4); };
    float2* parts = reinterpret_cast<float2*>(ring);
    int* tgt_col = reinterpret_cast<int*>(parts + kParts * S::BM);
    if (threadIdx.x < S::BM) {
        const int row = m0 + int(threadIdx.x);
        const int t = row < M ? g.target[row] - n0 : -1;
        tgt_col[threadIdx.x] = t >= 0 && t < S::BN && n0 + t < g.N ? t : -1;
    }
    __syncthreads();
    const int pidx = wn * 16 + (lane & 15);
#pragma unroll
    for (int i = 0; i < S::kRowTiles; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = row_of(i) + e;
            float m = acc[i][0][e];
#pragma unroll
            for (int j = 1; j < S::kColTiles; ++j) m = fmaxf(m, acc[i][j][e]);
            const float from = sum_from(m);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < S::kColTiles; ++j) sum += __builtin_amdgcn_exp2f((acc[i][j][e] - from) * kLog2eG);
            parts[pidx * S::BM + (r ^ part_row(pidx))] = make_float2(m, sum);
            const int tc = tgt_col[r];
#pragma unroll
            for (int j = 0; j < S::kColTiles; ++j)
                if (col_of(j) == tc && m0 + r < M) g.target_logit[m0 + r] = acc[i][j][e];
        }
    __syncthreads();
    const int rr = threadIdx.x / kMerge, first = threadIdx.x % kMerge * kShare, row = m0 + rr;
    float top = -__builtin_inff();
#pragma unroll 8
    for (int p = first; p < first + kShare; ++p) top = fmaxf(top, parts[p * S::BM + (rr ^ part_row(p))].x);
    top = fmaxf(top, quad_xor<1>(top));
    if constexpr (kMerge == 4) top = fmaxf(top, quad_xor<2>(top));
    const float from = sum_from(top);
    float sum = 0.0f;
#pragma unroll 8
    for (int p = first; p < first + kShare; ++p) {
        const float2 v = parts[p * S::BM + (rr ^ part_row(p))];
        sum += v.y * __builtin_amdgcn_exp2f((v.x - from) * kLog2eG);
    }
    sum += quad_xor<1>(sum);
    if constexpr (kMerge == 4) sum += quad_xor<2>(sum);
    if (threadIdx.x % kMerge == 0 && row < M)
        reinterpret_cast<float2*>(g.part)[int64_t(row) * g.tiles_n + tn] = make_float2(top, sum);
}

// dz of a piece's tiles whose logits were kept, bit for bit what ce_tile forms: a workgroup a tile, a wavefront its
// own blocks of it, each turned to whole rows in a strip of LDS of its own (1024 x 128256: 150 us, 5.3 TB/s).
template <typename T, typename S>
__global__ void __launch_bounds__(S::kThreads) ce_dz(const CeGemmArgs g) {
    constexpr int kPitch = 2 * S::kWaveN + 16, kLanes = S::kWaveN / 8;      // bytes of a row in the strip, lanes of its store
    __shared__ __attribute__((aligned(16))) char strips[S::kWaves][16 * kPitch];
    __shared__ float sums[S::kWavesM][S::BN];
    const int M = min(g.M, g.state->count);
    const uint32_t tiles_m = uint32_t(M + S::BM - 1) / uint32_t(S::BM);
    if (blockIdx.x >= tiles_m * g.tiles_n) return;
    const uint32_t tm = blockIdx.x % tiles_m, tn = blockIdx.x / tiles_m;
    const int m0 = int(tm) * S::BM, n0 = int(tn) * S::BN;
    if (!is_kept<S>(g, M, g.first + n0)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / S::kWavesN, wn = wave % S::kWavesN, odd = lane & 1;
    char* strip = strips[wave];
    float sum[S::kColTiles] = {};
#pragma unroll 2
    for (int i = 0; i < S::kRowTiles; ++i) {
        const int row0 = m0 + wm * S::kWaveM + i * 16;
        if (row0 >= M) break;
        const float* from = kept_at<S>(g, M, m0, g.first + n0, wm, wn, i, lane);
        floatx4 z[S::kColTiles];
#pragma unroll
        for (int j = 0; j < S::kColTiles; ++j) z[j] = *reinterpret_cast<const floatx4*>(from + 256 * j);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = row0 + 4 * (lane >> 4) + e;
            const float lse = row < M ? g.lse[row] : 0.0f;
            const float f = row < M ? g.dz_scale * (1.0f + g.z_loss2 * lse) : 0.0f;
            const int target = row < M ? g.target[row] - g.first : -1;
#pragma unroll
            for (int j = 0; j < S::kColTiles; ++j) {
                const int col = n0 + wn * S::kWaveN + j * 16 + (lane & 15);
                const float p = __builtin_amdgcn_exp2f((z[j][e] - lse) * kLog2eG);
                z[j][e] = (f != 0.0f ? f * p : 0.0f) - (col == target && col < g.N ? g.dz_scale : 0.0f);
                sum[j] += z[j][e];
            }
        }
#pragma unroll
        for (int e = 0; e < 4; e += 2)
#pragma unroll
            for (int j = 0; j < S::kColTiles; ++j) {
                const float a = z[j][e], b = z[j][e + 1], got = swap_pair(odd ? a : b);
                *reinterpret_cast<uint32_t*>(strip + (4 * (lane >> 4) + e + odd) * kPitch + 32 * j + 2 * ((lane & 15) - odd)) =
                    Elem<T>::pack(odd ? got : a, odd ? b : got);
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int c = lane % kLanes;
#pragma unroll
        for (int r = lane / kLanes; r < 16; r += 64 / kLanes)
            if (row0 + r < M)
                *reinterpret_cast<u32x4*>(static_cast<T*>(g.c) + int64_t(row0 + r) * g.ldc + n0 + wn * S::kWaveN + 8 * c) =
                    *reinterpret_cast<const u32x4*>(strip + r * kPitch + 16 * c);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    if (!g.col_part) return;
#pragma unroll
    for (int j = 0; j < S::kColTiles; ++j) {
        float s = sum[j];
        s += __shfl_xor(s, 16, 64);
        s += __shfl_xor(s, 32, 64);
        if (lane < 16) sums[wm][wn * S::kWaveN + j * 16 + lane] = s;
    }
    __syncthreads();
    const int col = n0 + int(threadIdx.x);
    if (threadIdx.x < S::BN && col < g.N)
        g.col_part[int64_t(tm) * g.col_ld + col] = sums[0][threadIdx.x] + sums[1][threadIdx.x];
}

template <typename T, typename S, int PRODUCT>
__global__ void __launch_bounds__(S::kThreads, 2) ce_gemm(const CeGemmArgs g) {
    ce_tile<T, S, PRODUCT, true, true>(g, blockIdx.x);
}
template <typename T, typename S>
__global__ void __launch_bounds__(S::kThreads, 2) ce_grads(const CeGradArgs a) {
    if (blockIdx.x < a.hidden_blocks) ce_tile<T, S, kCeHidden, true, false>(a.hidden, blockIdx.x);
    else ce_tile<T, S, kCeWeight, false, false>(a.weight, blockIdx.x - a.hidden_blocks);
}

// The time, in quarters of a K step, of the hidden product over `count` rows with its K (the longest piece's) in s
// splits, beside the weight's product over the same rows where that is wanted.  Both products' workgroups
// share the chip, so there a split pays only where a workgroup alone would outlast all of them; by themselves, the hidden
// product's run in rounds.  6001 x 2048 x 50021 with half of the rows kept takes two splits (five, the best without
// the weight's product, made the call 2.25 ms instead of 1.95), 16 x 4096 x 128256 six (690 us; 1548 with two, 745 with 32).
__device__ __forceinline__ uint64_t split_time(const CeRowArgs& a, const CeShape& shape, uint32_t count, uint32_t s) {
    const uint64_t tiles = uint64_t((count + shape.tile - 1) / shape.tile) * a.tiles_h, at_once = shape.at_once;
    const uint32_t steps = uint32_t(a.split_k + kGemmBK - 1) / kGemmBK, row_steps = (count + kGemmBK - 1) / kGemmBK;
    const uint64_t one = 4 * ((steps + s - 1) / s) + uint32_t(shape.extra);
    const uint64_t weight = uint64_t(a.weight_tiles) * (4 * row_steps + uint32_t(shape.weight_extra));
    const uint64_t all = (tiles * s * one + weight) / at_once, rounds = (tiles * s + at_once - 1) / at_once * one;
    return (a.weight_tiles == 0 ? rounds : all > one ? all : one) +
           s * (uint32_t(shape.plane) + tiles / uint32_t(shape.plane_tiles));
}

// A wavefront joins a kept row's tiles (each lane's in order, then the lane tree).  The workgroup that is done last
// sums the rows' losses in double (each lane's in order, then a tree), whichever it is: the rows' losses are written to
// and read from memory past the caches that compute units do not share, each before its workgroup counts itself
// done.  At most 512 workgroups count (a count takes about 12 ns, one after the other).
__global__ void __launch_bounds__(kCeThreads) ce_row(const CeRowArgs a) {
    __shared__ double sums[kCeThreads];
    __shared__ bool last;
    const int count = a.state->count, lane = threadIdx.x & 63;
    for (int row = blockIdx.x * (kCeThreads / 64) + (threadIdx.x >> 6); row < count; row += gridDim.x * (kCeThreads / 64)) {
        const float2* p = reinterpret_cast<const float2*>(a.part) + int64_t(row) * a.tiles;
        float top = -__builtin_inff();
#pragma unroll 8
        for (int t = lane; t < a.tiles; t += 64) top = fmaxf(top, p[t].x);
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
        float s = 0.0f;
#pragma unroll 8
        for (int t = lane; t < a.tiles; t += 64) s += p[t].y * __builtin_amdgcn_exp2f((p[t].x - top) * kLog2eG);
        s = wave_sum(s);
        if (lane == 0) {
            const float lse = top + __builtin_amdgcn_logf(s) * 0.6931471805599453f;
            a.lse[row] = lse;
            const float loss =
                a.target[row] >= 0 ? lse - a.target_logit[row] + a.z_loss * lse * lse : __builtin_nanf("");
            __hip_atomic_store(a.row_loss + row, loss, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));      // it has reached memory
            asm volatile("" ::: "memory");
        }
    }
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(&a.state->done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
    __syncthreads();
    if (!last) return;
    if (threadIdx.x < 64) {                // lane l: the time of l + 1 splits; the least, and of equal ones the fewest splits
        const CeShape shape = a.small ? kCeSmall : kCeLarge;
        const uint32_t rows = uint32_t((count + shape.tile - 1) / shape.tile);
        uint64_t best = ~uint64_t(0);
        if (lane == 0 || (lane < a.most && rows * uint32_t(lane + 1) <= a.plane_rows))
            best = split_time(a, shape, uint32_t(count), uint32_t(lane + 1)) << 8 | uint32_t(lane + 1);
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            const uint64_t other = __shfl_xor(best, off, 64);
            best = other < best ? other : best;
        }
        if (lane == 0) a.state->splits = uint32_t(best & 0xFF);
    }
    double s = 0.0;
    for (int i = threadIdx.x; i < count; i += kCeThreads)
        s += double(__hip_atomic_load(a.row_loss + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    sums[threadIdx.x] = s;
    for (int half = kCeThreads / 2; half > 0; half >>= 1) {
        __syncthreads();
        if (int(threadIdx.x) < half) sums[threadIdx.x] += sums[threadIdx.x + half];
    }
    if (threadIdx.x == 0) {
        const double n = a.mean ? double(count > 1 ? count : 1) : 1.0;
        *a.loss = float(sums[0] / n);
        a.state->scale = float(double(a.inv_dz_scale) / n);
    }
}

template <typename T>
__global__ void __launch_bounds__(kCeThreads) ce_finish(const CeFinishArgs a) {
    const float scale = a.state->scale;
    const int count = a.state->count;
    if (blockIdx.x >= a.row_blocks) {
        const int tiles = (count + a.col_tile - 1) / a.col_tile;
        const int col = int(blockIdx.x - a.row_blocks) * kCeThreads + threadIdx.x;
        if (col >= a.vocab) return;
        float s = 0.0f;
#pragma unroll 4
        for (int t = 0; t < tiles; ++t) s += a.col_part[int64_t(t) * a.vocab + col];
        s *= scale;
        if (a.out_f32) {
            float* out = static_cast<float*>(a.bias) + col;
            *out = a.accumulate ? *out + s : s;
        } else {
            static_cast<T*>(a.bias)[col] = from_f<T>(s);
        }
        return;
    }
    const int64_t plane = int64_t(count) * a.cols;
    const int splits = int(a.state->splits);
    for (int row = blockIdx.x; row < a.n; row += a.row_blocks) {
        const int k = a.place[row];
        const int64_t at = int64_t(row) * a.cols;
        for (int c = threadIdx.x * 8; c < a.cols; c += kCeThreads * 8) {
            float v[8] = {};
            if (k >= 0) {
                const float* p = a.part + int64_t(k) * a.cols + c;
#pragma unroll 4
                for (int z = 0; z < splits; ++z) {
                    float x[8];
                    load_row<8>(p + z * plane, x);
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] += x[q];
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] *= scale;
            }
            if (a.hidden_f32) store_row<8>(static_cast<float*>(a.out) + at + c, v);
            else store_row<8>(static_cast<T*>(a.out) + at + c, v);
        }
    }
}

// ----------------------------------------------------------------------------- host-side table

template <typename T, typename S>
static const void* ce_gemm_for(int product) {
    switch (product) {
    case kCeLogits: return reinterpret_cast<const void*>(&ce_gemm<T, S, kCeLogits>);
    case kCeDlogits: return reinterpret_cast<const void*>(&ce_gemm<T, S, kCeDlogits>);
    }
    return nullptr;
}

const void* pick_ce_gemm(int dtype, bool small, int product) {
    switch (dtype) {
    case kF16: return small ? ce_gemm_for<_Float16, Small>(product) : ce_gemm_for<_Float16, Large>(product);
    case kBF16: return small ? ce_gemm_for<__bf16, Small>(product) : ce_gemm_for<__bf16, Large>(product);
    }
    return nullptr;
}
const void* pick_ce_deep_logits(int dtype) {
    return dtype == kF16 ? reinterpret_cast<const void*>(&ce_gemm<_Float16, Deep, kCeLogits>)
                         : reinterpret_cast<const void*>(&ce_gemm<__bf16, Deep, kCeLogits>);
}
const void* pick_ce_grads(int dtype, bool small) {
    if (dtype == kF16)
        return small ? reinterpret_cast<const void*>(&ce_grads<_Float16, Small>)
                     : reinterpret_cast<const void*>(&ce_grads<_Float16, Large>);
    return small ? reinterpret_cast<const void*>(&ce_grads<__bf16, Small>)
                 : reinterpret_cast<const void*>(&ce_grads<__bf16, Large>);
}
const void* pick_ce_dz(int dtype, bool small) {
    if (dtype == kF16)
        return small ? reinterpret_cast<const void*>(&ce_dz<_Float16, Small>)
                     : reinterpret_cast<const void*>(&ce_dz<_Float16, Large>);
    return small ? reinterpret_cast<const void*>(&ce_dz<__bf16, Small>) : reinterpret_cast<const void*>(&ce_dz<__bf16, Large>);
}
const void* ce_prepare_kernel() { return reinterpret_cast<const void*>(&ce_prepare); }
const void* ce_compact_kernel() { return reinterpret_cast<const void*>(&ce_compact); }
const void* ce_gather_kernel() { return reinterpret_cast<const void*>(&ce_gather); }
const void* ce_row_kernel() { return reinterpret_cast<const void*>(&ce_row); }
const void* pick_ce_finish(int dtype) {
    return dtype == kF16 ? reinterpret_cast<const void*>(&ce_finish<_Float16>)
                         : reinterpret_cast<const void*>(&ce_finish<__bf16>);
}

}  // namespace rlpl
