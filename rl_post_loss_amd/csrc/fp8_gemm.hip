// Products of 8-bit operands with block scales over whole tiles on gfx950 (the
// formula stands in fp8_kernels.hip, which has the product of few rows).
//
// A tile of vocabulary entries by tokens, K in stages of 128 bytes through a
// ring of LDS that buffer-to-LDS copies fill, as the cross entropy's tiles do
// (a row of a stage has the same 128 bytes): a stage is one block of the scales.
// A block's product starts from zero on the matrix cores (fp8_mfma.h); its four
// results a lane are added to the accumulators times the block's scale, four
// vector operations beside an instruction of 32 cycles.  The entries of a
// wavefront share one scale of the projection; a lane's token has one for each
// column tile.
//
// A lane of a fragment takes 16-byte pieces q and q + 4 of a row's 128 bytes
// (q = lane / 16) in both operands: which of K's elements meet is all that counts.
//
// Six shapes (score_abi.cpp chooses by a time model), entries by tokens.  256 x 256, the loop of
// the cross entropy's large tile: 1.03 ms for 2048 x 4096 x 128256 (2.1 PFLOP/s), 0.47
// for 8192^3 (2.3; the library's product with one scale for each operand 0.86 to 0.98 and
// 0.36 to 0.38 ms).  A step has 2048 cycles of matrix instructions (1.47 us alone, 1.7 to
// 2.05 with its share of a tile's ends).  64 x 64 and 128 x 128, five and two
// workgroups a compute unit, for fewer results: 333 x 2048 x 5003 11 us, 2048 x 4096
// x 4096 46 us (1.5 PFLOP/s).  The projection's ring has a third stage at 128 x 128, where
// it comes from memory: 128 x 4096 x 128256 136 us instead of 149 (4 TB/s).  128 x 64 with three stages
// of both operands for up to 128 rows of a long projection (128 x 8192 x 30000 57 us; 67 by 64 x 64, 81 by
// 128 x 128).  64 x 64 with K shared by four or two groups of wavefronts, for tiles too few to fill the
// chip: a step of a workgroup alone is bound by its instructions, not by its copies (more stages change
// nothing), and four groups take 1.1 us for four steps of 0.6.  float32 outputs: 8192^3 0.97 ms at 128 x 128
// (1.13 PFLOP/s of 16-bit instructions; 1.26 ms at 64 x 64, whose wavefronts convert twice as much for each product).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "device_common.h"
#include "fp8_kernels.h"
#include "fp8_mfma.h"
#include "loss_kernels.h"
#include "mfma_ring.h"
#include "mfma_tile.h"
#include "row_io.h"

namespace rlpl {

namespace {

// Entries (M) by tokens (N), wavefronts along each, slots of the ring; groups of wavefronts that have a share of K (and a
// ring) each.
template <int BM_, int BN_, int WAVES_M, int WAVES_N, int SLOTS_A, int SLOTS_B, int GROUPS = 1>
struct Fp8Shape {
    static constexpr int BM = BM_, BN = BN_, kWavesM = WAVES_M, kWavesN = WAVES_N, kGroups = GROUPS;
    static constexpr int kWaves = WAVES_M * WAVES_N, kThreads = 64 * kWaves * GROUPS;
    static constexpr int kWaveM = BM / WAVES_M, kWaveN = BN / WAVES_N;
    static constexpr int kRowTiles = kWaveM / 16, kColTiles = kWaveN / 16;
    static constexpr int kBytesA = BM * 128, kBytesB = BN * 128;
    static constexpr int kSlotsA = SLOTS_A, kSlotsB = SLOTS_B;
    static constexpr int kRing = kSlotsA * kBytesA + kSlotsB * kBytesB, kLds = kRing * GROUPS;
    static constexpr int kCopiesA = kBytesA / 1024 / kWaves, kCopiesB = kBytesB / 1024 / kWaves;   // of a wavefront and stage
    static_assert(kCopiesA * kWaves * 1024 == kBytesA && kCopiesB * kWaves * 1024 == kBytesB, "whole copies");
    static_assert(kCopiesA % 2 == 0 && kCopiesB % 2 == 0, "a wavefront's first copy is an even one");
    static_assert(kWaveM <= kFp8Group && kFp8Group % kWaveM == 0, "a wavefront's entries share a scale");
    static constexpr bool launched_as(const Fp8TileShape& s) {
        return BM == s.vocab && BN == s.tokens && kThreads == s.threads && kLds == s.lds;
    }
};
using Large = Fp8Shape<256, 256, 2, 4, 3, 2>;
using Middle = Fp8Shape<128, 128, 2, 2, 3, 2>;
using Small = Fp8Shape<64, 64, 2, 2, 2, 2>;
using Deep = Fp8Shape<64, 64, 2, 2, 2, 2, 4>;
using Twice = Fp8Shape<64, 64, 2, 2, 2, 2, 2>;
using Narrow = Fp8Shape<128, 64, 2, 2, 3, 3>;
static_assert(Large::launched_as(kFp8Shapes[kFp8Large]) && Middle::launched_as(kFp8Shapes[kFp8Middle]) &&
              Small::launched_as(kFp8Shapes[kFp8Small]) && Deep::launched_as(kFp8Shapes[kFp8Deep]) &&
              Narrow::launched_as(kFp8Shapes[kFp8Narrow]) && Twice::launched_as(kFp8Shapes[kFp8Twice]), "as launched");

// A fragment from the two pieces that a lane read of it.
template <typename F>
__device__ __forceinline__ F whole(u32x4 lo, u32x4 hi) {
    return F(__builtin_bit_cast(v8i, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)));
}

// A stage's fragments for two by two tiles: v[0], v[1] and v[2], v[3] are the lower and upper pieces of the first operand's,
// v[4] to v[7] those of the second's.
__device__ __forceinline__ void read_stage(uint32_t la, uint32_t ha, uint32_t lb, uint32_t hb, u32x4 (&v)[8]) {
    asm volatile(
        "ds_read_b128 %0, %8\n\tds_read_b128 %1, %8 offset:2048\n\tds_read_b128 %2, %9\n\tds_read_b128 %3, %9 offset:2048\n\t"
        "ds_read_b128 %4, %10\n\tds_read_b128 %5, %10 offset:2048\n\tds_read_b128 %6, %11\n\tds_read_b128 %7, %11 offset:2048\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]), "=&v"(v[6]), "=&v"(v[7])
        : "v"(la), "v"(ha), "v"(lb), "v"(hb)
        : "memory");
}

// acc[i][j] += s[j] (a_i . b_j) for rows FIRST .. FIRST + R - 1 of the accumulators: the products run two ahead of the
// sums that take them (one ahead 1 % slower: 1037 us instead of 1027 for 2048 x 4096 x 128256).
template <int FIRST, typename F, int R, int C, int ALL>
__device__ __forceinline__ void multiply(const F (&a)[R], const F (&b)[C], const float (&s)[C], f32x4 (&acc)[ALL][C]) {
    constexpr int kAhead = 2;
    __builtin_amdgcn_s_setprio(1);
    f32x4 p[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) p[k] = block_product(a[k / C], b[k % C]);
#pragma unroll
    for (int k = 0; k < R * C; ++k) {
        f32x4 next = p[0];
        if (k + kAhead < R * C) next = block_product(a[(k + kAhead) / C], b[(k + kAhead) % C]);
        __builtin_amdgcn_sched_barrier(0);
        f32x4 sum = acc[FIRST + k / C][k % C];
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = fmaf(s[k % C], p[0][e], sum[e]);
        asm volatile("" : "+v"(sum));      // the sum stays here
        acc[FIRST + k / C][k % C] = sum;
        p[0] = p[1];
        p[1] = next;
    }
    __builtin_amdgcn_s_setprio(0);
}

// Where a token's results lie in the staged tile of BN rows of ROW bytes: 16-byte pieces swizzled by the row.
template <int ROW>
__device__ __forceinline__ int staged_at(int row, int byte) {
    return row * ROW + (byte ^ ((row & 7) << 4));
}

template <typename T, typename S>
__global__ void __launch_bounds__(S::kThreads, S::kGroups > 1 ? 4 : S::BM == 64 ? (sizeof(T) == 2 ? 5 : 4) : 2) fp8_tile(const Fp8LinearArgs g) {
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    uint32_t tm, tn, split;
    tile_of(blockIdx.x, g.tiles_v, g.tiles_t, 1u, tm, tn, split);
    const int m0 = int(tm) * S::BM, n0 = int(tn) * S::BN;
    const int lane = threadIdx.x & 63, all_waves = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = all_waves / S::kWaves, wave = all_waves % S::kWaves;
    const int wm = wave / S::kWavesN, wn = wave % S::kWavesN;
    // the group's stages are first .. nst - 1, `share` of them but for the last group's
    const int share = (g.blocks + S::kGroups - 1) / S::kGroups, first = group * share;
    const int nst = first + share < g.blocks ? first + share : g.blocks;
    char* const ring = lds + group * S::kRing;
    using F = Fragment<sizeof(T) == 4>;
    f32x4 acc[S::kRowTiles][S::kColTiles];
#pragma unroll
    for (auto& row : acc)
#pragma unroll
        for (auto& v : row) v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // Copy q of a stage brings rows 8 q .. 8 q + 7: lane l the piece that belongs in slot l % 8 of row 8 q + l / 8.  A
    // wavefront's copies start at an even q, and an odd one's pieces are four further.
    const int piece = (lane & 7) ^ (lane >> 4);
    const uint32_t odd = piece & 4 ? 0u - 64u : 64u;
    const uint32_t off_a = uint32_t(8 * S::kCopiesA * wave + (lane >> 3)) * uint32_t(g.K) + 16u * uint32_t(piece);
    const uint32_t off_b = uint32_t(8 * S::kCopiesB * wave + (lane >> 3)) * uint32_t(g.K) + 16u * uint32_t(piece);
    // The rows of an operand from `first` on; what lies past the last one reads as zeros.
    const auto rows_from = [&](const uint8_t* x, int first, int rows) {
        const int64_t left = int64_t(rows - first) * g.K;
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(x) + int64_t(first) * g.K, 0,
                                                 int(left < kBufferRecords ? left : kBufferRecords), 0x00020000);
    };
    const __amdgpu_buffer_rsrc_t from_a = rows_from(g.w, m0, g.vocab), from_b = rows_from(g.x, n0, g.n);
    // The wavefront's copies of stage s; of the last one, what lies past K reads as zeros.
    const auto issue = [&](auto copies, __amdgpu_buffer_rsrc_t from, uint32_t off, int s, char* to) {
        const int in_row = g.K - s * 128;
#pragma unroll
        for (int u = 0; u < copies; ++u) {
            uint32_t o = off + uint32_t(8 * u) * uint32_t(g.K) + (u & 1 ? odd : 0u);
            if (in_row < 128) o = 16 * (u & 1 ? piece ^ 4 : piece) < in_row ? o : kOutOfRange;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                from, (__attribute__((address_space(3))) void*)(to + (wave * copies + u) * 1024), 16, int(o), s * 128, 0, 0);
        }
    };
    char* const ring_b = ring + S::kSlotsA * S::kBytesA;
    const auto issue_a = [&](int s, int slot) {
        if (s < nst) issue(std::integral_constant<int, S::kCopiesA>(), from_a, off_a, s, ring + slot * S::kBytesA);
    };
    const auto issue_b = [&](int s, int slot) {
        if (s < nst) issue(std::integral_constant<int, S::kCopiesB>(), from_b, off_b, s, ring_b + slot * S::kBytesB);
    };
    // The scales of a stage: the lane's tokens' times the wavefront's entries'.  Tokens past the end take the last one's.
    const int block_v = (m0 + wm * S::kWaveM < g.vocab ? m0 + wm * S::kWaveM : g.vocab - 1) / kFp8Group;
    const float* sw = g.w_scale + int64_t(block_v) * g.blocks;
    const auto token = [&](int j) {
        const int t = wn * S::kWaveN + 16 * j + (lane & 15);
        return uint32_t(n0 + t < g.n ? t : g.n - 1 - n0);
    };
    const uint32_t la = k_base(ring, wm * S::kWaveM, 0, lane), ha = k_base(ring, wm * S::kWaveM, 1, lane);
    const uint32_t lb = k_base(ring_b, wn * S::kWaveN, 0, lane), hb = k_base(ring_b, wn * S::kWaveN, 1, lane);
    if constexpr (S::BM <= 128) {
        // One barrier a step: once stage s has landed and every wavefront is done with s - 1, stage s + 1 goes to that one's
        // slot.  A token's scales of four stages are one load, four stages ahead: each token's lie in a cache line of their
        // own (2048 x 4096 x 128256 by the 64 x 64 tile: 2.8 ms with a load a stage, 1.97 so).
        const int64_t left = int64_t(g.n - n0) * g.blocks * 4;
        const __amdgpu_buffer_rsrc_t from_s = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<float*>(g.x_scale) + int64_t(n0) * g.blocks, 0, int(left < kBufferRecords ? left : kBufferRecords), 0x00020000);
        f32x4 next[S::kColTiles], now[S::kColTiles];
        const auto load_scales = [&](int s) {
#pragma unroll
            for (int j = 0; j < S::kColTiles; ++j)
                next[j] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(from_s, int(token(j) * uint32_t(g.blocks) * 4u), s * 4, 0));
        };
        load_scales(first);
        issue_a(first, 0);
        issue_b(first, 0);
        if constexpr (S::kSlotsA == 3) issue_a(first + 1, 1);
        if constexpr (S::kSlotsB == 3) issue_b(first + 1, 1);
        int slot = 0;                      // of the rings of three
        for (int s0 = first; s0 < first + share; s0 += 4) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int s = s0 + u;
                if (s >= first + share) break;             // every group meets as often
                if (S::kSlotsA == 3 && s + 1 < nst) wait_copies<S::kCopiesA + (S::kSlotsB == 3 ? S::kCopiesB : 0)>();
                else wait_copies<0>();
                meet();
                if (S::kGroups > 1 && s >= nst) continue;
                if (u == 0) {
#pragma unroll
                    for (int j = 0; j < S::kColTiles; ++j) now[j] = next[j];
                    load_scales(s0 + 4);
                }
                const uint32_t slot_a = uint32_t((S::kSlotsA == 3 ? slot : u % 2) * S::kBytesA);
                const uint32_t slot_b = uint32_t((S::kSlotsB == 3 ? slot : u % 2) * S::kBytesB);
                const int after = slot == 0 ? 2 : slot - 1;            // the slot that stage s - 1 left
                if constexpr (S::kSlotsB == 3) issue_b(s + 2, after);
                else issue_b(s + 1, (u + 1) % 2);
                if constexpr (S::kSlotsA == 3) issue_a(s + 2, after);
                else issue_a(s + 1, (u + 1) % 2);
                slot = slot == 2 ? 0 : slot + 1;
                float scale[S::kColTiles];
#pragma unroll
                for (int j = 0; j < S::kColTiles; ++j) scale[j] = now[j][u] * sw[s];
                if constexpr (S::kRowTiles == 2) {
                    u32x4 v[8];
                    read_stage(la + slot_a, ha + slot_a, lb + slot_b, hb + slot_b, v);
                    const F a[2] = {whole<F>(v[0], v[2]), whole<F>(v[1], v[3])}, b[2] = {whole<F>(v[4], v[6]), whole<F>(v[5], v[7])};
                    multiply<0>(a, b, scale, acc);
                } else if constexpr (S::kColTiles == 2) {
                    u32x4 v[8], w[4];
                    read_k(la + slot_a, ha + slot_a, v);
                    read_k2(lb + slot_b, hb + slot_b, w);
                    const F b[2] = {whole<F>(w[0], w[2]), whole<F>(w[1], w[3])};
                    const F a[4] = {whole<F>(v[0], v[4]), whole<F>(v[1], v[5]), whole<F>(v[2], v[6]), whole<F>(v[3], v[7])};
                    multiply<0>(a, b, scale, acc);
                } else {
                    u32x4 v[16];
                    read_k(la + slot_a, ha + slot_a, lb + slot_b, hb + slot_b, v);
                    const F b[4] = {whole<F>(v[8], v[12]), whole<F>(v[9], v[13]), whole<F>(v[10], v[14]), whole<F>(v[11], v[15])};
                    if constexpr (sizeof(T) == 4) {        // a fragment is 16 registers: the first operand's one by one
                        const auto row = [&](auto i) {
                            const F a[1] = {whole<F>(v[i], v[4 + i])};
                            multiply<i>(a, b, scale, acc);
                        };
                        row(std::integral_constant<int, 0>());
                        row(std::integral_constant<int, 1>());
                        row(std::integral_constant<int, 2>());
                        row(std::integral_constant<int, 3>());
                    } else {
                        const F a[4] = {whole<F>(v[0], v[4]), whole<F>(v[1], v[5]), whole<F>(v[2], v[6]), whole<F>(v[3], v[7])};
                        multiply<0>(a, b, scale, acc);
                    }
                }
            }
        }
    } else {
        // A step in four turns, each ended by the workgroup's barrier: fragments of half of the wavefront's entries, their
        // products, and the same for the other half.  The wavefronts of the tile's lower half (one on each SIMD, as
        // those of the upper) run one turn behind, so that one group reads LDS while the other multiplies.  Copies run
        // two stages ahead: stage s + 2 of the projection goes to the slot that stage s - 1 left, that of the tokens to
        // stage s's own, whose fragments are all in registers after the step's first two turns.
        // The scales are a stage's side by side here (a row of g.scale_ld for each block of K).
        uint32_t off_s[S::kColTiles];
#pragma unroll
        for (int j = 0; j < S::kColTiles; ++j) off_s[j] = (uint32_t(n0) + token(j)) * 4u;
        float next[S::kColTiles], next_w, now[S::kColTiles];
        const auto load_scales = [&](int s) {
            if (s >= nst) return;
            next_w = sw[s];
            const char* at = reinterpret_cast<const char*>(g.x_scale + int64_t(s) * g.scale_ld);
#pragma unroll
            for (int j = 0; j < S::kColTiles; ++j) next[j] = *reinterpret_cast<const float*>(at + off_s[j]);
        };
        u32x4 va[8], v[16];
        load_scales(0);
        const auto wait_stage = [&](int s) {
            if (s + 1 < nst) wait_copies<S::kCopiesA + S::kCopiesB>();
            else wait_copies<0>();
        };
        issue_a(0, 0);
        issue_b(0, 0);
        issue_a(1, 1);
        issue_b(1, 1);
        wait_stage(0);
        meet();
        if (wm == 1) meet();
        int slot = 0;                      // of the projection's ring: s % 3
        for (int s = 0; s < nst; ++s) {
            const uint32_t at_a = uint32_t(slot * S::kBytesA), at_b = uint32_t(s % 2 * S::kBytesB);
#pragma unroll
            for (int j = 0; j < S::kColTiles; ++j) now[j] = next[j] * next_w;
            load_scales(s + 1);            // before the copies of stage s + 2: they have landed with stage s + 1
            issue_a(s + 2, slot == 0 ? 2 : slot - 1);
            read_k(la + at_a, ha + at_a, lb + at_b, hb + at_b, v);
            const F a[4] = {whole<F>(v[0], v[4]), whole<F>(v[1], v[5]), whole<F>(v[2], v[6]), whole<F>(v[3], v[7])};
            const F b[4] = {whole<F>(v[8], v[12]), whole<F>(v[9], v[13]), whole<F>(v[10], v[14]), whole<F>(v[11], v[15])};
            meet();
            multiply<0>(a, b, now, acc);
            meet();
            issue_b(s + 2, s % 2);
            read_k(la + at_a + 8192, ha + at_a + 8192, va);
            const F c[4] = {whole<F>(va[0], va[4]), whole<F>(va[1], va[5]), whole<F>(va[2], va[6]), whole<F>(va[3], va[7])};
            if (wm == 1) wait_stage(s + 1);
            meet();
            multiply<4>(c, b, now, acc);
            if (wm == 0) wait_stage(s + 1);
            meet();
            slot = slot == 2 ? 0 : slot + 1;
        }
        if (wm == 0) meet();
    }
    __syncthreads();                       // the ring is free
    if constexpr (S::kGroups > 1) {        // the groups' shares, in their order
        constexpr int kEach = S::kRowTiles * S::kColTiles;
        static_assert((S::kGroups - 1) * kEach * S::kWaves * 1024 <= S::kLds, "the shares");
        f32x4* part = reinterpret_cast<f32x4*>(lds) + threadIdx.x % (64 * S::kWaves);
        if (group > 0) {
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                part[((group - 1) * kEach + i) * 64 * S::kWaves] = acc[i / S::kColTiles][i % S::kColTiles];
        }
        __syncthreads();
        if (group == 0) {
#pragma unroll
            for (int o = 0; o < S::kGroups - 1; ++o)
#pragma unroll
                for (int i = 0; i < kEach; ++i) acc[i / S::kColTiles][i % S::kColTiles] += part[(o * kEach + i) * 64 * S::kWaves];
        }
        __syncthreads();
    }

    // Element e of accumulator (i, j) is entry m0 + wm kWaveM + 16 i + 4 (lane / 16) + e of token n0 + wn kWaveN + 16 j +
    // lane % 16.  The tile goes through LDS, so that a token's entries leave in whole rows.
    constexpr int kRow = S::BM * int(sizeof(T)), kRows = S::BN;
    static_assert(kRows * kRow <= S::kLds, "the staged tile");
    T* out = static_cast<T*>(g.out);
    const T* bias = static_cast<const T*>(g.bias);
#pragma unroll
    for (int i = 0; i < S::kRowTiles; ++i) {
        if (group > 0) break;
        const int m = wm * S::kWaveM + 16 * i + 4 * (lane >> 4);
        float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (bias) {                        // entries past the end take the last one's: they are not stored
#pragma unroll
            for (int e = 0; e < 4; ++e) b[e] = widen(bias[m0 + m + e < g.vocab ? m0 + m + e : g.vocab - 1]);
        }
#pragma unroll
        for (int j = 0; j < S::kColTiles; ++j) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e] + b[e];
            store_row<4>(reinterpret_cast<T*>(lds + staged_at<kRow>(wn * S::kWaveN + 16 * j + (lane & 15), m * int(sizeof(T)))), v);
        }
    }
    __syncthreads();
    constexpr int V = kVec16<T>, kLanes = S::BM / V;
    const int c = threadIdx.x % kLanes, v0 = m0 + V * c;
    for (int r = threadIdx.x / kLanes; r < kRows; r += S::kThreads / kLanes) {
        const int t = n0 + r;
        if (t >= g.n || v0 >= g.vocab) continue;
        const u32x4 d = *reinterpret_cast<const u32x4*>(lds + staged_at<kRow>(r, 16 * c));
        T* to = out + int64_t(t) * g.vocab + v0;
        if (v0 + V <= g.vocab) {
            *reinterpret_cast<typename Unaligned16<T>::type*>(to) = d;
        } else {
            const T* from = reinterpret_cast<const T*>(lds + staged_at<kRow>(r, 16 * c));
            for (int k = 0; v0 + k < g.vocab; ++k) to[k] = from[k];
        }
    }
}

template <typename S>
const void* tile_of_type(int out_dtype) {
    switch (out_dtype) {
    case kF16: return reinterpret_cast<const void*>(&fp8_tile<_Float16, S>);
    case kBF16: return reinterpret_cast<const void*>(&fp8_tile<__bf16, S>);
    }
    return nullptr;
}

}  // namespace

const void* pick_fp8_tile(int out_dtype, int kind) {
    if (out_dtype == kF32)
        return kind == kFp8Small    ? reinterpret_cast<const void*>(&fp8_tile<float, Small>)
               : kind == kFp8Middle ? reinterpret_cast<const void*>(&fp8_tile<float, Middle>)
               : kind == kFp8Deep   ? reinterpret_cast<const void*>(&fp8_tile<float, Deep>)
               : kind == kFp8Twice  ? reinterpret_cast<const void*>(&fp8_tile<float, Twice>)
               : kind == kFp8Narrow ? reinterpret_cast<const void*>(&fp8_tile<float, Narrow>)
                                    : nullptr;
    switch (kind) {
    case kFp8Deep: return tile_of_type<Deep>(out_dtype);
    case kFp8Twice: return tile_of_type<Twice>(out_dtype);
    case kFp8Narrow: return tile_of_type<Narrow>(out_dtype);
    case kFp8Small: return tile_of_type<Small>(out_dtype);
    case kFp8Middle: return tile_of_type<Middle>(out_dtype);
    case kFp8Large: return tile_of_type<Large>(out_dtype);
    }
    return nullptr;
}

}  // namespace rlpl
