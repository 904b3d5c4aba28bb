// Softmax cross entropy of an output projection over a large vocabulary on
// gfx950, with its gradients, in pieces of the vocabulary: no kernel writes
// logits.  For the rows i whose target y_i is not ignored (N of them),
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
// per piece of the vocabulary: the piece's logits are formed again (less
// traffic and memory than keeping n x V of them), dz goes to the workspace in
// the operand dtype, and two products take it from there.  The weight's
// gradient of a piece comes out whole, so it is rounded once and written once;
// the hidden states' is summed over the pieces in float32.
//
// dz is formed without s and held at a fixed scale (its largest value is
// about 1): s would push a long batch's small probabilities under fp16's
// range.  The factor is applied to the float32 results.
//
// The contraction and its tiles are those of mfma_tile.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ce_kernels.h"
#include "device_common.h"
#include "loss_kernels.h"
#include "mfma_tile.h"
#include "row_io.h"

namespace rlpl {

namespace {

template <typename T> constexpr float kDzScale = 1.0f;
template <> constexpr float kDzScale<_Float16> = 256.0f;

}  // namespace

// One workgroup scans the targets, eight consecutive ones a lane.
__global__ void __launch_bounds__(kCeCompactThreads) ce_compact(const CeCompactArgs a) {
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
            if (kept) {
                a.row[k0] = int(i + k);
                a.target[k0] = (t[k] >= 0 && t[k] < a.vocab) ? int(t[k]) : -1;
                ++k0;
            }
        }
        base += total;
    }
    if (threadIdx.x == 0) *a.state = CeState{base, 0.0f};
}

__global__ void __launch_bounds__(kCeThreads) ce_gather(const CeGatherArgs a) {
    const int count = a.state->count, words = a.cols / 8;
    for (int k = blockIdx.x; k < count; k += gridDim.x) {
        const u32x4* from = reinterpret_cast<const u32x4*>(a.hidden) + int64_t(a.row[k]) * words;
        u32x4* to = reinterpret_cast<u32x4*>(a.out) + int64_t(k) * words;
        for (int i = threadIdx.x; i < words; i += kCeThreads) to[i] = from[i];
    }
}

// One tile of a product.  A_KCONTIG, B_KCONTIG: the operands' layouts (mfma_tile.h).
template <typename T, int PRODUCT, bool A_KCONTIG, bool B_KCONTIG>
__global__ void __launch_bounds__(kGemmThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
ce_gemm(const CeGemmArgs g) {
    extern __shared__ __attribute__((aligned(1024))) uint16_t ring[];
    constexpr int BK = kGemmBK;
    using St = Stage<BK>;
    __shared__ float red_a[kGemmWavesM][kGemmBN];
    __shared__ int tgt_col[kGemmBM];

    const int count = g.state->count;
    const int M = PRODUCT == kCeWeight ? g.M : min(g.M, count);
    const int K = PRODUCT == kCeWeight ? min(g.K, count) : g.K;
    const uint32_t tiles_m = uint32_t(M + kGemmBM - 1) / kGemmBM;
    const uint32_t block = blockIdx.x + gridDim.x * blockIdx.z;
    if (block >= tiles_m * g.tiles_n * gridDim.z) return;     // the launch was sized for every row
    uint32_t tm, tn, split;
    tile_of(block, tiles_m, g.tiles_n, gridDim.z, tm, tn, split);
    const int m0 = int(tm) * kGemmBM, n0 = int(tn) * kGemmBN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / kGemmWavesN, wn = wave % kGemmWavesN;
    const int kb = PRODUCT == kCeHidden ? int(split) * g.k_split : 0;
    const int ke = PRODUCT == kCeHidden ? min(K, kb + g.k_split) : K;
    const uint16_t* __restrict__ A = static_cast<const uint16_t*>(g.a);
    const uint16_t* __restrict__ B = static_cast<const uint16_t*>(g.b);

    // Accumulator element e of tile (i, j) is tile row wm*kWaveM + i*32 + 8*(e/4) +
    // 4*(lane/32) + e%4 and column wn*kWaveN + j*32 + lane%32.
    auto row_of_e = [&](int i, int e) { return wm * kWaveM + i * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3); };
    auto col_of_j = [&](int j) { return wn * kWaveN + j * 32 + (lane & 31); };

    floatx16 acc[kFragM][kFragN];
#pragma unroll
    for (int i = 0; i < kFragM; ++i)
#pragma unroll
        for (int j = 0; j < kFragN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

    const int nst = kb < ke ? (ke - kb + BK - 1) / BK : 0;
    auto issue = [&](int s) {
        const int k0 = kb + s * BK;
        char* slot = reinterpret_cast<char*>(ring) + (s % St::kCount) * St::kBytes;
        const __amdgpu_buffer_rsrc_t a0 =
            buffer_at(A + (A_KCONTIG ? int64_t(m0) * g.lda + k0 : int64_t(k0) * g.lda + m0));
        const __amdgpu_buffer_rsrc_t b0 =
            buffer_at(B + (B_KCONTIG ? int64_t(n0) * g.ldb + k0 : int64_t(k0) * g.ldb + n0));
#pragma unroll
        for (int u = 0; u < St::kDmaA; ++u) {
            const int q = wave * St::kDmaA + u;
            dma16(a0, dma_source<A_KCONTIG, BK>(q, lane, uint32_t(g.lda), M, ke, m0, k0), slot + q * 1024);
        }
#pragma unroll
        for (int u = 0; u < St::kDmaB; ++u) {
            const int q = wave * St::kDmaB + u;
            dma16(b0, dma_source<B_KCONTIG, BK>(q, lane, uint32_t(g.ldb), g.N, ke, n0, k0),
                  slot + St::kBytesA + q * 1024);
        }
    };
    if (nst > 0) {
        for (int s = 0; s < St::kCount - 1; ++s) issue(s);
        for (int s = 0; s < nst; ++s) {
            wait_stages<St::kCount - 2, BK>();
            issue(s + St::kCount - 1);     // past the last stage: out of range, zeros
            const uint16_t* at = ring + (s % St::kCount) * (St::kBytes / 2);
            const uint16_t* bt = at + St::kBytesA / 2;
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
                uint4 af[kFragM], bf[kFragN];
#pragma unroll
                for (int i = 0; i < kFragM; ++i) af[i] = fragment<A_KCONTIG, kWaveM, BK>(at, wm, i, kk, lane);
#pragma unroll
                for (int j = 0; j < kFragN; ++j) bf[j] = fragment<B_KCONTIG, kWaveN, BK>(bt, wn, j, kk, lane);
#pragma unroll
                for (int i = 0; i < kFragM; ++i)
#pragma unroll
                    for (int j = 0; j < kFragN; ++j) acc[i][j] = Mfma<uint16_t>::run(af[i], bf[j], acc[i][j], T());
            }
        }
    }
    __syncthreads();

    if constexpr (PRODUCT == kCeHidden) {
        float* __restrict__ C = static_cast<float*>(g.c) + int64_t(split) * g.plane;
#pragma unroll
        for (int i = 0; i < kFragM; ++i) {
            float old[16][kFragN] = {};
            if (g.accumulate) {            // clamped to a valid element outside M x N, where nothing is stored
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int row = min(m0 + row_of_e(i, e), M - 1);
#pragma unroll
                    for (int j = 0; j < kFragN; ++j) old[e][j] = C[int64_t(row) * g.ldc + min(n0 + col_of_j(j), g.N - 1)];
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int row = m0 + row_of_e(i, e);
                if (row >= M) continue;
#pragma unroll
                for (int j = 0; j < kFragN; ++j) {
                    const int col = n0 + col_of_j(j);
                    if (col < g.N) C[int64_t(row) * g.ldc + col] = old[e][j] + acc[i][j][e];
                }
            }
        }
        return;
    }

    if constexpr (PRODUCT == kCeWeight) {
        const float scale = g.state->scale;
#pragma unroll
        for (int i = 0; i < kFragM; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int row = m0 + row_of_e(i, e);
                if (row >= M) continue;
#pragma unroll
                for (int j = 0; j < kFragN; ++j) {
                    const int col = n0 + col_of_j(j);
                    if (col >= g.N) continue;
                    const int64_t at = int64_t(row) * g.ldc + col;
                    const float v = acc[i][j][e] * scale;
                    if (g.out_f32) {
                        float* c = static_cast<float*>(g.c) + at;
                        *c = g.accumulate ? *c + v : v;
                    } else {
                        static_cast<T*>(g.c)[at] = from_f<T>(v);
                    }
                }
            }
        return;
    }

    // Logits: z = acc + bias; columns past N are -inf.
    const T* __restrict__ bias = static_cast<const T*>(g.bias);
#pragma unroll
    for (int j = 0; j < kFragN; ++j) {
        const int col = n0 + col_of_j(j);
        const float b = col < g.N ? (bias ? to_f<T>(bias[col]) : 0.0f) : -__builtin_inff();
#pragma unroll
        for (int i = 0; i < kFragM; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] += b;
    }

    if constexpr (PRODUCT == kCeDlogits) {
        float* row_lse = reinterpret_cast<float*>(ring);
        float* row_f = row_lse + kGemmBM;
        if (threadIdx.x < kGemmBM) {
            const int row = m0 + int(threadIdx.x);
            const float lse = row < M ? g.lse[row] : 0.0f;
            const int t = row < M ? g.target[row] - g.first - n0 : -1;
            row_lse[threadIdx.x] = lse;
            row_f[threadIdx.x] = kDzScale<T> * (1.0f + g.z_loss2 * lse);
            tgt_col[threadIdx.x] = t >= 0 && t < kGemmBN && n0 + t < g.N ? t : -1;
        }
        __syncthreads();
        T* __restrict__ D = static_cast<T*>(g.c);
        const bool odd = lane & 1;
        float csum[kFragN] = {};
#pragma unroll
        for (int i = 0; i < kFragM; ++i) {
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                float dz[2][kFragN];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = row_of_e(i, e + h);
                    const bool in = m0 + r < M;
                    const float l = row_lse[r], f = row_f[r];
                    const int tc = tgt_col[r];
#pragma unroll
                    for (int j = 0; j < kFragN; ++j) {
                        const int c = col_of_j(j);
                        const float p = __builtin_amdgcn_exp2f((acc[i][j][e + h] - l) * kLog2eG);
                        dz[h][j] = (in && n0 + c < g.N) ? f * p - (c == tc ? kDzScale<T> : 0.0f) : 0.0f;
                        csum[j] += dz[h][j];
                    }
                }
                const int row = m0 + row_of_e(i, e) + (odd ? 1 : 0);
#pragma unroll
                for (int j = 0; j < kFragN; ++j) {
                    const float got = swap_pair(odd ? dz[0][j] : dz[1][j]);
                    const float lo = odd ? got : dz[0][j];
                    const float hi = odd ? dz[1][j] : got;
                    const int col = n0 + col_of_j(j) - (odd ? 1 : 0);
                    // up to the row pitch: the padding past N is zeros, a K tail of the hidden product
                    if (row < M && col < g.ldc)
                        *reinterpret_cast<uint32_t*>(D + int64_t(row) * g.ldc + col) = Elem<T>::pack(lo, hi);
                }
            }
        }
        if (g.col_part) {
#pragma unroll
            for (int j = 0; j < kFragN; ++j) {
                const float s = csum[j] + __shfl_xor(csum[j], 32, 64);
                if (lane < 32) red_a[wm][col_of_j(j)] = s;
            }
            __syncthreads();
            const int col = n0 + int(threadIdx.x);
            if (threadIdx.x < kGemmBN && col < g.N) {
                float t = red_a[0][threadIdx.x];
#pragma unroll
                for (int w = 1; w < kGemmWavesM; ++w) t += red_a[w][threadIdx.x];
                g.col_part[int64_t(tm) * g.N + col] = t;
            }
        }
        return;
    }

    // kCeLogits: a lane reduces its own columns of a row; the 128 partials of a row
    // meet in LDS, half of the rows at a time, laid out [partial][row ^ part_swizzle(partial)]
    // (writes and reads free of bank conflicts), and four neighbouring lanes merge a row.
    constexpr int kParts = kGemmWavesN * 32;
    constexpr int kRoundRows = kGemmBM / kGemmWavesM;
    constexpr int kShare = kParts / 4;
    static_assert(kGemmThreads == 4 * kRoundRows && kParts * kRoundRows * 8 <= kGemmDynLds && kParts <= 256,
                  "four lanes a row; the partials fit");
    float2* parts = reinterpret_cast<float2*>(ring);
    if (threadIdx.x < kGemmBM) {
        const int row = m0 + int(threadIdx.x);
        const int t = row < M ? g.target[row] - n0 : -1;
        tgt_col[threadIdx.x] = t >= 0 && t < kGemmBN && n0 + t < g.N ? t : -1;
    }
    const int pidx = wn * 32 + (lane & 31);
#pragma unroll
    for (int w = 0; w < kGemmWavesM; ++w) {
        __syncthreads();                   // tgt_col written; parts free
        if (wm == w) {
#pragma unroll
            for (int i = 0; i < kFragM; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int r = row_of_e(i, e);
                    float m = acc[i][0][e];
#pragma unroll
                    for (int j = 1; j < kFragN; ++j) m = fmaxf(m, acc[i][j][e]);
                    float sum = 0.0f;
                    if (m != -__builtin_inff()) {
#pragma unroll
                        for (int j = 0; j < kFragN; ++j) sum += __builtin_amdgcn_exp2f((acc[i][j][e] - m) * kLog2eG);
                    }
                    parts[pidx * kRoundRows + ((r - w * kRoundRows) ^ part_swizzle(pidx))] = make_float2(m, sum);
                    const int tc = tgt_col[r];
#pragma unroll
                    for (int j = 0; j < kFragN; ++j)
                        if (col_of_j(j) == tc && m0 + r < M) g.target_logit[m0 + r] = acc[i][j][e];
                }
        }
        __syncthreads();
        const int rr = threadIdx.x / 4, qq = threadIdx.x % 4, row = m0 + w * kRoundRows + rr;
        float top = -__builtin_inff();
        for (int q = qq * kShare; q < (qq + 1) * kShare; ++q)
            top = fmaxf(top, parts[q * kRoundRows + (rr ^ part_swizzle(q))].x);
        top = fmaxf(top, quad_xor<1>(top));
        top = fmaxf(top, quad_xor<2>(top));
        float sum = 0.0f;
        for (int q = top == -__builtin_inff() ? kParts : qq * kShare; q < (qq + 1) * kShare; ++q) {   // none where all are -inf
            const float2 v = parts[q * kRoundRows + (rr ^ part_swizzle(q))];
            sum += v.y * __builtin_amdgcn_exp2f((v.x - top) * kLog2eG);
        }
        sum += quad_xor<1>(sum);
        sum += quad_xor<2>(sum);
        if (qq == 0 && row < M)
            reinterpret_cast<float2*>(g.part)[int64_t(row) * g.tiles_n + tn] = make_float2(top, sum);
    }
}

// A workgroup joins a kept row's tiles (each lane's in order, then the lane tree).
__global__ void __launch_bounds__(kCeThreads) ce_row(const CeRowArgs a) {
    __shared__ float red[kCeThreads / 64];
    const int count = a.state->count;
    for (int row = blockIdx.x; row < count; row += gridDim.x) {
        const float2* p = reinterpret_cast<const float2*>(a.part) + int64_t(row) * a.tiles;
        float m = -__builtin_inff();
        for (int t = threadIdx.x; t < a.tiles; t += kCeThreads) m = fmaxf(m, p[t].x);
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
        __syncthreads();
        float top = red[0];
#pragma unroll
        for (int i = 1; i < kCeThreads / 64; ++i) top = fmaxf(top, red[i]);
        float s = 0.0f;
        for (int t = threadIdx.x; t < a.tiles; t += kCeThreads)
            s += p[t].y * __builtin_amdgcn_exp2f((p[t].x - top) * kLog2eG);
        s = block_sum(s, red);
        if (threadIdx.x == 0) {
            const float lse = top + __builtin_amdgcn_logf(s) * 0.6931471805599453f;
            a.lse[row] = lse;
            a.row_loss[row] = a.target[row] >= 0 ? lse - a.target_logit[row] + a.z_loss * lse * lse : __builtin_nanf("");
        }
    }
}

// One workgroup sums the rows' losses in double (each lane's in order, then a tree in LDS).
__global__ void __launch_bounds__(kCeCompactThreads) ce_loss(const CeLossArgs a) {
    __shared__ double sums[kCeCompactThreads];
    const int count = a.state->count;
    double s = 0.0;
    for (int i = threadIdx.x; i < count; i += kCeCompactThreads) s += double(a.row_loss[i]);
    sums[threadIdx.x] = s;
    for (int half = kCeCompactThreads / 2; half > 0; half >>= 1) {
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
__global__ void __launch_bounds__(kCeThreads) ce_hidden(const CeHiddenArgs a) {
    const float scale = a.state->scale;
    for (int row = blockIdx.x; row < a.n; row += gridDim.x) {
        const int k = a.place[row];
        T* out = static_cast<T*>(a.out) + int64_t(row) * a.cols;
        for (int c = threadIdx.x * 8; c < a.cols; c += kCeThreads * 8) {
            float v[8] = {};
            if (k >= 0) {
                const float* p = a.part + int64_t(k) * a.cols + c;
                for (int z = 0; z < a.splits; ++z) {
                    float x[8];
                    load_row<8>(p + z * a.plane, x);
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] += x[q];
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] *= scale;
            }
            store_row<8>(out + c, v);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kCeThreads) ce_bias(const CeBiasArgs a) {
    const int col = blockIdx.x * kCeThreads + threadIdx.x;
    if (col >= a.cols) return;
    const int tiles = (a.state->count + kGemmBM - 1) / kGemmBM;
    float s = 0.0f;
    for (int t = 0; t < tiles; ++t) s += a.part[int64_t(t) * a.cols + col];
    s *= a.state->scale;
    if (a.out_f32) {
        float* out = static_cast<float*>(a.out) + col;
        *out = a.accumulate ? *out + s : s;
    } else {
        static_cast<T*>(a.out)[col] = from_f<T>(s);
    }
}

// ----------------------------------------------------------------------------- host-side table

template <typename T>
static const void* ce_gemm_for(int product) {
    switch (product) {
    case kCeLogits: return reinterpret_cast<const void*>(&ce_gemm<T, kCeLogits, true, true>);
    case kCeDlogits: return reinterpret_cast<const void*>(&ce_gemm<T, kCeDlogits, true, true>);
    case kCeHidden: return reinterpret_cast<const void*>(&ce_gemm<T, kCeHidden, true, false>);
    case kCeWeight: return reinterpret_cast<const void*>(&ce_gemm<T, kCeWeight, false, false>);
    }
    return nullptr;
}

const void* pick_ce_gemm(int dtype, int product) {
    return dtype == kF16 ? ce_gemm_for<_Float16>(product) : dtype == kBF16 ? ce_gemm_for<__bf16>(product) : nullptr;
}
const void* ce_compact_kernel() { return reinterpret_cast<const void*>(&ce_compact); }
const void* ce_gather_kernel() { return reinterpret_cast<const void*>(&ce_gather); }
const void* ce_row_kernel() { return reinterpret_cast<const void*>(&ce_row); }
const void* ce_loss_kernel() { return reinterpret_cast<const void*>(&ce_loss); }
const void* pick_ce_hidden(int dtype) {
    return dtype == kF16 ? reinterpret_cast<const void*>(&ce_hidden<_Float16>)
                         : reinterpret_cast<const void*>(&ce_hidden<__bf16>);
}
const void* pick_ce_bias(int dtype) {
    return dtype == kF16 ? reinterpret_cast<const void*>(&ce_bias<_Float16>)
                         : reinterpret_cast<const void*>(&ce_bias<__bf16>);
}

}  // namespace rlpl
