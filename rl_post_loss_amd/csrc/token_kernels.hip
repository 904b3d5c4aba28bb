// Log-probabilities of given tokens over rows of logits on gfx950, with each
// row's entropy and its most likely tokens, and the backward pass.
//
// For a row z at temperature T, with c = log2(e) / T and the running maximum b,
//
//   s = sum 2^(c z - c b),   t = sum (c z - c b) 2^(c z - c b)
//   lse = ln 2 (c b + log2 s),   logp = ln 2 (c z_y - c b - log2 s),   H = ln 2 (log2 s - t / s)
//
// in one pass: a lane keeps (b, s, t) over its vectors of 16 bytes and counts
// anew from a larger maximum once per 32 elements (s 2^d and (t + d s) 2^d for
// a maximum further by -d), and lanes, wavefronts and pieces of a row are joined in a
// fixed order by the same rule.  A logit of -inf adds nothing (its exponent is
// held at -1000, which 2^x takes to zero, by a maximum that lets NaN through).
//
// The k largest elements, the lowest index first among equal ones, come from
// the same pass without a list in its loop: each lane leaves the largest of
// every 32 of its elements in LDS.  The k-th of the largest of groups of lanes is a
// bound that k elements reach, so the row's k largest all do, and they lie in
// blocks of 32 whose own largest reaches it, little more than k of them: those are read a
// second time, their elements that reach the bound collected and ranked.  Where
// equal logits or their order make that many blocks or elements, the bound is
// taken by (logit, index), which no two elements share, and from the lanes that reach it,
// in steps if need be.
//
// The loop takes about ten vector operations an element (2^x counts four), a
// little less time than its reading: 3000 x 128256 bf16 143 us (5.4 TB/s of
// 0.77 GB), with 5 alternatives 144, with 20 146, with 64 159 (220 with 20, while
// the elements of the lanes that reach the bound were read again, each vector a cache line
// of its own).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "loss_kernels.h"
#include "row_io.h"
#include "token_kernels.h"

namespace rlpl {

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNone = -1000.0f;          // an exponent that 2^x takes to zero
constexpr int kTokenWaves = kTokenThreads / 64;

__device__ __forceinline__ float hold(float d) { return __builtin_elementwise_maximum(d, kNone); }
__device__ __forceinline__ float exp2_hw(float d) { return __builtin_amdgcn_exp2f(d); }
// What a sum counts from: its largest element, or 0 where that is -inf.
__device__ __forceinline__ float base_of(float top) { return top == -__builtin_inff() ? 0.0f : top; }

// The largest of a wavefront's values in every lane (NaN passed over), by DPP lane moves; lanes without a source keep theirs.
__device__ __forceinline__ float wave_top(float v) {
    const auto more = [&v](auto move) { v = fmaxf(v, __int_as_float(move(__float_as_int(v)))); };
    more([](int x) { return __builtin_amdgcn_update_dpp(x, x, 0xB1, 0xF, 0xF, false); });
    more([](int x) { return __builtin_amdgcn_update_dpp(x, x, 0x4E, 0xF, 0xF, false); });
    more([](int x) { return __builtin_amdgcn_update_dpp(x, x, 0x141, 0xF, 0xF, false); });
    more([](int x) { return __builtin_amdgcn_update_dpp(x, x, 0x140, 0xF, 0xF, false); });
    more([](int x) { return __builtin_amdgcn_update_dpp(x, x, 0x142, 0xA, 0xF, false); });
    more([](int x) { return __builtin_amdgcn_update_dpp(x, x, 0x143, 0xC, 0xF, false); });
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Exponents count from c b, rounded, as c z - c b by one operation, the same for a row's sums and its results, so that the
// rounding falls out of them.  Where c b is so large that its rounding is not small (a row of the type's lowest value; a tiny
// temperature) they are (z - b) c.  Either way c (z - from) - bc.
struct Base {
    float b, from, bc;
    __device__ __forceinline__ Base(float top, float c) : b(base_of(top)) {
#pragma clang fp contract(off)
        const float product = c * b;       // as it is rounded here, wherever it is used
        const bool near = fabsf(product) < 0x1p20f;
        from = near ? 0.0f : b;
        bc = near ? product : 0.0f;
    }
    // Of a wavefront's one maximum, in scalar registers.
    __device__ __forceinline__ Base uniform() const {
        const auto one = [](float v) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v))); };
        Base u = *this;
        u.b = one(b), u.from = one(from), u.bc = one(bc);
        return u;
    }
    __device__ __forceinline__ bool far() const { return from != 0.0f; }
    __device__ __forceinline__ float exponent(float z, float c) const { return fmaf(z - from, c, -bc); }
    // What exponents that count from here grow by when they count from `to`.  With the rounded products' difference nothing of
    // their rounding is left; c (b - b') gave log-probabilities off by 9e-6 and 1e-4 for logits around 300 and 3000.
    __device__ __forceinline__ float less(const Base& to, float c) const { return fmaf(from - to.from, c, bc - to.bc); }
};

// Sums that count from `top`.
struct Sums {
    float top, s, t;
    static __device__ __forceinline__ Sums none() { return Sums{-__builtin_inff(), 0.0f, 0.0f}; }
    // Counts from a larger maximum, whose base is `there`; `here` is the present one's.
    __device__ __forceinline__ void rise(float to, const Base& here, const Base& there, float c) {
        const bool none = top == -__builtin_inff();            // nothing but NaN is in the sums
        const float d = none ? 0.0f : hold(here.less(there, c));
        const float f = none ? 0.0f : exp2_hw(d);
        t = fmaf(d, s, t) * f;
        s *= f;
        top = to;
    }
    __device__ __forceinline__ void rise(float to, float c) { rise(to, Base(top, c), Base(to, c), c); }
    // One more term, with its exponent.
    __device__ __forceinline__ void add(float d) {
        d = hold(d);
        const float e = exp2_hw(d);
        s += e;
        t = fmaf(e, d, t);
    }
    // A wavefront's lanes joined, in each of them.
    __device__ __forceinline__ void join_lanes(float c) {
        rise(wave_top(top), c);
        s = wave_sum(s);
        t = wave_sum(t);
    }
};

// The workgroup's wavefronts' sums, in their order.
__device__ __forceinline__ Sums join_waves(const Sums* joined, float c) {
    Sums all = joined[0];
#pragma unroll
    for (int w = 1; w < kTokenWaves; ++w) {
        Sums o = joined[w];
        const float higher = fmaxf(all.top, o.top);
        all.rise(higher, c);
        o.rise(higher, c);
        all.s += o.s;
        all.t += o.t;
    }
    return all;
}

// A logit's place among others: larger keys are larger logits, of equal ones the one of the lower index.  Never 0.
__device__ __forceinline__ uint64_t key_of(float z, uint32_t index) {
    const uint32_t bits = __float_as_uint(z + 0.0f);           // -0 and 0 are equal
    return uint64_t(bits ^ (int32_t(bits) < 0 ? 0xFFFFFFFFu : 0x80000000u)) << 32 | uint32_t(~index);
}
__device__ __forceinline__ float key_logit(uint64_t key) {
    const uint32_t o = uint32_t(key >> 32);
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
constexpr uint32_t kKeyOfMinusInf = 0x007FFFFFu;               // a key's upper half
__device__ __forceinline__ uint32_t key_index(uint64_t key) { return ~uint32_t(key); }

// Where row r starts, in elements; r and inner are below 2^31.
__device__ __forceinline__ int64_t row_at(const TokenRows& in, int64_t row) {
    const uint32_t r = uint32_t(row), inner = uint32_t(in.inner), group = r / inner;
    return group * in.group_stride + int64_t(r - group * inner) * in.row_stride;
}

// A row: elements [0, head) and [head + V vectors, n) one by one, those between in 16-byte vectors of V.
template <typename T>
struct Row {
    static constexpr int V = kVec16<T>;
    const T* p;
    int32_t n, head, vectors;
    __device__ __forceinline__ Row(const TokenRows& in, int64_t row) {
        p = static_cast<const T*>(in.logits) + row_at(in, row);
        n = int32_t(in.vocab);
        head = int32_t((-reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
        if (head > n) head = n;
        vectors = (n - head) / V;
    }
    __device__ __forceinline__ u32x4 vector(int32_t i) const {
        return load_word<u32x4, true>(p + head + int64_t(i) * V);
    }
    __device__ __forceinline__ int32_t edges() const { return n - vectors * V; }
    // The place of edge element e.
    __device__ __forceinline__ int32_t edge(int32_t e) const { return e < head ? e : e + vectors * V; }
};

// The row's results from its joined sums.
struct Finish {
    Base base;
    float l2;                  // log2 s
    __device__ __forceinline__ Finish(const Base& base, float s) : base(base), l2(__log2f(s)) {}
    __device__ __forceinline__ Finish(const Sums& a, float c) : Finish(Base(a.top, c), a.s) {}
    // An exponent may be past float32 where ln 2 times it is not (a token that the lowest value of its type rules out).
    __device__ __forceinline__ float logp(float z, float c) const {
        const float l = kLn2 * (base.exponent(z, c) - l2);
        return l == -__builtin_inff() ? 2.0f * ((0.5f * z - 0.5f * base.b) * (c * kLn2)) : l;
    }
    // b c may be too large where b / T = ln 2 b c is not.
    __device__ __forceinline__ float lse(float c) const { return base.far() ? base.b * (c * kLn2) + kLn2 * l2 : kLn2 * (base.bc + l2); }
};

// The target's logit, NaN without one.
template <typename T>
__device__ __forceinline__ float target_logit(const T* p, int64_t y, int32_t n) {
    return y >= 0 && y < n ? widen(p[y]) : __builtin_nanf("");
}
__device__ __forceinline__ void write_row(const TokenFwdArgs& a, int64_t row, float zy, const Sums& j, const Finish& f) {
    a.logp[row] = f.logp(zy, a.scale);
    a.lse[row] = f.lse(a.scale);
    if (a.entropy) a.entropy[row] = kLn2 * (f.l2 - j.t / j.s);
}
template <int LANES>
__device__ __forceinline__ void write_masked(const TokenFwdArgs& a, int64_t row) {
    if (threadIdx.x % LANES == 0) {
        a.logp[row] = 0.0f;
        a.lse[row] = 0.0f;
        if (a.entropy) a.entropy[row] = 0.0f;
    }
    for (int i = threadIdx.x % LANES; i < a.top_k; i += LANES) {
        a.top_logp[row * a.top_k + i] = 0.0f;
        a.top_index[row * a.top_k + i] = -1;
    }
}
__device__ __forceinline__ void write_top(const TokenFwdArgs& a, int64_t row, int rank, uint64_t key, const Finish& f) {
    const bool bad = !(f.l2 < __builtin_inff());               // a NaN or +inf among the logits
    a.top_logp[row * a.top_k + rank] = bad ? __builtin_nanf("") : f.logp(key_logit(key), a.scale);
    a.top_index[row * a.top_k + rank] = bad ? -1 : int64_t(key_index(key));
}

// How many of n keys in LDS are larger than `mine`.
__device__ __forceinline__ int rank_of(uint64_t mine, const uint64_t* keys, int n) {
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) rank += keys[i] > mine ? 1 : 0;
    return rank;
}
// The larger of two lanes' keys.
template <int CTRL>
__device__ __forceinline__ uint64_t larger_of(uint64_t key) {
    const uint64_t other = uint64_t(dpp_move<CTRL>(uint32_t(key >> 32))) << 32 | dpp_move<CTRL>(uint32_t(key));
    return other > key ? other : key;
}
// The k-th largest of 64 G keys in LDS (none of them equal, but for zeros), or 1 where fewer than k are not zero; in every
// lane.
template <int G>
__device__ __forceinline__ uint64_t bound_of(const uint64_t* keys, int k) {
    uint64_t mine[G];
    int rank[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        mine[g] = keys[64 * g + (threadIdx.x & 63)];
        rank[g] = 0;
    }
#pragma unroll 16
    for (int i = 0; i < 64 * G; ++i) {
        const uint64_t other = keys[i];
#pragma unroll
        for (int g = 0; g < G; ++g) rank[g] += other > mine[g] ? 1 : 0;
    }
    uint64_t bound = 1;
#pragma unroll
    for (int g = 0; g < G; ++g) {
        const uint64_t at = __ballot(mine[g] != 0 && rank[g] == k - 1);
        if (!at) continue;
        const int lane = int(__builtin_ctzll(at));
        bound = uint64_t(uint32_t(__builtin_amdgcn_readlane(int(uint32_t(mine[g] >> 32)), lane))) << 32 |
                uint32_t(__builtin_amdgcn_readlane(int(uint32_t(mine[g])), lane));
    }
    return bound;
}
// The lanes' largest keys to LDS: the quads', where there are twice as many of them as alternatives (so that the k-th of
// them is near the k-th of all), else every lane's.
__device__ __forceinline__ bool by_quads(int32_t vectors, int k) { return min(vectors, int32_t(kTokenThreads)) >= 8 * k; }
__device__ __forceinline__ void leave_heads(uint64_t* heads, uint64_t key, int32_t vectors, int k) {
    const uint64_t quad = larger_of<0x4E>(larger_of<0xB1>(key));
    if (!by_quads(vectors, k)) heads[threadIdx.x] = key;
    else if ((threadIdx.x & 3) == 0) heads[threadIdx.x >> 2] = quad;
}
// After the workgroup's barrier, the k-th of those; `found` is a word of LDS that holds 1.
__device__ __forceinline__ uint64_t bound_of_heads(const uint64_t* heads, int32_t vectors, int k, uint64_t* found) {
    if (by_quads(vectors, k)) return bound_of<1>(heads, k);
    const int n = min(vectors, int32_t(kTokenThreads));        // the lanes that have elements are the first ones
    const uint64_t mine = heads[threadIdx.x];
    if (mine != 0 && rank_of(mine, heads, n) == k - 1) *found = mine;
    __syncthreads();
    return *found;
}

constexpr int kTokenFound = 1024;          // candidates that there is room for
constexpr int kTokenList = 256;            // blocks, and lanes, likewise
static_assert(kTokenList >= kTokenThreads, "every lane may be listed");

// One workgroup a row, or a piece of it.
template <typename T, bool TOP>
__global__ void __launch_bounds__(kTokenThreads) token_fwd(const TokenFwdArgs a) {
    constexpr int V = kVec16<T>, U = 32 / V;                   // 32 elements a lane at a time
    __shared__ Sums joined[kTokenWaves];
    __shared__ __attribute__((aligned(16))) uint64_t found[TOP ? kTokenFound : 2];
    __shared__ __attribute__((aligned(16))) uint64_t heads[TOP ? kTokenThreads : 2];
    __shared__ float tops[TOP ? kTokenBlocks : 1][TOP ? kTokenThreads : 1];
    __shared__ int listed[TOP ? kTokenList : 1];
    __shared__ uint64_t bounds[2];
    __shared__ int count, some;
    const int tid = threadIdx.x;
    const float c = a.scale;
    for (int64_t item = blockIdx.x; item < a.in.rows * a.pieces; item += gridDim.x) {
        const int64_t row = a.pieces == 1 ? item : item / a.pieces;
        const int piece = a.pieces == 1 ? 0 : int(item % a.pieces);
        if (a.in.mask && !a.in.mask[row]) {
            if (piece == 0) write_masked<kTokenThreads>(a, row);
            continue;
        }
        const Row<T> r(a.in, row);
        const int32_t first = int32_t(piece * a.piece_vectors) < r.vectors ? int32_t(piece * a.piece_vectors) : r.vectors;
        const int32_t last = piece == a.pieces - 1 || r.vectors - first < a.piece_vectors ? r.vectors : first + int32_t(a.piece_vectors);
        Sums mine = Sums::none();
        Base base(mine.top, c);
        int blocks = 0;                    // the lane's, of U vectors each
        const auto block = [&](const u32x4 (&raw)[U], int live) {
            float z[U][V];
            float top = -__builtin_inff();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                widen_raw<T>(raw[u], z[u]);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    if (u >= live) z[u][k] = -__builtin_inff();
                    top = fmaxf(top, z[u][k]);
                }
            }
            if constexpr (TOP) tops[blocks][tid] = top;
            ++blocks;
            if (top > mine.top) {
                const Base there(top, c);
                mine.rise(top, base, there, c);
                base = there;
            }
            if (base.far()) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int k = 0; k < V; ++k) mine.add((z[u][k] - base.from) * c);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int k = 0; k < V; ++k) mine.add(fmaf(z[u][k], c, -base.bc));
            }
        };
        int32_t i = first + tid;
        for (; i + (U - 1) * kTokenThreads < last; i += U * kTokenThreads) {
            u32x4 raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) raw[u] = r.vector(i + u * kTokenThreads);
            block(raw, U);
        }
        if (i < last) {
            u32x4 raw[U];
            int live = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                raw[u] = u32x4{0, 0, 0, 0};
                if (i + u * kTokenThreads < last) {
                    raw[u] = r.vector(i + u * kTokenThreads);
                    live = u + 1;
                }
            }
            block(raw, live);
        }
        Sums all = mine;
        if (piece == 0 && tid < r.edges()) {                   // at most 2 (V - 1) elements outside the vectors
            const float z = widen(r.p[r.edge(tid)]);
            if (z > all.top) all.rise(z, c);
            all.add(Base(all.top, c).exponent(z, c));
        }
        // lanes to wavefronts to the workgroup
        all.join_lanes(c);
        __syncthreads();                   // the last row's LDS may still be read
        if ((tid & 63) == 0) joined[tid >> 6] = all;
        if (tid == 0) {
            count = some = 0;
            if constexpr (TOP) bounds[0] = bounds[1] = 1;
        }
        if constexpr (TOP) leave_heads(heads, blocks > 0 ? key_of(mine.top, uint32_t(tid)) : 0, last - first, a.top_k);
        __syncthreads();
        all = join_waves(joined, c);
        const Finish f(all, c);
        if (tid == 0) {
            if (a.pieces == 1) write_row(a, row, target_logit(r.p, a.targets[row], r.n), all, f);
            else a.part[item] = TokenPart{all.top, all.s, all.t, 0.0f};
        }
        if constexpr (TOP) {
            uint64_t bound = bound_of_heads(heads, last - first, a.top_k, &bounds[0]);
            const auto take = [&](float z, uint32_t index) {
                const uint64_t key = key_of(z, index);
                if (key < bound) return;
                const int place = atomicAdd(&count, 1);
                if (place < kTokenFound) found[place] = key;
            };
            const auto take_vector = [&](int32_t i) {
                float z[V];
                widen_raw<T>(r.vector(i), z);
#pragma unroll
                for (int k = 0; k < V; ++k) take(z[k], uint32_t(r.head + i * V + k));
            };
            const auto take_edges = [&]() {
                if (piece == 0 && tid < r.edges()) take(widen(r.p[r.edge(tid)]), uint32_t(r.edge(tid)));
            };
            if (bound > 1) bound &= 0xFFFFFFFF00000000ull;     // any index
            const float least = key_logit(bound);
            for (int b = 0; b < blocks; ++b)
                if (bound == 1 || tops[b][tid] >= least) {
                    const int place = atomicAdd(&some, 1);
                    if (place < kTokenList) listed[place] = first + tid + b * (U * kTokenThreads);
                }
            take_edges();
            __syncthreads();
            if (some <= kTokenList) {
                for (int j = tid; j < some * U; j += kTokenThreads) {
                    const int32_t i = listed[j / U] + j % U * kTokenThreads;
                    if (i < last) take_vector(i);
                }
            }
            __syncthreads();
            if (some > kTokenList || count > kTokenFound) {    // uniform
                uint64_t best = 0;         // the lane's largest element at its first place
                for (int b = blocks - 1; b >= 0; --b)
                    if (tops[b][tid] == mine.top)
                        for (int u = U - 1; u >= 0; --u) {
                            const int32_t i = first + tid + (b * U + u) * kTokenThreads;
                            if (i >= last) continue;
                            float z[V];
                            widen_raw<T>(r.vector(i), z);
#pragma unroll
                            for (int k = V - 1; k >= 0; --k)
                                if (z[k] == mine.top) best = key_of(z[k], uint32_t(r.head + i * V + k));
                        }
                __syncthreads();
                leave_heads(heads, best, last - first, a.top_k);
                if (tid == 0) count = some = 0;
                __syncthreads();
                bound = bound_of_heads(heads, last - first, a.top_k, &bounds[1]);
                if (best >= bound) listed[atomicAdd(&some, 1)] = tid;
                take_edges();
                __syncthreads();
                const int32_t each = (last - first + kTokenThreads - 1) / kTokenThreads, all_vectors = some * each;
                constexpr int32_t kStep = (kTokenFound - kTokenMaxTop - 2 * V) / V;
                for (int32_t from = 0; from < all_vectors; from += kStep) {
                    const int32_t to = from + kStep < all_vectors ? from + kStep : all_vectors;
                    for (int32_t v = from + tid; v < to; v += kTokenThreads) {
                        const int32_t i = first + listed[v / each] + v % each * kTokenThreads;
                        if (i < last) take_vector(i);
                    }
                    __syncthreads();
                    const int n = count;
                    uint64_t held[kTokenFound / kTokenThreads];
                    int rank[kTokenFound / kTokenThreads];
#pragma unroll
                    for (int q = 0; q < kTokenFound / kTokenThreads; ++q) {
                        const int j = q * kTokenThreads + tid;
                        held[q] = j < n ? found[j] : 0;
                        rank[q] = j < n ? rank_of(held[q], found, n) : kTokenFound;
                    }
                    __syncthreads();       // every lane has read them
#pragma unroll
                    for (int q = 0; q < kTokenFound / kTokenThreads; ++q)
                        if (rank[q] < a.top_k) found[rank[q]] = held[q];
                    if (tid == 0 && n > a.top_k) count = a.top_k;
                    __syncthreads();
                    if (n >= a.top_k) bound = found[a.top_k - 1];
                }
            }
            const int n = count;
            for (int j = tid; j < n || j < a.top_k; j += kTokenThreads) {
                // a piece of fewer than k elements gives keys of 0 past them
                const uint64_t key = j < n ? found[j] : 0;
                const int rank = j < n ? rank_of(key, found, n) : j;
                if (rank >= a.top_k) continue;
                if (a.pieces == 1) write_top(a, row, rank, key, f);
                else a.part_top[item * a.top_k + rank] = key;
            }
        }
    }
}

constexpr int kShortFound = 256;           // candidates of a wavefront that there is room for
constexpr int kShortMany = 96;             // more of them cost more to rank than to thin out

// One wavefront a row of up to 64 E elements, which stay in its registers: one maximum for all lanes, no barrier, and the
// alternatives' elements are found again in registers.  Their bound is the k-th largest of the lanes' largest, raised by
// bisection where it leaves many; where equal logits still bring more than there is room for to it, the k-th largest key
// itself, bit by bit.  20480 rows of 1000 bf16 take 16.5 us (7 to read them), with 20 alternatives 37, with 64 73: a wavefront's
// instructions, 33 passes of a comparison and its count among them (with 64 and no bisection 325, a quarter of the rows bit by
// bit).
template <typename T, int E, bool TOP>
__global__ void __launch_bounds__(kTokenThreads, E > 32 && sizeof(T) == 2 ? 4 : 1) token_short(const TokenFwdArgs a) {
    constexpr int V = kVec16<T>, U = E / V;
    __shared__ uint64_t room[kTokenWaves][TOP ? kShortFound : 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
    const int32_t n = int32_t(a.in.vocab), vectors = n / V;
    const float c = a.scale;
    for (int64_t row = int64_t(blockIdx.x) * kTokenWaves + wave; row < a.in.rows; row += int64_t(gridDim.x) * kTokenWaves) {
        if (a.in.mask && !a.in.mask[row]) {
            write_masked<64>(a, row);
            continue;
        }
        const T* p = static_cast<const T*>(a.in.logits) + row_at(a.in, row);
        const int64_t y = a.targets[row];
        // vector u of a lane is the row's vector 64 u + lane; the elements past the last vector go to the first lanes
        u32x4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            raw[u] = u32x4{0, 0, 0, 0};
            if (64 * u + lane < vectors) raw[u] = load_word<typename Unaligned16<T>::type, true>(p + (64 * u + lane) * V);
        }
        const bool has_last = vectors * V + lane < n;
        const float last = has_last ? widen(p[vectors * V + lane]) : -__builtin_inff();
        const float zy = lane == 0 ? target_logit(p, y, n) : 0.0f;
        float z[U][V], mine = last == last ? last : -__builtin_inff();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            widen_raw<T>(raw[u], z[u]);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if (64 * u + lane >= vectors) z[u][k] = -__builtin_inff();
                mine = fmaxf(mine, z[u][k]);
            }
        }
        Sums all{wave_top(mine), 0.0f, 0.0f};
        const Base base = Base(all.top, c).uniform();
        all.add(base.exponent(last, c));
        if (base.far()) {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < V; ++k) all.add((z[u][k] - base.from) * c);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < V; ++k) all.add(fmaf(z[u][k], c, -base.bc));
        }
        all.s = wave_sum(all.s);
        all.t = wave_sum(all.t);
        const Finish f(base, all.s);
        if (lane == 0) write_row(a, row, zy, all, f);
        if constexpr (TOP) {
            if (!(f.l2 < __builtin_inff())) {                  // a NaN or +inf among the logits
                if (lane < a.top_k) write_top(a, row, lane, 0, f);
                continue;
            }
            // Calls f(logit, index, whether it is one of the row's) for the lane's elements, one after the other.
            const auto each = [&](auto&& f) {
                int at = lane;             // anew, so that no pass keeps all its indexes for the next
                asm volatile("" : "+v"(at));
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int k = 0; k < V; ++k) f(z[u][k], (64 * u + at) * V + k, 64 * u + at < vectors);
                f(last, vectors * V + at, vectors * V + at < n);
            };
            const auto how_many = [&](auto&& which) {
                int m = 0;
                each([&](float z, int index, bool live) { m += int(__popcll(__ballot(live && which(z, index)))); });
                return m;
            };
            uint64_t* found = room[wave];
            int count = 0;
            const auto collect = [&](auto&& which) {
                each([&](float z, int index, bool live) {
                    const bool take = live && which(z, index);
                    const uint64_t those = __ballot(take);
                    if (!those) return;
                    const int place = count + int(__builtin_amdgcn_mbcnt_hi(uint32_t(those >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(those), 0)));
                    if (take && place < kShortFound) found[place] = key_of(z, uint32_t(index));
                    count += int(__popcll(those));
                });
            };
            float bound = all.top;
            if (a.top_k > 1) {
                int larger = 0;
#pragma unroll
                for (int i = 0; i < 64; ++i) larger += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine), i)) > mine ? 1 : 0;
                bound = -wave_top(larger < a.top_k ? -mine : -__builtin_inff());
            }
            collect([&](float z, int) { return z >= bound; });
            if (count > kShortMany) {      // uniform: a tighter bound, nearer to the maximum
                if (bound == -__builtin_inff()) {          // fewer lanes than alternatives: the smallest logit above -inf
                    float low = __builtin_inff();
                    each([&](float z, int, bool live) { low = live && z > -__builtin_inff() ? fminf(low, z) : low; });
                    low = -wave_top(-low);
                    const int m = how_many([&](float z, int) { return z >= low; });
                    if (m >= a.top_k) {
                        bound = low;
                        count = m;
                    }
                }
                float above = bound == -__builtin_inff() ? bound : all.top;
#pragma unroll 1
                for (int i = 0; i < 8 && count > kShortMany && bound < above; ++i) {
                    const float middle = 0.5f * bound + 0.5f * above;
                    const int m = how_many([&](float z, int) { return z >= middle; });
                    if (m >= a.top_k) {
                        bound = middle;
                        count = m;
                    } else {
                        above = middle;
                    }
                }
                if (count <= kShortFound) {
                    count = 0;
                    collect([&](float z, int) { return z >= bound; });
                }
            }
            if (count > kShortFound) {
                // the k-th largest logit by the bits of its key, then the smallest index that leaves k of them
                uint32_t key = 0;
#pragma unroll 1
                for (int b = 31; b >= 0; --b) {
                    const uint32_t trial = key | 1u << b;
                    const float least = key_logit(uint64_t(trial) << 32);      // NaN below -inf
                    if (trial <= kKeyOfMinusInf || how_many([&](float z, int) { return z >= least; }) >= a.top_k) key = trial;
                }
                const float least = key_logit(uint64_t(key) << 32);
                int behind = 0;
#pragma unroll 1
                for (int b = 12; b >= 0; --b) {
                    const int trial = behind | ((1 << b) - 1);
                    if (how_many([&](float z, int index) { return z > least || (z == least && index <= trial); }) < a.top_k) behind |= 1 << b;
                }
                count = 0;
                collect([&](float z, int index) { return z > least || (z == least && index <= behind); });
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            for (int j = lane; j < count; j += 64) {
                const int rank = rank_of(found[j], found, count);
                if (rank < a.top_k) write_top(a, row, rank, found[j], f);
            }
            __builtin_amdgcn_wave_barrier();                   // the next row writes there
        }
    }
}

// A row's pieces joined: the sums in piece order, and the k largest of the pieces' k largest likewise.
template <typename T>
__global__ void __launch_bounds__(kTokenThreads) token_join(const TokenFwdArgs a) {
    __shared__ uint64_t heads[128];
    __shared__ uint64_t found[kTokenMaxKeys];
    __shared__ int count;
    const int tid = threadIdx.x, lane = tid & 63;
    const float c = a.scale;
    static_assert(kTokenMaxPieces <= 64, "a lane a piece");
    constexpr int kMine = kTokenMaxKeys / kTokenThreads;
    for (int64_t row = blockIdx.x; row < a.in.rows; row += gridDim.x) {
        if (a.in.mask && !a.in.mask[row]) continue;            // written by its first piece
        const int64_t y = a.targets[row];
        const uint64_t* keys = a.part_top + row * a.pieces * a.top_k;
        const int all_keys = a.pieces * a.top_k;
        Sums all = Sums::none();           // each wavefront joins the pieces, a lane a piece
        if (lane < a.pieces) {
            const TokenPart p = a.part[row * a.pieces + lane];
            all = Sums{p.top, p.sum, p.weighted};
        }
        uint64_t mine[kMine];              // all loads on their way at once
#pragma unroll
        for (int q = 0; q < kMine; ++q) mine[q] = q * kTokenThreads + tid < all_keys ? keys[q * kTokenThreads + tid] : 0;
        uint64_t head = 0;                 // the first few keys of each piece, k of them at least
        if (tid < 128 && a.top_k > 0) {
            const int few = min(a.top_k, 128 / a.pieces), p = tid / few;
            if (p < a.pieces) head = keys[p * a.top_k + tid % few];
        }
        const Row<T> r(a.in, row);
        const float zy = tid == 0 ? target_logit(r.p, y, r.n) : 0.0f;
        __syncthreads();                   // the last row's LDS may still be read
        if (tid < 128) heads[tid] = head;
        if (tid == 0) count = 0;
        all.join_lanes(c);
        const Finish f(all, c);
        if (!(f.l2 < __builtin_inff())) {  // a NaN or +inf among the logits: pieces of NaN alone may have left no keys
            if (tid < a.top_k) write_top(a, row, tid, 0, f);
        } else if (a.top_k > 0) {
            __syncthreads();
            const uint64_t bound = bound_of<2>(heads, a.top_k);
#pragma unroll
            for (int q = 0; q < kMine; ++q)
                if (q * kTokenThreads + tid < all_keys && mine[q] >= bound) found[atomicAdd(&count, 1)] = mine[q];
            __syncthreads();
            for (int j = tid; j < count; j += kTokenThreads) {
                const int rank = rank_of(found[j], found, count);
                if (rank < a.top_k) write_top(a, row, rank, found[j], f);
            }
        }
        if (tid == 0) write_row(a, row, zy, all, f);
    }
}

// A row's sums, in each of the LANES that have it.
template <typename T, int LANES>
__device__ __forceinline__ Sums sums_of_row(const T* x, int32_t n, int tid, float c, Sums* joined) {
    constexpr int V = kVec16<T>;
    const int32_t vectors = n / V;
    Sums all = Sums::none();
    const auto add = [&](float z) {
        if (z > all.top) all.rise(z, c);
        all.add(Base(all.top, c).exponent(z, c));
    };
#pragma unroll 1
    for (int32_t i = tid; i < vectors; i += LANES) {
        float z[V];
        widen_raw<T>(load_word<typename Unaligned16<T>::type, true>(x + int64_t(i) * V), z);
#pragma unroll
        for (int k = 0; k < V; ++k) add(z[k]);
    }
    if (vectors * V + tid < n) add(widen(x[vectors * V + tid]));
    all.join_lanes(c);
    if constexpr (LANES > 64) {
        __syncthreads();                   // the last row's LDS may still be read
        if ((tid & 63) == 0) joined[tid >> 6] = all;
        __syncthreads();
        all = join_waves(joined, c);
    }
    return all;
}

// The gradient of sum(grad_logp logp + grad_entropy H): with p = exp(z / T - lse),
//   dz_v = (grad_logp ((v == y) - p_v) - grad_entropy p_v (log p_v + H)) / T.
// Vectors are cut where the gradient's row is aligned, and stored past the caches, which then hold more of the logits:
// 3000 x 128256 bf16 287 us (5.4 TB/s) instead of 303, 4096 x 32000 79 instead of 106.  Rows whose lse is so large that float32
// does not hold its fraction (a mask that leaves nothing but the type's lowest value) form their sums anew.
template <typename T, int LANES>
__global__ void __launch_bounds__(kTokenThreads) token_bwd(const TokenBwdArgs a) {
    constexpr int V = kVec16<T>, ITEMS = kTokenThreads / LANES;
    __shared__ Sums joined[LANES > 64 ? kTokenWaves : 1];
    const int tid = threadIdx.x % LANES, which = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / LANES);
    for (int64_t item = int64_t(blockIdx.x) * ITEMS + which; item < a.in.rows * a.pieces; item += int64_t(gridDim.x) * ITEMS) {
        const int64_t row = a.pieces == 1 ? item : item / a.pieces;
        const int piece = a.pieces == 1 ? 0 : int(item % a.pieces);
        const int32_t n = int32_t(a.in.vocab);
        const T* x = static_cast<const T*>(a.in.logits) + row_at(a.in, row);
        T* out = static_cast<T*>(a.grad) + row * a.in.vocab;
        int32_t head = int32_t((-reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T));
        if (head > n) head = n;
        const int32_t vectors = (n - head) / V, edges = n - vectors * V;
        const int32_t first = int32_t(piece * a.piece_vectors) < vectors ? int32_t(piece * a.piece_vectors) : vectors;
        int32_t last = piece == a.pieces - 1 || vectors - first < a.piece_vectors ? vectors : first + int32_t(a.piece_vectors);
        const int32_t edge = tid < head ? tid : tid + vectors * V;
        if (a.in.mask && !a.in.mask[row]) {
            if (piece == 0 && tid < edges) out[edge] = T(0.0f);
            for (int32_t i = first + tid; i < last; i += LANES)
                store_word<true>(out + head + int64_t(i) * V, u32x4{0, 0, 0, 0});
            continue;
        }
        const float lse = a.lse[row], g = a.grad_logp ? a.grad_logp[row] : 0.0f;
        const float h = a.grad_entropy ? a.grad_entropy[row] : 0.0f;
        const float k0 = a.grad_entropy ? fmaf(h, a.entropy[row], g) : g;      // g + h H
        const int64_t target = a.targets[row];
        const int32_t y = target >= 0 && target < n ? int32_t(target) : -1;
        // Of an element with log-probability l.
        const auto value = [&](float l, int32_t v) {
            l = hold(l);
            const float p = exp2_hw(l * kLog2e);
            return a.inv_t * ((v == y ? g : 0.0f) - p * fmaf(h, l, k0));
        };
        const auto write_edge = [&](auto logp) {
            if (piece == 0 && tid < edges) out[edge] = T(value(logp(widen(x[edge])), edge));
        };
        const auto write_vector = [&](int32_t i, auto logp) {
            const int32_t v = head + i * V;
            float z[V];
            widen_raw<T>(load_word<typename Unaligned16<T>::type, true>(x + v), z);
#pragma unroll
            for (int k = 0; k < V; ++k) z[k] = value(logp(z[k]), v + k);
            __builtin_nontemporal_store(narrow_raw<T>(z), reinterpret_cast<u32x4*>(out + v));
        };
        const int run = (a.pieces + kTokenFarPieces - 1) / kTokenFarPieces;
        if (__builtin_expect(!(fabsf(lse) >= kTokenFar), 1)) {
            const auto logp = [&](float z) { return fmaf(z, a.inv_t, -lse); };
            write_edge(logp);
#pragma unroll 4
            for (int32_t i = first + tid; i < last; i += LANES) write_vector(i, logp);
        } else if (piece % run == 0) {                         // uniform in the lanes of a row
            const int64_t many = run * a.piece_vectors;
            last = vectors - first < many ? vectors : first + int32_t(many);
            const Finish f(sums_of_row<T, LANES>(x, n, tid, a.scale, joined), a.scale);
            const auto logp = [&](float z) { return kLn2 * (f.base.exponent(z, a.scale) - f.l2); };
            write_edge(logp);
#pragma unroll 1
            for (int32_t i = first + tid; i < last; i += LANES) write_vector(i, logp);
        }
    }
}

template <typename T, bool TOP>
const void* fwd_of(int64_t vocab) {
    if (vocab <= 512) return reinterpret_cast<const void*>(&token_short<T, 8, TOP>);
    if (vocab <= 2048) return reinterpret_cast<const void*>(&token_short<T, 32, TOP>);
    if (vocab <= kTokenShort) return reinterpret_cast<const void*>(&token_short<T, 64, TOP>);
    return reinterpret_cast<const void*>(&token_fwd<T, TOP>);
}
template <typename T>
const void* fwd_of(bool top, int64_t vocab) { return top ? fwd_of<T, true>(vocab) : fwd_of<T, false>(vocab); }

}  // namespace

const void* pick_token_fwd(int dtype, bool top, int64_t vocab) {
    switch (dtype) {
    case kF32: return fwd_of<float>(top, vocab);
    case kF16: return fwd_of<_Float16>(top, vocab);
    case kBF16: return fwd_of<__bf16>(top, vocab);
    }
    return nullptr;
}
const void* pick_token_join(int dtype) {
    switch (dtype) {
    case kF32: return reinterpret_cast<const void*>(&token_join<float>);
    case kF16: return reinterpret_cast<const void*>(&token_join<_Float16>);
    case kBF16: return reinterpret_cast<const void*>(&token_join<__bf16>);
    }
    return nullptr;
}
template <typename T>
const void* bwd_of(int64_t vocab) {
    return vocab <= kTokenShortBwd ? reinterpret_cast<const void*>(&token_bwd<T, 64>) : reinterpret_cast<const void*>(&token_bwd<T, kTokenThreads>);
}
const void* pick_token_bwd(int dtype, int64_t vocab) {
    switch (dtype) {
    case kF32: return bwd_of<float>(vocab);
    case kF16: return bwd_of<_Float16>(vocab);
    case kBF16: return bwd_of<__bf16>(vocab);
    }
    return nullptr;
}

}  // namespace rlpl
