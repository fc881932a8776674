// sft_logprob.hip -- log probabilities of given tokens from rows of logits,
// with the rows' entropy and likeliest alternatives, and the gradient.
//
//     logp = scale (z_t - M) - L,  L = ln S,  S = sum e^(scale (z_j - M)),  M = max z_j
//     entropy = L - (sum e^(scale (z_j - M)) scale (z_j - M)) / S
//     dz_j = scale (dlogp ([j = t] - p_j) - dentropy p_j (ln p_j + entropy))
//
// The forward pass reads a row once, keeping in every thread the largest logit
// so far, m, and relative to it the sums of e^(scale (z - m)) and of that
// times scale (z - m); the threads' parts are joined at the row's end.  The
// gradient reads a row and its statistics and writes a row.  Both are bound by
// HBM: 4096 x 32000 in bf16 takes 45.2 us (262 MB read, 5.8 TB/s; the vector
// units are busy for most of it, as an entropy needs about ten operations a
// logit), its gradient 82 us (5.8 TB/s, rows without one only written); 1003 x
// 50001 in fp32 with 5 alternatives 37 us.  Few long rows are bound by their
// CUs instead, about 70 ps a logit in bf16: 8 x 32000 takes 4.5 us, with 20
// alternatives 6.9, of which about 1.2 are passing over the logits that reach
// their bound.  Where the alternatives are looked for one by one, all logits
// equal, 4096 x 32000 with 20 takes about 1 ms, not 55 us.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "sft_blocks.h"
#include "sft_internal.h"
#include "sft_probe.h"
#include "sft_vec.h"

namespace {

using namespace sft;

constexpr float kInf = __builtin_huge_valf(), kLargest = __FLT_MAX__;
constexpr float kLn2 = 0.693147180559945309f;
// Powers of two below this one are 0 in fp32; a bound for exponents that may
// be minus infinity and get multiplied by 0.
constexpr float kNothing = -1000.0f;
// Products with c (scale in units of log2) up to this size are off by a quarter
// at most, which the differences from them carry and L takes off again.  Beyond,
// the rounding itself grows past what a power of two can hold: a thread whose
// logits are all below -kFar / c keeps -kFar, relative to which they are nothing,
// and a row whose largest is as far is summed again, differences first.
constexpr float kFar = 8388608.0f;
constexpr int kMaxTop = 64;

__device__ __forceinline__ float max3(float a, float b, float c) {
    // (a NaN among the logits may take m's place for a while; its row's sums
    // tell, and the row is then read in another way)
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float limit(float x, float lo, float hi) { return __builtin_amdgcn_fmed3f(x, lo, hi); }

// Order of floats (without NaN; the two zeros are one value) as unsigned integers; 0 is below all of them.
__host__ __device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = float_bits(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__host__ __device__ __forceinline__ float float_of(uint32_t order) {
    return bits_float(order & 0x80000000u ? order & 0x7fffffffu : ~order);
}
// Larger for a larger logit, of equal ones for the lower index.
__device__ __forceinline__ uint64_t key_of(float z, uint32_t at) { return uint64_t(order_of(z)) << 32 | (0xffffffffu - at); }

struct Logprob {
    const void *z;
    const int32_t *target;
    float *logp, *stats, *entropy, *top_logp;
    int32_t *top_index;
    int64_t ld;
    int32_t N, V, top;
    float scale, c;                // c = scale * log2(e)
};

// A row's running state in one slot, relative to m2, the largest logit so far times c.
struct Running {
    float m2, sum, along;
};

// Takes up n logits, after others where there are any (begun); returns the largest of them.
template <bool kEntropy, int n>
__device__ __forceinline__ float take_up(Running &r, const float (&z)[n], float c, bool begun) {
    float own = -kInf;
#pragma unroll
    for (int i = 0; i < n; i += 2) own = max3(own, z[i], z[i + 1]);
    const float m2 = __builtin_fmaxf(own * c, r.m2);      // (-kFar at first)
    if (begun) {
        const float less = limit(r.m2 - m2, kNothing, 0.0f), part = exp2_of(less);
        r.along = kEntropy ? part * __builtin_fmaf(r.sum, less, r.along) : 0.0f;
        r.sum *= part;
    }
    r.m2 = m2;
#pragma unroll
    for (int i = 0; i < n; ++i) {
        const float d = __builtin_fmaf(z[i], c, -m2), e = exp2_of(d);
        r.sum += e;
        if (kEntropy) r.along = __builtin_fmaf(e, __builtin_fmaxf(d, kNothing), r.along);
    }
    return own;
}

// Where 256 threads that sum four quarters of a row keep them.
template <int kThreads>
struct Quarters {
    static constexpr int kOf = kThreads == 256 ? 256 : 1;
    float m2[4][kOf], sum[4][kOf], along[4][kOf];
    __device__ __forceinline__ Running get(int q) const {
        return Running{m2[q][threadIdx.x], sum[q][threadIdx.x], along[q][threadIdx.x]};
    }
    __device__ __forceinline__ void put(int q, const Running &r) {
        m2[q][threadIdx.x] = r.m2, sum[q][threadIdx.x] = r.sum, along[q][threadIdx.x] = r.along;
    }
};

// Halves K values over pairs of lanes: the sums of the first half stay where
// `up` is false, those of the second in the others.
template <int kControl, int K>
__device__ __forceinline__ void halve(const float (&x)[K], bool up, float (&y)[(K + 1) / 2]) {
    if constexpr (K == 1) {
        y[0] = x[0] + dpp<kControl>(x[0]);
    } else {
#pragma unroll
        for (int i = 0; i < K / 2; ++i) y[i] = (up ? x[i + K / 2] : x[i]) + dpp<kControl>(up ? x[i] : x[i + K / 2]);
    }
}

// Sums of K values (1, 2, 4 or 8) over a wave, the k-th in lanes of k * 16 / K on.
// Lanes that would add the same share the values out between them, which makes
// 8 sums cost little more than 2; the order of a sum is the same for any K.
template <int K>
__device__ __forceinline__ float sums_of(const float (&x)[K]) {
    const int lane = static_cast<int>(threadIdx.x);
    float a[(K + 1) / 2], b[(K + 3) / 4], c[1];
    halve<0x128>(x, lane & 8, a);          // over lanes 8 apart, mirrored within 8, 2 apart, neighbours
    halve<0x141>(a, lane & 4, b);
    halve<0x4e>(b, lane & 2, c);
    float s = c[0] + dpp<0xb1>(c[0]);
    const u32x2 t = __builtin_amdgcn_permlane16_swap(float_bits(s), float_bits(s), false, false);
    s = bits_float(t.x) + bits_float(t.y);
    const u32x2 u = __builtin_amdgcn_permlane32_swap(float_bits(s), float_bits(s), false, false);
    return bits_float(u.x) + bits_float(u.y);
}

template <class Op, int kThreads>
__device__ __forceinline__ float block_of(float x, float *red) {
    x = lanes_of<Op, 64>(x);
    if constexpr (kThreads > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
        __syncthreads();
        x = red[0];
#pragma unroll
        for (int i = 1; i < kThreads / 64; ++i) x = Op::of(x, red[i]);
    }
    return x;
}

__device__ __forceinline__ uint64_t wave_max(uint64_t x) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint64_t y = __shfl_xor(x, d);
        x = y > x ? y : x;
    }
    return x;
}

template <class Z>
__device__ __forceinline__ float logit(const typename Z::type *z, int at) {
    return Z::up(z[at]);
}

// How a row's logits are shared out: by rounds of 4 waves (or of the single one
// that a short row has), of which a wave takes a run of R logits a lane, its lanes
// groups of it by turns.  Rows of up to kLong logits have 256 threads that
// take all rounds.  Longer rows have four quarters of the rounds, each summed on
// its own: 1024 threads take them side by side, 256 one after the other.  So the
// order of a row's sums goes by V and the type alone, whatever the address and
// however many rows there are.  A run's lines are whole but for the first and the
// last, which keeps loads past L2 worth while where rows start between lines.
constexpr int kRound = 32;
constexpr int kLong = 16384;

// wave: 0 to 3 (0 of a single one).
template <class Z, int kThreads, int R>
__device__ __forceinline__ int place_of(int round, int step, int wave, int lane) {
    return (round * (kThreads == 64 ? 1 : 4) + wave) * (64 * R) + (step * 64 + lane) * Z::kGroup;
}

// N elements of 2 bytes from an odd one on, by words: an access that starts
// between words takes longer (1000 x 50001 in bf16: 26.4 us, by words 21.1).  The
// first and the last word hold one of them each; their other halves may lie
// outside the row, but never on another page.
template <class Z, int N>
__device__ __forceinline__ Raw<Z, N> get_odd(const typename Z::type *p) {
    const Raw<Z, N> a = get<Z, N, true>(p - 1);
    const uint32_t next = *reinterpret_cast<const typename Z::word *>(p + N - 1);
    Raw<Z, N> r;
#pragma unroll
    for (int i = 0; i < words_of<Z, N>; ++i)
        r.w[i] = __builtin_amdgcn_alignbit(i + 1 < words_of<Z, N> ? a.w[i + 1] : next, a.w[i], 16);
    return r;
}

// The first logit behind those in groups: the last few of a row go to the first
// threads one each, but for the rows of a wave.
template <class Z, int kThreads>
__device__ __forceinline__ int grouped(int V) {
    return kThreads > 64 ? V & ~(Z::kGroup - 1) : V;
}

// What a workgroup looks for a row's alternatives with.  The rounds of a row
// are taken in up to kBlocks blocks of `rounds` rounds, and each thread's largest
// logit of each block is kept.  A wave has less room, so that many fit a CU.
template <int kThreads>
constexpr int kBlocks = kThreads == 64 ? 1 : 8;       // (a wave's rows are one round)

template <int kThreads, int kTop>
struct TopPlace {
    static constexpr int kFound = kThreads == 64 ? 512 : 1024;
    static constexpr int kItems = kTop == 1 ? 1 : kThreads == 64 ? 64 : 1024;
    union {
        struct {
            uint64_t found[kFound];
            int32_t item[kItems];
        };
        Quarters<kThreads> quarters;      // until the sums are joined
    };
    float mine[kThreads], block[kTop == 2 ? kBlocks<kThreads> : 1][kTop == 2 ? kThreads : 1];
    float threshold, M, L;
    bool plain;
    int items, n;
};

struct Or {
    static __device__ __forceinline__ float of(float a, float b) { return bits_float(float_bits(a) | float_bits(b)); }
};

// A bound that at least `want` and hardly more of `all` values reach (want <= all),
// found by halving from the first bit on in which they differ to the last (in bf16
// the lower half never does), two bits at a time.  one: any of them; differ: the
// bits in which another differs from it, not 0 (the loop's end needs one);
// reached(b): how many are b or larger.
template <class Reached>
__host__ __device__ __forceinline__ uint32_t bound_bits(uint32_t one, uint32_t differ, uint32_t want, uint32_t all,
                                                        const Reached &reached) {
    const uint32_t top = (31u - static_cast<uint32_t>(__builtin_clz(differ))) | 1u, least = differ & (0u - differ);
    uint32_t bound = one & ~((2u << top) - 1u), bit = 1u << top, reach = all;
    const uint32_t enough = want + want / 4, most = enough < all ? enough : all - 1u;      // (all of them reach the prefix alone)
    do {
        const uint32_t b1 = bound | bit >> 1, b2 = bound | bit, b3 = b1 | b2;
        const uint32_t r1 = reached(b1), r2 = reached(b2), r3 = reached(b3);
        if (r1 >= want) bound = b1, reach = r1;
        if (r2 >= want) bound = b2, reach = r2;
        if (r3 >= want) bound = b3, reach = r3;
        bit >>= 2;
    } while ((bit >= least) & (reach > most));
    return bound;
}

// The same of kParts values of each lane of a wave.
template <int kParts>
__device__ __forceinline__ float bound_among(const uint32_t (&o)[kParts], uint32_t want) {
    const uint32_t one = __builtin_amdgcn_readfirstlane(o[0]);
    uint32_t differ = 0;
#pragma unroll
    for (int i = 0; i < kParts; ++i) differ |= o[i] ^ one;
    differ = __builtin_amdgcn_readfirstlane(float_bits(lanes_of<Or, 64>(bits_float(differ))));
    if (differ == 0) return float_of(one);
    return float_of(bound_bits(one, differ, want, 64 * kParts, [&](uint32_t b) {
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < kParts; ++i) n += static_cast<uint32_t>(__builtin_popcountll(__ballot(o[i] >= b)));
        return n;
    }));
}

// A bound that at least K of a row's logits reach (K <= 64), by one wave: about
// the K-th largest of 64, each of them the largest of every 64th thread.  With the
// statistics computed meanwhile, 64 x 50001 in bf16 with 20 alternatives took
// 10.6 us, one after the other and to the last bit 11.7.  For many alternatives
// it is one of 128, or much more than they would reach it (4096 x 32000 in bf16
// with 64: 73 us, of 64 137; with 33: 56.5 and 58.7).
template <int kThreads>
__device__ __forceinline__ float bound_of(const float *mine, int K) {
    constexpr int kEach = kThreads / 64;
    const int lane = static_cast<int>(threadIdx.x) & 63;
    float x = mine[lane], y = -kInf;
    if constexpr (kEach > 1) {
        y = mine[lane + 64];
#pragma unroll
        for (int i = 2; i < kEach; i += 2) {
            x = __builtin_fmaxf(x, mine[lane + 64 * i]);
            y = __builtin_fmaxf(y, mine[lane + 64 * i + 64]);
        }
        if (K > 32) return bound_among<2>({order_of(x), order_of(y)}, K);
    }
    return bound_among<1>({order_of(__builtin_fmaxf(x, y))}, K);
}

// Logits of a row that reach the bound: those of rows of one round (kTop = 1)
// from the registers that still hold them, of others the blocks of a thread's
// turns that have one.  A wave on its own counts without atomics (50000 x 300
// in bf16, 5 alternatives: 55 us, with them 72; where the wave holds 2048 it
// loses, 30000 x 2000 62 us, by blocks 48).
template <class Z, int kThreads, int kTop, int R>
__device__ __forceinline__ void collect(const float (&last)[R], float behind, float mine, int whole, int count, int rounds,
                                        TopPlace<kThreads, kTop> &s) {
    constexpr int N = Z::kGroup, kFound = TopPlace<kThreads, kTop>::kFound;
    constexpr int kItems = TopPlace<kThreads, kTop>::kItems;
    int thread = static_cast<int>(threadIdx.x);
    if constexpr (kTop == 1) asm volatile("" : "+v"(thread));     // or the places of all logits stay in registers between rows
    const int wave = __builtin_amdgcn_readfirstlane(thread >> 6);
    const float threshold = s.threshold;
    const auto keep = [&](float x, int at) {
        const int k = atomicAdd(&s.n, 1);
        if (k < kFound) s.found[k] = key_of(x, at);
    };
    if constexpr (kTop == 1 && kThreads == 64) {
        static_assert(64 * R <= kFound);
        int n = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const uint64_t which = __ballot(last[i] >= threshold);      // (-infinity behind the row's end)
            if (which == 0) continue;
            const int k = n + __builtin_popcountll(which & ((uint64_t(1) << thread) - 1));
            if (last[i] >= threshold) s.found[k] = key_of(last[i], place_of<Z, 64, R>(0, i / N, 0, thread) + i % N);
            n += __builtin_popcountll(which);
        }
        if (thread == 0) s.n = n;
    } else if (mine >= threshold) {
        if (behind >= threshold) keep(behind, whole + thread);
        if constexpr (kTop == 1) {
#pragma unroll
            for (int g = 0; g < R; g += 8) {
                float most = last[g];
#pragma unroll
                for (int i = 1; i < 8; ++i) most = __builtin_fmaxf(most, last[g + i]);
                if (!(most >= threshold)) continue;
#pragma unroll
                for (int i = g; i < g + 8; ++i)
                    if (last[i] >= threshold) keep(last[i], place_of<Z, kThreads, R>(wave >> 2, i / N, wave & 3, thread & 63) + i % N);
            }
        } else {
            uint32_t hits = 0;
            const int blocks = (count + rounds - 1) / rounds;
#pragma unroll
            for (int b = kBlocks<kThreads> - 1; b >= 0; --b)
                hits += hits + (b < blocks && s.block[b][thread] >= threshold);
            for (; hits; hits &= hits - 1) {
                const int k = atomicAdd(&s.items, 1);
                if (k < kItems) s.item[k] = __builtin_ctz(hits) * kThreads + thread;
            }
        }
    }
}

// The K likeliest of a row, of what was collected (kTop = 2: after the blocks'
// logits were read again, by the whole workgroup), ranked by counting.  Where
// too much reaches the bound, or a NaN may have hidden a thread's largest, they
// are looked for one by one, the row read again for each.
template <class Z, int kThreads, int kTop, int R>
__device__ __forceinline__ void top_of(const Logprob &a, int64_t row, int end, int count, int rounds,
                                       TopPlace<kThreads, kTop> &s) {
    constexpr int N = Z::kGroup, kSteps = R / N, kFound = TopPlace<kThreads, kTop>::kFound, kWaves = kThreads / 64;
    constexpr int kItems = TopPlace<kThreads, kTop>::kItems;
    const int thread = static_cast<int>(threadIdx.x), lane = thread & 63;
    const float M = s.M, L = s.L;
    const typename Z::type *z = static_cast<const typename Z::type *>(a.z) + row * a.ld;
    float *top_logp = a.top_logp ? a.top_logp + row * a.top : nullptr;
    int32_t *top_index = a.top_index + row * a.top;
    const auto tell = [&](int rank, uint64_t key) {
        const int at = static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
        const uint32_t o = static_cast<uint32_t>(key >> 32);
        top_index[rank] = at;
        if (top_logp) top_logp[rank] = a.scale * (float_of(o) - M) - L;
    };
    const auto nothing = [&](int rank) {
        top_index[rank] = -1;
        if (top_logp) top_logp[rank] = -kInf;
    };
    if (s.plain) {
        bool whole = true;
        if constexpr (kTop == 2) {
            const int items = s.items;
            whole = items <= kItems;
            if (whole) {
                const float threshold = s.threshold;
                const int each = kSteps * rounds;            // groups of a block
                for (int p = thread; p < items * each; p += kThreads) {
                    const int k = p / each, item = s.item[k], b = item / kThreads, t = item - b * kThreads, g = p - k * each;
                    const int i = b * rounds + g / kSteps, round = kThreads == 1024 ? (t >> 8) * count + i : i;
                    const int at = place_of<Z, kThreads, R>(round, g % kSteps, t >> 6 & 3, t & 63);
                    const int n = i < count ? end - at : 0;
                    if (n <= 0) continue;
                    float x[N];
                    open<Z, N>(get_group<Z, N>(z + at, n), x);
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        if (i < n && x[i] >= threshold) {
                            const int k = atomicAdd(&s.n, 1);
                            if (k < kFound) s.found[k] = key_of(x[i], at + i);
                        }
                }
                __syncthreads();
            }
        }
        const int n = s.n;
        if (whole && n <= kFound) {
            if (kWaves > 1 && n <= 64) {          // (nearly always)
                const uint64_t key = lane < n ? s.found[lane] : 0;
                int rank = a.top;
                const uint32_t hi = static_cast<uint32_t>(key >> 32), lo = static_cast<uint32_t>(key);
                for (int k = __builtin_amdgcn_readfirstlane(thread >> 6); k < n; k += kWaves) {
                    const uint64_t other = uint64_t(static_cast<uint32_t>(__builtin_amdgcn_readlane(hi, k))) << 32 |
                                           static_cast<uint32_t>(__builtin_amdgcn_readlane(lo, k));
                    const int higher = __builtin_popcountll(__ballot(key > other));
                    if (lane == k) rank = higher;
                }
                if (rank < a.top) tell(rank, key);
            } else {
                for (int k = thread; k < n; k += kThreads) {
                    const uint64_t key = s.found[k];
                    int rank = 0;
#pragma unroll 8
                    for (int j = 0; j < n; ++j) rank += s.found[j] > key;
                    if (rank < a.top) tell(rank, key);
                }
            }
            for (int k = n + thread; k < a.top; k += kThreads) nothing(k);
            return;
        }
    }
    uint64_t before = ~uint64_t(0);
    for (int rank = 0; rank < a.top; ++rank) {
        uint64_t best = 0;
        for (int at = thread * N; at < a.V; at += kThreads * N) {
            float x[N];
            const int n = a.V - at;
            open<Z, N>(get_group<Z, N>(z + at, n), x);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint64_t key = key_of(x[i], at + i);
                if (i < n && x[i] > -kInf && key < before && key > best) best = key;
            }
        }
        best = wave_max(best);
        __syncthreads();
        if ((thread & 63) == 0) s.found[thread >> 6] = best;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kThreads / 64; ++i) best = s.found[i] > best ? s.found[i] : best;
        if (thread == 0) {
            if (best)
                tell(rank, best);
            else
                nothing(rank);
        }
        before = best;
    }
}

// kTop: 0 = no alternatives, 1 = of rows of at most one round a thread, 2 = of any.
// R: logits of a thread in a round.  kQuarters: of rows of four quarters.
template <class Z, int kThreads, int R, bool kQuarters, bool kEntropy, int kTop>
__global__ __launch_bounds__(kThreads, kTop == 0 ? 8 : kTop == 2 && kThreads == 256 ? 6 : 1) void k_logprob(const Logprob a) {
    constexpr int kWaves = kThreads / 64, N = Z::kGroup, kSteps = R / N, kSpan = R * (kThreads == 64 ? 64 : 256);
    constexpr int kEach = kQuarters && kThreads == 256 ? 4 : 1, kSums = kWaves * kEach;
    constexpr bool kOne = kTop == 1 || kThreads == 64;
    __shared__ float red[kWaves], sums[kEntropy ? 2 : 1][kSums];
    __shared__ typename std::conditional<(kTop > 0), TopPlace<kThreads, kTop>, char>::type top;
    __shared__ typename std::conditional<(kTop == 0 && kEach > 1), Quarters<kThreads>, char>::type room;
    const int thread = static_cast<int>(threadIdx.x), lane = thread & 63;
    const int wave = kThreads == 64 ? 0 : __builtin_amdgcn_readfirstlane(thread >> 6);
    auto &quarters = [&]() -> auto & {
        if constexpr (kTop > 0) return top.quarters;
        else return room;
    }();
    const int end = grouped<Z, kThreads>(a.V);
    // rounds of the row, of a quarter, of a thread, of a block; the wave's first one and the one behind its last
    const int all = (end + kSpan - 1) / kSpan, quarter = kQuarters ? (all + 3) / 4 : all;
    const int count = kOne ? 1 : kThreads == 1024 ? quarter : all;
    const int rounds = kTop == 2 ? (count + kBlocks<kThreads> - 1) / kBlocks<kThreads> : 1;
    const int begin = kThreads == 1024 ? (wave >> 2) * quarter : 0;
    const int behind_last = kOne ? begin + 1 : min(begin + count, (end - (wave & 3) * (64 * R) + kSpan - 1) / kSpan);
    for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
        const typename Z::type *z = static_cast<const typename Z::type *>(a.z) + row * a.ld;
        const int target = a.target ? a.target[row] : -1;
        const bool odd = Z::kType == SFT_BF16 && kThreads > 64 && (reinterpret_cast<uintptr_t>(z) & 2);
        float behind[2] = {-kInf, -kInf};
        if (end + thread < a.V) behind[0] = logit<Z>(z, end + thread);
        Running r{-kFar, 0.0f, 0.0f};
        float x[R], m = -kInf, most = -kInf;
        int block = 0, left = rounds, part = 0, round = begin;
        const auto take_round = [&]() {
            Raw<Z, N> raw[kSteps];
            const auto at = [&](int u) { return place_of<Z, kThreads, R>(round, u, wave & 3, lane); };
            if (!kOne && at(kSteps) - lane * N <= end) {
                if (odd) {
#pragma unroll
                    for (int u = 0; u < kSteps; ++u) raw[u] = get_odd<Z, N>(z + at(u));
                } else {
#pragma unroll
                    for (int u = 0; u < kSteps; ++u) raw[u] = get<Z, N, true>(z + at(u));
                }
            } else {
#pragma unroll
                for (int u = 0; u < kSteps; ++u) {
#pragma unroll
                    for (int i = 0; i < words_of<Z, N>; ++i) raw[u].w[i] = Z::kLowest;
                    if (at(u) + N <= end) {
                        if (odd) raw[u] = get_odd<Z, N>(z + at(u));
                        else raw[u] = get<Z, N, true>(z + at(u));
                    }
                }
            }
            if constexpr (kThreads == 64) {       // a group that the row ends in
#pragma unroll
                for (int u = 0; u < kSteps; ++u) {
                    const int n = end - at(u);
                    if (n > 0 && n < N) raw[u] = get_group<Z, N>(z + at(u), n);
                }
            }
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                open<Z, N>(raw[u], x + u * N);
                if constexpr (kThreads == 64) {
                    const int n = end - at(u);
                    if (n > 0 && n < N) {
#pragma unroll
                        for (int i = 0; i < N; ++i) x[u * N + i] = i < n ? x[u * N + i] : -kInf;
                    }
                }
            }
            const float own = take_up<kEntropy>(r, x, a.c, !kOne && round != (kEach > 1 ? part * quarter : begin));
            m = __builtin_fmaxf(m, own);
            if constexpr (kTop == 2) {
                most = __builtin_fmaxf(most, own);
                if (--left == 0) {
                    top.block[block][thread] = most;
                    ++block;
                    left = rounds;
                    most = -kInf;
                }
            }
        };
        if constexpr (kOne) {
            take_round();
        } else {
#pragma unroll 1
            for (; part < kEach; ++part) {
                const int stop = kEach > 1 ? min(behind_last, (part + 1) * quarter) : behind_last;
#pragma unroll 1
                for (; round < stop; ++round) take_round();
                if constexpr (kEach > 1) {
                    quarters.put(part, r);
                    r = Running{-kFar, 0.0f, 0.0f};
                }
            }
        }
        if constexpr (kTop == 2)
            if (left < rounds) top.block[block][thread] = most;
        const bool given = target >= 0 && target < a.V;
        const float at_target = given ? logit<Z>(z, target) : 0.0f;
        if constexpr (kEach > 1) r = quarters.get(0);
        if (end < a.V) m = __builtin_fmaxf(m, take_up<kEntropy>(r, behind, a.c, true));
        if constexpr (kTop > 0) {
            top.mine[thread] = m;
            if (thread == 0) top.items = top.n = 0;
            if (kThreads == 64) __syncthreads();
        }
        float M = block_of<Max, kThreads>(m, red);
        if constexpr (kTop > 0) {       // meanwhile one wave looks for the bound
            if (kThreads == 64 || wave == 1) {
                const float bound = bound_of<kThreads>(top.mine, a.top);
                if (lane == 0) top.threshold = __builtin_fmaxf(bound, -kLargest);      // (not minus infinity)
            }
        }
        const float m2 = __builtin_fmaxf(M * a.c, -kFar);
        // what m2 is off M * c by
        float off = __builtin_fmaf(M, a.c, -m2);
        const bool finite = __builtin_fabsf(M) < kInf, far = finite && !(__builtin_fabsf(M * a.c) < kFar);
        if (far) off = 0.0f;
        float own[(kEntropy ? 2 : 1) * kEach];      // of each quarter: the sums, then the others
#pragma unroll
        for (int q = 0; q < kEach; ++q) {
            float sum = 0.0f, along = 0.0f;
            if (far) {
#pragma unroll 1
                for (int i = q * kThreads + thread; i < a.V; i += kEach * kThreads) {
                    const float d = (logit<Z>(z, i) - M) * a.c, e = exp2_of(d);
                    sum += e;
                    along = __builtin_fmaf(e, __builtin_fmaxf(d, kNothing), along);
                }
            } else {
                if constexpr (kEach > 1)
                    if (q) r = quarters.get(q);
                const float less = limit(r.m2 - m2, kNothing, 0.0f), part = exp2_of(less);
                along = part * __builtin_fmaf(r.sum, less, r.along);
                sum = r.sum * part;
            }
            own[q] = sum;
            if constexpr (kEntropy) own[kEach + q] = along;
        }
        float sum = 0.0f, along = 0.0f;
        if constexpr (kThreads == 64) {
            sum = lanes_of<Sum, 64>(own[0]);
            if constexpr (kEntropy) along = lanes_of<Sum, 64>(own[1]);
        } else {
            constexpr int kGap = 16 / ((kEntropy ? 2 : 1) * kEach);
            const float s = sums_of(own);
            if (lane < 16 && lane % kGap == 0) sums[lane / kGap / kEach][lane / kGap % kEach * kWaves + wave] = s;
        }
        __syncthreads();
        if (thread < 64) {        // one wave finishes the row
            if constexpr (kThreads > 64) {
                sum = sums[0][0];
                if (kEntropy) along = sums[kEntropy][0];
#pragma unroll
                for (int i = 1; i < kSums; ++i) {
                    sum += sums[0][i];
                    if (kEntropy) along += sums[kEntropy][i];
                }
            }
            const bool none = M == -kInf && sum == 0.0f;      // a row without an allowed token
            float L = logf(sum), entropy = 0.0f;
            // neither is below 0, whatever the roundings
            if (kEntropy) entropy = __builtin_fmaxf(L - kLn2 * (along / sum), 0.0f);
            L = __builtin_fmaxf(L - kLn2 * off, 0.0f);
            if (!finite || sum != sum) {
                const float nan = __builtin_nanf("");
                M = none ? -kInf : nan;
                L = none ? -kInf : nan;
                entropy = none ? 0.0f : nan;
            }
            if (thread == 0) {
                if (a.logp) a.logp[row] = !given ? 0.0f : none ? -kInf : a.scale * (at_target - M) - L;
                if (a.stats) {
                    a.stats[2 * row] = M;
                    a.stats[2 * row + 1] = L;
                }
                if (kEntropy) a.entropy[row] = entropy;
            }
            if constexpr (kTop > 0)
                if (thread == 0) {
                    top.M = M, top.L = L;
                    top.plain = sum == sum;
                }
        }
        if constexpr (kTop > 0) {
            collect<Z, kThreads, kTop, R>(x, behind[0], m, end, behind_last - begin, rounds, top);
            __syncthreads();
            top_of<Z, kThreads, kTop, R>(a, row, end, count, rounds, top);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ gradient
struct LogprobGrad {
    const void *z;
    const int32_t *target;
    const float *stats, *entropy, *dlogp, *dentropy;
    void *dz;
    int64_t ld, ldd;
    int64_t pieces;                // of all rows
    int32_t N, V, per_row;         // pieces of a row
    float scale, c;
};

constexpr int kGradThreads = 256;

// A piece is kGradGroups groups of each of kLanes threads; short rows (kLanes =
// 64) are a piece each, without a head of their own.
template <class Z, class D, bool kEntropy, int kLanes, int kGradGroups>
__global__ __launch_bounds__(kGradThreads) void k_logprob_grad(const LogprobGrad a) {
    constexpr float kLog2e = 1.44269504088896340736f;
    constexpr int N = Z::kGroup, kPiece = kLanes * kGradGroups * N, kTeams = kGradThreads / kLanes;
    const int lane = static_cast<int>(threadIdx.x) % kLanes, team = static_cast<int>(threadIdx.x) / kLanes;
    for (int64_t p = int64_t(blockIdx.x) * kTeams + team; p < a.pieces; p += int64_t(gridDim.x) * kTeams) {
        const int64_t row = kLanes == 64 ? p : a.pieces >> 31 ? p / a.per_row : uint32_t(p) / uint32_t(a.per_row);
        const int piece = static_cast<int>(p - row * a.per_row);
        const typename Z::type *z = static_cast<const typename Z::type *>(a.z) + row * a.ld;
        typename D::type *dz = static_cast<typename D::type *>(a.dz) + row * a.ldd;
        // pieces start on whole cache lines of Z; the logits before go to the first one's first threads
        const int head = kLanes == 64 ? 0 : before_line<Z>(z, a.V), begin = head + piece * kPiece;
        const bool mine = piece == 0 && lane < head;
        const int target = a.target ? a.target[row] : -1;
        const bool given = target >= 0 && target < a.V;
        const float own = given && a.dlogp ? a.dlogp[row] : 0.0f;
        const float by_entropy = kEntropy ? a.dentropy[row] : 0.0f;
        const float M = a.stats[2 * row], L = a.stats[2 * row + 1];
        if ((own == 0.0f && by_entropy == 0.0f) || (M == -kInf && L == -kInf)) {
#pragma unroll
            for (int g = 0; g < kGradGroups; ++g) {
                const int at = begin + (g * kLanes + lane) * N;
                put_group<D, N, true>(dz + at, raw_zero<D, N>(), a.V - at);
            }
            if (mine) dz[lane] = D::down(0.0f);
            continue;
        }
        Raw<Z, N> raw[kGradGroups];
#pragma unroll
        for (int g = 0; g < kGradGroups; ++g) {
            const int at = begin + (g * kLanes + lane) * N, n = a.V - at;
            raw[g] = n >= N ? get<Z, N, true>(z + at) : get_group<Z, N>(z + at, n);
        }
        const float first = mine ? logit<Z>(z, lane) : 0.0f;
        // scale * (dlogp + dentropy * (logp + entropy)) as a line in log2(p)
        const float l2 = L * kLog2e, slope = a.scale * by_entropy * kLn2;
        const float level = a.scale * (own + (kEntropy ? by_entropy * a.entropy[row] : 0.0f));
        const float extra = a.scale * own;
        const auto slope_of = [&](float x) {
            const float d = __builtin_fmaf(x - M, a.c, -l2);
            const float weight = kEntropy ? __builtin_fmaf(__builtin_fmaxf(d, kNothing), slope, level) : level;
            return -exp2_of(d) * weight;
        };
#pragma unroll
        for (int g = 0; g < kGradGroups; ++g) {
            const int at = begin + (g * kLanes + lane) * N;
            float x[N];
            open<Z, N>(raw[g], x);
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = slope_of(x[i]);
            if (given && static_cast<uint32_t>(target - at) < uint32_t(N)) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (i == target - at) x[i] += extra;
            }
            put_group<D, N, true>(dz + at, close<D, N>(x), a.V - at);
        }
        if (mine) dz[lane] = D::down(slope_of(first) + (target == lane ? extra : 0.0f));
    }
}

// ------------------------------------------------------------------ host
int check(int64_t N, int64_t V, int64_t ld, const void *Z, int32_t type, float scale, const int32_t *target,
          const char *who, Block *z) {
    SFT_CHECK(N >= 0 && V >= 0, SFT_EINVAL, "%s: negative size", who);
    SFT_CHECK(V > 0, SFT_ESHAPE, "%s: V = 0", who);
    SFT_CHECK(V < (int64_t(1) << 30), SFT_ENOTSUP, "%s: V >= 2^30", who);
    SFT_CHECK(N < (int64_t(1) << 31), SFT_ENOTSUP, "%s: N >= 2^31", who);
    SFT_CHECK(ld >= V, SFT_ESHAPE, "%s: rows of Z are closer than V", who);
    SFT_CHECK(ld < (int64_t(1) << 40), SFT_ENOTSUP, "%s: rows of Z are 2^40 elements apart or more", who);
    SFT_CHECK(type == SFT_F32 || type == SFT_BF16, SFT_EINVAL, "%s: bad type %d", who, type);
    SFT_CHECK(scale > 0.0f && std::isfinite(scale), SFT_EINVAL, "%s: scale is not positive and finite", who);
    SFT_CHECK(Z || N == 0, SFT_EINVAL, "%s: Z is null", who);
    SFT_CHECK(aligned_to(Z, type_bytes(type)), SFT_EALIGN, "%s: Z not aligned to its type", who);
    SFT_CHECK(aligned_to(target, 4), SFT_EALIGN, "%s: target not 4-byte aligned", who);
    *z = rows_block(Z, N, ld, V, type_bytes(type));
    SFT_CHECK(extent(*z) >= 0, SFT_ENOTSUP, "%s: Z spans 2^46 bytes or more", who);
    return SFT_OK;
}

constexpr int64_t kMaxGrid = 1 << 21;

float scaled(float scale) { return static_cast<float>(double(scale) * 1.4426950408889634074); }

template <class Z, int kThreads, int R, bool kQuarters, int kTop>
void send(const Logprob &a, int64_t most, hipStream_t st) {
    const dim3 grid(static_cast<uint32_t>(std::min<int64_t>(a.N, most))), block(kThreads);
    if (a.entropy) hipLaunchKernelGGL((k_logprob<Z, kThreads, R, kQuarters, true, kTop>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_logprob<Z, kThreads, R, kQuarters, false, kTop>), grid, block, 0, st, a);
}

// Short rows go to a wave each, as many at a time as the device holds: starting
// a workgroup takes longer than reading one of them.  Long rows go to 1024
// threads where there is at most one for each CU (250 x 50001 in bf16, with 20
// alternatives: 10.8 us, by 256 threads 14.4), else to 256 (272 of them: 15.8, by
// 1024 threads 19.0), and beyond 16384 logits (16 x 20000 in fp32, with 5: 6.9
// and 8.8; when tried below, 16 x 16384 in bf16: 6.4 and 6.3, 16 x 5000 in fp32:
// 6.6 and 5.9).
template <class Z>
void send(const Logprob &a, hipStream_t st) {
    const int64_t waves = 32 * int64_t(num_cus());
    if (a.V <= 64 * 8) {
        if (a.top) send<Z, 64, 8, false, 1>(a, waves, st);
        else send<Z, 64, 8, false, 0>(a, waves, st);
    } else if (a.V <= 64 * kRound) {
        if (a.top) send<Z, 64, kRound, false, 2>(a, waves, st);
        else send<Z, 64, kRound, false, 0>(a, waves, st);
    } else if (a.V <= kLong) {
        if (a.top) send<Z, 256, kRound, false, 2>(a, kMaxGrid, st);
        else send<Z, 256, kRound, false, 0>(a, kMaxGrid, st);
    } else if (a.N <= num_cus()) {
        if (!a.top) send<Z, 1024, kRound, true, 0>(a, kMaxGrid, st);
        else if (a.V <= 1024 * kRound) send<Z, 1024, kRound, true, 1>(a, kMaxGrid, st);
        else send<Z, 1024, kRound, true, 2>(a, kMaxGrid, st);
    } else {
        if (a.top) send<Z, 256, kRound, true, 2>(a, kMaxGrid, st);
        else send<Z, 256, kRound, true, 0>(a, kMaxGrid, st);
    }
}

template <class Z, class D, int kLanes, int kGroups>
void send_grad(LogprobGrad a, int64_t most, hipStream_t st) {
    constexpr int kTeams = kGradThreads / kLanes, kPiece = kLanes * kGroups * Z::kGroup;
    a.per_row = (a.V + kPiece - 1) / kPiece;
    a.pieces = int64_t(a.N) * a.per_row;
    const dim3 grid(static_cast<uint32_t>(std::min((a.pieces + kTeams - 1) / kTeams, most))), block(kGradThreads);
    if (a.dentropy) hipLaunchKernelGGL((k_logprob_grad<Z, D, true, kLanes, kGroups>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_logprob_grad<Z, D, false, kLanes, kGroups>), grid, block, 0, st, a);
}

// Pieces of four groups a thread for either type (bf16: 4096 x 32000 85 us, two groups 90; fp32: 1000 x 32000 42.9 us,
// eight groups 45.3), and as above for short rows.
template <class Z, class D>
void send_grad(const LogprobGrad &a, hipStream_t st) {
    const int64_t held = 8 * int64_t(num_cus());
    if (a.V <= 64 * 8) send_grad<Z, D, 64, 8 / Z::kGroup>(a, held, st);
    else if (a.V <= 64 * kRound) send_grad<Z, D, 64, kRound / Z::kGroup>(a, held, st);
    else send_grad<Z, D, kGradThreads, 4>(a, 4 * kMaxGrid, st);
}

}  // namespace

extern "C" {

int sft_logprob(const sft_logprob_args *v, void *stream) {
    const char *const who = "sft_logprob";
    clear_error();
    SFT_CHECK(v, SFT_EINVAL, "%s: args is null", who);
    Block z;
    if (int rc = check(v->N, v->V, v->ldz, v->Z, v->z_type, v->scale, v->target, who, &z)) return rc;
    SFT_CHECK(std::isfinite(scaled(v->scale)), SFT_EINVAL, "%s: scale is too large", who);
    SFT_CHECK(v->top_k >= 0 && v->top_k <= kMaxTop, SFT_EINVAL, "%s: top_k outside [0, %d]", who, kMaxTop);
    SFT_CHECK(v->N == 0 || !v->target == !v->logp, SFT_EINVAL, "%s: one of target and logp is null", who);
    SFT_CHECK(v->N == 0 || v->top_index || !v->top_k, SFT_EINVAL, "%s: top_index is null", who);
    SFT_CHECK(aligned_to(v->logp, 4) && aligned_to(v->stats, 4) && aligned_to(v->entropy, 4) &&
                  aligned_to(v->top_logp, 4) && aligned_to(v->top_index, 4),
              SFT_EALIGN, "%s: an output not 4-byte aligned", who);
    const int64_t tops = v->N * v->top_k * 4;
    const Block written[] = {flat_block(v->logp, v->N * 4), flat_block(v->stats, v->N * 8),
                             flat_block(v->entropy, v->N * 4), flat_block(v->top_logp, tops),
                             flat_block(v->top_index, tops)};
    const Block target = flat_block(v->target, v->N * 4);
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < i; ++j)
            SFT_CHECK(apart(written[i], written[j]), SFT_EINVAL, "%s: two outputs overlap", who);
        SFT_CHECK(apart(written[i], z) && apart(written[i], target), SFT_EINVAL, "%s: an output overlaps an input", who);
    }
    if (v->N == 0) return SFT_OK;
    Logprob a{};
    a.z = v->Z, a.target = v->target, a.logp = v->logp, a.stats = v->stats, a.entropy = v->entropy;
    a.top_logp = v->top_logp, a.top_index = v->top_index;
    a.ld = v->ldz;
    a.N = static_cast<int32_t>(v->N), a.V = static_cast<int32_t>(v->V), a.top = v->top_k;
    a.scale = v->scale, a.c = scaled(v->scale);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (v->z_type == SFT_BF16) send<Bf16>(a, st);
    else send<Fp32>(a, st);
    const hipError_t e = hipGetLastError();
    SFT_CHECK(e == hipSuccess, SFT_EHIP, "%s: launch failed: %s", who, hipGetErrorString(e));
    return SFT_OK;
}

int sft_logprob_grad(const sft_logprob_grad_args *v, void *stream) {
    const char *const who = "sft_logprob_grad";
    clear_error();
    SFT_CHECK(v, SFT_EINVAL, "%s: args is null", who);
    Block z;
    if (int rc = check(v->N, v->V, v->ldz, v->Z, v->z_type, v->scale, v->target, who, &z)) return rc;
    SFT_CHECK(std::isfinite(scaled(v->scale)), SFT_EINVAL, "%s: scale is too large", who);
    SFT_CHECK(v->dz_type == v->z_type || v->dz_type == SFT_BF16, SFT_EINVAL, "%s: bad type of dZ", who);
    SFT_CHECK(v->lddz >= v->V, SFT_ESHAPE, "%s: rows of dZ are closer than V", who);
    SFT_CHECK(v->lddz < (int64_t(1) << 40), SFT_ENOTSUP, "%s: rows of dZ are 2^40 elements apart or more", who);
    SFT_CHECK(v->N == 0 || (v->dZ && v->stats), SFT_EINVAL, "%s: dZ or stats is null", who);
    SFT_CHECK(v->N == 0 || !v->target == !v->dlogp, SFT_EINVAL, "%s: one of target and dlogp is null", who);
    SFT_CHECK(v->N == 0 || !v->entropy == !v->dentropy, SFT_EINVAL, "%s: one of entropy and dentropy is null", who);
    SFT_CHECK(aligned_to(v->dZ, type_bytes(v->dz_type)) && aligned_to(v->stats, 4) && aligned_to(v->entropy, 4) &&
                  aligned_to(v->dlogp, 4) && aligned_to(v->dentropy, 4),
              SFT_EALIGN, "%s: an array not aligned to its type", who);
    const Block dz = rows_block(v->dZ, v->N, v->lddz, v->V, type_bytes(v->dz_type));
    SFT_CHECK(extent(dz) >= 0, SFT_ENOTSUP, "%s: dZ spans 2^46 bytes or more", who);
    SFT_CHECK(same(dz, z) || apart(dz, z), SFT_EINVAL, "%s: dZ overlaps Z", who);
    for (const Block &b : {flat_block(v->target, v->N * 4), flat_block(v->stats, v->N * 8),
                           flat_block(v->entropy, v->N * 4), flat_block(v->dlogp, v->N * 4),
                           flat_block(v->dentropy, v->N * 4)})
        SFT_CHECK(apart(dz, b), SFT_EINVAL, "%s: dZ overlaps an input", who);
    if (v->N == 0) return SFT_OK;
    LogprobGrad a{};
    a.z = v->Z, a.target = v->target, a.stats = v->stats, a.entropy = v->entropy;
    a.dlogp = v->dlogp, a.dentropy = v->dentropy, a.dz = v->dZ;
    a.ld = v->ldz, a.ldd = v->lddz;
    a.N = static_cast<int32_t>(v->N), a.V = static_cast<int32_t>(v->V);
    a.scale = v->scale, a.c = scaled(v->scale);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (v->z_type == SFT_BF16) send_grad<Bf16, Bf16>(a, st);
    else if (v->dz_type == SFT_BF16) send_grad<Fp32, Bf16>(a, st);
    else send_grad<Fp32, Fp32>(a, st);
    const hipError_t e = hipGetLastError();
    SFT_CHECK(e == hipSuccess, SFT_EHIP, "%s: launch failed: %s", who, hipGetErrorString(e));
    return SFT_OK;
}

int sft_probe_logprob_bound(const float *values, int32_t n, int32_t want, float *bound) {
    const char *const who = "sft_probe_logprob_bound";
    clear_error();
    SFT_CHECK(values && bound, SFT_EINVAL, "%s: null pointer", who);
    SFT_CHECK(n >= 1 && n <= 128 && want >= 1 && want <= n, SFT_EINVAL, "%s: n outside [1, 128] or want outside [1, n]", who);
    uint32_t order[128], differ = 0;
    for (int32_t i = 0; i < n; ++i) {
        SFT_CHECK(values[i] == values[i], SFT_EINVAL, "%s: a value is NaN", who);
        order[i] = order_of(values[i]);
        differ |= order[i] ^ order[0];
    }
    *bound = float_of(differ == 0 ? order[0] : bound_bits(order[0], differ, want, n, [&](uint32_t b) {
        return static_cast<uint32_t>(std::count_if(order, order + n, [&](uint32_t o) { return o >= b; }));
    }));
    return SFT_OK;
}

}  // extern "C"
