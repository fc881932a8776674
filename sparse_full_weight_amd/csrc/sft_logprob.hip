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
// HBM: 4096 x 32000 in bf16 takes 44.6 us (262 MB read, 5.9 TB/s; the vector
// units are busy for 87% of it, as an entropy needs about ten operations a
// logit), its gradient 82 us (5.8 TB/s, rows without one only written); 1003 x
// 50001 in fp32 with 5 alternatives 36.5 us.  Few long rows are bound by their
// CUs instead, about 70 ps a logit in bf16: 8 x 32000 takes 4.5 us, with 20
// alternatives 7.0, of which about 1.2 are passing over the logits that reach
// their bound.  Where the alternatives are looked for one by one, all logits
// equal, 4096 x 32000 with 20 takes about 1 ms, not 54 us.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "sft_blocks.h"
#include "sft_internal.h"
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
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = float_bits(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float float_of(uint32_t order) {
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

// A row's running state in one thread, relative to m2 = m * c.
struct Running {
    float m, m2, sum, along;
};

// Takes up n logits; returns the largest of them.
template <bool kEntropy, int n>
__device__ __forceinline__ float take_up(Running &r, const float (&z)[n], float c) {
    float own = -kInf;
#pragma unroll
    for (int i = 0; i < n; i += 2) own = max3(own, z[i], z[i + 1]);
    const float m = __builtin_fmaxf(own, r.m);
    const float m2 = __builtin_fmaxf(m * c, -kFar);       // (of minus infinity as well)
    const float less = limit(r.m2 - m2, kNothing, 0.0f), part = exp2_of(less);
    r.along = kEntropy ? part * __builtin_fmaf(r.sum, less, r.along) : 0.0f;
    r.sum *= part;
    r.m = m;
    r.m2 = m2;
#pragma unroll
    for (int i = 0; i < n; ++i) {
        const float d = __builtin_fmaf(z[i], c, -m2), e = exp2_of(d);
        r.sum += e;
        if (kEntropy) r.along = __builtin_fmaf(e, __builtin_fmaxf(d, kNothing), r.along);
    }
    return own;
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

// How a row's logits are shared out: those before the first whole cache line
// one each to the first threads, then groups by turns, as many turns at a time
// (a round) as make kRound logits of a thread.
constexpr int kRound = 32;

template <class Z, int kThreads>
__device__ __forceinline__ int place_of(int head, int turn, int thread) {
    return head + (turn * kThreads + thread) * Z::kGroup;
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
    uint64_t found[kFound];
    float mine[kThreads], block[kTop == 2 ? kBlocks<kThreads> : 1][kTop == 2 ? kThreads : 1];
    int32_t item[kItems];
    float threshold, M, L;
    bool plain;
    int items, n;
};

struct Or {
    static __device__ __forceinline__ float of(float a, float b) { return bits_float(float_bits(a) | float_bits(b)); }
};

// A bound that at least `want` and hardly more of a wave's values reach, found by
// halving from the first bit on in which they differ to the last (in bf16 the
// lower half never does), two bits at a time.
template <int kParts>
__device__ __forceinline__ float bound_among(const uint32_t (&o)[kParts], uint32_t want) {
    const uint32_t one = __builtin_amdgcn_readfirstlane(o[0]);
    uint32_t differ = 0;
#pragma unroll
    for (int i = 0; i < kParts; ++i) differ |= o[i] ^ one;
    differ = __builtin_amdgcn_readfirstlane(float_bits(lanes_of<Or, 64>(bits_float(differ))));
    if (differ == 0) return float_of(one);      // (no first bit: the loop's end needs one)
    const uint32_t top = (31u - static_cast<uint32_t>(__builtin_clz(differ))) | 1u, least = differ & (0u - differ);
    const auto reached = [&](uint32_t b) {
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < kParts; ++i) n += static_cast<uint32_t>(__builtin_popcountll(__ballot(o[i] >= b)));
        return n;
    };
    uint32_t bound = one & ~((2u << top) - 1u), bit = 1u << top, reach = 64 * kParts;
    const uint32_t most = min(want + want / 4, reach - 1u);         // (all of them reach the prefix alone)
    do {
        const uint32_t b1 = bound | bit >> 1, b2 = bound | bit, b3 = b1 | b2;
        const uint32_t r1 = reached(b1), r2 = reached(b2), r3 = reached(b3);
        if (r1 >= want) bound = b1, reach = r1;
        if (r2 >= want) bound = b2, reach = r2;
        if (r3 >= want) bound = b3, reach = r3;
        bit >>= 2;
    } while ((bit >= least) & (reach > most));
    return float_of(bound);
}

// A bound that at least K of a row's logits reach (K <= 64), by one wave: about
// the K-th largest of 64, each of them the largest of every 64th thread.  With the
// statistics computed meanwhile, 64 x 50001 in bf16 with 20 alternatives takes
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
__device__ __forceinline__ void collect(const float (&last)[R], float first, float mine, int head, int turns, int rounds,
                                        TopPlace<kThreads, kTop> &s) {
    constexpr int N = Z::kGroup, kSteps = R / N, kFound = TopPlace<kThreads, kTop>::kFound;
    constexpr int kItems = TopPlace<kThreads, kTop>::kItems;
    const int thread = static_cast<int>(threadIdx.x);
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
            if (last[i] >= threshold) s.found[k] = key_of(last[i], place_of<Z, 64>(0, i / N, thread) + i % N);
            n += __builtin_popcountll(which);
        }
        if (thread == 0) s.n = n;
    } else if (mine >= threshold) {
        if (first >= threshold) keep(first, thread);
        if constexpr (kTop == 1) {
            if (turns == 0) return;
#pragma unroll
            for (int g = 0; g < R; g += 8) {
                float most = last[g];
#pragma unroll
                for (int i = 1; i < 8; ++i) most = __builtin_fmaxf(most, last[g + i]);
                if (!(most >= threshold)) continue;
#pragma unroll
                for (int i = g; i < g + 8; ++i)
                    if (last[i] >= threshold) keep(last[i], place_of<Z, kThreads>(head, i / N, thread) + i % N);
            }
        } else {
            uint32_t hits = 0;
            const int blocks = (turns + kSteps * rounds - 1) / (kSteps * rounds);
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
__device__ __forceinline__ void top_of(const Logprob &a, int64_t row, int head, int rounds,
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
                const int each = kSteps * rounds;            // turns of a block
                for (int p = thread; p < items * each; p += kThreads) {
                    const int k = p / each, item = s.item[k], b = item / kThreads;
                    const int at = place_of<Z, kThreads>(head, b * each + p - k * each, item - b * kThreads), n = a.V - at;
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

// kTop: 0 = no alternatives, 1 = of rows of at most one round, 2 = of any.
// R: logits of a thread in a round.
template <class Z, int kThreads, int R, bool kEntropy, int kTop>
__global__ __launch_bounds__(kThreads) void k_logprob(const Logprob a) {
    constexpr int kWaves = kThreads / 64, N = Z::kGroup, kSteps = R / N;
    __shared__ float red[3][kWaves];
    __shared__ typename std::conditional<(kTop > 0), TopPlace<kThreads, kTop>, char>::type top;
    const int thread = static_cast<int>(threadIdx.x);
    for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
        const typename Z::type *z = static_cast<const typename Z::type *>(a.z) + row * a.ld;
        const int target = a.target ? a.target[row] : -1;
        const int head = kThreads > 64 ? before_line<Z>(z, a.V) : 0;     // (a short row's few loads may cross lines)
        const int turns = (a.V - head + kThreads * N - 1) / (kThreads * N);
        const int rounds = kTop == 2 ? (turns + kSteps * kBlocks<kThreads> - 1) / (kSteps * kBlocks<kThreads>) : 1;
        float first[2] = {-kInf, -kInf};
        if (thread < head) first[0] = logit<Z>(z, thread);
        Running r{-kInf, -kFar, 0.0f, 0.0f};
        float x[R], most = -kInf;
        int block = 0, left = rounds;
        const auto round_of = [&](const float (&x)[R]) {
            const float m = take_up<kEntropy>(r, x, a.c);
            if constexpr (kTop == 2) {
                most = __builtin_fmaxf(most, m);
                if (--left == 0) {
                    top.block[block][thread] = most;
                    ++block;
                    left = rounds;
                    most = -kInf;
                }
            }
        };
        Raw<Z, N> raw[kSteps];
        int turn = 0;
        for (; place_of<Z, kThreads>(head, turn + kSteps, 0) <= a.V; turn += kSteps) {
#pragma unroll
            for (int u = 0; u < kSteps; ++u) raw[u] = get<Z, N, true>(z + place_of<Z, kThreads>(head, turn + u, thread));
#pragma unroll
            for (int u = 0; u < kSteps; ++u) open<Z, N>(raw[u], x + u * N);
            round_of(x);
        }
        if (turn < turns) {       // the last round
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                const int at = place_of<Z, kThreads>(head, turn + u, thread);
                raw[u] = raw_zero<Z, N>();
                if (at + N <= a.V) raw[u] = get<Z, N, true>(z + at);
            }
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                const int at = place_of<Z, kThreads>(head, turn + u, thread), n = a.V - at;
                if (n > 0 && n < N) raw[u] = get_group<Z, N>(z + at, n);
            }
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                const int n = a.V - place_of<Z, kThreads>(head, turn + u, thread);
                open<Z, N>(raw[u], x + u * N);
                if (n < N) {
#pragma unroll
                    for (int i = 0; i < N; ++i) x[u * N + i] = i < n ? x[u * N + i] : -kInf;
                }
            }
            round_of(x);
        }
        if constexpr (kTop == 2)
            if (left < rounds) top.block[block][thread] = most;
        const bool given = target >= 0 && target < a.V;
        const float at_target = given ? logit<Z>(z, target) : 0.0f;
        if (head) take_up<kEntropy>(r, first, a.c);
        if constexpr (kTop > 0) {
            top.mine[thread] = r.m;
            if (thread == 0) top.items = top.n = 0;
            if (kThreads == 64) __syncthreads();
        }
        float M = block_of<Max, kThreads>(r.m, red[0]);
        if constexpr (kTop > 0) {       // meanwhile one wave looks for the bound
            if (kThreads == 64 || thread >> 6 == 1) {
                const float bound = bound_of<kThreads>(top.mine, a.top);
                if ((thread & 63) == 0) top.threshold = __builtin_fmaxf(bound, -kLargest);      // (not minus infinity)
            }
        }
        const float m2 = __builtin_fmaxf(M * a.c, -kFar);
        const float less = limit(r.m2 - m2, kNothing, 0.0f), part = exp2_of(less);
        float along = part * __builtin_fmaf(r.sum, less, r.along), sum = r.sum * part;
        // what m2 is off M * c by
        float off = __builtin_fmaf(M, a.c, -m2);
        const bool finite = __builtin_fabsf(M) < kInf;
        if (finite && !(__builtin_fabsf(M * a.c) < kFar)) {
            sum = along = off = 0.0f;
            for (int i = thread; i < a.V; i += kThreads) {
                const float d = (logit<Z>(z, i) - M) * a.c, e = exp2_of(d);
                sum += e;
                along = __builtin_fmaf(e, __builtin_fmaxf(d, kNothing), along);
            }
        }
        sum = lanes_of<Sum, 64>(sum);
        if (kEntropy) along = lanes_of<Sum, 64>(along);
        if (kWaves > 1 && (thread & 63) == 0) {
            red[1][thread >> 6] = sum;
            if (kEntropy) red[2][thread >> 6] = along;
        }
        __syncthreads();
        if (thread < 64) {        // one wave finishes the row
            if constexpr (kWaves > 1) {
                sum = red[1][0];
                if (kEntropy) along = red[2][0];
#pragma unroll
                for (int i = 1; i < kWaves; ++i) {
                    sum += red[1][i];
                    if (kEntropy) along += red[2][i];
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
            collect<Z, kThreads, kTop, R>(x, first[0], r.m, head, turns, rounds, top);
            __syncthreads();
            top_of<Z, kThreads, kTop, R>(a, row, head, rounds, top);
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

template <class Z, int kThreads, int R, int kTop>
void send(const Logprob &a, int64_t most, hipStream_t st) {
    const dim3 grid(static_cast<uint32_t>(std::min<int64_t>(a.N, most))), block(kThreads);
    if (a.entropy) hipLaunchKernelGGL((k_logprob<Z, kThreads, R, true, kTop>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_logprob<Z, kThreads, R, false, kTop>), grid, block, 0, st, a);
}

// Short rows go to a wave each, as many at a time as the device holds: starting
// a workgroup takes longer than reading one of them.  Long rows go to 1024
// threads where there is at most one for each CU (250 x 50001 in bf16, with 20
// alternatives: 11.1 us, by 256 threads 14.0), else to 256 (272 of them: 15.5, by
// 1024 threads 19.8), and from 16384 logits on (16 x 20000 in fp32, with 5: 7.0
// and 8.0; 16 x 16384 in bf16: 6.4 and 6.3; 16 x 5000 in fp32: 6.6 and 5.9).
template <class Z>
void send(const Logprob &a, hipStream_t st) {
    const int64_t waves = 32 * int64_t(num_cus());
    if (a.V <= 64 * 8) {
        if (a.top) send<Z, 64, 8, 1>(a, waves, st);
        else send<Z, 64, 8, 0>(a, waves, st);
    } else if (a.V <= 64 * kRound) {
        if (a.top) send<Z, 64, kRound, 2>(a, waves, st);
        else send<Z, 64, kRound, 0>(a, waves, st);
    } else if (a.N <= num_cus() && a.V >= 16384) {
        if (!a.top) send<Z, 1024, kRound, 0>(a, kMaxGrid, st);
        else if (a.V <= 1024 * kRound) send<Z, 1024, kRound, 1>(a, kMaxGrid, st);
        else send<Z, 1024, kRound, 2>(a, kMaxGrid, st);
    } else {
        if (a.top) send<Z, 256, kRound, 2>(a, kMaxGrid, st);
        else send<Z, 256, kRound, 0>(a, kMaxGrid, st);
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

}  // extern "C"
