// sft_vec.h -- groups of neighbouring elements between memory and registers,
// from any element's address, and sums and maxima over the lanes that share a
// row.  Shared by the row-wise kernels; not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "sft_internal.h"

namespace sft {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__host__ __device__ __forceinline__ float bits_float(uint32_t x) { return __builtin_bit_cast(float, x); }
__host__ __device__ __forceinline__ uint32_t float_bits(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ uint32_t bf16_bits(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));     // to nearest even
}

// The two storage types.  Groups are of 16 bytes where both sides have the
// same type (kGroup elements): a wave's loads and stores then are whole runs of
// a kilobyte.  They go to any element's address: memory takes accesses of that
// width from all of them, so rows of odd width or distance go the same way.
struct Fp32 {
    typedef float type;
    static constexpr int kGroup = 4;
    static constexpr int32_t kType = SFT_F32;
    static constexpr uint32_t kLowest = 0xff800000u;      // a word of minus infinity
    typedef u32x4 __attribute__((aligned(4))) quad;
    typedef u32x2 __attribute__((aligned(4))) twin;
    typedef uint32_t word;
    static __device__ __forceinline__ float up(float x) { return x; }
    static __device__ __forceinline__ float down(float x) { return x; }
    static __device__ __forceinline__ uint32_t bits(float x) { return float_bits(x); }
    static __device__ __forceinline__ float of_bits(uint32_t x) { return bits_float(x); }
};
struct Bf16 {
    typedef uint16_t type;
    static constexpr int kGroup = 8;
    static constexpr int32_t kType = SFT_BF16;
    static constexpr uint32_t kLowest = 0xff80ff80u;
    typedef u32x4 __attribute__((aligned(2))) quad;
    typedef u32x2 __attribute__((aligned(2))) twin;
    typedef uint32_t __attribute__((aligned(2))) word;
    static __device__ __forceinline__ float up(uint16_t x) { return bits_float(uint32_t(x) << 16); }
    static __device__ __forceinline__ uint16_t down(float x) { return static_cast<uint16_t>(bf16_bits(x)); }
    static __device__ __forceinline__ uint32_t bits(uint16_t x) { return x; }
    static __device__ __forceinline__ uint16_t of_bits(uint32_t x) { return static_cast<uint16_t>(x); }
};

// N elements (4 or 8) as they are in memory.
template <class E, int N>
constexpr int words_of = N * int(sizeof(typename E::type)) / 4;
template <class E, int N>
struct Raw {
    uint32_t w[words_of<E, N>];
};

template <class E, int N>
__device__ __forceinline__ Raw<E, N> raw_zero() {
    Raw<E, N> r;
#pragma unroll
    for (int i = 0; i < words_of<E, N>; ++i) r.w[i] = 0;
    return r;
}

// kPast: what is read once and lies on whole cache lines need not stay in L2.
template <class E, int N, bool kPast = false>
__device__ __forceinline__ Raw<E, N> get(const typename E::type *p) {
    Raw<E, N> r;
    if constexpr (words_of<E, N> == 2) {
        const u32x2 a = *reinterpret_cast<const typename E::twin *>(p);
        r.w[0] = a.x, r.w[1] = a.y;
    } else {
        const typename E::quad *q = reinterpret_cast<const typename E::quad *>(p);
#pragma unroll
        for (int i = 0; i < words_of<E, N> / 4; ++i) {
            const u32x4 a = kPast ? __builtin_nontemporal_load(q + i) : q[i];
            r.w[4 * i] = a.x, r.w[4 * i + 1] = a.y, r.w[4 * i + 2] = a.z, r.w[4 * i + 3] = a.w;
        }
    }
    return r;
}

// The first n < N of them, in pieces of half a group, a quarter and so on: n in
// binary.  Few holds the pieces as loaded, so that waiting for them can wait;
// whole() puts them together, zeros behind.
template <class E, int N>
struct Few {
    static constexpr int kWords = words_of<E, N> > N / 2 ? N - 1 : N / 2;      // a lone bf16 takes a word
    uint32_t w[kWords];
};

template <class E, int N>
__device__ __forceinline__ Few<E, N> few_zero() {
    Few<E, N> f;
#pragma unroll
    for (int i = 0; i < Few<E, N>::kWords; ++i) f.w[i] = 0;
    return f;
}

template <class E, int N>
__device__ __forceinline__ void get_few(const typename E::type *p, int n, Few<E, N> &f) {
    int k = 0;
#pragma unroll
    for (int half = N / 2; half; half /= 2) {
        const int words = half * int(sizeof(typename E::type)) / 4;
        if (n & half) {
            if (words == 4) {
                const u32x4 a = *reinterpret_cast<const typename E::quad *>(p);
                f.w[k] = a.x, f.w[k + 1] = a.y, f.w[k + 2] = a.z, f.w[k + 3] = a.w;
            } else if (words == 2) {
                const u32x2 a = *reinterpret_cast<const typename E::twin *>(p);
                f.w[k] = a.x, f.w[k + 1] = a.y;
            } else if (words == 1) {
                f.w[k] = *reinterpret_cast<const typename E::word *>(p);
            } else {
                f.w[k] = E::bits(*p);
            }
            p += half;
        }
        k += words ? words : 1;
    }
}

template <class E, int N>
__device__ __forceinline__ Raw<E, N> whole(const Few<E, N> &f, int n) {
    // the pieces from the last one on, each before what is there already
    constexpr int size = sizeof(typename E::type), W = words_of<E, N>;
    Raw<E, N> r = raw_zero<E, N>();
    int k = Few<E, N>::kWords;
#pragma unroll
    for (int half = 1; half < N; half *= 2) {
        const int words = half * size / 4;
        k -= words ? words : 1;
        if (n & half) {
            if (words == 0) {
                r.w[0] = f.w[k];
            } else {
#pragma unroll
                for (int i = W - 1; i >= 0; --i) r.w[i] = i >= words ? r.w[i - words] : f.w[k + i];
            }
        }
    }
    return r;
}

// n of them (whole from N on, none up to 0).
template <class E, int N, bool kEven = false>
__device__ __forceinline__ Raw<E, N> get_group(const typename E::type *p, int n) {
    if (n >= N) return get<E, N>(p);
    if (n <= 0 || kEven) return raw_zero<E, N>();
    Few<E, N> f = few_zero<E, N>();
    get_few<E, N>(p, n, f);
    return whole<E, N>(f, n);
}

template <class E, int N>
__device__ __forceinline__ void open(const Raw<E, N> &r, float *x) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (words_of<E, N> == N)
            x[i] = bits_float(r.w[i]);
        else
            x[i] = bits_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
    }
}

template <class E, int N>
__device__ __forceinline__ Raw<E, N> close(const float *x) {
    Raw<E, N> r;
#pragma unroll
    for (int i = 0; i < words_of<E, N>; ++i) {
        if constexpr (words_of<E, N> == N)
            r.w[i] = float_bits(x[i]);
        else
            r.w[i] = bf16_bits(x[2 * i]) | bf16_bits(x[2 * i + 1]) << 16;
    }
    return r;
}

// kPast: results that nothing near reads go past L2, which leaves it to what is still to be read.
template <class E, int N, bool kPast = false>
__device__ __forceinline__ void put(typename E::type *p, const Raw<E, N> &r) {
    if constexpr (words_of<E, N> == 2) {
        typename E::twin *q = reinterpret_cast<typename E::twin *>(p);
        const typename E::twin a = u32x2{r.w[0], r.w[1]};
        if constexpr (kPast)
            __builtin_nontemporal_store(a, q);
        else
            *q = a;
    } else {
        typename E::quad *q = reinterpret_cast<typename E::quad *>(p);
#pragma unroll
        for (int i = 0; i < words_of<E, N> / 4; ++i) {
            const typename E::quad a = u32x4{r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]};
            if constexpr (kPast)
                __builtin_nontemporal_store(a, q + i);
            else
                q[i] = a;
        }
    }
}

template <class E, int N>
__device__ __forceinline__ void put_few(typename E::type *p, Raw<E, N> r, int n) {
    constexpr int size = sizeof(typename E::type), W = words_of<E, N>;
#pragma unroll
    for (int half = N / 2; half; half /= 2) {
        const int words = half * size / 4;
        if (!(n & half)) continue;
        if (words == 4)
            *reinterpret_cast<typename E::quad *>(p) = u32x4{r.w[0], r.w[1], r.w[2], r.w[W - 1 < 3 ? W - 1 : 3]};
        else if (words == 2)
            *reinterpret_cast<typename E::twin *>(p) = u32x2{r.w[0], r.w[W - 1 < 1 ? W - 1 : 1]};
        else if (words == 1)
            *reinterpret_cast<typename E::word *>(p) = r.w[0];
        else
            *p = E::of_bits(r.w[0]);
        p += half;
#pragma unroll
        for (int i = 0; i < W; ++i) r.w[i] = i + words < W ? r.w[i + words] : 0;
    }
}

// n of them (whole from N on, none up to 0).
template <class E, int N, bool kPast = false, bool kEven = false>
__device__ __forceinline__ void put_group(typename E::type *p, const Raw<E, N> &r, int n) {
    if (n >= N)
        put<E, N, kPast>(p, r);
    else if (n > 0 && !kEven)
        put_few<E, N>(p, r, n);
}

// Elements of a row of n up to the first one at the start of a cache line.
template <class E>
__device__ __forceinline__ int before_line(const typename E::type *p, int n) {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 127u;
    return min(n, static_cast<int>(((128u - off) & 127u) / sizeof(typename E::type)));
}

// The groups of a row of n elements that lane `lane` of kLanes takes: group g
// starts at (g * kLanes + lane) * N.  The pieces of the one that ends inside wait
// in `few` for join_row, so that nothing here waits for a load; kEven: there is
// none, n is a multiple of N.
template <class E, int N, int kLanes, bool kEven, int kGroups>
__device__ __forceinline__ void get_row(const typename E::type *p, int lane, int n, Raw<E, N> (&r)[kGroups],
                                        Few<E, N> &few) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const int at = (g * kLanes + lane) * N;
        r[g] = raw_zero<E, N>();
        if (at + N <= n) r[g] = get<E, N>(p + at);
    }
    if (kEven) return;
    const int last = n & (N - 1);
    few = few_zero<E, N>();
    if (last && (n / N) % kLanes == lane) get_few<E, N>(p + (n - last), last, few);
}

template <class E, int N, int kLanes, bool kEven, int kGroups>
__device__ __forceinline__ void join_row(int lane, int n, Raw<E, N> (&r)[kGroups], const Few<E, N> &few) {
    const int last = n & (N - 1);
    if (kEven || !last) return;
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
        if (n / N == g * kLanes + lane) r[g] = whole<E, N>(few, last);
}

// ---- over the lanes of a wave
template <int kControl>
__device__ __forceinline__ float dpp(float x) {
    return bits_float(__builtin_amdgcn_update_dpp(0, float_bits(x), kControl, 0xf, 0xf, false));
}

struct Sum {
    static constexpr float kNone = 0.0f;
    static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
struct Max {
    static constexpr float kNone = -__builtin_huge_valf();
    static __device__ __forceinline__ float of(float a, float b) { return __builtin_fmaxf(a, b); }
};

// Over each run of kLanes (8, 16, 32 or 64) neighbouring lanes, the same bits in all of them.
template <class Op, int kLanes>
__device__ __forceinline__ float lanes_of(float x) {
    static_assert(kLanes == 8 || kLanes == 16 || kLanes == 32 || kLanes == 64, "lanes of a run");
    if constexpr (kLanes == 8) {           // neighbours, pairs, and the halves of 8 lanes mirrored
        x = Op::of(x, dpp<0xb1>(x));
        x = Op::of(x, dpp<0x4e>(x));
        x = Op::of(x, dpp<0x141>(x));
    } else {                               // rotations within 16 lanes
        x = Op::of(x, dpp<0x128>(x));
        x = Op::of(x, dpp<0x124>(x));
        x = Op::of(x, dpp<0x122>(x));
        x = Op::of(x, dpp<0x121>(x));
    }
    if constexpr (kLanes >= 32) {          // neighbouring halves exchanged
        const u32x2 s = __builtin_amdgcn_permlane16_swap(float_bits(x), float_bits(x), false, false);
        x = Op::of(bits_float(s.x), bits_float(s.y));
    }
    if constexpr (kLanes >= 64) {
        const u32x2 s = __builtin_amdgcn_permlane32_swap(float_bits(x), float_bits(x), false, false);
        x = Op::of(bits_float(s.x), bits_float(s.y));
    }
    return x;
}

}  // namespace sft
