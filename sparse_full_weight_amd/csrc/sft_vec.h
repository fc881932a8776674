// sft_vec.h -- groups of 8 neighbouring elements between memory and registers,
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

__device__ __forceinline__ float bits_float(uint32_t x) { return __builtin_bit_cast(float, x); }
__device__ __forceinline__ uint32_t float_bits(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ uint32_t bf16_bits(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));     // to nearest even
}

// The two storage types.  16 bytes are loaded at a time whatever the address:
// memory takes accesses of that width from any address of an element, so rows
// of odd width or distance go the same way as aligned ones.
struct Fp32 {
    typedef float type;
    static constexpr int kWords = 8;      // of 8 elements
    static constexpr int32_t kType = SFT_F32;
    typedef u32x4 __attribute__((aligned(4))) quad;
    static __device__ __forceinline__ float up(float x) { return x; }
    static __device__ __forceinline__ float down(float x) { return x; }
    static __device__ __forceinline__ float held(float x) { return x; }
};
struct Bf16 {
    typedef uint16_t type;
    static constexpr int kWords = 4;
    static constexpr int32_t kType = SFT_BF16;
    typedef u32x4 __attribute__((aligned(2))) quad;
    static __device__ __forceinline__ float up(uint16_t x) { return bits_float(uint32_t(x) << 16); }
    static __device__ __forceinline__ uint16_t down(float x) { return static_cast<uint16_t>(bf16_bits(x)); }
    static __device__ __forceinline__ float held(float x) { return bits_float(bf16_bits(x) << 16); }
};

// 8 elements as they are in memory.
template <class E>
struct Raw {
    uint32_t w[E::kWords];
};

template <class E>
__device__ __forceinline__ Raw<E> raw_zero() {
    Raw<E> r;
#pragma unroll
    for (int i = 0; i < E::kWords; ++i) r.w[i] = 0;
    return r;
}

template <class E>
__device__ __forceinline__ Raw<E> get8(const typename E::type *p) {
    Raw<E> r;
    const typename E::quad *q = reinterpret_cast<const typename E::quad *>(p);
#pragma unroll
    for (int i = 0; i < E::kWords / 4; ++i) {
        const u32x4 a = q[i];
        r.w[4 * i] = a.x, r.w[4 * i + 1] = a.y, r.w[4 * i + 2] = a.z, r.w[4 * i + 3] = a.w;
    }
    return r;
}

// The first n < 8 of them, zeros behind.
template <class E>
__device__ __forceinline__ Raw<E> get_few(const typename E::type *p, int n) {
    Raw<E> r = raw_zero<E>();
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        if (i >= n) continue;
        if constexpr (E::kWords == 8)
            r.w[i] = float_bits(p[i]);
        else
            r.w[i / 2] |= uint32_t(p[i]) << (16 * (i & 1));
    }
    return r;
}

template <class E>
__device__ __forceinline__ void open8(const Raw<E> &r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (E::kWords == 8)
            x[i] = bits_float(r.w[i]);
        else
            x[i] = bits_float(i & 1 ? r.w[i / 2] & 0xffff0000u : r.w[i / 2] << 16);
    }
}

template <class E>
__device__ __forceinline__ Raw<E> close8(const float (&x)[8]) {
    Raw<E> r;
#pragma unroll
    for (int i = 0; i < E::kWords; ++i) {
        if constexpr (E::kWords == 8)
            r.w[i] = float_bits(x[i]);
        else
            r.w[i] = bf16_bits(x[2 * i]) | bf16_bits(x[2 * i + 1]) << 16;
    }
    return r;
}

template <class E>
__device__ __forceinline__ void put8(typename E::type *p, const Raw<E> &r) {
    typename E::quad *q = reinterpret_cast<typename E::quad *>(p);
#pragma unroll
    for (int i = 0; i < E::kWords / 4; ++i)
        q[i] = u32x4{r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]};
}

template <class E>
__device__ __forceinline__ void put_few(typename E::type *p, const Raw<E> &r, int n) {
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        if (i >= n) continue;
        if constexpr (E::kWords == 8)
            p[i] = bits_float(r.w[i]);
        else
            p[i] = static_cast<uint16_t>(r.w[i / 2] >> (16 * (i & 1)));
    }
}

// A group of n elements (up to 8, whole above).
template <class E>
__device__ __forceinline__ void put_group(typename E::type *p, const Raw<E> &r, int n) {
    if (n >= 8)
        put8<E>(p, r);
    else if (n > 0)
        put_few<E>(p, r, n);
}

// The groups of a row of n elements that lane `lane` of kLanes takes: group g
// starts at (g * kLanes + lane) * 8.  Whole groups first, so that their loads
// are all under way before the one that ends inside is looked at.
template <class E, int kLanes, int kGroups>
__device__ __forceinline__ void get_row(const typename E::type *p, int lane, int n, Raw<E> (&r)[kGroups]) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const int at = (g * kLanes + lane) * 8;
        r[g] = raw_zero<E>();
        if (at + 8 <= n) r[g] = get8<E>(p + at);
    }
    if (n & 7) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int at = (g * kLanes + lane) * 8;
            if (at < n && at + 8 > n) r[g] = get_few<E>(p + at, n - at);
        }
    }
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

// Over each run of kLanes (a power of two from 2 to 64) neighbouring lanes, the same bits in all of them.
template <class Op, int kLanes>
__device__ __forceinline__ float lanes_of(float x) {
    if constexpr (kLanes >= 16) {          // rotations within 16 lanes
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
