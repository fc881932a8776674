// sft_dense.hip -- the optimizer step of what a model trains whole (norm
// gains, biases, routers, small matrices, experts): the global norm of many
// gradients with its clip factor, and AdamW over many tensors in one launch,
// with states in 32 bits or in 8.
//
// Both passes touch every element once and do little arithmetic, so both are
// bound by HBM, and by launch latency where the tensors are small.  A launch
// therefore takes as many tensors as a 4 KB kernel argument describes; a
// workgroup takes one chunk of one tensor and finds it by comparing its index
// with every tensor's first chunk at once, a lane each (one trip to the
// kernel argument instead of a chain of them).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <vector>

#include "sft_internal.h"

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

__device__ __forceinline__ float bf16_up(uint32_t h) { return __builtin_bit_cast(float, h << 16); }
__device__ __forceinline__ uint32_t bf16_rne(float x) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}

// Every array is read and written once in a pass far larger than the caches:
// past L2 (a layer's step in fp32 1138 -> 1100 us, its norm 78.7 -> 73.2).
template <class V>
__device__ __forceinline__ V stream_get(const void *p) {
    return __builtin_nontemporal_load(static_cast<const V *>(p));
}
template <class V>
__device__ __forceinline__ void stream_put(void *p, V v) {
    __builtin_nontemporal_store(v, static_cast<V *>(p));
}

// Element accessors of the two storage types; N consecutive elements from an
// address aligned to the access.
struct F32 {
    typedef float type;
    template <int N>
    static __device__ __forceinline__ void load(const float *p, float (&x)[N]) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const f32x4 a = stream_get<f32x4>(p + i);
            x[i] = a.x, x[i + 1] = a.y, x[i + 2] = a.z, x[i + 3] = a.w;
        }
    }
    template <int N>
    static __device__ __forceinline__ void store(float *p, const float (&x)[N]) {
#pragma unroll
        for (int i = 0; i < N; i += 4) stream_put(p + i, f32x4{x[i], x[i + 1], x[i + 2], x[i + 3]});
    }
    static __device__ __forceinline__ float one(const float *p) { return *p; }
    static __device__ __forceinline__ void put(float *p, float x) { *p = x; }
};

struct BF16 {
    typedef uint16_t type;
    template <int N>
    static __device__ __forceinline__ void load(const uint16_t *p, float (&x)[N]) {
        uint32_t w[N / 2];
        if constexpr (N % 8 == 0) {
#pragma unroll
            for (int i = 0; i < N / 2; i += 4) {
                const u32x4 a = stream_get<u32x4>(p + 2 * i);
                w[i] = a.x, w[i + 1] = a.y, w[i + 2] = a.z, w[i + 3] = a.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; i += 2) {
                const u32x2 a = stream_get<u32x2>(p + 2 * i);
                w[i] = a.x, w[i + 1] = a.y;
            }
        }
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            x[2 * i] = bf16_up(w[i] & 0xffffu);
            x[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
        }
    }
    template <int N>
    static __device__ __forceinline__ void store(uint16_t *p, const float (&x)[N]) {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = bf16_rne(x[2 * i]) | (bf16_rne(x[2 * i + 1]) << 16);
        if constexpr (N % 8 == 0) {
#pragma unroll
            for (int i = 0; i < N / 2; i += 4) stream_put(p + 2 * i, u32x4{w[i], w[i + 1], w[i + 2], w[i + 3]});
        } else {
#pragma unroll
            for (int i = 0; i < N / 2; i += 2) stream_put(p + 2 * i, u32x2{w[i], w[i + 1]});
        }
    }
    static __device__ __forceinline__ float one(const uint16_t *p) { return bf16_up(*p); }
    static __device__ __forceinline__ void put(uint16_t *p, float x) { *p = static_cast<uint16_t>(bf16_rne(x)); }
};

// The entry whose chunks hold chunk b: begin[] ascends from 0, unused entries
// hold UINT32_MAX.
template <int N>
__device__ __forceinline__ int entry_of(const uint32_t (&begin)[N], uint32_t b) {
    const int lane = threadIdx.x & 63;
    int at = -1;
#pragma unroll
    for (int k = 0; k < N; k += 64) {
        const uint32_t first = k + lane < N ? begin[k + lane] : UINT32_MAX;
        at += __builtin_popcountll(__ballot(first <= b));
    }
    return __builtin_amdgcn_readfirstlane(at);
}

// ------------------------------------------------------------------ norm and clip factor
constexpr int kNormVecs = 200;
constexpr int64_t kNormChunk = 8192;
constexpr int kNormGroups = 2048;      // workgroups of one launch: 8 on each CU

struct NormParams {
    const void *g[kNormVecs];
    int64_t n[kNormVecs];              // n << 2 | bf16 << 1 | 16-byte aligned
    uint32_t begin[kNormVecs];
    uint32_t chunks;
    double *part;                      // one sum a workgroup
};
static_assert(sizeof(NormParams) <= 4096, "kernel argument");

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
    return x;
}

__device__ __forceinline__ double square_on(double x, double sum) { return __builtin_fma(x, x, sum); }

template <class G>
__device__ __forceinline__ void norm_chunk(const typename G::type *g, int64_t n, bool vec, double &sum) {
    constexpr int kStep = 8;
    if (vec && n >= kNormChunk) {
#pragma unroll
        for (int k = 0; k < kNormChunk / (kThreads * kStep); ++k) {
            float x[kStep];
            G::load(g + (k * kThreads + threadIdx.x) * kStep, x);
#pragma unroll
            for (int i = 0; i < kStep; ++i) sum = square_on(x[i], sum);
        }
    } else {
        const int end = static_cast<int>(n < kNormChunk ? n : kNormChunk), runs = vec ? end / kStep * kStep : 0;
        for (int i = threadIdx.x * kStep; i < runs; i += kThreads * kStep) {
            float x[kStep];
            G::load(g + i, x);
#pragma unroll
            for (int j = 0; j < kStep; ++j) sum = square_on(x[j], sum);
        }
        for (int i = runs + threadIdx.x; i < end; i += kThreads) {
            const double x = G::one(g + i);
            sum = __builtin_fma(x, x, sum);
        }
    }
}

// Sum of squares: in fp64, where the square of every fp32 value is exact and
// in range.
__global__ __launch_bounds__(kThreads) void k_grad_norm(const NormParams p) {
    double sum = 0.0;
    for (uint32_t b = blockIdx.x; b < p.chunks; b += gridDim.x) {
        const int e = entry_of(p.begin, b);
        const int64_t at = static_cast<int64_t>(b - p.begin[e]) * kNormChunk, n = (p.n[e] >> 2) - at;
        const bool vec = p.n[e] & 1;
        if (p.n[e] & 2)
            norm_chunk<BF16>(static_cast<const uint16_t *>(p.g[e]) + at, n, vec, sum);
        else
            norm_chunk<F32>(static_cast<const float *>(p.g[e]) + at, n, vec, sum);
    }
    __shared__ double s[kThreads / 64];
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x == 0) p.part[blockIdx.x] = (s[0] + s[1]) + (s[2] + s[3]);
}

// The workgroups' sums in a fixed order, then the norm and the factor.
__global__ __launch_bounds__(kThreads) void k_grad_clip(const double *part, int32_t n, float max_norm, float *clip,
                                                        float *norm) {
    double sum = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) sum += part[i];
    __shared__ double s[kThreads / 64];
    sum = wave_sum(sum);
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = sum;
    __syncthreads();
    if (threadIdx.x) return;
    const double length = sqrt((s[0] + s[1]) + (s[2] + s[3]));
    const bool finite = length < __builtin_huge_val();
    *clip = !finite ? 0.0f : length > max_norm ? static_cast<float>(max_norm / length) : 1.0f;
    if (norm) *norm = static_cast<float>(length);
}

// ------------------------------------------------------------------ AdamW
struct AdamScalars {
    float lr, beta1, beta2, eps, c1, c2, decay;
    const float *bc1, *bc2;
    const float *clip;
    const int32_t *step_dev;
    int32_t step, t_max;
};

// What a workgroup needs of a step; go = false where the clip factor tells
// that the step is to be left out.
struct AdamStep {
    float k1, k2, clip;
    uint32_t t;
    bool go;
};

__device__ __forceinline__ AdamStep adam_step(const AdamScalars &h) {
    AdamStep s;
    s.clip = h.clip ? *h.clip : 1.0f;
    s.go = s.clip > 0.0f && s.clip < __builtin_huge_valf();
    const int32_t t = h.step_dev ? *h.step_dev : h.step;
    s.t = static_cast<uint32_t>(t);
    const int32_t at = min(max(t, 1), h.t_max);
    s.k1 = h.lr / h.bc1[at];
    s.k2 = 1.0f / __builtin_sqrtf(h.bc2[at]);
    return s;
}

// m and v from the gradient; p after decay and step.  IEEE fp32, each
// operation rounded on its own, in the order of the sparse update.
__device__ __forceinline__ void adam_moments(const AdamScalars &h, const AdamStep &s, float g, float &m, float &v) {
    g *= s.clip;
    m = h.beta1 * m + h.c1 * g;
    v = h.beta2 * v + h.c2 * (g * g);
}
// kRcp: the quotient as a product with the hardware's reciprocal, which is off
// by at most one unit in the last place.  The step with 8-bit states, whose
// arithmetic shows beside its few bytes, takes it (409 -> 372 us a layer); the
// one with fp32 states is bound by its bytes and divides.
template <bool kRcp>
__device__ __forceinline__ float adam_param(const AdamScalars &h, const AdamStep &s, float p, float m, float root) {
    const float den = root * s.k2 + h.eps, num = s.k1 * m;
    return p * h.decay - (kRcp ? num * __builtin_amdgcn_rcpf(den) : num / den);
}

// A group of elements with their moments in fp32.
template <int N>
__device__ __forceinline__ void adam_group(const AdamScalars &h, const AdamStep &s, float (&p)[N], const float (&g)[N],
                                           float (&m)[N], float (&v)[N]) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
        adam_moments(h, s, g[j], m[j], v[j]);
        p[j] = adam_param<false>(h, s, p[j], m[j], __builtin_sqrtf(v[j]));
    }
}

constexpr int kVecs32 = 74;
constexpr int64_t kChunk32 = 2048;

struct Adam32Params {
    void *p[kVecs32];
    const void *g[kVecs32];
    float *m[kVecs32];
    float *v[kVecs32];
    uint16_t *live[kVecs32];
    int64_t n[kVecs32];                // n << 1 | every pointer 16-byte aligned
    uint32_t begin[kVecs32];
    AdamScalars h;
};
static_assert(sizeof(Adam32Params) <= 4096, "kernel argument");

template <class P, class G>
__global__ __launch_bounds__(kThreads) void k_adamw32(const Adam32Params a) {
    const AdamStep s = adam_step(a.h);
    if (!s.go) return;
    const int e = entry_of(a.begin, blockIdx.x);
    const int64_t at = static_cast<int64_t>(blockIdx.x - a.begin[e]) * kChunk32, n = (a.n[e] >> 1) - at;
    typename P::type *p = static_cast<typename P::type *>(a.p[e]) + at;
    const typename G::type *g = static_cast<const typename G::type *>(a.g[e]) + at;
    float *m = a.m[e] + at, *v = a.v[e] + at;
    uint16_t *live = a.live[e] ? a.live[e] + at : nullptr;
    constexpr int N = 4, K = kChunk32 / (kThreads * N);
    float pp[K][N], gg[K][N], mm[K][N], vv[K][N];
    const bool aligned = a.n[e] & 1;
    // whole groups of N where the pointers allow it, one by one at the end and
    // in unaligned tensors
    if (aligned && n >= kChunk32) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = (k * kThreads + threadIdx.x) * N;
            P::load(p + i, pp[k]);
            G::load(g + i, gg[k]);
            F32::load(m + i, mm[k]);
            F32::load(v + i, vv[k]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = (k * kThreads + threadIdx.x) * N;
            adam_group(a.h, s, pp[k], gg[k], mm[k], vv[k]);
            P::store(p + i, pp[k]);
            F32::store(m + i, mm[k]);
            F32::store(v + i, vv[k]);
            if (live) BF16::store(live + i, pp[k]);
        }
        return;
    }
    const int end = static_cast<int>(n < kChunk32 ? n : kChunk32), runs = aligned ? end / N * N : 0;
    for (int i = threadIdx.x * N; i < runs; i += kThreads * N) {
        P::load(p + i, pp[0]);
        G::load(g + i, gg[0]);
        F32::load(m + i, mm[0]);
        F32::load(v + i, vv[0]);
        adam_group(a.h, s, pp[0], gg[0], mm[0], vv[0]);
        P::store(p + i, pp[0]);
        F32::store(m + i, mm[0]);
        F32::store(v + i, vv[0]);
        if (live) BF16::store(live + i, pp[0]);
    }
    for (int i = runs + threadIdx.x; i < end; i += kThreads) {
        float x[1] = {P::one(p + i)}, mi[1] = {m[i]}, vi[1] = {v[i]};
        const float gi[1] = {G::one(g + i)};
        adam_group(a.h, s, x, gi, mi, vi);
        P::put(p + i, x[0]);
        m[i] = mi[0];
        v[i] = vi[0];
        if (live) BF16::put(live + i, x[0]);
    }
}

// ---- states in 8 bits.  A block of 256 elements has a power of two for each
// state, chosen so that the block's largest magnitude lands in [128, 256);
// m / 2^k and sqrt(v) / 2^k are held in e4m3, whose exponent field then lines
// up with the fp32 field of the value times 2^(-k-120): the code is the top
// bits of that pattern.  Rounding to the nearest code would never let v decay
// (a step changes it by 1 - beta2 = 0.1%, a code is 6-12% wide), so a value is
// rounded up where a 20-bit sequence exceeds what is missing to the next code:
// w = i * 0xC2B2AE35 + t * 0x9E3779B9 (mod 2^32), which over the steps t of an
// element i fills [0, 1) evenly, so that the held state follows the true one
// without bias (relative deviation of sqrt(v) over 4000 steps 0.13, against
// 0.5 with nearest rounding and 0.3 growing with independent draws).
constexpr int kBlock = 256;
constexpr int kVecs8 = 64;
constexpr int64_t kChunk8 = 4096;
constexpr uint32_t kTurnM = 0x55555555u;   // m's place in the sequence against sqrt(v)'s

struct Adam8Params {
    void *p[kVecs8];
    const void *g[kVecs8];
    uint8_t *m[kVecs8];
    uint8_t *v[kVecs8];
    uint8_t *scale[kVecs8];
    uint16_t *live[kVecs8];
    int64_t n[kVecs8];
    uint32_t begin[kVecs8];
    AdamScalars h;
};
static_assert(sizeof(Adam8Params) <= 4096, "kernel argument");

// Largest value over the 32 lanes that share a block.
__device__ __forceinline__ uint32_t block_max(uint32_t x) {
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x128, 0xf, 0xf, false)));
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x124, 0xf, 0xf, false)));
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x122, 0xf, 0xf, false)));
    x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x121, 0xf, 0xf, false)));
    return max(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), 16)));
}

// The scale byte (k + 127; 255 = not finite) of a block whose largest
// magnitude has these bits (NaN and infinity compare above every number).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    if (top >= 0x7f800000u) return 255u;
    if (top == 0u) return 127u;
    return static_cast<uint32_t>(max(static_cast<int32_t>(top >> 23) - 7, 0));
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
    // 2^(byte - 127); byte 0 is the subnormal 2^-127, 255 is NaN
    return __builtin_bit_cast(float, byte == 255u ? 0x7fc00000u : byte ? byte << 23 : 0x00400000u);
}

template <bool kSigned>
__device__ __forceinline__ uint32_t code_of(float x, int32_t shift, uint32_t w) {
    const uint32_t bits = __builtin_bit_cast(uint32_t, x);
    const float y = __builtin_ldexpf(__builtin_bit_cast(float, bits & 0x7fffffffu), shift);
    uint32_t c = (__builtin_bit_cast(uint32_t, y) + (w >> 12)) >> 20;
    if constexpr (kSigned) return c | (bits >> 24 & 0x80u);
    return c ? c : (bits ? 1u : 0u);       // a root of zero would let m / eps through
}

__device__ __forceinline__ void codes_up(uint32_t w, float scale, float *x) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    x[0] = lo.x * scale, x[1] = lo.y * scale, x[2] = hi.x * scale, x[3] = hi.y * scale;
}

// A lane takes 8 consecutive elements, 32 lanes a block, so that every array
// is read in whole runs of 512 bytes and more; two rounds of a wave a chunk.
template <class P, class G>
__global__ __launch_bounds__(kThreads) void k_adamw8(const Adam8Params a) {
    const AdamStep s = adam_step(a.h);
    if (!s.go) return;
    const int e = entry_of(a.begin, blockIdx.x);
    const int64_t at = static_cast<int64_t>(blockIdx.x - a.begin[e]) * kChunk8, n = (a.n[e] >> 1) - at;
    typename P::type *p = static_cast<typename P::type *>(a.p[e]) + at;
    const typename G::type *g = static_cast<const typename G::type *>(a.g[e]) + at;
    uint8_t *m = a.m[e] + at, *v = a.v[e] + at, *scale = a.scale[e] + at / kBlock * 2;
    uint16_t *live = a.live[e] ? a.live[e] + at : nullptr;
    const bool aligned = a.n[e] & 1, whole = aligned && n >= kChunk8;
    constexpr int N = 8, K = kChunk8 / (kThreads * N);
    float pp[K][N], gg[K][N];
    uint32_t mc[K][2], vc[K][2], sm[K], sv[K];
    if (whole) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = (k * kThreads + threadIdx.x) * N;
            const u32x2 a0 = stream_get<u32x2>(m + i), a1 = stream_get<u32x2>(v + i);
            P::load(p + i, pp[k]);
            G::load(g + i, gg[k]);
            mc[k][0] = a0.x, mc[k][1] = a0.y, vc[k][0] = a1.x, vc[k][1] = a1.y;
            sm[k] = scale[i / kBlock * 2];
            sv[k] = scale[i / kBlock * 2 + 1];
        }
    } else {
        // a lane's group whole where it is inside, else one by one (on average
        // half of the last chunk of every tensor: 123 tensors of 26000
        // elements 18.1 us, one by one throughout 26.7)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = (k * kThreads + threadIdx.x) * N;
            sm[k] = i < n ? scale[i / kBlock * 2] : 127u;
            sv[k] = i < n ? scale[i / kBlock * 2 + 1] : 127u;
            if (aligned && i + N <= n) {
                const u32x2 a0 = stream_get<u32x2>(m + i), a1 = stream_get<u32x2>(v + i);
                P::load(p + i, pp[k]);
                G::load(g + i, gg[k]);
                mc[k][0] = a0.x, mc[k][1] = a0.y, vc[k][0] = a1.x, vc[k][1] = a1.y;
                continue;
            }
            mc[k][0] = mc[k][1] = vc[k][0] = vc[k][1] = 0;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const bool in = i + j < n;
                pp[k][j] = in ? P::one(p + i + j) : 0.0f;
                gg[k][j] = in ? G::one(g + i + j) : 0.0f;
                mc[k][j / 4] |= (in ? m[i + j] : 0u) << (8 * (j & 3));
                vc[k][j / 4] |= (in ? v[i + j] : 0u) << (8 * (j & 3));
            }
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = (k * kThreads + threadIdx.x) * N;
        float mm[N], rr[N];
        const float fm = scale_value(sm[k]), fv = scale_value(sv[k]);
        codes_up(mc[k][0], fm, mm);
        codes_up(mc[k][1], fm, mm + 4);
        codes_up(vc[k][0], fv, rr);
        codes_up(vc[k][1], fv, rr + 4);
        uint32_t top_m = 0, top_r = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float r = rr[j] * rr[j];
            adam_moments(a.h, s, gg[k][j], mm[j], r);
            rr[j] = __builtin_sqrtf(r);
            pp[k][j] = adam_param<true>(a.h, s, pp[k][j], mm[j], rr[j]);
            top_m = max(top_m, __builtin_bit_cast(uint32_t, mm[j]) & 0x7fffffffu);
            top_r = max(top_r, __builtin_bit_cast(uint32_t, rr[j]) & 0x7fffffffu);
        }
        const uint32_t bm = scale_byte(block_max(top_m)), br = scale_byte(block_max(top_r));
        // in a block that is not finite the codes mean nothing: its scale says so
        const int32_t shift_m = bm == 255u ? -1000 : 7 - static_cast<int32_t>(bm);
        const int32_t shift_r = br == 255u ? -1000 : 7 - static_cast<int32_t>(br);
        uint32_t w = (static_cast<uint32_t>(at) + static_cast<uint32_t>(i)) * 0xC2B2AE35u + s.t * 0x9E3779B9u;
        mc[k][0] = mc[k][1] = vc[k][0] = vc[k][1] = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            mc[k][j / 4] |= code_of<true>(mm[j], shift_m, w + kTurnM) << (8 * (j & 3));
            vc[k][j / 4] |= code_of<false>(rr[j], shift_r, w) << (8 * (j & 3));
            w += 0xC2B2AE35u;
        }
        if (whole || (aligned && i + N <= n)) {
            P::store(p + i, pp[k]);
            if (live) BF16::store(live + i, pp[k]);
            stream_put(m + i, u32x2{mc[k][0], mc[k][1]});
            stream_put(v + i, u32x2{vc[k][0], vc[k][1]});
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (i + j >= n) continue;
                P::put(p + i + j, pp[k][j]);
                if (live) BF16::put(live + i + j, pp[k][j]);
                m[i + j] = static_cast<uint8_t>(mc[k][j / 4] >> (8 * (j & 3)));
                v[i + j] = static_cast<uint8_t>(vc[k][j / 4] >> (8 * (j & 3)));
            }
        }
        if ((threadIdx.x & 31) == 0 && i < n) {
            scale[i / kBlock * 2] = static_cast<uint8_t>(bm);
            scale[i / kBlock * 2 + 1] = static_cast<uint8_t>(br);
        }
    }
}

// ------------------------------------------------------------------ host
size_t type_size(int32_t type) { return type == SFT_F32 ? 4 : 2; }
bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_grads(const sft_grad_vec *vecs, int32_t n_vecs, const char *who) {
    SFT_CHECK(n_vecs >= 0 && (n_vecs == 0 || vecs), SFT_EINVAL, "%s: bad vector list", who);
    for (int32_t i = 0; i < n_vecs; ++i) {
        const sft_grad_vec &v = vecs[i];
        SFT_CHECK(v.n >= 0, SFT_EINVAL, "%s: vector %d: n < 0", who, i);
        SFT_CHECK(v.n < (int64_t(1) << 42), SFT_ENOTSUP, "%s: vector %d: n >= 2^42", who, i);
        SFT_CHECK(v.type == SFT_F32 || v.type == SFT_BF16, SFT_EINVAL, "%s: vector %d: bad type %d", who, i, v.type);
        if (v.n == 0) continue;
        SFT_CHECK(v.grad, SFT_EINVAL, "%s: vector %d: null pointer", who, i);
        SFT_CHECK(aligned(v.grad, type_size(v.type)), SFT_EALIGN, "%s: vector %d: grad not aligned to its type", who,
                  i);
    }
    return SFT_OK;
}

// The launches of k_grad_norm: as many tensors each as an argument holds.
struct NormLaunch {
    int32_t lo, hi;      // vectors [lo, hi)
    uint32_t chunks, groups;
};

int plan_norm(const sft_grad_vec *vecs, int32_t n_vecs, std::vector<NormLaunch> &plan, const char *who) {
    for (int32_t i = 0; i < n_vecs;) {
        NormLaunch l{i, i, 0, 0};
        int64_t chunks = 0;
        for (int used = 0; l.hi < n_vecs && used < kNormVecs; ++l.hi) {
            if (vecs[l.hi].n == 0) continue;
            ++used;
            chunks += (vecs[l.hi].n + kNormChunk - 1) / kNormChunk;
        }
        SFT_CHECK(chunks < (int64_t(1) << 31), SFT_ENOTSUP, "%s: 2^31 chunks or more in one launch", who);
        l.chunks = static_cast<uint32_t>(chunks);
        l.groups = static_cast<uint32_t>(std::min<int64_t>(chunks, kNormGroups));
        if (l.groups) plan.push_back(l);
        i = l.hi;
    }
    return SFT_OK;
}

size_t norm_bytes(const std::vector<NormLaunch> &plan) {
    size_t n = 0;
    for (const NormLaunch &l : plan) n += l.groups;
    return n * sizeof(double);
}

struct Range {
    const uint8_t *lo, *hi;
};

// Whether written ranges overlap: an update of the same bytes from two places
// would be a race.  Lists usually come in ascending order already.
bool overlap(std::vector<Range> &r) {
    const auto by_lo = [](const Range &a, const Range &b) { return a.lo < b.lo; };
    if (!std::is_sorted(r.begin(), r.end(), by_lo)) std::sort(r.begin(), r.end(), by_lo);
    for (size_t i = 1; i < r.size(); ++i)
        if (r[i].lo < r[i - 1].hi) return true;
    return false;
}

// Whether the `bytes` bytes at p touch one of the ranges, which ascend and are
// apart; at: the range where the last search ended, tried first.
bool inside(const std::vector<Range> &r, const void *p, int64_t bytes, size_t &at) {
    const uint8_t *lo = static_cast<const uint8_t *>(p);
    if (!((at == 0 || r[at - 1].hi <= lo) && (at == r.size() || r[at].hi > lo)))
        at = static_cast<size_t>(std::partition_point(r.begin(), r.end(), [lo](const Range &x) { return x.hi <= lo; }) -
                                 r.begin());
    return at < r.size() && r[at].lo < lo + bytes;
}

template <class Params, int kMax, int64_t kChunk>
struct Launch {
    Params a{};
    int used = 0;
    int64_t chunks = 0;
    bool full() const { return used == kMax; }
    void reset() {
        used = 0;
        chunks = 0;
    }
    void close() {
        for (int i = used; i < kMax; ++i) a.begin[i] = UINT32_MAX;
    }
    int add(const sft_adamw_vec &v, bool vec) {
        const int i = used++;
        a.p[i] = v.p;
        a.g[i] = v.grad;
        a.live[i] = v.p_live;
        a.n[i] = v.n << 1 | int64_t(vec);
        a.begin[i] = static_cast<uint32_t>(chunks);
        chunks += (v.n + kChunk - 1) / kChunk;
        return i;
    }
};

typedef Launch<Adam32Params, kVecs32, kChunk32> Launch32;
typedef Launch<Adam8Params, kVecs8, kChunk8> Launch8;

template <class L>
int send(L &l, int p_type, int g_type, hipStream_t st);

#define SFT_SEND(kernel)                                                                                         \
    if (p_type == SFT_F32 && g_type == SFT_F32) hipLaunchKernelGGL((kernel<F32, F32>), grid, block, 0, st, l.a); \
    else if (p_type == SFT_F32) hipLaunchKernelGGL((kernel<F32, BF16>), grid, block, 0, st, l.a);                \
    else if (g_type == SFT_F32) hipLaunchKernelGGL((kernel<BF16, F32>), grid, block, 0, st, l.a);                \
    else hipLaunchKernelGGL((kernel<BF16, BF16>), grid, block, 0, st, l.a);

template <class L>
int send(L &l, int p_type, int g_type, hipStream_t st) {
    if (l.used == 0) return SFT_OK;
    l.close();
    const dim3 grid(static_cast<uint32_t>(l.chunks)), block(kThreads);
    if constexpr (std::is_same<L, Launch32>::value) {
        SFT_SEND(k_adamw32)
    } else {
        SFT_SEND(k_adamw8)
    }
    const hipError_t e = hipGetLastError();
    SFT_CHECK(e == hipSuccess, SFT_EHIP, "sft_adamw: launch failed: %s", hipGetErrorString(e));
    l.reset();
    return SFT_OK;
}

int grad_clip(const sft_grad_vec *vecs, int32_t n_vecs, float max_norm, float *clip, float *norm, void *ws,
              size_t ws_bytes, void *stream) {
    if (int rc = check_grads(vecs, n_vecs, "sft_grad_clip")) return rc;
    SFT_CHECK(max_norm > 0.0f, SFT_EINVAL, "sft_grad_clip: max_norm must be positive");
    SFT_CHECK(clip, SFT_EINVAL, "sft_grad_clip: clip is null");
    SFT_CHECK(aligned(clip, 4) && aligned(norm, 4), SFT_EALIGN, "sft_grad_clip: clip or norm not 4-byte aligned");
    std::vector<NormLaunch> plan;
    if (int rc = plan_norm(vecs, n_vecs, plan, "sft_grad_clip")) return rc;
    const size_t need = norm_bytes(plan);
    SFT_CHECK(ws_bytes >= need, SFT_ECAPACITY, "sft_grad_clip: workspace %zu < %zu bytes", ws_bytes, need);
    SFT_CHECK(need == 0 || ws, SFT_EINVAL, "sft_grad_clip: workspace is null");
    SFT_CHECK(sft::aligned16(ws), SFT_EALIGN, "sft_grad_clip: workspace not 16-byte aligned");
    SFT_CHECK(clip != norm, SFT_EINVAL, "sft_grad_clip: clip and norm overlap");
    const uint8_t *const lo = static_cast<const uint8_t *>(ws);
    for (int32_t i = 0; i < n_vecs; ++i) {
        const uint8_t *const g = static_cast<const uint8_t *>(vecs[i].grad);
        SFT_CHECK(vecs[i].n == 0 || g + vecs[i].n * int64_t(type_size(vecs[i].type)) <= lo || lo + need <= g, SFT_EINVAL,
                  "sft_grad_clip: vector %d and the workspace overlap", i);
    }
    const hipStream_t st = static_cast<hipStream_t>(stream);
    double *part = static_cast<double *>(ws);
    int32_t parts = 0;
    for (const NormLaunch &l : plan) {
        NormParams p{};
        int used = 0;
        int64_t chunks = 0;
        for (int32_t i = l.lo; i < l.hi; ++i) {
            if (vecs[i].n == 0) continue;
            p.g[used] = vecs[i].grad;
            p.n[used] = vecs[i].n << 2 | int64_t(vecs[i].type == SFT_BF16) << 1 | int64_t(sft::aligned16(vecs[i].grad));
            p.begin[used] = static_cast<uint32_t>(chunks);
            chunks += (vecs[i].n + kNormChunk - 1) / kNormChunk;
            ++used;
        }
        for (; used < kNormVecs; ++used) p.begin[used] = UINT32_MAX;
        p.chunks = l.chunks;
        p.part = part + parts;
        hipLaunchKernelGGL(k_grad_norm, dim3(l.groups), dim3(kThreads), 0, st, p);
        const hipError_t e = hipGetLastError();
        SFT_CHECK(e == hipSuccess, SFT_EHIP, "sft_grad_clip: launch failed: %s", hipGetErrorString(e));
        parts += static_cast<int32_t>(l.groups);
    }
    hipLaunchKernelGGL(k_grad_clip, dim3(1), dim3(kThreads), 0, st, part, parts, max_norm, clip, norm);
    const hipError_t e = hipGetLastError();
    SFT_CHECK(e == hipSuccess, SFT_EHIP, "sft_grad_clip: launch failed: %s", hipGetErrorString(e));
    return SFT_OK;
}

int adamw(const sft_adamw_vec *vecs, int32_t n_vecs, int32_t step, const int32_t *step_dev, const float *clip,
          const sft_adam *hp, void *stream) {
    SFT_CHECK(n_vecs >= 0 && (n_vecs == 0 || vecs), SFT_EINVAL, "sft_adamw: bad vector list");
    SFT_CHECK(hp && hp->bc1 && hp->bc2, SFT_EINVAL, "sft_adamw: missing Adam parameters or bias table");
    SFT_CHECK(hp->t_max >= 1, SFT_EINVAL, "sft_adamw: t_max < 1");
    SFT_CHECK(hp->beta1 >= 0.0f && hp->beta1 < 1.0f && hp->beta2 >= 0.0f && hp->beta2 < 1.0f, SFT_EINVAL,
              "sft_adamw: beta1 or beta2 outside [0, 1)");
    // (a subnormal eps alone in the denominator would have no reciprocal)
    SFT_CHECK(hp->eps == 0.0f || hp->eps >= FLT_MIN, SFT_EINVAL,
              "sft_adamw: eps is negative, subnormal or not a number");
    SFT_CHECK(step_dev || step >= 1, SFT_EINVAL, "sft_adamw: step %d < 1", step);
    SFT_CHECK(aligned(step_dev, 4) && aligned(clip, 4), SFT_EALIGN, "sft_adamw: step_dev or clip not 4-byte aligned");
    int64_t chunks = 0;
    const uint8_t *low = reinterpret_cast<const uint8_t *>(UINTPTR_MAX), *top = nullptr;    // of the gradients
    std::vector<Range> written;
    written.reserve(static_cast<size_t>(n_vecs) * 3);
    const auto writes = [&](const void *p, int64_t bytes) {
        const uint8_t *b = static_cast<const uint8_t *>(p);
        if (b) written.push_back({b, b + bytes});
    };
    for (int32_t i = 0; i < n_vecs; ++i) {
        const sft_adamw_vec &v = vecs[i];
        SFT_CHECK(v.n >= 0, SFT_EINVAL, "sft_adamw: vector %d: n < 0", i);
        SFT_CHECK(v.n < (int64_t(1) << 42), SFT_ENOTSUP, "sft_adamw: vector %d: n >= 2^42", i);
        SFT_CHECK((v.p_type == SFT_F32 || v.p_type == SFT_BF16) && (v.g_type == SFT_F32 || v.g_type == SFT_BF16),
                  SFT_EINVAL, "sft_adamw: vector %d: bad type", i);
        if (v.n == 0) continue;
        SFT_CHECK(v.p && v.grad && v.m && v.v, SFT_EINVAL, "sft_adamw: vector %d: null pointer", i);
        SFT_CHECK(aligned(v.p, type_size(v.p_type)) && aligned(v.grad, type_size(v.g_type)) &&
                      aligned(v.p_live, 2) && (v.scale || (aligned(v.m, 4) && aligned(v.v, 4))),
                  SFT_EALIGN, "sft_adamw: vector %d: a pointer is not aligned to its type", i);
        chunks += v.scale ? (v.n + kChunk8 - 1) / kChunk8 : (v.n + kChunk32 - 1) / kChunk32;
        const uint8_t *const g = static_cast<const uint8_t *>(v.grad);
        low = std::min(low, g);
        top = std::max(top, g + v.n * int64_t(type_size(v.g_type)));
    }
    // a launch has fewer than 2^32 threads
    SFT_CHECK(chunks < (int64_t(1) << 32) / kThreads, SFT_ENOTSUP, "sft_adamw: 2^24 chunks of values or more");
    // array by array: each ascends on its own where the tensors are views of flat buffers
    for (int32_t i = 0; i < n_vecs; ++i)
        if (vecs[i].n) writes(vecs[i].p, vecs[i].n * int64_t(type_size(vecs[i].p_type)));
    for (int32_t i = 0; i < n_vecs; ++i)
        if (vecs[i].n) writes(vecs[i].m, vecs[i].n * (vecs[i].scale ? 1 : 4));
    for (int32_t i = 0; i < n_vecs; ++i)
        if (vecs[i].n) writes(vecs[i].v, vecs[i].n * (vecs[i].scale ? 1 : 4));
    for (int32_t i = 0; i < n_vecs; ++i)
        if (vecs[i].n) {
            writes(vecs[i].scale, (vecs[i].n + kBlock - 1) / kBlock * 2);
            writes(vecs[i].p_live, vecs[i].n * 2);
        }
    SFT_CHECK(!overlap(written), SFT_EINVAL, "sft_adamw: two arrays that the step writes overlap");
    // other workgroups may still read what one of them writes; gradients often
    // share a buffer, so first from the lowest address to the highest
    size_t at = 0;
    if (top > low && inside(written, low, top - low, at))
        for (int32_t i = 0; i < n_vecs; ++i)
            SFT_CHECK(vecs[i].n == 0 || !inside(written, vecs[i].grad, vecs[i].n * int64_t(type_size(vecs[i].g_type)), at),
                      SFT_EINVAL, "sft_adamw: vector %d: the gradient overlaps an array that the step writes", i);
    const int64_t table = 4 * (int64_t(hp->t_max) + 1);
    SFT_CHECK(!inside(written, hp->bc1, table, at) && !inside(written, hp->bc2, table, at) &&
                  !(clip && inside(written, clip, 4, at)) && !(step_dev && inside(written, step_dev, 4, at)),
              SFT_EINVAL, "sft_adamw: a bias table, clip or step_dev overlaps an array that the step writes");

    AdamScalars h{};
    h.lr = hp->lr;
    h.beta1 = hp->beta1;
    h.beta2 = hp->beta2;
    h.eps = hp->eps;
    h.c1 = 1.0f - hp->beta1;
    h.c2 = 1.0f - hp->beta2;
    h.decay = 1.0f - hp->lr * hp->weight_decay;
    h.bc1 = hp->bc1;
    h.bc2 = hp->bc2;
    h.clip = clip;
    h.step_dev = step_dev;
    h.step = step;
    h.t_max = hp->t_max;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const auto kind_of = [](const sft_adamw_vec &v) { return v.p_type | v.g_type << 1 | int(v.scale != nullptr) << 2; };
    uint32_t kinds = 0;
    for (int32_t i = 0; i < n_vecs; ++i)
        if (vecs[i].n) kinds |= 1u << kind_of(vecs[i]);
    // one launch for the tensors of each kind
    for (int kind = 0; kind < 8; ++kind) {
        if (!(kinds >> kind & 1u)) continue;
        const int p_type = kind & 1, g_type = kind >> 1 & 1;
        const bool held = kind >> 2;
        Launch32 l32;
        Launch8 l8;
        l32.a.h = h;
        l8.a.h = h;
        for (int32_t i = 0; i < n_vecs; ++i) {
            const sft_adamw_vec &v = vecs[i];
            if (v.n == 0 || kind_of(v) != kind) continue;
            const bool vec = sft::aligned16(v.p) && sft::aligned16(v.grad) && sft::aligned16(v.m) &&
                             sft::aligned16(v.v) && sft::aligned16(v.p_live);
            if (held) {
                if (l8.full())
                    if (int rc = send(l8, p_type, g_type, st)) return rc;
                const int k = l8.add(v, vec);
                l8.a.m[k] = static_cast<uint8_t *>(v.m);
                l8.a.v[k] = static_cast<uint8_t *>(v.v);
                l8.a.scale[k] = v.scale;
            } else {
                if (l32.full())
                    if (int rc = send(l32, p_type, g_type, st)) return rc;
                const int k = l32.add(v, vec);
                l32.a.m[k] = static_cast<float *>(v.m);
                l32.a.v[k] = static_cast<float *>(v.v);
            }
        }
        if (int rc = send(l32, p_type, g_type, st)) return rc;
        if (int rc = send(l8, p_type, g_type, st)) return rc;
    }
    return SFT_OK;
}

}  // namespace

extern "C" {

// The lists built on the host may fail to allocate: no exception leaves here.
size_t sft_grad_clip_workspace(const sft_grad_vec *vecs, int32_t n_vecs) try {
    sft::clear_error();
    std::vector<NormLaunch> plan;
    if (check_grads(vecs, n_vecs, "sft_grad_clip_workspace") ||
        plan_norm(vecs, n_vecs, plan, "sft_grad_clip_workspace"))
        return static_cast<size_t>(-1);
    return norm_bytes(plan);
} catch (...) {
    (void)sft::fail(SFT_ECAPACITY, "sft_grad_clip_workspace: out of host memory");
    return static_cast<size_t>(-1);
}

int sft_grad_clip(const sft_grad_vec *vecs, int32_t n_vecs, float max_norm, float *clip, float *norm, void *ws,
                  size_t ws_bytes, void *stream) try {
    sft::clear_error();
    return grad_clip(vecs, n_vecs, max_norm, clip, norm, ws, ws_bytes, stream);
} catch (...) {
    return sft::fail(SFT_ECAPACITY, "sft_grad_clip: out of host memory");
}

int sft_adamw(const sft_adamw_vec *vecs, int32_t n_vecs, int32_t step, const int32_t *step_dev, const float *clip,
              const sft_adam *hp, void *stream) try {
    sft::clear_error();
    return adamw(vecs, n_vecs, step, step_dev, clip, hp, stream);
} catch (...) {
    return sft::fail(SFT_ECAPACITY, "sft_adamw: out of host memory");
}

}  // extern "C"
