// sft_rotary.hip -- rotary positions: pairs of elements of queries and keys
// turned by angles that grow with the token's position, and the table of those
// angles.
//
//     (a, b) -> amplitude (a cos t - b sin t, a sin t + b cos t),  t = position * angle; inverse: -t
//
// Every element is read and written once, so the call is bound by HBM: 4096
// tokens of 32 + 32 heads of 128 in bf16 take 21.6 us (134 MB, 6.2 TB/s).  The
// sines are the same for all heads of a token: a workgroup takes whole tokens
// (or a part of one's heads) and puts their sines into LDS once, while its
// elements are under way.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "sft_blocks.h"
#include "sft_internal.h"
#include "sft_vec.h"

namespace {

using namespace sft;

// Threads of a workgroup.  An item is two groups of elements of a head, whose
// loads are under way while the sines are computed; a workgroup takes an item a
// thread, of several tokens or of a part of one token's heads.  More items a
// thread leave too few workgroups on a CU (4096 tokens of 32 + 32 heads of 128
// in bf16, at the time: 23.4 us, two items 26.0; 512 threads 24.4).
constexpr int kThreads = 256;
constexpr int kMaxMats = 8;
constexpr int kMaxHead = 4096;

// n / d for n < 2^31.
struct Div {
    uint32_t mul, shift, by;
};
Div div_by(uint32_t d) {
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    return {static_cast<uint32_t>((uint64_t(1) << (31 + s)) / d + 1), 31 + s, d};
}
__device__ __forceinline__ uint32_t over(uint32_t n, const Div &d) {
    return static_cast<uint32_t>(uint64_t(n) * d.mul >> d.shift);
}

struct RotaryMat {
    const void *x;
    void *y;
    int64_t x_batch, x_row, x_head, y_batch, y_row, y_head;
    Div units, heads, parts;    // items of a head; heads; parts of a token's heads
    int32_t tokens, items;      // of a workgroup
    uint32_t begin;             // the first of its workgroups
};

struct Rotary {
    RotaryMat m[kMaxMats];
    const double *freq;
    const int32_t *pos;
    int64_t pos_batch;
    Div rows, pairs;            // tokens of a sequence; pairs of a head
    int32_t n_mats, D, rot, total;    // total: tokens of all sequences
    uint32_t blocks;
    float amplitude;
    bool inverse;
};

// One item: two groups of up to N elements, where they start in the head, how
// many there are, and the places of their first pairs' sines.  The second group
// is as far from the first as the units allow, so that a wave's accesses are
// whole runs: with SFT_ROTARY_HALF the pairs' other elements, else the second
// half of the groups.
struct Item {
    int64_t x, y;               // the head's first element in either array
    int32_t at0, at1, n0, n1;
    int32_t sine0, sine1;       // -1: to be copied
};

template <int N, bool kHalf>
__device__ __forceinline__ Item item_of(const Rotary &a, const RotaryMat &m, uint32_t i, uint32_t first) {
    Item it;
    const int half = a.rot / 2, pair_units = (half + N - 1) / N;
    const uint32_t q = over(i, m.units), t = over(q, m.heads);
    const int u = static_cast<int>(i - q * m.units.by);
    const int64_t head = q - t * m.heads.by;
    const uint32_t token = first + t, b = over(token, a.rows);
    const int64_t row = token - b * a.rows.by;
    it.x = b * m.x_batch + row * m.x_row + head * m.x_head;
    it.y = b * m.y_batch + row * m.y_row + head * m.y_head;
    if (u < pair_units) {
        const int sines = static_cast<int>(t) * half;
        if constexpr (kHalf) {
            it.at0 = N * u, it.at1 = half + N * u;
            it.n0 = it.n1 = min(N, half - N * u);
            it.sine0 = it.sine1 = sines + N * u;
        } else {
            it.at0 = N * u, it.at1 = N * (u + pair_units);
            it.n0 = min(N, a.rot - it.at0), it.n1 = min(N, a.rot - it.at1);
            it.sine0 = sines + it.at0 / 2, it.sine1 = sines + (it.n1 > 0 ? it.at1 / 2 : 0);
        }
    } else {
        it.sine0 = it.sine1 = -1;
        const int copy_units = static_cast<int>(m.units.by) - pair_units;
        it.at0 = a.rot + N * (u - pair_units), it.at1 = it.at0 + N * copy_units;
        it.n0 = min(N, a.D - it.at0), it.n1 = min(N, a.D - it.at1);
    }
    return it;
}

template <class E, bool kHalf, bool kPast>
__device__ __forceinline__ void turn_item(const Item &it, const Raw<E, E::kGroup> &r0, const Raw<E, E::kGroup> &r1,
                                          const float *sines, typename E::type *y) {
    constexpr int N = E::kGroup;
    y += it.y;
    if (it.sine0 < 0) {
        put_group<E, N, kPast>(y + it.at0, r0, it.n0);
        put_group<E, N, kPast>(y + it.at1, r1, it.n1);
        return;
    }
    float u[N], v[N];
    open<E, N>(r0, u);
    open<E, N>(r1, v);
    const float *s0 = sines + 2 * it.sine0, *s1 = sines + 2 * it.sine1;
    if constexpr (kHalf) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float p = u[i], q = v[i], c = s0[2 * i], s = s0[2 * i + 1];
            u[i] = __builtin_fmaf(p, c, -(q * s));
            v[i] = __builtin_fmaf(p, s, q * c);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float p = u[i], q = u[i + 1], f = v[i], g = v[i + 1];
            u[i] = __builtin_fmaf(p, s0[i], -(q * s0[i + 1]));
            u[i + 1] = __builtin_fmaf(p, s0[i + 1], q * s0[i]);
            v[i] = __builtin_fmaf(f, s1[i], -(g * s1[i + 1]));
            v[i + 1] = __builtin_fmaf(f, s1[i + 1], g * s1[i]);
        }
    }
    put_group<E, N, kPast>(y + it.at0, close<E, N>(u), it.n0);
    put_group<E, N, kPast>(y + it.at1, close<E, N>(v), it.n1);
}

// The turns that pos steps of `angle` make, but for whole ones.  Both products
// carry what their roundings leave out, and 1/(2 pi) its second part: rounded to
// fp64 alone, three of them would be 6 units of fp32 at position 2^30.
__device__ __forceinline__ double turns_of(double angle, int32_t pos) {
    constexpr double kTurn = 0x1.45f306dc9c883p-3, kTurnRest = -0x1.6b01ec5417056p-57;
    const double step = angle * kTurn, step_rest = __builtin_fma(angle, kTurn, -step) + angle * kTurnRest;
    const double all = step * pos, rest = __builtin_fma(step, double(pos), -all) + step_rest * pos;
    return (all - __builtin_rint(all)) + rest;
}

template <class E, bool kHalf, bool kPast>
__global__ __launch_bounds__(kThreads) void k_rotary(const Rotary a) {
    extern __shared__ f32x4 room[];       // cosine and sine of each token's pairs, and 8 pairs more for a last short group
    constexpr int N = E::kGroup;
    typedef typename E::type type;
    float *const sines = reinterpret_cast<float *>(room);
    const int half = a.rot / 2;
    for (uint32_t block = blockIdx.x; block < a.blocks; block += gridDim.x) {
        int k = 0;
        while (k + 1 < a.n_mats && a.m[k + 1].begin <= block) ++k;
        const RotaryMat &m = a.m[k];
        const uint32_t at = over(block - m.begin, m.parts), first = at * uint32_t(m.tokens);
        const uint32_t tokens = min(uint32_t(m.tokens), uint32_t(a.total) - first);
        const uint32_t i = (block - m.begin - at * m.parts.by) * uint32_t(m.items) + threadIdx.x;
        const bool live = threadIdx.x < uint32_t(m.items) && i < tokens * m.heads.by * m.units.by;
        const type *x = static_cast<const type *>(m.x);
        Item it;
        Raw<E, N> r0, r1;
        if (live) {
            it = item_of<N, kHalf>(a, m, i, first);
            r0 = get_group<E, N>(x + it.x + it.at0, it.n0);
            r1 = get_group<E, N>(x + it.x + it.at1, it.n1);
        }
        // in turns, of which whole ones do not matter
        for (uint32_t k = threadIdx.x; k < tokens * uint32_t(half); k += kThreads) {
            const uint32_t t = over(k, a.pairs), token = first + t, b = over(token, a.rows);
            const int32_t pos = a.pos[b * a.pos_batch + (token - b * a.rows.by)];
            const double turns = turns_of(a.freq[k - t * half], pos);
            float s, c;
            sincospif(static_cast<float>(2.0 * turns), &s, &c);
            sines[2 * k] = c * a.amplitude;
            sines[2 * k + 1] = (a.inverse ? -s : s) * a.amplitude;
        }
        __syncthreads();
        if (live) turn_item<E, kHalf, kPast>(it, r0, r1, sines, static_cast<type *>(m.y));
        __syncthreads();
    }
}

Block heads_block(const void *p, int64_t B, int64_t T, int64_t heads, int64_t batch, int64_t row, int64_t head,
                  int64_t D, int64_t size) {
    return Block{p, D * size, {{B, batch * size}, {T, row * size}, {heads, head * size}}};
}

}  // namespace

extern "C" {

int sft_rotary_table(int64_t rot, double base, int32_t kind, double factor, double context, double low, double high,
                     double *freq) {
    const char *const who = "sft_rotary_table";
    clear_error();
    SFT_CHECK(freq, SFT_EINVAL, "%s: freq is null", who);
    SFT_CHECK(kind >= SFT_ROTARY_PLAIN && kind <= SFT_ROTARY_BANDS, SFT_EINVAL, "%s: bad kind %d", who, kind);
    SFT_CHECK(rot >= 2 && rot % 2 == 0, SFT_ESHAPE, "%s: rot is odd or below 2", who);
    SFT_CHECK(std::isfinite(base) && base > 0.0, SFT_EINVAL, "%s: base is not positive and finite", who);
    SFT_CHECK(std::isfinite(factor) && factor >= 1.0, SFT_EINVAL, "%s: factor is below 1 or not finite", who);
    if (kind == SFT_ROTARY_BANDS) {
        SFT_CHECK(std::isfinite(context) && context > 0.0, SFT_EINVAL, "%s: context is not positive and finite", who);
        SFT_CHECK(std::isfinite(low) && std::isfinite(high) && high > low, SFT_EINVAL,
                  "%s: low and high are not finite and ascending", who);
    }
    const double n = static_cast<double>(rot);
    if (kind == SFT_ROTARY_BASE && rot > 2) base *= std::pow(factor, n / (n - 2.0));
    SFT_CHECK(std::isfinite(base), SFT_EINVAL, "%s: base * factor^(rot/(rot-2)) is not finite", who);
    for (int64_t j = 0; j < rot / 2; ++j) {
        double f = std::pow(base, -2.0 * static_cast<double>(j) / n);
        if (kind == SFT_ROTARY_LINEAR) f /= factor;
        if (kind == SFT_ROTARY_BANDS) {
            const double turns = context * f / 6.283185307179586477;
            const double w = std::min(1.0, std::max(0.0, (turns - low) / (high - low)));
            f *= w + (1.0 - w) / factor;
        }
        freq[j] = f;
    }
    return SFT_OK;
}

int sft_rotary(const sft_rotary_args *v, void *stream) {
    const char *const who = "sft_rotary";
    clear_error();
    SFT_CHECK(v, SFT_EINVAL, "%s: args is null", who);
    const sft_rotary_mat *const mats = v->mats;
    const int32_t n_mats = v->n_mats, layout = v->layout, type = v->type;
    const int64_t B = v->B, T = v->T, D = v->D, rot = v->rot, pos_batch = v->pos_batch;
    const double *const freq = v->freq;
    const int32_t *const pos = v->pos;
    SFT_CHECK(n_mats >= 0 && (n_mats == 0 || mats), SFT_EINVAL, "%s: bad list", who);
    SFT_CHECK(n_mats <= kMaxMats, SFT_ENOTSUP, "%s: more than %d arrays", who, kMaxMats);
    SFT_CHECK(B >= 0 && T >= 0 && D >= 0 && pos_batch >= 0, SFT_EINVAL, "%s: negative size or distance", who);
    SFT_CHECK(D <= kMaxHead, SFT_ENOTSUP, "%s: D > %d", who, kMaxHead);
    SFT_CHECK(B < (int64_t(1) << 30) && T < (int64_t(1) << 30) && B * T < (int64_t(1) << 30), SFT_ENOTSUP,
              "%s: 2^30 tokens or more", who);
    SFT_CHECK(rot >= 2 && rot % 2 == 0 && rot <= D, SFT_ESHAPE, "%s: rot is odd, below 2 or above D", who);
    SFT_CHECK(type == SFT_F32 || type == SFT_BF16, SFT_EINVAL, "%s: bad type %d", who, type);
    SFT_CHECK(layout == SFT_ROTARY_HALF || layout == SFT_ROTARY_PAIRS, SFT_EINVAL, "%s: bad layout %d", who, layout);
    SFT_CHECK(std::isfinite(v->amplitude), SFT_EINVAL, "%s: amplitude is not finite", who);
    const int64_t total = B * T, size = type_bytes(type), most = int64_t(1) << 40;
    const bool any = n_mats && total;
    SFT_CHECK(!any || (freq && pos), SFT_EINVAL, "%s: freq or pos is null", who);
    SFT_CHECK(aligned_to(freq, 8) && aligned_to(pos, 4), SFT_EALIGN, "%s: freq or pos not aligned to its type", who);
    SFT_CHECK(pos_batch < most, SFT_ENOTSUP, "%s: a distance of 2^40 or more", who);
    Block x[kMaxMats], y[kMaxMats];
    for (int32_t i = 0; i < n_mats; ++i) {
        const sft_rotary_mat &m = mats[i];
        SFT_CHECK(m.heads >= 0, SFT_EINVAL, "%s: array %d: negative size", who, i);
        SFT_CHECK(m.heads < (1 << 16), SFT_ENOTSUP, "%s: array %d: 2^16 heads or more", who, i);
        for (int64_t d : {m.x_batch, m.x_row, m.x_head, m.y_batch, m.y_row, m.y_head}) {
            SFT_CHECK(d >= 0, SFT_EINVAL, "%s: array %d: negative distance", who, i);
            SFT_CHECK(d < most, SFT_ENOTSUP, "%s: array %d: a distance of 2^40 or more", who, i);
        }
        SFT_CHECK(m.heads == 0 || !any || (m.X && m.Y), SFT_EINVAL, "%s: array %d: null pointer", who, i);
        SFT_CHECK(aligned_to(m.X, size) && aligned_to(m.Y, size), SFT_EALIGN, "%s: array %d not aligned to its type",
                  who, i);
        x[i] = heads_block(m.X, B, T, m.heads, m.x_batch, m.x_row, m.x_head, D, size);
        y[i] = heads_block(m.Y, B, T, m.heads, m.y_batch, m.y_row, m.y_head, D, size);
        SFT_CHECK(extent(x[i]) >= 0 && extent(y[i]) >= 0, SFT_ENOTSUP, "%s: array %d spans 2^46 bytes or more", who, i);
        SFT_CHECK(apart_within(y[i]), SFT_EINVAL, "%s: array %d: heads of Y overlap", who, i);
    }
    const Block table = flat_block(freq, rot / 2 * 8);
    const Block where{pos, T * 4, {{pos_batch ? B : 1, pos_batch * 4}, {1, 0}, {1, 0}}};
    SFT_CHECK(extent(where) >= 0, SFT_ENOTSUP, "%s: pos spans 2^46 bytes or more", who);
    for (int32_t i = 0; i < n_mats && total; ++i) {
        SFT_CHECK(apart(y[i], table) && apart(y[i], where), SFT_EINVAL, "%s: array %d overlaps freq or pos", who, i);
        for (int32_t j = 0; j < n_mats; ++j) {
            SFT_CHECK(i == j || apart(y[i], y[j]), SFT_EINVAL, "%s: two written arrays overlap", who);
            SFT_CHECK((i == j && same(y[i], x[j])) || apart(y[i], x[j]), SFT_EINVAL,
                      "%s: a written array overlaps an input", who);
        }
    }
    if (!any) return SFT_OK;
    Rotary a{};
    const int64_t half = rot / 2, group = 16 / size, pair_units = (half + group - 1) / group;
    int64_t blocks = 0, sines = 0;
    bool whole = true;          // every head of the results starts at a multiple of 64 bytes
    for (int32_t i = 0; i < n_mats; ++i) {
        const sft_rotary_mat &m = mats[i];
        if (m.heads == 0) continue;
        RotaryMat &r = a.m[a.n_mats++];
        // what lies behind the turned part stays where it is when Y is X
        const int64_t units = pair_units + (same(x[i], y[i]) ? 0 : (D - rot + 2 * group - 1) / (2 * group));
        r.x = m.X, r.y = m.Y;
        r.x_batch = m.x_batch, r.x_row = m.x_row, r.x_head = m.x_head;
        r.y_batch = m.y_batch, r.y_row = m.y_row, r.y_head = m.y_head;
        r.units = div_by(static_cast<uint32_t>(units));
        r.heads = div_by(static_cast<uint32_t>(m.heads));
        // as many tokens as give every thread an item, and at most two sines
        const int64_t tokens = std::max<int64_t>(
            1, std::min({total, kThreads / (units * m.heads), 2 * kThreads / half}));
        // a single token's heads in even parts
        const int64_t parts = (tokens * units * m.heads + kThreads - 1) / kThreads;
        r.parts = div_by(static_cast<uint32_t>(parts));
        r.tokens = static_cast<int32_t>(tokens);
        r.items = static_cast<int32_t>((tokens * units * m.heads + parts - 1) / parts);
        whole = whole && aligned_to(m.Y, 64) && (m.heads <= 1 || m.y_head * size % 64 == 0) &&
                (T <= 1 || m.y_row * size % 64 == 0) && (B <= 1 || m.y_batch * size % 64 == 0);
        r.begin = static_cast<uint32_t>(blocks);
        blocks += (total + tokens - 1) / tokens * parts;
        sines = std::max(sines, tokens * half);
    }
    SFT_CHECK(blocks < (int64_t(1) << 31), SFT_ENOTSUP, "%s: too many tokens and arrays", who);
    if (!blocks) return SFT_OK;
    a.freq = freq, a.pos = pos, a.pos_batch = pos_batch;
    a.rows = div_by(static_cast<uint32_t>(T));
    a.pairs = div_by(static_cast<uint32_t>(half));
    a.D = static_cast<int32_t>(D), a.rot = static_cast<int32_t>(rot), a.total = static_cast<int32_t>(total);
    a.blocks = static_cast<uint32_t>(blocks);
    a.amplitude = v->amplitude;
    a.inverse = v->inverse != 0;
    const dim3 grid(static_cast<uint32_t>(std::min<int64_t>(blocks, 1 << 23))), block(kThreads);
    const size_t lds = static_cast<size_t>(sines + 8) * 8;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    // Results go past L2 where a wave's stores are whole pieces of 64 bytes or long ones; others are put together in L2.
    // 132 MB in bf16, us past it and through it: heads of 128, 64 and 32 21 and 26, 26.0 and 26.5, 36.5 and 27.1; those of
    // 64 and 128 that start 16 bytes further on 37.3 and 28.5, 30.5 and 27.6; pieces of 7 groups (112) 30.0 and 27.1, of 9
    // that start anywhere (130) 40.1 and 40.2, of 10 (160) 23.9 and 26.2, of 16 that start anywhere (256) 24.5 and 26.8.
    const bool past = pair_units >= 10 || (whole && (layout == SFT_ROTARY_HALF ? half * size : pair_units * 16) % 64 == 0);
#define SFT_SEND(E, half)                                                                        \
    do {                                                                                         \
        if (past) hipLaunchKernelGGL((k_rotary<E, half, true>), grid, block, lds, st, a);        \
        else hipLaunchKernelGGL((k_rotary<E, half, false>), grid, block, lds, st, a);            \
    } while (0)
    if (type == SFT_BF16) {
        if (layout == SFT_ROTARY_HALF) SFT_SEND(Bf16, true);
        else SFT_SEND(Bf16, false);
    } else {
        if (layout == SFT_ROTARY_HALF) SFT_SEND(Fp32, true);
        else SFT_SEND(Fp32, false);
    }
#undef SFT_SEND
    const hipError_t e = hipGetLastError();
    SFT_CHECK(e == hipSuccess, SFT_EHIP, "%s: launch failed: %s", who, hipGetErrorString(e));
    return SFT_OK;
}

}  // extern "C"
