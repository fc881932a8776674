// sft_norm.hip -- layer norm and RMS norm of rows, with the residual's
// addition, and their backward pass with the gains' and biases' gradients.
//
//     h = x + res,  xhat = (h - mean) rstd,  rstd = 1 / sqrt(mean((h - mean)^2) + eps)
//     y = xhat gain + bias
//     g = dy gain,  dx = (g - xhat mean(g xhat) - mean(g)) rstd + dh   (mean(g) for a layer norm)
//     dgain = sum over rows of dy xhat,  dbias = sum over rows of dy
//
// A row is read once into the registers of a team of lanes, its mean and the
// squares of the centred values are summed over the team, and the results are
// written from the same registers, many of them past L2 (30 us through it): both
// passes are bound by HBM, and by launch latency where there are few rows.  4096 x 4096 in
// bf16: forward with residual 21.9 us (134 MB, 6.1 TB/s); backward with dh and
// dgain 27.3 us: under the tracer 24.5 the rows (139 MB with the partial sums, 5.7
// TB/s) and 3.9 the second launch that adds 256 workgroups' sums.  Rows of
// odd widths start between cache lines and cost a quarter more (16384 x 767 in
// bf16: backward 28.5 us, 768 22.0).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "sft_blocks.h"
#include "sft_internal.h"
#include "sft_vec.h"

namespace {

using namespace sft;

constexpr int kMaxWidth = 16384;

// The sum over a team, in all of its lanes.  red: one float a wave, of its own
// for each call (no barrier follows the reads).
template <int kLanes>
__device__ __forceinline__ float team_sum(float x, float *red) {
    x = lanes_of<Sum, (kLanes < 64 ? kLanes : 64)>(x);
    if constexpr (kLanes > 64) {
        constexpr int kWaves = kLanes / 64;
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
        __syncthreads();
        const float *own = red + threadIdx.x / kLanes * kWaves;
        x = own[0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) x += own[i];
    }
    return x;
}

// Elements of the vectors gain and bias, of either type.
template <int N, bool kEven>
__device__ __forceinline__ void get_vector(const void *v, bool w32, int at, int n, float *x) {
    if (w32)
        open<Fp32, N>(get_group<Fp32, N, kEven>(static_cast<const float *>(v) + at, n), x);
    else
        open<Bf16, N>(get_group<Bf16, N, kEven>(static_cast<const uint16_t *>(v) + at, n), x);
}

// Sums of up to 2^14 values are taken in this unit, so that those of finite rows
// are finite; it costs nothing, as a multiply-add is an addition's price.
constexpr float kSumUnit = 0x1p-14f;
static_assert(kMaxWidth <= 1 << 14, "sums of a row");
// Rows whose squares leave fp32 at either end are squared again in units of 2^75
// or 2^-75, in which every finite row's stay inside.
constexpr float kUnit = 0x1p75f, kLeast = 0x1p-90f;

// (squares that are nothing next to eps do not count; NaN leaves, too)
__device__ __forceinline__ bool leaves(float squares, int C, float eps) {
    const float variance = squares / static_cast<float>(C) + eps;
    return !(variance >= kLeast && variance < __builtin_huge_valf());
}

// The sum of a row's squares, of a row of C.
template <int N, int kLanes, int kGroups>
__device__ __forceinline__ float squares_of(const float (&x)[kGroups][N], int lane, int C, float *red) {
    float sum = 0.0f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const int n = C - (g * kLanes + lane) * N;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) sum = __builtin_fmaf(x[g][i], x[g][i], sum);
    }
    return team_sum<kLanes>(sum, red);
}

struct NormForward {
    const void *x, *res;
    void *h;
    const void *gain, *bias;
    void *y;
    float *mean, *rstd;
    int64_t ldx, ldr, ldh, ldy;
    int32_t T, C;
    float eps;
    bool layer, w32;
};

// Waves that a SIMD has to hold: odd rows in fp32 would take a few registers more
// than six of them leave (4096 x 3001: 23.4 us, with five 28.2).
constexpr int forward_waves(int type, int groups, bool even) { return type == SFT_F32 && groups == 2 && !even ? 6 : 1; }

// kEven: C is a multiple of a group.  kPast: results go past L2.
template <class X, class Y, int kLanes, int kGroups, bool kEven, bool kPast>
__global__ __launch_bounds__(kLanes < 256 ? 256 : kLanes, (forward_waves(X::kType, kGroups, kEven))) void k_norm_forward(const NormForward a) {
    constexpr int N = X::kGroup, kThreads = kLanes < 256 ? 256 : kLanes, kTeams = kThreads / kLanes;
    __shared__ float red[2][3][kThreads / 64];       // by turns, so that one barrier a sum is enough
    static_assert(kLanes <= 128 || kTeams == 1, "far rows");
    const int team = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const int C = a.C;
    typedef typename X::type xt;
    int turn = 0;
    for (int64_t first = int64_t(blockIdx.x) * kTeams; first < a.T; first += int64_t(gridDim.x) * kTeams, turn ^= 1) {
        const bool live = first + team < a.T;
        const int64_t row = live ? first + team : a.T - 1;      // a team without a row stays for the barriers
        Raw<X, N> raw[kGroups];
        Few<X, N> few;
        get_row<X, N, kLanes, kEven>(static_cast<const xt *>(a.x) + row * a.ldx, lane, C, raw, few);
        float x[kGroups][N];
        if (a.res) {
            Raw<X, N> other[kGroups];
            Few<X, N> other_few;
            get_row<X, N, kLanes, kEven>(static_cast<const xt *>(a.res) + row * a.ldr, lane, C, other, other_few);
            join_row<X, N, kLanes, kEven>(lane, C, raw, few);
            join_row<X, N, kLanes, kEven>(lane, C, other, other_few);
            xt *h = static_cast<xt *>(a.h) + row * a.ldh;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                float y[N];
                open<X, N>(raw[g], x[g]);
                open<X, N>(other[g], y);
#pragma unroll
                for (int i = 0; i < N; ++i) x[g][i] += y[i];
                const Raw<X, N> sum = close<X, N>(x[g]);
                open<X, N>(sum, x[g]);                    // what is normed is what is kept
                const int at = (g * kLanes + lane) * N;
                if (live) put_group<X, N, kPast, kEven>(h + at, sum, C - at);
            }
        } else {
            join_row<X, N, kLanes, kEven>(lane, C, raw, few);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) open<X, N>(raw[g], x[g]);
        }
        float mean = 0.0f;
        if (a.layer) {
            float sum = 0.0f;
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int i = 0; i < N; ++i) sum = __builtin_fmaf(x[g][i], kSumUnit, sum);      // zeros behind the row's end
            mean = team_sum<kLanes>(sum, red[turn][0]) / static_cast<float>(C) * (1.0f / kSumUnit);
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int i = 0; i < N; ++i) x[g][i] -= mean;
        }
        float squares = squares_of<N, kLanes>(x, lane, C, red[turn][1]), unit = 1.0f, eps = a.eps;
        bool far = leaves(squares, C, eps);
        if (far) unit = squares <= 1.0f ? kUnit : 1.0f / kUnit;
        if constexpr (kLanes == 128) {        // two teams that meet at barriers go the same way
            const float *other = red[turn][1] + (team ^ 1) * 2;
            far = far || leaves(other[0] + other[1], C, eps);
        }
        if (far) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int i = 0; i < N; ++i) x[g][i] *= unit;
            squares = squares_of<N, kLanes>(x, lane, C, red[turn][2]);
            eps = eps * unit * unit;
        }
        const float rstd = 1.0f / __builtin_sqrtf(squares / static_cast<float>(C) + eps);
        if (!live) continue;
        if (lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd * unit;
        }
        typename Y::type *y = static_cast<typename Y::type *>(a.y) + row * a.ldy;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int at = (g * kLanes + lane) * N, n = C - at;
            if (n <= 0) continue;
            float w[N];
#pragma unroll
            for (int i = 0; i < N; ++i) x[g][i] *= rstd;
            if (a.gain) {
                get_vector<N, kEven>(a.gain, a.w32, at, n, w);
#pragma unroll
                for (int i = 0; i < N; ++i) x[g][i] *= w[i];
            }
            if (a.bias) {
                get_vector<N, kEven>(a.bias, a.w32, at, n, w);
#pragma unroll
                for (int i = 0; i < N; ++i) x[g][i] += w[i];
            }
            put_group<Y, N, kPast, kEven>(y + at, close<Y, N>(x[g]), n);
        }
    }
}

// ------------------------------------------------------------------ backward
constexpr int kRowThreads = 1024;

struct NormBackward {
    const void *h, *gain;
    const float *mean, *rstd;
    const void *dy, *dh;
    void *dx;
    float *part;                  // [1 or 2][workgroups][C]
    int64_t ldh, ldy, ldr, ldx;
    int32_t T, C;
    bool layer, w32;
};

// What a team reads of a row.
template <class X, class Y, int kGroups>
struct NormRow {
    static constexpr int N = X::kGroup;
    Raw<X, N> h[kGroups], dh[kGroups];
    Raw<Y, N> dy[kGroups];
    Few<X, N> few_h, few_dh;
    Few<Y, N> few_dy;
    float mean, rstd;
};

template <class X, class Y, int kLanes, bool kEven, int kGroups>
__device__ __forceinline__ void get_norm_row(const NormBackward &a, int64_t row, int lane, NormRow<X, Y, kGroups> &r) {
    constexpr int N = X::kGroup;
    get_row<X, N, kLanes, kEven>(static_cast<const typename X::type *>(a.h) + row * a.ldh, lane, a.C, r.h, r.few_h);
    get_row<Y, N, kLanes, kEven>(static_cast<const typename Y::type *>(a.dy) + row * a.ldy, lane, a.C, r.dy, r.few_dy);
    if (a.dh) get_row<X, N, kLanes, kEven>(static_cast<const typename X::type *>(a.dh) + row * a.ldr, lane, a.C, r.dh, r.few_dh);
    r.rstd = a.rstd[row];
    r.mean = a.layer ? a.mean[row] : 0.0f;
}

// Each team takes rows in turn, kTeams * gridDim.x apart, the next one's loads
// under way while it works on one, and keeps its share of the sums over the
// rows in registers; a workgroup's teams are added at the end, by halves, and
// its sums go to its own place in the workspace.
// kSums: 0 = no sums over rows, 1 = dgain, 2 = dgain and dbias.  The widest
// rows leave no registers for a row ahead or for the gains.
template <class X, class Y, int kLanes, int kGroups, bool kEven, int kSums, bool kPast>
__device__ __forceinline__ void norm_rows(const NormBackward &a, uint32_t block, uint32_t blocks) {
    constexpr int N = X::kGroup, kTeams = kRowThreads / kLanes, kWidth = kLanes * kGroups * N;
    constexpr bool kAhead = kWidth <= 8192;
    __shared__ float red[2][2][kRowThreads / 64];
    __shared__ float total[kTeams > 1 && kSums ? kSums * kWidth * kTeams / 2 : 1];
    const int team = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const int C = a.C;
    typedef typename X::type xt;
    float dgain[kGroups][N], dbias[kGroups][N], gain[kGroups][N];
    const int64_t stride = int64_t(blocks) * kTeams;
    int64_t first = int64_t(block) * kTeams;           // there are never more workgroups than rows for them
    NormRow<X, Y, kGroups> next;
    if (kAhead) get_norm_row<X, Y, kLanes, kEven>(a, min(first + team, int64_t(a.T) - 1), lane, next);
    const auto get_gain = [&](int g) {
        const int at = (g * kLanes + lane) * N, n = C - at;
#pragma unroll
        for (int i = 0; i < N; ++i) gain[g][i] = 1.0f;
        if (a.gain && n > 0) get_vector<N, kEven>(a.gain, a.w32, at, n, gain[g]);
    };
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
        for (int i = 0; i < N; ++i) dgain[g][i] = dbias[g][i] = 0.0f;
        if (kAhead) get_gain(g);
    }
    const float per = 1.0f / static_cast<float>(C);
    for (int turn = 0; first < a.T; first += stride, turn ^= 1) {
        const bool live = first + team < a.T;           // a team without a row stays for the barriers
        const int64_t row = live ? first + team : a.T - 1;
        if (!kAhead) get_norm_row<X, Y, kLanes, kEven>(a, row, lane, next);
        NormRow<X, Y, kGroups> r = next;
        join_row<X, N, kLanes, kEven>(lane, C, r.h, r.few_h);
        join_row<Y, N, kLanes, kEven>(lane, C, r.dy, r.few_dy);
        if (a.dh) join_row<X, N, kLanes, kEven>(lane, C, r.dh, r.few_dh);
        if (kAhead && first + stride < a.T)
            get_norm_row<X, Y, kLanes, kEven>(a, min(first + stride + team, int64_t(a.T) - 1), lane, next);
        float x[kGroups][N], d[kGroups][N];
        float along = 0.0f, flat = 0.0f;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            open<X, N>(r.h[g], x[g]);
            open<Y, N>(r.dy[g], d[g]);          // zeros behind the row's end
            if (!kAhead) get_gain(g);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                x[g][i] = (x[g][i] - r.mean) * r.rstd;
                if (kSums && live) {
                    dgain[g][i] = __builtin_fmaf(d[g][i], x[g][i], dgain[g][i]);
                    if (kSums > 1) dbias[g][i] += d[g][i];
                }
                d[g][i] *= gain[g][i];
                // (Rounded before it is added: in rows of few columns, where the terms of dx nearly cancel, equal products
                // then leave nothing.  Fused, dx is off by as much: 1.07e-7 of its size at 2 columns, this way 1.10e-7.)
                along += d[g][i] * x[g][i];
                flat += d[g][i];
            }
        }
        if constexpr (kLanes > 64) {        // both sums behind one barrier
            constexpr int kWaves = kLanes / 64;
            along = lanes_of<Sum, 64>(along);
            flat = lanes_of<Sum, 64>(flat);
            if ((threadIdx.x & 63) == 0) {
                red[turn][0][threadIdx.x >> 6] = along;
                red[turn][1][threadIdx.x >> 6] = flat;
            }
            __syncthreads();                // the other turn's places are read until the next one
            along = flat = 0.0f;
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                along += red[turn][0][team * kWaves + i];
                flat += red[turn][1][team * kWaves + i];
            }
        } else {
            along = lanes_of<Sum, kLanes>(along);
            flat = lanes_of<Sum, kLanes>(flat);
        }
        along *= per;
        flat = a.layer ? flat * per : 0.0f;
        xt *dx = static_cast<xt *>(a.dx) + row * a.ldx;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int at = (g * kLanes + lane) * N;
#pragma unroll
            for (int i = 0; i < N; ++i) d[g][i] = (d[g][i] - x[g][i] * along - flat) * r.rstd;
            if (a.dh) {
                float other[N];
                open<X, N>(r.dh[g], other);
#pragma unroll
                for (int i = 0; i < N; ++i) d[g][i] += other[i];
            }
            if (live) put_group<X, N, kPast, kEven>(dx + at, close<X, N>(d[g]), C - at);
        }
    }
    if constexpr (kSums > 0) {
#pragma unroll
        for (int n = kTeams / 2; n; n /= 2) {
            // teams n .. 2n - 1 hand theirs to teams 0 .. n - 1
            const int place = (team - n) * kSums * kWidth, own = team * kSums * kWidth;
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int at = (g * N + i) * kLanes + lane;      // of one lane's values apart: no bank conflicts
                    if (team >= n && team < 2 * n) {
                        total[place + at] = dgain[g][i];
                        if (kSums > 1) total[place + kWidth + at] = dbias[g][i];
                    }
                }
            __syncthreads();
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int at = (g * N + i) * kLanes + lane;
                    if (team < n) {
                        dgain[g][i] += total[own + at];
                        if (kSums > 1) dbias[g][i] += total[own + kWidth + at];
                    }
                }
            __syncthreads();
        }
        if (team) return;
        float *part = a.part + int64_t(block) * C;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int at = (g * kLanes + lane) * N;
            put_group<Fp32, N, false, kEven>(part + at, close<Fp32, N>(dgain[g]), C - at);
            if (kSums > 1) put_group<Fp32, N, false, kEven>(part + int64_t(blocks) * C + at, close<Fp32, N>(dbias[g]), C - at);
        }
    }
}

// Where the sums over the rows end up.
struct NormSums {
    const float *part;
    void *out[2];                 // dgain, dbias
    int32_t groups, C;
    bool g32, accumulate;
};

__device__ __forceinline__ void put_sum(const NormSums &s, int which, int c, float sum) {
    if (!s.out[which]) return;
    if (s.g32) {
        float *out = static_cast<float *>(s.out[which]) + c;
        *out = s.accumulate ? *out + sum : sum;
    } else {
        static_cast<uint16_t *>(s.out[which])[c] = Bf16::down(sum);
    }
}

constexpr int kPartColumns = 32;    // whole cache lines of partial sums

// The sum of a column over its shares, in a fixed order, in the first of its threads.
template <int kColumns>
__device__ __forceinline__ float columns_sum(float sum, float *s) {
    constexpr int kWaves = kRowThreads / 64;
    const int column = threadIdx.x % kColumns;
#pragma unroll
    for (int d = kColumns; d < 64; d *= 2) sum += __shfl_xor(sum, d);
    if (threadIdx.x % 64 < kColumns) s[threadIdx.x / 64 * kColumns + column] = sum;
    __syncthreads();
    sum = 0.0f;
    if (threadIdx.x < kColumns)
#pragma unroll
        for (int i = 0; i < kWaves; ++i) sum += s[i * kColumns + column];
    __syncthreads();
    return sum;
}

// The sums over few rows, of kColumns columns a workgroup: the statistics are
// there already, so they need not wait for the rows' own sums, and one launch
// does for both.
template <class X, class Y, int kColumns>
__device__ __forceinline__ void norm_columns(const NormBackward &a, const NormSums &s, uint32_t block) {
    __shared__ float places[kRowThreads / 64 * kColumns];
    const int c = block * kColumns + threadIdx.x % kColumns;
    float dgain = 0.0f, dbias = 0.0f;
    if (c < a.C) {
        const typename X::type *h = static_cast<const typename X::type *>(a.h) + c;
        const typename Y::type *dy = static_cast<const typename Y::type *>(a.dy) + c;
#pragma unroll 16
        for (int t = threadIdx.x / kColumns; t < a.T; t += kRowThreads / kColumns) {
            const float d = Y::up(dy[t * a.ldy]), x = X::up(h[t * a.ldh]);
            dgain = __builtin_fmaf(d, (x - (a.layer ? a.mean[t] : 0.0f)) * a.rstd[t], dgain);
            dbias += d;
        }
    }
    dgain = columns_sum<kColumns>(dgain, places);
    dbias = columns_sum<kColumns>(dbias, places);
    if (threadIdx.x >= kColumns || c >= a.C) return;
    put_sum(s, 0, c, dgain);
    put_sum(s, 1, c, dbias);
}

// Columns a workgroup takes beside rows of up to `width` values: of narrow rows
// fewer, as their columns make few workgroups (1024 x 128 in bf16: 8 columns 3.9
// us, 32 6.2; 1024 x 700: 16 6.1, 32 6.6, and in fp32 7.2 and 9.6; 1024 x 2048: 16
// 9.7, 32 9.0).
constexpr int few_columns(int width) { return width <= 256 ? 8 : width <= 1024 ? 16 : 32; }

template <class X, class Y, int kLanes, int kGroups, bool kEven, int kSums>
__global__ __launch_bounds__(kRowThreads) void k_norm_backward(const NormBackward a) {
    norm_rows<X, Y, kLanes, kGroups, kEven, kSums, true>(a, blockIdx.x, gridDim.x);
}

// Rows and columns in one launch, the columns' workgroups first.  Results stay in
// L2, as forward (192 x 4096 in bf16 with the product that reads them 29.0 us past
// it, 28.4 through it, 512 41.1 and 41.2; alone 5.0 and 5.0, 8.0 and 8.1).
template <class X, class Y, int kLanes, int kGroups, bool kEven>
__global__ __launch_bounds__(kRowThreads) void k_norm_backward_few(const NormBackward a, const NormSums s,
                                                                   uint32_t columns) {
    if (blockIdx.x < columns)
        norm_columns<X, Y, few_columns(kLanes * kGroups * X::kGroup)>(a, s, blockIdx.x);
    else
        norm_rows<X, Y, kLanes, kGroups, kEven, 0, false>(a, blockIdx.x - columns, gridDim.x - columns);
}

// The workgroups' sums in a fixed order.
__global__ __launch_bounds__(kRowThreads) void k_norm_reduce(const NormSums a) {
    __shared__ float places[kRowThreads / 64 * kPartColumns];
    const int c = blockIdx.x * kPartColumns + threadIdx.x % kPartColumns;
    float sum = 0.0f;
    if (c < a.C && a.out[blockIdx.y]) {
        const float *p = a.part + int64_t(blockIdx.y) * a.groups * a.C + c;
#pragma unroll 8
        for (int g = threadIdx.x / kPartColumns; g < a.groups; g += kRowThreads / kPartColumns) sum += p[int64_t(g) * a.C];
    }
    sum = columns_sum<kPartColumns>(sum, places);
    if (threadIdx.x < kPartColumns && c < a.C) put_sum(a, blockIdx.y, c, sum);
}

// ------------------------------------------------------------------ host
bool known(int32_t type) { return type == SFT_F32 || type == SFT_BF16; }

int check_sizes(int64_t T, int64_t C, const char *who) {
    SFT_CHECK(T >= 0 && C >= 0, SFT_EINVAL, "%s: negative size", who);
    SFT_CHECK(C > 0, SFT_ESHAPE, "%s: C = 0", who);
    SFT_CHECK(C <= kMaxWidth, SFT_ENOTSUP, "%s: C > %d", who, kMaxWidth);
    SFT_CHECK(T < (int64_t(1) << 31), SFT_ENOTSUP, "%s: T >= 2^31", who);
    return SFT_OK;
}

int check_types(int32_t kind, int32_t x, int32_t w, int32_t y, const char *who) {
    SFT_CHECK(kind == SFT_NORM_LAYER || kind == SFT_NORM_RMS, SFT_EINVAL, "%s: bad kind %d", who, kind);
    SFT_CHECK(known(x) && known(w) && known(y) && (y == x || y == SFT_BF16), SFT_EINVAL, "%s: bad type", who);
    return SFT_OK;
}

// One array of rows: its pointer, distance and alignment; *b is filled.
int check_rows(const void *p, int64_t T, int64_t C, int64_t ld, int32_t type, const char *who, const char *name,
               Block *b) {
    SFT_CHECK(ld >= C, SFT_ESHAPE, "%s: rows of %s are closer than C", who, name);
    SFT_CHECK(ld < (int64_t(1) << 40), SFT_ENOTSUP, "%s: rows of %s are 2^40 elements apart or more", who, name);
    SFT_CHECK(p || T == 0, SFT_EINVAL, "%s: %s is null", who, name);
    SFT_CHECK(aligned_to(p, type_bytes(type)), SFT_EALIGN, "%s: %s not aligned to its type", who, name);
    *b = rows_block(p, T, ld, C, type_bytes(type));
    SFT_CHECK(extent(*b) >= 0, SFT_ENOTSUP, "%s: %s spans 2^46 bytes or more", who, name);
    return SFT_OK;
}

int check_apart(const Block *written, int n_written, const Block *read, int n_read, const char *who) {
    for (int i = 0; i < n_written; ++i) {
        for (int j = 0; j < i; ++j)
            SFT_CHECK(apart(written[i], written[j]), SFT_EINVAL, "%s: two written arrays overlap", who);
        for (int j = 0; j < n_read; ++j)
            SFT_CHECK(apart(written[i], read[j]), SFT_EINVAL, "%s: a written array overlaps an input", who);
    }
    return SFT_OK;
}

// Lanes of a team and eights of elements of a lane, narrowest first.  Forward,
// 32 bytes a lane are best for either type: two eights in bf16 (with residual,
// 16.8M values of rows of 512, 2048: 21.4 us, one eight 23.3, four 22.4), one in
// fp32 (8.4M values of rows of 512, 4096: 12.9 and 13.5 us, two 13.9 and 15.8),
// until there are 512 lanes.  Narrow rows take several turns of 16 workgroups a
// CU, as starting one takes longer than its few rows (131072 x 128: 22.3 ->
// 21.5 us).
#define SFT_FORWARD_BF16(go) \
    go(8, 1) go(16, 1) go(16, 2) go(32, 2) go(64, 2) go(128, 2) go(256, 2) go(512, 2) go(512, 4)
#define SFT_FORWARD_FP32(go) \
    go(8, 1) go(16, 1) go(32, 1) go(64, 1) go(128, 1) go(256, 1) go(512, 1) go(512, 2) go(1024, 2)
#define SFT_BACKWARD_WIDTHS(go) \
    go(16, 1) go(32, 1) go(64, 1) go(128, 1) go(256, 1) go(512, 1) go(1024, 1) go(1024, 2)

template <class X, class Y, bool kEven, bool kPast>
void send_forward(const NormForward &a, hipStream_t st) {
#define SFT_GO(lanes, eights)                                                                                   \
    if (a.C <= lanes * eights * 8) {                                                                            \
        constexpr int kGroups = eights * 8 / X::kGroup;                                                         \
        constexpr int kThreads = lanes < 256 ? 256 : lanes, kTeams = kThreads / lanes;                          \
        const int64_t rounds = (int64_t(a.T) + kTeams - 1) / kTeams;                                            \
        const uint32_t grid = static_cast<uint32_t>(std::min<int64_t>(rounds, 16 * num_cus()));                 \
        hipLaunchKernelGGL((k_norm_forward<X, Y, lanes, kGroups, kEven, kPast>), dim3(grid), dim3(kThreads), 0, st, a); \
        return;                                                                                                 \
    }
    if constexpr (X::kType == SFT_BF16) {
        SFT_FORWARD_BF16(SFT_GO)
    } else {
        SFT_FORWARD_FP32(SFT_GO)
    }
#undef SFT_GO
}

// Results of up to 2 MB stay in L2 for the product that reads them next: of 4096
// columns in bf16 with residual, norm and product of 8 rows take 18.5 us past it
// and 16.3 through it, of 192 36.5 and 31.0, of 256 26.0 and 23.5, of 2048 77.8 and
// 78.8; the norm alone 3.6 and 3.6, 3.9 and 4.1, 4.1 and 4.2, 12.4 and 13.4.
template <class X, class Y>
void send_forward(const NormForward &a, hipStream_t st) {
    const bool past = int64_t(a.T) * a.C * int64_t(sizeof(typename Y::type)) > (1 << 21), even = a.C % X::kGroup == 0;
    if (past) {
        if (even) send_forward<X, Y, true, true>(a, st);
        else send_forward<X, Y, false, true>(a, st);
    } else {
        if (even) send_forward<X, Y, true, false>(a, st);
        else send_forward<X, Y, false, false>(a, st);
    }
}

int backward_teams(int64_t C) {
#define SFT_GO(lanes, eights) \
    if (C <= lanes * eights * 8) return kRowThreads / lanes;
    SFT_BACKWARD_WIDTHS(SFT_GO)
#undef SFT_GO
    return 1;
}

// Workgroups of the rows' part: one on each CU, as each writes partial sums that are read again.
int backward_groups(int64_t T, int64_t C) {
    const int64_t teams = backward_teams(C);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((T + teams - 1) / teams, num_cus())));
}

template <class X, class Y, bool kEven>
void send_backward(const NormBackward &a, const NormSums *few, int sums, hipStream_t st) {
    const uint32_t rows = static_cast<uint32_t>(backward_groups(a.T, a.C));
    const dim3 block(kRowThreads);
#define SFT_GO(lanes, eights)                                                                                           \
    if (a.C <= lanes * eights * 8) {                                                                                    \
        constexpr int kGroups = eights * 8 / X::kGroup, kColumns = few_columns(lanes * eights * 8);                     \
        const uint32_t columns = few ? static_cast<uint32_t>((a.C + kColumns - 1) / kColumns) : 0;                      \
        const dim3 grid(rows + columns);                                                                                \
        if (few) hipLaunchKernelGGL((k_norm_backward_few<X, Y, lanes, kGroups, kEven>), grid, block, 0, st, a, *few, columns); \
        else if (sums == 0) hipLaunchKernelGGL((k_norm_backward<X, Y, lanes, kGroups, kEven, 0>), grid, block, 0, st, a); \
        else if (sums == 1) hipLaunchKernelGGL((k_norm_backward<X, Y, lanes, kGroups, kEven, 1>), grid, block, 0, st, a); \
        else hipLaunchKernelGGL((k_norm_backward<X, Y, lanes, kGroups, kEven, 2>), grid, block, 0, st, a);                \
        return;                                                                                                         \
    }
    SFT_BACKWARD_WIDTHS(SFT_GO)
#undef SFT_GO
}

template <class X, class Y>
void send_backward(const NormBackward &a, const NormSums *few, int sums, hipStream_t st) {
    if (a.C % X::kGroup) send_backward<X, Y, false>(a, few, sums, st);
    else send_backward<X, Y, true>(a, few, sums, st);
}

size_t backward_bytes(int64_t T, int64_t C, bool with_bias) {
    return size_t(backward_groups(T, C)) * size_t(C) * sizeof(float) * (with_bias ? 2 : 1);
}

// Where the sums over the rows are taken by columns in the same launch, which
// reads two arrays again but saves a launch: bf16, 256 x 4096 5.7 us (with
// partial sums 8.3), 512 x 1375 4.8 (9.5), 1024 x 300 4.6 (8.9), 512 x 4096 7.2
// (8.7), 2048 x 128 5.1 (8.1), 4096 x 33 6.3 (8.6); but 1024 x 4096 14.1 (10.6),
// 2048 x 256 9.7 (7.9), 4096 x 95 13.1 (9.5), 8192 x 8 9.5 (8.1).
bool few_rows(int64_t T, int64_t C) { return (T <= 1024 && T * C <= (1 << 21)) || (T <= 4096 && T * C <= (1 << 18)); }

}  // namespace

extern "C" {

int sft_norm_forward(const sft_norm_args *v, void *stream) {
    const char *const who = "sft_norm_forward";
    clear_error();
    SFT_CHECK(v, SFT_EINVAL, "%s: args is null", who);
    if (int rc = check_sizes(v->T, v->C, who)) return rc;
    if (int rc = check_types(v->kind, v->x_type, v->w_type, v->y_type, who)) return rc;
    SFT_CHECK(v->eps >= 0.0f && std::isfinite(v->eps), SFT_EINVAL, "%s: eps is negative or not finite", who);
    SFT_CHECK(!v->res == !v->H, SFT_EINVAL, "%s: one of res and H is null", who);
    Block x, res{}, h{}, y;
    if (int rc = check_rows(v->X, v->T, v->C, v->ldx, v->x_type, who, "X", &x)) return rc;
    if (int rc = check_rows(v->Y, v->T, v->C, v->ldy, v->y_type, who, "Y", &y)) return rc;
    if (v->res) {
        if (int rc = check_rows(v->res, v->T, v->C, v->ldr, v->x_type, who, "res", &res)) return rc;
        if (int rc = check_rows(v->H, v->T, v->C, v->ldh, v->x_type, who, "H", &h)) return rc;
    }
    const int64_t w = type_bytes(v->w_type);
    SFT_CHECK(aligned_to(v->gain, w) && aligned_to(v->bias, w), SFT_EALIGN, "%s: gain or bias not aligned to its type",
              who);
    SFT_CHECK(aligned_to(v->mean, 4) && aligned_to(v->rstd, 4), SFT_EALIGN, "%s: mean or rstd not 4-byte aligned", who);
    if (v->T == 0) return SFT_OK;
    const Block gain = flat_block(v->gain, v->C * w), bias = flat_block(v->bias, v->C * w);
    const Block mean = flat_block(v->mean, v->T * 4), rstd = flat_block(v->rstd, v->T * 4);
    {
        // H in the place of X or res: every lane has read what it writes there
        Block read[4];
        int n = 0;
        if (!same(h, x)) read[n++] = x;
        if (!same(h, res)) read[n++] = res;
        read[n++] = gain;
        read[n++] = bias;
        if (int rc = check_apart(&h, 1, read, n, who)) return rc;
        const Block written[] = {y, mean, rstd}, all[] = {x, res, h, gain, bias};
        if (int rc = check_apart(written, 3, all, 5, who)) return rc;
    }
    NormForward a{};
    a.x = v->X, a.res = v->res, a.h = v->H, a.gain = v->gain, a.bias = v->bias, a.y = v->Y;
    a.mean = v->mean, a.rstd = v->rstd;
    a.ldx = v->ldx, a.ldr = v->ldr, a.ldh = v->ldh, a.ldy = v->ldy;
    a.T = static_cast<int32_t>(v->T), a.C = static_cast<int32_t>(v->C);
    a.eps = v->eps;
    a.layer = v->kind == SFT_NORM_LAYER;
    a.w32 = v->w_type == SFT_F32;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (v->x_type == SFT_BF16)
        send_forward<Bf16, Bf16>(a, st);
    else if (v->y_type == SFT_BF16)
        send_forward<Fp32, Bf16>(a, st);
    else
        send_forward<Fp32, Fp32>(a, st);
    const hipError_t e = hipGetLastError();
    SFT_CHECK(e == hipSuccess, SFT_EHIP, "%s: launch failed: %s", who, hipGetErrorString(e));
    return SFT_OK;
}

size_t sft_norm_backward_workspace(int64_t T, int64_t C, int32_t with_bias) {
    clear_error();
    if (check_sizes(T, C, "sft_norm_backward_workspace")) return static_cast<size_t>(-1);
    return T ? backward_bytes(T, C, with_bias) : 0;
}

int sft_norm_backward(const sft_norm_grad_args *v, void *ws, size_t ws_bytes, void *stream) {
    const char *const who = "sft_norm_backward";
    clear_error();
    SFT_CHECK(v, SFT_EINVAL, "%s: args is null", who);
    if (int rc = check_sizes(v->T, v->C, who)) return rc;
    if (int rc = check_types(v->kind, v->x_type, v->w_type, v->y_type, who)) return rc;
    SFT_CHECK(known(v->g_type), SFT_EINVAL, "%s: bad type", who);
    SFT_CHECK(!v->accumulate || v->g_type == SFT_F32, SFT_EINVAL, "%s: accumulate asks for fp32 gradients", who);
    const bool layer = v->kind == SFT_NORM_LAYER, sums = v->dgain || v->dbias;
    SFT_CHECK(v->T == 0 || (v->rstd && (v->mean || !layer)), SFT_EINVAL, "%s: mean or rstd is null", who);
    Block h, dy, dh{}, dx;
    if (int rc = check_rows(v->H, v->T, v->C, v->ldh, v->x_type, who, "H", &h)) return rc;
    if (int rc = check_rows(v->dY, v->T, v->C, v->ldy, v->y_type, who, "dY", &dy)) return rc;
    if (int rc = check_rows(v->dX, v->T, v->C, v->ldx, v->x_type, who, "dX", &dx)) return rc;
    if (v->dH)
        if (int rc = check_rows(v->dH, v->T, v->C, v->ldr, v->x_type, who, "dH", &dh)) return rc;
    const int64_t w = type_bytes(v->w_type), gs = type_bytes(v->g_type);
    SFT_CHECK(aligned_to(v->gain, w), SFT_EALIGN, "%s: gain not aligned to its type", who);
    SFT_CHECK(aligned_to(v->mean, 4) && aligned_to(v->rstd, 4), SFT_EALIGN, "%s: mean or rstd not 4-byte aligned", who);
    SFT_CHECK(aligned_to(v->dgain, gs) && aligned_to(v->dbias, gs), SFT_EALIGN,
              "%s: dgain or dbias not aligned to its type", who);
    const size_t need = sums && v->T ? backward_bytes(v->T, v->C, v->dbias != nullptr) : 0;
    SFT_CHECK(ws_bytes >= need, SFT_ECAPACITY, "%s: workspace %zu < %zu bytes", who, ws_bytes, need);
    SFT_CHECK(need == 0 || ws, SFT_EINVAL, "%s: workspace is null", who);
    SFT_CHECK(aligned16(ws), SFT_EALIGN, "%s: workspace not 16-byte aligned", who);
    {
        const Block gain = flat_block(v->gain, v->C * w), mean = flat_block(layer ? v->mean : nullptr, v->T * 4);
        const Block rstd = flat_block(v->rstd, v->T * 4);
        const Block written[] = {flat_block(v->dgain, v->C * gs), flat_block(v->dbias, v->C * gs),
                                 flat_block(need ? ws : nullptr, static_cast<int64_t>(need))};
        const Block all[] = {h, dy, dh, dx, gain, mean, rstd};
        if (int rc = check_apart(written, 3, all, 7, who)) return rc;
        // dX in the place of dY or dH: every lane has read what it writes there
        Block read[6] = {h, gain, mean, rstd};
        int n = 4;
        if (!same(dx, dy)) read[n++] = dy;
        if (!same(dx, dh)) read[n++] = dh;
        if (int rc = check_apart(&dx, 1, read, n, who)) return rc;
    }
    const hipStream_t st = static_cast<hipStream_t>(stream);
    NormSums s{};
    s.part = static_cast<const float *>(ws);
    s.out[0] = v->dgain, s.out[1] = v->dbias;
    s.groups = v->T ? backward_groups(v->T, v->C) : 0, s.C = static_cast<int32_t>(v->C);
    s.g32 = v->g_type == SFT_F32, s.accumulate = v->accumulate != 0;
    // (dX in dY's place is written while other workgroups would still read dY for the columns)
    const bool few = sums && v->T > 0 && few_rows(v->T, v->C) && !same(dx, dy);
    if (v->T) {
        NormBackward a{};
        a.h = v->H, a.gain = v->gain, a.mean = v->mean, a.rstd = v->rstd, a.dy = v->dY, a.dh = v->dH, a.dx = v->dX;
        a.part = static_cast<float *>(ws);
        a.ldh = v->ldh, a.ldy = v->ldy, a.ldr = v->ldr, a.ldx = v->ldx;
        a.T = static_cast<int32_t>(v->T), a.C = s.C;
        a.layer = layer;
        a.w32 = v->w_type == SFT_F32;
        const int kind = !sums ? 0 : v->dbias ? 2 : 1;
        if (v->x_type == SFT_BF16)
            send_backward<Bf16, Bf16>(a, few ? &s : nullptr, kind, st);
        else if (v->y_type == SFT_BF16)
            send_backward<Fp32, Bf16>(a, few ? &s : nullptr, kind, st);
        else
            send_backward<Fp32, Fp32>(a, few ? &s : nullptr, kind, st);
        const hipError_t e = hipGetLastError();
        SFT_CHECK(e == hipSuccess, SFT_EHIP, "%s: launch failed: %s", who, hipGetErrorString(e));
    }
    if (sums && !few) {
        const dim3 grid(static_cast<uint32_t>((v->C + kPartColumns - 1) / kPartColumns), v->dbias ? 2 : 1);
        hipLaunchKernelGGL(k_norm_reduce, grid, dim3(kRowThreads), 0, st, s);
        const hipError_t e = hipGetLastError();
        SFT_CHECK(e == hipSuccess, SFT_EHIP, "%s: launch failed: %s", who, hipGetErrorString(e));
    }
    return SFT_OK;
}

}  // extern "C"
