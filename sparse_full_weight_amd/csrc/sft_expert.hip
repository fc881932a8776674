// sft_expert.hip -- matrix products grouped by expert, with ragged groups:
// tokens sorted by expert, rows first[e] .. first[e+1] of the token arrays
// belong to expert e, whose weight W_e is [R x C] (rows = output features).
//
//   forward          Y[t, r]    = sum_c X[t, c] W_e[r, c]
//   input gradient   dX[t, c]   = sum_r dY[t, r] W_e[r, c]
//   weight gradient  dW_e[r, c] = sum_t dY[t, r] X[t, c]
//
// One tiled product serves all three: out[m][n] = sum_k A[m][k] B[n][k].
//   forward          m = token, n = r, k = c: both operands have k contiguous
//   input gradient   m = token, n = c, k = r: B = W_e has n contiguous
//   weight gradient  m = r, n = c, k = token: both have m or n contiguous
// An operand with k contiguous is read from LDS 16 bytes a lane; one with the
// other axis contiguous goes to LDS as it lies in memory and is read by the
// transposing LDS loads (ds_read_b64_tr_b16), so no operand is ever laid out
// again in memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "sft_internal.h"
#include "sft_probe.h"

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;                 // 2 x 2 waves
constexpr uint32_t kOutside = 0x80000000u;    // an offset beyond every buffer's size: reads as zero
constexpr int kGroupM = 8;                    // m-tiles that are walked together along n

enum Op { kForward = 0, kDx = 1, kDw = 2 };

struct ExpertParams {
    const uint16_t *a, *b;
    void *out;
    const int32_t *first;
    int64_t T, R, C;
    int32_t E;
    int32_t chunk;          // consecutive units that one XCD takes
    int32_t cus;            // compute units: a launch that ends in a short round cuts its tiles in half
};

// s_waitcnt vmcnt(n) alone, and lgkmcnt(0) alone (gfx9 encoding).
#define SFT_WAIT_VMCNT(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | (((n) >> 4) << 14) | 0x0F70)
#define SFT_WAIT_LGKM0() __builtin_amdgcn_s_waitcnt(0xC07F)

template <int V>
using ic = std::integral_constant<int, V>;

__device__ __forceinline__ int32_t uniform(int32_t x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ uint64_t uniform64(uint64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x >> 32));
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// ------------------------------------------------------------------ tiles
// One output tile of an expert's product: its token rows [lo, lo + n), the
// tile's position, and which half of its columns (-1: all).
struct Tile {
    int32_t e, lo, n, mt, nt, half;
};

// Expert e's rows, whatever first[] holds: inside [0, T], never negative.
__device__ __forceinline__ int2 rows_of(const ExpertParams &p, int32_t e) {
    const int32_t T = static_cast<int32_t>(p.T);
    const int32_t lo = min(max(p.first[e], 0), T);
    return int2{lo, min(max(p.first[e + 1], lo), T) - lo};
}

// Workgroups are dealt to the 8 XCDs in turn; an XCD takes runs of `chunk`
// neighbouring units, which share operand panels in its L2.
__device__ __forceinline__ int32_t unit_index(const ExpertParams &p) {
    const int32_t b = blockIdx.x, x = b & 7, i = b >> 3;
    return ((i / p.chunk) * 8 + x) * p.chunk + i % p.chunk;
}

// Unit u of a launch of `tiles` tiles: whole tiles, and where the last round
// of workgroups would fill half of the CUs or less, that round's tiles as two
// halves along n (forward of 8 x 11008 x 4096 at 8192 tokens, 6.05 rounds: 692
// us, with whole tiles to the end 705).
__device__ __forceinline__ int32_t tile_of_unit(const ExpertParams &p, int32_t u, int32_t tiles, int32_t &half) {
    const int32_t last = tiles % p.cus, whole = tiles - (2 * last <= p.cus ? last : 0);
    half = u < whole ? -1 : (u - whole) & 1;
    return u < whole ? u : whole + ((u - whole) >> 1);
}

// Tiles of an expert in walking order: groups of kGroupM m-tiles, n outside,
// m inside, so that the tiles of a run share a few panels of both operands.
__device__ __forceinline__ void place(Tile &t, int32_t i, int32_t m_tiles, int32_t n_tiles) {
    const int32_t g = i / (kGroupM * n_tiles), r = i - g * kGroupM * n_tiles;
    const int32_t gm = min(kGroupM, m_tiles - g * kGroupM);
    t.nt = r / gm;
    t.mt = g * kGroupM + (r - t.nt * gm);
}

// Sum over the lanes up to each lane's own, without going through LDS.
__device__ __forceinline__ int32_t running_sum(int32_t x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);    // within 16 lanes: from 1, 2, 4, 8 lanes below
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // lane 15 to the next 16, 47 to the last
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);   // lane 31 to the upper half
    return x;
}

// The tile of this workgroup, or false where there is none: the host only
// knows how many tiles there can be at most.  64 experts at a time, a lane
// each: their tile counts, and the running sum whose range holds the index.
template <int BM, bool kHalves>
__device__ __forceinline__ bool token_tile(const ExpertParams &p, int32_t n_tiles, Tile &t) {
    const int32_t u = unit_index(p), lane = threadIdx.x & 63;
    int32_t v = u;
    t.half = -1;
    if constexpr (kHalves) {
        int32_t tiles = 0;
        for (int32_t e0 = 0; e0 < p.E; e0 += 64)
            tiles += e0 + lane < p.E ? (rows_of(p, e0 + lane).y + BM - 1) / BM : 0;
        v = tile_of_unit(p, u, __builtin_amdgcn_readlane(running_sum(tiles), 63) * n_tiles, t.half);
    }
    int32_t before = 0;
    for (int32_t e0 = 0; e0 < p.E; e0 += 64) {
        const int32_t e = e0 + lane;
        const int2 r = e < p.E ? rows_of(p, e) : int2{0, 0};
        const int32_t m_tiles = (r.y + BM - 1) / BM;
        const int32_t end = before + running_sum(m_tiles) * n_tiles;
        const uint64_t past = __ballot(v < end);
        if (past) {
            const int at = uniform(__builtin_ctzll(past));
            t.e = e0 + at;
            t.lo = __builtin_amdgcn_readlane(r.x, at);
            t.n = __builtin_amdgcn_readlane(r.y, at);
            const int32_t mt = __builtin_amdgcn_readlane(m_tiles, at);
            const int32_t i = v - (__builtin_amdgcn_readlane(end, at) - mt * n_tiles);
            if (i < 0 || i >= mt * n_tiles) return false;   // first[] does not ascend and the sums ran over
            place(t, i, mt, n_tiles);
            return true;
        }
        before = __builtin_amdgcn_readlane(end, 63);
    }
    return false;
}

// ------------------------------------------------------------------ operands
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) bf16x8 lds_bf16x8;
typedef __attribute__((address_space(3))) short4v lds_short4v;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;

__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, lds_u8 *lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)(lds), 16, voff, 0, 0, 0);
}

// One operand of a tile: how its stages of kBK k-values get into LDS and how
// a wave reads matrix fragments from there.  W: rows (m or n) of the tile.  A
// stage is copied by pieces of 1 KB, 16 bytes a lane, of which a wave takes
// every NW-th.
//
// kTr false (k contiguous): LDS row = one m, kBK values in groups of 16 bytes,
// each group in slot g ^ (row/2 % 8), or g ^ (row/4 % 4) of the shorter rows,
// so that 16 lanes reading one group of 16 rows hit all 64 banks.  kTr true (m
// contiguous): LDS row = one k, 2W bytes; a transposing read takes, by 32
// lanes, 64 bytes of four rows: group g sits in slot g ^ 4*(row % 4) where
// rows are whole multiples of 256 bytes, and in g ^ 4*(row/2 % 2) where every
// second row starts 128 bytes on, so that these hit all banks too.
template <bool kTr, int W, int kBK>
struct Operand {
    static constexpr int NW = kThreads / 64;
    static constexpr int kBytes = W * kBK * 2;
    static constexpr int kLoads = kBytes / 1024 / NW;
    static_assert(kLoads * 1024 * NW == kBytes, "a stage is its waves' pieces");
    static constexpr int kShift = kBK == 32 ? 2 : 1;
    static __device__ __forceinline__ int turn(int row) {
        if constexpr (!kTr) return row >> kShift & (kBK / 8 - 1);
        else return W % 128 ? 4 * (row >> 1 & 1) : 4 * (row & 3);
    }
    static constexpr int kRowLanes = kTr ? W / 8 : kBK / 8;     // groups of 16 bytes in an LDS row

    const uint8_t *base;      // of the next stage's first byte (wave-uniform)
    int64_t left;             // bytes from there to the end of what is valid
    int64_t step;             // bytes from one stage to the next
    uint32_t voff[kLoads];
    int32_t from[kTr ? 4 : 1];
    int32_t kgrp;             // k of the lane's 16 bytes inside a stage (k contiguous)

    // mem: first row of the tile (k contiguous) or first column (m contiguous)
    // in an array of `ld` elements a row; `valid` rows of memory are there
    // (tile rows or k), `cols` columns from the tile's first on (m contiguous).
    __device__ __forceinline__ void describe(const uint16_t *mem, int64_t ld, int64_t valid, int64_t cols) {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        base = reinterpret_cast<const uint8_t *>(uniform64(reinterpret_cast<uint64_t>(mem)));
        left = static_cast<int64_t>(uniform64(static_cast<uint64_t>(
            kTr ? (valid > 0 ? ((valid - 1) * ld + cols) * 2 : 0) : valid * ld * 2)));
        step = static_cast<int64_t>(uniform64(static_cast<uint64_t>(kTr ? kBK * ld * 2 : kBK * 2)));
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            const int at = 64 * (wave + NW * k) + lane, row = at / kRowLanes, grp = at % kRowLanes ^ turn(row);
            if constexpr (kTr) {
                voff[k] = 8 * grp < cols ? static_cast<uint32_t>((row * ld + 8 * grp) * 2) : kOutside;
            } else {
                voff[k] = row < valid ? static_cast<uint32_t>((row * ld + 8 * grp) * 2) : kOutside;
                kgrp = 8 * grp;   // the turn is the same for every piece of the lane
            }
        }
    }

    // Copies the next stage; k_left = valid k-values from it on.
    __device__ __forceinline__ void issue(lds_u8 *lds, int32_t k_left) {
        const int wave = uniform(threadIdx.x >> 6);
        const int32_t size = static_cast<int32_t>(left <= 0 ? 0 : left > 0x7fffffff ? 0x7fffffff : left);
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base),
                                                                           static_cast<short>(0), size, 0x00020000);
        const bool cut = !kTr && k_left < kBK;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
            uint32_t v = voff[k];
            if (cut) v = kgrp < k_left ? v : kOutside;
            dma16(r, v, lds + 1024 * (wave + NW * k));
        }
        base += step;
        left -= step;
    }

    // Where a wave reads its part of the tile, `at` = its first row.  The
    // empty asm keeps the compiler from taking the offset apart again: behind
    // a chain of pointer sums it loses track of which stage a read is from,
    // and waits for every copy in flight.
    __device__ __forceinline__ void read_from(int at) {
        const int lane = threadIdx.x & 63;
        if constexpr (kTr) {
            const int s = lane & 15, col = ((lane >> 4) & 1) * 16 + 4 * (s & 3);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int grp = (at + 32 * i) / 8 + (col >> 3);
                from[i] = (8 * (lane >> 5) + (s >> 2)) * (2 * W) + 16 * (grp ^ turn(s >> 2)) + 2 * (col & 7);
                asm volatile("" : "+v"(from[i]));
            }
        } else {
            from[0] = at + (lane & 31);
        }
    }

    // Fragments: 32 rows (m) of matrix step kk; lane l holds row l % 32,
    // k = 8 * (l / 32) + 0..7.
    template <int F>
    __device__ __forceinline__ void read(lds_u8 *lds, int kk, bf16x8 (&f)[F]) const {
        const int lane = threadIdx.x & 63;
        if constexpr (kTr) {
#pragma unroll
            for (int i = 0; i < F; ++i) {
                lds_u8 *q = lds + from[i];
                const short4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4v *)(q + 16 * kk * 2 * W));
                const short4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4v *)(q + (16 * kk + 4) * 2 * W));
                f[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
        } else {
            const int row = from[0];
#pragma unroll
            for (int i = 0; i < F; ++i)
                f[i] = *(lds_bf16x8 *)(lds + ((row + 32 * i) * (2 * kBK) + 16 * ((2 * kk + (lane >> 5)) ^ turn(lane))));
        }
    }
};

// The stages of each operand, as LDS variables of their own so that the
// compiler can tell copies into one from reads of the other; W: rows of the
// largest tile of the kernel.
template <int kBytes, int kOperand, int S>
__device__ __forceinline__ lds_u8 *stage() {
    __shared__ __attribute__((aligned(1024))) uint8_t m[kBytes];
    return (lds_u8 *)m;
}

// ------------------------------------------------------------------ the product
// Two values rounded to bf16, nearest even.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{static_cast<__bf16>(a), static_cast<__bf16>(b)});
}

// kStream: past L2.
template <bool kStream, class V>
__device__ __forceinline__ void put(V *p, V v) {
    if constexpr (kStream) __builtin_nontemporal_store(v, p);
    else *p = v;
}

constexpr int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// A kernel's tiles: kM x kN, by stages of kBK along k, kStages of them in LDS;
// per_cu workgroups share a CU.
constexpr int per_cu(int m, int n, int k, int stages) {
    const int fit = 160 * 1024 / ((m + n) * k * 2 * stages);
    return fit < 4 ? fit : 4;
}
template <int M_, int N_, int BK_, int STAGES_>
struct Shape {
    static constexpr int kM = M_, kN = N_, kBK = BK_, kStages = STAGES_;
    static constexpr int kPerCu = per_cu(kM, kN, kBK, kStages);
};
// The same as values.
struct ShapeOf {
    int m, n, k, stages;
    int per_cu() const { return ::per_cu(m, n, k, stages); }
    bool operator==(const ShapeOf &o) const { return m == o.m && n == o.n && k == o.k && stages == o.stages; }
    template <class S>
    static ShapeOf of() {
        return {S::kM, S::kN, S::kBK, S::kStages};
    }
};

// BM x BN from (m0, n0) on of expert t.e's product, by 2 x 2 waves, each
// (BM/2) x (BN/2) in blocks of 32 x 32.
template <int kOp, class S, int BM, int BN, class Out, bool kAdd>
__device__ __forceinline__ void multiply_part(const ExpertParams &p, const Tile &t, int64_t m0, int64_t n0) {
    constexpr int FM = BM / 64, FN = BN / 64, kBK = S::kBK, kStages = S::kStages, KK = kBK / 16;
    constexpr int SA = S::kM * kBK * 2, SB = S::kN * kBK * 2;
    typedef Operand<kOp == kDw, BM, kBK> A;
    typedef Operand<kOp != kForward, BN, kBK> B;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t N = kOp == kForward ? p.R : p.C;
    const int64_t K = kOp == kForward ? p.C : kOp == kDx ? p.R : t.n;
    const int64_t M = kOp == kDw ? p.R : t.n;

    A a;
    B b;
    if constexpr (kOp == kDw) {
        a.describe(p.a + t.lo * p.R + m0, p.R, K, p.R - m0);
        b.describe(p.b + t.lo * p.C + n0, p.C, K, p.C - n0);
    } else {
        a.describe(p.a + (t.lo + m0) * K, K, min(M - m0, static_cast<int64_t>(BM)), 0);
        const uint16_t *W = p.b + static_cast<int64_t>(t.e) * p.R * p.C;
        if constexpr (kOp == kForward)
            b.describe(W + n0 * K, K, min(N - n0, static_cast<int64_t>(BN)), 0);
        else
            b.describe(W + n0, p.C, K, p.C - n0);
    }

    floatx16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    const int am = (wave >> 1) * (BM / 2), bn = (wave & 1) * (BN / 2);
    a.read_from(am);
    b.read_from(bn);
    const int32_t k32 = static_cast<int32_t>(K), KT = (k32 + kBK - 1) / kBK;
    auto issue = [&](auto s, int32_t kt) __attribute__((always_inline)) {
        constexpr int I = decltype(s)::value;
        a.issue(stage<SA, 0, I>(), k32 - kt * kBK);
        b.issue(stage<SB, 1, I>(), k32 - kt * kBK);
    };
    auto read = [&](auto s, int kk, bf16x8 (&fa)[FM], bf16x8 (&fb)[FN]) __attribute__((always_inline)) {
        constexpr int I = decltype(s)::value;
        a.read(stage<SA, 0, I>(), kk, fa);
        b.read(stage<SB, 1, I>(), kk, fb);
    };
    auto multiply = [&](const bf16x8 (&fa)[FM], const bf16x8 (&fb)[FN]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
    };
    // The fragments of a matrix step are read while the step before is
    // multiplied, across stages too: a stage's last step needs nothing from
    // LDS, so the wait for the next stage and the barrier stand before it.
    // Behind the barrier every wave has read this stage whole, and the copies
    // of the stage kStages ahead go into its place.  Stages past K are copied
    // as zeros from an empty buffer, so every wave has the same copies in
    // flight at every wait.  The compiler would sink each read to its use:
    // the groups below spread reads and copies evenly between the products
    // (forward at 256 x 256: 742 us, 885 us as the compiler orders them).
    constexpr int kReads = FM * (kOp == kDw ? 2 : 1) + FN * (kOp == kForward ? 1 : 2), kMul = FM * FN;
    constexpr int kGroups = gcd(kReads, kMul), kCopies = (A::kLoads + B::kLoads + kGroups - 1) / kGroups;
    auto weave = [&](auto copies) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x100, kReads / kGroups, 0);                        // LDS reads
            if constexpr (decltype(copies)::value) __builtin_amdgcn_sched_group_barrier(0x020, kCopies, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, kMul / kGroups, 0);                          // MFMA
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int kInFlight = (kStages - 2) * (A::kLoads + B::kLoads);
    bf16x8 fa[2][FM], fb[2][FN];
    auto use = [&](auto s, int32_t kt) __attribute__((always_inline)) {
        constexpr int I = decltype(s)::value;
#pragma unroll
        for (int kk = 0; kk + 1 < KK; ++kk) {
            read(s, kk + 1, fa[(kk + 1) & 1], fb[(kk + 1) & 1]);
            multiply(fa[kk & 1], fb[kk & 1]);
            weave(ic<0>{});
        }
        SFT_WAIT_LGKM0();
        SFT_WAIT_VMCNT(kInFlight);
        __builtin_amdgcn_s_barrier();
        issue(s, kt + kStages);
        read(ic<(I + 1) % kStages>{}, 0, fa[0], fb[0]);
        multiply(fa[1], fb[1]);
        weave(ic<1>{});
    };
    auto each = [&](auto f) __attribute__((always_inline)) {
        f(ic<0>{});
        f(ic<1>{});
        if constexpr (kStages > 2) f(ic<2>{});
        if constexpr (kStages > 3) f(ic<3>{});
        if constexpr (kStages > 4) f(ic<4>{});
    };
    static_assert(kStages >= 2 && kStages <= 5 && KK % 2 == 0, "stages");
    // The loop takes kStages stages a turn; the KT % kStages stages that do not
    // fill a turn come first, by code of their own for each such number: the
    // first stage then sits in LDS where the loop's first turn will find its
    // own (the weight gradient of 64 experts with 64 rows each 160 -> 151 us).
    // Not for turns of two, nor for the largest tiles, whose sums are long:
    // there the loop takes stages of zeros.
    auto start = [&](auto first) __attribute__((always_inline)) {
        constexpr int I0 = decltype(first)::value;
        each([&](auto j) __attribute__((always_inline)) {
            constexpr int J = decltype(j)::value;
            issue(ic<(I0 + J) % kStages>{}, J);
        });
        SFT_WAIT_VMCNT((kStages - 1) * (A::kLoads + B::kLoads));
        __builtin_amdgcn_s_barrier();
        read(first, 0, fa[0], fb[0]);
        each([&](auto s) __attribute__((always_inline)) {
            constexpr int I = decltype(s)::value;
            if constexpr (I0 > 0 && I >= I0) use(s, I - I0);
        });
    };
    if (KT > 0) {
        constexpr bool kOdd = kStages > 2 && BM * BN <= 128 * 256;
        const int32_t odd = kOdd ? KT % kStages : 0;
        if constexpr (kOdd && kStages > 4) {
            if (odd == 4) start(ic<kStages - 4>{});
        }
        if constexpr (kOdd && kStages > 3) {
            if (odd == 3) start(ic<kStages - 3>{});
        }
        if constexpr (kOdd) {
            if (odd == 1) start(ic<kStages - 1>{});
            if (odd == 2) start(ic<kStages - 2>{});
        }
        if (odd == 0) start(ic<0>{});
        for (int32_t kt = odd; kt < KT; kt += kStages)
            each([&](auto s) __attribute__((always_inline)) { use(s, kt + decltype(s)::value); });
    }
    // Behind this every copy has landed and every wave has read its last
    // stage: LDS is free for the results.
    SFT_WAIT_VMCNT(0);
    __builtin_amdgcn_s_barrier();

    // Lane l holds, for row l % 32 of block (i, j), the columns
    // 8*(r/4) + 4*(l/32) + r%4 of register r: four neighbours a register quad.
    // A wave turns 32 rows of 128 bytes (one block of fp32, two of bf16, whose
    // halves of the wave first trade quads for eight neighbours a lane) at a
    // time through its own 4 KB of LDS, and stores whole cache lines: 16-byte
    // group c of row r sits in slot c ^ (r % 8) ^ (r/8 % 2), so that neither 16
    // rows of one group, nor 8 rows of two, nor a row's 8 collide on a bank.
    // Weight gradient of 8 x 11008 x 4096 at 8192 tokens, fp32: stored straight
    // from the registers, 32 bytes a row, 871 us; so 834; and past L2 803
    // (64 x 1376 x 4096 at 4099 tokens, bf16: 226, 211, 158).
    // The old values that a sum goes on from are read a block ahead where rows
    // start on cache lines (64 x 1376 x 4096: 676 -> 530 us), else just before
    // they are written (rows of 16416 bytes: 992 us ahead, 782 so).
    constexpr bool kF32 = std::is_same<Out, float>::value;
    constexpr int kJ = kF32 ? 1 : 2, kLane = kF32 ? 4 : 8;    // blocks at a time, values in 16 bytes
    static_assert(SA >= 8192 && SB >= 8192, "4 KB for each of 4 waves");
    lds_u8 *turn = (wave & 2 ? stage<SB, 1, 0>() : stage<SA, 0, 0>()) + 4096 * (wave & 1);
    Out *out = static_cast<Out *>(p.out) +
               (kOp == kDw ? static_cast<int64_t>(t.e) * p.R * p.C : static_cast<int64_t>(t.lo) * N);
    const int half = lane >> 5, row = lane & 31;
    static_assert(!kAdd || kF32, "sums go on in fp32");
    f32x4 old[2][4];
    auto read_old = [&](int block) __attribute__((always_inline)) {
        const int64_t n = n0 + bn + 32 * (block % FN) + 4 * (lane & 7);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t m = m0 + am + 32 * (block / FN) + 8 * k + (lane >> 3);
            if (m < M && n < N) old[block & 1][k] = *reinterpret_cast<const f32x4 *>(out + m * N + n);
        }
    };
    auto results = [&](auto past) __attribute__((always_inline)) {
        constexpr bool kAhead = kAdd && decltype(past)::value != 0;
        if constexpr (kAhead) read_old(0);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
#pragma unroll
            for (int j = 0; j < FN; j += kJ) {
                const int groups = (FN - j < kJ ? FN - j : kJ) * (32 / kLane);     // of 16 bytes in a row: 8, or 4
                auto slot = [&](int r, int c) __attribute__((always_inline)) {
                    return (lds_u32x4 *)(turn + (128 * r + 16 * (c ^ (r & 7) ^ (r >> 3 & 1))));
                };
#pragma unroll
                for (int b = j; b < j + kJ && b < FN; ++b) {
                    const floatx16 &x = acc[i][b];
                    if constexpr (kF32) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *slot(row, 2 * q + half) = __builtin_bit_cast(
                                u32x4, f32x4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]});
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; q += 2) {
                            uint32_t w[4];
#pragma unroll
                            for (int c = 0; c < 4; ++c) w[c] = pack2(x[4 * q + 2 * c], x[4 * q + 2 * c + 1]);
                            const auto lo = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
                            const auto hi = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
                            *slot(row, 4 * (b - j) + q + half) = u32x4{lo[0], hi[0], lo[1], hi[1]};
                        }
                    }
                }
                if constexpr (kAhead) {
                    if (i * FN + j + 1 < FM * FN) read_old(i * FN + j + 1);
                }
                const int rows = 64 / groups, c = lane % groups;                   // of one store
                const int64_t n = n0 + bn + 32 * j + kLane * c;
#pragma unroll
                for (int r0 = 0; r0 < 32; r0 += rows) {
                    const int r = r0 + lane / groups;
                    const int64_t m = m0 + am + 32 * i + r;
                    u32x4 v = *slot(r, c);
                    if (m < M && n < N) {
                        u32x4 *o = reinterpret_cast<u32x4 *>(out + m * N + n);
                        if constexpr (kAdd) {
                            f32x4 w;
                            if constexpr (kAhead)
                                w = old[(i * FN + j) & 1][r0 / 8];
                            else
                                w = *reinterpret_cast<const f32x4 *>(o);
                            v = __builtin_bit_cast(u32x4, w + __builtin_bit_cast(f32x4, v));
                        }
                        put<decltype(past)::value != 0>(o, v);
                    }
                }
            }
        }
    };
    // Weight gradients are written past L2: they are larger than every cache
    // and would push the operands out.  Only whole lines, though: where rows
    // do not start on one, L2 has to join the pieces (1.1 GB of zeros in rows
    // of 8416 bytes: 580 us past L2, 326 through it).
    if constexpr (kOp == kDw) {
        if ((N * sizeof(Out)) % 128 == 0 && reinterpret_cast<uintptr_t>(p.out) % 128 == 0) {
            results(ic<1>{});
            asm volatile("; past L2");   // or the ends of both versions become one, through L2
            return;
        }
    }
    results(ic<0>{});
}

// The weight gradient of an expert without rows: zeros, in whole lines
// whatever the rows' length; part i of `parts` (1.1 GB of rows of 8416 bytes
// 323 us by tiles, 202 so).
template <class Out>
__device__ __forceinline__ void zero_part(const ExpertParams &p, int32_t e, int32_t i, int32_t parts) {
    const int64_t groups = p.R * p.C * static_cast<int64_t>(sizeof(Out)) / 16;
    const int64_t each = ((groups + parts - 1) / parts + kThreads - 1) / kThreads * kThreads;
    u32x4 *o = reinterpret_cast<u32x4 *>(static_cast<Out *>(p.out) + static_cast<int64_t>(e) * p.R * p.C);
    const int64_t end = min((i + 1) * each, groups);
    for (int64_t g = i * each + threadIdx.x; g < end; g += kThreads) put<true>(o + g, u32x4{0, 0, 0, 0});
}

// The last rows of an expert take a tile of the height that they need, in
// steps of 64.
template <int kOp, class S, int BM, int BN, class Out, bool kAdd>
__device__ __forceinline__ void multiply_rows(const ExpertParams &p, const Tile &t, int64_t m0, int64_t n0,
                                              int64_t rows) {
    if constexpr (kOp != kDw && BM > 64) {
        if (rows <= BM - 64) return multiply_rows<kOp, S, BM - 64, BN, Out, kAdd>(p, t, m0, n0, rows);
    }
    multiply_part<kOp, S, BM, BN, Out, kAdd>(p, t, m0, n0);
}

template <int kOp, class S, class Out, bool kAdd>
__global__ __launch_bounds__(kThreads, S::kPerCu) void k_expert(const ExpertParams p) {
    constexpr bool kHalves = S::kPerCu == 1;
    const int64_t N = kOp == kForward ? p.R : p.C;
    const int32_t n_tiles = static_cast<int32_t>((N + S::kN - 1) / S::kN);
    Tile t;
    if constexpr (kOp == kDw) {
        const int32_t m_tiles = static_cast<int32_t>((p.R + S::kM - 1) / S::kM), each = m_tiles * n_tiles;
        const int32_t v = unit_index(p);
        t.e = v / each;
        if (t.e >= p.E) return;
        const int2 r = rows_of(p, t.e);
        t.lo = r.x;
        t.n = r.y;
        t.half = -1;
        if (t.n == 0) {
            if constexpr (!kAdd) zero_part<Out>(p, t.e, v - t.e * each, each);
            return;
        }
        place(t, v - t.e * each, m_tiles, n_tiles);
    } else {
        if (!token_tile<S::kM, kHalves>(p, n_tiles, t)) return;
    }
    const int64_t m0 = static_cast<int64_t>(t.mt) * S::kM, n0 = static_cast<int64_t>(t.nt) * S::kN;
    const int64_t rows = kOp == kDw ? S::kM : t.n - m0;
    if constexpr (kHalves && kOp != kDw) {
        if (t.half >= 0) {
            const int64_t n = n0 + t.half * (S::kN / 2);
            if (n < N) multiply_rows<kOp, S, S::kM, S::kN / 2, Out, kAdd>(p, t, m0, n, rows);
            return;
        }
    }
    multiply_rows<kOp, S, S::kM, S::kN, Out, kAdd>(p, t, m0, n0, rows);
}

// ------------------------------------------------------------------ host
// a_values, b_values, out_values: whether the arrays hold any.
int check(const char *who, int64_t E, int64_t T, int64_t R, int64_t C, const void *first, const void *a,
          bool a_values, const void *b, bool b_values, const void *out, bool out_values, int32_t out_type) {
    SFT_CHECK(E >= 0 && T >= 0 && R >= 0 && C >= 0, SFT_EINVAL, "%s: a size is negative", who);
    SFT_CHECK(out_type == SFT_F32 || out_type == SFT_BF16, SFT_EINVAL, "%s: bad out_type %d", who, out_type);
    SFT_CHECK(R % 8 == 0 && C % 8 == 0, SFT_ESHAPE, "%s: R and C must be multiples of 8", who);
    SFT_CHECK(T < (int64_t(1) << 30) && E <= 65536 && R <= (int64_t(1) << 20) && C <= (int64_t(1) << 20), SFT_ENOTSUP,
              "%s: T >= 2^30, E > 65536, or R or C > 2^20", who);
    if (!out_values) return SFT_OK;
    SFT_CHECK(first && out && (a || !a_values) && (b || !b_values), SFT_EINVAL, "%s: null pointer", who);
    SFT_CHECK(sft::aligned16(a) && sft::aligned16(b) && sft::aligned16(out), SFT_EALIGN,
              "%s: an array is not 16-byte aligned", who);
    SFT_CHECK((reinterpret_cast<uintptr_t>(first) & 3) == 0, SFT_EALIGN, "%s: first is not 4-byte aligned", who);
    return SFT_OK;
}

// Output tiles of a shape at most: the counts of the experts are on the device.
template <int kOp>
int64_t tiles_of(const ExpertParams &p, int64_t kM, int64_t kN) {
    const int64_t N = kOp == kForward ? p.R : p.C;
    const int64_t m = kOp == kDw ? p.E * ((p.R + kM - 1) / kM) : p.T / kM + std::min<int64_t>(p.E, p.T);
    return m * ((N + kN - 1) / kN);
}

// Workgroups of a launch (the XCDs' runs of units in p.chunk): fewer than 2^32
// threads.
constexpr int64_t kMaxGroups = (int64_t(1) << 32) / kThreads;
template <int kOp>
int64_t groups_of(const ExpertParams &p, const ShapeOf &s, int64_t cus, int32_t &chunk) {
    const int64_t units = tiles_of<kOp>(p, s.m, s.n) + (kOp != kDw && s.per_cu() == 1 ? cus / 2 : 0);
    // runs of a whole round of workgroups (per_cu() on each of an XCD's 32 CUs),
    // fewer where the launch has less than a round
    chunk = static_cast<int32_t>(std::min<int64_t>(32 * s.per_cu(), (units + 7) / 8));
    const int64_t run = 8 * int64_t(chunk);
    return (units + run - 1) / run * run;
}

// Whether the results share bytes with an array that other workgroups may
// still read.
template <int kOp>
bool writes_an_input(const ExpertParams &p, int32_t out_type) {
    const auto meet = [](const void *x, int64_t nx, const void *y, int64_t ny) {
        const uint8_t *a = static_cast<const uint8_t *>(x), *b = static_cast<const uint8_t *>(y);
        return nx && ny && a < b + ny && b < a + nx;
    };
    const int64_t W = int64_t(p.E) * p.R * p.C;
    const int64_t out = (kOp == kForward ? p.T * p.R : kOp == kDx ? p.T * p.C : W) * (out_type == SFT_F32 ? 4 : 2);
    return meet(p.out, out, p.a, 2 * p.T * (kOp == kForward ? p.C : p.R)) ||
           meet(p.out, out, p.b, 2 * (kOp == kDw ? p.T * p.C : W)) || meet(p.out, out, p.first, 4 * (int64_t(p.E) + 1));
}

template <int kOp, class S>
int launch(const char *who, ExpertParams p, int32_t out_type, bool add, hipStream_t st) {
    p.cus = sft::num_cus();
    const int64_t groups = groups_of<kOp>(p, ShapeOf::of<S>(), p.cus, p.chunk);
    SFT_CHECK(groups < kMaxGroups, SFT_ENOTSUP, "%s: 2^24 output tiles or more", who);
    SFT_CHECK(!writes_an_input<kOp>(p, out_type), SFT_EINVAL, "%s: the results overlap an input", who);
    const dim3 grid(static_cast<uint32_t>(groups)), block(kThreads);
    if (out_type == SFT_BF16)
        hipLaunchKernelGGL((k_expert<kOp, S, uint16_t, false>), grid, block, 0, st, p);
    else if (!add)
        hipLaunchKernelGGL((k_expert<kOp, S, float, false>), grid, block, 0, st, p);
    else if constexpr (kOp == kDw)
        hipLaunchKernelGGL((k_expert<kOp, S, float, true>), grid, block, 0, st, p);
    const hipError_t e = hipGetLastError();
    SFT_CHECK(e == hipSuccess, SFT_EHIP, "%s: launch failed: %s", who, hipGetErrorString(e));
    return SFT_OK;
}

// The shape of a product's tiles, by how much there is to fill the GPU with.
// Times in us on one MI355X, experts x R x C at T tokens, groups uneven:
//   256 x 256, one workgroup a CU: least traffic between L2 and LDS.
//     Forward, stages of 64 (whole cache lines of k): 8 x 11008 x 4096 at T =
//     4096 / 16384: 382 / 1309, 128 x 192 413 / 1408, 128 x 128 438 / 1520.
//     Input gradient, stages of 32, four of them: 103 / 468 / 1306 at 16 /
//     4096 / 16384, 128 x 192 171 / 479 / 1495; its weight rows are long
//     runs, so it also streams them best for few tokens.
//   128 x 192, two workgroups a CU, one stores while the other multiplies:
//     shorter sums or groups (64 x 1376 x 4096 at 16384, forward 275, 256 x
//     256 299; input gradient 265, 256 x 256 272, at 4096 143 and 162)
//   128 x 128: forward of groups about that long (8 x 11008 x 4096 at 1024:
//     177, 128 x 192 207, 256 x 256 202; 64 x 1376 x 4096 at 8192: 184, 221;
//     not where they take more rounds: 24 x 1536 x 2048 at 4096: 70, 49),
//     and where the rounds of workgroups come out much better (64 x 2816 x 2048
//     at 256 to 4096, input gradient: 125 to 143, 128 x 192 143 to 160; 16 x
//     1376 x 1000 at 4096, forward: 32, 42; but 64 x 1376 x 4096 at 4096: 190,
//     166)
//   128 x 256, stages of 32: the weight gradient, whose operands are both
//     read in long rows (8 x 11008 x 4096 at 64 / 4096 / 16384: 259 / 599 /
//     1412; 128 x 192 287 / 632 / 1553, 256 x 256 449 / 639 / 1409)
//   64 x 128: few tiles of longer groups (16 x 1024 x 1024 forward at 4096:
//     20.2, 128 x 192 26.1, 64 x 64 26.8); with three stages where there is
//     more than one 64 x 64 tile a CU, but one round of these (16 x 1376 x 1000
//     at 256 / 1024, input gradient 15.5 / 17.8, 64 x 64 18.1 / 20.8; forward at
//     1024 25.9 and 28.9; long sums need the loads of more tiles in flight: 8 x
//     4096 x 11008 forward at 64: 182, 64 x 64 136)
//   64 x 64 with four stages: the fewest tiles, and forward of short groups
//     (64 x 1376 x 4096 at 8 / 1024: 20 / 138, 128 x 192 34 / 159; 32 x 4096 x
//     4096 at 256: 196 and 220; 64 x 4096 x 1376: 124 and 145); five stages
//     where sums are long and no CU has more than one tile, so that only the
//     ring keeps loads in flight (the same 17.0, four stages 19.1; 12 x 1000 x
//     520 at 1003 tokens, of two tiles a CU and short sums, 9.3 and 8.9)
template <int kOp>
ShapeOf shape_by_sizes(const ExpertParams &p, int64_t cus) {
    // rounds of workgroups, two a CU, that so many tiles take
    [[maybe_unused]] const auto rounds = [cus](int64_t tiles) { return (tiles + 2 * cus - 1) / (2 * cus); };
    if constexpr (kOp == kDw) {
        if (tiles_of<kOp>(p, 128, 256) >= 256) return {128, 256, 32, 3};
        if (tiles_of<kOp>(p, 128, 128) >= 256) return {128, 128, 64, 2};
    } else {
        const int64_t rows = p.T / p.E;      // of an expert on average
        const int64_t K = kOp == kForward ? p.C : p.R;
        if constexpr (kOp == kForward) {
            if (rows >= 512 && tiles_of<kOp>(p, 256, 256) >= 1024) return {256, 256, 64, 2};
            if (rows >= 96 && rows <= 192 && tiles_of<kOp>(p, 128, 128) >= 512 &&
                2 * rounds(tiles_of<kOp>(p, 128, 128)) <= 3 * rounds(tiles_of<kOp>(p, 128, 192)))
                return {128, 128, 64, 2};
        } else {
            if (p.R >= 4096 && tiles_of<kOp>(p, 256, 256) >= 128) return {256, 256, 32, 4};
        }
        if (tiles_of<kOp>(p, 128, 192) >= 320 && (kOp == kDx || rows >= 48)) {
            // rounds times a tile's width; an expert has one tile a column, or
            // its rows and half a step of 64 more (between, whether one or two
            // is up to the groups: 64 x 1408 x 2048 at 8192, input gradient, 90
            // by this shape, 128 x 128 102)
            const int64_t N = kOp == kForward ? p.R : p.C;
            const int64_t high = p.E * (rows < 96 ? 128 : rows + 32) / 128;
            const int64_t narrow = 2 * rounds(high * ((N + 127) / 128)), wide = 3 * rounds(high * ((N + 191) / 192));
            if (rows >= 4 && (rows < 96 || rows > 192) && 10 * narrow <= 7 * wide) return {128, 128, 64, 2};
            return {128, 192, 64, 2};
        }
        if (tiles_of<kOp>(p, 64, 128) >= 256 && rows >= 128) return {64, 128, 64, 2};
        if (K <= 4096 && tiles_of<kOp>(p, 64, 64) > cus && tiles_of<kOp>(p, 64, 128) <= 2 * cus) return {64, 128, 64, 3};
    }
    if constexpr (kOp == kForward) {
        if (p.C >= 2048 && tiles_of<kOp>(p, 64, 64) <= cus) return {64, 64, 64, 5};
    }
    return {64, 64, 64, 4};
}

// The same, but where a launch does not hold so many tiles (one row on each of
// 16384 experts of 65536 x 8: 17 million of 64 x 64), larger ones.
template <int kOp>
ShapeOf shape_for(const ExpertParams &p, int64_t cus) {
    const ShapeOf s = shape_by_sizes<kOp>(p, cus);
    int32_t chunk;
    if (kOp != kDw && groups_of<kOp>(p, s, cus, chunk) >= kMaxGroups) return {128, 192, 64, 2};
    return s;
}

// The one of these kernels that the rule chose.
template <int kOp, class... S>
int launch_one(const ShapeOf &shape, const char *who, const ExpertParams &p, int32_t out_type, bool add,
               hipStream_t st) {
    int rc = SFT_ENOTSUP;
    (void)((shape == ShapeOf::of<S>() && (rc = launch<kOp, S>(who, p, out_type, add, st), true)) || ...);
    return rc;
}

template <int kOp>
int product(const char *who, const ExpertParams &p, int32_t out_type, bool add, void *stream) {
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const ShapeOf shape = shape_for<kOp>(p, sft::num_cus());
    if constexpr (kOp == kDw)
        return launch_one<kOp, Shape<128, 256, 32, 3>, Shape<128, 128, 64, 2>, Shape<64, 64, 64, 4>>(shape, who, p, out_type,
                                                                                                    add, st);
    else if constexpr (kOp == kDx)
        return launch_one<kOp, Shape<256, 256, 32, 4>, Shape<128, 192, 64, 2>, Shape<128, 128, 64, 2>,
                          Shape<64, 128, 64, 2>, Shape<64, 128, 64, 3>, Shape<64, 64, 64, 4>>(shape, who, p, out_type,
                                                                                             add, st);
    else
        return launch_one<kOp, Shape<256, 256, 64, 2>, Shape<128, 192, 64, 2>, Shape<128, 128, 64, 2>,
                          Shape<64, 128, 64, 2>, Shape<64, 128, 64, 3>, Shape<64, 64, 64, 5>, Shape<64, 64, 64, 4>>(
            shape, who, p, out_type, add, st);
}

}  // namespace

extern "C" {

int sft_expert_forward(int64_t E, int64_t T, int64_t R, int64_t C, const int32_t *first, const uint16_t *X,
                       const uint16_t *W, void *Y, int32_t out_type, void *stream) {
    sft::clear_error();
    if (int rc = check("sft_expert_forward", E, T, R, C, first, X, T && C, W, E && R && C, Y, E && T && R,
                       out_type))
        return rc;
    if (E == 0 || T == 0 || R == 0) return SFT_OK;
    return product<kForward>("sft_expert_forward", ExpertParams{X, W, Y, first, T, R, C, int32_t(E), 0, 0}, out_type,
                             false, stream);
}

int sft_expert_dx(int64_t E, int64_t T, int64_t R, int64_t C, const int32_t *first, const uint16_t *dY,
                  const uint16_t *W, void *dX, int32_t out_type, void *stream) {
    sft::clear_error();
    if (int rc = check("sft_expert_dx", E, T, R, C, first, dY, T && R, W, E && R && C, dX, E && T && C, out_type))
        return rc;
    if (E == 0 || T == 0 || C == 0) return SFT_OK;
    return product<kDx>("sft_expert_dx", ExpertParams{dY, W, dX, first, T, R, C, int32_t(E), 0, 0}, out_type, false,
                        stream);
}

int sft_expert_dw(int64_t E, int64_t T, int64_t R, int64_t C, const int32_t *first, const uint16_t *dY,
                  const uint16_t *X, void *dW, int32_t out_type, int32_t accumulate, void *stream) {
    sft::clear_error();
    if (int rc = check("sft_expert_dw", E, T, R, C, first, dY, T && R, X, T && C, dW, E && R && C, out_type))
        return rc;
    SFT_CHECK(!accumulate || out_type == SFT_F32, SFT_EINVAL, "sft_expert_dw: only fp32 gradients accumulate");
    if (E == 0 || R == 0 || C == 0) return SFT_OK;
    return product<kDw>("sft_expert_dw", ExpertParams{dY, X, dW, first, T, R, C, int32_t(E), 0, 0}, out_type,
                        accumulate != 0, stream);
}

int sft_probe_expert_tiles(int32_t op, int64_t E, int64_t T, int64_t R, int64_t C, int32_t cus, int32_t *out) {
    sft::clear_error();
    SFT_CHECK(op >= kForward && op <= kDw && cus >= 0 && out, SFT_EINVAL, "sft_probe_expert_tiles: bad arguments");
    if (int rc = check("sft_probe_expert_tiles", E, T, R, C, nullptr, nullptr, false, nullptr, false, nullptr, false,
                       SFT_F32))
        return rc;
    SFT_CHECK(E && R && C && (T || op == kDw), SFT_EINVAL, "sft_probe_expert_tiles: nothing to launch");
    const ExpertParams p{nullptr, nullptr, nullptr, nullptr, T, R, C, int32_t(E), 0, 0};
    const int64_t n = cus ? cus : sft::num_cus();
    ShapeOf s;
    int64_t groups;
    const auto look = [&](auto o) {
        constexpr int kOp = decltype(o)::value;
        int32_t chunk;
        s = shape_for<kOp>(p, n);
        groups = groups_of<kOp>(p, s, n, chunk);
    };
    op == kForward ? look(ic<kForward>{}) : op == kDx ? look(ic<kDx>{}) : look(ic<kDw>{});
    SFT_CHECK(groups < kMaxGroups, SFT_ENOTSUP, "sft_probe_expert_tiles: 2^24 output tiles or more");
    out[0] = s.m, out[1] = s.n, out[2] = s.k, out[3] = s.stages;
    return SFT_OK;
}

}  // extern "C"
