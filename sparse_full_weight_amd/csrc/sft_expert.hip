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

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kBK = 64;                       // k of one stage: four matrix steps of 16
constexpr uint32_t kOutside = 0x80000000u;    // an offset beyond every buffer's size: reads as zero
constexpr int kGroupM = 8;                    // m-tiles that are walked together along n

enum Op { kForward = 0, kDx = 1, kDw = 2 };

struct ExpertParams {
    const uint16_t *a, *b;
    void *out;
    const int32_t *first;
    int64_t T, R, C;
    int32_t E;
    int32_t chunk;          // consecutive tiles that one XCD takes
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
// One output tile: expert e, its token rows [lo, lo + n), tile position.
struct Tile {
    int32_t e, lo, n, mt, nt;
};

// Expert e's rows, whatever first[] holds: inside [0, T], never negative.
__device__ __forceinline__ int2 rows_of(const ExpertParams &p, int32_t e) {
    const int32_t T = static_cast<int32_t>(p.T);
    const int32_t lo = min(max(p.first[e], 0), T);
    return int2{lo, min(max(p.first[e + 1], lo), T) - lo};
}

// Workgroups are dealt to the 8 XCDs in turn; an XCD takes runs of `chunk`
// neighbouring tiles, which share operand panels in its L2.
__device__ __forceinline__ int32_t tile_index(const ExpertParams &p) {
    const int32_t b = blockIdx.x, x = b & 7, i = b >> 3;
    return ((i / p.chunk) * 8 + x) * p.chunk + i % p.chunk;
}

// Tiles of an expert in walking order: groups of kGroupM m-tiles, n outside,
// m inside, so that the tiles of a run share a few panels of both operands.
__device__ __forceinline__ void place(Tile &t, int32_t i, int32_t m_tiles, int32_t n_tiles) {
    const int32_t g = i / (kGroupM * n_tiles), r = i - g * kGroupM * n_tiles;
    const int32_t gm = min(kGroupM, m_tiles - g * kGroupM);
    t.nt = r / gm;
    t.mt = g * kGroupM + (r - t.nt * gm);
}

// The tile of this workgroup, or false where there is none: the host only
// knows how many tiles there can be at most.  64 experts at a time, a lane
// each: their tile counts, the running sum, and the lane whose range holds
// the index.
template <int BM, int BN>
__device__ __forceinline__ bool token_tile(const ExpertParams &p, int32_t n_tiles, Tile &t) {
    const int32_t v = tile_index(p), lane = threadIdx.x & 63;
    int32_t before = 0;
    for (int32_t e0 = 0; e0 < p.E; e0 += 64) {
        const int32_t e = e0 + lane;
        const int2 r = e < p.E ? rows_of(p, e) : int2{0, 0};
        const int32_t m_tiles = (r.y + BM - 1) / BM;
        int32_t end = m_tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t o = __shfl_up(end, d);
            end += lane >= d ? o : 0;
        }
        end = before + end * n_tiles;
        const uint64_t past = __ballot(v < end);
        if (past) {
            const int at = __builtin_ctzll(past);
            t.e = e0 + at;
            t.lo = uniform(__shfl(r.x, at));
            t.n = uniform(__shfl(r.y, at));
            const int32_t mt = uniform(__shfl(m_tiles, at));
            const int32_t i = v - (uniform(__shfl(end, at)) - mt * n_tiles);
            if (i < 0 || i >= mt * n_tiles) return false;   // first[] does not ascend and the sums ran over
            place(t, i, mt, n_tiles);
            return true;
        }
        before = uniform(__shfl(end, 63));
    }
    return false;
}

// ------------------------------------------------------------------ operands
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, void *lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)(lds), 16, voff, 0, 0, 0);
}
__device__ __forceinline__ short4v lds_tr16(const uint8_t *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4v *)(p));
}

// One operand of a tile: how its stages of kBK k-values get into LDS and how
// a wave reads matrix fragments from there.  W: rows (m or n) of the tile, NW:
// waves of the workgroup.  A stage is copied by pieces of 1 KB, 16 bytes a
// lane, of which a wave takes every NW-th.
//
// kTr false (k contiguous): LDS row = one m, 128 bytes, 8 groups of 16 bytes;
// group g sits in slot g ^ (row % 8), so that 8 lanes reading one group of 8
// rows hit all banks.  kTr true (m contiguous): LDS row = one k, 2W bytes;
// group g sits in slot g ^ 2*(row % 4), so that the four rows of a transposing
// read hit distinct banks.
template <bool kTr, int W, int NW>
struct Operand {
    static constexpr int kBytes = W * kBK * 2;
    static constexpr int kLoads = kBytes / 1024 / NW;
    static_assert(kLoads * 1024 * NW == kBytes, "a stage is its waves' pieces");
    static constexpr int kRowLanes = kTr ? W / 8 : 8;     // lanes of a piece that share an LDS row

    const uint8_t *base;      // of the next stage's first byte (wave-uniform)
    int64_t left;             // bytes from there to the end of what is valid
    int64_t step;             // bytes from one stage to the next
    uint32_t voff[kLoads];
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
            const int row = (64 / kRowLanes) * (wave + NW * k) + lane / kRowLanes;
            const int slot = lane % kRowLanes;
            const int grp = kTr ? slot ^ (2 * (row & 3)) : slot ^ (row & 7);
            if constexpr (kTr) {
                voff[k] = 8 * grp < cols ? static_cast<uint32_t>((row * ld + 8 * grp) * 2) : kOutside;
            } else {
                voff[k] = row < valid ? static_cast<uint32_t>((row * ld + 8 * grp) * 2) : kOutside;
                kgrp = 8 * grp;   // row % 8 is the same for every piece of the lane
            }
        }
    }

    // Copies the next stage; k_left = valid k-values from it on.
    __device__ __forceinline__ void issue(uint8_t *lds, int32_t k_left) {
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

    // Fragments: 32 rows (m) of matrix step kk; lane l holds row l % 32,
    // k = 8 * (l / 32) + 0..7.  at: first row of the wave's part of the tile.
    template <int F>
    __device__ __forceinline__ void read(const uint8_t *lds, int at, int kk, bf16x8 (&f)[F]) const {
        const int lane = threadIdx.x & 63;
        if constexpr (kTr) {
            const int s = lane & 15, row = 16 * kk + 8 * (lane >> 5) + (s >> 2);
            const int col = ((lane >> 4) & 1) * 16 + 4 * (s & 3);
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const int grp = (at + 32 * i) / 8 + (col >> 3);
                const uint8_t *q = lds + row * (2 * W) + 16 * (grp ^ (2 * (s >> 2))) + 2 * (col & 7);
                const short4v lo = lds_tr16(q), hi = lds_tr16(q + 4 * 2 * W);
                f[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            }
        } else {
            const int row = at + (lane & 31);
#pragma unroll
            for (int i = 0; i < F; ++i)
                f[i] = *reinterpret_cast<const bf16x8 *>(lds + (row + 32 * i) * 128 +
                                                         16 * ((2 * kk + (lane >> 5)) ^ (lane & 7)));
        }
    }
};

// Two stages of each operand, as LDS variables of their own so that the
// compiler can tell copies into one from reads of the other.
template <int BM, int BN, int S>
struct Stage {
    static __device__ __forceinline__ uint8_t *a() {
        __shared__ __attribute__((aligned(1024))) uint8_t m[BM * kBK * 2];
        return m;
    }
    static __device__ __forceinline__ uint8_t *b() {
        __shared__ __attribute__((aligned(1024))) uint8_t m[BN * kBK * 2];
        return m;
    }
};

// ------------------------------------------------------------------ the product
template <class Out, bool kAdd>
__device__ __forceinline__ void store4(Out *o, f32x4 x) {
    if constexpr (std::is_same<Out, float>::value) {
        f32x4 *q = reinterpret_cast<f32x4 *>(o);
        *q = kAdd ? *q + x : x;
    } else {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        *reinterpret_cast<u32x2 *>(o) = __builtin_bit_cast(
            u32x2, bf16x4{static_cast<__bf16>(x.x), static_cast<__bf16>(x.y), static_cast<__bf16>(x.z),
                          static_cast<__bf16>(x.w)});
    }
}

// WM x WN waves; each takes (BM/WM) x (BN/WN) of the tile in blocks of 32 x 32.
template <int kOp, int BM, int BN, int WM, int WN, class Out, bool kAdd>
__global__ __launch_bounds__(WM *WN * 64, 2) void k_expert(const ExpertParams p) {
    constexpr int NW = WM * WN, FM = BM / WM / 32, FN = BN / WN / 32;
    typedef Operand<kOp == kDw, BM, NW> A;
    typedef Operand<kOp != kForward, BN, NW> B;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int64_t N = kOp == kForward ? p.R : p.C;
    const int32_t n_tiles = static_cast<int32_t>((N + BN - 1) / BN);

    Tile t;
    if constexpr (kOp == kDw) {
        const int32_t m_tiles = static_cast<int32_t>((p.R + BM - 1) / BM), v = tile_index(p);
        t.e = v / (m_tiles * n_tiles);
        if (t.e >= p.E) return;
        const int2 r = rows_of(p, t.e);
        t.lo = r.x;
        t.n = r.y;
        place(t, v - t.e * m_tiles * n_tiles, m_tiles, n_tiles);
    } else {
        if (!token_tile<BM, BN>(p, n_tiles, t)) return;
    }
    const int64_t m0 = static_cast<int64_t>(t.mt) * BM, n0 = static_cast<int64_t>(t.nt) * BN;
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

    const int am = (wave / WN) * (BM / WM), bn = (wave % WN) * (BN / WN);
    const int32_t KT = static_cast<int32_t>((K + kBK - 1) / kBK), k32 = static_cast<int32_t>(K);
    auto issue = [&](auto s, int32_t kt) __attribute__((always_inline)) {
        constexpr int S = decltype(s)::value;
        a.issue(Stage<BM, BN, S>::a(), k32 - kt * kBK);
        b.issue(Stage<BM, BN, S>::b(), k32 - kt * kBK);
    };
    // One stage: its copies have landed for this wave (and, behind the
    // barrier, for all); the next stage's are on their way while it is used.
    auto use = [&](auto s, int32_t kt) __attribute__((always_inline)) {
        constexpr int S = decltype(s)::value;
        if (kt + 1 < KT) {
            issue(ic<1 - S>{}, kt + 1);
            SFT_WAIT_VMCNT(A::kLoads + B::kLoads);
        } else {
            SFT_WAIT_VMCNT(0);
        }
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk) {
            bf16x8 fa[FM], fb[FN];
            a.read(Stage<BM, BN, S>::a(), am, kk, fa);
            b.read(Stage<BM, BN, S>::b(), bn, kk, fb);
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
        }
        SFT_WAIT_LGKM0();
        __builtin_amdgcn_s_barrier();
    };
    if (KT > 0) issue(ic<0>{}, 0);
    for (int32_t kt = 0; kt < KT; kt += 2) {
        use(ic<0>{}, kt);
        if (kt + 1 < KT) use(ic<1>{}, kt + 1);
    }

    // Lane l holds, for row l % 32 of block (i, j), the columns
    // 8*(r/4) + 4*(l/32) + r%4 of register r: four neighbours a register quad.
    Out *out = static_cast<Out *>(p.out) +
               (kOp == kDw ? static_cast<int64_t>(t.e) * p.R * p.C : static_cast<int64_t>(t.lo) * N);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t m = m0 + am + 32 * i + (lane & 31);
        if (m >= M) continue;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t n = n0 + bn + 32 * j + 8 * q + 4 * (lane >> 5);
                if (n < N)
                    store4<Out, kAdd>(out + m * N + n, f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                                            acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]});
            }
    }
}

// ------------------------------------------------------------------ host
// a_values, b_values, out_values: whether the arrays hold any.
int check(const char *who, int64_t E, int64_t T, int64_t R, int64_t C, const void *first, const void *a,
          bool a_values, const void *b, bool b_values, const void *out, bool out_values, int32_t out_type) {
    SFT_CHECK(E >= 0 && T >= 0 && R >= 0 && C >= 0, SFT_EINVAL, "%s: a size is negative", who);
    SFT_CHECK(out_type == SFT_F32 || out_type == SFT_BF16, SFT_EINVAL, "%s: bad out_type %d", who, out_type);
    SFT_CHECK(R % 8 == 0 && C % 8 == 0, SFT_ESHAPE, "%s: R and C must be multiples of 8", who);
    SFT_CHECK(T < (int64_t(1) << 31) && E <= 65536 && R <= (int64_t(1) << 20) && C <= (int64_t(1) << 20), SFT_ENOTSUP,
              "%s: T >= 2^31, E > 65536, or R or C > 2^20", who);
    if (!out_values) return SFT_OK;
    SFT_CHECK(first && out && (a || !a_values) && (b || !b_values), SFT_EINVAL, "%s: null pointer", who);
    SFT_CHECK(sft::aligned16(a) && sft::aligned16(b) && sft::aligned16(out), SFT_EALIGN,
              "%s: an array is not 16-byte aligned", who);
    SFT_CHECK((reinterpret_cast<uintptr_t>(first) & 3) == 0, SFT_EALIGN, "%s: first is not 4-byte aligned", who);
    return SFT_OK;
}

template <int kOp, int BM, int BN, int WM, int WN>
int launch(const char *who, ExpertParams p, int32_t out_type, bool add, hipStream_t st) {
    const int64_t N = kOp == kForward ? p.R : p.C, n_tiles = (N + BN - 1) / BN;
    const int64_t m_tiles = kOp == kDw ? p.E * ((p.R + BM - 1) / BM) : p.T / BM + std::min<int64_t>(p.E, p.T);
    const int64_t tiles = m_tiles * n_tiles;
    if (tiles == 0) return SFT_OK;
    // runs of a whole round of workgroups (one or two on each of an XCD's 32
    // CUs), fewer where the launch has less than a round
    const int64_t round = 32 * (8 / (WM * WN));
    p.chunk = static_cast<int32_t>(std::min<int64_t>(round, (tiles + 7) / 8));
    const int64_t run = 8 * int64_t(p.chunk), groups = (tiles + run - 1) / run * run;
    SFT_CHECK(groups < (int64_t(1) << 31), SFT_ENOTSUP, "%s: 2^31 output tiles or more", who);
    const dim3 grid(static_cast<uint32_t>(groups)), block(WM * WN * 64);
    if (out_type == SFT_BF16)
        hipLaunchKernelGGL((k_expert<kOp, BM, BN, WM, WN, uint16_t, false>), grid, block, 0, st, p);
    else if (!add)
        hipLaunchKernelGGL((k_expert<kOp, BM, BN, WM, WN, float, false>), grid, block, 0, st, p);
    else if constexpr (kOp == kDw)
        hipLaunchKernelGGL((k_expert<kOp, BM, BN, WM, WN, float, true>), grid, block, 0, st, p);
    const hipError_t e = hipGetLastError();
    SFT_CHECK(e == hipSuccess, SFT_EHIP, "%s: launch failed: %s", who, hipGetErrorString(e));
    return SFT_OK;
}

template <int kOp>
int product(const char *who, const ExpertParams &p, int32_t out_type, bool add, void *stream) {
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return launch<kOp, 256, 256, 2, 4>(who, p, out_type, add, st);
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
    return product<kForward>("sft_expert_forward", ExpertParams{X, W, Y, first, T, R, C, int32_t(E), 0}, out_type,
                             false, stream);
}

int sft_expert_dx(int64_t E, int64_t T, int64_t R, int64_t C, const int32_t *first, const uint16_t *dY,
                  const uint16_t *W, void *dX, int32_t out_type, void *stream) {
    sft::clear_error();
    if (int rc = check("sft_expert_dx", E, T, R, C, first, dY, T && R, W, E && R && C, dX, E && T && C, out_type))
        return rc;
    if (E == 0 || T == 0 || C == 0) return SFT_OK;
    return product<kDx>("sft_expert_dx", ExpertParams{dY, W, dX, first, T, R, C, int32_t(E), 0}, out_type, false,
                        stream);
}

int sft_expert_dw(int64_t E, int64_t T, int64_t R, int64_t C, const int32_t *first, const uint16_t *dY,
                  const uint16_t *X, void *dW, int32_t out_type, int32_t accumulate, void *stream) {
    sft::clear_error();
    if (int rc = check("sft_expert_dw", E, T, R, C, first, dY, T && R, X, T && C, dW, E && R && C, out_type))
        return rc;
    SFT_CHECK(!accumulate || out_type == SFT_F32, SFT_EINVAL, "sft_expert_dw: only fp32 gradients accumulate");
    if (E == 0 || R == 0 || C == 0) return SFT_OK;
    return product<kDw>("sft_expert_dw", ExpertParams{dY, X, dW, first, T, R, C, int32_t(E), 0}, out_type,
                        accumulate != 0, stream);
}

}  // extern "C"
