// libssm2d: matrix products with an epilogue (include/ssm2d_block.h, linear):
//   C[m][n] = sum_k A[m][k] B[n][k], then bias, activation, residual,
// C's n contiguous in memory, A and B each with k or with m (n) contiguous. Token
// rows and channels-first maps, forward and both gradients, are such products
// with the sides chosen (linear.hip).
#pragma once

#include <cmath>

#include "block_common.h"

namespace ssm2d_impl {
namespace gemm {

using bfrag = __bf16 __attribute__((ext_vector_type(8)));
using facc = float __attribute__((ext_vector_type(4)));
using half4 = short __attribute__((ext_vector_type(4)));

struct GemmParams {
    const void *a, *b;
    long a_ld, b_ld;  // stride of the dim that is not contiguous
    long a_bs, b_bs;  // stride of the batch, or of the stretches of k that are summed (kb > 1)
    int M, N, K;
    int kb;           // stretches of K
    unsigned tiles_m, tiles_n, total;  // total: of all splits and batch entries
    long batch;
    unsigned splits;  // parts of the sum, each by workgroups of its own
    int steps, per;   // steps of BK in all stretches, and of one split
    // epilogue
    const float *bias;  // along n, or with bias_m along m
    int bias_m, act;
    const void *res;
    long r_ld, r_bs;
    void *c, *pre;
    long c_ld, c_bs;
    int straight;     // bf16 operands can be loaded straight to LDS
    float *part;      // splits > 1: [split][batch][M][N rounded up to 4]
    float *sums;      // [split][M] sums of A's rows over k (NULL: not wanted; batch 1)
    unsigned first;   // the launch's first workgroup
    // columns that the launch which joins the parts sums as well: [rows][n]
    const float *fold;
    float *fold_to;
    int fold_rows, fold_n;
    unsigned join_blocks;
};

template <typename T>
constexpr int kParts = sizeof(T) == 2 ? 1 : 3;
template <typename T>
constexpr int kStep = sizeof(T) == 2 ? 64 : 32;  // k of a step

// ------------------------------------------------------------------ epilogue

template <typename T>
constexpr int kWide = 16 / static_cast<int>(sizeof(T));  // elements of C that a lane finishes at once

template <typename T, int ACT>
__device__ __forceinline__ void act_all(float (&v)[kWide<T>])
{
#pragma unroll
    for (int j = 0; j < kWide<T>; ++j) v[j] = activate<T, ACT>(v[j]);
}

// The bias of columns n .. n + kWide - 1.
template <typename T>
__device__ __forceinline__ void column_bias(const GemmParams &p, int n, float (&b)[kWide<T>])
{
#pragma unroll
    for (int j = 0; j < kWide<T>; ++j) b[j] = p.bias && !p.bias_m && n < p.N ? p.bias[min(n + j, p.N - 1)] : 0.0f;
}

// The residual of row m from column n on, zeros where there is none.
template <typename T>
__device__ __forceinline__ void read_residual(const GemmParams &p, long b, int m, int n, Raw<T, kWide<T>> &w)
{
    constexpr int V = kWide<T>;
    w.clear();
    if (!p.res || m >= p.M || n >= p.N) return;
    const T *r = static_cast<const T *>(p.res) + b * p.r_bs + static_cast<long>(m) * p.r_ld + n;
    if (n + V <= p.N) {
        w.load_any(r);
    } else {
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = n + j < p.N ? widen1(r[j]) : 0.0f;
        w.set(v);
    }
}

// Neighbours of row m from column n on; bias: their columns', or the row's; RES: with a residual.
template <typename T, bool RES>
__device__ __forceinline__ void finish(const GemmParams &p, long b, int m, int n, float (&v)[kWide<T>], const float (&bias)[kWide<T>], float row,
                                       const Raw<T, kWide<T>> &res)
{
    constexpr int V = kWide<T>;
    if (m >= p.M || n >= p.N) return;
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] += p.bias_m ? row : bias[j];
    const long at = b * p.c_bs + static_cast<long>(m) * p.c_ld + n;
    const bool whole = n + V <= p.N;
    auto put = [&](void *c) __attribute__((always_inline)) {
        T *dst = static_cast<T *>(c) + at;
        if (whole) {
            Raw<T, V> r;
            r.set(v);
            r.store_any(dst);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (n + j < p.N) store1(dst + j, v[j]);
        }
    };
    if (p.pre) put(p.pre);
    switch (p.act) {
    case SSM2D_ACT_RELU: act_all<T, SSM2D_ACT_RELU>(v); break;
    case SSM2D_ACT_SILU: act_all<T, SSM2D_ACT_SILU>(v); break;
    case SSM2D_ACT_GELU: act_all<T, SSM2D_ACT_GELU>(v); break;
    default: break;
    }
    if constexpr (RES) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] += res.get(j);
    }
    put(p.c);
}

// ------------------------------------------------------------------ operands

__device__ __forceinline__ unsigned lds_at(const void *p) { return static_cast<unsigned>(reinterpret_cast<uintptr_t>(p)); }
__device__ __forceinline__ unsigned top_halves(unsigned hi, unsigned lo) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }

// A tile of an operand in LDS, R rows (of m or n) by BK of k, NP parts of bf16.
// KC (k contiguous in memory): [R][BK], the 16-byte chunks of a row turned by the
// row, so that a fragment's 16 rows lie in different banks. Else [BK][R], read
// by transposing reads: those take 32 bytes of 4 rows for each 16 lanes, turned
// by k so that the 8 rows of half a wave lie in different banks.
template <bool KC, int R, int BK, int NP>
struct OperandTile {
    static constexpr int kPart = R * BK, kElems = NP * kPart;
    static constexpr int kRow = KC ? BK : R, kChunks = kRow / 8;
    __device__ static __forceinline__ int turn(int row)
    {
        if constexpr (KC) return BK == 64 ? (row & 7) : ((row >> 1) & 3);
        else return (R == 128 ? ((row & 3) | ((row >> 1) & 4)) : (((row >> 1) & 1) | ((row >> 2) & 2))) << 1;
    }
    // the place of chunk c of a row
    __device__ static __forceinline__ int at(int row, int c) { return row * kRow + ((c ^ turn(row)) << 3); }
    // rows r0 .. r0 + 15 and k = 32 ks + 8 (lane / 16) .. + 7 of part n
    __device__ static __forceinline__ bfrag frag(const uint16_t *tile, int n, int r0, int ks)
    {
        const int l = threadIdx.x % 64;
        if constexpr (KC) {
            return *reinterpret_cast<const bfrag *>(tile + n * kPart + at(r0 + l % 16, ks * 4 + l / 16));
        } else {
            using lds4 = __attribute__((address_space(3))) half4 *;
            const int k = ks * 32 + 8 * (l / 16) + (l % 16) / 4;  // (rows k and k + 4 are turned alike)
            const unsigned a = lds_at(tile + n * kPart + at(k, r0 / 8 + (l % 4) / 2) + 4 * (l & 1));
            union {
                half4 h[2];
                bfrag f;
            } u;
            u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uintptr_t)a);
            u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uintptr_t)(a + 4 * kRow * 2));
            return u.f;
        }
    }
};

// 16 bytes of an operand on their way from memory to LDS (neighbouring lanes take
// neighbouring ones: two loads into the same line that is still under way
// would wait for each other).
template <typename T>
struct Chunk {
    static constexpr int kN = 16 / static_cast<int>(sizeof(T));
    Raw<T, kN> r;
    // the first `count` of the kN elements at p (0 or less: none), the others 0
    __device__ __forceinline__ void load(const T *p, long count)
    {
        if (count >= kN) {
            r.load_any(p);
        } else if (count > 0) {
            float v[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) v[i] = widen1(p[min(i, static_cast<int>(count) - 1)]);
#pragma unroll
            for (int i = 1; i < kN; ++i) v[i] = i < count ? v[i] : 0.0f;
            r.set(v);
        } else {
            r.clear();
        }
    }
    // to place c (in chunks) of a row of the tile, as NP parts
    template <typename Tile>
    __device__ __forceinline__ void store(uint16_t *tile, int row, int c) const
    {
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4 *>(tile + Tile::at(row, c)) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        } else {
            uint16_t *dst = tile + Tile::at(row, c / 2) + c % 2 * 4;
            // three parts of 8 bits each, cut off: exact
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = r.get(i);
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                unsigned w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const unsigned lo = __float_as_uint(v[2 * i]), hi = __float_as_uint(v[2 * i + 1]);
                    w[i] = top_halves(hi, lo);
                    v[2 * i] -= __uint_as_float(lo & 0xffff0000u);
                    v[2 * i + 1] -= __uint_as_float(hi & 0xffff0000u);
                }
                *reinterpret_cast<uint2 *>(dst + n * Tile::kPart) = make_uint2(w[0], w[1]);
            }
        }
    }
};

// acc += a b over the parts whose product reaches the last place kept, small ones first.
template <int NP>
__device__ __forceinline__ void mma(facc &acc, const bfrag (&a)[NP], const bfrag (&b)[NP])
{
#pragma unroll
    for (int s = NP - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[s - i], acc, 0, 0, 0);
}

// The tile of C, split and batch entry of a workgroup: workgroups go round the 8
// dies, so each die gets neighbouring tiles, which share operands in its L2.
struct TilePlace {
    int m0, n0, split;
    long b;
};
template <int BM, int BN>
__device__ __forceinline__ TilePlace tile_place(const GemmParams &p, unsigned id)
{
    const unsigned total = p.total, each = total / 8, more = total % 8;
    const unsigned die = id % 8;
    id = die * each + min(die, more) + id / 8;
    TilePlace t;
    t.n0 = static_cast<int>(id % p.tiles_n) * BN;
    id /= p.tiles_n;
    t.m0 = static_cast<int>(id % p.tiles_m) * BM;
    id /= p.tiles_m;
    t.split = static_cast<int>(id % p.splits);
    t.b = id / p.splits;
    return t;
}

// What a wave's lanes write to LDS and read of each other's stays in program order:
// the hardware keeps a wave's LDS accesses in theirs, and this the compiler. No instruction.
__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A wave's accumulators to memory, by way of LDS: there its lanes hold 16 rows by
// four columns each, and whole runs of rows go out (four times fewer requests).
// Every wave of the workgroup calls it, when none reads the operands' tiles any more.
template <typename T, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void finish_tile(const GemmParams &p, const TilePlace &t, facc (&acc)[WM / 16][WN / 16], void *lds, int slot)
{
    constexpr int V = kWide<T>, kLd = WN + 4, kLanes = WN / V, kRowsOnce = 64 / kLanes;
    const int l = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int m0 = t.m0 + wave / (BN / WN) * WM, n = t.n0 + wave % (BN / WN) * WN + l % kLanes * V;
    float *mine = static_cast<float *>(lds) + slot * 32 * kLd;  // 32 rows at a time
    const long ldp = (p.N + 3) / 4 * 4;
    constexpr int kPasses = 32 / kRowsOnce;
    float bias[V];
    column_bias<T>(p, n, bias);
    __syncthreads();
    auto all = [&](auto with_res) __attribute__((always_inline)) {
        constexpr bool RES = decltype(with_res)::value;
#pragma unroll
        for (int half = 0; half < WM / 32; ++half) {
            const int r0 = m0 + half * 32 + l / kLanes;
            // (all that is read, before anything is written that it might be)
            Raw<T, V> res[RES ? kPasses : 1];
            if constexpr (RES) {
#pragma unroll
                for (int k = 0; k < kPasses; ++k) read_residual<T>(p, t.b, r0 + k * kRowsOnce, n, res[k]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < WN / 16; ++j)
                    *reinterpret_cast<facc *>(mine + (i * 16 + l % 16) * kLd + j * 16 + 4 * (l / 16)) = acc[half * 2 + i][j];
            wave_order();  // (its own lanes' writes before its reads: no barrier)
            auto pass = [&](int k, const Raw<T, V> &w) __attribute__((always_inline)) {
                const int m = r0 + k * kRowsOnce;
                float v[V];
#pragma unroll
                for (int q = 0; q < V / 4; ++q) {
                    const facc f = *reinterpret_cast<const facc *>(mine + (l / kLanes + k * kRowsOnce) * kLd + l % kLanes * V + 4 * q);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[4 * q + j] = f[j];
                }
                if (p.splits > 1) {
                    if (m >= p.M) return;
                    float *part = p.part + ((static_cast<long>(t.split) * p.batch + t.b) * p.M + m) * ldp + n;
#pragma unroll
                    for (int q = 0; q < V / 4; ++q)
                        if (n + 4 * q < p.N) *reinterpret_cast<facc *>(part + 4 * q) = facc{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                } else {
                    finish<T, RES>(p, t.b, m, n, v, bias, p.bias && p.bias_m && m < p.M ? p.bias[m] : 0.0f, w);
                }
            };
            if constexpr (RES) {
#pragma unroll
                for (int k = 0; k < kPasses; ++k) pass(k, res[k]);
            } else {
#pragma unroll 2
                for (int k = 0; k < kPasses; ++k) pass(k, res[0]);
            }
            wave_order();  // (and those before the next rows' writes)
        }
    };
    if (p.res && p.splits == 1) all(std::true_type{});
    else all(std::false_type{});
}

// Sums of A's rows, by products with ones (the first column of tiles has them; a
// lane's all four are one row's), a wave's rows.
template <int WM>
struct RowSums {
    facc v[WM / 16];
    bool on;
    __device__ __forceinline__ void begin(bool wanted)
    {
        on = wanted;
#pragma unroll
        for (auto &f : v) f = facc{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __device__ __forceinline__ void add(int i, const bfrag &a)
    {
        const __bf16 one = static_cast<__bf16>(1.0f);
        const bfrag ones = {one, one, one, one, one, one, one, one};
        v[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, a, v[i], 0, 0, 0);
    }
    __device__ __forceinline__ void put(const GemmParams &p, const TilePlace &t, int wm) const
    {
        if (!on || threadIdx.x % 64 >= 16) return;
#pragma unroll
        for (int i = 0; i < WM / 16; ++i) {
            const int m = t.m0 + wm + i * 16 + static_cast<int>(threadIdx.x % 16);
            if (m < p.M) p.sums[static_cast<long>(t.split) * p.M + m] = v[i][0];
        }
    }
};

// Elements of LDS: both operands' tiles, the epilogue's place too.
template <typename T, bool A_KC, bool B_KC, int BM, int BN>
constexpr int kTileElems = std::max((BM + BN) * kStep<T> * kParts<T>, 4 * 32 * (BN / 2 + 4) * 2);

// Any alignment: operands go through registers to LDS, the next step's read
// while this one's products run. SUMS: A's row sums too. float32 is bound by the six
// products' matrix instructions (1.3 of 1.4 us of a full step of 128 x 128 x 32), at 128 channels also by
// memory: those of 196608 cells to 128, 87 us, 3.5 TB/s.
template <typename T, bool A_KC, bool B_KC, int BM, int BN, bool SUMS>
__device__ __forceinline__ void gemm_by_registers(const GemmParams &p, unsigned id, uint16_t *tiles)
{
    constexpr int NP = kParts<T>, BK = kStep<T>, WM = BM / 2, WN = BN / 2;
    using TA = OperandTile<A_KC, BM, BK, NP>;
    using TB = OperandTile<B_KC, BN, BK, NP>;
    uint16_t *const sa = tiles, *const sb = tiles + TA::kElems;
    const TilePlace t = tile_place<BM, BN>(p, id);
    const T *A = static_cast<const T *>(p.a), *B = static_cast<const T *>(p.b);
    if (p.kb == 1) A += t.b * p.a_bs, B += t.b * p.b_bs;
    const int s1 = t.split * p.per, s2 = min(s1 + p.per, p.steps), each = (p.K + BK - 1) / BK;
    constexpr int W = Chunk<T>::kN, CA = BM * BK / W / 256, CB = BN * BK / W / 256;
    Chunk<T> ra[CA], rb[CB];
    auto fetch = [&](int s) __attribute__((always_inline)) {
        const int kb = p.kb == 1 ? 0 : s / each, k0 = (s - kb * each) * BK;
        const T *ap = A + kb * p.a_bs, *bp = B + kb * p.b_bs;
        if (p.kb == 1) ap = A, bp = B;
        auto side = [&](auto kc, const T *src, long ld, int r0, int rows, auto &reg, auto row_len) __attribute__((always_inline)) {
            constexpr int kChunks = decltype(row_len)::value / W;
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(reg) / sizeof(reg[0])); ++i) {
                const int id = i * 256 + threadIdx.x, row = id / kChunks, col = id % kChunks * W;
                if constexpr (decltype(kc)::value) {
                    const long m = r0 + row, k = k0 + col;
                    reg[i].load(src + m * ld + k, m < rows ? p.K - k : 0);
                } else {
                    const long k = k0 + row, m = r0 + col;
                    reg[i].load(src + k * ld + m, k < p.K ? rows - m : 0);
                }
            }
        };
        using std::integral_constant;
        side(integral_constant<bool, A_KC>{}, ap, p.a_ld, t.m0, p.M, ra, integral_constant<int, TA::kRow>{});
        side(integral_constant<bool, B_KC>{}, bp, p.b_ld, t.n0, p.N, rb, integral_constant<int, TB::kRow>{});
    };
    facc acc[WM / 16][WN / 16];
#pragma unroll
    for (auto &r : acc)
#pragma unroll
        for (auto &v : r) v = facc{0.0f, 0.0f, 0.0f, 0.0f};
    const int wave = threadIdx.x / 64, wm = wave / 2 * WM, wn = wave % 2 * WN;
    RowSums<WM> sums;
    if constexpr (SUMS) sums.begin(p.sums && t.n0 == 0 && wave % 2 == 0);
    if (s1 < s2) fetch(s1);
    for (int s = s1; s < s2; ++s) {
        __syncthreads();  // (the last step's tiles have been read)
#pragma unroll
        for (int i = 0; i < CA; ++i) {
            const int id = i * 256 + threadIdx.x;
            ra[i].template store<TA>(sa, id / (TA::kRow / W), id % (TA::kRow / W));
        }
#pragma unroll
        for (int i = 0; i < CB; ++i) {
            const int id = i * 256 + threadIdx.x;
            rb[i].template store<TB>(sb, id / (TB::kRow / W), id % (TB::kRow / W));
        }
        __syncthreads();
        if (s + 1 < s2) fetch(s + 1);
#pragma unroll
        for (int ks = 0; ks < BK / 32; ++ks) {
            bfrag fb[WN / 16][NP];
#pragma unroll
            for (int j = 0; j < WN / 16; ++j)
#pragma unroll
                for (int n = 0; n < NP; ++n) fb[j][n] = TB::frag(sb, n, wn + j * 16, ks);
#pragma unroll
            for (int i = 0; i < WM / 16; ++i) {
                bfrag fa[NP];
#pragma unroll
                for (int n = 0; n < NP; ++n) fa[n] = TA::frag(sa, n, wm + i * 16, ks);
#pragma unroll
                for (int j = 0; j < WN / 16; ++j) mma<NP>(acc[i][j], fb[j], fa);  // (D's rows, a lane's registers, are n)
                if constexpr (SUMS) {
                    if (sums.on) {
#pragma unroll
                        for (int n = NP - 1; n >= 0; --n) sums.add(i, fa[n]);
                    }
                }
            }
        }
    }
    if constexpr (SUMS) sums.put(p, t, wm);
    finish_tile<T, BM, BN, WM, WN>(p, t, acc, tiles, wave);
}
template <typename T, bool A_KC, bool B_KC, int BM, int BN>
__global__ __launch_bounds__(256, 2) void gemm_kernel(const GemmParams p)
{
    __shared__ __align__(16) uint16_t tiles[kTileElems<T, A_KC, B_KC, BM, BN>];
    gemm_by_registers<T, A_KC, B_KC, BM, BN, false>(p, p.first + blockIdx.x, tiles);
}

// ------------------------------------------------------------------ straight to LDS

constexpr unsigned kNowhere = 0x80000000u;  // an offset behind every buffer: its load gives zeros

// One operand's loads, step after step, from memory straight to LDS: 16 bytes a
// lane, 64 lanes a kilobyte of the tile in the order of its places. The turn of
// a chunk (OperandTile) is in which chunk a lane asks for.
template <bool KC, int R, int BK>
struct StraightLoads {
    using Tile = OperandTile<KC, R, BK, 1>;
    static constexpr int kLoads = R * BK / 8 / 256;          // a thread's, of a step
    static constexpr int kRowsEach = 256 / Tile::kChunks;    // rows of the tile that 256 lanes cover
    const uint16_t *src;                                     // of the next step: the tile's first row (KC) or column
    long ld, stride;                                         // stride: between stretches of k
    unsigned off[KC ? kLoads : 1];
    int col;                                                 // KC: the lane's first k
    __device__ __forceinline__ void begin(const uint16_t *p, long ld_, long stride_, int r0, int rows, long kb, int k0)
    {
        ld = ld_, stride = stride_;
        const int row = threadIdx.x / Tile::kChunks, c = (threadIdx.x % Tile::kChunks) ^ Tile::turn(row);
        src = p + kb * stride + (KC ? r0 * ld + k0 : r0 + k0 * ld);
        if constexpr (KC) {
            col = c * 8;
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                off[i] = r0 + i * kRowsEach + row < rows ? static_cast<unsigned>(i * kRowsEach + row) * static_cast<unsigned>(ld * 2) + c * 16 : kNowhere;
        } else {
            col = 0;
            off[0] = r0 + c * 8 < rows ? static_cast<unsigned>(row) * static_cast<unsigned>(ld * 2) + c * 16 : kNowhere;
        }
    }
    // `left` of k: all BK, or what is left of a stretch, zeros past it (0: all zeros)
    __device__ __forceinline__ void issue(uint16_t *tile, int left) const
    {
        using lds = __attribute__((address_space(3))) void;
        const unsigned bytes = KC || left >= BK ? 0x7fffffffu : static_cast<unsigned>(left) * static_cast<unsigned>(ld * 2);
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(src), 0, static_cast<int>(bytes), 0x00020000);
        uint16_t *dst = tile + threadIdx.x / 64 * 512;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const unsigned o = KC ? (col < left ? off[i] : kNowhere) : off[0];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds *)(dst + i * 2048), 16, static_cast<int>(o),
                                                     KC ? 0 : static_cast<int>(i * kRowsEach * ld * 2), 0, 0);
        }
    }
    // to the next step, from the last of a stretch (it began `back` of k ago) to the next stretch
    __device__ __forceinline__ void next(bool over, int back)
    {
        if (over) src += stride - (KC ? static_cast<long>(back) : back * ld);
        else src += KC ? static_cast<long>(BK) : BK * ld;
    }
};

// bf16 operands whose rows are whole 16-byte chunks: two stages of tiles in LDS,
// one filled by loads that pass the registers by while the other is used. Each wave
// waits for its own loads of a stage before the barrier that opens it. Where both
// operands have k contiguous the other stage's loads are under way meanwhile. The
// transposing reads of the other layouts take a plain number as their address, from
// which the compiler cannot tell the stages apart, and has all loads wait before the
// first of them: there the two workgroups of a compute unit overlap, not the
// stages of one. Tiles of 128 x
// 128 keep the matrix instructions busy from two workgroups a compute unit: 4096-cubes 137 us,
// 1000 TFLOP/s, 8192-cubes 1190 us, 924; a ring of four stages of 32 and four workgroups of stages of 32 were
// slower. Short sums are bound by their rounds of tiles: 12544 x 768 to 1536 with GELU and
// a residual 51 to 54 us, 2.3 rounds, 10 of it at the tiles' ends.
template <bool A_KC, bool B_KC, int BM, int BN, bool SUMS>
__device__ __forceinline__ void gemm_by_lds(const GemmParams &p, unsigned id, uint16_t *ring0, uint16_t *ring1)
{
    constexpr int WM = BM / 2, WN = BN / 2, BK = kStep<uint16_t>;
    using TA = OperandTile<A_KC, BM, BK, 1>;
    using TB = OperandTile<B_KC, BN, BK, 1>;
    using LA = StraightLoads<A_KC, BM, BK>;
    using LB = StraightLoads<B_KC, BN, BK>;
    const TilePlace t = tile_place<BM, BN>(p, id);
    const uint16_t *A = static_cast<const uint16_t *>(p.a), *B = static_cast<const uint16_t *>(p.b);
    if (p.kb == 1) A += t.b * p.a_bs, B += t.b * p.b_bs;
    LA la;
    LB lb;
    const int s1 = t.split * p.per, s2 = min(s1 + p.per, p.steps), each = (p.K + BK - 1) / BK, kb = p.kb == 1 ? 0 : s1 / each;
    int k0 = (s1 - kb * each) * BK;
    la.begin(A, p.a_ld, p.kb == 1 ? 0 : p.a_bs, t.m0, p.M, kb, k0);
    lb.begin(B, p.b_ld, p.kb == 1 ? 0 : p.b_bs, t.n0, p.N, kb, k0);
    int ahead = s2 - s1;  // steps whose loads have not begun
    auto issue = [&](uint16_t *ring) __attribute__((always_inline)) {
        const int left = p.K - k0;
        la.issue(ring, left);
        lb.issue(ring + TA::kElems, left);
        const bool over = left <= BK;
        la.next(over, k0);
        lb.next(over, k0);
        k0 = over ? 0 : k0 + BK;
        --ahead;
    };
    facc acc[WM / 16][WN / 16];
#pragma unroll
    for (auto &r : acc)
#pragma unroll
        for (auto &v : r) v = facc{0.0f, 0.0f, 0.0f, 0.0f};
    const int wave = threadIdx.x / 64, wm = wave / 2 * WM, wn = wave % 2 * WN;
    RowSums<WM> sums;
    if constexpr (SUMS) sums.begin(p.sums && t.n0 == 0 && wave % 2 == 0);
    auto step = [&](const uint16_t *ring) __attribute__((always_inline)) {
#pragma unroll
        for (int ks = 0; ks < BK / 32; ++ks) {
            bfrag fb[WN / 16], fa[WM / 16];
#pragma unroll
            for (int j = 0; j < WN / 16; ++j) fb[j] = TB::frag(ring + TA::kElems, 0, wn + j * 16, ks);
#pragma unroll
            for (int i = 0; i < WM / 16; ++i) fa[i] = TA::frag(ring, 0, wm + i * 16, ks);
#pragma unroll
            for (int i = 0; i < WM / 16; ++i)
#pragma unroll
                for (int j = 0; j < WN / 16; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
            if constexpr (SUMS) {
                if (sums.on) {
#pragma unroll
                    for (int i = 0; i < WM / 16; ++i) sums.add(i, fa[i]);
                }
            }
        }
    };
    // the wave's own loads to LDS have arrived (vmcnt 0, the other counters as they are)
    auto arrived = [] __attribute__((always_inline)) { __builtin_amdgcn_s_waitcnt(0x0f70); };
    if (ahead > 0) issue(ring0);
    for (int left = s2 - s1; left > 0; left -= 2) {
        arrived();
        __syncthreads();  // (stage 0 is there, and stage 1 has been read)
        if (ahead > 0) issue(ring1);
        step(ring0);
        if (left == 1) break;
        arrived();
        __syncthreads();
        if (ahead > 0) issue(ring0);
        step(ring1);
    }
    if constexpr (SUMS) sums.put(p, t, wm);
    static_assert((BM + BN) * BK * 2 >= 2 * 32 * (WN + 4) * 4, "the epilogue's place");
    finish_tile<uint16_t, BM, BN, WM, WN>(p, t, acc, wave < 2 ? ring0 : ring1, wave % 2);
}
template <int BM, int BN>
constexpr int kRingElems = (BM + BN) * kStep<uint16_t>;
template <bool A_KC, bool B_KC, int BM, int BN>
__global__ __launch_bounds__(256, 2) void gemm_straight(const GemmParams p)
{
    __shared__ __align__(16) uint16_t ring0[kRingElems<BM, BN>], ring1[kRingElems<BM, BN>];
    gemm_by_lds<A_KC, B_KC, BM, BN, false>(p, p.first + blockIdx.x, ring0, ring1);
}

// ------------------------------------------------------------------ few rows

// NP bf16 parts of 8 neighbours of k, as a fragment holds them.
template <typename T>
__device__ __forceinline__ void to_parts(const Raw<T, 8> &r, bfrag (&f)[kParts<T>])
{
    union {
        unsigned w[4];
        bfrag f;
    } u;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) u.w[i] = r.w[i];
        f[0] = u.f;
    } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = r.get(i);
#pragma unroll
        for (int n = 0; n < 3; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const unsigned lo = __float_as_uint(v[2 * i]), hi = __float_as_uint(v[2 * i + 1]);
                u.w[i] = top_halves(hi, lo);
                v[2 * i] -= __uint_as_float(lo & 0xffff0000u);
                v[2 * i + 1] -= __uint_as_float(hi & 0xffff0000u);
            }
            f[n] = u.f;
        }
    }
}

// Few rows (serving): 16 rows by 16 columns a workgroup, the sum over k shared by its
// 8 waves, each with four (float32: two) steps of 32 under way from memory to registers:
// no LDS and no barrier until the waves' sums are added, and little code, whose way
// to the compute units counts here. Bound by the latencies of a launch and of a
// read. 768 to 1536 channels, one row, in a graph: 3.0 us, float32 4.2; by tiles of 64 6.1 and 9.1.
template <typename T>
__global__ __launch_bounds__(512) void gemm_few(const GemmParams p)
{
    constexpr int NP = kParts<T>, kWaves = 8, kAhead = sizeof(T) == 2 ? 4 : 2, kLd = 20;
    __shared__ float sums[kWaves][16 * kLd];
    const unsigned id = p.first + blockIdx.x;
    const int l = threadIdx.x % 64, wave = threadIdx.x / 64, n0 = static_cast<int>(id % p.tiles_n) * 16, m0 = static_cast<int>(id / p.tiles_n) * 16;
    const int k0 = l / 16 * 8;
    // (rows and columns past the last read it, and go nowhere)
    const T *a = static_cast<const T *>(p.a) + min(m0 + l % 16, p.M - 1) * p.a_ld + k0;
    const T *b = static_cast<const T *>(p.b) + static_cast<long>(min(n0 + l % 16, p.N - 1)) * p.b_ld + k0;
    facc acc = {0.0f, 0.0f, 0.0f, 0.0f};
    const int steps = (p.K + 31) / 32;
    for (int s = wave; s < steps; s += kWaves * kAhead) {
        Raw<T, 8> ra[kAhead], rb[kAhead];
        if ((s + kWaves * (kAhead - 1) + 1) * 32L <= p.K) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int k = (s + i * kWaves) * 32;
                ra[i].load_any(a + k);
                rb[i].load_any(b + k);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const long k = (s + i * kWaves) * 32L;
                const long left = p.K - k - k0;
                ra[i].clear();
                rb[i].clear();
                if (left >= 8) {
                    ra[i].load_any(a + k);
                    rb[i].load_any(b + k);
                } else if (left > 0) {
                    float x[8], y[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = j < left ? widen1(a[k + j]) : 0.0f, y[j] = j < left ? widen1(b[k + j]) : 0.0f;
                    ra[i].set(x);
                    rb[i].set(y);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            bfrag fa[NP], fb[NP];
            to_parts<T>(ra[i], fa);
            to_parts<T>(rb[i], fb);
            mma<NP>(acc, fb, fa);
        }
    }
    *reinterpret_cast<facc *>(&sums[wave][l % 16 * kLd + l / 16 * 4]) = acc;
    __syncthreads();
    // (an element a thread: little code, whose way to the compute units counts here)
    const int r = threadIdx.x / 16, c = threadIdx.x % 16, n = n0 + c;
    const long m = m0 + r;
    if (r >= 16 || m >= p.M || n >= p.N) return;
    float v = p.bias ? p.bias[n] : 0.0f, sum = 0.0f;
    const float res = p.res ? widen1(static_cast<const T *>(p.res)[m * p.r_ld + n]) : 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += sums[w][r * kLd + c];
    v += sum;
    const long at = m * p.c_ld + n;
    if (p.pre) store1(static_cast<T *>(p.pre) + at, v);
    if (p.act == SSM2D_ACT_RELU) v = activate<T, SSM2D_ACT_RELU>(v);
    else if (p.act == SSM2D_ACT_SILU) v = activate<T, SSM2D_ACT_SILU>(v);
    else if (p.act == SSM2D_ACT_GELU) v = activate<T, SSM2D_ACT_GELU>(v);
    store1(static_cast<T *>(p.c) + at, v + res);
}

// Both gradients of a projection in one launch: dweight's workgroups, then dx's (up
// to a whole round of the dies), so that the last ones of either share the chip
// (12544 x 768 by 768, bf16: 56 us, 37 + 32 one after the other; float32, 7755 x 200 by
// 97 maps: 17, 12 + 11).
struct PairParams {
    GemmParams dx, dw;
    unsigned first, dw_room;  // dw's total, rounded up to the 8 dies
};
template <typename T, bool X_MAPS, bool Y_MAPS, int BM, bool STRAIGHT>
__global__ __launch_bounds__(256, 2) void gemm_pair(const PairParams p)
{
    constexpr bool A_KC = !X_MAPS && !Y_MAPS, B_KC = X_MAPS && !Y_MAPS;  // (dx: dz by weight^T, of maps weight^T by dz)
    const unsigned id = p.first + blockIdx.x;
    if (id >= p.dw.total && id < p.dw_room) return;
    if constexpr (STRAIGHT) {
        __shared__ __align__(16) uint16_t ring0[kRingElems<BM, BM>], ring1[kRingElems<BM, BM>];
        if (id < p.dw.total) gemm_by_lds<Y_MAPS, X_MAPS, BM, BM, true>(p.dw, id, ring0, ring1);
        else gemm_by_lds<A_KC, B_KC, BM, BM, false>(p.dx, id - p.dw_room, ring0, ring1);
    } else {
        __shared__ __align__(16) uint16_t tiles[kTileElems<T, A_KC, B_KC, BM, BM>];
        if (id < p.dw.total) gemm_by_registers<T, Y_MAPS, X_MAPS, BM, BM, true>(p.dw, id, tiles);
        else gemm_by_registers<T, A_KC, B_KC, BM, BM, false>(p.dx, id - p.dw_room, tiles);
    }
}

// Adds the splits' sums, four threads a run of columns each every fourth, then
// those in order; then the epilogue. Workgroups behind them: sums of columns.
template <typename T>
__global__ __launch_bounds__(256) void gemm_join(const GemmParams p)
{
    constexpr int V = kWide<T>;
    __shared__ float sums[4][64][V + 1];
    if (p.first + blockIdx.x >= p.join_blocks) {
        float(&s)[16][17] = *reinterpret_cast<float(*)[16][17]>(sums);
        const int cx = threadIdx.x % 16, ry = threadIdx.x / 16, c = static_cast<int>(p.first + blockIdx.x - p.join_blocks) * 16 + cx;
        float v = 0.0f;
        if (c < p.fold_n) {
#pragma unroll 8
            for (int r = ry; r < p.fold_rows; r += 16) v += p.fold[static_cast<long>(r) * p.fold_n + c];
        }
        s[ry][cx] = v;
        __syncthreads();
        if (ry != 0 || c >= p.fold_n) return;
        v = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) v += s[r][cx];
        p.fold_to[c] = v;
        return;
    }
    const long ldp = (p.N + 3) / 4 * 4, runs = (p.N + V - 1) / V;
    const long i = static_cast<long>(p.first + blockIdx.x) * 64 + threadIdx.x % 64;
    const unsigned turn = threadIdx.x / 64;
    const bool live = i < p.batch * p.M * runs;
    const long row = i / runs;
    const int n = static_cast<int>(i % runs) * V, m = static_cast<int>(row % p.M);
    float v[V], bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = 0.0f;
    Raw<T, V> res;
    res.clear();
    if (live) {
#pragma unroll 8
        for (unsigned s = turn; s < p.splits; s += 4) {
            const float *part = p.part + (s * p.batch * p.M + row) * ldp + n;
#pragma unroll
            for (int k = 0; k < V / 4; ++k) {
                if (n + 4 * k >= p.N) continue;
                const facc f = *reinterpret_cast<const facc *>(part + 4 * k);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * k + j] += f[j];
            }
        }
        if (turn == 0) read_residual<T>(p, row / p.M, m, n, res);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) sums[turn][threadIdx.x % 64][j] = v[j];
    __syncthreads();
    if (turn != 0 || !live) return;
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = (v[j] + sums[1][threadIdx.x][j]) + (sums[2][threadIdx.x][j] + sums[3][threadIdx.x][j]);
    column_bias<T>(p, n, bias);
    finish<T, true>(p, row / p.M, m, n, v, bias, p.bias && p.bias_m ? p.bias[m] : 0.0f, res);
}

// ------------------------------------------------------------------ launches

constexpr long round_up_to(long v, long to) { return (v + to - 1) / to * to; }

// How a product is cut: the side of its tiles, and the parts of its sum. From its
// sizes alone, so that the workspace is known without the pointers.
struct GemmPlan {
    int bm, splits;
    int steps, per;
    int64_t bytes;  // of the splits' sums
    double us;      // as counted
    bool few;       // gemm_few
};

// The choice with the least time by this count, in us, of what was measured (bf16;
// float32): a workgroup alone takes 0.4 (1.1) a step of 64 x 64 and 0.8 (2.0) of
// 128 x 128, a compute unit full of them 0.22 (0.48) and 0.5 (1.4) for each; and parts
// cost 4 for the launch that joins them and their sums' way to memory and back.
// 768 x 768 over 12544 rows: 33 to 34 us of bf16 in 7 parts of 64 x 64 or 14 of 128 x 128, 115 and
// 193 undivided; 196 x 768 of 768: 7.4 us undivided, 11.5 in two parts. Short float32 sums of
// few steps are taken in tiles of 64, whose loads more workgroups keep under way
// (128 of 128 channels by 196608 cells: 84 us, 93 in tiles of 128).
struct GemmCost {
    double alone, full;  // of a workgroup alone, of the chip full of them
};
template <typename T>
GemmCost gemm_cost(const GemmPlan &g, long batch, long M, long N, int bm, int parts)
{
    constexpr bool kHalf = sizeof(T) == 2;
    const double tiles = static_cast<double>((M + bm - 1) / bm) * static_cast<double>((N + bm - 1) / bm) * static_cast<double>(batch);
    const double per = (g.steps + parts - 1) / parts;
    return {per * (bm == 64 ? (kHalf ? 0.4 : 1.1) : (kHalf ? 0.8 : 2.0)), per * tiles * parts / 256.0 * (bm == 64 ? (kHalf ? 0.22 : 0.48) : (kHalf ? 0.5 : 1.4))};
}
// What parts cost, or 0 of one; less than 0: not taken.
inline double parts_cost(const GemmPlan &g, long batch, long M, long N, int bm, int parts)
{
    if (parts == 1) return 0.0;
    const double tiles = static_cast<double>((M + bm - 1) / bm) * static_cast<double>((N + bm - 1) / bm) * static_cast<double>(batch);
    if ((g.steps + parts - 1) / parts < 4 || tiles * parts > 2048.0) return -1.0;
    return 4.0 + parts * static_cast<double>(batch) * static_cast<double>(M) * static_cast<double>(N) * 8.0 / 4e6;
}
constexpr int kGemmParts[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};

inline void cut_plan(GemmPlan &g, long batch, long M, long N, int bm, int parts)
{
    g.bm = bm;
    g.per = std::max((g.steps + parts - 1) / parts, 1);
    g.splits = std::max((g.steps + g.per - 1) / g.per, 1);
    g.bytes = g.splits > 1 ? static_cast<int64_t>(g.splits) * batch * M * round_up_to(N, 4) * 4 : 0;
}

template <typename T>
GemmPlan plan_gemm(long batch, long M, long N, long K, long kb)
{
    GemmPlan g{};
    g.steps = static_cast<int>((K + kStep<T> - 1) / kStep<T> * kb);  // (less than 2^31: checked at the entries)
    int side = 64, cuts = 1;
    g.us = -1.0;
    for (const int bm : {64, 128}) {
        if (bm == 128 && sizeof(T) == 4 && K <= 256 && kb == 1) continue;
        for (const int parts : kGemmParts) {
            const double extra = parts_cost(g, batch, M, N, bm, parts);
            if (extra < 0.0) continue;
            const GemmCost c = gemm_cost<T>(g, batch, M, N, bm, parts);
            const double us = std::max(c.alone, c.full) + extra;
            if (g.us < 0.0 || us < g.us) g.us = us, side = bm, cuts = parts;
        }
    }
    cut_plan(g, batch, M, N, side, cuts);
    return g;
}

// Whether rows are few, by the time gemm_few is counted to take (us): 2.1 and for each
// round of 256 workgroups 0.3 and 1.6 (float32 3.5) a thousand of k; the count of tiles is
// without their launch, 2.3 (1.5). (One row of 2048 to 8192 channels,
// bf16: 7.4 us, 10.8 by tiles; 32 rows: 17 and 12; 64 of 768 to 1536: 5.0 and 6.6.)
template <typename T>
bool few_rows(const GemmPlan &g, long M, long N, long K)
{
    const double rounds = std::ceil(static_cast<double>((M + 15) / 16) * static_cast<double>((N + 15) / 16) / 256.0);
    return 2.1 + rounds * (0.3 + static_cast<double>(K) * (sizeof(T) == 2 ? 0.0016 : 0.0035)) < g.us + (sizeof(T) == 2 ? 2.3 : 1.5);
}

// Both of a projection's gradients in one launch with tiles of one size, where
// that is counted to take less than one after the other (a launch is 3).
template <typename T>
bool plan_pair(GemmPlan &dx, GemmPlan &dw, long batch, long M, long N, long n, long k)
{
    double best = dx.us + dw.us + 3.0;
    bool pair = false;
    const GemmPlan x = dx, w = dw;
    for (const int bm : {64, 128})
        for (const int parts : kGemmParts) {
            const double extra = parts_cost(w, 1, n, k, bm, parts);
            if (extra < 0.0) continue;
            const GemmCost a = gemm_cost<T>(x, batch, M, N, bm, 1), b = gemm_cost<T>(w, 1, n, k, bm, parts);
            const double us = std::max({a.alone, b.alone, a.full + b.full}) + extra;
            if (us >= best) continue;
            best = us, pair = true;
            cut_plan(dx, batch, M, N, bm, 1);
            cut_plan(dw, 1, n, k, bm, parts);
        }
    return pair;
}

// A product as planned; ws: its parts' sums. Columns that p.fold names are summed too, in the joining launch or one more.
template <typename T>
int run_gemm(GemmParams p, const GemmPlan &g, bool a_kc, bool b_kc, void *ws, hipStream_t s);
// dx (undivided) and dw as planned together, in tiles of one size.
template <typename T>
int run_pair(GemmParams dx, const GemmPlan &gx, GemmParams dw, const GemmPlan &gw, bool x_maps, bool y_maps, void *ws, hipStream_t s);

template <typename F>
int gemm_launch(unsigned &at, long groups, F &&f)
{
    const long most = most_groups(256) / 8 * 8;
    for (long first = 0; first < groups; first += most) {
        at = static_cast<unsigned>(first);
        f(dim3(static_cast<unsigned>(std::min(groups - first, most))));
        const int st = launched();
        if (st != SSM2D_OK) return st;
    }
    return SSM2D_OK;
}

inline void lay_out(GemmParams &p, const GemmPlan &g, void *ws)
{
    p.splits = g.splits, p.steps = g.steps, p.per = g.per, p.part = static_cast<float *>(ws);
    p.tiles_m = (p.M + g.bm - 1) / g.bm, p.tiles_n = (p.N + g.bm - 1) / g.bm;
    p.total = p.tiles_m * p.tiles_n * static_cast<unsigned>(p.batch) * p.splits;
}

template <typename T>
int run_join(GemmParams &p, hipStream_t s)
{
    if (p.splits == 1 && !p.fold) return SSM2D_OK;
    const long blocks = p.splits == 1 ? 0 : (p.batch * p.M * ((p.N + kWide<T> - 1) / kWide<T>) + 63) / 64;
    p.join_blocks = static_cast<unsigned>(blocks);
    return gemm_launch(p.first, blocks + (p.fold ? (p.fold_n + 15) / 16 : 0), [&](dim3 grid) { gemm_join<T><<<grid, dim3(256), 0, s>>>(p); });
}

template <typename T>
int run_gemm_of(GemmParams p, const GemmPlan &g, bool a_kc, bool b_kc, void *ws, hipStream_t s)
{
    if (g.few) {
        p.tiles_n = (p.N + 15) / 16;
        return gemm_launch(p.first, static_cast<long>(p.tiles_n) * ((p.M + 15) / 16), [&](dim3 grid) { gemm_few<T><<<grid, dim3(512), 0, s>>>(p); });
    }
    lay_out(p, g, ws);
    auto go = [&](auto size) {
        constexpr int BM = decltype(size)::value;
        return gemm_launch(p.first, p.total, [&](dim3 grid) {
            if constexpr (sizeof(T) == 2) {
                if (p.straight) {
                    if (a_kc && b_kc) gemm_straight<true, true, BM, BM><<<grid, dim3(256), 0, s>>>(p);
                    else if (a_kc) gemm_straight<true, false, BM, BM><<<grid, dim3(256), 0, s>>>(p);
                    else if (b_kc) gemm_straight<false, true, BM, BM><<<grid, dim3(256), 0, s>>>(p);
                    else gemm_straight<false, false, BM, BM><<<grid, dim3(256), 0, s>>>(p);
                    return;
                }
            }
            if (a_kc && b_kc) gemm_kernel<T, true, true, BM, BM><<<grid, dim3(256), 0, s>>>(p);
            else if (a_kc) gemm_kernel<T, true, false, BM, BM><<<grid, dim3(256), 0, s>>>(p);
            else if (b_kc) gemm_kernel<T, false, true, BM, BM><<<grid, dim3(256), 0, s>>>(p);
            else gemm_kernel<T, false, false, BM, BM><<<grid, dim3(256), 0, s>>>(p);
        });
    };
    const int st = g.bm == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 64>{});
    return st == SSM2D_OK ? run_join<T>(p, s) : st;
}

template <typename T>
int run_pair_of(GemmParams dx, const GemmPlan &gx, GemmParams dw, const GemmPlan &gw, bool x_maps, bool y_maps, void *ws, hipStream_t s)
{
    lay_out(dx, gx, nullptr);
    lay_out(dw, gw, ws);
    PairParams p{dx, dw, 0, static_cast<unsigned>(round_up_to(dw.total, 8))};
    auto go = [&](auto size, auto straight) {
        constexpr int BM = decltype(size)::value;
        constexpr bool L = decltype(straight)::value;
        return gemm_launch(p.first, static_cast<long>(p.dw_room) + dx.total, [&](dim3 grid) {
            if (x_maps && y_maps) gemm_pair<T, true, true, BM, L><<<grid, dim3(256), 0, s>>>(p);
            else if (x_maps) gemm_pair<T, true, false, BM, L><<<grid, dim3(256), 0, s>>>(p);
            else if (y_maps) gemm_pair<T, false, true, BM, L><<<grid, dim3(256), 0, s>>>(p);
            else gemm_pair<T, false, false, BM, L><<<grid, dim3(256), 0, s>>>(p);
        });
    };
    auto sized = [&](auto straight) {
        return gw.bm == 128 ? go(std::integral_constant<int, 128>{}, straight) : go(std::integral_constant<int, 64>{}, straight);
    };
    int st;
    if constexpr (sizeof(T) == 2) st = dx.straight && dw.straight ? sized(std::true_type{}) : sized(std::false_type{});
    else st = sized(std::false_type{});
    return st == SSM2D_OK ? run_join<T>(dw, s) : st;
}

}  // namespace gemm
}  // namespace ssm2d_impl
