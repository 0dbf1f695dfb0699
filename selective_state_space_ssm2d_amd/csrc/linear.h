// libssm2d: matrix products with an epilogue (include/ssm2d_block.h, linear):
//   C[m][n] = sum_k A[m][k] B[n][k], then bias, activation, residual,
// C's n contiguous in memory, A and B each with k or with m (n) contiguous. Token
// rows and channels-first maps, forward and both gradients, are such products
// with the sides chosen (linear.hip).
#pragma once

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
    int tiles_m, tiles_n;
    long batch;
    int splits;       // parts of the sum, each by workgroups of its own
    long steps, per;  // steps of BK in all stretches, and of one split
    // epilogue
    const float *bias;  // along n, or with bias_m along m
    int bias_m, act;
    const void *res;
    long r_ld, r_bs;
    void *c, *pre;
    long c_ld, c_bs;
    int straight;     // bf16 operands can be loaded straight to LDS
    float *part;      // splits > 1: [split][batch][M][N rounded up to 4]
    long first;       // the launch's first workgroup
};

template <typename T>
constexpr int kParts = sizeof(T) == 2 ? 1 : 3;
template <typename T>
constexpr int kStep = sizeof(T) == 2 ? 64 : 32;  // k of a step

// ------------------------------------------------------------------ epilogue

template <typename T, int ACT>
__device__ __forceinline__ void act4(float (&v)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = activate<T, ACT>(v[j]);
}

// Four neighbours of row m from column n on.
template <typename T>
__device__ __forceinline__ void finish4(const GemmParams &p, long b, int m, int n, float (&v)[4])
{
    if (m >= p.M || n >= p.N) return;
    if (p.bias) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += p.bias[p.bias_m ? m : min(n + j, p.N - 1)];
    }
    const long at = b * p.c_bs + static_cast<long>(m) * p.c_ld + n;
    T *c = static_cast<T *>(p.c) + at;
    const bool four = n + 4 <= p.N;
    auto put = [&](T *dst) __attribute__((always_inline)) {
        if (four) {
            Raw<T, 4> r;
            r.set(v);
            r.store_any(dst);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < p.N) store1(dst + j, v[j]);
        }
    };
    if (p.pre) put(static_cast<T *>(p.pre) + at);
    switch (p.act) {
    case SSM2D_ACT_RELU: act4<T, SSM2D_ACT_RELU>(v); break;
    case SSM2D_ACT_SILU: act4<T, SSM2D_ACT_SILU>(v); break;
    case SSM2D_ACT_GELU: act4<T, SSM2D_ACT_GELU>(v); break;
    default: break;
    }
    if (p.res) {
        const T *r = static_cast<const T *>(p.res) + b * p.r_bs + static_cast<long>(m) * p.r_ld + n;
        if (four) {
            Raw<T, 4> w;
            w.load_any(r);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += w.get(j);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < p.N) v[j] += widen1(r[j]);
        }
    }
    put(c);
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

// Eight elements of an operand on their way from memory to LDS.
template <typename T>
struct Chunk {
    Raw<T, 8> r;
    // the first `count` of the 8 at p (0 or less: none), the others 0
    __device__ __forceinline__ void load(const T *p, long count)
    {
        if (count >= 8) {
            r.load_any(p);
        } else if (count > 0) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = widen1(p[min(i, static_cast<int>(count) - 1)]);
#pragma unroll
            for (int i = 1; i < 8; ++i) v[i] = i < count ? v[i] : 0.0f;
            r.set(v);
        } else {
            r.clear();
        }
    }
    // as NP parts, kPart elements apart
    __device__ __forceinline__ void store(uint16_t *dst, int part) const
    {
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        } else {
            // three parts of 8 bits each, cut off: exact
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = r.get(i);
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                unsigned w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const unsigned lo = __float_as_uint(v[2 * i]), hi = __float_as_uint(v[2 * i + 1]);
                    w[i] = top_halves(hi, lo);
                    v[2 * i] -= __uint_as_float(lo & 0xffff0000u);
                    v[2 * i + 1] -= __uint_as_float(hi & 0xffff0000u);
                }
                *reinterpret_cast<uint4 *>(dst + n * part) = make_uint4(w[0], w[1], w[2], w[3]);
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
__device__ __forceinline__ TilePlace tile_place(const GemmParams &p)
{
    const long total = static_cast<long>(p.tiles_m) * p.tiles_n * p.batch * p.splits;
    long id = p.first + blockIdx.x;
    const long each = total / 8, more = total % 8, die = id % 8;
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

template <typename T, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void finish_tile(const GemmParams &p, const TilePlace &t, facc (&acc)[WM / 16][WN / 16])
{
    const int l = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int m0 = t.m0 + wave / (BN / WN) * WM + l % 16, n0 = t.n0 + wave % (BN / WN) * WN + 4 * (l / 16);
    const long ldp = (p.N + 3) / 4 * 4;
#pragma unroll
    for (int i = 0; i < WM / 16; ++i)
#pragma unroll
        for (int j = 0; j < WN / 16; ++j) {
            const int m = m0 + i * 16, n = n0 + j * 16;
            if (p.splits > 1) {
                if (m < p.M && n < p.N)
                    *reinterpret_cast<facc *>(p.part + ((t.split * p.batch + t.b) * p.M + m) * ldp + n) = acc[i][j];
            } else {
                float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
                finish4<T>(p, t.b, m, n, v);
            }
        }
}

// Any alignment: operands go through registers to LDS, the next step's read
// while this one's products run.
template <typename T, bool A_KC, bool B_KC, int BM, int BN>
__global__ __launch_bounds__(256) void gemm_kernel(const GemmParams p)
{
    constexpr int NP = kParts<T>, BK = kStep<T>, WM = BM / 2, WN = BN / 2;
    using TA = OperandTile<A_KC, BM, BK, NP>;
    using TB = OperandTile<B_KC, BN, BK, NP>;
    __shared__ __align__(16) uint16_t sa[TA::kElems], sb[TB::kElems];
    const TilePlace t = tile_place<BM, BN>(p);
    const T *A = static_cast<const T *>(p.a), *B = static_cast<const T *>(p.b);
    if (p.kb == 1) A += t.b * p.a_bs, B += t.b * p.b_bs;
    const long s1 = t.split * p.per, s2 = min(s1 + p.per, p.steps), each = (p.K + BK - 1) / BK;
    constexpr int CA = BM * BK / 8 / 256, CB = BN * BK / 8 / 256;
    Chunk<T> ra[CA], rb[CB];
    auto fetch = [&](long s) __attribute__((always_inline)) {
        const long kb = p.kb == 1 ? 0 : s / each, k0 = (s - kb * each) * BK;
        const T *ap = A + kb * p.a_bs, *bp = B + kb * p.b_bs;
        if (p.kb == 1) ap = A, bp = B;
        auto side = [&](auto kc, const T *src, long ld, int r0, int rows, auto &reg, auto row_len) __attribute__((always_inline)) {
            constexpr int kChunks = decltype(row_len)::value / 8;
#pragma unroll
            for (int i = 0; i < static_cast<int>(sizeof(reg) / sizeof(reg[0])); ++i) {
                const int id = i * 256 + threadIdx.x, row = id / kChunks, col = id % kChunks * 8;
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
    if (s1 < s2) fetch(s1);
    for (long s = s1; s < s2; ++s) {
        __syncthreads();  // (the last step's tiles have been read)
#pragma unroll
        for (int i = 0; i < CA; ++i) {
            const int id = i * 256 + threadIdx.x;
            ra[i].store(sa + TA::at(id / TA::kChunks, id % TA::kChunks), TA::kPart);
        }
#pragma unroll
        for (int i = 0; i < CB; ++i) {
            const int id = i * 256 + threadIdx.x;
            rb[i].store(sb + TB::at(id / TB::kChunks, id % TB::kChunks), TB::kPart);
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
            }
        }
    }
    finish_tile<T, BM, BN, WM, WN>(p, t, acc);
}

// ------------------------------------------------------------------ straight to LDS

constexpr unsigned kNowhere = 0x80000000u;  // an offset behind every buffer: its load gives zeros

// One operand's loads of a step, from memory straight to LDS: 16 bytes a lane,
// 64 lanes a kilobyte of the tile in the order of its places. The turn of a
// chunk (OperandTile) is in which chunk a lane asks for.
template <bool KC, int R>
struct StraightLoads {
    using Tile = OperandTile<KC, R, 64, 1>;
    static constexpr int kLoads = R * 8 / 256;               // a thread's, of a step of 64
    static constexpr int kRowsEach = 256 / Tile::kChunks;    // rows of the tile that 256 lanes cover
    const uint16_t *base;                                    // the tile's first row (KC) or column
    long ld;
    int K;
    unsigned off[KC ? kLoads : 1];
    int col;                                                 // KC: the lane's first k
    __device__ __forceinline__ void begin(const uint16_t *src, long ld_, int r0, int rows, int K_)
    {
        ld = ld_, K = K_;
        const int row = threadIdx.x / Tile::kChunks, c = (threadIdx.x % Tile::kChunks) ^ Tile::turn(row);
        if constexpr (KC) {
            base = src + r0 * ld, col = c * 8;
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                off[i] = r0 + i * kRowsEach + row < rows ? static_cast<unsigned>(i * kRowsEach + row) * static_cast<unsigned>(ld * 2) + c * 16 : kNowhere;
        } else {
            base = src + r0, col = 0;
            off[0] = r0 + c * 8 < rows ? static_cast<unsigned>(row) * static_cast<unsigned>(ld * 2) + c * 16 : kNowhere;
        }
    }
    // k0 .. k0 + 63 of the stretch that lies `at` elements on
    __device__ __forceinline__ void issue(uint16_t *tile, long at, int k0) const
    {
        using lds = __attribute__((address_space(3))) void;
        const int left = K - k0;
        const uint16_t *src = base + at + (KC ? static_cast<long>(k0) : k0 * ld);
        // (of the last rows of k no more than there are)
        const unsigned bytes = KC || left >= 64 ? 0x7fffffffu : static_cast<unsigned>(left) * static_cast<unsigned>(ld * 2);
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(src), 0, static_cast<int>(bytes), 0x00020000);
        uint16_t *dst = tile + threadIdx.x / 64 * 512;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const unsigned o = KC ? (left >= 64 || col < left ? off[i] : kNowhere) : off[0];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds *)(dst + i * 2048), 16, static_cast<int>(o),
                                                     KC ? 0 : static_cast<int>(i * kRowsEach * ld * 2), 0, 0);
        }
    }
};

// bf16 operands whose rows are whole 16-byte chunks: two stages of tiles in LDS,
// one filled by loads that pass the registers by while the other is used.
template <bool A_KC, bool B_KC, int BM, int BN>
__global__ __launch_bounds__(256) void gemm_straight(const GemmParams p)
{
    constexpr int WM = BM / 2, WN = BN / 2;
    using TA = OperandTile<A_KC, BM, 64, 1>;
    using TB = OperandTile<B_KC, BN, 64, 1>;
    // (variables of their own, so that a read waits for its own stage's loads alone)
    __shared__ __align__(16) uint16_t a0[TA::kElems], b0[TB::kElems], a1[TA::kElems], b1[TB::kElems];
    const TilePlace t = tile_place<BM, BN>(p);
    const uint16_t *A = static_cast<const uint16_t *>(p.a), *B = static_cast<const uint16_t *>(p.b);
    if (p.kb == 1) A += t.b * p.a_bs, B += t.b * p.b_bs;
    StraightLoads<A_KC, BM> la;
    StraightLoads<B_KC, BN> lb;
    la.begin(A, p.a_ld, t.m0, p.M, p.K);
    lb.begin(B, p.b_ld, t.n0, p.N, p.K);
    const long s1 = t.split * p.per, s2 = min(s1 + p.per, p.steps), each = (p.K + 63) / 64;
    auto issue = [&](long s, uint16_t *a, uint16_t *b) __attribute__((always_inline)) {
        const long kb = p.kb == 1 ? 0 : s / each;
        const int k0 = static_cast<int>((s - kb * each) * 64);
        la.issue(a, kb * p.a_bs, k0);
        lb.issue(b, kb * p.b_bs, k0);
    };
    facc acc[WM / 16][WN / 16];
#pragma unroll
    for (auto &r : acc)
#pragma unroll
        for (auto &v : r) v = facc{0.0f, 0.0f, 0.0f, 0.0f};
    const int wave = threadIdx.x / 64, wm = wave / 2 * WM, wn = wave % 2 * WN;
    auto step = [&](const uint16_t *a, const uint16_t *b) __attribute__((always_inline)) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            bfrag fb[WN / 16], fa[WM / 16];
#pragma unroll
            for (int j = 0; j < WN / 16; ++j) fb[j] = TB::frag(b, 0, wn + j * 16, ks);
#pragma unroll
            for (int i = 0; i < WM / 16; ++i) fa[i] = TA::frag(a, 0, wm + i * 16, ks);
#pragma unroll
            for (int i = 0; i < WM / 16; ++i)
#pragma unroll
                for (int j = 0; j < WN / 16; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
        }
    };
    if (s1 < s2) issue(s1, a0, b0);
    for (long s = s1; s < s2; s += 2) {
        __syncthreads();  // (stage 0 is there, and stage 1 has been read)
        if (s + 1 < s2) issue(s + 1, a1, b1);
        step(a0, b0);
        __syncthreads();
        if (s + 2 < s2) issue(s + 2, a0, b0);
        if (s + 1 < s2) step(a1, b1);
    }
    finish_tile<uint16_t, BM, BN, WM, WN>(p, t, acc);
}

// Adds the splits' sums in order, then the epilogue.
template <typename T>
__global__ __launch_bounds__(256) void gemm_join(const GemmParams p)
{
    const long ldp = (p.N + 3) / 4 * 4, quads = ldp / 4;
    const long i = (p.first + blockIdx.x) * 256 + threadIdx.x;
    if (i >= p.batch * p.M * quads) return;
    const long row = i / quads;
    facc sum = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < p.splits; ++s) sum += *reinterpret_cast<const facc *>(p.part + (s * p.batch * p.M + row) * ldp + i % quads * 4);
    float v[4] = {sum[0], sum[1], sum[2], sum[3]};
    finish4<T>(p, row / p.M, static_cast<int>(row % p.M), static_cast<int>(i % quads) * 4, v);
}

// ------------------------------------------------------------------ launches

constexpr long round_up_to(long v, long to) { return (v + to - 1) / to * to; }

// How a product is cut. From its sizes alone, so that the workspace is known without the pointers.
struct GemmPlan {
    int bm, splits;
    long steps, per;
    int64_t bytes;  // of the splits' sums
};
template <typename T>
GemmPlan plan_gemm(long batch, long M, long N, long K, long kb)
{
    GemmPlan g{};
    auto tiles = [&](long t) { return static_cast<double>((M + t - 1) / t) * static_cast<double>((N + t - 1) / t) * static_cast<double>(batch); };
    g.steps = (K + kStep<T> - 1) / kStep<T> * kb;
    g.bm = tiles(128) >= 256 ? 128 : 64;
    g.splits = 1;
    const double have = tiles(g.bm);
    if (have < 384 && g.steps >= 8) g.splits = static_cast<int>(std::min<double>(std::min<long>(g.steps / 4, 64), 768.0 / std::max(have, 1.0)));
    g.splits = std::max(g.splits, 1);
    g.per = (g.steps + g.splits - 1) / g.splits;
    g.splits = static_cast<int>(std::max<long>((g.steps + g.per - 1) / std::max<long>(g.per, 1), 1));
    g.bytes = g.splits > 1 ? static_cast<int64_t>(g.splits) * batch * M * round_up_to(N, 4) * 4 : 0;
    return g;
}

template <typename T>
int run_gemm(GemmParams p, bool a_kc, bool b_kc, void *ws, hipStream_t s);

template <typename F>
int gemm_launch(GemmParams &p, long groups, F &&f)
{
    const long most = most_groups(256) / 8 * 8;
    for (p.first = 0; p.first < groups; p.first += most) {
        f(dim3(static_cast<unsigned>(std::min(groups - p.first, most))));
        const int st = launched();
        if (st != SSM2D_OK) return st;
    }
    return SSM2D_OK;
}

#define SSM2D_DEFINE_RUN_GEMM(T)                                                                                     \
    template <>                                                                                                      \
    int run_gemm<T>(GemmParams p, bool a_kc, bool b_kc, void *ws, hipStream_t s)                                     \
    {                                                                                                                \
        return run_gemm_of<T>(p, a_kc, b_kc, ws, s);                                                                 \
    }

template <typename T>
int run_gemm_of(GemmParams p, bool a_kc, bool b_kc, void *ws, hipStream_t s)
{
    const GemmPlan g = plan_gemm<T>(p.batch, p.M, p.N, p.K, p.kb);
    p.splits = g.splits, p.steps = g.steps, p.per = g.per, p.part = static_cast<float *>(ws);
    auto go = [&](auto size) {
        constexpr int BM = decltype(size)::value;
        p.tiles_m = (p.M + BM - 1) / BM, p.tiles_n = (p.N + BM - 1) / BM;
        return gemm_launch(p, static_cast<long>(p.tiles_m) * p.tiles_n * p.batch * p.splits, [&](dim3 grid) {
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
    int st = g.bm == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 64>{});
    if (st == SSM2D_OK && p.splits > 1) {
        const long quads = p.batch * p.M * (round_up_to(p.N, 4) / 4);
        st = gemm_launch(p, (quads + 255) / 256, [&](dim3 grid) { gemm_join<T><<<grid, dim3(256), 0, s>>>(p); });
    }
    return st;
}

}  // namespace gemm
}  // namespace ssm2d_impl
