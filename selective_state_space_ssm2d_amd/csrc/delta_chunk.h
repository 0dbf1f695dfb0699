// libssm2d: the gated delta rule in chunks of 64 tokens, forward and backward.
//
// With G_i the running sum of g over a chunk, gamma_i = e^G_i and
// Gam_ij = e^(G_i - G_j), a chunk that starts from S0 has (rows = tokens)
//   R = V - gamma K S0,   N_ij = Gam_ij k_i . k_j (j < i),   B = diag(beta)
//   E = (I + N B)^-1 R,   U = B E
//   O = scale (gamma Q S0 + P U),   P_ij = Gam_ij q_i . k_j (j <= i)
//   S1 = gamma_last S0 + K^T (Gam_last U)
// With M = (I + N B)^-1 N (strictly lower; no division by beta) both inverses
// the passes need are products: E = R - M (B R), and for the adjoint of U,
// dR = dU - M^T (B dU). Given dO and the adjoint D1 of S1:
//   dU = scale P^T dO + Gam_last K D1
//   dV = B dR,   dbeta_i = dR_i . E_i
//   D0 = gamma_last D1 + Q^T (scale gamma dO) - K^T (gamma B dR)
// and, with Pd_ij = scale Gam_ij dO_i . U_j (j <= i) and
// Nd_ij = -beta_i Gam_ij dR_i . U_j (j < i),
//   dQ = scale gamma dO S0^T + Pd K
//   dK = Rk + Ck,   Rk = -gamma B dR S0^T + Nd K,   Ck = Gam_last U D1^T + Pd^T Q + Nd^T K
//   dG_i = q_i . dQ_i + k_i . Rk_i - k_i . Ck_i, and at the chunk's end
//   also gamma_last <S0, D1> + sum_j k_j . (Gam_last U D1^T)_j;  dg = suffix sums of dG.
//
// Kernels: delta_prep (per chunk: the gates, M and for the forward P), delta_z
// (scale P^T dO), delta_seq (the chain over chunks: in the forward O as it goes,
// in the backward S0 and E, and at the same time the chain of adjoints, D1 and
// dR), delta_join (first states of the chains' segments) and delta_local (the
// gradients of a chunk). Only delta_seq and delta_join are sequential.
//
// What bounds them is not memory (4 heads of 32 x 32 over 196608 tokens, fp32, have
// 409 MB to move, 80 us, and take 430): a chunk's step is a chain of products of
// one wave's 16 columns, each waiting for the one before, and cutting operands
// into parts takes twice the issue cycles of the matrix instructions (SQ
// counters: of delta_seq's wave cycles 25 to 43 % issue vector instructions, 14 to 21
// matrix ones, 27 to 42 wait).
//
// Precision: an fp32 operand goes through the matrix cores as the sum of
// three bf16 parts, cut off exactly (8 + 8 + 8 bits); products keep six
// terms, and the three left out are under 2^-21 of the product and of its sign, at 6/16
// of the matrix instructions' time of fp32. bf16 inputs are one part (three
// terms against an fp32 operand). Outputs are rounded once, from sums like these.
//
// Fragments: v_mfma_f32_16x16x32_bf16 with lane l holding row (column) l % 16
// and, of the 32 summed indices, 4 (l / 16) + j and 16 + 4 (l / 16) + j, j < 4.
// That is the order in which the accumulators of two stacked 16 x 16 tiles
// lie, so a result becomes the next product's operand in registers; LDS tiles
// give it by two 8-byte reads along rows, or two transposing reads down rows.
#pragma once

#include "delta.h"
#include "delta_plan.h"

namespace ssm2d_impl {

using word4 = unsigned __attribute__((ext_vector_type(4)));  // (a register value; the uint4 struct is copied through memory)

struct ChunkParams : Cuts {
    const void *q, *k, *v, *dout;
    const float *g, *beta, *h_init, *dh_last;
    void *o, *dq, *dk, *dv;
    float *h_last, *dg, *dbeta, *dh_init;
    // workspace, by [slot][head of this pass]
    float *gates;                       // [5][kC]: gamma, Gam_last, beta, G and its rounding error
    // -M, -M^T and P: their 10 tiles that are not zero, as operands: row lane % 16, columns 4 (lane / 16) + j
    float *m, *mt, *pm;
    // (matrices as accumulator tiles: 16 columns after 16, of each 16 rows after
    // 16, of each the 64 lanes' four values: column lane % 16, rows 4 (lane / 16) + j)
    float *s0, *d1;                     // [KD][dvp]
    float *e, *dr, *z;                  // [kC][dvp]
    // by [place of a segment][head of this pass]: a segment's transition
    // [KD][KD] (as operands of its columns, for adjoints, and of its rows, in three
    // parts), its state from zero and then its first state (forward and adjoint)
    // [KD][dvp]
    word4 *seg_a, *seg_at;
    float *seg_s, *seg_d;
    float *sum;                         // dQ and dK of shared heads so far, by [slot][key head]
    int turn;                           // which of the heads that share a key head (delta_local)
    int hk, h, rep, dk_, dv_, dvp;
    int hk0, nhk, nh;                   // this pass: key heads hk0 .. hk0 + nhk - 1, nh = nhk * rep heads
    long qs[3], ks[3], vs[3], os[3], gs[3], bs[3];
    float scale;
    int vec_qk, vec_do, vec_v;          // rows of q and k, of dout, of v can be read 16 bytes at a time
    int vec_o, vec_dqk;                 // rows of o, of dq and dk can be written four elements at a time
};

// 16-byte words of 16 rows (columns) of a segment's transition
template <int KD>
constexpr int kSegTile = KD / 32 * 3 * 64;

using bfrag = __bf16 __attribute__((ext_vector_type(8)));
using facc = float __attribute__((ext_vector_type(4)));
using half4 = short __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ parts

__device__ __forceinline__ unsigned top16(unsigned hi, unsigned lo) { return __builtin_amdgcn_perm(hi, lo, 0x07060302u); }

// N parts of two values, each part's pair in one word.
template <int N>
__device__ __forceinline__ void split2(float a, float b, unsigned (&w)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const unsigned ua = __float_as_uint(a), ub = __float_as_uint(b);
        w[i] = top16(ub, ua);
        if (i + 1 < N) {
            a -= __uint_as_float(ua & 0xffff0000u);
            b -= __uint_as_float(ub & 0xffff0000u);
        }
    }
}

union FragBits {
    bfrag f;
    unsigned w[4];
    word4 q;
    half4 h[2];
};

// The operand that two stacked accumulator tiles make.
template <int N>
__device__ __forceinline__ void split_acc(const facc &lo, const facc &hi, bfrag (&f)[N])
{
    FragBits b[N];
    unsigned w[N];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        split2<N>(lo[2 * i], lo[2 * i + 1], w);
#pragma unroll
        for (int n = 0; n < N; ++n) b[n].w[i] = w[n];
        split2<N>(hi[2 * i], hi[2 * i + 1], w);
#pragma unroll
        for (int n = 0; n < N; ++n) b[n].w[2 + i] = w[n];
    }
#pragma unroll
    for (int n = 0; n < N; ++n) f[n] = b[n].f;
}

// 4 x 4 values of four neighbouring lanes, turned: lane b's j-th was lane j's b-th.
__device__ __forceinline__ facc turn4(facc v)
{
    const int b = threadIdx.x % 4;
    auto swap = [&](int i, int j, bool high, auto ctrl) __attribute__((always_inline)) {
        const float r = __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(high ? v[i] : v[j]), decltype(ctrl)::value, 0xf, 0xf, true));
        if (high) v[i] = r;
        else v[j] = r;
    };
    constexpr std::integral_constant<int, 0xb1> one{};  // lanes 1 apart
    constexpr std::integral_constant<int, 0x4e> two{};  // lanes 2 apart
    swap(0, 1, b & 1, one);
    swap(2, 3, b & 1, one);
    swap(0, 2, b & 2, two);
    swap(1, 3, b & 2, two);
    return v;
}

// acc += a b over the parts whose product reaches the last place kept.
template <int NA, int NB>
__device__ __forceinline__ void mma(facc &acc, const bfrag (&a)[NA], const bfrag (&b)[NB])
{
    constexpr int kMax = NA > NB ? NA : NB;
#pragma unroll
    for (int s = kMax - 1; s >= 0; --s)  // small terms first
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = s - i;
            if (j >= 0 && j < NB) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc, 0, 0, 0);
        }
}

// acc[t] += a[t] b for all t, the same terms: one term of every t before the
// next, so that no product waits for the one before it.
template <int NA, int NB, int NT>
__device__ __forceinline__ void mma_each(facc (&acc)[NT], const bfrag (&a)[NT][NA], const bfrag (&b)[NB])
{
    constexpr int kMax = NA > NB ? NA : NB;
#pragma unroll
    for (int s = kMax - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = s - i;
            if (j < 0 || j >= NB) continue;
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][i], b[j], acc[t], 0, 0, 0);
        }
}

// The same with the operands' sides changed: acc[t]^T += b^T a[t]^T.
template <int NA, int NB, int NT>
__device__ __forceinline__ void mma_each_t(facc (&acc)[NT], const bfrag (&a)[NT][NA], const bfrag (&b)[NB])
{
    constexpr int kMax = NA > NB ? NA : NB;
#pragma unroll
    for (int s = kMax - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = s - i;
            if (j < 0 || j >= NB) continue;
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], a[t][i], acc[t], 0, 0, 0);
        }
}

// Two or three sums whose terms take turns, so that none waits for itself.
template <int NP>
__device__ __forceinline__ void mma_turns(facc &q, const bfrag (&fq)[NP], facc &r, const bfrag (&fr)[3], const bfrag (&a)[3], facc &c,
                                          const bfrag (&d)[3], const bfrag (&fc)[3])
{
#pragma unroll
    for (int s = 2; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i) {
            r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], fr[s - i], r, 0, 0, 0);
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(d[i], fc[s - i], c, 0, 0, 0);
            if (s - i < NP) q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], fq[s - i], q, 0, 0, 0);
        }
}
template <int NA, int NB, int NC, int ND>
__device__ __forceinline__ void mma_two(facc &x, const bfrag (&a)[NA], const bfrag (&b)[NB], facc &y, const bfrag (&c)[NC], const bfrag (&d)[ND])
{
    constexpr int kX = NA > NB ? NA : NB, kY = NC > ND ? NC : ND, kMax = kX > kY ? kX : kY;
#pragma unroll
    for (int s = kMax - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i <= s; ++i) {
            if (s < kX && i < NA && s - i < NB) x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[s - i], x, 0, 0, 0);
            if (s < kY && i < NC && s - i < ND) y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(c[i], d[s - i], y, 0, 0, 0);
        }
}

// A workgroup barrier for what goes through LDS alone: unlike __syncthreads it
// does not wait for global loads and stores still in flight.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The LDS address behind a pointer into it: its low half (a cast between the
// address spaces would test for null first).
__device__ __forceinline__ unsigned lds_offset(const void *p) { return static_cast<unsigned>(reinterpret_cast<uintptr_t>(p)); }

// A tile in LDS: NP parts of [ROWS][COLS] bf16, rows padded by 16 bytes (the
// 16 rows of a fragment then start 4 banks apart, both ways of reading).
template <int NP, int ROWS, int COLS>
struct Tile {
    static constexpr int kLd = COLS + 8, kPart = ROWS * kLd, kBytes = NP * kPart * 2;
    uint16_t *p;
    // rows r0 .. r0 + 15, summed index along the rows from c0
    __device__ __forceinline__ void rows(int r0, int c0, bfrag (&f)[NP]) const
    {
        const int l = threadIdx.x % 64;
        const uint16_t *a = p + (r0 + l % 16) * kLd + c0 + 4 * (l / 16);
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            FragBits b;
            b.h[0] = *reinterpret_cast<const half4 *>(a + n * kPart);
            b.h[1] = *reinterpret_cast<const half4 *>(a + n * kPart + 16);
            f[n] = b.f;
        }
    }
    // columns c0 .. c0 + 15, summed index down the rows from r0
    __device__ __forceinline__ void cols(int r0, int c0, bfrag (&f)[NP]) const
    {
        using lds4 = __attribute__((address_space(3))) half4 *;
        const int l = threadIdx.x % 64;
        const unsigned at = lds_offset(p + (r0 + 4 * (l / 16) + (l % 16) / 4) * kLd + c0 + 4 * (l % 4));
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            FragBits b;
            b.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at + n * kPart * 2));
            b.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(at + (n * kPart + 16 * kLd) * 2));
            f[n] = b.f;
        }
    }
    // four neighbours of a row
    __device__ __forceinline__ void put4(int r, int c, float x0, float x1, float x2, float x3) const
    {
        unsigned a[NP], b[NP];
        split2<NP>(x0, x1, a);
        split2<NP>(x2, x3, b);
#pragma unroll
        for (int n = 0; n < NP; ++n) *reinterpret_cast<uint2 *>(p + n * kPart + r * kLd + c) = make_uint2(a[n], b[n]);
    }
    __device__ __forceinline__ void get4(int r, int c, float (&x)[4]) const
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = 0.0f;
#pragma unroll
        for (int n = NP - 1; n >= 0; --n) {
            const uint2 w = *reinterpret_cast<const uint2 *>(p + n * kPart + r * kLd + c);
            x[0] += bf16_lo(w.x), x[1] += bf16_hi(w.x), x[2] += bf16_lo(w.y), x[3] += bf16_hi(w.y);
        }
    }
};

template <typename T>
constexpr int kParts = sizeof(T) == 2 ? 1 : 3;  // parts of an input

// ------------------------------------------------------------------ staging

// A chunk's rows of q, k or dO (COLS wide, zeros past n and past the chunk):
// read to registers, later put into LDS. Places outside are read at the nearest
// one inside (len >= 1, n >= 1) and cleared when they are put: anything that
// looks at a load's result right after it would wait for it there.
template <typename T, int COLS, int THREADS>
struct Stage {
    static constexpr int N = 16 / static_cast<int>(sizeof(T)), kRow = COLS / N, kAll = kC * kRow, kEach = (kAll + THREADS - 1) / THREADS;
    word4 r[kEach];
    int len, n;
    __device__ __forceinline__ void load(const T *base, long stride, int len_, int n_, bool vec)
    {
        len = len_, n = n_;
        if (vec) {  // (n is a multiple of N)
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int at = i * THREADS + threadIdx.x, row = at / kRow, c = (at % kRow) * N;
                r[i] = *reinterpret_cast<const word4 *>(base + min(row, len - 1) * stride + min(c, n - N));
            }
        } else {
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int at = i * THREADS + threadIdx.x, row = at / kRow, c = (at % kRow) * N;
                r[i] = gather(base + min(row, len - 1) * stride, c, n);
            }
        }
    }
    // 16 bytes element by element; past n: the last element
    static __device__ __forceinline__ word4 gather(const T *src, int c, int n)
    {
        unsigned w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 2) w[j] = src[min(c + 2 * j, n - 1)] | (static_cast<unsigned>(src[min(c + 2 * j + 1, n - 1)]) << 16);
            else w[j] = __float_as_uint(src[min(c + j, n - 1)]);
        }
        return word4{w[0], w[1], w[2], w[3]};
    }
    __device__ __forceinline__ void put(const Tile<kParts<T>, kC, COLS> &t) const
    {
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = i * THREADS + threadIdx.x, row = at / kRow, c = (at % kRow) * N;
            if (kAll % THREADS != 0 && at >= kAll) continue;
            const int left = row < len ? n - c : 0;  // elements that are inside
            unsigned w[4] = {r[i][0], r[i][1], r[i][2], r[i][3]};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 2) w[j] = left > 2 * j + 1 ? w[j] : (left > 2 * j ? w[j] & 0xffffu : 0u);
                else w[j] = left > j ? w[j] : 0u;
            }
            if constexpr (sizeof(T) == 2) *reinterpret_cast<word4 *>(t.p + row * t.kLd + c) = word4{w[0], w[1], w[2], w[3]};
            else t.put4(row, c, __uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]));
        }
    }
};

// ------------------------------------------------------------------ gates

// gamma, Gam_last, beta, G's two parts of a chunk into out[5][kC], by the
// first wave. G is summed in fp64 and kept as two floats in units of log 2 (the
// hardware's exponential, exact to a unit of the last place, takes powers of
// two), so that differences of large sums stay exact. Below -1e4 a decay is 0 in any sum: held there,
// so that -inf gives 0 and not inf - inf.
// g and beta of the chunk's tokens, one a lane of the first wave (clamped reads;
// tokens past the end count as g = beta = 0).
struct GateIn {
    float g, b;
    __device__ __forceinline__ void load(const ChunkParams &p, const Place &c, int head)
    {
        const long t = c.t0 + min(static_cast<int>(threadIdx.x), c.len - 1);
        g = p.g[c.b * p.gs[0] + t * p.gs[1] + head * p.gs[2]];
        b = p.beta[c.b * p.bs[0] + t * p.bs[1] + head * p.bs[2]];
    }
};
__device__ __forceinline__ void make_gates(const Place &c, const GateIn &in, float *out)
{
    const int i = threadIdx.x;
    if (i >= kC) return;
    const float g = i < c.len ? (in.g < -1e4f ? -1e4f : in.g) : 0.0f, b = i < c.len ? in.b : 0.0f;
    double s = g * 1.4426950408889634;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        const double u = __shfl_up(s, m, 64);
        if (i >= m) s += u;
    }
    const double last = __shfl(s, 63, 64);
    out[i] = __builtin_amdgcn_exp2f(static_cast<float>(s));
    out[kC + i] = __builtin_amdgcn_exp2f(static_cast<float>(last - s));
    out[2 * kC + i] = b;
    const float hi = static_cast<float>(s);
    out[3 * kC + i] = hi;
    out[4 * kC + i] = static_cast<float>(s - hi);
}
__device__ __forceinline__ float gam(const float *gt, int i, int j)
{
    return __builtin_amdgcn_exp2f((gt[3 * kC + i] - gt[3 * kC + j]) + (gt[4 * kC + i] - gt[4 * kC + j]));
}

__device__ __forceinline__ int tri_row(int tile) { return tile < 1 ? 0 : (tile < 3 ? 1 : (tile < 6 ? 2 : 3)); }
__host__ __device__ constexpr int tri_tile(int a, int b) { return a * (a + 1) / 2 + b; }
// fragment of M (P) for rows 16 rt .., columns 32 ks .. (ks <= rt / 2)
__host__ __device__ constexpr int m_frag(int rt, int ks) { return rt < 2 ? rt : 2 * rt - 2 + ks; }
// fragment of M^T for rows 16 rt .., columns 32 ks .. (ks >= rt / 2)
__host__ __device__ constexpr int mt_frag(int rt, int ks) { return rt < 2 ? 2 * rt + ks : 2 + rt; }

// ------------------------------------------------------------------ delta_prep

__device__ __forceinline__ facc mfma4(float a, float b, facc c) { return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0); }

// Gates, M and (for the forward) P of one chunk for the heads that share key
// head hk0 + blockIdx.y. M block by block: the 16 x 16 blocks on the diagonal by
// substitution, a column a lane, then the blocks below by
// M21 = (I - M22 B2) N21 (I - B1 M11) for halves of 32 and of 64, in fp32 matrix
// instructions (20 products of 16^3 a head: small beside the split products
// elsewhere). Bound by the substitution's 14 dependent steps and the barriers
// between the phases, so by workgroups a compute unit. 12288 chunks and heads of d_k
// 32, fp32: 130 us (172 with the rows below read all at once, in registers that
// halve the workgroups); 2508 of d_k 128, bf16: 36 us.
template <typename T, int KD, bool BWD>
__global__ __launch_bounds__(256, KD == 128 && sizeof(T) == 4 ? 3 : 4) void delta_prep(ChunkParams p)
{
    // Q, then K, then N and M share one place, so that several workgroups fit a
    // compute unit (the phases below wait for one another)
    constexpr int NP = kParts<T>, kLdM = 68, kNM = 2 * kC * kLdM * 4, kK = Tile<NP, kC, KD>::kBytes;
    __shared__ __align__(16) unsigned char buf[kK > kNM ? kK : kNM];
    __shared__ __align__(16) float gt[kGates];
    uint16_t *kbuf = reinterpret_cast<uint16_t *>(buf);
    float *sn = reinterpret_cast<float *>(buf), *sm = sn + kC * kLdM;
    const long slot = blockIdx.x;
    const Place c = find_chunk(p, slot);
    if (c.len == 0) return;
    const int hk = p.hk0 + blockIdx.y, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = threadIdx.x % 64;
    int g4 = l / 16, l16 = l % 16;
    const Tile<NP, kC, KD> kt{kbuf};
    facc kk[4], qk[4];  // K K^T: rows 16 wave + 4 g4 + r, columns 16 ct + l16; Q K^T transposed: rows 16 ct + .., columns 16 wave + ..
    // (the gates' inputs are read first, and for the next head a head ahead: their
    // sums over the chunk go on while the rows of q and k come)
    GateIn gates;
    gates.load(p, c, hk * p.rep);
    {
        Stage<T, KD, 256> sq, sk;
        bfrag fq[KD / 32][NP];
        if constexpr (!BWD) sq.load(static_cast<const T *>(p.q) + c.b * p.qs[0] + c.t0 * p.qs[1] + hk * p.qs[2], p.qs[1], c.len, p.dk_, p.vec_qk);
        sk.load(static_cast<const T *>(p.k) + c.b * p.ks[0] + c.t0 * p.ks[1] + hk * p.ks[2], p.ks[1], c.len, p.dk_, p.vec_qk);
        make_gates(c, gates, gt);
        if constexpr (!BWD) {
            sq.put(kt);
            lds_barrier();
#pragma unroll
            for (int ks = 0; ks < KD / 32; ++ks) kt.rows(16 * wave, 32 * ks, fq[ks]);
            lds_barrier();
        }
        sk.put(kt);
        lds_barrier();
#pragma unroll
        for (int ct = 0; ct < 4; ++ct) {
            kk[ct] = qk[ct] = facc{0, 0, 0, 0};
            if (ct > wave) continue;
#pragma unroll
            for (int ks = 0; ks < KD / 32; ++ks) {
                bfrag a[NP], b[NP];
                kt.rows(16 * wave, 32 * ks, a);
                kt.rows(16 * ct, 32 * ks, b);
                if constexpr (BWD) mma<NP, NP>(kk[ct], a, b);
                else mma_two<NP, NP, NP, NP>(kk[ct], a, b, qk[ct], b, fq[ks]);
            }
        }
    }
    for (int r = 0; r < p.rep; ++r) {
        const int hl = blockIdx.y * p.rep + r;  // head of this pass
        asm volatile("" : "+v"(g4), "+v"(l16));  // (else the addresses of the whole body are kept across heads, in 200 registers)
        lds_barrier();
        if (r > 0) {
            make_gates(c, gates, gt);
            lds_barrier();
        }
        if (r + 1 < p.rep) gates.load(p, c, hk * p.rep + r + 1);
        const long at = slot * p.nh + hl;
        for (int i = threadIdx.x; i < kGates; i += 256) p.gates[at * kGates + i] = gt[i];
        if constexpr (!BWD) {  // P: token i = 16 wave + l16, four neighbouring j a lane, which is an operand's layout
            const int i = 16 * wave + l16;
            const float hi = gt[3 * kC + i], lo = gt[4 * kC + i];
#pragma unroll
            for (int ct = 0; ct < 4; ++ct) {
                if (ct > wave) continue;
                const int j0 = 16 * ct + 4 * g4;
                const facc jhi = *reinterpret_cast<const facc *>(gt + 3 * kC + j0), jlo = *reinterpret_cast<const facc *>(gt + 4 * kC + j0);
                facc x;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    x[j] = j0 + j <= i ? p.scale * __builtin_amdgcn_exp2f((hi - jhi[j]) + (lo - jlo[j])) * qk[ct][j] : 0.0f;
                *reinterpret_cast<facc *>(p.pm + at * kTriFloats + tri_tile(wave, ct) * 256 + l * 4) = x;
            }
        }
        {   // N (in the blocks on the diagonal with its mirror image, read below)
            const facc hi = *reinterpret_cast<const facc *>(gt + 3 * kC + 16 * wave + 4 * g4), lo = *reinterpret_cast<const facc *>(gt + 4 * kC + 16 * wave + 4 * g4);
#pragma unroll
            for (int ct = 0; ct < 4; ++ct) {
                const int col = 16 * ct + l16;
                const float chi = gt[3 * kC + col], clo = gt[4 * kC + col];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = 16 * wave + 4 * g4 + j;
                    if (ct > wave) {
                        sm[row * kLdM + col] = 0.0f;
                    } else {
                        const float d = (hi[j] - chi) + (lo[j] - clo);
                        sn[row * kLdM + col] = col == row ? 0.0f : __builtin_amdgcn_exp2f(col < row ? d : -d) * kk[ct][j];
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        __syncthreads();
        const float *beta = gt + 2 * kC;
        {   // diagonal block `wave`, column l16 (each 16 lanes the same)
            const int o = 16 * wave;
            // (row i is final once rows before it have been taken off; then it
            // is taken off the rows below, which do not wait for one another)
            float m[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = sn[(o + i) * kLdM + o + l16];
                m[i] = i > l16 ? x : 0.0f;
            }
            facc be[4], next[4];  // N below row i in column i, from its mirror image
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                be[k] = *reinterpret_cast<const facc *>(beta + o + 4 * k);
                next[k] = *reinterpret_cast<const facc *>(sn + (o + 1) * kLdM + o + 4 * k);
            }
#pragma unroll
            for (int i = 1; i < 15; ++i) {
                facc row[4];
                int zero = 0;
                asm volatile("" : "+v"(zero) : "v"(m[i]));  // (the next row is read now: all rows at once would take 120 registers)
#pragma unroll
                for (int k = i / 4; k < 4; ++k) {
                    row[k] = next[k];
                    if (i < 14) next[k] = *reinterpret_cast<const facc *>(sn + (o + i + 1) * kLdM + o + 4 * k + zero);
                }
                const float x = be[i / 4][i % 4] * m[i];
#pragma unroll
                for (int k = i + 1; k < 16; ++k) m[k] = fmaf(-row[k / 4][k % 4], x, m[k]);
            }
            if (g4 == 0) {
#pragma unroll
                for (int i = 0; i < 16; ++i) sm[(o + i) * kLdM + o + l16] = m[i];
            }
        }
        __syncthreads();
        if (wave < 2) {  // blocks (1, 0) and (3, 2); summed index 4 g4 + s
            const int r0 = 32 * wave + 16, c0 = 32 * wave;
            facc x;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = sn[(r0 + 4 * g4 + j) * kLdM + c0 + l16];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = c0 + 4 * g4 + s;
                x = mfma4(-sn[(r0 + l16) * kLdM + k] * beta[k], sm[k * kLdM + c0 + l16], x);
            }
            facc y = x;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = r0 + 4 * g4 + s;
                y = mfma4(-sm[(r0 + l16) * kLdM + k] * beta[k], x[s], y);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) sm[(r0 + 4 * g4 + j) * kLdM + c0 + l16] = y[j];
        }
        __syncthreads();
        {   // rows 32 .. 63, columns 0 .. 31: one tile a wave
            const int r0 = 32 + 16 * (wave / 2), c0 = 16 * (wave % 2);
            facc x;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = sn[(r0 + 4 * g4 + j) * kLdM + c0 + l16];
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int k = 16 * (s / 4) + 4 * g4 + s % 4;
                x = mfma4(-sn[(r0 + l16) * kLdM + k] * beta[k], sm[k * kLdM + c0 + l16], x);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) sm[(r0 + 4 * g4 + j) * kLdM + c0 + l16] = x[j];
            __syncthreads();
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int k = 32 + 16 * (s / 4) + 4 * g4 + s % 4;
                x = mfma4(-sm[(r0 + l16) * kLdM + k] * beta[k], sm[k * kLdM + c0 + l16], x);
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) sm[(r0 + 4 * g4 + j) * kLdM + c0 + l16] = x[j];
        }
        __syncthreads();
#pragma unroll 1
        for (int t = wave; t < kTriTiles; t += 4) {
            const int ra = tri_row(t), rb = t - tri_tile(ra, 0);
            *reinterpret_cast<facc *>(p.m + at * kTriFloats + t * 256 + l * 4) =
                -*reinterpret_cast<const facc *>(sm + (16 * ra + l16) * kLdM + 16 * rb + 4 * g4);
            if constexpr (BWD) {
                facc x;
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = -sm[(16 * ra + 4 * g4 + j) * kLdM + 16 * rb + l16];
                *reinterpret_cast<facc *>(p.mt + at * kTriFloats + t * 256 + l * 4) = x;
            }
        }
    }
}

// ------------------------------------------------------------------ P

// Rows 16 rt .. of scale Gam_ij q_i . k_j (j <= i), by one wave: column (token)
// i = 16 rt + l % 16, rows j; fq: the wave's rows of q.
template <typename T, int KD>
__device__ __forceinline__ void make_p(const bfrag (&fq)[KD / 32][kParts<T>], const Tile<kParts<T>, kC, KD> &kt, const float *gt, float scale,
                                       int rt, facc (&out)[4])
{
    constexpr int NP = kParts<T>;
    const int l = threadIdx.x % 64, i = 16 * rt + l % 16;
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
        out[jt] = facc{0, 0, 0, 0};
        if (jt > rt) continue;
        facc acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};  // two sums, so that a product does not wait for the one before
#pragma unroll
        for (int ks = 0; ks < KD / 32; ++ks) {
            bfrag a[NP];
            kt.rows(16 * jt, 32 * ks, a);
            mma<NP, NP>(acc[ks % 2], a, fq[ks]);
        }
        const int j0 = 16 * jt + 4 * (l / 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) out[jt][j] = j0 + j <= i ? scale * gam(gt, i, j0 + j) * (acc[0][j] + acc[1][j]) : 0.0f;
    }
}
template <int NPP>
__device__ __forceinline__ void put_p(const facc (&x)[4], int rt, const Tile<NPP, kC, kC> &out)
{
    const int l = threadIdx.x % 64;
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) out.put4(16 * rt + l % 16, 16 * jt + 4 * (l / 16), x[jt][0], x[jt][1], x[jt][2], x[jt][3]);
}

// Z = scale P^T dO of one chunk and head: workgroup (slot, head). Q and K give
// their place to P and dO. Its own kernel, since it needs no state: 3072 chunks
// and heads of 64 x 64, bf16, take 29 us, bound by the latency of one chunk's
// phases (58 % of its wave cycles wait).
template <typename T, int KD>
struct ZLds {
    static constexpr int NP = kParts<T>, VS = 32;
    using KT = Tile<NP, kC, KD>;
    using PT = Tile<3, kC, kC>;
    using VT = Tile<NP, kC, VS>;
    static constexpr int kAfter = PT::kBytes + VT::kBytes, kMain = 2 * KT::kBytes > kAfter ? 2 * KT::kBytes : kAfter;
    static constexpr int kBytes = kMain + kGates * 4;
};

template <typename T, int KD>
__global__ __launch_bounds__(256) void delta_z(ChunkParams p)
{
    using L = ZLds<T, KD>;
    constexpr int NP = L::NP, VS = L::VS;
    extern __shared__ __align__(16) uint16_t lds[];
    const long slot = blockIdx.x;
    const Place c = find_chunk(p, slot);
    if (c.len == 0) return;
    const int hl = blockIdx.y, head = p.hk0 * p.rep + hl, hk = head / p.rep, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = threadIdx.x % 64;
    const typename L::KT qt{lds}, kt{lds + L::KT::kBytes / 2};
    const typename L::PT pt{lds};
    const typename L::VT ot{lds + L::PT::kBytes / 2};
    float *gt = reinterpret_cast<float *>(lds + L::kMain / 2);
    const T *op = static_cast<const T *>(p.dout) + c.b * p.os[0] + c.t0 * p.os[1] + head * p.os[2];
    Stage<T, VS, 256> so;
    facc x[4];
    {
        Stage<T, KD, 256> a, b;
        float gates[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) gates[i] = p.gates[(slot * p.nh + hl) * kGates + min(i * 256 + static_cast<int>(threadIdx.x), kGates - 1)];
        a.load(static_cast<const T *>(p.q) + c.b * p.qs[0] + c.t0 * p.qs[1] + hk * p.qs[2], p.qs[1], c.len, p.dk_, p.vec_qk);
        b.load(static_cast<const T *>(p.k) + c.b * p.ks[0] + c.t0 * p.ks[1] + hk * p.ks[2], p.ks[1], c.len, p.dk_, p.vec_qk);
        so.load(op, p.os[1], c.len, p.dv_, p.vec_do);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (i * 256 + static_cast<int>(threadIdx.x) < kGates) gt[i * 256 + threadIdx.x] = gates[i];
        a.put(qt);
        b.put(kt);
        lds_barrier();
        bfrag fq[KD / 32][NP];
#pragma unroll
        for (int ks = 0; ks < KD / 32; ++ks) qt.rows(16 * wave, 32 * ks, fq[ks]);
        make_p<T, KD>(fq, kt, gt, p.scale, wave, x);
    }
    lds_barrier();
    put_p<3>(x, wave, pt);
    float *zp = p.z + (slot * p.nh + hl) * kC * p.dvp;
    for (int v0 = 0; v0 < p.dvp; v0 += VS) {
        so.put(ot);
        lds_barrier();
        if (v0 + VS < p.dvp) so.load(op + v0 + VS, p.os[1], c.len, p.dv_ - v0 - VS, p.vec_do);
        // rows tokens j = 16 wave .., columns v
        facc acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            if (32 * ks + 31 < 16 * wave) continue;  // i >= j
            bfrag a[3], b[2][NP];
            pt.cols(32 * ks, 16 * wave, a);
#pragma unroll
            for (int vt = 0; vt < 2; ++vt) ot.cols(32 * ks, 16 * vt, b[vt]);
            mma_two<3, NP, 3, NP>(acc[0], a, b[0], acc[1], a, b[1]);
        }
        lds_barrier();
#pragma unroll
        for (int vt = 0; vt < 2; ++vt) *reinterpret_cast<facc *>(zp + (v0 + 16 * vt) * kC + wave * 256 + l * 4) = acc[vt];
    }
}

// ------------------------------------------------------------------ delta_seq

// What a chunk's step reads from LDS: K (and Q, but for the forward's chain of
// a backward), M's fragments (and P's, for the outputs), the gates and, of bf16
// inputs, the columns of v (dO).
template <typename T, int KD, bool BWD, bool OUT, int THREADS>
struct SeqBuf {
    static constexpr int kCols = THREADS / 4;
    static constexpr bool kStaged = sizeof(T) == 2, kQ = BWD || OUT;
    static constexpr int kTile = Tile<kParts<T>, kC, KD>::kBytes;
    static constexpr int kTri = kTriFrags * 1024 * 3, kTriP = OUT ? kTri : 0;
    static constexpr int kOne = (kQ ? 2 : 1) * kTile + kTri + kTriP + 3 * kC * 4;
    static constexpr int kV = kStaged ? Tile<1, kC, kCols>::kBytes : 0;
    // two buffers where that costs no second workgroup a compute unit: a large
    // state fills its registers with one anyway
    static constexpr int kBufs = (THREADS == 512 || KD == 128) && 2 * kOne + kV <= 160 * 1024 ? 2 : 1;
    static constexpr int kBytes = kBufs * kOne + kV;
};

// The next step's inputs, on their way through registers into LDS.
template <typename T, int KD, bool BWD, bool OUT, int THREADS>
struct SeqStage {
    using Buf = SeqBuf<T, KD, BWD, OUT, THREADS>;
    static constexpr int kTiles = OUT ? 2 * kTriTiles : kTriTiles, kWaves = THREADS / 64, kEach = (kTiles + kWaves - 1) / kWaves;
    static constexpr int kGateEach = (3 * kC + THREADS - 1) / THREADS;
    Stage<T, KD, THREADS> k, q;
    Stage<T, Buf::kCols, THREADS> v;
    facc m[kEach];
    float g[kGateEach];
    __device__ __forceinline__ void load(const ChunkParams &p, long b, long t0, int len, int hk, long at)
    {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = threadIdx.x % 64;
        k.load(static_cast<const T *>(p.k) + b * p.ks[0] + t0 * p.ks[1] + hk * p.ks[2], p.ks[1], len, p.dk_, p.vec_qk);
        if constexpr (Buf::kQ) q.load(static_cast<const T *>(p.q) + b * p.qs[0] + t0 * p.qs[1] + hk * p.qs[2], p.qs[1], len, p.dk_, p.vec_qk);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int t = min(i * kWaves + wave, kTiles - 1);
            const float *src = (OUT && t >= kTriTiles ? p.pm - kTriFloats : (BWD ? p.mt : p.m)) + at * kTriFloats + t * 256;
            m[i] = *reinterpret_cast<const facc *>(src + l * 4);
        }
#pragma unroll
        for (int i = 0; i < kGateEach; ++i) g[i] = p.gates[at * kGates + min(i * THREADS + static_cast<int>(threadIdx.x), 3 * kC - 1)];
    }
    // the workgroup's columns of v (dO) from c0 on: n of them
    __device__ __forceinline__ void load_v(const T *base, long stride, int len, int n, bool vec)
    {
        if constexpr (Buf::kStaged) v.load(base, stride, len, n, vec);
    }
    // a tile's four values into their fragment's parts
    static __device__ __forceinline__ void put_tile(uint16_t *area, int frag, int half, const facc &x)
    {
        const int l = threadIdx.x % 64;
        unsigned a[3], b[3];
        split2<3>(x[0], x[1], a);
        split2<3>(x[2], x[3], b);
#pragma unroll
        for (int n = 0; n < 3; ++n) *reinterpret_cast<uint2 *>(area + ((frag * 3 + n) * 64 + l) * 8 + half * 4) = make_uint2(a[n], b[n]);
    }
    __device__ __forceinline__ void put(uint16_t *one, uint16_t *vbuf) const
    {
        constexpr int kTile = Buf::kTile / 2;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
        if constexpr (Buf::kStaged) v.put(Tile<1, kC, Buf::kCols>{vbuf});
        k.put(Tile<kParts<T>, kC, KD>{one});
        if constexpr (Buf::kQ) q.put(Tile<kParts<T>, kC, KD>{one + kTile});
        uint16_t *mm = one + (Buf::kQ ? 2 : 1) * kTile, *pp = mm + Buf::kTri / 2;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int t = i * kWaves + wave;
            if (t >= kTiles) break;
            const int u = t < kTriTiles ? t : t - kTriTiles, a = tri_row(u), b = u - tri_tile(a, 0);
            if (BWD) put_tile(mm, mt_frag(b, a / 2), a % 2, m[i]);
            else put_tile(OUT && t >= kTriTiles ? pp : mm, m_frag(a, b / 2), b % 2, m[i]);
        }
        float *gates = reinterpret_cast<float *>(pp + Buf::kTriP / 2);
#pragma unroll
        for (int i = 0; i < kGateEach; ++i)
            if (i * THREADS + static_cast<int>(threadIdx.x) < 3 * kC) gates[i * THREADS + threadIdx.x] = g[i];
    }
    // the two halves of fragments that no tile fills, once
    static __device__ __forceinline__ void clear(uint16_t *one)
    {
        uint16_t *mm = one + (Buf::kQ ? 2 : 1) * (Buf::kTile / 2), *pp = mm + Buf::kTri / 2;
        const facc zero = {0, 0, 0, 0};
        if (threadIdx.x >= 64) return;
        if constexpr (BWD) {
            put_tile(mm, mt_frag(1, 0), 0, zero);
            put_tile(mm, mt_frag(3, 1), 0, zero);
        } else {
            put_tile(mm, m_frag(0, 0), 1, zero);
            put_tile(mm, m_frag(2, 1), 1, zero);
            if constexpr (OUT) {
                put_tile(pp, m_frag(0, 0), 1, zero);
                put_tile(pp, m_frag(2, 1), 1, zero);
            }
        }
    }
};

// The chain over a sequence's chunks for 16 columns of the state a wave (32, 64 or
// 128 a workgroup). Columns are independent, so waves only share what they read.
// The state [KD][16] stays in accumulators, from which it is cut into operands.
//
// A sequence whose chain would leave most of the chip idle is cut into
// segments: the chain is linear in its first state, S_end = A S_start + b, so
// PROBE runs every segment from zero (b) and, in the forward, with KD more
// columns from the unit matrix and v = 0 (A); delta_join goes over the
// segments; then they run at once from their true first states. The adjoint's
// transition is A^T.
//
// OUT: the outputs come from the same step, O = scale gamma Q S0 + P U, in
// transposed tiles (the parts of S and U are operands as they are, and a lane
// gets four neighbours of a token's row); else S0 and E are kept for
// delta_local.
//
// Measured: 8 heads of 128 x 128, bf16, 20034 packed tokens: probe 138 us, outputs
// 113 us (443 us for the whole forward with 64 columns a workgroup, 283 with 128,
// which read a chunk's K, Q and M once for 8 waves); 4 heads of 32 x 32, fp32, 196608
// tokens: 109 and 184 us (290 with four waves, two of them idle). With 128 columns
// the backward's chains took 147 and 130 us instead of 137 and 113 (2 x 4099
// tokens, 8 heads of 128 x 128).
template <typename T, int KD, bool BWD, bool PROBE, bool OUT, int THREADS>
__device__ __forceinline__ void seq_chain(const ChunkParams &p, uint16_t *lds)
{
    constexpr int NP = kParts<T>, NT = KD / 16;
    using Buf = SeqBuf<T, KD, BWD, OUT, THREADS>;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = threadIdx.x % 64, g4 = l / 16, l16 = l % 16;
    const long x = blockIdx.x / p.nh;
    const int hl = static_cast<int>(blockIdx.x - x * p.nh), head = p.hk0 * p.rep + hl, hk = head / p.rep;
    const Segment sg = find_segment<PROBE>(p, x);
    if (sg.of == 0) return;
    const Seq q = sg.q;
    const long s = sg.s, n_all = (q.len + kC - 1) / kC;
    const long c0 = static_cast<long>(sg.at) * p.seg_len, c1 = min(n_all, c0 + p.seg_len), n = c1 - c0;
    int v0 = blockIdx.y * (THREADS / 4) + wave * 16;
    const bool unit = PROBE && !BWD && v0 >= p.dvp;  // this wave's columns are the unit matrix's
    if (unit) v0 -= p.dvp;
    const bool act = v0 < (unit ? KD : p.dvp);  // this wave has columns
    if (PROBE && BWD && static_cast<int>(blockIdx.y) * (THREADS / 4) >= p.dvp) return;
    const int col = v0 + l16;
    const bool live = !unit && col < p.dv_;  // this lane's column is not padding
    const int colv = min(col, p.dv_ - 1);  // (where lanes without a column read)
    const long state = ((s * p.h + head) * p.dk_) * p.dv_;
    const float *init = BWD ? p.dh_last : p.h_init;
    const long place = sg.place * p.nh + hl;
    float *joined = (BWD ? p.seg_d : p.seg_s) + place * KD * p.dvp + v0 * KD + l * 4;
    facc S[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        if (!PROBE && sg.of > 1) {
            S[t] = act ? *reinterpret_cast<const facc *>(joined + t * 256) : facc{0, 0, 0, 0};
            continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 16 * t + 4 * g4 + j;
            if constexpr (PROBE) {
                S[t][j] = (unit && row == col) ? 1.0f : 0.0f;
            } else {
                S[t][j] = init ? init[state + static_cast<long>(min(row, p.dk_ - 1)) * p.dv_ + colv] : 0.0f;
                S[t][j] = (live && row < p.dk_) ? S[t][j] : 0.0f;
            }
        }
    }
    auto len_of = [&](long c) { return static_cast<int>(q.len - c * kC < kC ? q.len - c * kC : kC); };
    auto chunk = [&](long i) { return BWD ? c1 - 1 - i : c0 + i; };
    // a column of the chunk's rows of v (dO and Z in the backward), 16 tokens a lane
    T x0[16];
    facc x1[4];
    const T *vp = BWD ? static_cast<const T *>(p.dout) + q.b * p.os[0] + head * p.os[2] : static_cast<const T *>(p.v) + q.b * p.vs[0] + head * p.vs[2];
    const long vstep = BWD ? p.os[1] : p.vs[1];
    SeqStage<T, KD, BWD, OUT, THREADS> st;
    uint16_t *vbuf = lds + Buf::kBufs * (Buf::kOne / 2);
    const int wg0 = min(static_cast<int>(blockIdx.y) * Buf::kCols, (p.dv_ - 1) / 16 * 16);  // (workgroups of the unit matrix alone read any)
    auto load_cols = [&](long c) __attribute__((always_inline)) {
        const int len = len_of(c);
        const T *src = vp + (q.t0 + c * kC) * vstep;
        if constexpr (Buf::kStaged) {
            st.load_v(src + wg0, vstep, len, p.dv_ - wg0, BWD ? p.vec_do : p.vec_v);
        } else if (len == kC) {  // (the lane's part of the offset in 32 bits: see the limit on strides)
            const unsigned lane = 4 * g4 * static_cast<unsigned>(vstep) + colv;
#pragma unroll
            for (int t = 0; t < 16; ++t) x0[t] = (src + (16 * (t / 4) + t % 4) * vstep)[lane];
        } else {
#pragma unroll
            for (int t = 0; t < 16; ++t) x0[t] = (src + colv)[min(16 * (t / 4) + 4 * g4 + t % 4, len - 1) * vstep];
        }
        if constexpr (BWD) {
            const float *z = p.z + ((q.slot0 + c) * p.nh + hl) * kC * p.dvp + (act && !unit ? v0 : 0) * kC + l * 4;
#pragma unroll
            for (int t = 0; t < 4; ++t) x1[t] = *reinterpret_cast<const facc *>(z + t * 256);
        }
    };
    auto fetch = [&](long c) __attribute__((always_inline)) { st.load(p, q.b, q.t0 + c * kC, len_of(c), hk, (q.slot0 + c) * p.nh + hl); };
    facc y0[4], y1[4];  // the step's rows of v (dO) and Z
    auto take_cols = [&](long c) __attribute__((always_inline)) {
        const int len = len_of(c);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if constexpr (!Buf::kStaged) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    y0[t][j] = (live && 16 * t + 4 * g4 + j < len) ? widen1(x0[4 * t + j]) : 0.0f;
                    asm volatile("" : "+v"(y0[t][j]));  // (here, and not where it is used)
                }
            }
            if constexpr (BWD) {
                y1[t] = x1[t];
                asm volatile("" : "+v"(y1[t]));
            }
        }
    };
    // (staged columns: 16 tokens of column l16 by a transposing read, which gives an accumulator's rows)
    auto staged_cols = [&]() __attribute__((always_inline)) {
        if constexpr (Buf::kStaged) {
            const Tile<1, kC, Buf::kCols> vt{vbuf};
#pragma unroll
            for (int t = 0; t < 4; t += 2) {
                bfrag f[1];
                vt.cols(16 * t, 16 * wave, f);
                FragBits x;
                x.f = f[0];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    y0[t + w / 2][2 * (w % 2)] = live ? bf16_lo(x.w[w]) : 0.0f;
                    y0[t + w / 2][2 * (w % 2) + 1] = live ? bf16_hi(x.w[w]) : 0.0f;
                }
            }
        }
    };
    auto keep_state = [&](long c) __attribute__((always_inline)) {
        float *keep = (BWD ? p.d1 : p.s0) + ((q.slot0 + c) * p.nh + hl) * KD * p.dvp + v0 * KD + l * 4;
#pragma unroll
        for (int t = 0; t < NT; ++t) *reinterpret_cast<facc *>(keep + t * 256) = S[t];
    };
    if (n > 0) {
        fetch(chunk(0));
        load_cols(chunk(0));
        st.clear(lds);
        if constexpr (Buf::kBufs == 2) st.clear(lds + Buf::kOne / 2);
        st.put(lds, vbuf);
        take_cols(chunk(0));
        if (!PROBE && !OUT && act) keep_state(chunk(0));
    }
    // One step: read the next chunk, compute this one, put what was read, store
    // this one's results. The stores come last: loads and stores share one
    // counter, so a wait for a load would also wait for the stores before it,
    // and these get a whole step to finish.
    for (long i = 0; i < n; ++i) {
        const long c = chunk(i), at = (q.slot0 + c) * p.nh + hl;
        uint16_t *buf = lds + (Buf::kBufs == 2 ? (i & 1) * (Buf::kOne / 2) : 0);
        uint16_t *next = lds + (Buf::kBufs == 2 ? ((i + 1) & 1) * (Buf::kOne / 2) : 0);
        lds_barrier();
        if (act) staged_cols();
        if constexpr (Buf::kBufs == 2 && Buf::kStaged) lds_barrier();  // (there is one place for the columns)
        if (i + 1 < n) {
            fetch(chunk(i + 1));
            load_cols(chunk(i + 1));
        }
        facc X[4], O[4];
        float o0[16];
        if (act) {
            const Tile<NP, kC, KD> kt{buf}, qt{buf + Buf::kTile / 2};
            uint16_t *rest = buf + (Buf::kQ ? 2 : 1) * (Buf::kTile / 2);
            const word4 *mm = reinterpret_cast<const word4 *>(rest), *pp = reinterpret_cast<const word4 *>(rest + Buf::kTri / 2);
            const float *gt = reinterpret_cast<const float *>(rest + (Buf::kTri + Buf::kTriP) / 2);
            // Y = K S, then the right-hand side: V - gamma Y, or Z + Gam_last Y
            facc Y[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) Y[t] = O[t] = facc{0, 0, 0, 0};
#pragma unroll
            for (int ks = 0; ks < KD / 32; ++ks) {
                bfrag b[3], a[4][NP];
#pragma unroll
                for (int t = 0; t < 4; ++t) kt.rows(16 * t, 32 * ks, a[t]);
                split_acc<3>(S[2 * ks], S[2 * ks + 1], b);
                mma_each<NP, 3, 4>(Y, a, b);
                if constexpr (OUT) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) qt.rows(16 * t, 32 * ks, a[t]);
                    mma_each_t<NP, 3, 4>(O, a, b);
                }
            }
            // (gamma, Gam_last and beta of the lane's tokens come from LDS at each use: kept, they take 48 registers)
            auto gate = [&](int which, int t) { return *reinterpret_cast<const facc *>(gt + which * kC + 16 * t + 4 * g4); };
            facc W[4];  // beta times the right-hand side
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const facc f = gate(BWD ? 1 : 0, t);
#pragma unroll
                for (int j = 0; j < 4; ++j) X[t][j] = BWD ? fmaf(f[j], Y[t][j], y1[t][j]) : fmaf(-f[j], Y[t][j], y0[t][j]);
                W[t] = gate(2, t) * X[t];
            }
            // E = R - M (B R), or dR = dU - M^T (B dU)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                bfrag b[3], a[4][3];
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (BWD ? ks >= t / 2 : ks <= t / 2)
#pragma unroll
                        for (int n3 = 0; n3 < 3; ++n3) {
                            FragBits fb;
                            fb.q = mm[((BWD ? mt_frag(t, ks) : m_frag(t, ks)) * 3 + n3) * 64 + l];
                            a[t][n3] = fb.f;
                        }
                split_acc<3>(W[2 * ks], W[2 * ks + 1], b);
#pragma unroll
                for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                    for (int u = 0; u <= sum; ++u)
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            if (BWD ? ks >= t / 2 : ks <= t / 2) X[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][u], b[sum - u], X[t], 0, 0, 0);
            }
            facc W2[4];
            if constexpr (OUT) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    W2[t] = gate(2, t) * X[t];           // U
                    O[t] *= p.scale * gt[16 * t + l16];  // (this lane's token)
                }
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    bfrag b[3], a[4][3];
                    split_acc<3>(W2[2 * ks], W2[2 * ks + 1], b);
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        if (ks <= t / 2)
#pragma unroll
                            for (int n3 = 0; n3 < 3; ++n3) {
                                FragBits fb;
                                fb.q = pp[(m_frag(t, ks) * 3 + n3) * 64 + l];
                                a[t][n3] = fb.f;
                            }
#pragma unroll
                    for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                        for (int u = 0; u <= sum; ++u)
#pragma unroll
                            for (int t = 0; t < 4; ++t)
                                if (ks <= t / 2) O[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[sum - u], a[t][u], O[t], 0, 0, 0);
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const facc bx = gate(2, t) * X[t];
                if constexpr (BWD) {
                    const facc ga = gate(0, t);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o0[4 * t + j] = bx[j];
                    W[t] = -ga * bx;
                    W2[t] = p.scale * ga * y0[t];
                } else {
                    W[t] = gate(1, t) * bx;
                }
            }
            const float last = gt[kC - 1];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) S[t][j] *= last;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                bfrag b[3], a[NT][NP];
#pragma unroll
                for (int t = 0; t < NT; ++t) kt.cols(32 * ks, 16 * t, a[t]);
                split_acc<3>(W[2 * ks], W[2 * ks + 1], b);
                mma_each<NP, 3, NT>(S, a, b);
                if constexpr (BWD) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) qt.cols(32 * ks, 16 * t, a[t]);
                    split_acc<3>(W2[2 * ks], W2[2 * ks + 1], b);
                    mma_each<NP, 3, NT>(S, a, b);
                }
            }
        }
        if (i + 1 < n) {
            if constexpr (Buf::kBufs == 1) lds_barrier();
            st.put(next, vbuf);
            take_cols(chunk(i + 1));
        }
        asm volatile("" ::: "memory");  // (no store goes up past the waits above)
        if (OUT && act) {
            const int len = len_of(c), v = v0 + 4 * g4;
            T *op = static_cast<T *>(p.o) + ((q.b * p.tokens + q.t0 + c * kC + l16) * p.h + head) * p.dv_ + v;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (16 * t + l16 >= len) continue;
                T *to = op + static_cast<long>(16 * t) * p.h * p.dv_;
                if (p.vec_o && v + 4 <= p.dv_) {
                    Raw<T, 4> r;
                    float y[4] = {O[t][0], O[t][1], O[t][2], O[t][3]};
                    r.set(y);
                    r.store(to);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (v + j < p.dv_) store1(to + j, O[t][j]);
                }
            }
        }
        if (!PROBE && !OUT && act) {
            float *ep = (BWD ? p.dr : p.e) + at * kC * p.dvp + v0 * kC + l * 4;
#pragma unroll
            for (int t = 0; t < 4; ++t) *reinterpret_cast<facc *>(ep + t * 256) = X[t];
            if (i + 1 < n) keep_state(chunk(i + 1));
            if constexpr (BWD) {
                const int len = len_of(c);
                const long step = static_cast<long>(p.h) * p.dv_;
                T *dvo = static_cast<T *>(p.dv) + ((q.b * p.tokens + q.t0 + c * kC) * p.h + head) * p.dv_ + 4 * g4 * step + col;
                if (live) {
                    if (len == kC) {
#pragma unroll
                        for (int t = 0; t < 16; ++t) store1(dvo + (16 * (t / 4) + t % 4) * step, o0[t]);
                    } else {
#pragma unroll
                        for (int t = 0; t < 16; ++t)
                            if (16 * (t / 4) + 4 * g4 + t % 4 < len) store1(dvo + (16 * (t / 4) + t % 4) * step, o0[t]);
                    }
                }
            }
        }
    }
    if constexpr (PROBE) {
        if (!act) return;
        if (unit) {
            // A for delta_join, in parts: its rows' operands (four columns of a row
            // a lane), and for the adjoint its columns'
            const long at = place * (kSegTile<KD> * NT);
            uint2 *rows = reinterpret_cast<uint2 *>(p.seg_at + at + v0 / 32 * 3 * 64 + 4 * g4 + l16 % 4 + 16 * (l16 / 4)) + v0 / 16 % 2;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const facc r = turn4(S[t]);
                unsigned w0[3], w1[3];
                split2<3>(r[0], r[1], w0);
                split2<3>(r[2], r[3], w1);
#pragma unroll
                for (int n = 0; n < 3; ++n) rows[2 * (t * kSegTile<KD> + n * 64)] = make_uint2(w0[n], w1[n]);
            }
            if (!p.seg_a) return;
#pragma unroll
            for (int ks = 0; ks < NT / 2; ++ks) {
                bfrag f[3];
                split_acc<3>(S[2 * ks], S[2 * ks + 1], f);
#pragma unroll
                for (int n = 0; n < 3; ++n) p.seg_a[at + v0 / 16 * kSegTile<KD> + (ks * 3 + n) * 64 + l] = FragBits{.f = f[n]}.q;
            }
            return;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) *reinterpret_cast<facc *>(joined + t * 256) = S[t];
        return;
    }
    float *out = BWD ? p.dh_init : p.h_last;
    if (out && live && sg.at == (BWD ? 0 : sg.of - 1)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = 16 * t + 4 * g4 + j;
                if (row < p.dk_) out[state + static_cast<long>(row) * p.dv_ + col] = S[t][j];
            }
    }
}

// Workgroups (segment and head, 32, 64 or 128 columns); with GRAD those of blockIdx.z
// = 1 run the adjoints' chain, at the same time.
template <typename T, int KD, bool GRAD, bool PROBE, int THREADS>
__global__ __launch_bounds__(THREADS, THREADS == 256 && KD <= 64 ? 2 : 1) void delta_seq(ChunkParams p)
{
    extern __shared__ __align__(16) uint16_t lds[];
    if constexpr (GRAD) {
        if (blockIdx.z == 1) {
            seq_chain<T, KD, true, PROBE, false, THREADS>(p, lds);
            return;
        }
    }
    seq_chain<T, KD, false, PROBE, !GRAD && !PROBE, THREADS>(p, lds);
}

// First states of the segments: S over a sequence's segments, S <- A S + b
// (adjoint: D <- A^T D + b from the last one), each stored in b's place.
// Workgroup (sequence, or the place of its first segment, and head; 16 columns; forward
// or adjoint). What a step
// waits for is its own chain (the state's parts, products), so a wave has few
// rows: 16, with the state's parts through LDS and one barrier a segment, or a
// small state's 32, whose parts stay in registers. A comes as operands, split
// by the probe. A step takes 2 us of 128 x 128, 0.3 of 32 x 32; with 64 columns a
// workgroup, all rows a wave and A through LDS 5.7 and 0.6.
template <typename T, int KD, bool GRAD>
__global__ __launch_bounds__(KD == 32 ? 64 : KD * 4, 1) void delta_join(ChunkParams p)
{
    constexpr int NT = KD / 16, KS = KD / 32, WT = KD == 32 ? 2 : 1, DEPTH = KD == 128 ? 2 : (KD == 64 ? 4 : 6);
    __shared__ __align__(16) word4 parts[2][3][KS][64];  // [turn][part]: two tiles' parts, a lane's 16 bytes
    const bool bwd = GRAD && blockIdx.z == 1;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = threadIdx.x % 64, g4 = l / 16, l16 = l % 16;
    const long x = blockIdx.x / p.nh;
    const int hl = static_cast<int>(blockIdx.x - x * p.nh), head = p.hk0 * p.rep + hl;
    const Segment sg = find_joined(p, x);
    if (sg.of == 0) return;
    const long s = sg.s;
    const int ns = sg.of;
    const int v0 = blockIdx.y * 16, col = v0 + l16;
    const float *init = bwd ? p.dh_last : p.h_init;
    const long state = ((s * p.h + head) * p.dk_) * p.dv_;
    facc S[WT];
#pragma unroll
    for (int t = 0; t < WT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 16 * (wave * WT + t) + 4 * g4 + j;
            S[t][j] = init ? init[state + static_cast<long>(min(row, p.dk_ - 1)) * p.dv_ + min(col, p.dv_ - 1)] : 0.0f;
            S[t][j] = (col < p.dv_ && row < p.dk_) ? S[t][j] : 0.0f;
        }
    // A and b of the next DEPTH segments, read that far ahead: another XCD wrote
    // them, so they come from memory, later than a step or two
    word4 a[DEPTH][WT][KS][3];
    facc b[DEPTH][WT];
    auto seg = [&](int i) { return (sg.place + (bwd ? ns - 1 - i : i)) * p.nh + hl; };
    auto place = [&](int i) { return (bwd ? p.seg_d : p.seg_s) + seg(i) * KD * p.dvp + v0 * KD + wave * WT * 256 + l * 4; };
    auto fetch = [&](int i, int at) __attribute__((always_inline)) {  // (past the end the last segment's, which are not used)
        i = min(i, ns - 1);
        const word4 *src = (bwd ? p.seg_a : p.seg_at) + seg(i) * kSegTile<KD> * NT + wave * WT * kSegTile<KD> + l;
#pragma unroll
        for (int t = 0; t < WT; ++t) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int n = 0; n < 3; ++n) a[at][t][ks][n] = src[t * kSegTile<KD> + (ks * 3 + n) * 64];
            b[at][t] = *reinterpret_cast<const facc *>(place(i) + t * 256);
        }
    };
    {
#pragma unroll
        for (int u = 0; u < DEPTH; ++u) fetch(u, u);
        for (int i0 = 0; i0 + 1 < ns; i0 += DEPTH) {
#pragma unroll
            for (int u = 0; u < DEPTH; ++u) {
                const int i = i0 + u;
                if (i + 1 >= ns) break;
                const int turn = i & 1;
                bfrag f[KS][3];
                if constexpr (WT == NT) {
                    split_acc<3>(S[0], S[1], f[0]);
                } else {
                    unsigned w0[3], w1[3];
                    split2<3>(S[0][0], S[0][1], w0);
                    split2<3>(S[0][2], S[0][3], w1);
#pragma unroll
                    for (int n = 0; n < 3; ++n)
                        reinterpret_cast<uint2 *>(&parts[turn][n][wave / 2][l])[wave % 2] = make_uint2(w0[n], w1[n]);
                    lds_barrier();
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int n = 0; n < 3; ++n) f[ks][n] = FragBits{.q = parts[turn][n][ks][l]}.f;
                }
                float *to = place(i);
                facc out[WT], x[WT], y[WT];
#pragma unroll
                for (int t = 0; t < WT; ++t) out[t] = S[t], x[t] = b[u][t], y[t] = facc{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    bfrag m[WT][3];
#pragma unroll
                    for (int t = 0; t < WT; ++t)
#pragma unroll
                        for (int n = 0; n < 3; ++n) m[t][n] = FragBits{.q = a[u][t][ks][n]}.f;
                    if (ks % 2) mma_each<3, 3, WT>(y, m, f[ks]);
                    else mma_each<3, 3, WT>(x, m, f[ks]);
                }
                fetch(i + DEPTH, u);
#pragma unroll
                for (int t = 0; t < WT; ++t) {
                    S[t] = KS > 1 ? x[t] + y[t] : x[t];
                    *reinterpret_cast<facc *>(to + t * 256) = out[t];
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < WT; ++t) *reinterpret_cast<facc *>(place(ns - 1) + t * 256) = S[t];
}

// ------------------------------------------------------------------ delta_local

// LDS of delta_local: slices of 32 columns first, then Q, K and the two
// triangular matrices in the same place.
template <typename T, int KD>
struct LocalLds {
    static constexpr int NP = kParts<T>, VS = 32;
    using KT = Tile<NP, kC, KD>;
    using PT = Tile<3, kC, kC>;
    using OT = Tile<NP, kC, VS>;
    using UT = Tile<3, VS, kC>;  // transposed
    using ST = Tile<3, VS, KD>;
    static constexpr int kSlices = OT::kBytes + 2 * UT::kBytes + 2 * ST::kBytes, kAfter = 2 * KT::kBytes + 2 * PT::kBytes;
    static constexpr int kMain = kSlices > kAfter ? kSlices : kAfter;
    // gates, sums of dG and dbeta (a row a wave or half), sums over the chunk
    static constexpr int kSums = kGates + 2 * kC + 2 * kC + 16;
    static constexpr int kBytes = kMain + kSums * 4;
};

// Gradients of one chunk for head p.turn of those that share key head
// hk0 + blockIdx.y: workgroup (slot, key head), a launch a turn, dQ and dK
// summed from turn to turn. Wave w holds tokens 16 (w % 4) .. and, of eight
// waves, half of the dims: the three d_k-wide sums of its tokens stay in
// accumulators over all slices of 32 columns, the next slice's matrices are
// read while this one's are multiplied. Four waves where that leaves two
// workgroups a compute unit (d_k' <= 64): their phases overlap. Bound by the
// waits between its phases (43 % of wave cycles) and the splits (23 %): 3072
// chunks and heads of 64 x 64, bf16: 104 us; 520 chunks and key heads of 128 x 128:
// 65 us a turn.
template <typename T, int KD, int WAVES>
__global__ __launch_bounds__(WAVES * 64, WAVES == 4 ? 2 : 1) void delta_local(ChunkParams p)
{
    using L = LocalLds<T, KD>;
    constexpr int NP = L::NP, VS = L::VS, THREADS = WAVES * 64, HALVES = WAVES / 4, NT = KD / 16 / HALVES, JT = 4 / HALVES;
    constexpr int kE = kC * VS / 4 / THREADS, kS = (KD * VS / 4 + THREADS - 1) / THREADS;
    static_assert(KD * VS / 4 % THREADS == 0 || KD * VS / 4 < THREADS, "pieces of a slice");
    extern __shared__ __align__(16) uint16_t lds[];
    const long slot = blockIdx.x;
    const Place c = find_chunk(p, slot);
    if (c.len == 0) return;
    const int hk = p.hk0 + blockIdx.y, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l = threadIdx.x % 64, g4 = l / 16;
    const int rt = wave % 4, half = wave / 4, i = 16 * rt + l % 16;  // this wave's tokens; its part of the dims and of the columns j
    const typename L::OT ot{lds};
    const typename L::UT ut{lds + L::OT::kBytes / 2}, rt_{ut.p + L::UT::kBytes / 2};
    const typename L::ST st{rt_.p + L::UT::kBytes / 2}, dt{st.p + L::ST::kBytes / 2};
    const typename L::KT qt{lds}, kt{lds + L::KT::kBytes / 2};
    const typename L::PT pt{lds + L::KT::kBytes}, nt{pt.p + L::PT::kBytes / 2};
    float *gt = reinterpret_cast<float *>(lds + L::kMain / 2), *sg = gt + kGates, *sb = sg + 2 * kC, *sw = sb + 2 * kC;
    const int hl = blockIdx.y * p.rep + p.turn, head = hk * p.rep + p.turn;
    const long at = slot * p.nh + hl;
    const T *op = static_cast<const T *>(p.dout) + c.b * p.os[0] + c.t0 * p.os[1] + head * p.os[2];
    const float *e0 = p.e + at * kC * p.dvp, *r0 = p.dr + at * kC * p.dvp, *s0 = p.s0 + at * KD * p.dvp, *d0 = p.d1 + at * KD * p.dvp;
    // one slice in registers
    Stage<T, VS, THREADS> so;
    facc xe[kE], xr[kE], xs[kS], xd[kS];
    auto fetch = [&](int v0) __attribute__((always_inline)) {
        so.load(op + v0, p.os[1], c.len, p.dv_ - v0, p.vec_do);
#pragma unroll
        for (int k = 0; k < kE; ++k) {
            xe[k] = *reinterpret_cast<const facc *>(e0 + v0 * kC + (k * THREADS + threadIdx.x) * 4);
            xr[k] = *reinterpret_cast<const facc *>(r0 + v0 * kC + (k * THREADS + threadIdx.x) * 4);
        }
#pragma unroll
        for (int k = 0; k < kS; ++k) {
            const int w = min(k * THREADS + static_cast<int>(threadIdx.x), KD * VS / 4 - 1);
            xs[k] = *reinterpret_cast<const facc *>(s0 + v0 * KD + w * 4);
            xd[k] = *reinterpret_cast<const facc *>(d0 + v0 * KD + w * 4);
        }
    };
    fetch(0);
    for (int w = threadIdx.x; w < kGates; w += THREADS) gt[w] = p.gates[at * kGates + w];
    __syncthreads();
    facc aq[NT], ar[NT], ac[NT], ap[JT], an[JT];
#pragma unroll
    for (int t = 0; t < NT; ++t) aq[t] = ar[t] = ac[t] = facc{0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < JT; ++t) ap[t] = an[t] = facc{0, 0, 0, 0};
    float sd = 0.0f;         // <S0, D1>, this thread's part
    facc db = {0, 0, 0, 0};  // dR . E of this thread's four tokens and its columns
    const int tok = 16 * rt + 4 * g4;
    for (int v0 = 0; v0 < p.dvp; v0 += VS) {
        so.put(ot);
#pragma unroll
        for (int k = 0; k < kE; ++k) {  // 64 x 32: a piece is four tokens of a column
            const int pcol = 16 * ((k * THREADS + static_cast<int>(threadIdx.x)) / 256) + l % 16;
            const facc u = xe[k] * *reinterpret_cast<const facc *>(gt + 2 * kC + tok);
            ut.put4(pcol, tok, u[0], u[1], u[2], u[3]);
            rt_.put4(pcol, tok, xr[k][0], xr[k][1], xr[k][2], xr[k][3]);
            db += xe[k] * xr[k];
        }
#pragma unroll
        for (int k = 0; k < kS; ++k) {
            const int w = k * THREADS + threadIdx.x, tile = w / 64, row = 16 * (tile % (KD / 16)) + 4 * g4, col = 16 * (tile / (KD / 16)) + l % 16;
            if (KD * VS / 4 % THREADS == 0 || w < KD * VS / 4) {
                st.put4(col, row, xs[k][0], xs[k][1], xs[k][2], xs[k][3]);
                dt.put4(col, row, xd[k][0], xd[k][1], xd[k][2], xd[k][3]);
                const facc m = xs[k] * xd[k];
                sd += (m[0] + m[1]) + (m[2] + m[3]);
            }
        }
        lds_barrier();
        if (v0 + VS < p.dvp) fetch(v0 + VS);
        bfrag fo[NP], fr[3], fu[3];
        ot.rows(16 * rt, 0, fo);
        rt_.cols(0, 16 * rt, fr);
        ut.cols(0, 16 * rt, fu);
#pragma unroll
        for (int t = 0; t < JT; ++t) {
            const int jt = JT * half + t;
            if (jt > rt) continue;
            bfrag a[3];
            ut.cols(0, 16 * jt, a);
            mma_two<3, NP, 3, 3>(ap[t], a, fo, an[t], a, fr);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            bfrag a[3], d[3];
            st.cols(0, 16 * (half * NT + t), a);
            dt.cols(0, 16 * (half * NT + t), d);
            mma_turns<NP>(aq[t], fo, ar[t], fr, a, ac[t], d, fu);
        }
        lds_barrier();
    }
    {   // rows' factors, and the triangular matrices into LDS
        Stage<T, KD, THREADS> a, b;
        a.load(static_cast<const T *>(p.q) + c.b * p.qs[0] + c.t0 * p.qs[1] + hk * p.qs[2], p.qs[1], c.len, p.dk_, p.vec_qk);
        b.load(static_cast<const T *>(p.k) + c.b * p.ks[0] + c.t0 * p.ks[1] + hk * p.ks[2], p.ks[1], c.len, p.dk_, p.vec_qk);
        const float ga = gt[i], gl = gt[kC + i], be = gt[2 * kC + i];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            aq[t] *= p.scale * ga;
            ar[t] *= -ga * be;
            ac[t] *= gl;
        }
#pragma unroll
        for (int t = 0; t < JT; ++t) {
            const int j0 = 16 * (JT * half + t) + 4 * g4;
            float x[4], y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float f = j0 + j <= i ? gam(gt, i, j0 + j) : 0.0f;
                x[j] = j0 + j <= i ? p.scale * f * ap[t][j] : 0.0f;
                y[j] = j0 + j < i ? -be * f * an[t][j] : 0.0f;
            }
            pt.put4(i, j0, x[0], x[1], x[2], x[3]);
            nt.put4(i, j0, y[0], y[1], y[2], y[3]);
        }
        a.put(qt);
        b.put(kt);
    }
    lds_barrier();
    float end = 0.0f;  // sum over this lane's dims of k . (Gam_last U D1^T)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float x[4];
        kt.get4(i, 16 * (half * NT + t) + 4 * g4, x);
#pragma unroll
        for (int j = 0; j < 4; ++j) end += x[j] * ac[t][j];
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
        if (32 * ks <= 16 * rt + 15) {  // j <= i
            bfrag fp[3], fn[3];
            pt.rows(16 * rt, 32 * ks, fp);
            nt.rows(16 * rt, 32 * ks, fn);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                bfrag a[NP];
                kt.cols(32 * ks, 16 * (half * NT + t), a);
                mma_two<NP, 3, NP, 3>(aq[t], a, fp, ar[t], a, fn);
            }
        }
        if (32 * ks + 31 >= 16 * rt) {  // this wave's tokens as j, i >= j
            bfrag fp[3], fn[3];
            pt.cols(32 * ks, 16 * rt, fp);
            nt.cols(32 * ks, 16 * rt, fn);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                bfrag a[NP], d[NP];
                facc x = {0, 0, 0, 0};
                qt.cols(32 * ks, 16 * (half * NT + t), a);
                kt.cols(32 * ks, 16 * (half * NT + t), d);
                mma_two<NP, 3, NP, 3>(ac[t], a, fp, x, d, fn);
                ac[t] += x;
            }
        }
    }
    float dg = 0.0f;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float x[4], y[4];
        qt.get4(i, 16 * (half * NT + t) + 4 * g4, x);
        kt.get4(i, 16 * (half * NT + t) + 4 * g4, y);
#pragma unroll
        for (int j = 0; j < 4; ++j) dg += x[j] * aq[t][j] + y[j] * (ar[t][j] - ac[t][j]);
    }
    dg = pair_sum<32>(pair_sum<16>(dg));
    if (g4 == 0) sg[half * kC + i] = dg;
#pragma unroll
    for (int j = 0; j < 4; ++j) db[j] = lane_sum<16>(db[j]);
    if (l % 16 == 0) *reinterpret_cast<facc *>(sb + half * kC + tok) = db;
    end = lane_sum<64>(end);
    sd = lane_sum<64>(sd);
    if (l == 0) sw[wave] = end, sw[8 + wave] = sd;
    lds_barrier();
    if (threadIdx.x < kC) {
        const int t = threadIdx.x;
        float e = 0.0f, d = 0.0f, s = sg[t], be = sb[t];
#pragma unroll
        for (int w = 0; w < WAVES; ++w) e += sw[w], d += sw[8 + w];
        if constexpr (HALVES == 2) s += sg[kC + t], be += sb[kC + t];
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
            const float u = __shfl_down(s, m, 64);
            if (t + m < 64) s += u;
        }
        if (t < c.len) {
            const long out = (c.b * p.tokens + c.t0 + t) * p.h + head;
            p.dg[out] = s + e + gt[kC - 1] * d;
            p.dbeta[out] = be;
        }
    }
    // dQ in aq, dK in ar: rows 16 (half NT + t) + 4 g4 + j (dims), column i
#pragma unroll
    for (int t = 0; t < NT; ++t) ar[t] += ac[t];
    if (p.rep > 1) {
        facc *sum = reinterpret_cast<facc *>(p.sum) + (slot * p.nhk + blockIdx.y) * (2 * NT * THREADS) + threadIdx.x;
        if (p.turn > 0) {
#pragma unroll
            for (int t = 0; t < NT; ++t) aq[t] += sum[(2 * t) * THREADS], ar[t] += sum[(2 * t + 1) * THREADS];
        }
        if (p.turn + 1 < p.rep) {
#pragma unroll
            for (int t = 0; t < NT; ++t) sum[(2 * t) * THREADS] = aq[t], sum[(2 * t + 1) * THREADS] = ar[t];
            return;
        }
    }
    if (i < c.len) {
        const long row = ((c.b * p.tokens + c.t0 + i) * p.hk + hk) * p.dk_;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const facc vq = aq[t], vk = ar[t];
            const int d0 = 16 * (half * NT + t) + 4 * g4;
            T *a = static_cast<T *>(p.dq) + row + d0, *b = static_cast<T *>(p.dk) + row + d0;
            if (p.vec_dqk && d0 + 4 <= p.dk_) {
                float x[4] = {vq[0], vq[1], vq[2], vq[3]}, y[4] = {vk[0], vk[1], vk[2], vk[3]};
                Raw<T, 4> w;
                w.set(x);
                w.store(a);
                w.set(y);
                w.store(b);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (d0 + j < p.dk_) store1(a + j, vq[j]), store1(b + j, vk[j]);
            }
        }
    }
}

// ------------------------------------------------------------------ host

template <typename T>
bool rows_aligned(const void *p, const long (&st)[3], int n)
{
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    return !off_by(p, 16) && n % N == 0 && st[0] % N == 0 && st[1] % N == 0 && st[2] % N == 0;
}

template <typename F>
int big_lds(F *kernel, int bytes)
{
    if (bytes <= 64 * 1024) return SSM2D_OK;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return e == hipSuccess ? SSM2D_OK : hip_fail(e);
}

template <typename T, int KD, bool GRAD>
int chunk_passes(const DeltaArgs &a)
{
    ChunkParams p{};
    p.q = a.q, p.k = a.k, p.v = a.v, p.dout = a.dout, p.g = a.g, p.beta = a.beta, p.h_init = a.h_init, p.dh_last = a.dh_last, p.cu = a.cu;
    p.o = a.o, p.dq = a.dq, p.dk = a.dk, p.dv = a.dv, p.h_last = a.h_last, p.dg = a.dg, p.dbeta = a.dbeta, p.dh_init = a.dh_init;
    p.batch = a.batch, p.tokens = a.tokens, p.n_seq = a.n_seq, p.chunks_b = (a.tokens + kC - 1) / kC;
    // (a lane's offset in a chunk's rows of v and dout is kept in 32 bits)
    if (a.tokens > 1 && (a.vs[1] < 0 || a.vs[1] >= (1 << 26) || (GRAD && (a.os[1] < 0 || a.os[1] >= (1 << 26))))) return SSM2D_ERR_UNSUPPORTED;
    if (chunk_slots(p) >= (1 << 22)) return SSM2D_ERR_UNSUPPORTED;  // (grids; far beyond memory but for tiny heads)
    p.hk = a.hk, p.h = a.h, p.rep = a.h / a.hk, p.dk_ = a.dk_, p.dv_ = a.dv_, p.dvp = (a.dv_ + 31) / 32 * 32;
    for (int i = 0; i < 3; ++i) {
        p.qs[i] = a.qs[i], p.ks[i] = a.ks[i], p.vs[i] = a.vs[i], p.os[i] = a.os[i], p.gs[i] = a.gs[i], p.bs[i] = a.bs[i];
    }
    p.scale = a.scale;
    p.vec_qk = rows_aligned<T>(a.q, a.qs, a.dk_) && rows_aligned<T>(a.k, a.ks, a.dk_);
    p.vec_do = GRAD && rows_aligned<T>(a.dout, a.os, a.dv_);
    p.vec_v = rows_aligned<T>(a.v, a.vs, a.dv_);
    p.vec_o = !GRAD && a.dv_ % 4 == 0 && !off_by(a.o, 4 * sizeof(T));
    p.vec_dqk = GRAD && a.dk_ % 4 == 0 && !off_by(a.dq, 4 * sizeof(T)) && !off_by(a.dk, 4 * sizeof(T));
    constexpr int kDirs = GRAD ? 2 : 1;
    // columns a workgroup of the chains: 128 share what they read of a chunk,
    // narrower states would leave waves idle (both measured at seq_chain)
    const bool wide = !GRAD && p.dvp > 64, slim = !GRAD && p.dvp <= 32;
    const int cols = wide ? 128 : 64, vb = (p.dvp + cols - 1) / cols, pb = (p.dvp + KD + cols - 1) / cols;
    // Measured: a join takes 2 us of d_k' = 128, 0.3 of 32, a step 5 and 3.3 us. Two
    // workgroups fit a compute unit where the state is small (2 x 12 heads of 32 x 32,
    // 12544 tokens, bf16 forward and backward: 440 us planned with one, 355 with two).
    const Extent x{a.batch, a.tokens, a.n_seq, a.hk, p.rep, KD, p.dvp, cols, GRAD, KD <= 64 ? 512 : 256, KD == 128 ? 0.4 : (KD == 64 ? 0.3 : 0.1)};
    const Passes plan = plan_passes(x);
    const Share &share = plan.share;
    p.nseg = plan.cuts.nseg, p.seg_len = plan.cuts.seg_len;
    // (so many chains at once take a workspace of 170 GiB and more)
    if (seg_count(p) * plan.nhk * p.rep > most_groups(512)) return SSM2D_ERR_UNSUPPORTED;
    void *ws = nullptr;
    int rc = get_aux_ws(a.dev, a.stream, kSlotDelta, plan.bytes(x), &ws);
    if (rc != SSM2D_OK) return rc;
    const hipStream_t s = static_cast<hipStream_t>(a.stream);
    for (p.hk0 = 0; p.hk0 < a.hk; p.hk0 += plan.nhk) {
        p.nhk = std::min(plan.nhk, a.hk - p.hk0);
        p.nh = p.nhk * p.rep;
        unsigned char *w = static_cast<unsigned char *>(ws);
        auto take = [&](size_t bytes) {
            unsigned char *at = w;
            w += bytes * p.nh;
            return at;
        };
        p.m = reinterpret_cast<float *>(take(share.tri));
        (GRAD ? p.mt : p.pm) = reinterpret_cast<float *>(take(share.tri));
        if (GRAD) {
            p.s0 = reinterpret_cast<float *>(take(share.state));
            p.e = reinterpret_cast<float *>(take(share.row));
            p.d1 = reinterpret_cast<float *>(take(share.state));
            p.dr = reinterpret_cast<float *>(take(share.row));
            p.z = reinterpret_cast<float *>(take(share.row));
        }
        p.gates = reinterpret_cast<float *>(take(share.gates));
        if (p.nseg > 1) {
            p.seg_at = reinterpret_cast<word4 *>(take(share.seg_a));
            if (GRAD) p.seg_a = reinterpret_cast<word4 *>(take(share.seg_a));
            p.seg_s = reinterpret_cast<float *>(take(share.seg_s));
            if (GRAD) p.seg_d = reinterpret_cast<float *>(take(share.seg_s));
        }
        p.sum = reinterpret_cast<float *>(w);
        const unsigned slots = static_cast<unsigned>(chunk_slots(p)), nk = static_cast<unsigned>(p.nhk), nh = static_cast<unsigned>(p.nh);
        delta_prep<T, KD, GRAD><<<dim3(slots, nk), dim3(256), 0, s>>>(p);
        if ((rc = launched()) != SSM2D_OK) return rc;
        if constexpr (GRAD) {
            constexpr int kZ = ZLds<T, KD>::kBytes;
            if ((rc = big_lds(delta_z<T, KD>, kZ)) != SSM2D_OK) return rc;
            delta_z<T, KD><<<dim3(slots, nh), dim3(256), kZ, s>>>(p);
            if ((rc = launched()) != SSM2D_OK) return rc;
        }
        auto run_chains = [&](auto probe, auto threads) -> int {
            constexpr bool PROBE = decltype(probe)::value;
            constexpr int THREADS = decltype(threads)::value;
            constexpr int kF = SeqBuf<T, KD, false, !GRAD && !PROBE, THREADS>::kBytes, kB = SeqBuf<T, KD, true, false, THREADS>::kBytes;
            constexpr int kSeq = GRAD && kB > kF ? kB : kF;
            const int st2 = big_lds(delta_seq<T, KD, GRAD, PROBE, THREADS>, kSeq);
            if (st2 != SSM2D_OK) return st2;
            const unsigned groups = static_cast<unsigned>((PROBE ? seg_places(p) : seg_count(p)) * p.nh);
            delta_seq<T, KD, GRAD, PROBE, THREADS><<<dim3(groups, static_cast<unsigned>(PROBE ? pb : vb), kDirs), dim3(THREADS), kSeq, s>>>(p);
            return launched();
        };
        auto chains_of = [&](auto probe) -> int {
            if constexpr (!GRAD) {
                if (wide) return run_chains(probe, std::integral_constant<int, 512>{});
                if constexpr (!decltype(probe)::value) {
                    if (slim) return run_chains(probe, std::integral_constant<int, 128>{});
                }
            }
            return run_chains(probe, std::integral_constant<int, 256>{});
        };
        if (p.nseg > 1) {
            if ((rc = chains_of(std::true_type{})) != SSM2D_OK) return rc;
            const unsigned joins = static_cast<unsigned>(join_count(p) * p.nh);
            delta_join<T, KD, GRAD><<<dim3(joins, static_cast<unsigned>(p.dvp / 16), kDirs), dim3(KD == 32 ? 64 : KD * 4), 0, s>>>(p);
            if ((rc = launched()) != SSM2D_OK) return rc;
        }
        if ((rc = chains_of(std::false_type{})) != SSM2D_OK) return rc;
        if constexpr (GRAD) {
            constexpr int kL = LocalLds<T, KD>::kBytes, kWaves = KD <= 64 ? 4 : 8;
            if ((rc = big_lds(delta_local<T, KD, kWaves>, kL)) != SSM2D_OK) return rc;
            for (p.turn = 0; p.turn < p.rep; ++p.turn) {
                delta_local<T, KD, kWaves><<<dim3(slots, nk), dim3(kWaves * 64), kL, s>>>(p);
                if ((rc = launched()) != SSM2D_OK) return rc;
            }
        }
    }
    return SSM2D_OK;
}

template <typename T, bool GRAD>
int chunk_kd(const DeltaArgs &a)
{
    if (a.dk_ <= 32) return chunk_passes<T, 32, GRAD>(a);
    if (a.dk_ <= 64) return chunk_passes<T, 64, GRAD>(a);
    return chunk_passes<T, 128, GRAD>(a);
}

}  // namespace ssm2d_impl
