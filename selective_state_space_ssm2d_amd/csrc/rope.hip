// libssm2d: rotary positions with several axes (include/ssm2d_ops.h has the
// formulas), queries and keys in one launch.
//
// Memory-bound: every element is read and written once. A workgroup takes a
// few tokens, first puts the cosine and sine of their angles into LDS (each
// angle serves all heads of its token), then walks the tokens' heads with
// 16-byte accesses where the addresses allow.
// The angle pos * inv_freq is kept as a product and its rounding error, and
// reduced by multiples of pi/2 in three parts (Cody and Waite), so cosine and
// sine are as exact at an angle of 2^20 as at 1; on [-pi/4, pi/4] they are
// their Taylor polynomials (the first term left out is below 2^-36). Angles
// beyond 2^20 go through fp64.
// Measured: q and k of 32 maps of 56 x 56 with 6 heads of 32 each, bf16: 27 us,
// 32 from memory (4.8 TB/s); 5 heads and 1 of 72 at 27918 positions, fp32,
// interleaved: 22 us, 4.4 TB/s.
// A bf16 output is rounded once, from the fp32 turn.
#include "ops_common.h"

namespace ssm2d_impl {
namespace {

constexpr int kMaxTable = 4096;  // (cos, sin) pairs a workgroup holds: 32 KiB

struct RopeParams {
    const void *q, *k;
    const int *pos;
    const float *freq;
    void *qo, *ko;
    long batch, tokens;
    int hq, hk, d, pairs, sec_end[SSM2D_ROPE_MAX_AXES];
    long qs[3], ks[3], pos_axis, pos_batch;
    float sign;
    int tok;  // tokens a workgroup
};

// cos and sin of pos * freq.
__device__ __forceinline__ float2 cos_sin(int pos, float freq)
{
    // (the sums of parts below rely on every operation rounding by itself)
#pragma clang fp contract(off)
    // pos in two parts, of 20 bits (with the sign) and 12, exact in fp32; the products' errors by fma
    const float ph = static_cast<float>(pos >> 12) * 4096.0f, pl = static_cast<float>(pos & 4095);
    const float a = ph * freq, ae = fmaf(ph, freq, -a);
    const float b = pl * freq, be = fmaf(pl, freq, -b);
    // a + b = hi + lo
    const float hi = a + b, z = hi - a;
    const float lo = (a - (hi - z)) + (b - z) + (ae + be);
    if (!(fabsf(hi) <= 1048576.0f)) {
        double sd, cd;
        sincos(static_cast<double>(pos) * static_cast<double>(freq), &sd, &cd);
        return make_float2(static_cast<float>(cd), static_cast<float>(sd));
    }
    // hi + lo - k pi/2, k = round(hi 2/pi); pi/2 as a sum of three floats: the
    // first product's remainder is a multiple of 2^-24 below 1, so exact
    const float k = rintf(hi * 0.636619772367581343f);
    const float r = fmaf(k, -1.57079637050628662109375f, hi);
    const float e = k * 4.37113882867379e-8f;
    const float e2 = fmaf(k, 4.37113882867379e-8f, -e) + k * 1.7151245100e-15f;
    float s = r + e;
    const float t = s - r;
    s += ((r - (s - t)) + (e - t)) + (lo + e2);
    const float s2 = s * s;
    // Taylor: 1/3! .. 1/11!, 1/2! .. 1/12!
    float sn = fmaf(s2, -2.5052108385441719e-8f, 2.7557319223985891e-6f);
    sn = fmaf(s2, sn, -1.9841269841269841e-4f);
    sn = fmaf(s2, sn, 8.3333333333333333e-3f);
    sn = fmaf(s2, sn, -1.6666666666666667e-1f);
    sn = fmaf(s * s2, sn, s);
    float cn = fmaf(s2, 2.0876756987868099e-9f, -2.7557319223985891e-7f);
    cn = fmaf(s2, cn, 2.4801587301587302e-5f);
    cn = fmaf(s2, cn, -1.3888888888888889e-3f);
    cn = fmaf(s2, cn, 4.1666666666666667e-2f);
    cn = fmaf(s2, cn, -0.5f);
    cn = fmaf(s2, cn, 1.0f);
    const int quad = static_cast<int>(k) & 3;
    const float c = (quad & 1) ? sn : cn, q = (quad & 1) ? cn : sn;
    return make_float2((quad == 1 || quad == 2) ? -c : c, (quad & 2) ? -q : q);
}

// All heads of the tokens [t0, t0 + nt) of batch b of one tensor. VEC
// elements at a time; pairs (p, P + p), or (2p, 2p + 1) when INTER.
template <typename T, int VEC, bool INTER>
__device__ __forceinline__ void turn(const T *in, T *out, const float2 *table, const RopeParams &p, const long (&st)[3], int heads,
                                     long b, long t0, int nt)
{
    const int P = p.pairs, d = p.d;
    // pieces of a head: the pairs' (VEC pairs from the two halves, or VEC / 2
    // neighbouring pairs, one where VEC = 1), then the copied dims'
    const int np = (INTER && VEC > 1) ? 2 * P / VEC : P / VEC, rest = (d - 2 * P) / VEC, per = np + rest;
    const int total = nt * heads * per;
    for (int i = threadIdx.x; i < total; i += 256) {
        const int th = i / per, piece = i - th * per;
        const int tok = th / heads, h = th - tok * heads;
        const T *src = in + b * st[0] + (t0 + tok) * st[1] + h * st[2];
        T *dst = out + ((b * p.tokens + t0 + tok) * heads + h) * d;
        const float2 *cs = table + tok * P;
        if (piece >= np) {
            const int at = 2 * P + (piece - np) * VEC;
            Raw<T, VEC> r;
            r.load(src + at);
            r.store(dst + at);
        } else if constexpr (INTER && VEC == 1) {
            const float2 a = cs[piece];
            const float x1 = widen1(src[2 * piece]), x2 = widen1(src[2 * piece + 1]);
            store1(dst + 2 * piece, x1 * a.x - x2 * a.y);
            store1(dst + 2 * piece + 1, x2 * a.x + x1 * a.y);
        } else if constexpr (INTER) {
            const int at = piece * VEC;
            Raw<T, VEC> r;
            r.load(src + at);
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
                const float2 a = cs[at / 2 + j];
                const float x1 = r.get(2 * j), x2 = r.get(2 * j + 1);
                o[2 * j] = x1 * a.x - x2 * a.y;
                o[2 * j + 1] = x2 * a.x + x1 * a.y;
            }
            r.set(o);
            r.store(dst + at);
        } else {
            const int at = piece * VEC;
            Raw<T, VEC> r1, r2;
            r1.load(src + at);
            r2.load(src + P + at);
            float o1[VEC], o2[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float2 a = cs[at + j];
                const float x1 = r1.get(j), x2 = r2.get(j);
                o1[j] = x1 * a.x - x2 * a.y;
                o2[j] = x2 * a.x + x1 * a.y;
            }
            r1.set(o1);
            r2.set(o2);
            r1.store(dst + at);
            r2.store(dst + P + at);
        }
    }
}

template <typename T, int VEC, bool INTER>
__global__ __launch_bounds__(256) void rope_kernel(RopeParams p)
{
    extern __shared__ float2 table[];
    const long tiles = (p.tokens + p.tok - 1) / p.tok;
    for (long w = blockIdx.x; w < tiles * p.batch; w += gridDim.x) {
        const long b = w / tiles, t0 = (w - b * tiles) * p.tok;
        const int nt = static_cast<int>(min(static_cast<long>(p.tok), p.tokens - t0));
        for (int i = threadIdx.x; i < nt * p.pairs; i += 256) {
            const int tok = i / p.pairs, q = i - tok * p.pairs;
            int axis = 0;
            while (q >= p.sec_end[axis]) ++axis;  // (q < pairs = the last section's end)
            const float2 cs = cos_sin(p.pos[axis * p.pos_axis + b * p.pos_batch + t0 + tok], p.freq[q]);
            table[i] = make_float2(cs.x, p.sign * cs.y);
        }
        __syncthreads();
        turn<T, VEC, INTER>(static_cast<const T *>(p.q), static_cast<T *>(p.qo), table, p, p.qs, p.hq, b, t0, nt);
        if (p.hk > 0) turn<T, VEC, INTER>(static_cast<const T *>(p.k), static_cast<T *>(p.ko), table, p, p.ks, p.hk, b, t0, nt);
        __syncthreads();
    }
}

template <typename T>
int rope_entry(const T *q, const T *k, const int32_t *pos, const float *freq, T *qo, T *ko, const ssm2d_rope_shape *sh, uint32_t flags,
               void *stream)
{
    if (flags & ~(SSM2D_ROPE_INTERLEAVED | SSM2D_ROPE_INVERSE)) return SSM2D_ERR_BAD_FLAGS;
    if (!sh) return SSM2D_ERR_NULLPTR;
    if (sh->batch < 0 || sh->tokens < 0 || sh->heads_q < 0 || sh->heads_k < 0 || sh->d < 0) return SSM2D_ERR_BAD_DIM;
    if (sh->n_axes < 1 || sh->n_axes > SSM2D_ROPE_MAX_AXES || sh->d > SSM2D_ROPE_MAX_D) return SSM2D_ERR_UNSUPPORTED;
    RopeParams p{};
    int64_t pairs = 0;
    for (int a = 0; a < SSM2D_ROPE_MAX_AXES; ++a) {
        if (a < sh->n_axes) {
            if (sh->sections[a] < 0 || sh->sections[a] > SSM2D_ROPE_MAX_D) return SSM2D_ERR_BAD_DIM;
            pairs += sh->sections[a];
        }
        p.sec_end[a] = static_cast<int>(pairs);
    }
    if (2 * pairs > sh->d) return SSM2D_ERR_BAD_DIM;
    if (sh->batch == 0 || sh->tokens == 0 || sh->d == 0 || (sh->heads_q == 0 && sh->heads_k == 0)) return SSM2D_OK;
    // (32-bit counts within a workgroup's tokens)
    if (sh->heads_q > 65536 || sh->heads_k > 65536 || static_cast<double>(sh->batch) * sh->tokens > 1e12) return SSM2D_ERR_UNSUPPORTED;
    if ((sh->heads_q > 0 && (!q || !qo)) || (sh->heads_k > 0 && (!k || !ko)) || (pairs > 0 && (!pos || !freq))) return SSM2D_ERR_NULLPTR;
    if (off_by(q, sizeof(T)) || off_by(k, sizeof(T)) || off_by(qo, sizeof(T)) || off_by(ko, sizeof(T)) || off_by(pos, 4) || off_by(freq, 4))
        return SSM2D_ERR_MISALIGNED;
    p.q = q, p.k = k, p.pos = pos, p.freq = freq, p.qo = qo, p.ko = ko;
    p.batch = sh->batch, p.tokens = sh->tokens;
    p.hq = static_cast<int>(sh->heads_q), p.hk = static_cast<int>(sh->heads_k), p.d = static_cast<int>(sh->d);
    p.pairs = static_cast<int>(pairs);
    for (int i = 0; i < 3; ++i) p.qs[i] = sh->q_stride[i], p.ks[i] = sh->k_stride[i];
    p.pos_axis = sh->pos_stride[0], p.pos_batch = sh->pos_stride[1];
    p.sign = (flags & SSM2D_ROPE_INVERSE) ? -1.0f : 1.0f;
    // Tokens a workgroup: about 64 KiB of reads and writes (the maps above: 27 us, 31
    // with 16 KiB, 29 with 256), within the table, fewer where that would leave
    // compute units without one.
    const int64_t row = (sh->heads_q + sh->heads_k) * sh->d * static_cast<int64_t>(sizeof(T)) * 2;
    int64_t tok = std::max<int64_t>(1, 65536 / row);
    if (pairs > 0) tok = std::min<int64_t>(tok, kMaxTable / pairs);
    while (tok > 1 && sh->batch * ((sh->tokens + tok - 1) / tok) < 1024) tok /= 2;
    tok = std::min(tok, sh->tokens);
    p.tok = static_cast<int>(tok);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(sh->batch * ((sh->tokens + tok - 1) / tok), 1 << 20));
    const size_t lds = static_cast<size_t>(tok * std::max<int64_t>(pairs, 1)) * sizeof(float2);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool inter = flags & SSM2D_ROPE_INTERLEAVED;
    // V elements at a time: pieces must not cross the halves of a head, and
    // every row of both tensors must start at a multiple of V. (Element by element
    // the same sizes reach half the bandwidth: bf16 heads of 50, 2.5 TB/s.)
    auto fits = [&](int v) {
        if (sh->d % v || (inter ? 2 * pairs : pairs) % v) return false;
        auto rows = [&](const T *in, const T *out, const int64_t (&st)[3]) {
            return !off_by(in, v * sizeof(T)) && !off_by(out, v * sizeof(T)) && st[0] % v == 0 && st[1] % v == 0 && st[2] % v == 0;
        };
        return (sh->heads_q == 0 || rows(q, qo, sh->q_stride)) && (sh->heads_k == 0 || rows(k, ko, sh->k_stride));
    };
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    return guarded([&] {
        std::lock_guard<std::recursive_mutex> lock(g_mutex);
        auto go = [&](auto vec) {
            constexpr int VEC = decltype(vec)::value;
            if (inter) rope_kernel<T, VEC, true><<<dim3(grid), dim3(256), lds, s>>>(p);
            else rope_kernel<T, VEC, false><<<dim3(grid), dim3(256), lds, s>>>(p);
            return launched();
        };
        if (fits(V)) return go(std::integral_constant<int, V>{});
        if (fits(V / 2)) return go(std::integral_constant<int, V / 2>{});
        return go(std::integral_constant<int, 1>{});
    });
}

}  // namespace
}  // namespace ssm2d_impl

extern "C" {

int ssm2d_rope(const float *q, const float *k, const int32_t *positions, const float *inv_freq, float *q_out, float *k_out,
               const ssm2d_rope_shape *shape, uint32_t flags, void *stream)
{
    return ssm2d_impl::rope_entry<float>(q, k, positions, inv_freq, q_out, k_out, shape, flags, stream);
}

int ssm2d_rope_bf16(const uint16_t *q, const uint16_t *k, const int32_t *positions, const float *inv_freq, uint16_t *q_out,
                    uint16_t *k_out, const ssm2d_rope_shape *shape, uint32_t flags, void *stream)
{
    return ssm2d_impl::rope_entry<uint16_t>(q, k, positions, inv_freq, q_out, k_out, shape, flags, stream);
}

}  // extern "C"
