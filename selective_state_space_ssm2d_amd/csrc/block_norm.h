// libssm2d: the norms after a block and before the next one, fused with the
// block's gate, its scale and the residual stream (include/ssm2d_block.h has the
// formulas), forward and backward.
//
// Memory-bound: each input is read once and each output written once (12544 rows of
// 768, bf16 with a float32 residual: 26 us, 5.1 TB/s; backward, 12408 rows of 771: 42 us, 3.6
// TB/s, where two waves a SIMD, as many as its 206 registers allow, do not ask for all). A row
// belongs to 16 lanes up to 16 waves, a lane holds NCH pieces of VEC consecutive
// channels in registers as they were read, and both norms' statistics and the
// outputs come from there. The backward computes the forward again from the
// same registers, so nothing of it is kept in memory: it has three rounds of
// sums a row (the squares of the normed input; the squares of out together with
// dy next_weight out, which the norm before the next block needs; and the
// product for the norm after the block).
// dweight, dscale and dnext_weight: each workgroup loops over rows, keeps its
// sums in registers and writes one partial row; fold_rows adds them in a fixed
// order.
// Statistics, sums and out as y sees it are fp32; bf16 outputs are rounded once.
// Two forms are far from memory's rate. Groups that neighbouring lanes do not hold (not
// 2^i pieces, or more than 64): each lane adds up its whole group, so that
// a row costs channels by pieces a group, and where a group is no whole number of 16-byte pieces the
// pieces are single channels: 12544 rows of 4092 in 12 groups 1.25 ms forward and 4.7 backward, of 4004 in
// 4 3.2 and 13; of 4096 in one 0.12 and 0.14. And the backward of more than 4096 channels,
// whose 16 waves have 128 registers a lane and spill: 4096 rows of 8192 0.15 ms, of 16384 0.8.
#pragma once

#include "block_common.h"

namespace ssm2d_impl {
namespace norm {

struct NormParams {
    const void *x, *gate, *res, *dout, *dy;
    const float *weight, *scale, *next;
    void *out, *y, *dx, *dgate, *dres;
    float *part;  // [workgroup][3][n]: dweight, dscale, dnext_weight
    long rows;
    int n, groups, per;  // per: pieces of VEC channels a group has
    long ldx, ldg, ldr, ldo, ldy;
    float eps, inv_n, inv_g;
    int on, first, sigmoid, sums;
};

template <int LPR>
constexpr int kThreads = LPR > 256 ? LPR : 256;
template <int LPR>
constexpr int kRows = LPR >= 256 ? 1 : 256 / LPR;  // rows a workgroup holds at once

// Sum over the LPR lanes of a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float *buf)
{
    v = lane_sum<(LPR > 64 ? 64 : LPR)>(v);
    if constexpr (LPR > 64) {
        constexpr int kWaves = LPR / 64;
        const int wave = threadIdx.x / 64;
        __syncthreads();  // (the last use of buf has been read)
        if (threadIdx.x % 64 == 0) buf[wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += buf[(wave / kWaves) * kWaves + w];
    }
    return v;
}

// Groups of 2^i pieces that neighbouring lanes hold.
template <int LPR>
__host__ __device__ constexpr bool in_lanes(int per)
{
    return (per & (per - 1)) == 0 && per <= (LPR > 64 ? 64 : LPR);
}

// For each of a lane's pieces the sum over its group's pieces, from sums of each
// piece. Groups that no neighbouring lanes hold go through `pieces` (LDS, one
// float a piece of the row), each lane adding up its group.
template <int NCH, int LPR>
__device__ __forceinline__ void group_sums(float (&s)[NCH], const NormParams &p, float *buf, float *pieces)
{
    if (p.groups == 1) {
        float v = 0.0f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) v += s[c];
        v = row_sum<LPR>(v, buf);
#pragma unroll
        for (int c = 0; c < NCH; ++c) s[c] = v;
        return;
    }
    if (in_lanes<LPR>(p.per)) {
        auto lanes = [&](auto w) __attribute__((always_inline)) {
#pragma unroll
            for (int c = 0; c < NCH; ++c) s[c] = lane_sum<decltype(w)::value>(s[c]);
        };
        using std::integral_constant;
        switch (p.per) {
        case 1: return;
        case 2: return lanes(integral_constant<int, 2>{});
        case 4: return lanes(integral_constant<int, 4>{});
        case 8: return lanes(integral_constant<int, 8>{});
        case 16: return lanes(integral_constant<int, 16>{});
        case 32: return lanes(integral_constant<int, 32>{});
        default: return lanes(integral_constant<int, 64>{});
        }
    }
    const int t = static_cast<int>(threadIdx.x) % LPR;
    float *mine = pieces + (threadIdx.x / LPR) * NCH * LPR;
    __syncthreads();  // (the last use of pieces has been read)
#pragma unroll
    for (int c = 0; c < NCH; ++c) mine[c * LPR + t] = s[c];
    __syncthreads();
    const int last = p.groups - 1;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        // (pieces past the row read its last group)
        const float *g = mine + min((c * LPR + t) / p.per, last) * p.per;
        float v = 0.0f;
        for (int i = 0; i < p.per; ++i) v += g[i];
        s[c] = v;
    }
}

// Where a lane's pieces lie: piece q of a row is channels VEC q .. VEC q + VEC - 1,
// at any alignment. TAIL: the last piece of a row reaches back over the one
// before, so that it is whole too; the channels that both hold get the same
// values from both, and count once in sums. Pieces past the row are its last
// one again, and count nowhere.
template <int VEC, int NCH, int LPR, bool TAIL>
struct Pieces {
    int n;
    __device__ __forceinline__ int place(int c) const { return (c * LPR + static_cast<int>(threadIdx.x) % LPR) * VEC; }
    __device__ __forceinline__ int first(int c) const { return min(place(c), n - VEC); }
    __device__ __forceinline__ bool in(int c) const { return place(c) < n; }
    // whether element j of piece c is this piece's own
    __device__ __forceinline__ bool own(int c, int j) const { return in(c) && (!TAIL || first(c) + j >= place(c)); }
    __device__ __forceinline__ float count(int c, int j) const { return TAIL && !own(c, j) ? 0.0f : 1.0f; }
    template <typename U>
    __device__ __forceinline__ void load(const void *p, long at, Raw<U, VEC> (&v)[NCH]) const
    {
#pragma unroll
        for (int c = 0; c < NCH; ++c) v[c].load_any(static_cast<const U *>(p) + at + first(c));
    }
    // zeros past the row (where there is no TAIL to tell what counts)
    template <typename U>
    __device__ __forceinline__ void trim(Raw<U, VEC> (&v)[NCH]) const
    {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
            if (!TAIL && !in(c)) v[c].clear();
    }
    // Channel parameters, without a branch a load.
    __device__ __forceinline__ void params(const float *src, float (&out)[NCH][VEC]) const
    {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int j = 0; j < VEC; ++j) out[c][j] = 1.0f;
        if (!src) return;
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int j = 0; j < VEC; ++j) out[c][j] = src[first(c) + j];
    }
    template <typename U>
    __device__ __forceinline__ void store(void *p, long at, int c, const float (&v)[VEC]) const
    {
        if (!in(c)) return;
        Raw<U, VEC> o;
        o.set(v);
        o.store_any(static_cast<U *>(p) + at + first(c));
    }
};

enum : int { kNoGate = 0, kGateAfter = 1, kGateFirst = 2 };

// T: x, gate and y; TR: residual and out.
template <typename T, typename TR, int VEC, int NCH, int LPR, int GATE, bool TAIL>
__global__ __launch_bounds__(kThreads<LPR>) void block_norm_fwd_kernel(const NormParams p)
{
    __shared__ float red[2][16];
    extern __shared__ float pieces[];
    const int sub = threadIdx.x / LPR % kRows<LPR>;
    const long row0 = static_cast<long>(blockIdx.x) * kRows<LPR> + sub, step = static_cast<long>(gridDim.x) * kRows<LPR>;
    const Pieces<VEC, NCH, LPR, TAIL> lay{p.n};
    float w[NCH][VEC], sc[NCH][VEC], nw[NCH][VEC];
    lay.params(p.weight, w);
    lay.params(p.scale, sc);
    lay.params(p.next, nw);
    for (long row = row0; row - sub < p.rows; row += step) {
        const bool live = row < p.rows;
        const long at = live ? row : p.rows - 1;  // (rows past the end read the last one, and are not written)
        Raw<T, VEC> vx[NCH], vg[NCH];
        Raw<TR, VEC> vr[NCH];
        lay.load(p.x, at * p.ldx, vx);
        if (GATE != kNoGate) lay.load(p.gate, at * p.ldg, vg);
        if (p.res) {
            lay.load(p.res, at * p.ldr, vr);
        } else {
#pragma unroll
            for (int c = 0; c < NCH; ++c) vr[c].clear();
        }
        lay.trim(vx);
        if (GATE != kNoGate) lay.trim(vg);
        lay.trim(vr);
        auto act = [&](int c, int j) __attribute__((always_inline)) {
            const float z = vg[c].get(j);
            return sigmoid_for<T>(z) * (p.sigmoid ? 1.0f : z);
        };
        float u[NCH][VEC], s[NCH];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            s[c] = 0.0f;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                u[c][j] = vx[c].get(j);
                if (GATE == kGateFirst) u[c][j] *= act(c, j);
                s[c] += u[c][j] * u[c][j] * lay.count(c, j);
            }
        }
        if (p.on) {
            group_sums<NCH, LPR>(s, p, red[0], pieces);
#pragma unroll
            for (int c = 0; c < NCH; ++c) s[c] = lay.in(c) ? 1.0f / sqrtf(s[c] * p.inv_g + p.eps) : 0.0f;  // (past the row: of an empty group)
        } else {
#pragma unroll
            for (int c = 0; c < NCH; ++c) s[c] = 1.0f;
        }
        float q = 0.0f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                u[c][j] *= s[c] * w[c][j];
                if (GATE == kGateAfter) u[c][j] *= act(c, j);
                u[c][j] = u[c][j] * sc[c][j] + vr[c].get(j);
                q += u[c][j] * u[c][j] * lay.count(c, j);
            }
        }
        // (TAIL over several waves: out may be the residual's buffer, and two of
        // them read what one writes: not before all have what they read)
        const bool sum = p.y || (TAIL && LPR > 64);
        const float r2 = sum ? 1.0f / sqrtf(row_sum<LPR>(q, red[1]) * p.inv_n + p.eps) : 0.0f;
        if (!live) continue;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            lay.template store<TR>(p.out, row * p.n, c, u[c]);
            if (!p.y) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[c][j] *= r2 * nw[c][j];
            lay.template store<T>(p.y, row * p.n, c, u[c]);
        }
    }
}

template <typename T, typename TR, int VEC, int NCH, int LPR, int GATE, bool TAIL>
__global__ __launch_bounds__(kThreads<LPR>) void block_norm_bwd_kernel(const NormParams p)
{
    __shared__ float red[3][16];
    extern __shared__ float pieces[];
    const int t = static_cast<int>(threadIdx.x) % LPR, sub = threadIdx.x / LPR % kRows<LPR>;
    const long row0 = static_cast<long>(blockIdx.x) * kRows<LPR> + sub, step = static_cast<long>(gridDim.x) * kRows<LPR>;
    const Pieces<VEC, NCH, LPR, TAIL> lay{p.n};
    float w[NCH][VEC], sc[NCH][VEC], nw[NCH][VEC], sums[3][NCH][VEC];
    lay.params(p.weight, w);
    lay.params(p.scale, sc);
    lay.params(p.next, nw);
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int j = 0; j < VEC; ++j) sums[i][c][j] = 0.0f;
    // The next row is read while this one is worked on (not with 16 waves, whose
    // registers are all taken).
    constexpr bool kAhead = LPR < 1024;
    struct Row {
        Raw<T, VEC> x[NCH], g[NCH], y[NCH];
        Raw<TR, VEC> r[NCH], o[NCH];
    } next;
    auto fetch = [&](long row) __attribute__((always_inline)) {
        const long at = row < p.rows ? row : p.rows - 1;
        auto read = [&](const void *src, long ld, auto &v) __attribute__((always_inline)) {
            if (src) {
                lay.load(src, at * ld, v);
            } else {
#pragma unroll
                for (int c = 0; c < NCH; ++c) v[c].clear();
            }
        };
        read(p.x, p.ldx, next.x);
        if (GATE != kNoGate) read(p.gate, p.ldg, next.g);
        read(p.dout, p.ldo, next.o);
        read(p.dy, p.ldy, next.y);
        read(p.dy ? p.res : nullptr, p.ldr, next.r);
    };
    if (kAhead) fetch(row0);
    for (long row = row0; row - sub < p.rows; row += step) {
        const bool live = row < p.rows;
        if (!kAhead) fetch(row);
        Row now = next;
        if (kAhead && row + step - sub < p.rows) fetch(row + step);
        auto &vx = now.x;
        auto &vg = now.g;
        auto &vy = now.y;
        auto &vr = now.r;
        auto &vo = now.o;
        lay.trim(vx);
        if (GATE != kNoGate) lay.trim(vg);
        lay.trim(vo);
        lay.trim(vy);
        lay.trim(vr);
        // the gate's sigmoid f (act = f, or z f), the normed input, and 1 / rms of each piece's group
        float f[NCH][VEC], u[NCH][VEC], r[NCH];
        auto act = [&](int c, int j) __attribute__((always_inline)) { return f[c][j] * (p.sigmoid ? 1.0f : vg[c].get(j)); };
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            r[c] = 0.0f;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (GATE != kNoGate) f[c][j] = sigmoid_for<T>(vg[c].get(j));
                u[c][j] = vx[c].get(j);
                if (GATE == kGateFirst) u[c][j] *= act(c, j);
                r[c] += u[c][j] * u[c][j] * lay.count(c, j);
            }
        }
        if (p.on) {
            group_sums<NCH, LPR>(r, p, red[0], pieces);
#pragma unroll
            for (int c = 0; c < NCH; ++c) r[c] = lay.in(c) ? 1.0f / sqrtf(r[c] * p.inv_g + p.eps) : 0.0f;  // (as in the forward)
        } else {
#pragma unroll
            for (int c = 0; c < NCH; ++c) r[c] = 1.0f;
        }
        // (u becomes rms(u), or stays; then rms(u) weight, and m)
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[c][j] *= r[c];
        auto m_of = [&](int c, int j) __attribute__((always_inline)) {
            const float v = u[c][j] * w[c][j];
            return GATE == kGateAfter ? v * act(c, j) : v;
        };
        float r2 = 0.0f, mean = 0.0f;
        if (p.dy) {
            float q = 0.0f, k = 0.0f;
#pragma unroll
            for (int c = 0; c < NCH; ++c)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float out = m_of(c, j) * sc[c][j] + vr[c].get(j);
                    const float once = out * lay.count(c, j);
                    q += out * once;
                    k += vy[c].get(j) * nw[c][j] * once;
                }
            r2 = 1.0f / sqrtf(row_sum<LPR>(q, red[1]) * p.inv_n + p.eps);
            mean = row_sum<LPR>(k, red[2]) * r2 * p.inv_n;  // of dy next_weight rms(out)
        }
        float D[NCH][VEC], k[NCH];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            k[c] = 0.0f;
            float d[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                // (without dy nothing of out enters: a 0 by it would be NaN where out is not finite)
                const float m = m_of(c, j), dy = vy[c].get(j), xh = p.dy ? (m * sc[c][j] + vr[c].get(j)) * r2 : 0.0f;
                d[j] = vo[c].get(j);
                if (p.dy) d[j] += r2 * (dy * nw[c][j] - xh * mean);
                const float e = d[j] * sc[c][j], g = GATE == kGateAfter ? e * act(c, j) : e;
                D[c][j] = e;
                k[c] += g * w[c][j] * u[c][j] * lay.count(c, j);
                if (live) {
                    sums[2][c][j] += dy * xh;
                    sums[1][c][j] += d[j] * m;
                    sums[0][c][j] += g * u[c][j];
                }
            }
            if (p.dres && live) lay.template store<TR>(p.dres, row * p.n, c, d);
        }
        if (p.on) {
            group_sums<NCH, LPR>(k, p, red[0], pieces);
        } else {
#pragma unroll
            for (int c = 0; c < NCH; ++c) k[c] = 0.0f;
        }
        if (!live) continue;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            float dx[VEC], dg[VEC];
            const float kk = k[c] * p.inv_g;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float d = D[c][j], da = 0.0f;
                if (GATE == kGateAfter) da = d * u[c][j] * w[c][j], d *= act(c, j);
                if (p.on) d = r[c] * (d * w[c][j] - u[c][j] * kk);
                if (GATE == kGateFirst) da = d * vx[c].get(j), d *= act(c, j);
                dx[j] = d;
                if (GATE != kNoGate) {
                    const float rest = 1.0f - f[c][j];
                    dg[j] = da * f[c][j] * (p.sigmoid ? rest : 1.0f + vg[c].get(j) * rest);
                }
            }
            if (p.dx) lay.template store<T>(p.dx, row * p.n, c, dx);
            if (GATE != kNoGate && p.dgate) lay.template store<T>(p.dgate, row * p.n, c, dg);
        }
    }
    if (!p.sums) return;
    // the workgroup's partial row: its rows' waves one after the other
    float *part = p.part + static_cast<long>(blockIdx.x) * 3 * p.n;
    if constexpr (kRows<LPR> == 1) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int c = 0; c < NCH; ++c)
#pragma unroll
                for (int j = 0; j < VEC; ++j)
                    if (lay.own(c, j)) part[i * p.n + lay.first(c) + j] = sums[i][c][j];
    } else {
        __shared__ float fold[LPR * NCH * VEC];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            for (int k = 0; k < kRows<LPR>; ++k) {
                __syncthreads();
                if (sub == k) {
#pragma unroll
                    for (int c = 0; c < NCH; ++c)
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            const int at = (c * VEC + j) * LPR + t;
                            if (k == 0) fold[at] = sums[i][c][j];
                            else fold[at] += sums[i][c][j];
                        }
                }
            }
            __syncthreads();
            for (int col = threadIdx.x; col < p.n; col += kThreads<LPR>) {
                const int piece = col / VEC, j = col - min(piece * VEC, p.n - VEC);
                part[i * p.n + col] = fold[(piece / LPR * VEC + j) * LPR + piece % LPR];
            }
        }
    }
}

// ------------------------------------------------------------------ host

// Calls f(NCH, lanes a row) with what holds a row of n channels in pieces of VEC:
// 16 channels a lane in the forward where a wave has a row, 8 in the backward,
// where 16 take more than 256 registers with the parameters and sums of each (beyond 8192
// channels there is no other way, and 16 waves have 128).
template <int VEC, bool BWD, typename F>
int pick_row(int n, F &&f)
{
    using std::integral_constant;
#define SSM2D_ROW(NCH, LPR) f(integral_constant<int, NCH>{}, integral_constant<int, LPR>{})
    constexpr int k8 = 8 / VEC, k16 = 16 / VEC;
    if (n <= 128) return SSM2D_ROW(k8, 16);
    if constexpr (VEC <= 4) {
        if (n <= 256) return SSM2D_ROW(4 / VEC, 64);
    }
    if (n <= 512) return SSM2D_ROW(k8, 64);
    if constexpr (BWD) {
        if (n <= 1024) return SSM2D_ROW(k8, 128);
        if (n <= 2048) return SSM2D_ROW(k8, 256);
        if (n <= 4096) return SSM2D_ROW(k8, 512);
    } else {
        if (n <= 1024) return SSM2D_ROW(k16, 64);
        if (n <= 2048) return SSM2D_ROW(k8, 256);
        if (n <= 4096) return SSM2D_ROW(k16, 256);
    }
    if (n <= 8192) return SSM2D_ROW(k8, 1024);
    return SSM2D_ROW(k16, 1024);
#undef SSM2D_ROW
}

constexpr int kMaxParts = 512;  // partial rows of the channel sums

// Workgroups: as many rows each as fit evenly.
inline unsigned even_blocks(long groups, long most)
{
    const long rounds = (groups + most - 1) / most;
    return static_cast<unsigned>((groups + rounds - 1) / rounds);
}

// One type's kernels, forward or backward (block_norm_*.hip).
template <typename T, typename TR, bool BWD>
int launch_norm(NormParams p, float *dweight, float *dscale, float *dnext, hipStream_t s)
{
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const int per = p.n / p.groups;
    auto with = [&](auto vec, auto tail, auto gate) {
        constexpr int VEC = decltype(vec)::value, GATE = decltype(gate)::value;
        constexpr bool TAIL = decltype(tail)::value;
        p.per = per / VEC;
        return pick_row<VEC, BWD>(p.n, [&](auto nch, auto lanes) {
            constexpr int NCH = decltype(nch)::value, LPR = decltype(lanes)::value;
            const bool lds = p.on && p.groups > 1 && !in_lanes<LPR>(p.per);
            const size_t bytes = lds ? static_cast<size_t>(kRows<LPR>) * NCH * LPR * sizeof(float) : 0;
            const long groups = (p.rows + kRows<LPR> - 1) / kRows<LPR>;
            if constexpr (!BWD) {
                // (enough to fill the chip; a workgroup reads the parameters once for its rows)
                const unsigned grid = even_blocks(groups, LPR == 1024 ? 1024 : 4096);
                block_norm_fwd_kernel<T, TR, VEC, NCH, LPR, GATE, TAIL><<<dim3(grid), dim3(kThreads<LPR>), bytes, s>>>(p);
                return launched();
            } else {
                const unsigned grid = even_blocks(groups, LPR == 1024 ? 256 : kMaxParts);
                block_norm_bwd_kernel<T, TR, VEC, NCH, LPR, GATE, TAIL><<<dim3(grid), dim3(kThreads<LPR>), bytes, s>>>(p);
                const int st = launched();
                if (st != SSM2D_OK || !p.sums) return st;
                fold_three<<<dim3(fold_blocks(p.n), 3), dim3(kFoldThreads), 0, s>>>(p.part, static_cast<int>(grid), p.n, dweight, dscale, dnext);
                return launched();
            }
        });
    };
    using std::integral_constant;
    auto gates = [&](auto vec, auto tail) {
        if (!p.gate) return with(vec, tail, integral_constant<int, kNoGate>{});
        if (p.first) return with(vec, tail, integral_constant<int, kGateFirst>{});
        return with(vec, tail, integral_constant<int, kGateAfter>{});
    };
    // (a piece belongs to one group)
    if (p.n < V || (p.groups > 1 && per % V != 0)) return gates(integral_constant<int, 1>{}, std::false_type{});
    return p.n % V ? gates(integral_constant<int, V>{}, std::true_type{}) : gates(integral_constant<int, V>{}, std::false_type{});
}

}  // namespace norm
}  // namespace ssm2d_impl
