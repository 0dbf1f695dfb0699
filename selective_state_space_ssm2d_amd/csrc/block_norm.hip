// libssm2d: the norms after a block and before the next one, fused with the
// block's gate, its scale and the residual stream (include/ssm2d_block.h has the
// formulas), forward and backward.
//
// Memory-bound: each input is read once and each output written once. A row
// belongs to 1, 4 or 16 waves, a lane holds NCH pieces of VEC consecutive
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
#include "block_common.h"

namespace ssm2d_impl {
namespace {

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

template <int WPR>
constexpr int kThreads = WPR * 64 > 256 ? WPR * 64 : 256;
template <int WPR>
constexpr int kRows = WPR >= 4 ? 1 : 4 / WPR;  // rows a workgroup holds at once

template <int WPR>
__device__ __forceinline__ float row_sum(float v, float *buf)
{
    v = lane_sum<64>(v);
    if constexpr (WPR > 1) {
        const int wave = threadIdx.x / 64;
        __syncthreads();  // (the last use of buf has been read)
        if (threadIdx.x % 64 == 0) buf[wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) v += buf[(wave / WPR) * WPR + w];
    }
    return v;
}

// For each of a lane's pieces the sum over its group's pieces, from sums of each
// piece. Groups of 2^i <= 64 pieces are neighbouring lanes; others go through
// `pieces` (LDS, one float a piece of the row), each lane adding up its group.
template <int NCH, int WPR>
__device__ __forceinline__ void group_sums(float (&s)[NCH], const NormParams &p, float *buf, float *pieces)
{
    if (p.groups == 1) {
        float v = 0.0f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) v += s[c];
        v = row_sum<WPR>(v, buf);
#pragma unroll
        for (int c = 0; c < NCH; ++c) s[c] = v;
        return;
    }
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
    case 64: return lanes(integral_constant<int, 64>{});
    default: break;
    }
    const int t = static_cast<int>(threadIdx.x) % (WPR * 64);
    float *mine = pieces + (threadIdx.x / (WPR * 64)) * NCH * WPR * 64;
    __syncthreads();  // (the last use of pieces has been read)
#pragma unroll
    for (int c = 0; c < NCH; ++c) mine[c * WPR * 64 + t] = s[c];
    __syncthreads();
    const int last = p.groups - 1;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        // (pieces past the row read its last group)
        const float *g = mine + min((c * WPR * 64 + t) / p.per, last) * p.per;
        float v = 0.0f;
        for (int i = 0; i < p.per; ++i) v += g[i];
        s[c] = v;
    }
}

// A lane's channel parameters; channels past the row get 0.
template <int VEC, int NCH, int WPR>
__device__ __forceinline__ void row_params(const float *src, int n, float (&out)[NCH][VEC])
{
    const int t = static_cast<int>(threadIdx.x) % (WPR * 64);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const int col = (c * WPR * 64 + t) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) out[c][j] = col < n ? (src ? src[col + j] : 1.0f) : 0.0f;
    }
}

template <typename T, int VEC, int NCH, int WPR>
__device__ __forceinline__ void row_load(const void *src, long at, int n, Raw<T, VEC> (&v)[NCH])
{
    const int t = static_cast<int>(threadIdx.x) % (WPR * 64);
#pragma unroll
    for (int c = 0; c < NCH; ++c) v[c].load(static_cast<const T *>(src) + at + min((c * WPR * 64 + t) * VEC, n - VEC));
}
template <typename T, int VEC, int NCH, int WPR>
__device__ __forceinline__ void row_trim(int n, Raw<T, VEC> (&v)[NCH])
{
    const int t = static_cast<int>(threadIdx.x) % (WPR * 64);
#pragma unroll
    for (int c = 0; c < NCH; ++c)
        if ((c * WPR * 64 + t) * VEC >= n) v[c].clear();
}

// T: x, gate and y; TR: residual and out.
template <typename T, typename TR, int VEC, int NCH, int WPR>
__global__ __launch_bounds__(kThreads<WPR>) void block_norm_fwd_kernel(const NormParams p)
{
    __shared__ float red[2][16];
    extern __shared__ float pieces[];
    const int t = static_cast<int>(threadIdx.x) % (WPR * 64);
    float w[NCH][VEC], sc[NCH][VEC], nw[NCH][VEC];
    row_params<VEC, NCH, WPR>(p.weight, p.n, w);
    row_params<VEC, NCH, WPR>(p.scale, p.n, sc);
    row_params<VEC, NCH, WPR>(p.next, p.n, nw);
    for (long r0 = static_cast<long>(blockIdx.x) * kRows<WPR>; r0 < p.rows; r0 += static_cast<long>(gridDim.x) * kRows<WPR>) {
        const long row = r0 + (WPR >= 4 ? 0 : threadIdx.x / (WPR * 64));
        const bool live = row < p.rows;
        const long at = live ? row : p.rows - 1;  // (rows past the end read the last one, and are not written)
        Raw<T, VEC> vx[NCH], vg[NCH];
        Raw<TR, VEC> vr[NCH];
        row_load<T, VEC, NCH, WPR>(p.x, at * p.ldx, p.n, vx);
        if (p.gate) row_load<T, VEC, NCH, WPR>(p.gate, at * p.ldg, p.n, vg);
        if (p.res) row_load<TR, VEC, NCH, WPR>(p.res, at * p.ldr, p.n, vr);
        row_trim<T, VEC, NCH, WPR>(p.n, vx);
        float u[NCH][VEC], s[NCH];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            s[c] = 0.0f;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                u[c][j] = vx[c].get(j);
                if (p.gate && p.first) {
                    const float z = vg[c].get(j), f = sigmoid_for<T>(z);
                    u[c][j] *= p.sigmoid ? f : z * f;
                }
                s[c] += u[c][j] * u[c][j];
            }
        }
        if (p.on) {
            group_sums<NCH, WPR>(s, p, red[0], pieces);
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                const float r = 1.0f / sqrtf(s[c] * p.inv_g + p.eps);
#pragma unroll
                for (int j = 0; j < VEC; ++j) u[c][j] *= r * w[c][j];
            }
        }
        float q = 0.0f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int col = (c * WPR * 64 + t) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (p.gate && !p.first) {
                    const float z = vg[c].get(j), f = sigmoid_for<T>(z);
                    u[c][j] *= p.sigmoid ? f : z * f;
                }
                u[c][j] *= sc[c][j];
                if (p.res) u[c][j] += vr[c].get(j);
                if (col < p.n) q += u[c][j] * u[c][j];
            }
            if (live && col < p.n) {
                Raw<TR, VEC> o;
                o.set(u[c]);
                o.store(static_cast<TR *>(p.out) + row * p.n + col);
            }
        }
        if (!p.y) continue;
        const float r2 = 1.0f / sqrtf(row_sum<WPR>(q, red[1]) * p.inv_n + p.eps);
        if (!live) continue;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int col = (c * WPR * 64 + t) * VEC;
            if (col >= p.n) continue;
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] = u[c][j] * r2 * nw[c][j];
            Raw<T, VEC> v;
            v.set(o);
            v.store(static_cast<T *>(p.y) + row * p.n + col);
        }
    }
}

template <typename T, typename TR, int VEC, int NCH, int WPR>
__global__ __launch_bounds__(kThreads<WPR>) void block_norm_bwd_kernel(const NormParams p)
{
    __shared__ float red[3][16];
    extern __shared__ float pieces[];
    const int t = static_cast<int>(threadIdx.x) % (WPR * 64);
    float w[NCH][VEC], sc[NCH][VEC], nw[NCH][VEC], sums[3][NCH][VEC];
    row_params<VEC, NCH, WPR>(p.weight, p.n, w);
    row_params<VEC, NCH, WPR>(p.scale, p.n, sc);
    row_params<VEC, NCH, WPR>(p.next, p.n, nw);
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int j = 0; j < VEC; ++j) sums[i][c][j] = 0.0f;
    const bool gated = p.gate != nullptr;
    for (long r0 = static_cast<long>(blockIdx.x) * kRows<WPR>; r0 < p.rows; r0 += static_cast<long>(gridDim.x) * kRows<WPR>) {
        const long row = r0 + (WPR >= 4 ? 0 : threadIdx.x / (WPR * 64));
        const bool live = row < p.rows;
        const long at = live ? row : p.rows - 1;
        Raw<T, VEC> vx[NCH], vg[NCH], vy[NCH];
        Raw<TR, VEC> vr[NCH], vo[NCH];
        row_load<T, VEC, NCH, WPR>(p.x, at * p.ldx, p.n, vx);
        if (gated) row_load<T, VEC, NCH, WPR>(p.gate, at * p.ldg, p.n, vg);
        if (p.dout) row_load<TR, VEC, NCH, WPR>(p.dout, at * p.ldo, p.n, vo);
        if (p.dy) {
            row_load<T, VEC, NCH, WPR>(p.dy, at * p.ldy, p.n, vy);
            if (p.res) row_load<TR, VEC, NCH, WPR>(p.res, at * p.ldr, p.n, vr);
            row_trim<T, VEC, NCH, WPR>(p.n, vy);
            if (p.res) row_trim<TR, VEC, NCH, WPR>(p.n, vr);
        }
        row_trim<T, VEC, NCH, WPR>(p.n, vx);
        if (p.dout) row_trim<TR, VEC, NCH, WPR>(p.n, vo);
        if (gated) row_trim<T, VEC, NCH, WPR>(p.n, vg);
        // the gate's sigmoid f (act = f, or z f), and 1 / rms of each piece's group
        float f[NCH][VEC], r[NCH];
        auto act = [&](int c, int j) __attribute__((always_inline)) { return p.sigmoid ? f[c][j] : vg[c].get(j) * f[c][j]; };
        auto u_of = [&](int c, int j) __attribute__((always_inline)) {
            return gated && p.first ? vx[c].get(j) * act(c, j) : vx[c].get(j);
        };
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            r[c] = 0.0f;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (gated) f[c][j] = sigmoid_for<T>(vg[c].get(j));
                const float u = u_of(c, j);
                r[c] += u * u;
            }
        }
        if (p.on) {
            group_sums<NCH, WPR>(r, p, red[0], pieces);
#pragma unroll
            for (int c = 0; c < NCH; ++c) r[c] = 1.0f / sqrtf(r[c] * p.inv_g + p.eps);
        }
        // (rms(u) weight, or u), and m
        auto n_of = [&](int c, int j) __attribute__((always_inline)) { return p.on ? u_of(c, j) * r[c] * w[c][j] : u_of(c, j); };
        auto m_of = [&](int c, int j) __attribute__((always_inline)) { return gated && !p.first ? n_of(c, j) * act(c, j) : n_of(c, j); };
        float D[NCH][VEC];
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int j = 0; j < VEC; ++j) D[c][j] = p.dout ? vo[c].get(j) : 0.0f;
        if (p.dy) {
            float q = 0.0f, k = 0.0f;
#pragma unroll
            for (int c = 0; c < NCH; ++c)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float out = m_of(c, j) * sc[c][j] + (p.res ? vr[c].get(j) : 0.0f);
                    q += out * out;
                    k += vy[c].get(j) * nw[c][j] * out;
                }
            const float r2 = 1.0f / sqrtf(row_sum<WPR>(q, red[1]) * p.inv_n + p.eps);
            const float mean = row_sum<WPR>(k, red[2]) * r2 * p.inv_n;  // of dy next_weight rms(out)
#pragma unroll
            for (int c = 0; c < NCH; ++c)
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float xh = (m_of(c, j) * sc[c][j] + (p.res ? vr[c].get(j) : 0.0f)) * r2, dy = vy[c].get(j);
                    D[c][j] += r2 * (dy * nw[c][j] - xh * mean);
                    if (live) sums[2][c][j] += dy * xh;
                }
        }
        float k[NCH];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int col = (c * WPR * 64 + t) * VEC;
            if (p.dres && live && col < p.n) {
                Raw<TR, VEC> o;
                o.set(D[c]);
                o.store(static_cast<TR *>(p.dres) + row * p.n + col);
            }
            k[c] = 0.0f;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (live) sums[1][c][j] += D[c][j] * m_of(c, j);
                D[c][j] *= sc[c][j];
                if (p.on) {
                    const float xh = u_of(c, j) * r[c], d = gated && !p.first ? D[c][j] * act(c, j) : D[c][j];
                    if (live) sums[0][c][j] += d * xh;
                    k[c] += d * w[c][j] * xh;
                }
            }
        }
        if (p.on) group_sums<NCH, WPR>(k, p, red[0], pieces);
        if (!live) continue;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int col = (c * WPR * 64 + t) * VEC;
            if (col >= p.n) continue;
            float dx[VEC], dg[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float d = D[c][j], da = 0.0f;
                if (gated && !p.first) da = d * n_of(c, j), d *= act(c, j);
                if (p.on) d = r[c] * (d * w[c][j] - u_of(c, j) * r[c] * k[c] * p.inv_g);
                if (gated && p.first) da = d * vx[c].get(j), d *= act(c, j);
                dx[j] = d;
                if (gated) dg[j] = da * f[c][j] * (p.sigmoid ? 1.0f - f[c][j] : 1.0f + vg[c].get(j) * (1.0f - f[c][j]));
            }
            Raw<T, VEC> o;
            if (p.dx) {
                o.set(dx);
                o.store(static_cast<T *>(p.dx) + row * p.n + col);
            }
            if (gated && p.dgate) {
                o.set(dg);
                o.store(static_cast<T *>(p.dgate) + row * p.n + col);
            }
        }
    }
    if (!p.sums) return;
    // the workgroup's partial row: its rows' waves one after the other
    float *part = p.part + static_cast<long>(blockIdx.x) * 3 * p.n;
    if constexpr (kRows<WPR> == 1) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                const int col = (c * WPR * 64 + t) * VEC;
                if (col >= p.n) continue;
#pragma unroll
                for (int j = 0; j < VEC; ++j) part[i * p.n + col + j] = sums[i][c][j];
            }
    } else {
        __shared__ float fold[WPR * 64 * NCH * VEC];
        const int sub = threadIdx.x / (WPR * 64);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            for (int k = 0; k < kRows<WPR>; ++k) {
                __syncthreads();
                if (sub == k) {
#pragma unroll
                    for (int c = 0; c < NCH; ++c)
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            const int at = (c * VEC + j) * WPR * 64 + t;
                            if (k == 0) fold[at] = sums[i][c][j];
                            else fold[at] += sums[i][c][j];
                        }
                }
            }
            __syncthreads();
            for (int col = threadIdx.x; col < p.n; col += kThreads<WPR>) {
                const int piece = col / VEC;
                part[i * p.n + col] = fold[(piece / (WPR * 64) * VEC + col % VEC) * WPR * 64 + piece % (WPR * 64)];
            }
        }
    }
}

// ------------------------------------------------------------------ host

// Calls f(NCH, WPR) with what holds a row of n channels in pieces of VEC.
template <int VEC, typename F>
int pick_row(int n, F &&f)
{
    using std::integral_constant;
#define SSM2D_ROW(NCH, WPR) f(integral_constant<int, NCH>{}, integral_constant<int, WPR>{})
    constexpr int k8 = 8 / VEC, k16 = 16 / VEC;
    if constexpr (VEC <= 4) {
        if (n <= 256) return SSM2D_ROW(4 / VEC, 1);
    }
    if (n <= 512) return SSM2D_ROW(k8, 1);
    if (n <= 1024) return SSM2D_ROW(k16, 1);
    if (n <= 2048) return SSM2D_ROW(k8, 4);
    if (n <= 4096) return SSM2D_ROW(k16, 4);
    if (n <= 8192) return SSM2D_ROW(k8, 16);
    return SSM2D_ROW(k16, 16);
#undef SSM2D_ROW
}

constexpr int kMaxParts = 512;  // partial rows of the channel sums

// Workgroups: as many rows each as fit evenly.
unsigned even_blocks(long groups, long most)
{
    const long rounds = (groups + most - 1) / most;
    return static_cast<unsigned>((groups + rounds - 1) / rounds);
}

bool rows_by(const void *p, long stride, int v, size_t size) { return !p || (!off_by(p, v * size) && stride % v == 0); }

template <typename T, typename TR, bool BWD>
int launch_norm(NormParams p, float *dweight, float *dscale, float *dnext, hipStream_t s)
{
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const int per = p.n / p.groups;
    bool wide = p.n % V == 0 && per % V == 0;
    for (const auto &[ptr, ld] : {std::pair<const void *, long>{p.x, p.ldx}, {p.gate, p.ldg}, {p.dy, p.ldy}, {p.y, 0}, {p.dx, 0}, {p.dgate, 0}})
        wide = wide && rows_by(ptr, ld, V, sizeof(T));
    // (V elements of a wider residual are read 16 bytes at a time)
    for (const auto &[ptr, ld] : {std::pair<const void *, long>{p.res, p.ldr}, {p.dout, p.ldo}, {p.out, 0}, {p.dres, 0}})
        wide = wide && (!ptr || (!off_by(ptr, 16) && ld % V == 0));
    auto go = [&](auto vec) {
        constexpr int VEC = decltype(vec)::value;
        p.per = per / VEC;
        return pick_row<VEC>(p.n, [&](auto nch, auto wpr) {
            constexpr int NCH = decltype(nch)::value, WPR = decltype(wpr)::value;
            const bool lds = p.on && p.groups > 1 && !(p.per <= 64 && (p.per & (p.per - 1)) == 0);
            const size_t bytes = lds ? static_cast<size_t>(kRows<WPR>) * NCH * WPR * 64 * sizeof(float) : 0;
            const long groups = (p.rows + kRows<WPR> - 1) / kRows<WPR>;
            if constexpr (!BWD) {
                // (enough to fill the chip; a workgroup reads the parameters once for its rows)
                block_norm_fwd_kernel<T, TR, VEC, NCH, WPR><<<dim3(even_blocks(groups, WPR == 16 ? 1024 : 4096)), dim3(kThreads<WPR>), bytes, s>>>(p);
                return launched();
            } else {
                const unsigned grid = even_blocks(groups, WPR == 16 ? 256 : kMaxParts);
                block_norm_bwd_kernel<T, TR, VEC, NCH, WPR><<<dim3(grid), dim3(kThreads<WPR>), bytes, s>>>(p);
                int st = launched();
                float *dst[3] = {dweight, dscale, dnext};
                for (int i = 0; i < 3 && st == SSM2D_OK; ++i)
                    if (dst[i]) {
                        fold_rows<<<dim3(fold_blocks(p.n)), dim3(kFoldThreads), 0, s>>>(p.part + static_cast<long>(i) * p.n, static_cast<int>(grid), p.n,
                                                                                 3L * p.n, dst[i]);
                        st = launched();
                    }
                return st;
            }
        });
    };
    return wide ? go(std::integral_constant<int, V>{}) : go(std::integral_constant<int, 1>{});
}

constexpr uint32_t kNormFlags = SSM2D_NORM_ON | SSM2D_NORM_GATE_SIGMOID | SSM2D_NORM_GATE_FIRST | SSM2D_NORM_RESIDUAL_F32;

// SSM2D_OK and *work, or what is wrong with the shape.
int check_norm(const ssm2d_block_norm_shape *a, uint32_t flags, bool *work)
{
    *work = false;
    if (flags & ~kNormFlags) return SSM2D_ERR_BAD_FLAGS;
    if (!a) return SSM2D_ERR_NULLPTR;
    if (a->rows < 0 || a->n < 0 || a->groups < 1 || a->n % a->groups != 0) return SSM2D_ERR_BAD_DIM;
    if (a->n > SSM2D_NORM_MAX_N) return SSM2D_ERR_UNSUPPORTED;
    if (a->rows > (int64_t{1} << 50) / std::max<int64_t>(a->n, 1)) return SSM2D_ERR_UNSUPPORTED;
    for (const int64_t st : {a->x_stride, a->gate_stride, a->res_stride, a->dout_stride, a->dy_stride})
        if (st < 0) return SSM2D_ERR_BAD_DIM;
    *work = a->rows > 0 && a->n > 0;
    return SSM2D_OK;
}

NormParams norm_params(const ssm2d_block_norm_shape &a, float eps, uint32_t flags)
{
    NormParams p{};
    p.rows = a.rows, p.n = static_cast<int>(a.n), p.groups = static_cast<int>(a.groups);
    p.ldx = a.x_stride, p.ldg = a.gate_stride, p.ldr = a.res_stride, p.ldo = a.dout_stride, p.ldy = a.dy_stride;
    p.eps = eps, p.inv_n = 1.0f / static_cast<float>(a.n), p.inv_g = 1.0f / static_cast<float>(a.n / a.groups);
    p.on = (flags & SSM2D_NORM_ON) != 0, p.first = (flags & SSM2D_NORM_GATE_FIRST) != 0;
    p.sigmoid = (flags & SSM2D_NORM_GATE_SIGMOID) != 0;
    return p;
}

template <typename T>
int norm_fwd(const T *x, const T *gate, const void *res, const float *weight, const float *scale, const float *next, void *out, T *y,
             const ssm2d_block_norm_shape *a, float eps, uint32_t flags, void *stream)
{
    bool work = false;
    const int st = check_norm(a, flags, &work);
    if (st != SSM2D_OK || !work) return st;
    if (!x || !out) return SSM2D_ERR_NULLPTR;
    const bool f32 = sizeof(T) == 4 || (flags & SSM2D_NORM_RESIDUAL_F32);
    const size_t tr = f32 ? 4 : 2;
    if (off_by(x, sizeof(T)) || off_by(gate, sizeof(T)) || off_by(y, sizeof(T)) || off_by(res, tr) || off_by(out, tr) || off_by(weight, 4) ||
        off_by(scale, 4) || off_by(next, 4))
        return SSM2D_ERR_MISALIGNED;
    NormParams p = norm_params(*a, eps, flags);
    p.x = x, p.gate = gate, p.res = res, p.weight = weight, p.scale = scale, p.next = next, p.out = out, p.y = y;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return f32 ? launch_norm<T, float, false>(p, nullptr, nullptr, nullptr, s) : launch_norm<T, T, false>(p, nullptr, nullptr, nullptr, s);
}

int64_t norm_workspace(const ssm2d_block_norm_shape *a, uint32_t flags)
{
    bool work = false;
    const int st = check_norm(a, flags, &work);
    if (st != SSM2D_OK) return -st;
    return work ? std::min<int64_t>(a->rows, kMaxParts) * 3 * a->n * 4 : 0;
}

template <typename T>
int norm_bwd(const T *x, const T *gate, const void *res, const float *weight, const float *scale, const float *next, const void *dout,
             const T *dy, T *dx, T *dgate, void *dres, float *dweight, float *dscale, float *dnext, const ssm2d_block_norm_shape *a, float eps,
             uint32_t flags, void *ws, int64_t ws_bytes, void *stream)
{
    bool work = false;
    const int st = check_norm(a, flags, &work);
    if (st != SSM2D_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (off_by(dweight, 4) || off_by(dscale, 4) || off_by(dnext, 4)) return SSM2D_ERR_MISALIGNED;
    if (!work) {  // (sums over no rows)
        for (float *d : {dweight, dscale, dnext})
            if (d && a->n > 0) {
                clear_floats<<<dim3(static_cast<unsigned>((a->n + 255) / 256)), dim3(256), 0, s>>>(d, a->n);
                const int e = launched();
                if (e != SSM2D_OK) return e;
            }
        return SSM2D_OK;
    }
    if (!x) return SSM2D_ERR_NULLPTR;
    const bool f32 = sizeof(T) == 4 || (flags & SSM2D_NORM_RESIDUAL_F32);
    const size_t tr = f32 ? 4 : 2;
    if (off_by(x, sizeof(T)) || off_by(gate, sizeof(T)) || off_by(dy, sizeof(T)) || off_by(dx, sizeof(T)) || off_by(dgate, sizeof(T)) ||
        off_by(res, tr) || off_by(dout, tr) || off_by(dres, tr) || off_by(weight, 4) || off_by(scale, 4) || off_by(next, 4) || off_by(ws, 16))
        return SSM2D_ERR_MISALIGNED;
    NormParams p = norm_params(*a, eps, flags);
    p.x = x, p.gate = gate, p.res = res, p.weight = weight, p.scale = scale, p.next = next, p.dout = dout, p.dy = dy;
    p.dx = dx, p.dgate = dgate, p.dres = dres, p.sums = dweight || dscale || dnext;
    if (p.sums && (!ws || ws_bytes < norm_workspace(a, flags))) return SSM2D_ERR_NOMEM;
    p.part = static_cast<float *>(ws);
    return f32 ? launch_norm<T, float, true>(p, dweight, dscale, dnext, s) : launch_norm<T, T, true>(p, dweight, dscale, dnext, s);
}

}  // namespace
}  // namespace ssm2d_impl

extern "C" {

int ssm2d_block_norm_fwd(const float *x, const float *gate, const void *residual, const float *weight, const float *scale,
                         const float *next_weight, void *out, float *y, const ssm2d_block_norm_shape *shape, float eps, uint32_t flags,
                         void *stream)
{
    return ssm2d_impl::norm_fwd<float>(x, gate, residual, weight, scale, next_weight, out, y, shape, eps, flags, stream);
}

int ssm2d_block_norm_fwd_bf16(const uint16_t *x, const uint16_t *gate, const void *residual, const float *weight, const float *scale,
                              const float *next_weight, void *out, uint16_t *y, const ssm2d_block_norm_shape *shape, float eps,
                              uint32_t flags, void *stream)
{
    return ssm2d_impl::norm_fwd<uint16_t>(x, gate, residual, weight, scale, next_weight, out, y, shape, eps, flags, stream);
}

int64_t ssm2d_block_norm_bwd_workspace(const ssm2d_block_norm_shape *shape, uint32_t flags)
{
    return ssm2d_impl::norm_workspace(shape, flags);
}

int ssm2d_block_norm_bwd(const float *x, const float *gate, const void *residual, const float *weight, const float *scale,
                         const float *next_weight, const void *dout, const float *dy, float *dx, float *dgate, void *dresidual,
                         float *dweight, float *dscale, float *dnext_weight, const ssm2d_block_norm_shape *shape, float eps, uint32_t flags,
                         void *workspace, int64_t workspace_bytes, void *stream)
{
    return ssm2d_impl::norm_bwd<float>(x, gate, residual, weight, scale, next_weight, dout, dy, dx, dgate, dresidual, dweight, dscale,
                                       dnext_weight, shape, eps, flags, workspace, workspace_bytes, stream);
}

int ssm2d_block_norm_bwd_bf16(const uint16_t *x, const uint16_t *gate, const void *residual, const float *weight, const float *scale,
                              const float *next_weight, const void *dout, const uint16_t *dy, uint16_t *dx, uint16_t *dgate, void *dresidual,
                              float *dweight, float *dscale, float *dnext_weight, const ssm2d_block_norm_shape *shape, float eps,
                              uint32_t flags, void *workspace, int64_t workspace_bytes, void *stream)
{
    return ssm2d_impl::norm_bwd<uint16_t>(x, gate, residual, weight, scale, next_weight, dout, dy, dx, dgate, dresidual, dweight, dscale,
                                          dnext_weight, shape, eps, flags, workspace, workspace_bytes, stream);
}

}  // extern "C"
