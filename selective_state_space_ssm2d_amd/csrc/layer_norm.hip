// libssm2d: layer norm over the channels of token rows and of channels-first
// maps, forward and backward (include/ssm2d_ops.h has the formulas).
//
// Memory-bound: the forward reads x and writes y once, the backward reads x
// and dy and writes dx once. So a row (or a tile of a map's cells with all its
// channels) is held in registers as it was read, and the mean, the variance
// around it (two passes over registers, no difference of moments) and the
// output come from there. Statistics and sums are fp32.
//   * Token rows: a row belongs to 1, 4 or 16 waves, a lane holds NCH pieces
//     of VEC consecutive channels.
//   * Channels-first maps: a workgroup holds TX * VEC neighbouring cells
//     (16 lanes of 16 bytes: 256-byte runs) times all channels, TY channels at
//     a time; the sums over channels go across the workgroup through LDS.
//   * dweight and dbias: each workgroup loops over rows or tiles and keeps the
//     sums of its channels in registers, writes one partial row a workgroup,
//     and a second kernel adds the partial rows in a fixed order.
// Only y and dx of bf16 tensors are rounded to fewer bits, once each.
// Measured, inputs from memory (a large copy runs at 5.1 TB/s): forward of 32 x
// 192 x 56 x 56 maps, bf16: 17 us, 4.6 TB/s; backward of 12544 rows of 768, bf16:
// 18 us, 3.3 TB/s, 4 of them ln_fold; of a 128 x 384 x 512 map, fp32: 71 us, 4.3
// TB/s. One row of 768 takes 2.2 us. What bounds the smaller ones is the start
// and the end of a launch, then the fold. Far from memory's rate, warm inputs: 64 x
// 768 x 196 maps backward (read again: 53 us bf16, 74 fp32, 1.1 and 1.6 TB/s), 64 x 768 x
// 49 (odd rows of cells: 10 and 13 us forward, 42 and 44 backward), 4 x 96 x 50175 (56 us
// forward; 64 and 70 backward, 1.8 and 3.3 TB/s).
#include "ops_common.h"

namespace ssm2d_impl {
namespace {

// ------------------------------------------------------------------ token rows

// Sum over the WPR waves of a row; `buf`: 16 floats of LDS for this use alone.
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

// A lane's weights or biases, without a branch a load: channels past the end
// (VEC divides n) read the last ones, and are not used.
template <int VEC, int NCH, int WPR>
__device__ __forceinline__ void row_params(const float *src, int n, float missing, float (&out)[NCH][VEC])
{
    const int t = static_cast<int>(threadIdx.x) % (WPR * 64);
    if (src) {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const float *at = src + min((c * WPR * 64 + t) * VEC, n - VEC);
#pragma unroll
            for (int j = 0; j < VEC; ++j) out[c][j] = at[j];
        }
    } else {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int j = 0; j < VEC; ++j) out[c][j] = missing;
    }
}

template <typename T, int VEC, int NCH, int WPR>
__global__ __launch_bounds__(WPR * 64 > 256 ? WPR * 64 : 256) void ln_row_fwd(const T *x, const float *weight, const float *bias, T *y,
                                                                  float *mean, float *rstd, long rows, int n, long ldx, float eps)
{
    constexpr int kRows = WPR >= 4 ? 1 : 4 / WPR;  // rows a workgroup holds at once
    __shared__ float red[2][16];
    const int t = static_cast<int>(threadIdx.x) % (WPR * 64);
    float w[NCH][VEC], b[NCH][VEC];
    row_params<VEC, NCH, WPR>(weight, n, 1.0f, w);
    row_params<VEC, NCH, WPR>(bias, n, 0.0f, b);
    const float inv_n = 1.0f / static_cast<float>(n);
    for (long r0 = static_cast<long>(blockIdx.x) * kRows; r0 < rows; r0 += static_cast<long>(gridDim.x) * kRows) {
        const long row = r0 + (WPR >= 4 ? 0 : threadIdx.x / (WPR * 64));
        const bool live = row < rows;
        const T *xr = x + (live ? row : rows - 1) * ldx;
        Raw<T, VEC> v[NCH];
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int col = (c * WPR * 64 + t) * VEC;
            v[c].load(xr + min(col, n - VEC));
        }
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const bool in = (c * WPR * 64 + t) * VEC < n;
#pragma unroll
            for (int j = 0; j < VEC; ++j) s += in ? v[c].get(j) : 0.0f;
        }
        const float mu = row_sum<WPR>(s, red[0]) * inv_n;
#pragma unroll
        for (int c = 0; c < NCH; ++c) v[c].forget();
        float q = 0.0f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int col = (c * WPR * 64 + t) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float d = v[c].get(j) - mu;
                q += col < n ? d * d : 0.0f;
            }
        }
        const float rs = 1.0f / sqrtf(row_sum<WPR>(q, red[1]) * inv_n + eps);
#pragma unroll
        for (int c = 0; c < NCH; ++c) v[c].forget();
        if (!live) continue;
        if (t == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = rs;
        }
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int col = (c * WPR * 64 + t) * VEC;
            if (col >= n) continue;
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] = (v[c].get(j) - mu) * rs * w[c][j] + b[c][j];
            Raw<T, VEC> out;
            out.set(o);
            out.store(y + row * n + col);
        }
    }
}

template <typename T, int VEC, int NCH, int WPR>
__global__ __launch_bounds__(WPR * 64 > 256 ? WPR * 64 : 256) void ln_row_bwd(const T *x, const float *weight, const float *mean,
                                                                  const float *rstd, const T *dy, T *dx, float *part, long rows,
                                                                  int n, long ldx, long ldy)
{
    constexpr int kRows = WPR >= 4 ? 1 : 4 / WPR;
    __shared__ float red[2][16];
    __shared__ float fold[kRows > 1 ? 64 * NCH * VEC : 1];
    const int t = static_cast<int>(threadIdx.x) % (WPR * 64);
    float w[NCH][VEC], dw[NCH][VEC], db[NCH][VEC];
    row_params<VEC, NCH, WPR>(weight, n, 1.0f, w);
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int j = 0; j < VEC; ++j) dw[c][j] = db[c][j] = 0.0f;
    const float inv_n = 1.0f / static_cast<float>(n);
    // the next row is read while this one is worked on (where registers allow)
    constexpr bool kAhead = NCH * VEC <= 16 && WPR < 16;
    Raw<T, VEC> nx[NCH], ng[NCH];
    float nmu = 0.0f, nrs = 0.0f;
    auto fetch = [&](long row) __attribute__((always_inline)) {
        const long at = row < rows ? row : rows - 1;  // (rows past the end read the last one, and are not used)
        nmu = mean[at], nrs = rstd[at];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int col = min((c * WPR * 64 + t) * VEC, n - VEC);
            nx[c].load(x + at * ldx + col);
            ng[c].load(dy + at * ldy + col);
        }
    };
    const long first = static_cast<long>(blockIdx.x) * kRows, step = static_cast<long>(gridDim.x) * kRows;
    const int sub = WPR >= 4 ? 0 : threadIdx.x / (WPR * 64);
    if (kAhead) fetch(first + sub);
    for (long r0 = first; r0 < rows; r0 += step) {
        const long row = r0 + sub;
        const bool live = row < rows;
        if (!kAhead) fetch(row);
        Raw<T, VEC> vx[NCH], vg[NCH];
        const float mu = nmu, rs = nrs;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            vx[c] = nx[c], vg[c] = ng[c];
            if ((c * WPR * 64 + t) * VEC >= n) vx[c].clear(), vg[c].clear();
        }
        if (kAhead && r0 + step < rows) fetch(row + step);
        // (columns past n: x = dy = 0, their terms of both sums are 0 * (-mu rs) = 0
        // unless the row's statistics are not finite, where dx is not either)
        float sa = 0.0f, sc = 0.0f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int col = (c * WPR * 64 + t) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float g = vg[c].get(j), xh = (vx[c].get(j) - mu) * rs;
                const float gw = g * w[c][j];
                sa += gw;
                sc += gw * xh;
                if (live && col < n) {
                    dw[c][j] += g * xh;
                    db[c][j] += g;
                }
            }
        }
        const float a = row_sum<WPR>(sa, red[0]) * inv_n, cc = row_sum<WPR>(sc, red[1]) * inv_n;
#pragma unroll
        for (int c = 0; c < NCH; ++c) vx[c].forget(), vg[c].forget();
        if (!live) continue;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int col = (c * WPR * 64 + t) * VEC;
            if (col >= n) continue;
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float xh = (vx[c].get(j) - mu) * rs;
                o[j] = rs * (vg[c].get(j) * w[c][j] - a - xh * cc);
            }
            Raw<T, VEC> out;
            out.set(o);
            out.store(dx + row * n + col);
        }
    }
    if (!part) return;
    // one partial row of dweight and dbias a workgroup: its waves' sums added in order
    float *mine = part + static_cast<long>(blockIdx.x) * 2 * n;
    if constexpr (kRows > 1) {
        const int wave = threadIdx.x / 64;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            for (int u = 0; u < kRows; ++u) {
                __syncthreads();
                if (wave == u) {
#pragma unroll
                    for (int c = 0; c < NCH; ++c)
#pragma unroll
                        for (int j = 0; j < VEC; ++j) {
                            const int at = (c * 64 + t) * VEC + j;
                            const float add = k ? db[c][j] : dw[c][j];
                            fold[at] = u ? fold[at] + add : add;
                        }
                }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < n; i += static_cast<int>(blockDim.x)) mine[k * n + i] = fold[i];
        }
    } else {
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int col = (c * WPR * 64 + t) * VEC;
            if (col >= n) continue;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                mine[col + j] = dw[c][j];
                mine[n + col + j] = db[c][j];
            }
        }
    }
}

// A few MB at most, so latency: 4 us for 512 rows of 2 x 768.
// dweight (columns 0 .. n - 1 of the partial rows) and dbias (n .. 2n - 1): 16
// columns a workgroup, so that few columns still make several workgroups; 64
// groups of rows, then the groups in order.
__global__ __launch_bounds__(1024) void ln_fold(const float *part, int np, int n, float *dweight, float *dbias)
{
    __shared__ float s[64][17];
    const int lx = threadIdx.x % 16, ly = threadIdx.x / 16;
    const int col = static_cast<int>(blockIdx.x) * 16 + lx, at = min(col, 2 * n - 1);
    float acc = 0.0f;
    int p = ly;
    for (; p + 7 * 64 < np; p += 8 * 64) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = part[static_cast<long>(p + 64 * k) * 2 * n + at];
#pragma unroll
        for (int k = 0; k < 8; ++k) acc += v[k];
    }
    for (; p < np; p += 64) acc += part[static_cast<long>(p) * 2 * n + at];
    s[ly][lx] = acc;
    __syncthreads();
    if (threadIdx.x < 64) {  // 16 columns by 4 groups of 16 rows
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) v += s[16 * ly + k][lx];
        v = pair_sum<32>(pair_sum<16>(v));
        if (ly == 0 && col < 2 * n) {
            float *out = col < n ? dweight : dbias;
            if (out) out[col < n ? col : col - n] = v;
        }
    }
}

// ------------------------------------------------------------------ channels-first maps

// Sum over a tile's TY channel groups of VEC values a lane column: within each
// wave first, then over the waves through LDS, every thread in the same order.
template <int VEC, int TX, int TY>
__device__ __forceinline__ void tile_sum(float (&v)[VEC], float *buf)
{
    constexpr int kWaves = TX * TY / 64;
    const int tx = threadIdx.x % TX, wave = threadIdx.x / 64;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        static_assert(TX == 16 || TX == 64, "lanes of a channel group");
        if constexpr (TX == 16) v[j] = pair_sum<32>(pair_sum<16>(v[j]));
    }
    __syncthreads();  // (the last use of buf has been read)
    if (threadIdx.x % 64 < TX) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) buf[(wave * VEC + j) * TX + tx] = v[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = 0.0f;
#pragma unroll 2
    for (int u = 0; u < kWaves; ++u)
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] += buf[(u * VEC + j) * TX + tx];
}

// A lane's place within a workgroup's channels, beside a base the workgroup
// shares. In 32 bits one register serves every channel group; strides of 2^26
// elements or more take the kernels of single cells, which keep 64.
template <int VEC>
__device__ __forceinline__ auto lane_offset(int ty, int at, long stride)
{
    if constexpr (VEC == 1) return ty * stride + at;
    else return static_cast<unsigned>(ty) * static_cast<unsigned>(stride) + static_cast<unsigned>(at);
}

// The channels' weights or biases in LDS (a load each where they are used would
// be waited for one by one); a barrier comes before their use.
template <int THREADS>
__device__ __forceinline__ void map_params(const float *src, int n, float missing, float *out)
{
    for (int i = threadIdx.x; i < n; i += THREADS) out[i] = src ? src[i] : missing;
}

// KEEP: the tile stays in registers (n <= TY * NCH); else it is read again for
// each pass (from cache: a tile is TX * VEC * n elements) and dweight and
// dbias are left to ln_map_sums.
template <typename T, int VEC, int TX, int TY, int NCH, bool KEEP>
__global__ __launch_bounds__(TX *TY) void ln_map_fwd(const T *x, const float *weight, const float *bias, T *y, float *mean,
                                                     float *rstd, long tiles, int tiles_b, int n, long cells, long sb, long sn,
                                                     float eps)
{
    __shared__ float buf[TX * TY / 64 * VEC * TX];
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    const float inv_n = 1.0f / static_cast<float>(n);
    __shared__ float ws[KEEP ? TY * NCH : 1], bs[KEEP ? TY * NCH : 1];
    if constexpr (KEEP) {
        map_params<TX * TY>(weight, n, 1.0f, ws);
        map_params<TX * TY>(bias, n, 0.0f, bs);
    }
    const int nc = KEEP ? NCH : (n + TY - 1) / TY;
    for (long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const long b = tile / tiles_b;
        const long cell0 = (tile - b * tiles_b) * (TX * VEC), cell = cell0 + tx * VEC;
        const bool live = cell < cells;
        const T *xb = x + b * sb + cell0;
        const auto lane = lane_offset<VEC>(ty, tx * VEC, sn);
        Raw<T, VEC> v[KEEP ? NCH : 1];
        auto get = [&](int c) -> const Raw<T, VEC> & {
            if constexpr (KEEP) return v[c];
            if (live && c * TY + ty < n) v[0].load(xb + c * TY * sn + lane);
            else v[0].clear();
            return v[0];
        };
        if constexpr (KEEP) {
#pragma unroll
            for (int c = 0; c < NCH; ++c) {
                if (live && c * TY + ty < n) v[c].load(xb + c * TY * sn + lane);
                else v[c].clear();
            }
        }
        float mu[VEC], q[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) mu[j] = q[j] = 0.0f;
#pragma unroll(KEEP ? NCH : 1)
        for (int c = 0; c < nc; ++c) {
            const Raw<T, VEC> &r = get(c);
#pragma unroll
            for (int j = 0; j < VEC; ++j) mu[j] += r.get(j);
        }
        tile_sum<VEC, TX, TY>(mu, buf);
#pragma unroll
        for (int j = 0; j < VEC; ++j) mu[j] *= inv_n;
        if constexpr (KEEP) {
#pragma unroll
            for (int c = 0; c < NCH; ++c) v[c].forget();
        }
#pragma unroll(KEEP ? NCH : 1)
        for (int c = 0; c < nc; ++c) {
            const Raw<T, VEC> &r = get(c);
            if (c * TY + ty < n)
#pragma unroll
                for (int j = 0; j < VEC; ++j) q[j] += (r.get(j) - mu[j]) * (r.get(j) - mu[j]);
        }
        tile_sum<VEC, TX, TY>(q, buf);
#pragma unroll
        for (int j = 0; j < VEC; ++j) q[j] = 1.0f / sqrtf(q[j] * inv_n + eps);
        if constexpr (KEEP) {
#pragma unroll
            for (int c = 0; c < NCH; ++c) v[c].forget();
        }
        if (!live) continue;
        if (ty == 0) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (mean) mean[b * cells + cell + j] = mu[j];
                if (rstd) rstd[b * cells + cell + j] = q[j];
            }
        }
#pragma unroll(KEEP ? NCH : 1)
        for (int c = 0; c < nc; ++c) {
            const int ch = c * TY + ty;
            const Raw<T, VEC> &r = get(c);
            if (ch >= n) continue;
            const float w = KEEP ? ws[ch] : (weight ? weight[ch] : 1.0f), bi = KEEP ? bs[ch] : (bias ? bias[ch] : 0.0f);
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] = (r.get(j) - mu[j]) * q[j] * w + bi;
            Raw<T, VEC> out;
            out.set(o);
            out.store(y + (b * n + c * TY) * cells + cell0 + lane_offset<VEC>(ty, tx * VEC, cells));
        }
    }
}

template <typename T, int VEC, int TX, int TY, int NCH, bool KEEP>
__global__ __launch_bounds__(TX *TY) void ln_map_bwd(const T *x, const float *weight, const float *mean, const float *rstd,
                                                     const T *dy, T *dx, float *part, long tiles, int tiles_b, int n, long cells,
                                                     long sb, long sn, long gb, long gn)
{
    __shared__ float buf[TX * TY / 64 * VEC * TX];
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    const float inv_n = 1.0f / static_cast<float>(n);
    const int nc = KEEP ? NCH : (n + TY - 1) / TY;
    __shared__ float ws[KEEP ? TY * NCH : 1];
    float dw[KEEP ? NCH : 1], db[KEEP ? NCH : 1];
    if constexpr (KEEP) {
        map_params<TX * TY>(weight, n, 1.0f, ws);
        __syncthreads();
#pragma unroll
        for (int c = 0; c < NCH; ++c) dw[c] = db[c] = 0.0f;
    }
    for (long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const long b = tile / tiles_b;
        const long cell0 = (tile - b * tiles_b) * (TX * VEC), cell = cell0 + tx * VEC;
        const bool live = cell < cells;
        const T *xb = x + b * sb + cell0, *yb = dy + b * gb + cell0;
        const auto xl = lane_offset<VEC>(ty, tx * VEC, sn);
        const auto yl = lane_offset<VEC>(ty, tx * VEC, gn);
        Raw<T, VEC> vx[KEEP ? NCH : 1], vg[KEEP ? NCH : 1];
        auto fetch = [&](int c, int k) {
            if (live && c * TY + ty < n) {
                vx[k].load(xb + c * TY * sn + xl);
                vg[k].load(yb + c * TY * gn + yl);
            } else {
                vx[k].clear();
                vg[k].clear();
            }
        };
        if constexpr (KEEP) {
#pragma unroll
            for (int c = 0; c < NCH; ++c) fetch(c, c);
        }
        float mu[VEC], rs[VEC], a[VEC], cc[VEC];
        const long stat = b * cells + (live ? cell : cell0);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            mu[j] = mean[stat + j];
            rs[j] = rstd[stat + j];
            a[j] = cc[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) mu[j] = live ? mu[j] : 0.0f, rs[j] = live ? rs[j] : 0.0f;
#pragma unroll(KEEP ? NCH : 1)
        for (int c = 0; c < nc; ++c) {
            const int k = KEEP ? c : 0, ch = c * TY + ty;
            if constexpr (!KEEP) fetch(c, 0);
            const float w = KEEP ? ws[min(ch, n - 1)] : (weight ? weight[min(ch, n - 1)] : 1.0f);
            float sw = 0.0f, sg = 0.0f;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float g = vg[k].get(j), xh = (vx[k].get(j) - mu[j]) * rs[j];
                a[j] += g * w;
                cc[j] += g * w * xh;
                sw += g * xh;
                sg += g;
            }
            if constexpr (KEEP) dw[c] += sw, db[c] += sg;
            vx[k].forget(), vg[k].forget();
        }
        tile_sum<VEC, TX, TY>(a, buf);
        tile_sum<VEC, TX, TY>(cc, buf);
        if constexpr (KEEP) {
#pragma unroll
            for (int c = 0; c < NCH; ++c) vx[c].forget(), vg[c].forget();
        }
        if (!live) continue;
#pragma unroll(KEEP ? NCH : 1)
        for (int c = 0; c < nc; ++c) {
            const int k = KEEP ? c : 0, ch = c * TY + ty;
            if constexpr (!KEEP) fetch(c, 0);
            if (ch >= n) continue;
            const float w = KEEP ? ws[ch] : (weight ? weight[ch] : 1.0f);
            float o[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float xh = (vx[k].get(j) - mu[j]) * rs[j];
                o[j] = rs[j] * (vg[k].get(j) * w - a[j] * inv_n - xh * (cc[j] * inv_n));
            }
            Raw<T, VEC> out;
            out.set(o);
            out.store(dx + (b * n + c * TY) * cells + cell0 + lane_offset<VEC>(ty, tx * VEC, cells));
        }
    }
    if constexpr (KEEP) {
        if (!part) return;
        float *mine = part + static_cast<long>(blockIdx.x) * 2 * n;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const int ch = c * TY + ty;
            const float sw = lane_sum<TX>(dw[c]), sg = lane_sum<TX>(db[c]);
            if (tx == 0 && ch < n) {
                mine[ch] = sw;
                mine[n + ch] = sg;
            }
        }
    }
}

// dweight and dbias of maps whose tiles are not kept: workgroup (channel,
// slice of the cells) to one entry of a partial row. x and dy come a second
// time, from cache or memory; it is the part of a backward of more than 512
// channels that bounds it (bf16, 21 x 1536 x 448: 54 us in all, 1.6 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void ln_map_sums(const T *x, const float *mean, const float *rstd, const T *dy, float *part,
                                                   long batch, int n, long cells, long sb, long sn, long gb, long gn)
{
    __shared__ float red[2][4];
    const int ch = blockIdx.x;
    float sw = 0.0f, sg = 0.0f;
    const long total = batch * cells, step = static_cast<long>(gridDim.y) * 256;
    for (long i = static_cast<long>(blockIdx.y) * 256 + threadIdx.x; i < total; i += step) {
        const long b = i / cells, cell = i - b * cells;
        const float g = widen1(dy[b * gb + ch * gn + cell]);
        sw += g * (widen1(x[b * sb + ch * sn + cell]) - mean[i]) * rstd[i];
        sg += g;
    }
    sw = lane_sum<64>(sw);
    sg = lane_sum<64>(sg);
    if (threadIdx.x % 64 == 0) red[0][threadIdx.x / 64] = sw, red[1][threadIdx.x / 64] = sg;
    __syncthreads();
    if (threadIdx.x == 0) {
        float *mine = part + static_cast<long>(blockIdx.y) * 2 * n;
        mine[ch] = red[0][0] + red[0][1] + red[0][2] + red[0][3];
        mine[n + ch] = red[1][0] + red[1][1] + red[1][2] + red[1][3];
    }
}

__global__ void ln_zero(float *a, float *b, int n)
{
    const int i = static_cast<int>(blockIdx.x * blockDim.x + threadIdx.x);
    if (i >= n) return;
    if (a) a[i] = 0.0f;
    if (b) b[i] = 0.0f;
}

// The statistics of no channels: sums over nothing are zeros.
__global__ void ln_no_channels(float *mean, float *rstd, long rows, float eps)
{
    const long step = static_cast<long>(gridDim.x) * blockDim.x;
    for (long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x; i < rows; i += step) {
        if (mean) mean[i] = 0.0f;
        if (rstd) rstd[i] = 1.0f / sqrtf(eps);
    }
}

// ------------------------------------------------------------------ host

struct NormArgs {
    int64_t batch, n, cells, sb, sn, gb, gn;
    hipStream_t s;
};

constexpr int64_t kFar = int64_t{1} << 26;
inline bool near(int64_t stride) { return stride >= 0 && stride < kFar; }
// Partial rows of dweight and dbias: the workgroups of a backward launch, two a
// compute unit. Fewer leave the reads short (bf16, 8 x 192 x 12544: 42 us with 256,
// 33 with 512, 34 with 1024), more make the fold longer (bf16 rows, 8192 x 2048: 25,
// 26 and 31 us).
constexpr int kMaxParts = 512;

// Workgroups for `work` turns of a loop: at most `most`, all with as many turns (but the last).
unsigned even_blocks(int64_t work, int64_t most)
{
    const int64_t turns = (work + most - 1) / most;
    return static_cast<unsigned>(turns > 0 ? (work + turns - 1) / turns : 1);
}
unsigned blocks_for(int64_t work, int64_t most) { return static_cast<unsigned>(std::max<int64_t>(1, std::min(work, most))); }

// The row kernels' variant: waves a row and pieces a lane, the fewest that
// hold n channels with VEC channels a piece. A wave a row needs no barrier: the
// backward of 12544 x 768 (bf16) takes 21 us with one, 32 with four. Four from
// 2048 channels of bf16 on: 4096 x 4096 takes 36 us with four, 60 with one. Rows
// that are not aligned are read by single elements (12544 x 767: 14 us forward and
// 31 backward; 9.7 and 19 of 768).
template <typename T, int VEC, typename F>
int pick_row(int64_t n, F &&f)
{
    const int64_t per = VEC * 64;
    using std::integral_constant;
#define SSM2D_ROW(NCH, WPR) f(integral_constant<int, NCH>{}, integral_constant<int, WPR>{})
    if (n <= per) return SSM2D_ROW(1, 1);
    if (n <= 2 * per) return SSM2D_ROW(2, 1);
    if (n <= 4 * per) return SSM2D_ROW(4, 1);
    if (n <= 8 * per) return SSM2D_ROW(2, 4);
    if (n <= 16 * per) return SSM2D_ROW(4, 4);
    if constexpr (VEC == 1) {
        if (n <= 64 * per) return SSM2D_ROW(4, 16);
        return SSM2D_ROW(16, 16);
    } else {
        return SSM2D_ROW(16 / VEC, 16);
    }
#undef SSM2D_ROW
}

// The map kernels' variants. Lanes run over 16 pieces of VEC cells, or over 64
// pieces of few cells where rows of cells are not aligned; channels over TY
// groups of NCH at most, which a thread keeps (the backward those of two tensors
// and two sums a channel). The widest piece is taken with which nothing spills:
//   * forward: 16 bytes up to 384 channels, 8 up to 1024, single cells or 4
//     bytes where rows allow no more; beyond, the tile is read again each pass
//     (bf16, 21 x 1536 x 448: 36 us, 1.6 TB/s; 4 x 1024 x 3136 kept: 15 us, 3.5).
//   * backward: 16 bytes up to 64 channels of bf16 and 128 of fp32 (bf16,
//     4 x 96 x 50176: 45 us with 8-byte pieces, 71 with 16; fp32: 58 and 50),
//     8 up to 384 and 512, single cells up to 128 (4 x 96 x 50175, bf16: 61 us, and
//     136 with 1024 threads of 128 registers, which spill); beyond, read again
//     (bf16, 4 x 768 x 3136: 37 us; 53 with 4-byte pieces kept by 1024 threads;
//     8 x 512 x 3136: 43 us).
enum : int { kCells16 = 0, kCells8 = 1, kCells4 = 2, kCellsFew = 3 };

template <int LEVEL, int VEC, bool BWD, typename F>
int pick_map(int64_t n, F &&f)
{
    using std::integral_constant;
#define SSM2D_MAP(TX, TY, NCH, KEEP) \
    f(integral_constant<int, TX>{}, integral_constant<int, TY>{}, integral_constant<int, NCH>{}, std::bool_constant<KEEP>{})
    if constexpr (LEVEL == kCellsFew) {
        if (n <= 64) return SSM2D_MAP(64, 4, 16, true);
        if constexpr (BWD && VEC == 1) {
            if (n <= 128) return SSM2D_MAP(64, 8, 16, true);
        }
        if constexpr (!BWD) {
            if (n <= 256) return SSM2D_MAP(64, 16, 16, true);
        }
        return SSM2D_MAP(64, 16, 16, false);
    } else if constexpr (LEVEL == kCells16) {
        if (n <= 64 || (BWD && VEC == 8)) return SSM2D_MAP(16, 16, 4, true);
        if constexpr (BWD && VEC == 4) return SSM2D_MAP(16, 16, 8, true);
        if constexpr (!BWD) {
            if (n <= 128) return SSM2D_MAP(16, 16, 8, true);
            if (n <= 192) return SSM2D_MAP(16, 16, 12, true);
            if (n <= 256) return SSM2D_MAP(16, 32, 8, true);
            return SSM2D_MAP(16, 32, 12, true);
        }
    } else if constexpr (LEVEL == kCells8) {
        if (n > (BWD ? (VEC == 2 ? 512 : 384) : 1024)) return SSM2D_MAP(16, 64, 16, false);
        if (n <= 128) return SSM2D_MAP(16, 16, 8, true);
        if (n <= 192) return SSM2D_MAP(16, 16, 12, true);
        if (n <= 256) return SSM2D_MAP(16, 32, 8, true);
        if (n <= 384) return SSM2D_MAP(16, 32, 12, true);
        if constexpr (BWD) {
            return SSM2D_MAP(16, 32, VEC == 2 ? 16 : 12, true);
        } else {
            if (n <= 512) return SSM2D_MAP(16, 32, 16, true);
            if (n <= 768) return SSM2D_MAP(16, 64, 12, true);
            return SSM2D_MAP(16, 64, 16, true);
        }
    } else {
        if (n <= 768) return SSM2D_MAP(16, 64, 12, true);
        return SSM2D_MAP(16, 64, 16, true);
    }
#undef SSM2D_MAP
}

// The piece for n channels; fits(v): v cells can be read at once everywhere.
// Two cells of bf16 a lane are kept for up to 64 channels of the backward (more
// spill: 8 x 192 x 12546 took 112 us, and 88 with one cell).
template <int V, bool BWD, typename P, typename F>
int pick_cells(int64_t n, P &&fits, F &&go)
{
    using std::integral_constant;
    if (n <= (BWD ? 512 / V : 384) && fits(V)) return go(integral_constant<int, V>{}, integral_constant<int, kCells16>{});
    if (fits(V / 2)) return go(integral_constant<int, V / 2>{}, integral_constant<int, kCells8>{});
    const bool middle = n > 256 && n <= 1024;
    if constexpr (V / 4 > 1) {
        const bool few = BWD ? n <= 64 || n > 128 : !middle;
        if (few && fits(V / 4)) return go(integral_constant<int, V / 4>{}, integral_constant<int, kCellsFew>{});
        if constexpr (!BWD) {
            if (middle && fits(V / 4)) return go(integral_constant<int, V / 4>{}, integral_constant<int, kCells4>{});
        }
    }
    if constexpr (!BWD) {
        if (middle) return go(integral_constant<int, 1>{}, integral_constant<int, kCells4>{});
    }
    return go(integral_constant<int, 1>{}, integral_constant<int, kCellsFew>{});
}

// Whether rows of `stride` elements from p can be read V elements at a time.
template <typename T>
bool aligned_to(const T *p, int64_t stride_a, int64_t stride_b, int v)
{
    return !off_by(p, static_cast<size_t>(v) * sizeof(T)) && stride_a % v == 0 && stride_b % v == 0;
}

template <typename T>
int norm_fwd(const T *x, const float *weight, const float *bias, T *y, float *mean, float *rstd, const NormArgs &a, float eps)
{
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const int n = static_cast<int>(a.n);
    if (a.cells == 1 && (a.sn == 1 || a.n == 1)) {
        auto go = [&](auto vec) {
            constexpr int VEC = decltype(vec)::value;
            return pick_row<T, VEC>(a.n, [&](auto nch, auto wpr) {
                constexpr int NCH = decltype(nch)::value, WPR = decltype(wpr)::value;
                constexpr int kRows = WPR >= 4 ? 1 : 4 / WPR;
                // (enough to fill the chip; a workgroup reads the weights once for its rows)
                const unsigned grid = blocks_for((a.batch + kRows - 1) / kRows, WPR == 16 ? 1024 : 4096);
                ln_row_fwd<T, VEC, NCH, WPR><<<dim3(grid), dim3(WPR * 64 > 256 ? WPR * 64 : 256), 0, a.s>>>(
                    x, weight, bias, y, mean, rstd, a.batch, n, a.sb, eps);
                return launched();
            });
        };
        const bool wide = a.n % V == 0 && aligned_to(x, a.sb, 0, V) && !off_by(y, 16);
        return wide ? go(std::integral_constant<int, V>{}) : go(std::integral_constant<int, 1>{});
    }
    auto go = [&](auto vec, auto level) {
        constexpr int VEC = decltype(vec)::value;
        return pick_map<decltype(level)::value, VEC, false>(a.n, [&](auto tx, auto ty, auto nch, auto keep) {
            constexpr int TX = decltype(tx)::value, TY = decltype(ty)::value, NCH = decltype(nch)::value;
            const int64_t tiles_b = (a.cells + TX * VEC - 1) / (TX * VEC), tiles = tiles_b * a.batch;
            ln_map_fwd<T, VEC, TX, TY, NCH, decltype(keep)::value><<<dim3(blocks_for(tiles, 1 << 20)), dim3(TX * TY), 0, a.s>>>(
                x, weight, bias, y, mean, rstd, tiles, static_cast<int>(tiles_b), n, a.cells, a.sb, a.sn, eps);
            return launched();
        });
    };
    auto fits = [&](int v) {
        return a.cells < kFar && near(a.sn) && a.cells % v == 0 && aligned_to(x, a.batch > 1 ? a.sb : 0, a.n > 1 ? a.sn : 0, v) &&
               !off_by(y, v * sizeof(T));
    };
    return pick_cells<V, false>(a.n, fits, go);
}

template <typename T>
int norm_bwd(const T *x, const float *weight, const float *mean, const float *rstd, const T *dy, T *dx, float *dweight,
             float *dbias, const NormArgs &a, void *stream)
{
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    const int n = static_cast<int>(a.n);
    const bool sums = dweight || dbias;
    float *part = nullptr;
    auto parts = [&](unsigned np) -> int {
        if (!sums) return SSM2D_OK;
        int dev = 0;
        const hipError_t e = hipGetDevice(&dev);
        if (e != hipSuccess) return hip_fail(e);
        void *p = nullptr;
        const int st = get_aux_ws(dev, stream, kSlotNorm, static_cast<size_t>(np) * 2 * n * sizeof(float), &p);
        part = static_cast<float *>(p);
        return st;
    };
    auto fold = [&](unsigned np) -> int {
        if (!sums) return SSM2D_OK;
        ln_fold<<<dim3(static_cast<unsigned>((2 * n + 15) / 16)), dim3(1024), 0, a.s>>>(part, static_cast<int>(np), n, dweight, dbias);
        return launched();
    };
    if (a.cells == 1 && ((a.sn == 1 && a.gn == 1) || a.n == 1)) {
        auto go = [&](auto vec) {
            constexpr int VEC = decltype(vec)::value;
            return pick_row<T, VEC>(a.n, [&](auto nch, auto wpr) {
                constexpr int NCH = decltype(nch)::value, WPR = decltype(wpr)::value;
                constexpr int kRows = WPR >= 4 ? 1 : 4 / WPR;
                // (of 16 waves one workgroup fits a compute unit)
                const unsigned grid = even_blocks((a.batch + kRows - 1) / kRows, WPR == 16 ? 256 : kMaxParts);
                int st = parts(grid);
                if (st != SSM2D_OK) return st;
                ln_row_bwd<T, VEC, NCH, WPR><<<dim3(grid), dim3(WPR * 64 > 256 ? WPR * 64 : 256), 0, a.s>>>(
                    x, weight, mean, rstd, dy, dx, part, a.batch, n, a.sb, a.gb);
                st = launched();
                return st == SSM2D_OK ? fold(grid) : st;
            });
        };
        const bool wide = a.n % V == 0 && aligned_to(x, a.sb, 0, V) && aligned_to(dy, a.gb, 0, V) && !off_by(dx, 16);
        return wide ? go(std::integral_constant<int, V>{}) : go(std::integral_constant<int, 1>{});
    }
    auto go = [&](auto vec, auto level) {
        constexpr int VEC = decltype(vec)::value;
        return pick_map<decltype(level)::value, VEC, true>(a.n, [&](auto tx, auto ty, auto nch, auto keep) {
            constexpr int TX = decltype(tx)::value, TY = decltype(ty)::value, NCH = decltype(nch)::value;
            constexpr bool KEEP = decltype(keep)::value;
            const int64_t tiles_b = (a.cells + TX * VEC - 1) / (TX * VEC), tiles = tiles_b * a.batch;
            const unsigned grid = KEEP ? even_blocks(tiles, kMaxParts) : blocks_for(tiles, 1 << 20);
            const unsigned slices = KEEP ? grid : blocks_for((a.batch * a.cells + 2047) / 2048, 64);
            int st = parts(slices);
            if (st != SSM2D_OK) return st;
            ln_map_bwd<T, VEC, TX, TY, NCH, KEEP><<<dim3(grid), dim3(TX * TY), 0, a.s>>>(
                x, weight, mean, rstd, dy, dx, part, tiles, static_cast<int>(tiles_b), n, a.cells, a.sb, a.sn, a.gb, a.gn);
            st = launched();
            if (st != SSM2D_OK) return st;
            if (!KEEP && sums) {
                ln_map_sums<T><<<dim3(static_cast<unsigned>(n), slices), dim3(256), 0, a.s>>>(x, mean, rstd, dy, part, a.batch, n,
                                                                                             a.cells, a.sb, a.sn, a.gb, a.gn);
                st = launched();
                if (st != SSM2D_OK) return st;
            }
            return fold(slices);
        });
    };
    auto fits = [&](int v) {
        const int64_t b = a.batch > 1, c = a.n > 1;
        return a.cells < kFar && near(a.sn) && near(a.gn) && a.cells % v == 0 && aligned_to(x, b * a.sb, c * a.sn, v) &&
               aligned_to(dy, b * a.gb, c * a.gn, v) && !off_by(dx, v * sizeof(T));
    };
    return pick_cells<V, true>(a.n, fits, go);
}

int check_sizes(int64_t batch, int64_t n, int64_t cells)
{
    if (batch < 0 || n < 0 || cells < 0) return SSM2D_ERR_BAD_DIM;
    if (n > SSM2D_LN_MAX_N) return SSM2D_ERR_UNSUPPORTED;
    return SSM2D_OK;
}
// Tensors of 2^62 bytes and more would wrap the offsets; far beyond memory.
bool beyond(int64_t batch, int64_t n, int64_t cells)
{
    return static_cast<double>(batch) * static_cast<double>(std::max<int64_t>(n, 1)) * static_cast<double>(cells) > 1e15;
}

template <typename T>
int norm_fwd_entry(const T *x, const float *weight, const float *bias, T *y, float *mean, float *rstd, int64_t batch, int64_t n,
                   int64_t cells, int64_t sb, int64_t sn, float eps, void *stream)
{
    int st = check_sizes(batch, n, cells);
    if (st != SSM2D_OK) return st;
    if (batch == 0 || cells == 0 || (n == 0 && !mean && !rstd)) return SSM2D_OK;
    if (beyond(batch, n, cells)) return SSM2D_ERR_UNSUPPORTED;
    if (n == 0) {
        if (off_by(mean, 4) || off_by(rstd, 4)) return SSM2D_ERR_MISALIGNED;
        ln_no_channels<<<dim3(blocks_for((batch * cells + 255) / 256, 1 << 20)), dim3(256), 0, static_cast<hipStream_t>(stream)>>>(
            mean, rstd, batch * cells, eps);
        return launched();
    }
    if (!x || !y) return SSM2D_ERR_NULLPTR;
    if (off_by(x, sizeof(T)) || off_by(y, sizeof(T)) || off_by(weight, 4) || off_by(bias, 4) || off_by(mean, 4) || off_by(rstd, 4))
        return SSM2D_ERR_MISALIGNED;
    return guarded([&] {
        std::lock_guard<std::recursive_mutex> lock(g_mutex);
        return norm_fwd(x, weight, bias, y, mean, rstd, NormArgs{batch, n, cells, sb, sn, 0, 0, static_cast<hipStream_t>(stream)}, eps);
    });
}

template <typename T>
int norm_bwd_entry(const T *x, const float *weight, const float *mean, const float *rstd, const T *dy, T *dx, float *dweight,
                   float *dbias, int64_t batch, int64_t n, int64_t cells, int64_t sb, int64_t sn, int64_t gb, int64_t gn, void *stream)
{
    int st = check_sizes(batch, n, cells);
    if (st != SSM2D_OK) return st;
    if (n == 0) return SSM2D_OK;
    if (off_by(dweight, 4) || off_by(dbias, 4)) return SSM2D_ERR_MISALIGNED;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (batch == 0 || cells == 0) {
        if (!dweight && !dbias) return SSM2D_OK;
        ln_zero<<<dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, s>>>(dweight, dbias, static_cast<int>(n));
        return launched();
    }
    if (beyond(batch, n, cells)) return SSM2D_ERR_UNSUPPORTED;
    if (!x || !mean || !rstd || !dy || !dx) return SSM2D_ERR_NULLPTR;
    if (off_by(x, sizeof(T)) || off_by(dy, sizeof(T)) || off_by(dx, sizeof(T)) || off_by(weight, 4) || off_by(mean, 4) || off_by(rstd, 4))
        return SSM2D_ERR_MISALIGNED;
    return guarded([&] {
        std::lock_guard<std::recursive_mutex> lock(g_mutex);
        return norm_bwd(x, weight, mean, rstd, dy, dx, dweight, dbias, NormArgs{batch, n, cells, sb, sn, gb, gn, s}, stream);
    });
}

}  // namespace
}  // namespace ssm2d_impl

extern "C" {

int ssm2d_layer_norm_fwd(const float *x, const float *weight, const float *bias, float *y, float *mean, float *rstd, int64_t batch,
                         int64_t n, int64_t cells, int64_t x_stride_b, int64_t x_stride_n, float eps, void *stream)
{
    return ssm2d_impl::norm_fwd_entry<float>(x, weight, bias, y, mean, rstd, batch, n, cells, x_stride_b, x_stride_n, eps, stream);
}

int ssm2d_layer_norm_fwd_bf16(const uint16_t *x, const float *weight, const float *bias, uint16_t *y, float *mean, float *rstd,
                              int64_t batch, int64_t n, int64_t cells, int64_t x_stride_b, int64_t x_stride_n, float eps,
                              void *stream)
{
    return ssm2d_impl::norm_fwd_entry<uint16_t>(x, weight, bias, y, mean, rstd, batch, n, cells, x_stride_b, x_stride_n, eps, stream);
}

int ssm2d_layer_norm_bwd(const float *x, const float *weight, const float *mean, const float *rstd, const float *dy, float *dx,
                         float *dweight, float *dbias, int64_t batch, int64_t n, int64_t cells, int64_t x_stride_b,
                         int64_t x_stride_n, int64_t dy_stride_b, int64_t dy_stride_n, void *stream)
{
    return ssm2d_impl::norm_bwd_entry<float>(x, weight, mean, rstd, dy, dx, dweight, dbias, batch, n, cells, x_stride_b, x_stride_n,
                                             dy_stride_b, dy_stride_n, stream);
}

int ssm2d_layer_norm_bwd_bf16(const uint16_t *x, const float *weight, const float *mean, const float *rstd, const uint16_t *dy,
                              uint16_t *dx, float *dweight, float *dbias, int64_t batch, int64_t n, int64_t cells,
                              int64_t x_stride_b, int64_t x_stride_n, int64_t dy_stride_b, int64_t dy_stride_n, void *stream)
{
    return ssm2d_impl::norm_bwd_entry<uint16_t>(x, weight, mean, rstd, dy, dx, dweight, dbias, batch, n, cells, x_stride_b,
                                                x_stride_n, dy_stride_b, dy_stride_n, stream);
}

}  // extern "C"
