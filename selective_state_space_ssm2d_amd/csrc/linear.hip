// libssm2d: linear's entries: checks, the products behind the forward and the
// gradients, and the pass that makes dz and dbias (linear.h has the products).
//
// With rows as token rows [r][channel] and maps [channel][r], all of them are
// C = A B^T with C's n contiguous:
//   forward    y rows: m = r, n = j, A = x, B = weight;    y maps: m = j, n = r, A = weight, B = x
//   dx         x rows: m = r, n = i, A = dz, B = weight^T;  x maps: m = i, n = r, A = weight^T, B = dz
//   dweight    m = j, n = i, A = dz^T, B = x^T, the sum over r and the batch
// and each operand has its summed index contiguous or the other one.
#include "linear.h"

namespace ssm2d_impl {
namespace gemm {

template <>
int run_gemm<uint16_t>(GemmParams p, const GemmPlan &g, bool a_kc, bool b_kc, void *ws, hipStream_t s);
template <>
int run_gemm<float>(GemmParams p, const GemmPlan &g, bool a_kc, bool b_kc, void *ws, hipStream_t s);
template <>
int run_pair<uint16_t>(GemmParams dx, const GemmPlan &gx, GemmParams dw, const GemmPlan &gw, bool x_maps, bool y_maps, void *ws, hipStream_t s);
template <>
int run_pair<float>(GemmParams dx, const GemmPlan &gx, GemmParams dw, const GemmPlan &gw, bool x_maps, bool y_maps, void *ws, hipStream_t s);

}  // namespace gemm

namespace {

using namespace gemm;

// ------------------------------------------------------------------ dz and dbias

struct SlopeParams {
    const void *dy, *pre;
    // NULL: not stored. In T, as the products take it: bf16 dz is rounded once on its way (dx and
    // dweight err by 0.0024 of their size, 0.0017 without); two parts of it would take twice
    // the matrix instructions, which bound that call.
    void *dz;
    float *part;     // [slice][n] sums; NULL: not wanted
    long batch, rows, n;
    long d_b, d_s;   // dy: batch; row, or channel of maps
    int act, slices; // slices of the rows (of each batch entry)
    long each;       // rows of a slice
    long first;
};

template <typename T, int V>
__device__ __forceinline__ void slope_of(const SlopeParams &p, const T *dy, const T *pre, T *dz, float (&v)[V])
{
    Raw<T, V> d;
    d.load_any(dy);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = d.get(j);
    if (p.act != SSM2D_ACT_NONE) {
        Raw<T, V> z;
        z.load_any(pre);
        switch (p.act) {
        case SSM2D_ACT_RELU:
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = z.get(j) > 0.0f ? v[j] : 0.0f;
            break;
        case SSM2D_ACT_SILU:
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] *= act_slope<T, SSM2D_ACT_SILU>(z.get(j));
            break;
        default:
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] *= act_slope<T, SSM2D_ACT_GELU>(z.get(j));
            break;
        }
        if (dz) {
            Raw<T, V> o;
            o.set(v);
            o.store_any(dz);
        }
    }
}

// Token rows: 32 lanes of V channels by 8 rows; a slice of rows a workgroup (12544 x 768,
// bf16, with SiLU: 14.6 us, memory). The
// last lane of a row reaches back over the one before, and counts what is its own.
template <typename T, int V>
__global__ __launch_bounds__(256) void slope_rows(const SlopeParams p)
{
    __shared__ float sum[8][32 * V + 1];
    const int cx = threadIdx.x % 32, ry = threadIdx.x / 32;
    const long tiles = (p.n + 32 * V - 1) / (32 * V), id = p.first + blockIdx.x;
    const long c0 = (id % tiles * 32 + cx) * V, c = min(c0, p.n - V), slice = id / tiles, b = slice / p.slices;
    const long r1 = slice % p.slices * p.each, r2 = min(r1 + p.each, p.rows);
    float s[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = 0.0f;
    if (c0 < p.n) {
#pragma unroll 4
        for (long r = r1 + ry; r < r2; r += 8) {
            float v[V];
            const long at = (b * p.rows + r) * p.n + c;
            slope_of<T, V>(p, static_cast<const T *>(p.dy) + b * p.d_b + r * p.d_s + c, static_cast<const T *>(p.pre) + at,
                           p.dz ? static_cast<T *>(p.dz) + at : nullptr, v);
#pragma unroll
            for (int j = 0; j < V; ++j) s[j] += v[j];
        }
    }
    if (!p.part) return;
    const int back = static_cast<int>(c0 - c);
    if (c0 < p.n) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j >= back) sum[ry][cx * V + j - back] = s[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * V; i += 256) {
        const long col = id % tiles * 32 * V + i;
        if (col >= p.n) continue;
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += sum[k][i];
        p.part[slice * p.n + col] = t;
    }
}

// Maps: a slice of one channel's cells a workgroup.
template <typename T, int V>
__global__ __launch_bounds__(256) void slope_maps(const SlopeParams p)
{
    __shared__ float sum[4];
    const long id = p.first + blockIdx.x, c = id % p.n, slice = id / p.n, b = slice / p.slices;
    const long r1 = slice % p.slices * p.each, r2 = min(r1 + p.each, p.rows), at = (b * p.n + c) * p.rows;
    const T *dy = static_cast<const T *>(p.dy) + b * p.d_b + c * p.d_s, *pre = static_cast<const T *>(p.pre) + at;
    T *dz = p.dz ? static_cast<T *>(p.dz) + at : nullptr;
    float s = 0.0f;
    long r = r1 + threadIdx.x * V;
#pragma unroll 2
    for (; r + V <= r2; r += 256 * V) {
        float v[V];
        slope_of<T, V>(p, dy + r, pre + r, dz ? dz + r : nullptr, v);
#pragma unroll
        for (int j = 0; j < V; ++j) s += v[j];
    }
    for (const long end = min(r + V, r2); r < end; ++r) {  // (one thread's, at the end of the row)
        float v[1];
        slope_of<T, 1>(p, dy + r, pre + r, dz ? dz + r : nullptr, v);
        s += v[0];
    }
    if (!p.part) return;
    s = lane_sum<64>(s);
    if (threadIdx.x % 64 == 0) sum[threadIdx.x / 64] = s;
    __syncthreads();
    if (threadIdx.x == 0) p.part[slice * p.n + c] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// Slices of a batch entry's rows: enough workgroups to fill the chip, and whole
// vectors. At most 512 partial rows where the batch allows.
void slope_slices(const ssm2d_linear_shape &a, bool maps, int *slices, long *each)
{
    const long tiles = maps ? a.n : (a.n + 127) / 128, unit = maps ? 2048 : 32;
    long want = std::max(1L, std::min(2048 / std::max(1L, std::min<long>(tiles * a.batch, 2048)), std::max(1L, 512 / static_cast<long>(a.batch))));
    want = std::min(want, static_cast<long>((a.rows + unit - 1) / unit));
    *each = round_up_to((a.rows + want - 1) / std::max(want, 1L), 8);
    *slices = static_cast<int>((a.rows + *each - 1) / std::max(*each, 1L));
}

template <typename T>
int run_slope(SlopeParams p, bool maps, hipStream_t s)
{
    constexpr int V = 16 / static_cast<int>(sizeof(T));
    auto go = [&](auto vec) {
        constexpr int W = decltype(vec)::value;
        const long groups = p.slices * p.batch * (maps ? p.n : (p.n + 32 * W - 1) / (32 * W)), most = most_groups(256);
        for (p.first = 0; p.first < groups; p.first += most) {
            const dim3 grid(static_cast<unsigned>(std::min(groups - p.first, most)));
            if (maps) slope_maps<T, W><<<grid, dim3(256), 0, s>>>(p);
            else slope_rows<T, W><<<grid, dim3(256), 0, s>>>(p);
            const int st = launched();
            if (st != SSM2D_OK) return st;
        }
        return static_cast<int>(SSM2D_OK);
    };
    return maps || p.n >= V ? go(std::integral_constant<int, V>{}) : go(std::integral_constant<int, 1>{});
}

// ------------------------------------------------------------------ checks

constexpr uint32_t kLinearFlags = SSM2D_LINEAR_X_MAPS | SSM2D_LINEAR_Y_MAPS;

int check_linear(const ssm2d_linear_shape *a, int act, uint32_t flags)
{
    if ((flags & ~kLinearFlags) || act < SSM2D_ACT_NONE || act > SSM2D_ACT_GELU) return SSM2D_ERR_BAD_FLAGS;
    if (!a) return SSM2D_ERR_NULLPTR;
    if (a->batch < 0 || a->rows < 0 || a->n < 0 || a->k < 0) return SSM2D_ERR_BAD_DIM;
    for (const int64_t st : {a->x_stride[0], a->x_stride[1], a->r_stride[0], a->r_stride[1], a->w_stride}) {
        if (st < 0) return SSM2D_ERR_BAD_DIM;
        if (st >= (int64_t{1} << 40)) return SSM2D_ERR_UNSUPPORTED;
    }
    const int64_t most = (int64_t{1} << 31) - 256;
    if (a->rows >= most || a->n >= most || a->k >= most || a->batch >= most) return SSM2D_ERR_UNSUPPORTED;
    const double b = static_cast<double>(a->batch), r = static_cast<double>(a->rows), n = static_cast<double>(a->n), k = static_cast<double>(a->k);
    for (const double t : {b * (r / 64 + 1) * (n / 64 + 1), b * (r / 64 + 1) * (k / 64 + 1), (k / 64 + 1) * (n / 64 + 1)})
        if (t >= 2147483648.0) return SSM2D_ERR_UNSUPPORTED;
    if (b * (r / 32 + 1) >= 2147483648.0) return SSM2D_ERR_UNSUPPORTED;  // (steps of dweight's sum)
    return SSM2D_OK;
}

// Whether rows of `len` at strides s0 and s1 are whole 16-byte words.
bool in_words(const void *p, long len, long s0, long s1, size_t size)
{
    const long v = 16 / static_cast<long>(size);
    return len % v == 0 && s0 % v == 0 && s1 % v == 0 && !off_by(p, 16);
}

// The operand with index pairs (rows, len) at p, `ld` between rows, contiguous along len.
struct Side {
    const void *p;
    long ld, bs;
    bool kc;
};

template <typename T>
void sides(GemmParams &g, const Side &a, const Side &b)
{
    const long kb = g.kb > 1 ? g.kb : g.batch;
    g.a = a.p, g.a_ld = a.ld, g.a_bs = a.bs, g.b = b.p, g.b_ld = b.ld, g.b_bs = b.bs;
    // (a tile's offsets within 31 bits, and rows that do not lie over each other)
    auto straight = [&](const Side &x, long len) {
        return in_words(x.p, len, x.ld, kb > 1 ? x.bs : 0, sizeof(T)) && x.ld >= len && x.ld < (1L << 22);
    };
    g.straight = sizeof(T) == 2 && straight(a, a.kc ? g.K : g.M) && straight(b, b.kc ? g.K : g.N);
}

template <typename T>
GemmPlan plan_fwd(const ssm2d_linear_shape &a, uint32_t flags)
{
    GemmPlan g = flags & SSM2D_LINEAR_Y_MAPS ? plan_gemm<T>(a.batch, a.n, a.rows, a.k, 1) : plan_gemm<T>(a.batch, a.rows, a.n, a.k, 1);
    g.few = !flags && a.batch == 1 && few_rows<T>(g, a.rows, a.n, a.k);
    if (g.few) g.bytes = 0;
    return g;
}

template <typename T>
int64_t fwd_workspace(const ssm2d_linear_shape *a, uint32_t flags)
{
    const int st = check_linear(a, 0, flags);
    if (st != SSM2D_OK) return -st;
    if (a->batch == 0 || a->rows == 0 || a->n == 0) return 0;
    return plan_fwd<T>(*a, flags).bytes;
}

template <typename T>
int linear_fwd(const T *x, const T *weight, const float *bias, const T *res, T *y, T *pre, const ssm2d_linear_shape *a, int act, uint32_t flags,
               void *ws, int64_t ws_bytes, void *stream)
{
    const int st = check_linear(a, act, flags);
    if (st != SSM2D_OK) return st;
    if (a->batch == 0 || a->rows == 0 || a->n == 0) return SSM2D_OK;
    if ((a->k > 0 && (!x || !weight)) || !y) return SSM2D_ERR_NULLPTR;
    if (off_by(x, sizeof(T)) || off_by(weight, sizeof(T)) || off_by(res, sizeof(T)) || off_by(y, sizeof(T)) || off_by(pre, sizeof(T)) ||
        off_by(bias, 4) || off_by(ws, 16))
        return SSM2D_ERR_MISALIGNED;
    const GemmPlan plan = plan_fwd<T>(*a, flags);
    if (plan.bytes > 0 && (!ws || ws_bytes < plan.bytes)) return SSM2D_ERR_NOMEM;
    const bool xm = flags & SSM2D_LINEAR_X_MAPS, ym = flags & SSM2D_LINEAR_Y_MAPS;
    GemmParams g{};
    g.batch = a->batch, g.kb = 1, g.K = static_cast<int>(a->k);
    g.bias = bias, g.bias_m = ym, g.act = act, g.res = res, g.c = y, g.pre = pre;
    g.r_bs = a->r_stride[0], g.r_ld = a->r_stride[1], g.c_bs = a->rows * a->n;
    const Side w{weight, a->w_stride, 0, true}, in{x, a->x_stride[1], a->x_stride[0], !xm};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (ym) {
        g.M = static_cast<int>(a->n), g.N = static_cast<int>(a->rows), g.c_ld = a->rows;
        sides<T>(g, w, in);
    } else {
        g.M = static_cast<int>(a->rows), g.N = static_cast<int>(a->n), g.c_ld = a->n;
        sides<T>(g, in, w);
    }
    return run_gemm<T>(g, plan, ym || !xm, !ym || !xm, ws, s);
}

// The backward's workspace: dz, the slices' sums (or those of dweight's parts: not
// both), and the parts' sums.
struct BwdPlan {
    int slices;
    long each;
    int64_t dz, sums, parts;
    GemmPlan dx, dw, pair_dx, pair_dw;
    bool pair;
};
template <typename T>
BwdPlan plan_bwd(const ssm2d_linear_shape &a, int act, uint32_t flags)
{
    BwdPlan p{};
    slope_slices(a, flags & SSM2D_LINEAR_Y_MAPS, &p.slices, &p.each);
    p.dz = act != SSM2D_ACT_NONE ? round_up_to(a.batch * a.rows * a.n * static_cast<int64_t>(sizeof(T)), 256) : 0;
    const long M = flags & SSM2D_LINEAR_X_MAPS ? a.k : a.rows, N = flags & SSM2D_LINEAR_X_MAPS ? a.rows : a.k;
    p.pair_dx = p.dx = plan_gemm<T>(a.batch, M, N, a.n, 1);
    p.pair_dw = p.dw = plan_gemm<T>(1, a.n, a.k, a.rows, a.batch);
    p.pair = a.k > 0 && plan_pair<T>(p.pair_dx, p.pair_dw, a.batch, M, N, a.n, a.k);
    p.sums = round_up_to(std::max<int64_t>(p.slices * a.batch, std::max(p.dw.splits, p.pair_dw.splits)) * a.n * 4, 16);
    p.parts = std::max({p.dx.bytes, p.dw.bytes, p.pair_dw.bytes});
    return p;
}

template <typename T>
int64_t bwd_workspace(const ssm2d_linear_shape *a, int act, uint32_t flags)
{
    const int st = check_linear(a, act, flags);
    if (st != SSM2D_OK) return -st;
    if (a->batch == 0 || a->rows == 0 || a->n == 0) return 0;
    const BwdPlan p = plan_bwd<T>(*a, act, flags);
    return p.dz + p.sums + p.parts;
}

template <typename T>
__global__ void clear_all(T *p, long n)
{
    const long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < n) p[i] = T{0};
}
template <typename T>
int clear(T *p, long n, hipStream_t s)
{
    if (!p || n == 0) return SSM2D_OK;
    const long most = most_groups(256) * 256;
    for (long at = 0; at < n; at += most) {
        const long m = std::min(most, n - at);
        clear_all<T><<<dim3(static_cast<unsigned>((m + 255) / 256)), dim3(256), 0, s>>>(p + at, m);
        const int st = launched();
        if (st != SSM2D_OK) return st;
    }
    return SSM2D_OK;
}

template <typename T>
int linear_bwd(const T *x, const T *weight, const T *pre, const T *dy, T *dx, T *dweight, float *dbias, const ssm2d_linear_shape *a, int act,
               uint32_t flags, void *ws, int64_t ws_bytes, void *stream)
{
    int st = check_linear(a, act, flags);
    if (st != SSM2D_OK) return st;
    if (off_by(x, sizeof(T)) || off_by(weight, sizeof(T)) || off_by(pre, sizeof(T)) || off_by(dy, sizeof(T)) || off_by(dx, sizeof(T)) ||
        off_by(dweight, sizeof(T)) || off_by(dbias, 4) || off_by(ws, 16))
        return SSM2D_ERR_MISALIGNED;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const long B = a->batch, R = a->rows, n = a->n, k = a->k;
    if (B == 0 || R == 0 || n == 0) {  // sums over nothing
        if ((st = clear(dx, B * R * k, s)) != SSM2D_OK || (st = clear(dweight, n * k, s)) != SSM2D_OK) return st;
        return clear(dbias, n, s);
    }
    if (k == 0) dx = nullptr, dweight = nullptr;
    if (!dx && !dweight && !dbias) return SSM2D_OK;
    if (!dy || (act != SSM2D_ACT_NONE && !pre) || (dx && !weight) || (dweight && !x)) return SSM2D_ERR_NULLPTR;
    const BwdPlan plan = plan_bwd<T>(*a, act, flags);
    if (!ws || ws_bytes < plan.dz + plan.sums + plan.parts) return SSM2D_ERR_NOMEM;
    const bool xm = flags & SSM2D_LINEAR_X_MAPS, ym = flags & SSM2D_LINEAR_Y_MAPS;
    float *sums = reinterpret_cast<float *>(static_cast<char *>(ws) + plan.dz);
    void *parts = static_cast<char *>(ws) + plan.dz + plan.sums;
    const bool pair = plan.pair && dx && dweight;
    // dbias without an activation: dweight's product sums dy's rows with the rest
    // (with one, its slopes are summed as they were before dz was rounded).
    const bool by_product = pair && dbias && act == SSM2D_ACT_NONE;
    Side dz{dy, a->r_stride[1], a->r_stride[0], true};  // (contiguous: channels of rows, cells of maps)
    int sum_rows = 0;
    if (act != SSM2D_ACT_NONE || (dbias && !by_product)) {
        SlopeParams p{};
        p.dy = dy, p.pre = pre, p.dz = act != SSM2D_ACT_NONE && (dx || dweight) ? ws : nullptr, p.part = dbias ? sums : nullptr;
        p.batch = B, p.rows = R, p.n = n, p.d_b = a->r_stride[0], p.d_s = a->r_stride[1], p.act = act, p.slices = plan.slices, p.each = plan.each;
        if ((st = run_slope<T>(p, ym, s)) != SSM2D_OK) return st;
        if (dbias) sum_rows = static_cast<int>(plan.slices * B);
        if (act != SSM2D_ACT_NONE) dz = Side{ws, ym ? R : n, R * n, true};
    }
    if (dbias && !dweight) {
        fold_rows<<<dim3(fold_blocks(n)), dim3(kFoldThreads), 0, s>>>(sums, sum_rows, n, dbias);
        if ((st = launched()) != SSM2D_OK) return st;
    }
    auto along = [](Side side, bool kc) {
        side.kc = kc;
        return side;
    };
    GemmParams gx{}, gw{};
    if (dx) {
        gx.batch = B, gx.kb = 1, gx.K = static_cast<int>(n), gx.c = dx, gx.c_bs = R * k;
        const Side w{weight, a->w_stride, 0, false};
        if (xm) {
            gx.M = static_cast<int>(k), gx.N = static_cast<int>(R), gx.c_ld = R;
            sides<T>(gx, w, along(dz, !ym));
        } else {
            gx.M = static_cast<int>(R), gx.N = static_cast<int>(k), gx.c_ld = k;
            sides<T>(gx, along(dz, !ym), w);
        }
        if (!pair && (st = run_gemm<T>(gx, plan.dx, !xm && !ym, xm && !ym, parts, s)) != SSM2D_OK) return st;
    }
    if (dweight) {
        gw.batch = 1, gw.kb = static_cast<int>(B), gw.K = static_cast<int>(R), gw.M = static_cast<int>(n), gw.N = static_cast<int>(k);
        gw.c = dweight, gw.c_ld = k;
        sides<T>(gw, along(dz, ym), Side{x, a->x_stride[1], a->x_stride[0], xm});
        if (by_product) {
            gw.sums = plan.pair_dw.splits > 1 ? sums : dbias;
            sum_rows = plan.pair_dw.splits > 1 ? plan.pair_dw.splits : 0;
        }
        if (dbias && sum_rows > 0) gw.fold = sums, gw.fold_to = dbias, gw.fold_rows = sum_rows, gw.fold_n = static_cast<int>(n);
        st = pair ? run_pair<T>(gx, plan.pair_dx, gw, plan.pair_dw, xm, ym, parts, s) : run_gemm<T>(gw, plan.dw, ym, xm, parts, s);
    }
    return st;
}

}  // namespace
}  // namespace ssm2d_impl

extern "C" {

int64_t ssm2d_linear_fwd_workspace(const ssm2d_linear_shape *shape, uint32_t flags) { return ssm2d_impl::fwd_workspace<float>(shape, flags); }
int64_t ssm2d_linear_fwd_workspace_bf16(const ssm2d_linear_shape *shape, uint32_t flags)
{
    return ssm2d_impl::fwd_workspace<uint16_t>(shape, flags);
}
int64_t ssm2d_linear_bwd_workspace(const ssm2d_linear_shape *shape, int act, uint32_t flags)
{
    return ssm2d_impl::bwd_workspace<float>(shape, act, flags);
}
int64_t ssm2d_linear_bwd_workspace_bf16(const ssm2d_linear_shape *shape, int act, uint32_t flags)
{
    return ssm2d_impl::bwd_workspace<uint16_t>(shape, act, flags);
}

int ssm2d_linear_fwd(const float *x, const float *weight, const float *bias, const float *residual, float *y, float *pre,
                     const ssm2d_linear_shape *shape, int act, uint32_t flags, void *workspace, int64_t workspace_bytes, void *stream)
{
    return ssm2d_impl::linear_fwd<float>(x, weight, bias, residual, y, pre, shape, act, flags, workspace, workspace_bytes, stream);
}

int ssm2d_linear_fwd_bf16(const uint16_t *x, const uint16_t *weight, const float *bias, const uint16_t *residual, uint16_t *y, uint16_t *pre,
                          const ssm2d_linear_shape *shape, int act, uint32_t flags, void *workspace, int64_t workspace_bytes, void *stream)
{
    return ssm2d_impl::linear_fwd<uint16_t>(x, weight, bias, residual, y, pre, shape, act, flags, workspace, workspace_bytes, stream);
}

int ssm2d_linear_bwd(const float *x, const float *weight, const float *pre, const float *dy, float *dx, float *dweight, float *dbias,
                     const ssm2d_linear_shape *shape, int act, uint32_t flags, void *workspace, int64_t workspace_bytes, void *stream)
{
    return ssm2d_impl::linear_bwd<float>(x, weight, pre, dy, dx, dweight, dbias, shape, act, flags, workspace, workspace_bytes, stream);
}

int ssm2d_linear_bwd_bf16(const uint16_t *x, const uint16_t *weight, const uint16_t *pre, const uint16_t *dy, uint16_t *dx, uint16_t *dweight,
                          float *dbias, const ssm2d_linear_shape *shape, int act, uint32_t flags, void *workspace, int64_t workspace_bytes,
                          void *stream)
{
    return ssm2d_impl::linear_bwd<uint16_t>(x, weight, pre, dy, dx, dweight, dbias, shape, act, flags, workspace, workspace_bytes, stream);
}

}  // extern "C"
