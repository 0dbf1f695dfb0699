// libssm2d: the gated linear recurrence's entries: checks, how tokens are cut
// into segments, and the join between the launches (recurrence.h has the kernels).
#include "recurrence.h"

#include <cmath>

namespace ssm2d_impl {

extern template int rec_run<uint16_t, false>(const RecParams &, const RecPlan &, long, bool, hipStream_t);
extern template int rec_run<uint16_t, true>(const RecParams &, const RecPlan &, long, bool, hipStream_t);
extern template int rec_run<float, false>(const RecParams &, const RecPlan &, long, bool, hipStream_t);
extern template int rec_run<float, true>(const RecParams &, const RecPlan &, long, bool, hipStream_t);

namespace {

// Per channel: what enters each segment, from the segments' products and sums
// (H, and F from the last segment to the first), in place. 16 threads a channel
// take as many segments each, then join.
template <bool PACKED>
__global__ __launch_bounds__(256) void rec_join(const RecParams p)
{
    __shared__ float sP[16][17], sc[16][17];
    const int cx = threadIdx.x % 16, k = threadIdx.x / 16;
    const long chan = static_cast<long>(blockIdx.x % p.tiles) * 16 + cx, b = p.first + blockIdx.x / p.tiles;
    const bool live = chan < p.n;
    const long base = b * p.S * p.n + (live ? chan : 0);
    const int each = (p.S + 15) / 16, s0 = min(k * each, p.S), s1 = min(s0 + each, p.S);
    auto at = [&](int s) { return base + static_cast<long>(s) * p.n; };
    auto both = [&](float *buf, bool down, float enter) {
        float P = 1.0f, c = 0.0f;
        for (int i = s0; i < s1; ++i) {
            const int s = down ? s1 - 1 - (i - s0) : i;
            float q = p.P[at(s)], d = buf[at(s)];
            join<PACKED, true>(P, c, q, d);
            P = q, c = d;
        }
        sP[k][cx] = P, sc[k][cx] = c;
        __syncthreads();
        float h = enter;
        for (int i = 0; i < (down ? 15 - k : k); ++i) h = pass<PACKED, true>(sP[down ? 15 - i : i][cx], sc[down ? 15 - i : i][cx], h);
        for (int i = s0; i < s1; ++i) {
            const int s = down ? s1 - 1 - (i - s0) : i;
            const float q = p.P[at(s)], d = buf[at(s)];
            if (live) buf[at(s)] = h;
            h = pass<PACKED, true>(q, d, h);
        }
        __syncthreads();
    };
    both(p.H, false, !PACKED && p.h_init && live ? p.h_init[b * p.n + chan] : 0.0f);
    both(p.F, true, !PACKED && p.dh_last && live ? p.dh_last[b * p.n + chan] : 0.0f);
}

// Before a relay: no word is there, and no ticket drawn.
__global__ __launch_bounds__(256) void relay_open(uint4 *words, long quads, unsigned *tickets, long chains, long first)
{
    const long i = (first + blockIdx.x) * 256 + threadIdx.x;
    if (i < quads) words[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
    if (i < chains) tickets[i * kTicketWords] = 0u;
}

// Set where a relay's wait was given up, read and cleared by ssm2d_sync_check.
__device__ unsigned relay_gave_up;

// How long the relay's workgroups of a call on the current device wait, and where they say that they did not.
int bound_waits(RecParams &p)
{
    return guarded([&] {
        int dev = 0;
        hipError_t e = hipGetDevice(&dev);
        if (e != hipSuccess) return hip_fail(e);
        std::lock_guard<std::recursive_mutex> lock(g_mutex);
        auto it = g_gave_up.find(dev);
        if (it == g_gave_up.end()) {
            void *at = nullptr;
            e = hipGetSymbolAddress(&at, HIP_SYMBOL(relay_gave_up));
            if (e != hipSuccess) return hip_fail(e);
            it = g_gave_up.emplace(dev, static_cast<unsigned *>(at)).first;
        }
        p.gave_up = it->second;
        p.polls = g_spin_limit > 0 ? static_cast<int>(std::min<long long>(g_spin_limit, kMostPolls)) : kMostPolls;
        return static_cast<int>(SSM2D_OK);
    });
}

__global__ void copy_floats(const float *src, float *dst, long n)
{
    const long i = static_cast<long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < n) dst[i] = src[i];
}

constexpr uint32_t kRecFlags = SSM2D_RECUR_SIGMOID | SSM2D_RECUR_MAPS | SSM2D_RECUR_REVERSE;

int check_rec(const ssm2d_recurrence_shape *a, uint32_t flags)
{
    if (flags & ~kRecFlags) return SSM2D_ERR_BAD_FLAGS;
    if (!a) return SSM2D_ERR_NULLPTR;
    if (a->n_seq > 0 && (flags & (SSM2D_RECUR_MAPS | SSM2D_RECUR_REVERSE))) return SSM2D_ERR_BAD_FLAGS;
    if (a->batch < 0 || a->tokens < 0 || a->channels < 0 || a->n_seq < 0 || (a->n_seq > 0 && a->batch != 1)) return SSM2D_ERR_BAD_DIM;
    for (const auto &st : {a->x_stride, a->g_stride, a->dh_stride})
        if (st[0] < 0 || st[1] < 0) return SSM2D_ERR_BAD_DIM;
    const int64_t most = (int64_t{1} << 31) - 65536;
    if (a->batch >= most || a->tokens >= most || a->channels >= most || a->n_seq >= most) return SSM2D_ERR_UNSUPPORTED;
    // (states: one launch copies or clears them)
    if (a->batch * a->channels >= (int64_t{1} << 31) || a->n_seq * a->channels > 256 * most_groups(256)) return SSM2D_ERR_UNSUPPORTED;
    if (static_cast<double>(a->batch) * static_cast<double>(a->tokens) * static_cast<double>(a->channels) > 1e14) return SSM2D_ERR_UNSUPPORTED;
    return SSM2D_OK;
}

// Token rows that are walked over by a thread for each few channels.
bool few_tokens(const ssm2d_recurrence_shape &a, uint32_t flags) { return a.tokens <= 8 && a.n_seq == 0 && !(flags & SSM2D_RECUR_MAPS); }

// How many tokens a segment has (whole chunks); token rows: for v channels a lane.
struct Cut {
    long seg;
    int S, tiles;
    int groups;    // forward: of the relay
    int64_t chains;
};
template <typename T, bool BWD>
Cut cut_tokens(const ssm2d_recurrence_shape &a, uint32_t flags, int v)
{
    Cut c{};
    // A workgroup's chunk: of one that walks over them, and of a relay or the backward's.
    long chunk, wide, groups;
    int relay = 64;  // segments of a group
    double fit;      // workgroups that the chip takes at once, of those that walk
    if (flags & SSM2D_RECUR_MAPS) {
        int rows = 1;
        chunk = wide = with_map_dims<T>(a.tokens, [&](auto dims) {
            rows = decltype(dims)::kRows;
            return static_cast<long>(decltype(dims)::template kChunk<T>);
        });
        groups = (a.batch * a.channels + rows - 1) / rows;
        fit = 2048.0;
    } else {
        auto dims = [&](auto vec) {
            using N = RowDims<T, decltype(vec)::value, false>;
            using W = RowDims<T, decltype(vec)::value, true>;
            chunk = N::kChunk, wide = W::kChunk, relay = 4 * W::kThreads / (W::kBX * v);
            c.tiles = static_cast<int>((a.channels + N::kBX * v - 1) / (N::kBX * v));
        };
        if (v > 1) dims(std::integral_constant<int, kRowV<T>>{});
        else dims(std::integral_constant<int, 1>{});
        groups = a.batch * c.tiles;
        fit = 1024.0;
    }
    // Segments of one chunk, or of all tokens: the forward walks over all chunks where
    // its channels make workgroups enough, by what rounds of as many workgroups as
    // fit the chip take. (A relay's start and its waits are as long as two rounds.)
    const long chunks = (a.tokens + chunk - 1) / chunk;
    const double walk = std::ceil(groups / fit) * chunks, cut = std::ceil(static_cast<double>(groups) * chunks / fit) + 2.0;
    c.seg = BWD || walk > cut ? wide : std::max(chunks, 1L) * chunk;
    c.S = static_cast<int>((a.tokens + c.seg - 1) / c.seg);
    c.groups = (c.S + relay - 1) / relay;
    c.chains = a.batch * (flags & SSM2D_RECUR_MAPS ? a.channels : c.tiles);
    return c;
}

constexpr int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Whether workgroups read states that another one writes, so that one written in
// place is read from a copy: packed sequences begin and end anywhere, the last
// lane of a row reaches back over channels of other lanes, and all of a relay's
// first group read what enters it.
template <typename T>
bool shares_states(const ssm2d_recurrence_shape &a, uint32_t flags, bool relay)
{
    return a.n_seq > 0 || relay || (!(flags & SSM2D_RECUR_MAPS) && a.channels % kRowV<T> != 0);
}
// Bytes of a relay's words: products and sums, then states, in whole 16 bytes; behind them the counters.
int64_t relay_words(const Cut &c, int64_t lines) { return round_up(lines * (int64_t{8} * c.S + int64_t{4} * c.groups), 16); }

template <typename T, bool BWD>
int64_t rec_workspace(const ssm2d_recurrence_shape *a, uint32_t flags)
{
    const int st = check_rec(a, flags);
    if (st != SSM2D_OK) return -st;
    if (a->batch == 0 || a->tokens == 0 || a->channels == 0) return 0;
    int64_t bytes = 0;
    bool relay = false;
    for (const int v : {kRowV<T>, 1}) {
        const Cut c = cut_tokens<T, BWD>(*a, flags, v);
        const int64_t lines = a->batch * a->channels;
        if (c.S > 1) bytes = std::max(bytes, BWD ? 3 * lines * c.S * 4 : relay_words(c, lines) + c.chains * kTicketWords * 4);
        relay = relay || (!BWD && c.S > 1);
    }
    if (shares_states<T>(*a, flags, relay) && (BWD || !few_tokens(*a, flags))) bytes = round_up(bytes, 16) + std::max(a->n_seq, a->batch) * a->channels * 4;
    return bytes;
}

template <typename T, bool BWD>
int rec_entry(const T *x, const T *g, const float *h_init, const int32_t *cu, const T *dh, const float *dh_last, T *out, T *dg, float *last,
              const ssm2d_recurrence_shape *a, uint32_t flags, void *ws, int64_t ws_bytes, void *stream)
{
    // (`last`: h_last of the forward, dh_init of the backward; `state`: what an empty sequence passes on)
    int st = check_rec(a, flags);
    if (st != SSM2D_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const long B = a->batch, T_ = a->tokens, n = a->channels, states = (a->n_seq > 0 ? a->n_seq : B) * n;
    const float *state = BWD ? dh_last : h_init;
    if (states == 0 || (T_ == 0 && !last)) return SSM2D_OK;
    if (off_by(h_init, 4) || off_by(dh_last, 4) || off_by(last, 4)) return SSM2D_ERR_MISALIGNED;
    auto blocks = [](long m) { return dim3(static_cast<unsigned>((m + 255) / 256)); };
    if (T_ == 0) {
        if (last == state) return SSM2D_OK;
        if (state) copy_floats<<<blocks(states), dim3(256), 0, s>>>(state, last, states);
        else clear_floats<<<blocks(states), dim3(256), 0, s>>>(last, states);
        return launched();
    }
    if (!x || !g || !out || (BWD && (!dh || !dg)) || (a->n_seq > 0 && !cu)) return SSM2D_ERR_NULLPTR;
    if (off_by(x, sizeof(T)) || off_by(g, sizeof(T)) || off_by(out, sizeof(T)) || off_by(dh, sizeof(T)) || off_by(dg, sizeof(T)) ||
        off_by(ws, 16) || (a->n_seq > 0 && off_by(cu, 4)))
        return SSM2D_ERR_MISALIGNED;
    const int64_t need = rec_workspace<T, BWD>(a, flags);
    if (need > 0 && (!ws || ws_bytes < need)) return SSM2D_ERR_NOMEM;
    RecPlan plan{};
    plan.maps = flags & SSM2D_RECUR_MAPS, plan.packed = a->n_seq > 0, plan.sig = flags & SSM2D_RECUR_SIGMOID;
    plan.rev = flags & SSM2D_RECUR_REVERSE;
    // (a chunk of tokens spans less than 2^31 bytes)
    const int64_t far = std::max({a->x_stride[1], a->g_stride[1], a->dh_stride[1], a->channels});
    plan.v = n >= kRowV<T> && far < (int64_t{1} << 20) ? kRowV<T> : 1;
    plan.few = !BWD && few_tokens(*a, flags);
    const Cut c = cut_tokens<T, BWD>(*a, flags, plan.v);
    plan.cells = T_;
    RecParams p{};
    p.x = x, p.g = g, p.dh = dh, p.h_init = h_init, p.dh_last = dh_last, p.cu = cu;
    p.T = T_, p.seg = c.seg, p.S = c.S, p.n = static_cast<int>(n), p.n_seq = static_cast<int>(a->n_seq), p.tiles = c.tiles;
    p.x_b = a->x_stride[0], p.g_b = a->g_stride[0], p.d_b = a->dh_stride[0];
    p.x_t = a->x_stride[1], p.g_t = a->g_stride[1], p.d_t = a->dh_stride[1], p.rev = plan.rev;
    if (BWD) p.dx = out, p.dg = dg, p.dh_init = last;
    else p.h = out, p.h_last = last;
    const long plane = B * p.S * n;
    if (BWD) {
        p.P = static_cast<float *>(ws), p.H = p.P + plane, p.F = p.H + plane;
    } else {
        p.parts = static_cast<unsigned long *>(ws), p.enter = reinterpret_cast<unsigned *>(p.parts + plane);
        p.tickets = reinterpret_cast<unsigned *>(static_cast<char *>(ws) + relay_words(c, B * n)), p.chains = c.chains;
    }
    if (last && last == state) {
        if (shares_states<T>(*a, flags, !BWD && p.S > 1) && !plan.few) {
            float *copy = reinterpret_cast<float *>(static_cast<char *>(ws) + (need - states * 4));
            copy_floats<<<blocks(states), dim3(256), 0, s>>>(state, copy, states);
            if ((st = launched()) != SSM2D_OK) return st;
            (BWD ? p.dh_last : p.h_init) = copy;
        }
    } else {
        p.pass_on = plan.packed && last;
    }
    if (!BWD) {
        if (p.S > 1) {
            if ((st = bound_waits(p)) != SSM2D_OK) return st;
            const long quads = relay_words(c, B * n) / 16;
            const int opened = rec_launch(p, (std::max<long>(quads, c.chains) + 255) / 256, 256, [&](const RecParams &q, dim3 grid) {
                relay_open<<<grid, dim3(256), 0, s>>>(static_cast<uint4 *>(ws), quads, p.tickets, c.chains, q.first);
            });
            if (opened != SSM2D_OK) return opened;
        }
        return rec_run<T, BWD>(p, plan, B, p.S > 1, s);
    }
    if (p.S > 1) {
        if ((st = rec_run<T, BWD>(p, plan, B, true, s)) != SSM2D_OK) return st;
        RecParams q = p;
        q.tiles = static_cast<int>((n + 15) / 16);
        const long most = std::max(1L, most_groups(256) / q.tiles);
        for (q.first = 0; q.first < B; q.first += most) {
            const dim3 grid(static_cast<unsigned>(std::min(B - q.first, most) * q.tiles));
            if (plan.packed) rec_join<true><<<grid, dim3(256), 0, s>>>(q);
            else rec_join<false><<<grid, dim3(256), 0, s>>>(q);
            if ((st = launched()) != SSM2D_OK) return st;
        }
    }
    return rec_run<T, BWD>(p, plan, B, false, s);
}

}  // namespace
}  // namespace ssm2d_impl

extern "C" {

int64_t ssm2d_recurrence_fwd_workspace(const ssm2d_recurrence_shape *shape, uint32_t flags)
{
    return ssm2d_impl::rec_workspace<float, false>(shape, flags);
}
int64_t ssm2d_recurrence_fwd_workspace_bf16(const ssm2d_recurrence_shape *shape, uint32_t flags)
{
    return ssm2d_impl::rec_workspace<uint16_t, false>(shape, flags);
}
int64_t ssm2d_recurrence_bwd_workspace(const ssm2d_recurrence_shape *shape, uint32_t flags)
{
    return ssm2d_impl::rec_workspace<float, true>(shape, flags);
}
int64_t ssm2d_recurrence_bwd_workspace_bf16(const ssm2d_recurrence_shape *shape, uint32_t flags)
{
    return ssm2d_impl::rec_workspace<uint16_t, true>(shape, flags);
}

int ssm2d_recurrence_fwd(const float *x, const float *g, const float *h_init, const int32_t *cu_seqlens, float *h, float *h_last,
                         const ssm2d_recurrence_shape *shape, uint32_t flags, void *workspace, int64_t workspace_bytes, void *stream)
{
    return ssm2d_impl::rec_entry<float, false>(x, g, h_init, cu_seqlens, nullptr, nullptr, h, nullptr, h_last, shape, flags, workspace,
                                               workspace_bytes, stream);
}

int ssm2d_recurrence_fwd_bf16(const uint16_t *x, const uint16_t *g, const float *h_init, const int32_t *cu_seqlens, uint16_t *h,
                              float *h_last, const ssm2d_recurrence_shape *shape, uint32_t flags, void *workspace, int64_t workspace_bytes,
                              void *stream)
{
    return ssm2d_impl::rec_entry<uint16_t, false>(x, g, h_init, cu_seqlens, nullptr, nullptr, h, nullptr, h_last, shape, flags, workspace,
                                                  workspace_bytes, stream);
}

int ssm2d_recurrence_bwd(const float *x, const float *g, const float *h_init, const int32_t *cu_seqlens, const float *dh,
                         const float *dh_last, float *dx, float *dg, float *dh_init, const ssm2d_recurrence_shape *shape, uint32_t flags,
                         void *workspace, int64_t workspace_bytes, void *stream)
{
    return ssm2d_impl::rec_entry<float, true>(x, g, h_init, cu_seqlens, dh, dh_last, dx, dg, dh_init, shape, flags, workspace,
                                              workspace_bytes, stream);
}

int ssm2d_recurrence_bwd_bf16(const uint16_t *x, const uint16_t *g, const float *h_init, const int32_t *cu_seqlens, const uint16_t *dh,
                              const float *dh_last, uint16_t *dx, uint16_t *dg, float *dh_init, const ssm2d_recurrence_shape *shape,
                              uint32_t flags, void *workspace, int64_t workspace_bytes, void *stream)
{
    return ssm2d_impl::rec_entry<uint16_t, true>(x, g, h_init, cu_seqlens, dh, dh_last, dx, dg, dh_init, shape, flags, workspace,
                                                 workspace_bytes, stream);
}

}  // extern "C"
