// libssm2d: the gated linear recurrence h[t] = a[t] h[t - 1] + w[t] x[t]
// (include/ssm2d_block.h), forward and backward, for token rows and for
// channels-first maps.
//
// Memory-bound. A stretch of tokens maps a state h to P h + c, with P the
// product of its a's, so stretches are worked on at once and joined in a fixed
// order: a thread takes neighbouring tokens of its channels one after the other,
// threads are joined within a wave and over the workgroup's waves, workgroups
// through a small workspace. A workgroup holds a chunk of tokens in registers and
// needs each input once. The forward walks over all tokens of its channels, or
// where there are too few channels for that (the host's choice) chunks go to
// workgroups of their own, which hand the state on (Relay). The backward, which
// goes both ways, has a first launch that reads the inputs for P and c alone.
// It joins both ways: e[t] = dh[t] + a[t + 1] e[t + 1] is the same
// recurrence from the end, and what flows out of a stretch, f = a e, is P f' + c'.
// States are fp32 throughout, also in the backward, which computes them again.
//
// Packed sequences: a first token of a sequence does not see the one before. Its
// stretch has P = -0: a product with it stays -0 until another cut, and joins
// select instead of multiply there, so that no Inf or NaN of one sequence
// reaches another.
#pragma once

#include "block_common.h"

namespace ssm2d_impl {

struct RecParams {
    const void *x, *g, *dh;
    const float *h_init, *dh_last;
    const int *cu;
    void *h, *dx, *dg;
    float *h_last, *dh_init;
    float *P, *H, *F;              // backward, [batch][segment][channel]: a segment's product and sums, then what enters it
    unsigned long *parts;          // forward, from workgroup to workgroup
    unsigned *tickets, *enter;
    unsigned *gave_up;             // set by a workgroup that waited for all its polls
    int polls;
    long chains;                   // rows of maps, or tiles of channels, of the batch
    long T;                        // tokens
    long seg;                      // tokens of a segment
    int S;                         // segments
    long first;                    // the launch's first workgroup (a grid has less than 2^32 threads)
    int n, n_seq, tiles;
    long x_b, g_b, d_b, x_t, g_t, d_t;  // strides of batch and token (rows) or channel (maps)
    int rev;                       // rows: from the last token to the first
    int pass_on;                   // packed: empty sequences' states are to be written
};

constexpr float kCut = -0.0f;
template <bool PACKED>
__device__ __forceinline__ bool is_cut(float p)
{
    return PACKED && __float_as_uint(p) == 0x80000000u;
}
// Gates that grow (g > 0) may multiply to Inf where the state is 0 and stays 0,
// token by token: c is then what is left, not the NaN of Inf by 0. Products of
// gates, none of which is negative, are 0 where one of them is, not that NaN (where a
// gate is NaN, c has it). GROW: gates may; a sigmoid's do not (64 x 196 tokens of 768,
// bf16, backward: 28.4 us, 29.8 with what growing takes; decays, of inputs in the caches, forward 12.7 for
// 11.7 and backward 23.4 for 22.6; long rows and maps 0 to 3 %).
template <bool GROW>
__device__ __forceinline__ float state_after(float P, float c, float h)
{
    return GROW && h == 0.0f ? c : fmaf(P, h, c);
}
template <bool GROW>
__device__ __forceinline__ float no_nan(float P)
{
    return GROW ? fmaxf(P, 0.0f) : P;
}
// The stretch (P, c) after (p0, c0).
template <bool PACKED, bool GROW>
__device__ __forceinline__ void join(float p0, float c0, float &P, float &c)
{
    if (is_cut<PACKED>(P)) return;
    c = state_after<GROW>(P, c, c0);
    P = is_cut<PACKED>(p0) ? p0 : no_nan<GROW>(P * p0);
}
// The state after a stretch (P, c) entered with h.
template <bool PACKED, bool GROW>
__device__ __forceinline__ float pass(float P, float c, float h)
{
    return is_cut<PACKED>(P) ? c : state_after<GROW>(P, c, h);
}

// a and w of a gate; for bf16 the sigmoid's two sides share their exponential.
template <typename T, bool SIG>
__device__ __forceinline__ void gates(float g, float &a, float &w)
{
    if constexpr (SIG) {
        // of e = exp(-|g|): 1 / (1 + e) and e / (1 + e), neither a difference
        const float e = exp_for<T>(-fabsf(g)), r = inverse_for<T>(1.0f + e), s = e * r;
        a = g < 0.0f ? s : r, w = g < 0.0f ? r : s;
    } else {
        a = exp_for<T>(g), w = 1.0f;
    }
}

// A gate that leaves the state as it is, where x is 0: for tokens past the last.
template <typename T, bool SIG>
__device__ __forceinline__ float idle() { return SIG ? INFINITY : 0.0f; }

// ------------------------------------------------------------------ packed sequences

// Where a token stands: its sequence (-1: none), whether it is its first, and
// the next token at which that changes.
struct Place {
    int seq;
    bool first;
    long end, next;
};
__device__ __forceinline__ long in_tokens(const RecParams &p, long v) { return v < 0 ? 0 : (v > p.T ? p.T : v); }
__device__ __forceinline__ long cu_at(const RecParams &p, long i) { return in_tokens(p, p.cu[i]); }
// (by halves at each change: any contents end, and stay within the tokens)
template <typename F>
__device__ __forceinline__ Place locate_by(const RecParams &p, long t, F &&at)
{
    int lo = -1, hi = p.n_seq;  // at(lo) <= t < at(hi), as far as they ascend
    while (hi - lo > 1) {
        const int m = static_cast<int>((static_cast<unsigned>(lo) + static_cast<unsigned>(hi)) / 2);  // (as ints the sum may be beyond them)
        if (at(m) <= t) lo = m;
        else hi = m;
    }
    Place w{-1, false, -1, 0x7fffffffffffffffL};
    if (lo < 0) {
        w.next = at(0);
    } else {
        const long end = at(lo + 1);
        if (t < end) w = Place{lo, at(lo) == t, end, end};
    }
    return w;
}
__device__ __forceinline__ Place locate(const RecParams &p, long t)
{
    return locate_by(p, t, [&](int i) { return cu_at(p, i); });
}
// Of the workgroup's first token, by scalar loads (nothing writes the offsets
// meanwhile): vector loads would wait for all that were asked for before.
__device__ __forceinline__ Place locate_first(const RecParams &p, long t)
{
    const auto *cu = reinterpret_cast<const __attribute__((address_space(4))) int *>(reinterpret_cast<uintptr_t>(p.cu));
    return locate_by(p, t, [&](int i) { return in_tokens(p, cu[i]); });
}

// ------------------------------------------------------------------ from workgroup to workgroup

// A forward in segments of one chunk. Each workgroup puts down its segment's
// product and sum, and takes what enters it from those before it in its group of
// segments and from what enters the group, which the last segment of the group
// before puts down. So sums are taken in one order whatever comes first, the
// inputs are read once, and only groups wait for each other.
// Every wait ends: a channel's segments are taken by tickets in their order, so all
// that a workgroup waits for belongs to workgroups that run already; they put their
// products down before they wait, and the first of those that wait has all it
// needs. (A counter for each row of maps or tile of channels: all workgroups at one
// counter took 13 ns each, 175 us for the 71 below.) (196608 cells of 128 channels, float32: 71 us; 95 with a launch for the products,
// one that joins them and one for the states. 16698 packed tokens of 1024, bf16: 43, 69 so.)
// Words say for themselves that they are there: all bits set, a NaN that nothing
// else is put down as, they are not. No order between them is needed.
constexpr unsigned long kNotYet = ~0ul;
constexpr int kMostPolls = 1 << 22;  // (seconds, before it goes on with a NaN rather than never, and says so)

__device__ __forceinline__ void put_down(unsigned long *to, float P, float c)
{
    unsigned long w = static_cast<unsigned long>(__float_as_uint(P)) << 32 | __float_as_uint(c);
    if (w == kNotYet) w = 0x7fc000007fc00000ul;
    __hip_atomic_store(to, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void put_down(unsigned *to, float h)
{
    const unsigned w = __float_as_uint(h);
    __hip_atomic_store(to, w == ~0u ? 0x7fc00000u : w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Waits for the first `count` of V words. (Polls first, so that no path leaves w
// unset: asked for the bound first, packed bf16 rows spill 11 registers, 50 us for the 43 above.)
template <int V, typename W>
__device__ __forceinline__ void take_up(const RecParams &p, const W *from, long step, int count, W (&w)[V])
{
    int polls = 0;
    do {
        bool there = true;
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] = __hip_atomic_load(from + min(j, count - 1) * step, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int j = 0; j < V; ++j) there = there && w[j] != static_cast<W>(kNotYet);
        if (there) return;
        __builtin_amdgcn_s_sleep(2);
    } while (++polls < p.polls);
    __hip_atomic_store(p.gave_up, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The workgroup's segment of a row of maps or tile of channels.
constexpr int kTicketWords = 32;  // from counter to counter, a line of their own
__device__ __forceinline__ int draw_ticket(const RecParams &p, long chain)
{
    __shared__ unsigned drawn;
    if (threadIdx.x == 0) drawn = __hip_atomic_fetch_add(p.tickets + chain * kTicketWords, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(static_cast<int>(drawn));
}

// ------------------------------------------------------------------ token rows

// How a workgroup holds token rows: 16 lanes of 8 bytes (128-byte runs; single channels
// by 32 lanes, where there are fewer or rows are far apart) by 16 lots of 8 tokens, WIDE 32,
// where a workgroup has one chunk. (Relays of 16384 x 1024, bf16: 35 us; lots of 4
// tokens, more workgroups that each wait: 60, when those of 8 took 49.)
template <typename T, int V, bool WIDE>
struct RowDims {
    static constexpr int kBX = V > 1 ? 16 : 32, kBY = (WIDE ? 512 : 256) / kBX, kThreads = kBX * kBY, kWaves = kThreads / 64;
    static constexpr int kL = 8, kChunk = kBY * kL;
};

template <typename T>
constexpr int kRowV = 8 / static_cast<int>(sizeof(T));  // channels a lane holds

// Where a thread's tokens of a chunk lie in a tensor: token `k` of the chunk, in
// the order of the recurrence, at base + offset. Offsets are 32 bits where
// channels are read together (the host sees to it that a chunk spans less).
template <int V>
struct Line {
    using Offset = std::conditional_t<V == 1, unsigned long, unsigned>;
    long base;            // elements from the tensor's start, the same for the workgroup
    Offset first, step;   // of token `lot` of the chunk (or the last there is), and to the next one
    // tokens t1 .. t1 + last; the thread's first is `lot`
    __device__ __forceinline__ void begin(const RecParams &p, long batch, long stride, long t1, int last, int lot, int channel)
    {
        base = batch + (p.rev ? p.T - 1 - t1 - last : t1) * stride;
        const int k = min(lot, last);
        first = static_cast<Offset>(p.rev ? last - k : k) * static_cast<Offset>(stride) + channel;
        step = p.rev ? -static_cast<Offset>(stride) : static_cast<Offset>(stride);
    }
};

// Joins the threads' stretches (P, c) of a workgroup in token order. lots_up: within
// the waves, whose totals go to `tot`; eP, ec: what is before a thread's in its wave.
// lots_in: `in` gets the state before each thread's stretch given `carry` before
// the workgroup's, and carry (with carryP, the product so far) moves to its end. DOWN:
// in reverse token order. tot: LDS for this use alone until the next barrier but one.
template <int V, int BX, bool PACKED, bool GROW, bool DOWN>
__device__ __forceinline__ void lots_up(float (&P)[V], float (&c)[V], float (&eP)[V], float (&ec)[V], float (*tot)[BX * V][2])
{
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, cx = lane % BX, sub = lane / BX;
    constexpr int kSubs = 64 / BX;
#pragma unroll
    for (int d = 1; d < kSubs; d *= 2)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float p0 = DOWN ? __shfl_down(P[j], d * BX) : __shfl_up(P[j], d * BX);
            const float c0 = DOWN ? __shfl_down(c[j], d * BX) : __shfl_up(c[j], d * BX);
            if (DOWN ? sub + d < kSubs : sub >= d) join<PACKED, GROW>(p0, c0, P[j], c[j]);
        }
    if (sub == (DOWN ? 0 : kSubs - 1)) {
#pragma unroll
        for (int j = 0; j < V; ++j) tot[wave][cx * V + j][0] = P[j], tot[wave][cx * V + j][1] = c[j];
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        eP[j] = DOWN ? __shfl_down(P[j], BX) : __shfl_up(P[j], BX);
        ec[j] = DOWN ? __shfl_down(c[j], BX) : __shfl_up(c[j], BX);
    }
    __syncthreads();
}
template <int V, int BX, int WAVES, bool PACKED, bool GROW, bool DOWN>
__device__ __forceinline__ void lots_in(const float (&eP)[V], const float (&ec)[V], float (&carry)[V], float (&carryP)[V], float (&in)[V],
                                        const float (*tot)[BX * V][2])
{
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, cx = lane % BX, sub = lane / BX;
    constexpr int kSubs = 64 / BX;
    // (two waves at a time: all at once would take the registers of the lots)
    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = carry[j];
#pragma unroll 2
    for (int i = 0; i < WAVES; ++i) {
        const int w = DOWN ? WAVES - 1 - i : i;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float wP = tot[w][cx * V + j][0], wc = tot[w][cx * V + j][1];
            if (w == wave) in[j] = h[j];
            h[j] = pass<PACKED, GROW>(wP, wc, h[j]);
            float p = wP, q = 0.0f;
            join<PACKED, GROW>(carryP[j], 0.0f, p, q);
            carryP[j] = p;
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        carry[j] = h[j];
        if (sub != (DOWN ? kSubs - 1 : 0)) in[j] = pass<PACKED, GROW>(eP[j], ec[j], in[j]);
    }
}
template <int V, int BX, int WAVES, bool PACKED, bool GROW, bool DOWN>
__device__ __forceinline__ void join_lots(float (&P)[V], float (&c)[V], float (&carry)[V], float (&carryP)[V], float (&in)[V],
                                          float (*tot)[BX * V][2])
{
    float eP[V], ec[V];
    lots_up<V, BX, PACKED, GROW, DOWN>(P, c, eP, ec, tot);
    lots_in<V, BX, WAVES, PACKED, GROW, DOWN>(eP, ec, carry, carryP, in, tot);
}

// Which of a thread's L tokens from t on are the first or the last of a packed
// sequence, and which are in none.
template <int L>
struct Marks {
    unsigned firsts, ends, outs;
    // t0: the workgroup's first token, of `chunk`
    __device__ __forceinline__ void find(const RecParams &p, long t0, int chunk, long t)
    {
        firsts = ends = outs = 0;
        Place w = locate_first(p, t0);
        if (w.seq >= 0 && !w.first && w.end > t0 + chunk) return;  // (most: inside one sequence)
        w = locate(p, t);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (i > 0) {
                if (t + i >= w.next) w = locate(p, t + i);
                else w.first = false;
            }
            firsts |= (w.seq >= 0 && w.first ? 1u : 0u) << i;
            ends |= (w.seq >= 0 && t + i + 1 == w.end ? 1u : 0u) << i;
            outs |= (w.seq < 0 ? 1u : 0u) << i;
        }
    }
    __device__ __forceinline__ bool first(int i) const { return (firsts >> i) & 1u; }
    __device__ __forceinline__ bool end(int i) const { return (ends >> i) & 1u; }
    __device__ __forceinline__ bool none(int i) const { return (outs >> i) & 1u; }
    __device__ __forceinline__ bool any() const { return (firsts | ends | outs) != 0; }
};
// A state of the sequence that token t belongs to (NULL: zeros). (Where offsets are out
// of order a token may be marked by the look-up of one before it, and itself be in none.)
__device__ __forceinline__ float state_at(const RecParams &p, const float *state, long t, long c)
{
    if (!state) return 0.0f;
    const long s = locate(p, t).seq;
    return s >= 0 ? state[s * p.n + c] : 0.0f;
}

// A few tokens (serving: one): a thread walks over them all for V channels (the
// last one of a row for those that are left: the state may be written in place,
// so that no two threads may share one).
template <typename T, int V, bool SIG>
__global__ __launch_bounds__(256) void rec_few(const RecParams p, long threads)
{
    const long id = (p.first + blockIdx.x) * 256 + threadIdx.x;
    if (id >= threads) return;
    const long b = id / p.tiles;
    const int c = static_cast<int>(id % p.tiles) * V, left = min(p.n - c, V);
    const T *x = static_cast<const T *>(p.x) + b * p.x_b + c, *g = static_cast<const T *>(p.g) + b * p.g_b + c;
    T *out = static_cast<T *>(p.h) + b * p.T * p.n + c;
    const long at = b * p.n + c;
    float h[V];
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = p.h_init && j < left ? p.h_init[at + j] : 0.0f;
    for (long i = 0; i < p.T; ++i) {
        const long t = p.rev ? p.T - 1 - i : i;
        Raw<T, V> vx, vg, o;
        if (left == V) {
            vx.load_any(x + t * p.x_t);
            vg.load_any(g + t * p.g_t);
        } else {
            float fx[V], fg[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                fx[j] = j < left ? widen1(x[t * p.x_t + j]) : 0.0f;
                fg[j] = j < left ? widen1(g[t * p.g_t + j]) : 0.0f;
            }
            vx.set(fx);
            vg.set(fg);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float a, w;
            gates<T, SIG>(vg.get(j), a, w);
            h[j] = fmaf(a, h[j], SIG ? w * vx.get(j) : vx.get(j));
        }
        if (left == V) {
            o.set(h);
            o.store_any(out + t * p.n);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < left) store1(out + t * p.n + j, h[j]);
        }
    }
    if (!p.h_last) return;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j < left) p.h_last[at + j] = h[j];
}

// Sequences without tokens pass their state on (NULL: zeros): for V channels, a
// share of the sequences each.
template <int V>
__device__ __forceinline__ void pass_on(const RecParams &p, const float *src, float *dst, int c, int first, int step)
{
    for (long s = first; s < p.n_seq; s += step) {
        if (cu_at(p, s + 1) > cu_at(p, s)) continue;
        const long at = s * p.n + c;
#pragma unroll
        for (int j = 0; j < V; ++j) dst[at + j] = src ? src[at + j] : 0.0f;
    }
}

// RELAY: a segment a workgroup, of one chunk. Otherwise all tokens.
template <typename T, int V, bool PACKED, bool SIG, bool RELAY>
__global__ __launch_bounds__(RELAY ? 512 : 256, 4) void rec_rows_fwd(const RecParams p)
{
    using D = RowDims<T, V, RELAY>;
    constexpr bool GROW = !SIG;
    __shared__ float tot[2][D::kWaves][D::kBX * V][2];
    const int cx = threadIdx.x % D::kBX, ty = threadIdx.x / D::kBX;
    const long id = p.first + blockIdx.x, chain = RELAY ? id % p.chains : id, b = chain / p.tiles;
    const int tile = static_cast<int>(chain % p.tiles), seg = RELAY ? draw_ticket(p, chain) : 0;
    const int c0 = (tile * D::kBX + cx) * V;
    const bool live = c0 < p.n;
    // (the last lane of a row reaches back over the one before: both get the same values)
    const int c = min(c0, p.n - V);
    const T *x = static_cast<const T *>(p.x), *g = static_cast<const T *>(p.g);
    T *h_out = static_cast<T *>(p.h);
    const long t1 = static_cast<long>(seg) * p.seg, t2 = min(t1 + p.seg, p.T);
    float carry[V], carryP[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        carryP[j] = 1.0f, carry[j] = 0.0f;
        if (!RELAY && !PACKED && p.h_init) carry[j] = p.h_init[b * p.n + c + j];
    }
    if (PACKED && p.pass_on && live) pass_on<V>(p, p.h_init, p.h_last, c, seg * D::kBY + ty, p.S * D::kBY);
    int buf = 0;
    for (long t0 = t1; t0 < t2; t0 += D::kChunk, buf ^= 1) {
        const long mine = t0 + ty * D::kL;
        const int last = static_cast<int>(min(t2 - t0, static_cast<long>(D::kChunk))) - 1, cnt = min(last + 1 - ty * D::kL, D::kL);
        Raw<T, V> rx[D::kL], rg[D::kL];
        Line<V> lx, lg, lo;
        lx.begin(p, b * p.x_b, p.x_t, t0, last, ty * D::kL, c);
        lg.begin(p, b * p.g_b, p.g_t, t0, last, ty * D::kL, c);
        lo.begin(p, b * p.T * p.n, p.n, t0, last, ty * D::kL, c);
#pragma unroll
        for (int i = 0; i < D::kL; ++i) {  // (tokens past the segment read its last, and are not used)
            rx[i].load_any(x + lx.base + lx.first);
            rg[i].load_any(g + lg.base + lg.first);
            if (i + 1 < cnt) lx.first += lx.step, lg.first += lg.step;
        }
        Marks<D::kL> marks;
        if constexpr (PACKED) marks.find(p, t0, D::kChunk, mine);
        // what each token does to the state: h = a h + wx (a first one of a sequence: h = wx)
        float a[D::kL][V], wx[D::kL][V], P[V], h[V], in[V], eP[V], ec[V];
#pragma unroll
        for (int j = 0; j < V; ++j) P[j] = 1.0f, h[j] = 0.0f;
        // (whole lots inside one sequence, which are most, go without a branch)
        const bool whole = cnt == D::kL && !(PACKED && marks.any());
#pragma unroll
        for (int i = 0; i < D::kL; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float w;
                gates<T, SIG>(rg[i].get(j), a[i][j], w);
                wx[i][j] = SIG ? w * rx[i].get(j) : rx[i].get(j);
            }
        if (whole) {
#pragma unroll
            for (int i = 0; i < D::kL; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) P[j] *= a[i][j], h[j] = fmaf(a[i][j], h[j], wx[i][j]);
#pragma unroll
            for (int j = 0; j < V; ++j) P[j] = no_nan<GROW>(P[j]);
        } else {
#pragma unroll
            for (int i = 0; i < D::kL; ++i) {
                if (i >= cnt) continue;
                const bool cut = PACKED && (marks.first(i) || marks.none(i));
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (cut) {
                        if (marks.none(i)) wx[i][j] = 0.0f;
                        else wx[i][j] = fmaf(a[i][j], state_at(p, p.h_init, mine + i, c + j), wx[i][j]);
                        P[j] = kCut, h[j] = wx[i][j];
                    } else {
                        if (!is_cut<PACKED>(P[j])) P[j] = no_nan<GROW>(P[j] * a[i][j]);
                        h[j] = fmaf(a[i][j], h[j], wx[i][j]);
                    }
                }
            }
        }
        lots_up<V, D::kBX, PACKED, GROW, false>(P, h, eP, ec, tot[buf]);
        if constexpr (RELAY) {
            // A lane a channel here, so that words are asked for in whole lines and few
            // registers are held beside the tokens' (lanes of V channels, 4 times the
            // requests past the caches, and spills: 71 us for those 43).
            constexpr int C = D::kBX * V, kShares = D::kThreads / C, kGroup = 4 * kShares;  // segments of a group
            __shared__ float before[kShares][C][2], into[D::kWaves][C];
            const int l = threadIdx.x % C, share = threadIdx.x / C, first = (tile * D::kBX + l / V) * V;
            const bool here = first < p.n;
            const int ch = min(first, p.n - V) + l % V;
            const int k = seg % kGroup, group = seg / kGroup, groups = (p.S + kGroup - 1) / kGroup;
            unsigned *enter = p.enter + (b * groups + group) * p.n + ch;
            float q = 1.0f, d = 0.0f;
            auto also = [&](const float(&w)[2]) __attribute__((always_inline)) {
                float P1 = w[0], c1 = w[1];
                join<PACKED, GROW>(q, d, P1, c1);
                q = P1, d = c1;
            };
            if (share == 0 && here && seg + 1 < p.S) {
                for (int w = 0; w < D::kWaves; ++w) also(tot[buf][w][l]);
                put_down(p.parts + (b * p.S + seg) * p.n + ch, q, d);
                q = 1.0f, d = 0.0f;
            }
            if (here && share * 4 < k) {
                unsigned long w[4];
                take_up<4>(p, p.parts + (b * p.S + seg - k + share * 4) * p.n + ch, static_cast<long>(p.n), min(k - share * 4, 4), w);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (share * 4 + i < k) also({__uint_as_float(static_cast<unsigned>(w[i] >> 32)), __uint_as_float(static_cast<unsigned>(w[i]))});
            }
            before[share][l][0] = q, before[share][l][1] = d;
            unsigned w[1] = {0u};
            if (share == 0 && here) {
                if (group > 0) take_up<1>(p, enter, 0, 1, w);
                else if (!PACKED && p.h_init) w[0] = __float_as_uint(p.h_init[b * p.n + ch]);
            }
            __syncthreads();
            if (share == 0 && here) {
                float state = __uint_as_float(w[0]);
                for (int i = 0; i * 4 < k; ++i) state = pass<PACKED, GROW>(before[i][l][0], before[i][l][1], state);
                for (int i = 0; i < D::kWaves; ++i) {
                    into[i][l] = state;
                    state = pass<PACKED, GROW>(tot[buf][i][l][0], tot[buf][i][l][1], state);
                }
                if (k + 1 == kGroup && seg + 1 < p.S) put_down(enter + p.n, state);
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < V; ++j) {
                in[j] = into[threadIdx.x / 64][cx * V + j];
                if (threadIdx.x % 64 >= D::kBX) in[j] = pass<PACKED, GROW>(eP[j], ec[j], in[j]);
            }
        } else {
            lots_in<V, D::kBX, D::kWaves, PACKED, GROW, false>(eP, ec, carry, carryP, in, tot[buf]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = in[j];
        auto put = [&](int i) __attribute__((always_inline)) {
            Raw<T, V> v;
            v.set(h);
            v.store_any(h_out + lo.base + (lo.first + i * lo.step));
        };
        auto keep = [&](long s) __attribute__((always_inline)) {
            if (PACKED && s < 0) return;  // (as in state_at)
#pragma unroll
            for (int j = 0; j < V; ++j) p.h_last[s * p.n + c + j] = h[j];
        };
        if (whole) {
#pragma unroll
            for (int i = 0; i < D::kL; ++i) {
#pragma unroll
                for (int j = 0; j < V; ++j) h[j] = fmaf(a[i][j], h[j], wx[i][j]);
                if (live) put(i);
            }
            if (!PACKED && p.h_last && live && mine + D::kL == p.T) keep(b);
        } else {
#pragma unroll
            for (int i = 0; i < D::kL; ++i) {
                if (i >= cnt) continue;
                const bool cut = PACKED && (marks.first(i) || marks.none(i));
#pragma unroll
                for (int j = 0; j < V; ++j) h[j] = cut ? wx[i][j] : fmaf(a[i][j], h[j], wx[i][j]);
                if (!live || (PACKED && marks.none(i))) continue;
                put(i);
                if (p.h_last && (PACKED ? marks.end(i) : mine + i + 1 == p.T)) keep(PACKED ? locate(p, mine + i).seq : b);
            }
        }
    }
}

// A workgroup's chunk is a segment. AGG: its product, state from zero and flow from zero, into P, H and F.
// (64 x 196 tokens of 768, bf16: 28 us, 3.4 TB/s, 64 x 256 4.0; bound by what two workgroups a
// compute unit, as many as the registers allow, ask for, and by the gates' exponentials.)
template <typename T, int V, bool PACKED, bool SIG, bool AGG>
__global__ __launch_bounds__(512, 4) void rec_rows_bwd(const RecParams p)
{
    using D = RowDims<T, V, true>;
    constexpr int L = D::kL;
    constexpr bool GROW = !SIG;
    __shared__ float tot[2][D::kWaves][D::kBX * V][2];
    const int cx = threadIdx.x % D::kBX, ty = threadIdx.x / D::kBX;
    const int tile = static_cast<int>((p.first + blockIdx.x) % p.tiles);
    const long rest = (p.first + blockIdx.x) / p.tiles;
    const int seg = static_cast<int>(rest % p.S);
    const long b = rest / p.S;
    const int c0 = (tile * D::kBX + cx) * V;
    const bool live = c0 < p.n;
    // (the last lane of a row reaches back over the one before: both get the same values)
    const int c = min(c0, p.n - V);
    const T *x = static_cast<const T *>(p.x), *g = static_cast<const T *>(p.g), *d = static_cast<const T *>(p.dh);
    const long t1 = static_cast<long>(seg) * p.seg, t2 = min(t1 + p.seg, p.T);
    const long place = (b * p.S + seg) * p.n + c;
    const long mine = t1 + ty * L;
    const int last = static_cast<int>(t2 - t1) - 1, cnt = min(last + 1 - ty * L, L);
    Raw<T, V> rx[L], rg[L], rd[L];
    Line<V> lx, lg, ld, lo;
    lx.begin(p, b * p.x_b, p.x_t, t1, last, ty * L, c);
    lg.begin(p, b * p.g_b, p.g_t, t1, last, ty * L, c);
    ld.begin(p, b * p.d_b, p.d_t, t1, last, ty * L, c);
    lo.begin(p, b * p.T * p.n, p.n, t1, last, ty * L, c);
#pragma unroll
    for (int i = 0; i < L; ++i) {
        rx[i].load_any(x + lx.base + lx.first);
        rg[i].load_any(g + lg.base + lg.first);
        rd[i].load_any(d + ld.base + ld.first);
        if (i + 1 < cnt) lx.first += lx.step, lg.first += lg.step, ld.first += ld.step;
    }
    if (PACKED && !AGG && p.pass_on && live) pass_on<V>(p, p.dh_last, p.dh_init, c, seg * D::kBY + ty, p.S * D::kBY);
    float enter[V], flow[V], one[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        enter[j] = flow[j] = 0.0f;
        if (AGG) continue;
        if (p.S > 1) {
            enter[j] = p.H[place + j], flow[j] = p.F[place + j];
        } else if (!PACKED) {
            if (p.h_init) enter[j] = p.h_init[b * p.n + c + j];
            if (p.dh_last) flow[j] = p.dh_last[b * p.n + c + j];
        }
    }
    Marks<L> marks;
    if constexpr (PACKED) marks.find(p, t1, D::kChunk, mine);
    const bool whole = cnt == L && !(PACKED && marks.any());
    // the thread's stretch, forward and (f) backward; CUT: with what a lot that is not whole has to look at
    float P[V], h[V], f[V], in[V];
#pragma unroll
    for (int j = 0; j < V; ++j) P[j] = 1.0f, h[j] = 0.0f, f[j] = 0.0f;
    auto stretch = [&](auto cut) __attribute__((always_inline)) {
        constexpr bool CUT = decltype(cut)::value;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (CUT && i >= cnt) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float a, w;
                gates<T, SIG>(rg[i].get(j), a, w);
                const float wx = SIG ? w * rx[i].get(j) : rx[i].get(j);
                if (PACKED && CUT && (marks.first(i) || marks.none(i))) {
                    h[j] = marks.none(i) ? 0.0f : fmaf(a, state_at(p, p.h_init, mine + i, c + j), wx);
                    P[j] = kCut;
                } else {
                    h[j] = fmaf(a, h[j], wx);
                    if (!(CUT && is_cut<PACKED>(P[j]))) P[j] = no_nan<GROW>(P[j] * a);
                }
            }
        }
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            if (CUT && i >= cnt) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float a, w;
                gates<T, SIG>(rg[i].get(j), a, w);
                const float after = PACKED && CUT && marks.end(i) ? state_at(p, p.dh_last, mine + i, c + j) : f[j];
                f[j] = PACKED && CUT && (marks.first(i) || marks.none(i)) ? 0.0f : a * (rd[i].get(j) + after);
            }
        }
    };
    if (whole) stretch(std::false_type{});
    else stretch(std::true_type{});
    float P2[V], out[V];
#pragma unroll
    for (int j = 0; j < V; ++j) P2[j] = P[j], one[j] = 1.0f;
    join_lots<V, D::kBX, D::kWaves, PACKED, GROW, false>(P, h, enter, one, in, tot[0]);
    if (AGG && live && ty == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) p.P[place + j] = one[j], p.H[place + j] = enter[j];
    }
    join_lots<V, D::kBX, D::kWaves, PACKED, GROW, true>(P2, f, flow, one, out, tot[1]);
    if (AGG) {
        if (live && ty == 0) {
#pragma unroll
            for (int j = 0; j < V; ++j) p.F[place + j] = flow[j];
        }
        return;
    }
    if (!live) return;
#pragma unroll
    for (int i = 0; i < L; ++i) rg[i].forget(), rx[i].forget(), rd[i].forget();
    auto finish = [&](auto cut) __attribute__((always_inline)) {
        constexpr bool CUT = decltype(cut)::value;
        // what e is to be multiplied by for dg, of each token
        float q[L][V];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (CUT && i >= cnt) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float a, w;
                gates<T, SIG>(rg[i].get(j), a, w);
                const float xv = rx[i].get(j), before = PACKED && CUT && marks.first(i) ? state_at(p, p.h_init, mine + i, c + j) : in[j];
                q[i][j] = SIG ? a * w * (before - xv) : a * before;
                in[j] = fmaf(a, before, SIG ? w * xv : xv);
            }
        }
#pragma unroll
        for (int i = 0; i < L; ++i) rg[i].forget();
#pragma unroll
        for (int i = L - 1; i >= 0; --i) {
            if (CUT && i >= cnt) continue;
            float dx[V], dg[V], fl[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float a, w;
                gates<T, SIG>(rg[i].get(j), a, w);
                const float e = rd[i].get(j) + (PACKED && CUT && marks.end(i) ? state_at(p, p.dh_last, mine + i, c + j) : out[j]);
                dx[j] = SIG ? w * e : e;
                dg[j] = q[i][j] * e;
                fl[j] = a * e;
                out[j] = PACKED && CUT && (marks.first(i) || marks.none(i)) ? 0.0f : fl[j];
            }
            if (PACKED && CUT && marks.none(i)) continue;
            const auto at = lo.first + i * lo.step;
            Raw<T, V> v;
            v.set(dx);
            v.store_any(static_cast<T *>(p.dx) + lo.base + at);
            v.set(dg);
            v.store_any(static_cast<T *>(p.dg) + lo.base + at);
            if ((PACKED ? CUT : i == 0) && p.dh_init && (PACKED ? marks.first(i) : mine == 0)) {
                const long s = PACKED ? locate(p, mine + i).seq : b;  // (a first token is marked by its own look-up)
#pragma unroll
                for (int j = 0; j < V; ++j) p.dh_init[s * p.n + c + j] = fl[j];
            }
        }
    };
    if (whole) finish(std::false_type{});
    else finish(std::true_type{});
}

// ------------------------------------------------------------------ maps

template <typename T>
constexpr int kMapV = 16 / static_cast<int>(sizeof(T));  // tokens of a vector
// How a row of cells is held: LPR lanes (16 .. 256: four waves) with U vectors each.
template <int LPR_, int U_>
struct MapDims {
    static constexpr int kLpr = LPR_, kU = U_, kWaves = LPR_ > 64 ? LPR_ / 64 : 1, kWidth = LPR_ > 64 ? 64 : LPR_, kRows = 256 / LPR_;
    template <typename T>
    static constexpr int kChunk = LPR_ * kMapV<T> * U_;
};

// Inclusive join over aligned groups of W lanes.
template <int W, bool GROW>
__device__ __forceinline__ void wave_join(float &P, float &c)
{
    auto step = [&](auto ctrl, auto rows) __attribute__((always_inline)) {
        constexpr int kCtrl = decltype(ctrl)::value, kRowMask = decltype(rows)::value;
        const float p0 = __int_as_float(__builtin_amdgcn_update_dpp(0x3f800000, __float_as_int(P), kCtrl, kRowMask, 0xf, false));
        const float c0 = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(c), kCtrl, kRowMask, 0xf, false));
        c = state_after<GROW>(P, c, c0);
        P = no_nan<GROW>(P * p0);
    };
    using std::integral_constant;
    step(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});  // row_shr:1, 2, 4, 8
    step(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});
    step(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});
    step(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});
    // the rows' last lanes to the next row, and to the second half
    if constexpr (W > 16) step(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});
    if constexpr (W > 32) step(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});
}
// The value of the lane before, `none` for the first of a group.
template <int W>
__device__ __forceinline__ float lane_before(float v, float none)
{
    constexpr int kCtrl = W == 16 ? 0x111 : 0x138;  // row_shr:1, wave_shr:1
    const float r = __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(none), __float_as_int(v), kCtrl, 0xf, 0xf, false));
    return W == 32 && threadIdx.x % 32 == 0 ? none : r;
}
template <int W>
__device__ __forceinline__ float last_lane(float v)
{
    if constexpr (W == 64) return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
    else return __shfl(v, W - 1, W);
}

// The product and sum of U stretches of each lane of a group (in token order: all
// lanes' first, then all lanes' second); P, c become the joined ones up to each lane.
template <int W, bool GROW, int U>
__device__ __forceinline__ void wave_total(float (&P)[U], float (&c)[U], float &wP, float &wc)
{
    wP = 1.0f, wc = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        wave_join<W, GROW>(P[u], c[u]);
        const float lP = last_lane<W>(P[u]), lc = last_lane<W>(c[u]);
        wc = state_after<GROW>(lP, lc, wc);
        wP = no_nan<GROW>(wP * lP);
    }
}
// The states before each of a lane's stretches given h before the group's.
template <int W, bool GROW, int U>
__device__ __forceinline__ void wave_states(const float (&P)[U], const float (&c)[U], float h, float (&in)[U])
{
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const float eP = lane_before<W>(P[u], 1.0f), ec = lane_before<W>(c[u], 0.0f);
        in[u] = state_after<GROW>(eP, ec, h);
        h = state_after<GROW>(last_lane<W>(P[u]), last_lane<W>(c[u]), h);
    }
}

// V tokens from place i in the order of the recurrence, at any alignment; `fill`
// past the last of the row's n.
template <typename T, int V, bool REV>
struct Run {
    Raw<T, V> r;
    __device__ __forceinline__ void load(const T *row, long i, long n, float fill)
    {
        if (i + V <= n) {
            r.load_any(row + (REV ? n - V - i : i));
            return;
        }
        float f[V];
#pragma unroll
        for (int j = 0; j < V; ++j) f[REV ? V - 1 - j : j] = i + j < n ? widen1(row[REV ? n - 1 - i - j : i + j]) : fill;
        r.set(f);
    }
    __device__ __forceinline__ float get(int j) const { return r.get(REV ? V - 1 - j : j); }
    __device__ __forceinline__ void forget() { r.forget(); }
};
template <typename T, int V, bool REV>
__device__ __forceinline__ void store_run(T *row, long i, long n, const float (&v)[V])
{
    if (i + V > n) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (i + j < n) store1(row + (REV ? n - 1 - i - j : i + j), v[j]);
        return;
    }
    float o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = v[REV ? V - 1 - j : j];
    Raw<T, V> r;
    r.set(o);
    r.store_any(row + (REV ? n - V - i : i));
}

// Over the workgroup's WPR waves of one row: the state before this wave given
// `carry` before the first; carry and its product move to the end. Every wave
// of the workgroup calls it. DOWN: from the last wave to the first.
template <int WPR, bool GROW, bool DOWN>
__device__ __forceinline__ float join_waves(float wP, float wc, float &carry, float &carryP, float (*tot)[2])
{
    float in = carry;
    if constexpr (WPR > 1) {
        const int wave = threadIdx.x / 64;
        if (threadIdx.x % 64 == 0) tot[wave][0] = wP, tot[wave][1] = wc;
        __syncthreads();
        float h = carry;
#pragma unroll
        for (int i = 0; i < WPR; ++i) {
            const int w = DOWN ? WPR - 1 - i : i;
            if (w == wave) in = h;
            h = state_after<GROW>(tot[w][0], tot[w][1], h);
            carryP = no_nan<GROW>(carryP * tot[w][0]);
        }
        carry = h;
    } else {
        carry = state_after<GROW>(wP, wc, carry);
        carryP = no_nan<GROW>(carryP * wP);
    }
    return in;
}

// RELAY: a segment a workgroup, of one chunk. Otherwise all tokens.
template <typename T, typename DIMS, bool REV, bool SIG, bool RELAY>
__global__ __launch_bounds__(256) void rec_maps_fwd(const RecParams p, long units)
{
    constexpr bool GROW = !SIG;
    constexpr int V = kMapV<T>, U = DIMS::kU, W = DIMS::kWidth, kWaves = DIMS::kWaves, kChunk = DIMS::template kChunk<T>;
    __shared__ float tot[2][4][2];
    const int place_in = threadIdx.x % DIMS::kLpr, wave = place_in / 64, lane = place_in % 64;  // of the row
    const long unit = (p.first + blockIdx.x) * DIMS::kRows + threadIdx.x / DIMS::kLpr;
    // (rows past the last: whole waves or parts of them, and no barrier follows)
    if (DIMS::kRows > 1 && unit >= units) return;
    const long row = RELAY ? unit % p.chains : unit, b = row / p.n, c = row % p.n;
    const int seg = RELAY ? draw_ticket(p, row) : 0;
    const T *x = static_cast<const T *>(p.x) + b * p.x_b + c * p.x_t, *g = static_cast<const T *>(p.g) + b * p.g_b + c * p.g_t;
    T *h_out = static_cast<T *>(p.h) + row * p.T;
    const long t1 = static_cast<long>(seg) * p.seg, t2 = min(t1 + p.seg, p.T);
    float carry = !RELAY && p.h_init ? p.h_init[row] : 0.0f, carryP = 1.0f;
    int buf = 0;
    for (long t0 = t1; t0 < t2; t0 += kChunk, buf ^= 1) {
        Run<T, V, REV> rx[U], rg[U];
        float a[U][V], wx[U][V], P[U], h[U], in[U];
        auto at = [&](int u) { return t0 + (static_cast<long>(wave * U + u) * W + lane) * V; };
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // (segments end with whole chunks or with the row)
            rx[u].load(x, at(u), p.T, 0.0f);
            rg[u].load(g, at(u), p.T, idle<T, SIG>());
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            P[u] = 1.0f, h[u] = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float w;
                gates<T, SIG>(rg[u].get(j), a[u][j], w);
                wx[u][j] = SIG ? w * rx[u].get(j) : rx[u].get(j);
                h[u] = fmaf(a[u][j], h[u], wx[u][j]);
                P[u] *= a[u][j];
            }
            P[u] = no_nan<GROW>(P[u]);
        }
        float wP, wc;
        wave_total<W, GROW>(P, h, wP, wc);
        float enter;
        if constexpr (RELAY) {
            __shared__ float entering;
            constexpr int kGroup = 64;  // segments of a group: a lane each
            const int k = seg % kGroup, group = seg / kGroup, groups = (p.S + kGroup - 1) / kGroup;
            if (lane == 0) tot[0][wave][0] = wP, tot[0][wave][1] = wc;
            __syncthreads();
            if (wave == 0) {
                float sP = 1.0f, sc = 0.0f;
#pragma unroll
                for (int i = 0; i < kWaves; ++i) sc = state_after<GROW>(tot[0][i][0], tot[0][i][1], sc), sP = no_nan<GROW>(sP * tot[0][i][0]);
                if (lane == 0 && seg + 1 < p.S) put_down(p.parts + row * p.S + seg, sP, sc);
                float pP = 1.0f, pc = 0.0f;
                if (lane < k) {
                    unsigned long w[1];
                    take_up<1>(p, p.parts + row * p.S + seg - k + lane, 0, 1, w);
                    pP = __uint_as_float(static_cast<unsigned>(w[0] >> 32)), pc = __uint_as_float(static_cast<unsigned>(w[0]));
                }
                unsigned w[1] = {0u};
                if (group > 0) take_up<1>(p, p.enter + row * groups + group, 0, 1, w);
                else if (p.h_init) w[0] = __float_as_uint(p.h_init[row]);
                wave_join<64, GROW>(pP, pc);
                const float into = state_after<GROW>(last_lane<64>(pP), last_lane<64>(pc), __uint_as_float(w[0]));
                if (lane == 0) {
                    entering = into;
                    if (k + 1 == kGroup && seg + 1 < p.S) put_down(p.enter + row * groups + group + 1, state_after<GROW>(sP, sc, into));
                }
            }
            __syncthreads();
            enter = entering;
#pragma unroll
            for (int i = 0; i < kWaves; ++i)
                if (i < wave) enter = state_after<GROW>(tot[0][i][0], tot[0][i][1], enter);
        } else {
            enter = join_waves<kWaves, GROW, false>(wP, wc, carry, carryP, tot[buf]);
        }
        wave_states<W, GROW>(P, h, enter, in);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float o[V], v = in[u];
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] = v = fmaf(a[u][j], v, wx[u][j]);
            store_run<T, V, REV>(h_out, at(u), p.T, o);
            if (p.h_last && at(u) < p.T && at(u) + V >= p.T) p.h_last[row] = v;  // (past the last token it stays)
        }
    }
}

template <typename T, typename DIMS, bool REV, bool SIG, bool AGG>
__global__ __launch_bounds__(256) void rec_maps_bwd(const RecParams p, long units)
{
    constexpr bool GROW = !SIG;
    constexpr int V = kMapV<T>, U = DIMS::kU, W = DIMS::kWidth, kWaves = DIMS::kWaves;
    __shared__ float tot[2][4][2];
    const int place_in = threadIdx.x % DIMS::kLpr, wave = place_in / 64, lane = place_in % 64;  // of the row
    const long unit = (p.first + blockIdx.x) * DIMS::kRows + threadIdx.x / DIMS::kLpr;
    // (rows past the last: whole waves or parts of them, and no barrier follows)
    if (DIMS::kRows > 1 && unit >= units) return;
    const int seg = static_cast<int>(unit % p.S);
    const long row = unit / p.S, b = row / p.n, c = row % p.n;
    const T *x = static_cast<const T *>(p.x) + b * p.x_b + c * p.x_t, *g = static_cast<const T *>(p.g) + b * p.g_b + c * p.g_t;
    const T *d = static_cast<const T *>(p.dh) + b * p.d_b + c * p.d_t;
    const long t1 = static_cast<long>(seg) * p.seg, place = (b * p.S + seg) * p.n + c;
    auto at = [&](int u) { return t1 + (static_cast<long>(wave * U + u) * W + lane) * V; };
    Run<T, V, REV> rx[U], rg[U], rd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        rx[u].load(x, at(u), p.T, 0.0f);
        rg[u].load(g, at(u), p.T, idle<T, SIG>());
        rd[u].load(d, at(u), p.T, 0.0f);
    }
    float enter = 0.0f, flow = 0.0f, product = 1.0f, unused = 1.0f;
    if (!AGG) {
        if (p.S > 1) enter = p.H[place], flow = p.F[place];
        else enter = p.h_init ? p.h_init[row] : 0.0f, flow = p.dh_last ? p.dh_last[row] : 0.0f;
    }
    // each lane's stretches, forward, and backward with the lanes and stretches mirrored
    float P[U], h[U], Q[U], f[U], in[U], out[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        P[u] = 1.0f, h[u] = 0.0f, f[u] = 0.0f;
        float a[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float w;
            gates<T, SIG>(rg[u].get(j), a[j], w);
            h[u] = fmaf(a[j], h[u], SIG ? w * rx[u].get(j) : rx[u].get(j));
            P[u] *= a[j];
        }
        P[u] = no_nan<GROW>(P[u]);
#pragma unroll
        for (int j = V - 1; j >= 0; --j) f[u] = a[j] * (rd[u].get(j) + f[u]);
    }
    float G[U];
#pragma unroll
    for (int u = 0; u < U; ++u) Q[u] = __shfl(P[U - 1 - u], W - 1 - lane, W), G[u] = __shfl(f[U - 1 - u], W - 1 - lane, W);
    float wP, wc;
    wave_total<W, GROW>(P, h, wP, wc);
    const float enter_w = join_waves<kWaves, GROW, false>(wP, wc, enter, product, tot[0]);
    wave_total<W, GROW>(Q, G, wP, wc);
    const float flow_w = join_waves<kWaves, GROW, true>(wP, wc, flow, unused, tot[1]);
    if (AGG) {
        if (lane == 0 && wave == 0) p.P[place] = product, p.H[place] = enter, p.F[place] = flow;
        return;
    }
    wave_states<W, GROW>(P, h, enter_w, in);
    wave_states<W, GROW>(Q, G, flow_w, f);
#pragma unroll
    for (int u = 0; u < U; ++u) out[u] = __shfl(f[U - 1 - u], W - 1 - lane, W);
#pragma unroll
    for (int u = 0; u < U; ++u) rg[u].forget();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float a[V], w[V], q[V], dx[V], dg[V], v = in[u], e = out[u];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            gates<T, SIG>(rg[u].get(j), a[j], w[j]);
            const float xv = rx[u].get(j);
            q[j] = SIG ? a[j] * w[j] * (v - xv) : a[j] * v;
            v = fmaf(a[j], v, SIG ? w[j] * xv : xv);
        }
#pragma unroll
        for (int j = V - 1; j >= 0; --j) {
            e += rd[u].get(j);
            dx[j] = SIG ? w[j] * e : e;
            dg[j] = q[j] * e;
            e *= a[j];
        }
        store_run<T, V, REV>(static_cast<T *>(p.dx) + row * p.T, at(u), p.T, dx);
        store_run<T, V, REV>(static_cast<T *>(p.dg) + row * p.T, at(u), p.T, dg);
        if (p.dh_init && at(u) == 0) p.dh_init[row] = e;
    }
}

// ------------------------------------------------------------------ launches

// How a call is cut, and which kernels run it.
struct RecPlan {
    bool maps, packed, sig, rev;
    bool few;  // forward of few tokens: a thread walks over them
    int v;       // token rows: channels a lane holds
    long cells;  // maps: tokens of a row
};

template <typename F>
int rec_launch(RecParams p, long groups, int threads, F &&f)
{
    const long most = most_groups(threads);
    for (p.first = 0; p.first < groups; p.first += most) {
        f(p, dim3(static_cast<unsigned>(std::min(groups - p.first, most))));
        const int st = launched();
        if (st != SSM2D_OK) return st;
    }
    return SSM2D_OK;
}

// f(bool_constant...) for the values of some flags.
template <typename F>
int with_flags(F &&f)
{
    return f();
}
template <typename F, typename... B>
int with_flags(F &&f, bool first, B... rest)
{
    if (first) return with_flags([&](auto... r) { return f(std::true_type{}, r...); }, rest...);
    return with_flags([&](auto... r) { return f(std::false_type{}, r...); }, rest...);
}

// Calls f with how rows of so many cells are held: as few lanes as hold them, so
// that a wave has several short rows (64 maps of 768 channels, bf16, 14 x 14 cells: 22 us
// from 62 with a wave a row, 7 x 7: 10 from 56).
template <typename T, typename F>
auto with_map_dims(long cells, F &&f)
{
    if (cells <= MapDims<16, 1>::kChunk<T>) return f(MapDims<16, 1>{});
    if (cells <= MapDims<32, 1>::kChunk<T>) return f(MapDims<32, 1>{});
    if (cells <= MapDims<64, 1>::kChunk<T>) return f(MapDims<64, 1>{});
    if (cells <= MapDims<64, 2>::kChunk<T>) return f(MapDims<64, 2>{});
    return f(MapDims<256, 2>{});
}

template <typename T>
int rec_run_few(RecParams p, const RecPlan &plan, long batch, hipStream_t s)
{
    auto go = [&](auto vec) {
        constexpr int V = decltype(vec)::value;
        p.tiles = (p.n + V - 1) / V;
        const long threads = batch * p.tiles;
        return rec_launch(p, (threads + 255) / 256, 256, [&](const RecParams &q, dim3 grid) {
            if (plan.sig) rec_few<T, V, true><<<grid, dim3(256), 0, s>>>(q, threads);
            else rec_few<T, V, false><<<grid, dim3(256), 0, s>>>(q, threads);
        });
    };
    return plan.v > 1 ? go(std::integral_constant<int, kRowV<T>>{}) : go(std::integral_constant<int, 1>{});
}

template <typename T, bool BWD>
int rec_run(const RecParams &p, const RecPlan &plan, long batch, bool agg, hipStream_t s)
{
    if constexpr (!BWD) {
        if (plan.few) return rec_run_few<T>(p, plan, batch, s);
    }
    if (!plan.maps) {
        auto go = [&](auto vec) {
            constexpr int V = decltype(vec)::value;
            return with_flags(
                [&](auto packed, auto sig, auto only) {
                    constexpr bool K = decltype(packed)::value, G = decltype(sig)::value, A = decltype(only)::value;
                    constexpr int kThreads = RowDims<T, V, BWD || A>::kThreads;
                    return rec_launch(p, batch * p.S * p.tiles, kThreads, [&](const RecParams &q, dim3 grid) {
                        if constexpr (BWD) rec_rows_bwd<T, V, K, G, A><<<grid, dim3(kThreads), 0, s>>>(q);
                        else rec_rows_fwd<T, V, K, G, A><<<grid, dim3(kThreads), 0, s>>>(q);
                    });
                },
                plan.packed, plan.sig, agg);
        };
        return plan.v > 1 ? go(std::integral_constant<int, kRowV<T>>{}) : go(std::integral_constant<int, 1>{});
    }
    const long units = batch * p.n * p.S;
    return with_map_dims<T>(plan.cells, [&](auto dims) {
        using D = decltype(dims);
        return with_flags(
            [&](auto rev, auto sig, auto only) {
                constexpr bool R = decltype(rev)::value, G = decltype(sig)::value, A = decltype(only)::value;
                if constexpr (A && D::kWaves == 1) {  // (rows of a wave or less are one chunk)
                    return static_cast<int>(SSM2D_ERR_UNSUPPORTED);
                } else {
                    return rec_launch(p, (units + D::kRows - 1) / D::kRows, 256, [&](const RecParams &q, dim3 grid) {
                        if constexpr (BWD) rec_maps_bwd<T, D, R, G, A><<<grid, dim3(256), 0, s>>>(q, units);
                        else rec_maps_fwd<T, D, R, G, A><<<grid, dim3(256), 0, s>>>(q, units);
                    });
                }
            },
            plan.rev, plan.sig, agg);
    });
}

}  // namespace ssm2d_impl
