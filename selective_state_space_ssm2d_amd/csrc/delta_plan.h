// libssm2d: how the gated delta rule's sequences are cut: into chunks of 64
// tokens, chains of chunks into segments, heads into passes. Host and device
// agree on it here; packed sequences' lengths are known to the device alone.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstddef>

namespace ssm2d_impl {

constexpr int kC = 64;  // tokens a chunk

struct Cuts {
    const int *cu;
    long batch, tokens, n_seq, chunks_b;  // chunks_b: chunks of a batch entry
    int nseg, seg_len;                    // segments of the longest sequence, chunks a segment
};

// Where a chunk lies.
struct Place {
    long b;   // batch entry (addresses)
    long t0;  // its first token there
    int len;  // tokens, 1 .. kC (0: no such chunk)
};

struct Seq {
    long b, t0, len, slot0;  // slot0: the slot of its first chunk
};

__host__ __device__ inline long packed_at(const Cuts &p, long s)
{
    const long c = p.cu[s];
    return c < 0 ? 0 : (c > p.tokens ? p.tokens : c);
}

// Sequence s. Packed sequences' chunks get slots from cu / 64 + s on: at
// least as many as they need before the next sequence's, without a table.
__host__ __device__ inline Seq find_seq(const Cuts &p, long s)
{
    if (p.n_seq == 0) return {s, 0, p.tokens, s * p.chunks_b};
    const long a = packed_at(p, s), e = packed_at(p, s + 1);
    return {0, a, e > a ? e - a : 0, a / kC + s};
}

// The last packed sequence whose key is x or below (the first one, if none is).
template <typename F>
__host__ __device__ inline long last_at(const Cuts &p, long x, F &&key)
{
    long lo = 0, hi = p.n_seq - 1;
    while (lo < hi) {
        const long mid = (lo + hi + 1) / 2;
        if (key(mid) <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__host__ __device__ inline long chunk_slots(const Cuts &p) { return p.n_seq > 0 ? p.tokens / kC + p.n_seq : p.batch * p.chunks_b; }

__host__ __device__ inline Place find_chunk(const Cuts &p, long slot)
{
    const Seq q = find_seq(p, p.n_seq == 0 ? slot / p.chunks_b : last_at(p, slot, [&](long s) { return packed_at(p, s) / kC + s; }));
    const long at = (slot - q.slot0) * kC;
    if (at < 0 || at >= q.len) return {0, 0, 0};
    return {q.b, q.t0 + at, static_cast<int>(q.len - at < kC ? q.len - at : kC)};
}

// Segments. Packed sequences' first ones are numbered as the sequences are; the
// others, with W tokens a segment, from n_seq + offset / W on: of a sequence of len
// tokens there are ceil(len / W) - 1 more, and len / W or more numbers before the next
// one's. Where a segment's transition and states are kept (its place), only
// sequences of several have any, from 2 offset / W on: a sequence of len > W tokens
// needs ceil(len / W) places, and 2 len / W or more lie before the next one's.
struct Segment {
    Seq q;
    long s;
    int at, of;  // segment `at` of its sequence's `of` (of = 0: no such segment)
    long place;
};

__host__ __device__ inline unsigned seg_tokens(const Cuts &p) { return static_cast<unsigned>(p.seg_len) * kC; }
__host__ __device__ inline long seg_places(const Cuts &p) { return p.n_seq > 0 ? 2 * p.tokens / seg_tokens(p) : p.batch * p.nseg; }
__host__ __device__ inline long seg_count(const Cuts &p) { return p.n_seq > 0 ? p.tokens / seg_tokens(p) + p.n_seq : p.batch * p.nseg; }
// (32-bit divisions: there are less than 2^22 chunks)
__host__ __device__ inline long first_place(const Cuts &p, long s) { return 2 * static_cast<unsigned>(packed_at(p, s)) / seg_tokens(p); }
__host__ __device__ inline long next_segment(const Cuts &p, long s) { return static_cast<unsigned>(packed_at(p, s)) / seg_tokens(p); }

// Segment `at` of packed sequence s; CUT: of sequences of several.
template <bool CUT>
__host__ __device__ inline Segment packed_segment(const Cuts &p, long s, long at)
{
    const Seq q = find_seq(p, s);
    const long of = q.len > 0 ? (static_cast<unsigned>(q.len) + seg_tokens(p) - 1) / seg_tokens(p) : 1;
    const bool is = at >= 0 && at < of && !(CUT && of == 1);
    return {q, s, static_cast<int>(at), is ? static_cast<int>(of) : 0, first_place(p, s) + at};
}
// Segment x of all, or (CUT) that of place x.
template <bool CUT>
__host__ __device__ inline Segment find_segment(const Cuts &p, long x)
{
    if (p.n_seq == 0) {
        const long s = static_cast<unsigned>(x) / static_cast<unsigned>(p.nseg);
        return {find_seq(p, s), s, static_cast<int>(x - s * p.nseg), p.nseg, x};
    }
    if constexpr (CUT) {
        const long s = last_at(p, x, [&](long i) { return first_place(p, i); });
        return packed_segment<true>(p, s, x - first_place(p, s));
    } else {
        if (x < p.n_seq) return packed_segment<false>(p, x, 0);
        x -= p.n_seq;
        const long s = last_at(p, x, [&](long i) { return next_segment(p, i); });
        const Segment g = packed_segment<false>(p, s, x - next_segment(p, s) + 1);
        return g.at > 0 ? g : Segment{g.q, g.s, 0, 0, 0};
    }
}

// Workgroups of the join go by sequence, or by place where that makes far fewer (only
// a sequence's first place does anything, and finding it takes a search, which empty
// workgroups wait for: of 7 sequences with 49 places, 8 heads of 128 x 128, 22 us by
// sequence and 47 by place).
__host__ __device__ inline bool join_by_place(const Cuts &p) { return p.n_seq > 4 * seg_places(p); }
__host__ __device__ inline long join_count(const Cuts &p) { return p.n_seq == 0 ? p.batch : (join_by_place(p) ? seg_places(p) : p.n_seq); }
__host__ __device__ inline Segment find_joined(const Cuts &p, long x)
{
    if (p.n_seq == 0) return find_segment<true>(p, x * p.nseg);
    const Segment g = join_by_place(p) ? find_segment<true>(p, x) : packed_segment<true>(p, x, 0);
    return g.at == 0 ? g : Segment{g.q, g.s, 0, 0, 0};
}

// ------------------------------------------------------------------ host

// A call, as far as its cutting goes. cols: columns a workgroup of the chains.
struct Extent {
    long batch, tokens, n_seq;
    int hk, rep, kd, dvp, cols;  // kd, dvp: d_k and d_v rounded up
    bool grad;
    long units;                  // workgroups of the chains the chip holds at once
    double join;                 // a segment's step of the join, in steps of a chain
};

// Segments of the chains. Whole, a chain of n chunks takes n steps, and the
// `chains` * vb workgroups of all chains (twice that with the adjoints') may
// leave compute units idle. In P segments: ceil(n / P) steps of the probes
// (pb blocks of columns a chain), `join` of a step a segment to join them, and
// ceil(n / P) steps again. The P with the fewest steps is taken, counting
// rounds of `units` workgroups. Packed sequences' lengths are on the device:
// there it is planned for one that holds all tokens, since any number of short ones
// may lie beside a long one, whose chain alone then bounds the call (127 sequences of
// 500 tokens and one of 200000, 8 heads of 128 x 128, bf16 forward: 3.3 ms, 22.3 when
// that many chains count as filling the chip; 1000 of 66 tokens, which nothing cuts,
// pay 844 us instead of 806 for a probe and a join without work). A sequence no longer
// than a segment is not cut; those that are may end in a part of one, which is
// counted for half as many as there are segments.
inline Cuts plan_segments(const Extent &x, long heads)
{
    Cuts p{};
    p.batch = x.batch, p.tokens = x.tokens, p.n_seq = x.n_seq, p.chunks_b = (x.tokens + kC - 1) / kC;
    const bool packed = x.n_seq > 0;
    const long n = packed ? x.tokens / kC + 1 : p.chunks_b, dirs = x.grad ? 2 : 1;
    const long chains = packed ? heads : x.batch * heads;
    const long vb = (x.dvp + x.cols - 1) / x.cols, pb = (x.dvp + x.kd + x.cols - 1) / x.cols;
    auto rounds = [&](long workgroups) { return (workgroups + x.units - 1) / x.units; };
    p.nseg = 1;
    p.seg_len = static_cast<int>(n);
    if (chains * vb * dirs >= 4 * x.units) return p;
    double best = static_cast<double>(n * rounds(chains * vb * dirs));
    for (long k = 2; k <= std::min<long>(n / 4, 256); ++k) {
        const long len = (n + k - 1) / k, segs = (k + std::min(x.n_seq, k / 2)) * chains;
        const double steps =
            static_cast<double>(len * (rounds(segs * (pb + (x.grad ? vb : 0))) + rounds(segs * vb * dirs))) + x.join * static_cast<double>(k);
        if (steps < best) best = steps, p.seg_len = static_cast<int>(len), p.nseg = static_cast<int>((n + len - 1) / len);
    }
    return p;
}

constexpr int kGates = 5 * kC;
// The triangular matrices of a chunk are kept as 10 tiles of 16 x 16, tile
// (a, b), a >= b, at a (a + 1) / 2 + b, and multiplied as 6 fragments of 16 x 32.
constexpr int kTriTiles = 10, kTriFloats = kTriTiles * 256, kTriFrags = 6;

// Bytes of the workspace, of one head each but `sums` (of one key head).
struct Share {
    size_t gates, tri, state, row;  // of its chunks: gates; M, and M^T or P; S0 and D1; E, dR and Z
    size_t seg_a, seg_s;            // of its segments: transitions, states
    size_t sums;                    // dQ and dK of heads that share the key head
    size_t head(bool grad) const { return gates + 2 * tri + (grad ? 2 * state + 3 * row : 0) + (grad ? 2 : 1) * (seg_a + seg_s); }
};

struct Passes {
    Cuts cuts;
    Share share;
    int nhk;  // key heads a pass
    size_t bytes(const Extent &x) const { return (share.head(x.grad) * x.rep + share.sums) * nhk; }
};

// Workspace of one pass at most (heads beyond it take another pass).
constexpr double kMostBytes = 16.0 * (1u << 30);

inline Passes plan_passes(const Extent &x)
{
    Passes r{};
    for (r.nhk = x.hk;;) {
        r.cuts = plan_segments(x, static_cast<long>(x.rep) * r.nhk);
        const size_t n = static_cast<size_t>(chunk_slots(r.cuts)), places = r.cuts.nseg > 1 ? static_cast<size_t>(seg_places(r.cuts)) : 0;
        const size_t kd = static_cast<size_t>(x.kd), dvp = static_cast<size_t>(x.dvp);
        r.share = {n * kGates * 4,   n * kTriFloats * 4,    n * kd * dvp * 4, n * kC * dvp * 4, places * kd * kd * 6,
                   places * kd * dvp * 4, x.grad && x.rep > 1 ? n * 2 * kC * kd * 4 : 0};
        const double all = static_cast<double>(r.bytes(x));
        if (all <= kMostBytes || r.nhk == 1) return r;
        // (fewer heads may be cut into more segments: again, with fewer)
        r.nhk = std::max(1, std::min(r.nhk - 1, static_cast<int>(r.nhk * (kMostBytes / all))));
    }
}

}  // namespace ssm2d_impl
