"""How the gated delta rule cuts its sequences (csrc/delta_plan.h), on the CPU:
every chunk and segment of packed sequences is found once, by host code built
from the header that the kernels use, and a pass's workspace stays within its bound."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

import selective_state_space_ssm2d_amd as pkg

CSRC = os.path.join(os.path.dirname(pkg.LIB_PATH), "csrc")
SOURCE = r"""
#include <map>
#include <vector>
#include "delta_plan.h"
using namespace ssm2d_impl;

extern "C" void plan(const long *in, double join, double *out)
{
    Extent x{in[0], in[1], in[2], int(in[3]), int(in[4]), int(in[5]), int(in[6]), int(in[7]), in[8] != 0, in[9], join};
    const Passes p = plan_passes(x);
    const bool cut = p.cuts.nseg > 1;
    const double o[] = {double(p.cuts.nseg), double(p.cuts.seg_len), double(p.nhk), double(p.bytes(x)), double(chunk_slots(p.cuts)),
                        cut ? double(seg_places(p.cuts)) : 0.0, double(seg_count(p.cuts))};
    for (int i = 0; i < 7; ++i) out[i] = o[i];
}

// 0, or the number of the rule that does not hold. `sorted`: the offsets are valid.
extern "C" int check(const int *cu, long batch, long n_seq, long tokens, int seg_len, bool sorted)
{
    Cuts c{};
    c.cu = cu, c.batch = batch, c.n_seq = n_seq, c.tokens = tokens, c.chunks_b = (tokens + kC - 1) / kC, c.seg_len = seg_len;
    const long n = n_seq ? tokens / kC + 1 : c.chunks_b, seqs = n_seq ? n_seq : batch, W = long(seg_len) * kC;
    c.nseg = int((n + seg_len - 1) / seg_len);
    std::vector<int> seen(batch * tokens);
    for (long slot = 0; slot < chunk_slots(c); ++slot) {
        const Place p = find_chunk(c, slot);
        for (int t = 0; t < p.len; ++t) {
            if (p.t0 + t >= tokens) return 1;
            ++seen[p.b * tokens + p.t0 + t];
        }
    }
    for (int t : seen)
        if (sorted && t != 1) return 2;
    std::map<std::pair<long, int>, long> chains, places;
    for (long x = 0; x < seg_count(c); ++x) {
        const Segment g = find_segment<false>(c, x);
        if (g.of == 0) continue;
        if (g.s < 0 || g.s >= seqs || g.at < 0 || g.at >= g.of || g.q.t0 < 0 || g.q.t0 + g.q.len > tokens) return 3;
        if (g.of > 1 && (g.place < 0 || g.place >= seg_places(c))) return 4;
        if (g.of != std::max(1L, (g.q.len + W - 1) / W) && n_seq) return 5;
        if (chains.count({g.s, g.at}) && sorted) return 6;
        chains[{g.s, g.at}] = g.of > 1 ? g.place : -1;
    }
    if (c.nseg > 1)
        for (long x = 0; x < seg_places(c); ++x) {
            const Segment g = find_segment<true>(c, x);
            if (g.of == 0) continue;
            if (g.of < 2 || g.place != x || g.at < 0 || g.at >= g.of) return 7;
            places[{g.s, g.at}] = x;
        }
    std::map<long, int> joined;
    for (long x = 0; c.nseg > 1 && x < join_count(c); ++x) {
        const Segment g = find_joined(c, x);
        if (g.of == 0) continue;
        if (g.of < 2 || g.at != 0 || g.place < 0 || g.place + g.of > seg_places(c)) return 11;
        ++joined[g.s];
    }
    if (!sorted) return 0;
    for (long s = 0; s < seqs; ++s) {
        const Seq q = find_seq(c, s);
        const long of = std::max(1L, (q.len + W - 1) / W);
        for (int i = 0; i < of; ++i) {
            if (!chains.count({s, i})) return 8;
            if (of > 1 && (!places.count({s, i}) || places[{s, i}] != chains[{s, i}])) return 9;
        }
        if (chains.count({s, int(of)})) return 10;
        if (joined[s] != (of > 1 ? 1 : 0)) return 12;
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if shutil.which("hipcc") is None:
        pytest.skip("hipcc not found")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    out = str(d / "libplan.so")
    subprocess.run(["hipcc", "-x", "hip", "--offload-host-only", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "plan.cpp"), "-o", out],
                   check=True)
    return ctypes.CDLL(out)


def _check(lib, lens, seg_len, batch=1, cu=None):
    if isinstance(lens, int):  # a batch of one length
        return lib.check(None, ctypes.c_long(batch), ctypes.c_long(0), ctypes.c_long(lens), seg_len, True)
    valid = cu is None
    cu = cu or [sum(lens[:i]) for i in range(len(lens) + 1)]
    return lib.check((ctypes.c_int * len(cu))(*cu), ctypes.c_long(1), ctypes.c_long(len(cu) - 1), ctypes.c_long(sum(lens)), seg_len, valid)


def test_every_chunk_and_segment_is_found_once(lib):
    rng = random.Random(1)
    lists = [[1], [64], [65, 1], [0, 0, 5], [512] * 64, [196] * 64, [66] * 300, [5120, 1, 0, 777, 4099, 64, 9973], [0, 20000, 0, 1]]
    for _ in range(60):
        most = rng.choice([3, 70, 700, 5000])
        lists.append([rng.choice([0, 1, 63, 64, 65, rng.randint(0, most)]) for _ in range(rng.randint(1, 60))] + [rng.randint(1, most)])
    for lens in lists:
        n = sum(lens) // 64 + 1
        for seg_len in {1, 2, 3, rng.randint(1, n), max(1, n // 7), n}:
            assert _check(lib, lens, seg_len) == 0, (lens, seg_len)
    for tokens in (1, 64, 65, 1000, 4096):
        for seg_len in (1, 3, (tokens + 63) // 64):
            assert _check(lib, tokens, seg_len, batch=3) == 0, (tokens, seg_len)


def test_offsets_out_of_order_stay_in_range(lib):
    rng = random.Random(2)
    for _ in range(60):
        tokens = rng.choice([10, 1000, 9000])
        cu = [rng.choice([rng.randint(-100, 2 * tokens), -2 ** 31, 2 ** 31 - 1]) for _ in range(rng.randint(2, 40))]
        assert _check(lib, [tokens], rng.randint(1, tokens // 64 + 1), cu=cu) == 0, (tokens, cu)


def _plan(lib, tokens, n_seq, hk, rep=1, kd=128, dv=128, grad=False, batch=1):
    dvp = -(-dv // 32) * 32
    cols = 128 if not grad and dvp > 64 else 64
    units, join = (512 if kd <= 64 else 256), {128: 0.4, 64: 0.3, 32: 0.1}[kd]
    out = (ctypes.c_double * 7)()
    lib.plan((ctypes.c_long * 10)(batch, tokens, n_seq, hk, rep, kd, dvp, cols, grad, units), ctypes.c_double(join), out)
    return dict(zip(("nseg", "seg_len", "nhk", "bytes", "slots", "places", "groups"), out))


@pytest.mark.parametrize("grad", [False, True])
def test_packed_workspaces_follow_the_tokens(lib, grad):
    """The chunks' share is what the tokens need (at most one more chunk a sequence); segments add less than 513
    places a head, whatever the number of sequences, and a pass more than one key head only within 16 GiB."""
    for n_seq, tokens, hk, rep, kd, dv in [(64, 32768, 8, 1, 128, 128), (64, 12544, 12, 1, 64, 64), (1000, 66000, 1, 1, 128, 128),
                                           (1000, 1000000, 1, 1, 128, 128), (64, 262144, 8, 1, 128, 128), (200, 1 << 20, 4, 1, 128, 128),
                                           (128, 262144, 4, 2, 128, 128), (3, 100000, 16, 2, 32, 1024), (100000, 400000, 1, 1, 32, 32)]:
        p = _plan(lib, tokens, n_seq, hk, rep, kd, dv, grad)
        dirs, dvp = 1 + grad, -(-dv // 32) * 32
        chunk = 21760 + (4 * (2 * kd + 192) * dvp if grad else 0) + (512 * kd if grad and rep > 1 else 0) / rep
        heads = p["nhk"] * rep
        chunks = (tokens // 64 + n_seq) * chunk * heads
        segments = p["places"] * dirs * kd * (6 * kd + 4 * dvp) * heads
        assert abs(p["bytes"] - chunks - segments) < 1, p
        assert p["places"] <= 512 and p["nseg"] <= 256, p
        assert p["nhk"] == 1 or p["bytes"] <= 16 << 30, p
        # groups of the chains beyond one a sequence: one more for each segment's length of tokens
        assert p["groups"] <= n_seq + 256, p
        if not grad and n_seq in (64, 1000) and tokens < 100000:
            assert p["bytes"] < 1 << 30, p


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("tokens,hk,kd", [(32768, 8, 128), (263500, 8, 128), (1 << 20, 4, 64), (100000, 24, 32)])
def test_short_sequences_beside_a_long_one_do_not_keep_it_whole(lib, tokens, hk, kd, grad):
    """The host does not know the lengths: whatever their number, one sequence may hold nearly all tokens. Its chains
    (rounds of a segment's chunks, twice, and the join) take at most twice the steps that they are planned to take alone."""
    join, units, dirs = {128: 0.4, 64: 0.3, 32: 0.1}[kd], (512 if kd <= 64 else 256), 1 + grad
    cols = 128 if not grad and kd > 64 else 64
    vb, pb = -(-kd // cols), -(-2 * kd // cols)

    def steps(n_seq):
        p = _plan(lib, tokens, n_seq, hk, kd=kd, dv=kd, grad=grad)
        groups = p["nseg"] * hk
        main = p["seg_len"] * -(-groups * vb * dirs // units)
        probe = p["seg_len"] * -(-groups * (pb + (vb if grad else 0)) // units) + join * p["nseg"]
        return main + (probe if p["nseg"] > 1 else 0)

    alone = steps(1)
    for n_seq in (2, 7, 64, 127, 128, 129, 500, 1000):
        assert steps(n_seq) <= 2 * alone, (n_seq, steps(n_seq), alone)
