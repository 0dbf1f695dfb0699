"""GPU tests of the gated delta rule where its dispatch and its roundings are
easiest to get wrong: how a bf16 output is rounded, wide values, and many packed
sequences. The bars are those of the operator's own tests unless a test
derives another.
"""
import math

import pytest

import selective_state_space_ssm2d_amd as pkg
import test_gpu_delta as D

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = D.U
DT = D.DT


def _reference_terms(q, k, v, g, beta, scale):
    """o in 64 bits, and the sum of the magnitudes of the terms that make each of its elements."""
    h = v.shape[2]
    q, k, v, g, beta = (t.double() for t in (q, k, v, g, beta))
    q, k = (t.repeat_interleave(h // t.shape[2], 2) for t in (q, k))
    S = torch.zeros(v.shape[0], h, q.shape[3], v.shape[3], dtype=torch.float64, device=v.device)
    o, terms = torch.zeros_like(v), torch.zeros_like(v)
    for t in range(v.shape[1]):
        S = torch.exp(g[:, t])[..., None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(2))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        o[:, t] = scale * (S * q[:, t, :, :, None]).sum(2)
        terms[:, t] = scale * (S * q[:, t, :, :, None]).abs().sum(2)
    return o, terms


# (batch, tokens, hk, h, dk, dv): the state's parts, the chunk's own (P U), both, and segments
@pytest.mark.parametrize("case", [(256, 24, 4, 4, 32, 32), (128, 64, 2, 4, 32, 32), (64, 70, 2, 2, 64, 64), (24, 130, 4, 8, 128, 128),
                                  (1, 1500, 2, 4, 32, 64)], ids=str)
def test_bf16_outputs_are_rounded_once(case):
    """A bf16 output is an fp32 sum's, rounded once: it is another neighbour than the 64-bit result's only where
    that lies within the sum's error of the middle between two. With roundings of u = 2^-24 that add like a random
    walk over T tokens and d terms, an error is about u sqrt(T + d) times the magnitude of its terms, and
    falls across the middle for error / spacing of the elements; twice that is allowed, and 5 standard deviations."""
    B, T, hk, h, dk, dv = case
    x = D.make(B, T, hk, h, dk, dv, "bf16", 90 + T)
    ref, terms = _reference_terms(*x, dk ** -0.5)
    o = pkg.gated_delta_fwd(*x).double()
    spacing = torch.exp2(torch.floor(torch.log2(ref.abs().clamp_min(1e-30))) - 7)
    want = ref.to(torch.bfloat16).double()  # (64 bits to bf16 through fp32: a second rounding of 2^-16 of the spacing)
    allowed = float((2 * U * math.sqrt(T + dk) * terms / spacing + 2.0 ** -15).clamp_max(1.0).sum())
    other = int((o != want).sum())
    print(f"{case}: {other} of {o.numel()} on the other side, {allowed:.0f} allowed")
    assert other <= allowed + 5 * math.sqrt(allowed), (other, allowed, o.numel())


# ------------------------------------------------------------------ many packed sequences

def _lens(kind):
    g = torch.Generator().manual_seed(len(kind))
    if kind == "short":  # a few hundred, some empty
        return torch.randint(0, 131, (300,), generator=g).tolist()
    if kind == "one long":  # among many short ones
        return torch.randint(0, 40, (150,), generator=g).tolist() + [2300] + torch.randint(0, 40, (100,), generator=g).tolist()
    return [196] * 64  # "equal"


def _padded(x, lens):
    """Packed tensors as a batch of the longest length; what is past a sequence's end is zero, which leaves a state as it is."""
    out = []
    for t in x:
        p = torch.zeros(len(lens), max(lens), *t.shape[2:], dtype=t.dtype, device=t.device)
        at = 0
        for i, n in enumerate(lens):
            p[i, :n] = t[0, at:at + n]
            at += n
        out.append(p)
    return out


def _unpadded(t, lens):
    return torch.cat([t[i, :n] for i, n in enumerate(lens)])[None]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,dk,dv", [("short", 32, 32), ("one long", 32, 40), ("one long", 128, 96), ("equal", 64, 64)])
def test_many_packed_sequences(kind, dk, dv, dtype):
    lens, hk, h = _lens(kind), 1, 2
    x, cu, h0 = D._packed(lens, hk, h, dk, dv, dtype, 35)
    pad, T = _padded(x, lens), max(lens)
    ref, S, top = D.reference(*pad, dk ** -0.5, h0)
    ref = _unpadded(ref, lens)
    o, last = pkg.gated_delta_fwd(*x, h_init=h0, cu_seqlens=cu, return_last_state=True)
    D._close(o, ref, D._bar(T, dk, top, ref, dtype), "o")
    D._close(last, S, D._bar(T, dk, top, S, "f32"), "h_last")
    # gradients: those of the batch, one sequence an entry, which other tests hold against 64 bits (both within the bar)
    do = torch.randn(1, sum(lens), h, dv, generator=D._gen(36), device="cuda").to(DT[dtype])
    dh = torch.randn(h0.shape, generator=D._gen(37), device="cuda")
    r = pkg.gated_delta_bwd(*x, do, h_init=h0, dh_last=dh, cu_seqlens=cu)
    e = pkg.gated_delta_bwd(*pad, _padded([do], lens)[0], h_init=h0, dh_last=dh)
    terms = ((x[0].double() * r["dq"].double()).abs().sum(-1) + (x[1].double() * r["dk"].double()).abs().sum(-1)).max() * (h // hk)
    for n, t in e.items():
        want = (t if n == "dh_init" else _unpadded(t, lens)).double()
        size = float(want.abs().max())
        size = max(size, float(terms)) if n == "dg" else size
        D._close(r[n], want, 2 * D._bar(T, dk + dv, size, want, dtype if n in ("dq", "dk", "dv") else "f32", 32), n)


def _workspace(call):
    """What a first call takes besides its outputs."""
    torch.cuda.synchronize()
    pkg.release_workspaces()
    torch.cuda.empty_cache()
    before = torch.cuda.mem_get_info()[0]
    call()
    torch.cuda.synchronize()
    used = before - torch.cuda.mem_get_info()[0]
    pkg.release_workspaces()
    return used


@pytest.mark.parametrize("n_seq,tokens,h,dk,dv", [(64, 512, 8, 128, 128), (1000, 66, 1, 128, 128), (64, 196, 12, 64, 64)])
def test_packed_workspaces(n_seq, tokens, h, dk, dv):
    """Many short sequences take what their tokens need (a chunk's 21760 bytes a head, one more chunk a sequence) and at
    most 512 segments' transitions and states: below 1 GiB for each of these."""
    x = D.make(1, n_seq * tokens, h, h, dk, dv, "bf16", 38)
    cu = torch.arange(0, n_seq * tokens + 1, tokens, dtype=torch.int32, device="cuda")
    o = torch.empty_like(x[2])
    used = _workspace(lambda: pkg.gated_delta_fwd(*x, cu_seqlens=cu, o=o))
    most = ((n_seq * tokens // 64 + n_seq) * 21760 + 512 * dk * (6 * dk + 4 * dv)) * h
    assert used <= most + (64 << 20) and used < 1 << 30, (used, most)  # (an allocation is rounded up to whole MB)


# ------------------------------------------------------------------ wide values, segments of every width

# (batch, tokens, hk, h, dk, dv): probes whose workgroups hold columns of values and of the unit matrix, several blocks of columns
WIDE = [(1, 1500, 1, 1, 32, 96), (1, 1500, 1, 2, 64, 128), (1, 1300, 1, 1, 128, 260), (1, 600, 1, 1, 24, 1024), (2, 150, 1, 2, 64, 1000)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", WIDE, ids=str)
def test_wide_values(case, dtype):
    B, T, hk, h, dk, dv = case
    x = D.make(B, T, hk, h, dk, dv, dtype, T + dv)
    g = D._gen(39)
    h0, dh = torch.randn(B, h, dk, dv, generator=g, device="cuda"), torch.randn(B, h, dk, dv, generator=g, device="cuda")
    do = torch.randn(B, T, h, dv, generator=g, device="cuda").to(DT[dtype])
    ref, S, top = D.reference(*x, dk ** -0.5, h0)
    o, last = pkg.gated_delta_fwd(*x, h_init=h0, return_last_state=True)
    D._close(o, ref, D._bar(T, dk, top, ref, dtype), f"o {case}")
    D._close(last, S, D._bar(T, dk, top, S, "f32"), f"h_last {case}")
    D._check_bwd(x, do, h0, dh, dtype, f"{case}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 128), (32, 200)])
def test_wide_values_packed(dk, dv, dtype):
    lens, hk, h = [1200, 3, 0, 700, 64, 129], 1, 2
    x, cu, h0 = D._packed(lens, hk, h, dk, dv, dtype, 43)
    do = torch.randn(1, sum(lens), h, dv, generator=D._gen(44), device="cuda").to(DT[dtype])
    dh = torch.randn(h0.shape, generator=D._gen(45), device="cuda")
    o, last = pkg.gated_delta_fwd(*x, h_init=h0, cu_seqlens=cu, return_last_state=True)
    r = pkg.gated_delta_bwd(*x, do, h_init=h0, dh_last=dh, cu_seqlens=cu)
    at = 0
    for i, t in enumerate(lens):
        sl, one = slice(at, at + t), slice(i, i + 1)
        ref, S, top = D.reference(*(y[:, sl] for y in x), dk ** -0.5, h0[one])
        D._close(o[:, sl], ref, D._bar(t, dk, top, ref, dtype), f"o {i}")
        D._close(last[one], S, D._bar(t, dk, top, S, "f32"), f"h_last {i}")
        if t:
            got = {n: r[n][:, sl] for n in ("dq", "dk", "dv", "dg", "dbeta")} | {"dh_init": r["dh_init"][one]}
            D._check_bwd([y[:, sl] for y in x], do[:, sl], h0[one], dh[one], dtype, f"{i}", got=got)
        at += t


# ------------------------------------------------------------------ beyond the threads of one launch

@pytest.fixture
def large():
    """Room for tens of GB, given back afterwards."""
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free GPU memory")
    yield
    pkg.release_workspaces()
    torch.cuda.empty_cache()


def test_step_of_2_to_the_23_heads(large):
    """Two blocks of columns a head: 2^24 workgroups of 256 threads, which HIP does not take at once. Heads of one key are
    formulas of one element, each rounding a few times in fp32."""
    B, h, dv = 1 << 20, 8, 128
    g = D._gen(46)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k, gate, beta = rn(B, h, 1), rn(B, h, 1).clamp_(-1, 1), -torch.rand(B, h, generator=g, device="cuda"), torch.rand(B, h, generator=g, device="cuda")
    v, state = rn(B, h, dv), rn(B, h, 1, dv)
    parts = [slice(i, i + (B >> 3)) for i in range(0, B, B >> 3)]
    first = state.clone()
    o = pkg.gated_delta_step(q, k, v, gate, beta, state, scale=0.5)
    for p in parts:
        S = torch.exp(gate[p])[..., None] * first[p, :, 0]
        S = S + k[p] * (beta[p][..., None] * (v[p] - S * k[p]))
        size = first[p, :, 0].abs() + v[p].abs()  # (|k| <= 1: what is added up is no larger)
        assert bool(((state[p, :, 0] - S).abs() <= 16 * U * size).all()), p
        assert bool(((o[p] - 0.5 * q[p] * S).abs() <= 16 * U * size * (1 + q[p].abs())).all()), p


def test_no_tokens_of_2_to_the_32_state_elements(large):
    h0 = torch.empty(1 << 15, 1, 128, 1024, device="cuda")
    h0.view(-1)[::12345] = 1.0
    none = [torch.empty(1 << 15, 0, 1, d, device="cuda") for d in (128, 128, 1024)] + [torch.empty(1 << 15, 0, 1, device="cuda")] * 2
    _, last = pkg.gated_delta_fwd(*none, h_init=h0, return_last_state=True)
    assert all(torch.equal(last[i:i + 4096].view(torch.int32), h0[i:i + 4096].view(torch.int32)) for i in range(0, 1 << 15, 4096))


def test_no_keys_of_2_to_the_32_outputs(large):
    B, T, dv = 1 << 12, 1 << 10, 1024
    v = torch.empty(B, T, 1, dv, dtype=torch.bfloat16, device="cuda")
    q, g = torch.empty(B, T, 1, 0, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, T, 1, device="cuda")
    o = torch.full_like(v, 3.0)
    pkg.gated_delta_fwd(q, q, v, g, g, o=o)
    assert not any(bool(o[i:i + 512].any()) for i in range(0, B, 512))


# ------------------------------------------------------------------ gradients of a state that is not given

def test_bwd_writes_the_state_gradient_it_is_given():
    """dh_init in ``out`` is asked for, also where the forward started from zeros."""
    x = D.make(2, 70, 1, 2, 32, 32, "f32", 47)
    do = torch.randn(2, 70, 2, 32, generator=D._gen(48), device="cuda")
    want = pkg.gated_delta_bwd(*x, do, h_init=torch.zeros(2, 2, 32, 32, device="cuda"))["dh_init"]
    into = torch.full((2, 2, 32, 32), 3.0, device="cuda")
    r = pkg.gated_delta_bwd(*x, do, out={"dh_init": into})
    assert r["dh_init"] is into and torch.equal(into, want)
    assert "dh_init" not in pkg.gated_delta_bwd(*x, do)


# ------------------------------------------------------------------ many segments

@pytest.mark.parametrize("T,dk,dv,dtype", [(12000, 32, 32, "f32"), (9000, 64, 48, "bf16"), (9000, 128, 64, "bf16")])
def test_long_chains(T, dk, dv, dtype):
    """One sequence in as many segments as the plan makes of it, against the recurrence over all of its tokens."""
    x = D.make(1, T, 1, 1, dk, dv, dtype, T + dk)
    h0 = torch.randn(1, 1, dk, dv, generator=D._gen(49), device="cuda")
    ref, S, top = D.reference(*x, dk ** -0.5, h0)
    o, last = pkg.gated_delta_fwd(*x, h_init=h0, return_last_state=True)
    D._close(o, ref, D._bar(T, dk, top, ref, dtype), "o")
    D._close(last, S, D._bar(T, dk, top, S, "f32"), "h_last")
    x, T = tuple(t[:, :4500] for t in x), 4500
    do = torch.randn(1, T, 1, dv, generator=D._gen(50), device="cuda").to(DT[dtype])
    D._check_bwd(x, do, h0, torch.randn(h0.shape, generator=D._gen(51), device="cuda"), dtype, "long")
