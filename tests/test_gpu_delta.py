"""GPU tests of the gated delta rule against the recurrence in 64 bits.

Bars: with unit keys, beta in [0, 1] and decays <= 1 a token's update does not
enlarge an error already in the state, and adds u = 2^-24 of each product and
sum it forms, over dots of d_k (d_v) terms. Errors of independent roundings add
like a random walk, so after T tokens an output errs by about
u sqrt(T d) times the largest values around; the bar is 8 times that (32 for
gradients, which pass through the recurrence twice). A bf16 output adds half a
unit of its last place, 2^-9 of its value.
"""
import math

import pytest

import selective_state_space_ssm2d_amd as pkg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make(B, T, hk, h, dk, dv, dtype, seed, decay=0.05):
    g = _gen(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
    q, k = unit(rn(B, T, hk, dk)).to(DT[dtype]), unit(rn(B, T, hk, dk) + 0.3).to(DT[dtype])
    v = rn(B, T, h, dv).to(DT[dtype])
    gate = -decay * torch.nn.functional.softplus(2 * rn(B, T, h))
    return q, k, v, gate, torch.sigmoid(rn(B, T, h))


def reference(q, k, v, g, beta, scale, S0=None):
    """o, last state and the largest state entry, token by token in 64 bits (on the CPU for tiny sizes, else the GPU)."""
    h = v.shape[2]
    q, k, v, g, beta = (t.double() for t in (q, k, v, g, beta))
    q, k = (t.repeat_interleave(h // t.shape[2], 2) for t in (q, k))
    S = torch.zeros(v.shape[0], h, q.shape[3], v.shape[3], dtype=torch.float64, device=v.device) if S0 is None else S0.double().clone()
    o, top = torch.zeros_like(v), S.abs().amax() if S.numel() else torch.zeros(())
    for t in range(v.shape[1]):
        S = torch.exp(g[:, t])[..., None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(2))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        o[:, t] = scale * (S * q[:, t, :, :, None]).sum(2)
        top = torch.maximum(top, S.abs().amax())
    return o, S, float(top)


def _bar(T, d, size, ref, dtype, c=8):
    return c * U * math.sqrt(max(T, 1) * d) * size + (2.0 ** -8 * ref.abs() if dtype == "bf16" else 0.0) + 1e-30


def _close(got, ref, tol, what):
    d = (got.double() - ref).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), (what, float(d[bad].max()), int(bad.sum()), d.numel())


# (batch, hk, h, dk, dv)
STEP = [(1, 1, 1, 1, 1), (2, 1, 3, 5, 7), (3, 2, 4, 16, 24), (1, 4, 8, 128, 128), (64, 4, 8, 64, 64), (2, 3, 3, 96, 130), (5, 2, 2, 33, 64),
        (1, 2, 2, 127, 20), (40, 8, 16, 128, 128), (1, 1, 2, 128, 1024)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", STEP, ids=str)
def test_step(case, dtype):
    B, hk, h, dk, dv = case
    state = torch.randn(B, h, dk, dv, generator=_gen(1), device="cuda")
    for n in range(3):
        q, k, v, g, beta = make(B, 1, hk, h, dk, dv, dtype, 100 + n)
        scale = None if n else 0.7
        ref, S, top = reference(q, k, v, g, beta, dk ** -0.5 if scale is None else scale, state)
        o = pkg.gated_delta_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], state, scale=scale)
        _close(o, ref[:, 0], _bar(1, dk, top, ref[:, 0], dtype), f"o {case} {n}")
        _close(state, S, _bar(1, dk, top, S, "f32"), f"state {case} {n}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_of_a_few_tokens(dtype):
    q, k, v, g, beta = make(3, 7, 2, 4, 40, 36, dtype, 7)
    state = torch.randn(3, 4, 40, 36, generator=_gen(2), device="cuda")
    ref, S, top = reference(q, k, v, g, beta, 40 ** -0.5, state)
    o = pkg.gated_delta_step(q, k, v, g, beta, state)
    _close(o, ref, _bar(7, 40, top, ref, dtype), "o")
    _close(state, S, _bar(7, 40, top, S, "f32"), "state")


def test_step_views_and_resets():
    """Tokens sliced out of a longer sequence, misaligned states, decays that clear the state, beta of 0 and 1."""
    q, k, v, g, beta = make(2, 9, 2, 4, 32, 20, "bf16", 8)
    g[0, 4], g[1, 4, 1] = -math.inf, -200.0
    beta[0, 4, 0], beta[1, 4, 2] = 0.0, 1.0
    flat = torch.randn(2 * 4 * 32 * 20 + 1, generator=_gen(3), device="cuda")
    state = flat[1:].view(2, 4, 32, 20)
    ref, S, top = reference(q[:, 4:5], k[:, 4:5], v[:, 4:5], g[:, 4:5], beta[:, 4:5], 32 ** -0.5, state)
    o = pkg.gated_delta_step(q[:, 4], k[:, 4], v[:, 4], g[:, 4], beta[:, 4], state)
    _close(o, ref[:, 0], _bar(1, 32, top, ref[:, 0], "bf16"), "o")
    _close(state, S, _bar(1, 32, top, S, "f32"), "state")


# (batch, tokens, hk, h, dk, dv)
SEQ = [(1, 1, 1, 1, 1, 1), (1, 2, 1, 2, 3, 5), (2, 15, 1, 1, 16, 16), (2, 16, 2, 2, 32, 32), (1, 17, 1, 2, 20, 40), (3, 63, 2, 4, 64, 64),
       (2, 64, 1, 1, 128, 128), (1, 65, 2, 2, 128, 64), (2, 100, 1, 3, 33, 17), (1, 129, 2, 4, 96, 100), (2, 196, 3, 3, 64, 64),
       (1, 777, 1, 2, 128, 128), (1, 640, 4, 4, 32, 32), (4, 130, 1, 1, 8, 130),
       # long chains of few heads, cut into segments
       (1, 2100, 1, 2, 128, 96), (2, 1500, 2, 2, 30, 20), (1, 1793, 1, 1, 64, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", SEQ, ids=str)
def test_fwd(case, dtype):
    B, T, hk, h, dk, dv = case
    q, k, v, g, beta = make(B, T, hk, h, dk, dv, dtype, T + dk)
    h0 = torch.randn(B, h, dk, dv, generator=_gen(4), device="cuda")
    for init in (None, h0):
        ref, S, top = reference(q, k, v, g, beta, dk ** -0.5, init)
        o, last = pkg.gated_delta_fwd(q, k, v, g, beta, h_init=init, return_last_state=True)
        _close(o, ref, _bar(T, dk, top, ref, dtype), f"o {case}")
        _close(last, S, _bar(T, dk, top, S, "f32"), f"h_last {case}")
    only = pkg.gated_delta_fwd(q, k, v, g, beta, h_init=h0)
    assert torch.equal(only, o)


LENS = [[1], [64], [65, 1], [0, 3, 0, 130, 64, 0], [200, 17, 128, 1, 1, 63], [0, 0, 5], [1300, 5, 0, 700, 64]]


def _packed(lens, hk, h, dk, dv, dtype, seed):
    x = make(1, sum(lens), hk, h, dk, dv, dtype, seed)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    return x, cu, torch.randn(len(lens), h, dk, dv, generator=_gen(seed + 1), device="cuda")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_fwd_packed(lens, dtype):
    hk, h, dk, dv = 2, 4, 48, 40
    x, cu, h0 = _packed(lens, hk, h, dk, dv, dtype, 31)
    for init in (None, h0):
        o, last = pkg.gated_delta_fwd(*x, h_init=init, cu_seqlens=cu, return_last_state=True)
        at = 0
        for i, t in enumerate(lens):
            part = [y[:, at:at + t] for y in x]
            ref, S, top = reference(*part, dk ** -0.5, None if init is None else init[i:i + 1])
            _close(o[:, at:at + t], ref, _bar(t, dk, top, ref, dtype), f"o {lens} {i}")
            _close(last[i:i + 1], S, _bar(t, dk, top, S, "f32"), f"h_last {lens} {i}")
            at += t


def test_fwd_state_in_place_and_bands():
    """A sequence in bands, each band's last state written over its initial one, is the whole sequence's."""
    x = make(2, 300, 1, 2, 64, 32, "f32", 40)
    want, S = pkg.gated_delta_fwd(*x, return_last_state=True)
    state = torch.zeros(2, 2, 64, 32, device="cuda")
    got = torch.cat([pkg.gated_delta_fwd(*(t[:, a:b] for t in x), h_init=state, h_last=state) for a, b in ((0, 100), (100, 107), (107, 300))], 1)
    ref, _, top = reference(*x, 64 ** -0.5)
    _close(got, ref, _bar(300, 64, top, ref, "f32"), "bands")
    _close(want, ref, _bar(300, 64, top, ref, "f32"), "whole")
    _close(state, S.double(), _bar(300, 64, top, S.double(), "f32"), "state")


def _views(x, dtype):
    """The same values in other layouts: heads before tokens, odd offsets, tokens of one fused row."""
    q, k, v, g, beta = x
    B, T, hk, dk = q.shape
    h, dv = v.shape[2:]
    pad = torch.zeros(B, T, 2 * hk * dk + h * dv + 3, dtype=q.dtype, device="cuda")
    fused = pad[..., 3:]
    fused[..., :hk * dk], fused[..., hk * dk:2 * hk * dk], fused[..., 2 * hk * dk:] = q.flatten(2), k.flatten(2), v.flatten(2)
    yield (fused[..., :hk * dk].unflatten(-1, (hk, dk)), fused[..., hk * dk:2 * hk * dk].unflatten(-1, (hk, dk)),
           fused[..., 2 * hk * dk:].unflatten(-1, (h, dv)), g, beta)
    yield tuple(t.transpose(1, 2).contiguous().transpose(1, 2) for t in x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_views(dtype):
    x = make(2, 97, 2, 4, 64, 48, dtype, 41)
    do = torch.randn(2, 97, 4, 48, generator=_gen(42), device="cuda").to(DT[dtype])
    o = pkg.gated_delta_fwd(*x)
    r = pkg.gated_delta_bwd(*x, do)
    for y in _views(x, dtype):
        assert torch.equal(pkg.gated_delta_fwd(*y), o)
        e = pkg.gated_delta_bwd(*y, do.transpose(1, 2).contiguous().transpose(1, 2))
        assert all(torch.equal(e[n], r[n]) for n in r)


def test_resets_and_extreme_gates():
    """Decays of -inf (the state is cleared), of -300 and of 0, beta of 0 and 1, in the middle of a chunk."""
    x = make(1, 150, 1, 2, 32, 32, "f32", 43)
    g, beta = x[3], x[4]
    g[0, 40, 0], g[0, 70, 1], g[0, 64:70, 0] = -math.inf, -300.0, 0.0
    beta[0, 10:14, 0], beta[0, 20, 1] = 0.0, 1.0
    ref, S, top = reference(*x, 32 ** -0.5)
    o, last = pkg.gated_delta_fwd(*x, return_last_state=True)
    _close(o, ref, _bar(150, 32, top, ref, "f32"), "o")
    _close(last, S, _bar(150, 32, top, S, "f32"), "state")
    do = torch.randn(1, 150, 2, 32, generator=_gen(44), device="cuda")
    _check_bwd(x, do, None, None, "f32", "resets")


def test_nan_does_not_go_back():
    """A NaN at a token leaves the chunks before its own, and the other sequences, as they are."""
    x = make(2, 200, 1, 1, 32, 32, "f32", 45)
    clean = pkg.gated_delta_fwd(*x)
    x[2][0, 100, 0, 5] = float("nan")
    o = pkg.gated_delta_fwd(*x)
    assert torch.equal(o[1], clean[1]) and torch.equal(o[0, :64], clean[0, :64])
    assert bool(torch.isnan(o[0, 100:, 0, 5]).all())


def _grads(x, do, h0, dh, dk):
    """Gradients of the recurrence in 64 bits, by autograd over its tokens."""
    leaf = [t.detach().double().requires_grad_(True) for t in (*x, *([h0] if h0 is not None else []))]
    q, k, v, g, beta = leaf[:5]
    rep = v.shape[2] // q.shape[2]
    q, k = q.repeat_interleave(rep, 2), k.repeat_interleave(rep, 2)
    S = leaf[5] if h0 is not None else torch.zeros(v.shape[0], v.shape[2], q.shape[3], v.shape[3], dtype=torch.float64, device=v.device)
    loss = torch.zeros((), dtype=torch.float64, device=v.device)
    for t in range(v.shape[1]):
        S = torch.exp(g[:, t])[..., None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(2))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        loss = loss + (dk ** -0.5 * (S * q[:, t, :, :, None]).sum(2) * do[:, t].double()).sum()
    if dh is not None:
        loss = loss + (S * dh.double()).sum()
    got = torch.autograd.grad(loss, leaf, allow_unused=True)
    return [torch.zeros_like(t) if r is None else r for t, r in zip(leaf, got)]


def _check_bwd(x, do, h0, dh, dtype, what, got=None):
    dk, dv, T = x[0].shape[3], x[2].shape[3], x[0].shape[1]
    r = got if got is not None else pkg.gated_delta_bwd(*x, do, h_init=h0, dh_last=dh)
    ref = _grads(x, do, h0, dh, dk)
    names = ["dq", "dk", "dv", "dg", "dbeta"] + (["dh_init"] if h0 is not None else [])
    rep = x[2].shape[2] // x[0].shape[2]
    terms = ((x[0].double() * ref[0]).abs().sum(-1) + (x[1].double() * ref[1]).abs().sum(-1)).max() * rep
    for n, e in zip(names, ref):
        size = float(e.abs().max()) if e.numel() else 0.0
        if n == "dg":
            size = max(size, float(terms))  # dg is a difference of sums of these
        _close(r[n], e, _bar(T, dk + dv, size, e, dtype if n in ("dq", "dk", "dv") else "f32", 32), f"{n} {what}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [c for c in SEQ if c[1] != 777], ids=str)
def test_bwd(case, dtype):
    B, T, hk, h, dk, dv = case
    x = make(B, T, hk, h, dk, dv, dtype, T + dk + 1)
    g = _gen(50)
    do = torch.randn(B, T, h, dv, generator=g, device="cuda").to(DT[dtype])
    h0, dh = torch.randn(B, h, dk, dv, generator=g, device="cuda"), torch.randn(B, h, dk, dv, generator=g, device="cuda")
    _check_bwd(x, do, h0, dh, dtype, f"{case} with states")
    _check_bwd(x, do, None, None, dtype, f"{case}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_bwd_packed(lens, dtype):
    hk, h, dk, dv = 2, 4, 48, 40
    x, cu, h0 = _packed(lens, hk, h, dk, dv, dtype, 33)
    do = torch.randn(1, sum(lens), h, dv, generator=_gen(51), device="cuda").to(DT[dtype])
    dh = torch.randn(h0.shape, generator=_gen(52), device="cuda")
    r = pkg.gated_delta_bwd(*x, do, h_init=h0, dh_last=dh, cu_seqlens=cu)
    at = 0
    for i, t in enumerate(lens):
        sl = slice(at, at + t)
        part = {n: r[n][:, sl] for n in ("dq", "dk", "dv", "dg", "dbeta")} | {"dh_init": r["dh_init"][i:i + 1]}
        if t == 0:
            assert torch.equal(part["dh_init"], dh[i:i + 1])
            continue
        _check_bwd([y[:, sl] for y in x], do[:, sl], h0[i:i + 1], dh[i:i + 1], dtype, f"{lens} {i}", got=part)
        at += t


def test_bwd_against_differences():
    """Central differences of the 64-bit recurrence along random directions of all inputs together."""
    x = make(1, 70, 1, 2, 24, 20, "f32", 60)
    g = _gen(61)
    do = torch.randn(1, 70, 2, 20, generator=g, device="cuda")
    h0, dh = torch.randn(1, 2, 24, 20, generator=g, device="cuda"), torch.randn(1, 2, 24, 20, generator=g, device="cuda")
    r = pkg.gated_delta_bwd(*x, do, h_init=h0, dh_last=dh)

    def loss(t):
        o, S, _ = reference(*t[:5], 24 ** -0.5, t[5])
        return (o * do.double()).sum() + (S * dh.double()).sum()

    full = [t.double() for t in (*x, h0)]
    for n, name in enumerate(["dq", "dk", "dv", "dg", "dbeta", "dh_init"]):
        d = torch.randn(full[n].shape, generator=g, device="cuda").double()
        e = 1e-6
        up, dn = ([t + s * e * d if i == n else t for i, t in enumerate(full)] for s in (1, -1))
        want = float((loss(up) - loss(dn)) / (2 * e))
        got = float((r[name].double() * d).sum())
        # e^2 of the third derivative and 2^-52 |loss| / e of rounding stay below 1e-5 of the terms' size
        size = float((r[name].double() * d).abs().sum())
        assert abs(got - want) <= 2e-5 * size, (name, got, want)


def test_bwd_is_deterministic_and_replays_in_a_graph():
    x = make(2, 130, 2, 4, 64, 64, "bf16", 62)
    do = torch.randn(2, 130, 4, 64, generator=_gen(63), device="cuda").bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = pkg.gated_delta_bwd(*x, do, stream=s)
    o = pkg.gated_delta_fwd(*x, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        pkg.gated_delta_bwd(*x, do, out=out)
        pkg.gated_delta_fwd(*x, o=o)
    for n in range(3):
        do.copy_(torch.randn(do.shape, generator=_gen(70 + n), device="cuda"))
        x[2].copy_(torch.randn(x[2].shape, generator=_gen(80 + n), device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        e = pkg.gated_delta_bwd(*x, do)
        assert all(torch.equal(e[k], out[k]) for k in e) and torch.equal(pkg.gated_delta_fwd(*x), o)


def test_workspaces_are_released():
    x = make(1, 100, 1, 1, 32, 32, "f32", 64)
    o = pkg.gated_delta_fwd(*x)
    pkg.release_workspaces()
    assert torch.equal(pkg.gated_delta_fwd(*x), o)


def test_fwd_without_tokens():
    q, k, v, g, beta = make(2, 0, 1, 2, 8, 8, "f32", 1)
    h0 = torch.randn(2, 2, 8, 8, device="cuda")
    o, last = pkg.gated_delta_fwd(q, k, v, g, beta, h_init=h0, return_last_state=True)
    assert o.shape == (2, 0, 2, 8) and torch.equal(last, h0)
    o, last = pkg.gated_delta_fwd(q, k, v, g, beta, return_last_state=True)
    assert bool((last == 0).all())


def test_refusals():
    q, k, v, g, beta = make(2, 4, 2, 4, 8, 8, "f32", 1)
    st = torch.zeros(2, 4, 8, 8, device="cuda")
    F, S = pkg.gated_delta_fwd, pkg.gated_delta_step
    cu = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    wide = make(1, 4, 1, 1, 129, 8, "f32", 1)
    bad = [(ValueError, lambda: F(q, k[:, :3], v, g, beta)), (TypeError, lambda: F(q, k.bfloat16(), v, g, beta)),
           (ValueError, lambda: F(q, k, v[:, :, :3], g[:, :, :3], beta[:, :, :3])), (ValueError, lambda: F(q, k, v, g[:, :, :2], beta)),
           (ValueError, lambda: F(q, k, v, g.double(), beta)), (ValueError, lambda: F(q, k, v, g, beta.bfloat16())),
           (ValueError, lambda: F(q, k, v, g, beta, h_init=st[:1])), (ValueError, lambda: F(q, k, v, g, beta, h_init=st.double())),
           (ValueError, lambda: F(q, k, v, g, beta, cu_seqlens=cu)), (ValueError, lambda: F(q[:1], k[:1], v[:1], g[:1], beta[:1], cu_seqlens=cu.long())),
           (ValueError, lambda: F(q[:1], k[:1], v[:1], g[:1], beta[:1], cu_seqlens=cu[:1])),
           (ValueError, lambda: F(q.transpose(2, 3), k.transpose(2, 3), v, g, beta)), (ValueError, lambda: F(q, k, v.cpu(), g, beta)),
           (TypeError, lambda: F(q.half(), k.half(), v.half(), g, beta)), (pkg.Ssm2dError, lambda: F(*wide)),
           (ValueError, lambda: pkg.gated_delta_bwd(q, k, v, g, beta, v[:, :3])),
           (ValueError, lambda: pkg.gated_delta_bwd(q, k, v, g, beta, v, dh_last=st[:1])),
           (ValueError, lambda: S(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], st[:1])),
           (ValueError, lambda: S(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], st.transpose(2, 3))),
           (ValueError, lambda: S(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], None))]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            pytest.fail(f"case {i} was not refused")
