"""GPU tests of the operators' edges: strides and offsets past 32 bits, sizes at
the limits of the map kernels' variants, heads of no dims, packed offsets out of
range, other streams, graphs; and of the example that runs them together.
The bars are those of the operators' own tests."""
import importlib.util
import math
import os

import pytest

import selective_state_space_ssm2d_amd as pkg
import test_gpu_delta as D
import test_gpu_norm_rope as N

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = N.DT


# ------------------------------------------------------------------ layer norm

# cells of whole 16, 8 and 4 bytes and odd ones, around the channels where a tile takes another shape
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [64, 65, 128, 129, 256, 257, 384, 512, 513, 768, 1024, 1025])
@pytest.mark.parametrize("cells", [64, 68, 70, 71])
def test_map_variants(n, cells, dtype):
    x, w, b, dy = N._norm_case((2, n, cells), dtype, n + cells, 0.5)
    N._check_norm(x, w, b, dy, dtype, True, what=f"{n} {cells}")


def _spread(t, strides):
    """t's values in a view of the given strides."""
    size = 1 + sum((s - 1) * st for s, st in zip(t.shape, strides))
    out = torch.empty(size, dtype=t.dtype, device="cuda").as_strided(t.shape, strides)
    return out.copy_(t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_far_strides(dtype):
    x, w, b, dy = N._norm_case((2, 9, 70), dtype, 1, 0.0)
    far = (9 * (1 << 26) + 8, 1 << 26, 1)  # channels 2^26 apart, the last more than 2^30
    N._check_norm(_spread(x, far), w, b, _spread(dy, far), dtype, True, what="far channels")
    near = (1 << 31, 72, 1)
    N._check_norm(_spread(x, near), w, b, _spread(dy, near), dtype, True, what="far maps")
    x, w, b, dy = N._norm_case((3, 136), dtype, 2, 0.0)
    N._check_norm(_spread(x, ((1 << 31) + 8, 1)), w, b, _spread(dy, ((1 << 30) + 8, 1)), dtype, False, what="far rows")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_channels_upwards(dtype):
    """Channels from the last to the first: a negative stride, through the C entry."""
    from selective_state_space_ssm2d_amd import ops
    x, w, b, _ = N._norm_case((1, 20, 64), dtype, 3, 0.0)
    want = pkg.layer_norm_fwd(x.flip(1), w, b, channels_first=True)
    y = torch.empty_like(x)
    last = x.data_ptr() + 19 * 64 * x.element_size()
    st = ops._entry("ssm2d_layer_norm_fwd", x.dtype)(last, w.data_ptr(), b.data_ptr(), y.data_ptr(), None, None, 1, 20, 64, 20 * 64, -64, 1e-5,
                                                   torch.cuda.current_stream().cuda_stream)
    assert st == pkg.OK
    # (another order of the same sums)
    N._close(y, want.double(), 128 * U * (1 + want.double().abs() ** 2) * w.double().abs().max() + N._half_ulp(want.double(), dtype), "upwards")


# ------------------------------------------------------------------ rotary positions

def test_rope_far_strides_and_graph():
    q = torch.randn(2, 3, 2, 32, generator=N._gen(4), device="cuda")
    pos = torch.randint(0, 99, (2, 3), generator=N._gen(5), device="cuda", dtype=torch.int32)
    freq = torch.rand(16, generator=N._gen(6), device="cuda")
    far = _spread(q, (64, (1 << 31) + 4, 32, 1))
    want = pkg.rope_fwd(q, q, pos, freq, (8, 8))
    got = pkg.rope_fwd(far, far, pos, freq, (8, 8))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = [torch.empty_like(q) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.rope_fwd(q, q, pos, freq, (8, 8), q_out=out[0], k_out=out[1])
    for _ in range(3):
        q.mul_(-0.5)
        want = pkg.rope_fwd(q, None, pos, freq, (8, 8))[0]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want) and torch.equal(out[1], want)


# ------------------------------------------------------------------ gated delta rule

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_delta_far_strides(dtype):
    """Tokens up to 2^25 elements apart: offsets past 32 bits, as dense tensors."""
    x = D.make(1, 70, 1, 2, 32, 32, dtype, 50)
    do = torch.randn(1, 70, 2, 32, generator=D._gen(51), device="cuda").to(DT[dtype])
    st = (1 << 25) + 8
    spread = [_spread(t, (70 * st, st, 32, 1)) for t in (*x[:3], do)]
    assert torch.equal(pkg.gated_delta_fwd(*spread[:3], *x[3:]), pkg.gated_delta_fwd(*x))
    want, got = pkg.gated_delta_bwd(*x, do), pkg.gated_delta_bwd(*spread[:3], *x[3:], spread[3])
    assert all(torch.equal(got[n], want[n]) for n in want)
    assert torch.equal(pkg.gated_delta_fwd(*(t[:, :5] for t in (*spread[:3], *x[3:]))), pkg.gated_delta_fwd(*(t[:, :5].contiguous() for t in x)))
    if dtype == "f32":
        with pytest.raises(pkg.Ssm2dError):
            beyond = torch.empty(20 << 26, device="cuda").as_strided((1, 20, 2, 32), (0, 1 << 26, 32, 1))
            pkg.gated_delta_fwd(x[0][:, :20], x[1][:, :20], beyond, x[3][:, :20], x[4][:, :20])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 2, 8, 9, 16, 17, 63, 64, 65])
def test_delta_lengths(tokens, dtype):
    x = D.make(3, tokens, 2, 4, 40, 72, dtype, 60 + tokens)
    ref, S, top = D.reference(*x, 40 ** -0.5)
    o, last = pkg.gated_delta_fwd(*x, return_last_state=True)
    D._close(o, ref, D._bar(tokens, 72, top, ref, dtype), "o")
    D._close(last, S, D._bar(tokens, 72, top, S, "f32"), "state")


def test_delta_packed_offsets_out_of_range():
    x = D.make(1, 100, 1, 2, 32, 32, "f32", 52)
    do = torch.randn(1, 100, 2, 32, generator=D._gen(53), device="cuda")
    cu = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    a, b = cu(0, 40, 100), cu(-7, 40, 1 << 30)
    assert torch.equal(pkg.gated_delta_fwd(*x, cu_seqlens=b), pkg.gated_delta_fwd(*x, cu_seqlens=a))
    want, got = pkg.gated_delta_bwd(*x, do, cu_seqlens=a), pkg.gated_delta_bwd(*x, do, cu_seqlens=b)
    assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(0, 16), (16, 0), (0, 0)])
def test_delta_heads_of_no_dims(dk, dv, dtype):
    """Sums over nothing are zeros."""
    t = lambda *s: torch.ones(*s, device="cuda", dtype=DT[dtype])  # noqa: E731
    q, v, g = t(2, 70, 2, dk), t(2, 70, 4, dv), torch.zeros(2, 70, 4, device="cuda")
    full = lambda x: torch.full_like(x, 3.0)  # noqa: E731
    o, last = pkg.gated_delta_fwd(q, q, v, g, g, o=full(v), return_last_state=True)
    assert bool((o == 0).all()) and last.shape == (2, 4, dk, dv)
    out = dict(dq=full(q), dk=full(q), dv=full(v), dg=full(g), dbeta=full(g))
    r = pkg.gated_delta_bwd(q, q, v, g, g, v, out=out)
    assert all(bool((r[n] == 0).all()) for n in out)
    o = pkg.gated_delta_step(q[:, 0], q[:, 0], v[:, 0], g[:, 0], g[:, 0], torch.zeros(2, 4, dk, dv, device="cuda"), o=full(v[:, 0]).contiguous())
    assert bool((o == 0).all())


@pytest.fixture
def large():
    """Room for tens of GB, given back afterwards."""
    free, _ = torch.cuda.mem_get_info()
    if free < 100 << 30:
        pytest.skip("needs 100 GB of free GPU memory")
    yield
    pkg.release_workspaces()
    torch.cuda.empty_cache()


def _some_heads(x, hk, rep):
    """One key head's inputs and the heads that share it."""
    q, k, v, g, beta = x
    own = slice(hk * rep, (hk + 1) * rep)
    return tuple(t.contiguous() for t in (q[:, :, hk:hk + 1], k[:, :, hk:hk + 1], v[:, :, own], g[:, :, own], beta[:, :, own])), own


def test_delta_fwd_in_passes(large):
    """Workspaces beyond 16 GiB: heads go in passes, each head as by itself (cut into other
    segments, so with other roundings; two roundings of a bf16 output)."""
    T = 65536
    x = D.make(16, T, 64, 64, 32, 32, "bf16", 70)
    o, last = pkg.gated_delta_fwd(*x, return_last_state=True)
    for head in (0, 31, 63):
        one, own = _some_heads(x, head, 1)
        want, S = pkg.gated_delta_fwd(*one, return_last_state=True)
        ref, top = want.double(), float(S.abs().amax())
        D._close(o[:, :, own], ref, 2 * D._bar(T, 32, top, ref, "bf16"), f"head {head}")
        D._close(last[:, own], S.double(), 2 * D._bar(T, 32, top, S.double(), "f32"), f"state {head}")


def test_delta_bwd_in_passes(large):
    T = 32768
    x = D.make(4, T, 20, 40, 128, 128, "bf16", 71)
    do = torch.randn(4, T, 40, 128, generator=D._gen(72), device="cuda").to(torch.bfloat16)
    r = pkg.gated_delta_bwd(*x, do)
    for hk in (0, 15, 16, 19):
        one, own = _some_heads(x, hk, 2)
        want = pkg.gated_delta_bwd(*one, do[:, :, own].contiguous())
        for n, t in want.items():
            got = r[n][:, :, hk:hk + 1] if n in ("dq", "dk") else r[n][:, :, own]
            ref = t.double()
            D._close(got, ref, 2 * D._bar(T, 128, ref.abs().amax(), ref, "bf16" if n in ("dq", "dk", "dv") else "f32", 32), f"{n} {hk}")


# ------------------------------------------------------------------ streams

def test_operators_on_other_streams():
    """On a stream given, and on the current stream of a block: each call sees what its stream did before."""
    x = D.make(2, 130, 2, 2, 32, 32, "f32", 54)
    do = torch.randn(2, 130, 2, 32, generator=D._gen(55), device="cuda")
    pos = torch.arange(130, dtype=torch.int32, device="cuda").repeat(2, 1)
    freq = torch.rand(16, generator=D._gen(56), device="cuda")
    m = torch.randn(2, 32, 130, generator=D._gen(57), device="cuda")

    def chain(stream, q, m):
        kw = {} if stream is None else {"stream": stream}
        y, mean, rstd = pkg.layer_norm_fwd(m, channels_first=True, return_stats=True, **kw)
        dn = pkg.layer_norm_bwd(m, None, mean, rstd, y, channels_first=True, **kw)
        q, k = pkg.rope_fwd(q, x[1], pos, freq, (8, 8), **kw)
        o, last = pkg.gated_delta_fwd(q, k, *x[2:], return_last_state=True, **kw)
        r = pkg.gated_delta_bwd(q, k, *x[2:], do, dh_last=last, **kw)
        s = pkg.gated_delta_step(q[:, 0], k[:, 0], *(t[:, 0] for t in x[2:]), last, **kw)
        return [y, *dn.values(), q, k, o, *r.values(), s, last]

    want = chain(None, x[0] * 2, m * 2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for given in (False, True):
        with torch.cuda.stream(side):
            busy = torch.randn(2048, 2048, device="cuda")
            for _ in range(8):
                busy = busy @ busy
            q, mm = x[0] * 2, m * 2  # (ready on the side stream only)
            got = chain(None, q, mm) if not given else None
        if given:
            got = chain(side, q, mm)
        side.synchronize()
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ the example

@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "map_mixer.py")
    spec = importlib.util.spec_from_file_location("map_mixer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _plain(m, x):
    """The block in plain 64-bit torch, with gradients."""
    p = {n: t.detach().double().requires_grad_() for n, t in m.named_parameters()}
    x = x.detach().double().requires_grad_()
    B, C, H, W = x.shape
    y = torch.nn.functional.layer_norm(x.permute(0, 2, 3, 1), (C,), p["norm_weight"], p["norm_bias"], 1e-5).flatten(1, 2)
    z, d, hk, h = y @ p["w_in"], 2 * m.pairs, m.heads_qk, m.heads
    q, k, v = z[..., :m.wide].split([hk * d, hk * d, h * m.d_v], -1)
    gate, beta = z[..., m.wide:].split(h, -1)
    axis = m.positions(range(H), W).double()
    pair = torch.cat([torch.full((s,), i) for i, s in enumerate(m.sections)]).cuda()
    ang = axis[pair].T * m.inv_freq.double()  # [cells, pairs]
    cos, sin = torch.cos(ang)[:, None], torch.sin(ang)[:, None]

    def turned(t):
        t = torch.nn.functional.normalize(t.unflatten(-1, (hk, d)), dim=-1)
        a, b = t.split(m.pairs, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).repeat_interleave(h // hk, 2)

    q, k, v = turned(q), turned(k), v.unflatten(-1, (h, m.d_v))
    g, beta = torch.exp(-0.1 * torch.nn.functional.softplus(gate)), torch.sigmoid(beta)
    S, out = torch.zeros(B, h, d, m.d_v, dtype=torch.float64, device="cuda"), []
    for t in range(H * W):
        S = g[:, t, :, None, None] * S
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, :, None]).sum(2))
        S = S + k[:, t, :, :, None] * u[:, :, None]
        out.append(d ** -0.5 * (S * q[:, t, :, :, None]).sum(2))
    o = torch.stack(out, 1)
    return p, x, x + (o.flatten(2) @ p["w_out"]).transpose(1, 2).reshape(x.shape)


def test_example_trains_like_plain_torch(example):
    """Outputs and every gradient of the block, each within 64 u sqrt(T d) of its largest value."""
    torch.manual_seed(7)
    m = example.MapMixer(24, 4, heads_qk=2, pairs=6, d_v=10)
    x = torch.randn(2, 24, 9, 11, device="cuda", requires_grad=True)
    dy = torch.randn_like(x)
    y = m(x)
    y.backward(dy)
    p, xd, yd = _plain(m, x)
    yd.backward(dy.double())
    bar = 64 * U * math.sqrt(99 * 24)
    pairs = {"y": (y.detach(), yd.detach()), "x": (x.grad, xd.grad), **{n: (t.grad, p[n].grad) for n, t in m.named_parameters()}}
    for name, (got, ref) in pairs.items():
        D._close(got, ref, bar * ref.abs().max(), name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_example_serves_what_it_trains(example, dtype):
    """Rows at once and then cell by cell give the whole map's outputs: within the bar in fp32; in
    bf16 each step's roundings (2^-9 of its values, four in a row) may fall otherwise."""
    torch.manual_seed(8)
    m = example.MapMixer(32, 4, heads_qk=2)
    x = torch.randn(2, 32, 10, 12, device="cuda").to(DT[dtype])
    with torch.no_grad():
        want = m(x).double()
    bar = 64 * U * math.sqrt(120 * 32) + (4 * 2.0 ** -7 if dtype == "bf16" else 0)
    D._close(m.serve(x, 7), want, bar * want.abs().max(), "served")


# ------------------------------------------------------------------ rows of no channels

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,cf", [((5, 0), False), ((2, 7, 0), False), ((2, 0, 7), True)])
def test_norm_of_no_channels(shape, cf, dtype):
    """Sums over nothing are zeros: the mean 0, the variance 0, so rstd = 1 / sqrt(eps)."""
    x = torch.empty(shape, dtype=DT[dtype], device="cuda")
    stale = [torch.full((s,), 3.0, device="cuda") for s in (5, 14) for _ in range(64)]  # (what an allocation without writing would show)
    del stale
    y, mean, rstd = pkg.layer_norm_fwd(x, eps=0.25, channels_first=cf, return_stats=True)
    assert y.shape == x.shape and mean.shape == (shape[:1] + shape[2:] if cf else shape[:-1])
    assert bool((mean == 0).all()) and bool((rstd == 2).all())
    r = pkg.layer_norm_bwd(x, None, mean, rstd, x, channels_first=cf)
    assert r["dx"].shape == x.shape and r["dweight"].shape == (0,)
