"""GPU tests of the recurrent block's operators where calls meet: captured and
replayed graphs (several at once), other streams, far strides, refusals of the
binding, and the example that runs them together."""
import importlib.util
import math
import os

import pytest

import selective_state_space_ssm2d_amd as pkg
import test_gpu_block_norm as N
import test_gpu_linear as L
import test_gpu_recurrence as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = L.DT


def _calls(dtype, seed):
    """Each operator once, both ways, on inputs of its own: (inputs, function of them giving a list of outputs)."""
    x, w, dy = L._randn((700, 200), dtype, seed), L._randn((96, 200), dtype, seed + 1, 0.1), L._randn((700, 96), dtype, seed + 2)
    b = torch.randn(96, generator=L._gen(seed + 3), device="cuda")
    t = N.make(600, 192, dtype, seed + 4)
    s = R.make(2, 1500, 40, dtype, seed + 5)
    m = R.make(2, 5000, 3, dtype, seed + 6, maps=True, sig=True)
    p = R.make(1, 900, 64, dtype, seed + 7, lens=[400, 0, 500])

    def linear(x, w, dy):
        y, pre = pkg.linear_fwd(x, w, b, act="silu", return_pre=True)
        return [y, *pkg.linear_bwd(x, w, dy, pre, act="silu").values()]

    def norm(x, gate, residual):
        args = {k: t[k] for k in ("weight", "scale", "next_weight")}
        return [*pkg.block_norm_fwd(x, gate=gate, residual=residual, groups=3, **args),
                *pkg.block_norm_bwd(x, t["dout"], t["dy"], gate=gate, residual=residual, groups=3, **args).values()]

    def rec(v, **kw):
        def run(x, g, dh):
            h, last = pkg.recurrence_fwd(x, g, h_init=v["h_init"], cu_seqlens=v["cu"], return_last_state=True, **kw)
            return [h, last, *pkg.recurrence_bwd(x, g, dh, h_init=v["h_init"], dh_last=v["dh_last"], cu_seqlens=v["cu"], **kw).values()]
        return run

    return {"linear": ([x, w, dy], linear), "norm": ([t["x"], t["gate"], t["residual"]], norm),
            "rows": ([s["x"], s["g"], s["dh"]], rec(s)), "maps": ([m["x"], m["g"], m["dh"]], rec(m, gates="sigmoid", channels_first=True)),
            "packed": ([p["x"], p["g"], p["dh"]], rec(p))}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", ["linear", "norm", "rows", "maps", "packed"])
def test_graphs(name, dtype):
    """Two captured graphs of a call, replayed in turn with new inputs, with eager calls of other sizes in between."""
    graphs = []
    for seed in (20, 60):
        inputs, run = _calls(dtype, seed)[name]
        run(*inputs)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(*inputs)
        graphs.append((inputs, run, g, out))
    larger = L._randn((5000, 300), dtype, 1), L._randn((300, 300), dtype, 2, 0.05)
    for turn in range(3):
        for inputs, run, g, out in graphs:
            for i, t in enumerate(inputs):
                t.copy_(t.roll(turn + i + 1, 0) if name != "packed" else t.flip(1))
            g.replay()
        pkg.linear_bwd(*larger, larger[0], None)
        torch.cuda.synchronize()
        for inputs, run, g, out in graphs:
            want = run(*inputs)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (name, turn)


@pytest.mark.parametrize("name", ["linear", "norm", "rows", "maps", "packed"])
def test_streams_at_once(name):
    inputs, run = _calls("bf16", 30)[name]
    want = run(*inputs)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(run(*inputs))
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_stream_argument():
    x, w = L._randn((500, 512), "bf16", 1), L._randn((64, 512), "bf16", 2)
    t, s = N.make(100, 96, "bf16", 3), R.make(1, 900, 32, "bf16", 4)
    want = [pkg.linear_fwd(x, w), pkg.linear_bwd(x, w, x[:, :64].contiguous())["dweight"], pkg.block_norm_fwd(t["x"]),
            pkg.block_norm_bwd(t["x"], t["dout"], weight=t["weight"])["dweight"], pkg.recurrence_fwd(s["x"], s["g"]),
            pkg.recurrence_bwd(s["x"], s["g"], s["dh"])["dg"], pkg.recurrence_step(s["x"][:, 0], s["g"][:, 0], s["h_init"].clone())]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    state = s["h_init"].clone()
    dy = x[:, :64].contiguous()
    torch.cuda.synchronize()
    got = [pkg.linear_fwd(x, w, stream=st), pkg.linear_bwd(x, w, dy, stream=st)["dweight"], pkg.block_norm_fwd(t["x"], stream=st),
           pkg.block_norm_bwd(t["x"], t["dout"], weight=t["weight"], stream=st)["dweight"], pkg.recurrence_fwd(s["x"], s["g"], stream=st),
           pkg.recurrence_bwd(s["x"], s["g"], s["dh"], stream=st)["dg"], pkg.recurrence_step(s["x"][:, 0], s["g"][:, 0], state, stream=st)]
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def _spread(t, strides):
    """t's values in a view of the given strides."""
    size = 1 + sum((s - 1) * st for s, st in zip(t.shape, strides))
    return torch.empty(size, dtype=t.dtype, device="cuda").as_strided(t.shape, strides).copy_(t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_far_strides(dtype):
    """Offsets past 31 bits give what dense tensors give."""
    x, w = L._randn((5, 64), dtype, 1), L._randn((24, 64), dtype, 2)
    far = (1 << 29) + 8
    assert torch.equal(pkg.linear_fwd(_spread(x, (far, 1)), w), pkg.linear_fwd(x, w))
    g = pkg.linear_bwd(_spread(x, (far, 1)), w, x[:, :24])
    want = pkg.linear_bwd(x, w, x[:, :24].contiguous())
    assert all(torch.equal(g[k], want[k]) for k in want)
    m = L._randn((2, 20, 72), dtype, 3)
    assert torch.equal(pkg.linear_fwd(_spread(m, (1 << 31, 72, 1)), w[:, :20], channels_first=True), pkg.linear_fwd(m, w[:, :20], channels_first=True))
    assert torch.equal(pkg.linear_fwd(_spread(m[:1], (0, 1 << 27, 1)), w[:, :20], channels_first=True),
                       pkg.linear_fwd(m[:1], w[:, :20], channels_first=True))
    t = N.make(4, 64, dtype, 4)
    assert torch.equal(pkg.block_norm_fwd(_spread(t["x"], (1 << 30, 1)), t["weight"]), pkg.block_norm_fwd(t["x"], t["weight"]))
    s = R.make(1, 20, 40, dtype, 5)
    st = (1 << 27) + 8
    assert torch.equal(pkg.recurrence_fwd(_spread(s["x"], (0, st, 1)), s["g"]), pkg.recurrence_fwd(s["x"], s["g"]))
    assert torch.equal(pkg.recurrence_fwd(_spread(s["x"], (0, st, 1)), s["g"], reverse=True), pkg.recurrence_fwd(s["x"], s["g"], reverse=True))


def test_guard_bands():
    """Nothing is written around outputs of odd sizes."""
    def inside(shape, dtype):
        n = math.prod(shape)
        buf = torch.full((n + 512,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[256:256 + n].view(shape)

    for dtype in ("f32", "bf16"):
        dt = DT[dtype]
        for rows, k, n in ((65, 33, 67), (129, 72, 200), (3, 100, 50), (1, 16, 24)):
            x, w = L._randn((rows, k), dtype, 1), L._randn((n, k), dtype, 2)
            buf, y = inside((rows, n), dt)
            pkg.linear_fwd(x, w, y=y)
            bufs = {"dx": inside((rows, k), dt), "dweight": inside((n, k), dt), "dbias": inside((n,), torch.float32)}
            pkg.linear_bwd(x, w, y, out={a: b[1] for a, b in bufs.items()})
            for b in [buf] + [v[0] for v in bufs.values()]:
                assert (b[:256] == 7).all() and (b[-256:] == 7).all()
        t = N.make(7, 101, dtype, 3)
        bufs = {"out": inside((7, 101), dt), "y": inside((7, 101), dt)}
        pkg.block_norm_fwd(t["x"], next_weight=t["next_weight"], **{a: b[1] for a, b in bufs.items()})
        s = R.make(1, 333, 21, dtype, 4)
        bufs["h"], bufs["dx"], bufs["dg"] = (inside((1, 333, 21), dt) for _ in range(3))
        pkg.recurrence_fwd(s["x"], s["g"], h=bufs["h"][1])
        pkg.recurrence_bwd(s["x"], s["g"], s["dh"], out={a: bufs[a][1] for a in ("dx", "dg")})
        for b, _ in bufs.values():
            assert (b[:256] == 7).all() and (b[-256:] == 7).all()


def test_refusals():
    x, w, b = L._randn((4, 16), "bf16", 1), L._randn((8, 16), "bf16", 2), torch.zeros(8, device="cuda")
    y = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(2, 16, 5, dtype=torch.bfloat16, device="cuda")
    s = torch.zeros(2, 6, 16, device="cuda")
    st, cu = torch.zeros(2, 16, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    f = torch.zeros(4, 16, device="cuda")
    for call in (lambda: pkg.linear_fwd(x, w.float()), lambda: pkg.linear_fwd(x, w[:, :8]), lambda: pkg.linear_fwd(x, w, b.bfloat16()),
                 lambda: pkg.linear_fwd(x, w, b[:4]), lambda: pkg.linear_fwd(x, w, act="tanh"), lambda: pkg.linear_fwd(x, w, residual=y.float()),
                 lambda: pkg.linear_fwd(x, w, residual=y[:2]), lambda: pkg.linear_fwd(x.t(), w), lambda: pkg.linear_fwd(x, w.t().contiguous().t()),
                 lambda: pkg.linear_fwd(x, w, out_channels_first=True), lambda: pkg.linear_fwd(x, w, y=y.t()), lambda: pkg.linear_fwd(x, w.cpu()),
                 lambda: pkg.linear_fwd(m.transpose(1, 2), w, channels_first=True), lambda: pkg.linear_bwd(x, w, y, act="silu"),
                 lambda: pkg.linear_bwd(x, w, y, y.float(), act="silu"), lambda: pkg.linear_bwd(x, w, y.float()), lambda: pkg.linear_bwd(x, w, y[:2]),
                 lambda: pkg.linear_bwd(x, w, y, out={"dx": f}),
                 lambda: pkg.block_norm_fwd(f, groups=3), lambda: pkg.block_norm_fwd(f, groups=0), lambda: pkg.block_norm_fwd(f, gate_act="relu"),
                 lambda: pkg.block_norm_fwd(f, b), lambda: pkg.block_norm_fwd(f, gate=x), lambda: pkg.block_norm_fwd(f, residual=x),
                 lambda: pkg.block_norm_fwd(f, torch.ones(16, device="cuda"), norm=False), lambda: pkg.block_norm_fwd(f, y=f),
                 lambda: pkg.block_norm_fwd(f, out_dtype=torch.bfloat16), lambda: pkg.block_norm_bwd(f, None), lambda: pkg.block_norm_bwd(f, f, f),
                 lambda: pkg.block_norm_bwd(x, f, residual=x), lambda: pkg.block_norm_fwd(f[:, ::2]),
                 lambda: pkg.recurrence_fwd(s, s.bfloat16()), lambda: pkg.recurrence_fwd(s, s[:, :3]), lambda: pkg.recurrence_fwd(s, s, gates="x"),
                 lambda: pkg.recurrence_fwd(s, s, h_init=st[:1]), lambda: pkg.recurrence_fwd(s, s, cu_seqlens=cu),
                 lambda: pkg.recurrence_fwd(s[:1], s[:1], cu_seqlens=cu, reverse=True), lambda: pkg.recurrence_fwd(s[:1], s[:1], cu_seqlens=cu.long()),
                 lambda: pkg.recurrence_fwd(s[:1], s[:1], cu_seqlens=cu, channels_first=True), lambda: pkg.recurrence_fwd(s[..., ::2], s[..., ::2]),
                 lambda: pkg.recurrence_bwd(s, s, s[:, :2]), lambda: pkg.recurrence_bwd(s, s, s, dh_last=st.double()), lambda: pkg.recurrence_step(s, s, st),
                 lambda: pkg.recurrence_step(st, st, None), lambda: pkg.recurrence_step(st, st, st[:1]), lambda: pkg.recurrence_fwd(s, s.cpu())):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(pkg.Ssm2dError):
        pkg.block_norm_fwd(torch.zeros(1, pkg.block.NORM_MAX_N + 1, device="cuda"))


# ------------------------------------------------------------------ together

@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_block.py")
    spec = importlib.util.spec_from_file_location("recurrent_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _plain(model, x):
    """The example's forward in torch calls of x's type."""
    def rms(v, groups=1):
        u = v.unflatten(-1, (groups, -1))
        return (u / torch.sqrt((u * u).mean(-1, keepdim=True) + 1e-5)).flatten(-2)

    p = {k: v for k, v in model.items()}
    e = torch.nn.functional.silu(x.flatten(2).transpose(1, 2) @ p["embed"].t() + p["embed_bias"])
    stream, n = e, len({k.split(".")[1] for k in p if k.startswith("blocks.")})
    y = rms(stream) * p["blocks.0.pre"]
    for i in range(n):
        b = {k: p[f"blocks.{i}.{k}"] for k in ("pre", "post", "head", "scale", "w_in", "b_in", "w_out")}
        u, g, z = (y @ b["w_in"].t() + b["b_in"]).chunk(3, -1)
        a, h, hs = torch.sigmoid(g), torch.zeros_like(u[:, 0]), []
        for t in range(u.shape[1]):
            h = a[:, t] * h + (1 - a[:, t]) * u[:, t]
            hs.append(h)
        o = (rms(torch.stack(hs, 1), 4) * b["head"] * torch.nn.functional.silu(z)) @ b["w_out"].t()
        stream = stream + b["scale"] * rms(o) * b["post"]
        y = rms(stream) * (p[f"blocks.{i + 1}.pre"] if i + 1 < n else p["last"])
    return x + (y @ p["readout"].t()).transpose(1, 2).reshape(x.shape)


def test_example_against_64_bits(example):
    torch.manual_seed(1)
    model = example.RecurrentBlocks(24, 64, 2)
    x = torch.randn(2, 24, 5, 7, device="cuda")
    dy = torch.randn_like(x)
    y = model(x)
    (y * dy).sum().backward()
    params = {k: v.detach().double().cpu().requires_grad_(True) for k, v in model.named_parameters()}
    want = _plain(params, x.double().cpu())
    (want * dy.double().cpu()).sum().backward()
    # (fp32 through two blocks: sums of up to 64 terms and 35 tokens, and what two norms in a row do to them)
    assert (y.double().cpu() - want).abs().max() <= 1e-4
    for k, v in model.named_parameters():
        g = params[k].grad
        assert (v.grad.double().cpu() - g).norm() <= 1e-4 * g.norm() + 1e-6, k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_example_serves_what_it_trains(example, dtype):
    torch.manual_seed(2)
    model = example.RecurrentBlocks(32, 64, 2)
    x = torch.randn(2, 32, 6, 8, device="cuda").to(DT[dtype])
    with torch.no_grad():
        full = model(x).float()
    # (fp32: other orders of the same sums; bf16: roundings on the other side, each up to 2^-7 of values of a few units)
    assert (model.serve(x, 4).float() - full).abs().max() <= (1e-4 if dtype == "f32" else 0.15)
