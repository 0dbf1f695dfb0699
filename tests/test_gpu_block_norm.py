"""GPU tests of the block norm (include/ssm2d_block.h) against 64 bits.

Bars. Every output is a sum of products, computed in fp32 with at most K = 160
roundings on any path (three rounds of sums of at most 40 additions a lane and
its levels, and about 40 operations around them; a sigmoid's exp adds 2 |z|), so
it errs by at most (K + 2 |z|) 2^-24 of the same formula with every term taken by
its magnitude; a bf16 output rounds once more, 2^-8 of the value."""
import pytest

import selective_state_space_ssm2d_amd as pkg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, dtype, seed):
    return torch.randn(*shape, generator=_gen(seed), device="cuda").to(DT[dtype])


def _near(got, want, bar, what):
    bad = ~((got.double() - want).abs() <= bar + 1e-30)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {((got.double() - want).abs() / (bar + 1e-30)).max().item():.2f} bars"


def _half(v, dtype):
    return v.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else U)


def make(rows, n, dtype, seed, gate=True, res=True, weight=True, scale=True, nxt=True, rf32=False):
    rt = "f32" if rf32 else dtype
    p = lambda s, a: (1 + a * torch.randn(n, generator=_gen(s), device="cuda"))  # noqa: E731
    spread = torch.exp(0.5 * torch.randn(n, generator=_gen(seed + 9), device="cuda"))
    return {"x": (_randn((rows, n), "f32", seed) * spread).to(DT[dtype]), "gate": _randn((rows, n), dtype, seed + 1) if gate else None,
            "residual": _randn((rows, n), rt, seed + 2) if res else None, "weight": p(seed + 3, 0.2) if weight else None,
            "scale": 0.5 * p(seed + 4, 0.3) if scale else None, "next_weight": p(seed + 5, 0.2) if nxt else None,
            "dout": _randn((rows, n), rt, seed + 6), "dy": _randn((rows, n), dtype, seed + 7) if nxt else None}


def formula(t, norm, groups, act, first, mag=False):
    """The forward and its gradients in 64 bits; `mag`: with every term by its
    magnitude (the rms and the gates' factors are what they are)."""
    o = {}
    d = {k: v.double() if v is not None else None for k, v in t.items()}
    z = d["gate"]
    s = torch.sigmoid(z) if z is not None else None
    a = None if z is None else (s if act == "sigmoid" else z * s)
    da_dz = None if z is None else (s * (1 - s) if act == "sigmoid" else s * (1 + z * (1 - s)))
    n = d["x"].shape[-1]
    grp = lambda v: v.unflatten(-1, (groups, n // groups))  # noqa: E731
    one = torch.ones(n, dtype=torch.float64, device="cuda")
    w, sc, nw = (d[k] if d[k] is not None else one for k in ("weight", "scale", "next_weight"))
    x, res = d["x"], d["residual"] if d["residual"] is not None else torch.zeros_like(d["x"])
    u = x * a if z is not None and first else x
    r = grp(torch.zeros_like(u)) + 1 / torch.sqrt((grp(u) ** 2).mean(-1, keepdim=True) + EPS) if norm else None
    r = r.flatten(-2) if norm else 1.0
    m = u * r * w if norm else u
    if z is not None and not first:
        m = m * a
    out = res + sc * m
    r2 = 1 / torch.sqrt((out ** 2).mean(-1, keepdim=True) + EPS)
    sign = 1.0
    if mag:
        x, res, w, sc, nw, u, m = (v.abs() for v in (x, res, w, sc, nw, u, m))
        a, da_dz = (None, None) if z is None else (a.abs(), s * (1 + z.abs()))
        out = res + sc * m
        sign = -1.0
        d["dout"] = d["dout"].abs() if d["dout"] is not None else None
        d["dy"] = d["dy"].abs() if d["dy"] is not None else None
    o["out"] = out
    D = d["dout"] if d["dout"] is not None else torch.zeros_like(x)
    if d["next_weight"] is not None:
        o["y"] = out * r2 * nw * (1 if not mag else 1 + r2 * r2 * (out * out).mean(-1, keepdim=True))
        if d["dy"] is not None:
            xh, gw = out * r2, d["dy"] * nw
            o["dnext_weight"] = (d["dy"] * xh).sum(0)
            D = D + r2 * (gw - sign * xh * (gw * xh).mean(-1, keepdim=True))
            if mag:  # (an error of out passes through rms(out) again)
                D = D * (1 + (r2 * r2 * (out * out).mean(-1, keepdim=True)))
    o["dresidual"] = D
    o["dscale"] = (D * m).sum(0)
    D = D * sc
    nn = u * r * w if norm else u
    if z is not None and not first:
        da, D = D * nn, D * a
    if norm:
        xh = u * r
        o["dweight"] = (D * xh).sum(0)
        gw = D * w
        D = r * (gw - sign * (grp(xh) * grp(gw * xh).mean(-1, keepdim=True)).flatten(-2))
    if z is not None and first:
        da, D = D * x, D * a
    o["dx"] = D
    if z is not None:
        o["dgate"] = da * da_dz
    return o


def check(t, norm=True, groups=1, act="silu", first=False, what="", views=None):
    args = {k: t[k] for k in ("weight", "gate", "residual", "scale", "next_weight")}
    args.update(norm=norm, groups=groups, gate_act=act, gate_first=first, eps=EPS)
    rt = t["residual"].dtype if t["residual"] is not None else t["dout"].dtype
    r = pkg.block_norm_fwd(t["x"], **args, out_dtype=rt)
    got = dict(zip(("out", "y"), r)) if t["next_weight"] is not None else {"out": r}
    got.update(pkg.block_norm_bwd(t["x"], t["dout"], t["dy"], **args))
    want, mag = formula(t, norm, groups, act, first), formula(t, norm, groups, act, first, mag=True)
    rows = t["x"].shape[0]
    zmax = t["gate"].abs().max().item() if t["gate"] is not None else 0.0
    for name, g in got.items():
        k = 160 + 2 * zmax + (rows if g.dim() == 1 else 0)
        if name not in want:  # (no dy: no gradient of the norm that it comes through)
            assert name == "dnext_weight" and not g.any()
            continue
        assert g.dtype == (torch.float32 if g.dim() == 1 else (rt if name in ("out", "dresidual") else t["x"].dtype)), name
        _near(g, want[name], k * U * mag[name] + _half(want[name], g.dtype), f"{what} {name}")


SIZES = [(1, 1), (1, 768), (3, 7), (5, 64), (9, 100), (4, 511), (4, 512), (6, 513), (3, 768), (7, 771), (3, 1024), (2, 1025), (3, 2048), (2, 2056),
         (2, 4096), (2, 4099), (2, 8192), (1, 8200), (2, 16384), (1, 16383)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", SIZES)
def test_sizes(rows, n, dtype):
    check(make(rows, n, dtype, rows + n), what=f"{rows}x{n}")
    check(make(rows, n, dtype, rows + n, rf32=True), first=True, act="sigmoid", what=f"{rows}x{n} first")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("off", ["", "gate", "res", "weight", "scale", "nxt", "gate res", "gate res weight scale", "gate res weight scale nxt"])
def test_parts(off, first, norm, dtype):
    t = make(11, 96, dtype, 5, **{k: False for k in off.split()})
    if not norm:
        t["weight"] = None
    check(t, norm=norm, first=first, what=off)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,groups", [(768, 12), (768, 6), (768, 8), (96, 96), (96, 3), (96, 4), (99, 33), (771, 3), (1024, 2), (1024, 1024), (2048, 16), (1536, 2),
                                      (4096, 64), (4096, 8), (16384, 4), (16383, 3), (16384, 128), (15360, 5)])
def test_groups(n, groups, dtype):
    check(make(6, n, dtype, n + groups), groups=groups, what=f"{n}/{groups}")
    check(make(5, n, dtype, n + groups, rf32=True), groups=groups, first=True, act="sigmoid", what=f"{n}/{groups} first")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", [(2500, 96), (3001, 200), (1030, 1030), (700, 2048), (300, 9000), (20000, 16)])
def test_many_rows(rows, n, dtype):
    check(make(rows, n, dtype, 3), what=f"{rows}x{n}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides(dtype):
    base = make(40, 400, dtype, 1)
    for lo, n in ((0, 64), (8, 256), (3, 100), (4, 96)):
        t = {k: (v[:, lo:lo + n] if v is not None and v.dim() == 2 else v[lo:lo + n].contiguous() if v is not None else None) for k, v in base.items()}
        check(t, what=f"columns from {lo}")
        check({k: (v[::3] if v is not None and v.dim() == 2 else v) for k, v in t.items()}, what=f"every third row, columns from {lo}")
    t = dict(base, gate=base["gate"][:1].expand(40, 400), residual=base["residual"][:1].expand(40, 400), dy=base["dy"][:1].expand(40, 400))
    check(t, what="one row for all")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_zeros_and_large_values(dtype):
    t = make(5, 96, dtype, 1)
    for name in ("x", "residual", "gate"):
        check(dict(t, **{name: torch.zeros_like(t[name])}), what=f"{name} 0")
    check(dict(t, x=torch.zeros_like(t["x"]), residual=torch.zeros_like(t["residual"])), what="all 0")
    check(dict(t, gate=(t["gate"].float() * 40).to(t["gate"].dtype)), what="large gates")
    check(dict(t, x=(t["x"].float() * 1e6).to(t["x"].dtype)), what="large x")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_not_finite_stays_in_its_row(bad, dtype):
    t = make(9, 200, dtype, 1)
    args = {k: t[k] for k in ("weight", "gate", "residual", "scale", "next_weight")}
    run = lambda: (*pkg.block_norm_fwd(t["x"], **args), *(pkg.block_norm_bwd(t["x"], t["dout"], t["dy"], **args)[k] for k in ("dx", "dgate", "dresidual")))  # noqa: E731
    want = run()
    for name in ("x", "gate", "residual"):
        keep = t[name].clone()
        t[name][4, 199] = bad
        got = run()
        t[name].copy_(keep)
        rows = torch.arange(9, device="cuda") != 4
        for a, b in zip(got, want):
            assert torch.equal(a[rows], b[rows]), name


def test_leading_dims_in_place_and_missing_gradients():
    t = make(12, 64, "bf16", 1)
    args = {k: t[k] for k in ("weight", "scale", "next_weight")}
    want = pkg.block_norm_fwd(t["x"], gate=t["gate"], residual=t["residual"], **args)
    shaped = [t[k].view(2, 2, 3, 64) for k in ("x", "gate", "residual")]
    got = pkg.block_norm_fwd(shaped[0], gate=shaped[1], residual=shaped[2], **args)
    assert got[0].shape == (2, 2, 3, 64) and all(torch.equal(a.flatten(0, 2), b) for a, b in zip(got, want))
    r = t["residual"].clone()
    out, y = pkg.block_norm_fwd(t["x"], gate=t["gate"], residual=r, out=r, **args)
    assert out is r and torch.equal(r, want[0]) and torch.equal(y, want[1])
    check(dict(t, dy=None), what="no dy")
    zero = pkg.block_norm_bwd(t["x"], torch.zeros_like(t["dout"]), t["dy"], gate=t["gate"], residual=t["residual"], **args)
    none = pkg.block_norm_bwd(t["x"], None, t["dy"], gate=t["gate"], residual=t["residual"], **args)
    assert all(torch.equal(zero[k], none[k]) for k in zero)


def test_empty():
    x, w = torch.zeros(0, 8, device="cuda"), torch.ones(8, device="cuda")
    out, y = pkg.block_norm_fwd(x, w, next_weight=w)
    assert out.shape == (0, 8) and y.shape == (0, 8)
    g = pkg.block_norm_bwd(x, x, x, w, scale=w, next_weight=w, out={k: torch.full((8,), 3.0, device="cuda") for k in ("dweight", "dscale", "dnext_weight")})
    assert all(not g[k].any() for k in ("dweight", "dscale", "dnext_weight"))
    assert pkg.block_norm_fwd(torch.zeros(4, 0, device="cuda")).shape == (4, 0)


@pytest.mark.parametrize("first", [False, True])
def test_gradients_against_differences(first):
    t = make(4, 12, "f32", 2)
    names = ("x", "gate", "residual", "weight", "scale", "next_weight")
    g = pkg.block_norm_bwd(t["x"], t["dout"], t["dy"], **{k: t[k] for k in names[1:]}, groups=3, gate_first=first)
    f = lambda d: sum((formula({**t, **d}, True, 3, "silu", first)[o] * t[k].double()).sum() for o, k in (("out", "dout"), ("y", "dy")))  # noqa: E731
    for k in names:
        d, h = torch.randn(t[k].shape, generator=_gen(8), device="cuda").double(), 1e-6
        slope = (f({k: t[k].double() + h * d}) - f({k: t[k].double() - h * d})) / (2 * h)
        got = g["d" + k].double() * d
        assert abs(got.sum() - slope) <= 1e-5 * got.abs().sum() + 1e-7, k


def test_deterministic():
    t = make(5000, 768, "bf16", 1)
    args = {k: t[k] for k in ("weight", "gate", "residual", "scale", "next_weight")}
    a, b = (pkg.block_norm_bwd(t["x"], t["dout"], t["dy"], **args) for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
def test_weight_without_the_norm_is_left_out(gate, dtype):
    """The C entries, given a weight without SSM2D_NORM_ON: as without the weight, whose gradient is zeros."""
    from selective_state_space_ssm2d_amd import block

    t = make(9, 200, dtype, 1, gate=gate)
    stream = torch.cuda.current_stream().cuda_stream
    ptr = lambda k: t[k].data_ptr() if t[k] is not None else None  # noqa: E731
    args = (False, 1, False, False)
    fn, _, s, flags, _, _, _ = block._norm_plan(False, t["x"], None, t["gate"], t["residual"], t["scale"], t["next_weight"], *args, None, None)
    want = pkg.block_norm_fwd(t["x"], gate=t["gate"], residual=t["residual"], scale=t["scale"], next_weight=t["next_weight"], norm=False)
    out, y = torch.empty_like(t["residual"]), torch.empty_like(t["x"])
    assert fn(t["x"].data_ptr(), ptr("gate"), ptr("residual"), ptr("weight"), ptr("scale"), ptr("next_weight"), out.data_ptr(), y.data_ptr(), s, EPS, flags,
              stream) == 0
    assert torch.equal(out, want[0]) and torch.equal(y, want[1])
    fn, _, s, flags, need, _, _ = block._norm_plan(True, t["x"], None, t["gate"], t["residual"], t["scale"], t["next_weight"], *args, t["dout"], t["dy"])
    want = pkg.block_norm_bwd(t["x"], t["dout"], t["dy"], gate=t["gate"], residual=t["residual"], scale=t["scale"], next_weight=t["next_weight"], norm=False)
    like = {"dx": t["x"], "dgate": t["gate"], "dresidual": t["residual"], "dweight": t["weight"], "dscale": t["scale"], "dnext_weight": t["next_weight"]}
    got = {k: torch.full_like(v, 7.0) if v is not None else None for k, v in like.items()}
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert fn(t["x"].data_ptr(), ptr("gate"), ptr("residual"), ptr("weight"), ptr("scale"), ptr("next_weight"), ptr("dout"), ptr("dy"),
              *(v.data_ptr() if v is not None else None for v in got.values()), s, EPS, flags, work.data_ptr(), need, stream) == 0
    for k, v in want.items():
        assert torch.equal(got[k], v), k
    assert not got["dweight"].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,groups", [(768, 12), (768, 6), (96, 3), (40, 5), (200, 25), (1536, 24), (4096, 64), (100, 1), (771, 3)])
def test_eps_of_zero(n, groups, dtype, monkeypatch):
    """No eps: lanes that hold nothing of the row (pieces behind it) do not reach what the row sums."""
    monkeypatch.setitem(globals(), "EPS", 0.0)
    for nxt in (True, False):
        check(make(7, n, dtype, n + groups, nxt=nxt), groups=groups, what=f"{n}/{groups}")
        check(make(5, n, dtype, n + groups, nxt=nxt, rf32=True), groups=groups, first=True, act="sigmoid", what=f"{n}/{groups} first")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [96, 771, 2048])
def test_gradients_of_values_that_are_not_finite(n, dtype):
    """Without the norm a gradient is dout by the scale, whatever x holds; and
    without dy nothing is taken from the norm before the next block."""
    t = make(6, n, dtype, 2, gate=False, weight=False)
    t["x"][1, 3], t["x"][2, n - 1], t["x"][4, 0] = float("nan"), float("inf"), float("-inf")
    g = pkg.block_norm_bwd(t["x"], t["dout"], None, residual=t["residual"], scale=t["scale"], next_weight=t["next_weight"], norm=False)
    want = t["dout"].double() * t["scale"].double()
    _near(g["dx"], want, U * want.abs() + _half(want, g["dx"].dtype), "dx")
    assert torch.equal(g["dresidual"], t["dout"]) and not g["dnext_weight"].any()
    # through y rows that hold such a value are lost, the others are not
    g = pkg.block_norm_bwd(t["x"], t["dout"], t["dy"], residual=t["residual"], scale=t["scale"], next_weight=t["next_weight"], norm=False)
    keep = torch.tensor([0, 3, 5], device="cuda")
    assert all(torch.isfinite(g[k][keep]).all() for k in ("dx", "dresidual"))
