"""GPU tests of linear (include/ssm2d_block.h) against 64 bits: layouts, types,
activations, odd sizes and strides, gradients.

Bars. A bf16 output is off by its rounding (2^-8 of the value) and the fp32 sum
before it; products of bf16 are exact, so a sum of k terms errs by at most
(k + 2) 2^-24 of the sum of their magnitudes. A float32 product drops the three
smallest of nine partial products: parts cut off after 8 bits leave remainders
under 2^-7 and 2^-15 of the value, so that is under 2^-21 of a term; the six kept
ones are 6 k additions. An activation passes an error on by its slope (at most
1.13) and adds its own: sigmoid and erf by a few roundings, exp's argument |z| of
them, erf's published approximation 1.5e-7 for bf16."""
import math

import pytest

import selective_state_space_ssm2d_amd as pkg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(shape, dtype, seed, scale=1.0):
    return (scale * torch.randn(*shape, generator=_gen(seed), device="cuda")).to(DT[dtype])


def _act(z, act):
    return {None: lambda v: v, "relu": lambda v: v.clamp_min(0), "silu": lambda v: v * torch.sigmoid(v),
            "gelu": lambda v: 0.5 * v * torch.erfc(-v / math.sqrt(2))}[act](z)


def _slope(z, act):
    s = torch.sigmoid(z)
    return {None: torch.ones_like, "relu": lambda v: (v > 0).double(), "silu": lambda v: s * (1 + v * (1 - s)),
            "gelu": lambda v: 0.5 * torch.erfc(-v / math.sqrt(2)) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)}[act](z)


def _sum_bar(k, dtype):
    """The error of a sum of k products, relative to the sum of their magnitudes."""
    return (k + 2) * U if dtype == "bf16" else (6 * k + 2) * U + 2.0 ** -21


def _half(v, dtype):
    return v.abs() * (2.0 ** -8 if dtype == "bf16" else U)


def _near(got, want, bar, what):
    got = got.double()
    bad = ~((got - want).abs() <= bar + 1e-30)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {((got - want).abs() / (bar + 1e-30)).max().item():.2f} bars"


def _rows(t, maps):
    """[..., rows, channels] of a tensor in either layout."""
    return t.flatten(2).transpose(1, 2) if maps else t


def check(x, w, b=None, res=None, act=None, cf=False, ocf=None, dtype="bf16", dy=None, what=""):
    ocf = cf if ocf is None else ocf
    k, n = w.shape[1], w.shape[0]
    y, pre = pkg.linear_fwd(x, w, b, res, act=act, channels_first=cf, out_channels_first=ocf, return_pre=True)
    xr, w64 = _rows(x, cf).double(), w.double()
    z = xr @ w64.t() + (b.double() if b is not None else 0.0)
    mag = xr.abs() @ w64.t().abs() + (b.double().abs() if b is not None else 0.0)
    zbar = _sum_bar(k + 1, dtype) * mag
    _near(_rows(pre, ocf), z, zbar + _half(z, dtype), what + " pre")
    want = _act(z, act)
    bar = 1.13 * zbar + (0.0 if act in (None, "relu") else (z * z + 10 * z.abs()) * 2.0 ** -23)
    if res is not None:
        want = want + _rows(res, ocf).double()
        bar = bar + U * want.abs()
    _near(_rows(y, ocf), want, bar + _half(want, dtype), what + " y")
    if dy is None:
        return
    g = pkg.linear_bwd(x, w, dy, pre if act else None, act=act, bias=True, channels_first=cf, out_channels_first=ocf)
    zz, up = _rows(pre, ocf).double(), _rows(dy, ocf).double()
    dz = up * _slope(zz, act)
    # dz's own error: the slope's, and its rounding for the products
    own = up.abs() * (0.0 if act in (None, "relu") else 1.0) * (zz * zz + 10 * zz.abs() + 4) * 2.0 ** -23
    rnd = own + (_half(dz, dtype) if act else 0.0)
    dx = dz @ w64
    bar = rnd @ w64.abs() + _sum_bar(n, dtype) * ((dz.abs() + rnd) @ w64.abs()) + _half(dx, dtype)
    _near(_rows(g["dx"], cf), dx, bar, what + " dx")
    flat, fx, fr = dz.reshape(-1, n), xr.reshape(-1, k), (rnd + dz * 0).reshape(-1, n)
    dw = flat.t() @ fx
    bar = fr.t() @ fx.abs() + _sum_bar(flat.shape[0], dtype) * ((flat.abs() + fr).t() @ fx.abs()) + _half(dw, dtype)
    _near(g["dweight"], dw, bar, what + " dweight")
    db = flat.sum(0)
    _near(g["dbias"], db, own.reshape(-1, n).sum(0) + (flat.shape[0] + 2) * U * flat.abs().sum(0), what + " dbias")


def case(batch, rows, k, n, cf, ocf, act, res, dtype, seed, bias=True):
    mixed = cf or ocf
    xs = (batch, k, rows) if cf else ((batch, rows, k) if mixed or batch > 1 else (rows, k))
    ys = (batch, n, rows) if ocf else ((batch, rows, n) if mixed or batch > 1 else (rows, n))
    x, w = _randn(xs, dtype, seed), _randn((n, k), dtype, seed + 1, max(k, 1) ** -0.5)
    b = torch.randn(n, generator=_gen(seed + 2), device="cuda") if bias else None
    r = _randn(ys, dtype, seed + 3) if res else None
    check(x, w, b, r, act, cf, ocf, dtype, _randn(ys, dtype, seed + 4), f"{batch}x{rows}x{k}->{n} cf={cf} ocf={ocf} {act} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,k,n", [(1, 1, 1), (1, 8, 16), (3, 7, 5), (17, 33, 129), (64, 64, 64), (65, 63, 127), (128, 72, 136), (130, 100, 196),
                                      (257, 768, 96)])
def test_rows(rows, k, n, dtype):
    case(1, rows, k, n, False, False, "silu", True, dtype, rows + k)
    case(1, rows, k, n, False, False, None, False, dtype, rows + n, bias=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cf,ocf", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("batch,rows,k,n", [(1, 1, 3, 2), (2, 49, 40, 24), (3, 196, 64, 96), (2, 200, 33, 65), (1, 1024, 128, 128), (5, 131, 96, 17)])
def test_maps(batch, rows, k, n, cf, ocf, dtype):
    case(batch, rows, k, n, cf, ocf, "gelu", True, dtype, rows + k + n)
    case(batch, rows, k, n, cf, ocf, None, False, dtype, rows + k, bias=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu"])
def test_activations(act, dtype):
    case(1, 100, 48, 80, False, False, act, False, dtype, 7)
    x = torch.cat([torch.linspace(-30, 30, 601), torch.tensor([0.0, -0.0, 1e-8, 100.0, -100.0])]).to(DT[dtype]).cuda()[:, None]
    check(x, torch.ones(1, 1, dtype=DT[dtype], device="cuda"), act=act, dtype=dtype, dy=torch.ones_like(x), what=f"values {act}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,k,n", [(2, 4096, 64), (1, 2048, 1000), (16, 1000, 72), (700, 4100, 40), (4097, 16, 24), (20000, 24, 16), (2200, 1024, 1100)])
def test_long(rows, k, n, dtype):
    """Long sums that are split, many rows, and sizes of the larger tile."""
    case(1, rows, k, n, False, False, "silu", True, dtype, 11)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", range(1, 20))
def test_each_small_row_count(rows, dtype):
    for k, n in ((768, 200), (520, 33), (100, 64), (1025, 16)):
        x, w = _randn((rows, k), dtype, rows), _randn((n, k), dtype, k, k ** -0.5)
        b = torch.randn(n, generator=_gen(2), device="cuda")
        check(x, w, b, _randn((rows, n), dtype, 3), "silu", dtype=dtype, what=f"{rows} {k} {n}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strides(dtype):
    x = _randn((70, 100), dtype, 1)
    w = _randn((48, 90), dtype, 2, 0.1)
    b = torch.randn(48, generator=_gen(3), device="cuda")
    dy = _randn((70, 96), dtype, 4)
    for x0, k, wk in ((8, 64, 64), (3, 64, 64), (0, 61, 61), (4, 88, 88)):
        check(x[:, x0:x0 + k], w[:, :wk], b, dy[:, 7:55], "relu", dtype=dtype, dy=dy[:, 40:88], what=f"from {x0}")
        check(x[::2, x0:x0 + k], w[::3, 90 - wk:], b[:16].contiguous(), None, None, dtype=dtype, dy=dy[::2, 8:24], what=f"every other row from {x0}")
    m = _randn((3, 40, 6, 10), dtype, 5)
    check(m[:, 4:36], w[:, :32], b, None, "silu", True, True, dtype, _randn((3, 50, 6, 10), dtype, 6)[:, 1:49], "channels of maps")
    check(m[::2, ::2], w[:, :20], b, None, None, True, False, dtype, _randn((2, 60, 50), dtype, 7)[..., 1:49], "every other channel")
    same = _randn((1, 100), dtype, 8).expand(33, 100)
    check(same, _randn((48, 100), dtype, 10, 0.1), b, None, None, dtype=dtype, dy=_randn((1, 48), dtype, 9).expand(33, 48), what="one row many times")


def test_leading_dims_and_in_place():
    x, w = _randn((2, 3, 5, 64), "bf16", 1), _randn((64, 64), "bf16", 2, 0.1)
    r = _randn((2, 3, 5, 64), "bf16", 3)
    want = pkg.linear_fwd(x, w, None, r)
    assert want.shape == (2, 3, 5, 64)
    assert torch.equal(want.flatten(0, 2), pkg.linear_fwd(x.flatten(0, 2), w, None, r.flatten(0, 2)))
    assert pkg.linear_fwd(x, w, None, r, y=r) is r
    assert torch.equal(r, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty(dtype):
    z = lambda *s: torch.zeros(*s, dtype=DT[dtype], device="cuda")  # noqa: E731
    b, r = torch.randn(6, device="cuda"), _randn((3, 6), dtype, 1)
    y = pkg.linear_fwd(z(3, 0), z(6, 0), b, r)
    assert torch.equal(y, (b + r.float()).to(DT[dtype]))
    assert pkg.linear_fwd(z(0, 5), z(6, 5)).shape == (0, 6)
    assert pkg.linear_fwd(z(4, 5), z(0, 5)).shape == (4, 0)
    g = pkg.linear_bwd(z(0, 5), z(6, 5), z(0, 6), out={"dweight": z(6, 5).fill_(7), "dbias": torch.full((6,), 7.0, device="cuda")})
    assert not g["dweight"].any() and not g["dbias"].any()
    g = pkg.linear_bwd(z(4, 5), z(0, 5), z(4, 0), out={"dx": z(4, 5).fill_(7)})
    assert not g["dx"].any()
    g = pkg.linear_bwd(z(3, 0), z(6, 0), r)
    assert torch.allclose(g["dbias"], r.float().sum(0)) and g["dx"].shape == (3, 0) and g["dweight"].shape == (6, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_not_finite_stays_in_its_row(bad, dtype):
    for rows, k, n in ((5, 64, 40), (200, 100, 130)):
        x, w = _randn((rows, k), dtype, 1), _randn((n, k), dtype, 2)
        want = pkg.linear_fwd(x, w)
        x[3, k - 1] = bad
        y = pkg.linear_fwd(x, w)
        assert not torch.isfinite(y[3][w[:, k - 1] != 0]).any()
        keep = torch.arange(rows, device="cuda") != 3
        assert torch.equal(y[keep], want[keep])
        # beyond a view's rows and columns: not read into the sums
        big = torch.full((rows + 2, k + 8), bad, dtype=DT[dtype], device="cuda")
        big[1:-1, 4:-4] = x.nan_to_num(0.5, 0.5, 0.5)
        clean = big[1:-1, 4:-4].contiguous()
        assert torch.equal(pkg.linear_fwd(big[1:-1, 4:-4], w), pkg.linear_fwd(clean, w))


@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu"])
def test_gradients_against_differences(act):
    x, w = _randn((6, 10), "f32", 1), _randn((7, 10), "f32", 2)
    b, dy = torch.randn(7, generator=_gen(3), device="cuda"), _randn((6, 7), "f32", 4)
    _, pre = pkg.linear_fwd(x, w, b, act=act, return_pre=True)
    if act == "relu":  # away from the corner
        b = b + torch.where(pre.abs().amin(0) < 0.02, 0.05, 0.0)
        _, pre = pkg.linear_fwd(x, w, b, act=act, return_pre=True)
    g = pkg.linear_bwd(x, w, dy, pre, act=act)
    f = lambda x, w, b: (_act(x.double() @ w.double().t() + b.double(), act) * dy.double()).sum()  # noqa: E731
    for name, t in (("dx", 0), ("dweight", 1), ("dbias", 2)):
        args, d = [x, w, b], torch.randn((x, w, b)[t].shape, generator=_gen(5), device="cuda").double()
        h = 1e-6  # in 64 bits: the second differences leave 1e-12, the roundings 1e-10
        up, dn = (list(args) for _ in range(2))
        up[t], dn[t] = args[t].double() + h * d, args[t].double() - h * d
        slope = (f(*up) - f(*dn)) / (2 * h)
        assert abs((g[name].double() * d).sum() - slope) <= 1e-5 * (g[name].double() * d).abs().sum() + 1e-7, name


def test_many_batches_and_deterministic():
    case(300, 5, 24, 40, True, True, "silu", True, "bf16", 3)
    x, w, dy = _randn((9000, 64), "bf16", 1), _randn((96, 64), "bf16", 2), _randn((9000, 96), "bf16", 3)
    a, b = (pkg.linear_bwd(x, w, dy) for _ in range(2))
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cf,ocf", [(False, False), (False, True), (True, False), (True, True)])
def test_each_gradient_alone(cf, ocf, dtype):
    """The C entry leaves out the gradients it has no pointer for; the others are right in any company."""
    from selective_state_space_ssm2d_amd import block

    B, R, k, n = 2, 1500, 72, 40
    x, w, dy = _randn((B, k, R) if cf else (B, R, k), dtype, 1), _randn((n, k), dtype, 2), _randn((B, n, R) if ocf else (B, R, n), dtype, 3)
    fn, _, s, flags, need, _, _ = block._linear_plan(True, x, w, None, dy, None, 0, cf, ocf)
    up, xr = _rows(dy, ocf).double(), _rows(x, cf).double()
    flat, fx = up.reshape(-1, n), xr.reshape(-1, k)
    dx, dw, db = up @ w.double(), flat.t() @ fx, flat.sum(0)
    bars = {"dx": _sum_bar(n, dtype) * (up.abs() @ w.double().abs()) + _half(dx, dtype),
            "dweight": _sum_bar(B * R, dtype) * (flat.abs().t() @ fx.abs()) + _half(dw, dtype),
            "dbias": (3 * B * R + 2) * U * flat.abs().sum(0)}  # (float32 as three parts: additions of each)
    for wanted in range(1, 8):
        out = {"dx": torch.full_like(x, 7.0), "dweight": torch.full_like(w, 7.0), "dbias": torch.full((n,), 7.0, device="cuda")}
        work = torch.empty(need, dtype=torch.uint8, device="cuda")
        ptr = [t.data_ptr() if wanted >> i & 1 else None for i, t in enumerate(out.values())]
        assert fn(x.data_ptr(), w.data_ptr(), None, dy.data_ptr(), *ptr, s, 0, flags, work.data_ptr(), need, torch.cuda.current_stream().cuda_stream) == 0
        for i, (name, want) in enumerate(zip(out, (dx, dw, db))):
            got = _rows(out[name], cf) if name == "dx" else out[name]
            if wanted >> i & 1:
                _near(got, want, bars[name], f"{name} of {wanted}")
            else:
                assert (got == 7.0).all(), (name, wanted)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,k,n,act", [(2, 16, 16, "silu"), (3, 2000, 5, None), (40000, 16, 24, None), (40000, 20, 9, "gelu"), (12544, 136, 264, None)])
def test_gradients_of_few_and_many_rows(rows, k, n, act, dtype):
    """Sums undivided and in parts, one gradient's workgroups few beside the other's."""
    x, w = _randn((rows, k), dtype, rows), _randn((n, k), dtype, 1, k ** -0.5)
    check(x, w, torch.zeros(n, device="cuda"), None, act, dtype=dtype, dy=_randn((rows, n), dtype, 2), what=f"{rows} rows")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("k,n", [(768, 1536), (1, 3), (31, 17), (32, 16), (33, 15), (1000, 100), (1031, 33), (2047, 8)])
def test_few_rows(k, n, dtype):
    """Tiles of 16 rows and one row more, with the epilogue's parts, at strides, and into the residual."""
    for i, rows in enumerate((1, 2, 5, 15, 16, 17, 33, 64)):
        act = (None, "silu", "gelu", "relu")[i % 4]
        case(1, rows, k, n, False, False, act, i % 2 == 0, dtype, rows + k, bias=i % 3 != 0)
    wide, w = _randn((8, k + 5), dtype, 1), _randn((n + 2, k + 3), dtype, 2, k ** -0.5)
    check(wide[::2, 3:3 + k], w[1:1 + n, 1:1 + k], None, None, "silu", dtype=dtype, what="strides")
    x, r = wide[:3, :k], _randn((3, n), dtype, 3)
    want = pkg.linear_fwd(x, w[:n, :k], None, r, act="gelu")
    y = r.clone()
    assert pkg.linear_fwd(x, w[:n, :k], None, y, act="gelu", y=y) is y and torch.equal(y, want)
    # (both are few rows) a row alone, and with others: the same bits
    assert torch.equal(pkg.linear_fwd(x[1:2], w[:n, :k]), pkg.linear_fwd(x, w[:n, :k])[1:2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cf,ocf", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("rows,k,n", [(256, 64, 128), (300, 200, 136), (1030, 1000, 264), (4100, 520, 520), (70, 4096, 72)])
def test_whole_numbers(rows, k, n, cf, ocf, dtype):
    """Sums of small whole numbers are exact in any order: every element of every
    tile, several times over, forward and both gradients."""
    whole = lambda shape, seed: torch.randint(-3, 4, shape, generator=_gen(seed), device="cuda").to(DT[dtype])  # noqa: E731
    mixed = cf or ocf
    xs = (1, k, rows) if cf else ((1, rows, k) if mixed else (rows, k))
    ys = (1, n, rows) if ocf else ((1, rows, n) if mixed else (rows, n))
    x, w, r, dy = whole(xs, 1), whole((n, k), 2), whole(ys, 3), whole(ys, 4)
    xr, up, res = (_rows(t, m).reshape(rows, -1).double() for t, m in ((x, cf), (dy, ocf), (r, ocf)))
    # (all below 9 * 4100 + 3 < 2^24; a bf16 output is the sum rounded)
    want = {"y": xr @ w.double().t() + res, "dx": up @ w.double(), "dweight": up.t() @ xr, "dbias": up.sum(0)}
    for _ in range(3):
        got = {"y": pkg.linear_fwd(x, w, None, r, channels_first=cf, out_channels_first=ocf),
               **pkg.linear_bwd(x, w, dy, channels_first=cf, out_channels_first=ocf)}
        for name, v in want.items():
            g = got[name]
            g = _rows(g, ocf if name == "y" else cf).reshape(rows, -1) if name in ("y", "dx") else g
            assert torch.equal(g, v.to(g.dtype)), name
