"""GPU tests of layer norm and rotary positions against plain 64-bit
implementations: sizes around every variant's limits, strided and misaligned
views, both directions, streams and graph replays.

Bars, from the arithmetic: every fp32 operation rounds by at most u = 2^-24
relative; sums run over a tree of registers, lanes and waves (depth below 64
for the sizes here), so a sum of terms t errs by at most 64 u sum|t|, and
x - mean inherits u (|x| + mean|x|) from cancellation. A bf16 output adds half
a unit of its last place, 2^-9 of its value.
"""
import pytest

import selective_state_space_ssm2d_amd as pkg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _half_ulp(ref, dtype):
    return 2.0 ** -8 * ref.abs() if dtype == "bf16" else 0.0


def _close(got, ref, tol, what):
    d = (got.double() - ref).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), (what, float(d[bad].max()), int(bad.sum()))


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# (batch, n, cells): rows
ROWS = [(1, 1), (3, 2), (5, 7), (1, 64), (4, 65), (70, 96), (9, 128), (33, 192), (2, 255), (6, 256), (7, 257), (5, 768), (3, 1000),
        (2, 1024), (2, 1032), (3, 2048), (2, 2056), (2, 4097), (3, 8192), (2, 8200), (2, 16384), (1, 16383), (5000, 40)]
# (batch, n, cells): maps
MAPS = [(1, 1, 1), (2, 3, 5), (1, 16, 64), (2, 64, 49), (1, 65, 196), (3, 128, 130), (2, 129, 96), (1, 192, 3136), (2, 193, 196),
        (1, 256, 77), (2, 257, 40), (1, 384, 196), (1, 385, 72), (2, 768, 196), (1, 769, 33), (1, 1024, 68), (1, 1030, 64), (1, 1500, 12),
        (2, 300, 7)]


def _norm_case(shape, dtype, seed, offset):
    g = _gen(seed)
    n = shape[1]
    one = (1, n) + (1,) * (len(shape) - 2)
    x = torch.randn(shape, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(one, generator=g, device="cuda")) + offset
    w, b = torch.randn(n, generator=g, device="cuda"), torch.randn(n, generator=g, device="cuda")
    dy = torch.randn(shape, generator=g, device="cuda")
    return x.to(DT[dtype]), w, b, dy.to(DT[dtype])


def _check_norm(x, w, b, dy, dtype, cf, eps=1e-5, what=""):
    y, mean, rstd = pkg.layer_norm_fwd(x, w, b, eps, channels_first=cf, return_stats=True)
    xd, n = x.double(), x.shape[1]
    col = (lambda t: t.double().view(1, n, *([1] * (x.dim() - 2))))
    mu = xd.mean(1, keepdim=True)
    rs = 1.0 / torch.sqrt(((xd - mu) ** 2).mean(1, keepdim=True) + eps)
    wd = col(w) if w is not None else torch.ones_like(mu)
    bd = col(b) if b is not None else torch.zeros_like(mu)
    size = (xd.abs() + xd.abs().mean(1, keepdim=True)) * rs  # of x - mean before cancellation, normalised
    ref = (xd - mu) * rs * wd + bd
    # the statistics' errors: the mean's 64 u mean|x|; the variance's, relative, 64 u plus the shift of the mean
    shift = 64 * U * size.amax(1, keepdim=True)
    _close(y, ref, shift * wd.abs() * (1 + ((xd - mu) * rs).abs()) + 8 * U * (ref.abs() + bd.abs()) + _half_ulp(ref, dtype), what + " y")
    _close(mean, mu.squeeze(1), 64 * U * xd.abs().mean(1) + 1e-30, what + " mean")
    _close(rstd, rs.squeeze(1), (64 * U + shift.squeeze(1) + shift.squeeze(1) ** 2) * rs.squeeze(1), what + " rstd")
    # the gradient takes the statistics it is given
    r = pkg.layer_norm_bwd(x, w, mean, rstd, dy, channels_first=cf)
    mu, rs, gd = mean.double().unsqueeze(1), rstd.double().unsqueeze(1), dy.double()
    xh, gw = (xd - mu) * rs, gd * wd
    exh = 4 * U * (xd.abs() + mu.abs()) * rs  # of xh
    a, c = gw.mean(1, keepdim=True), (gw * xh).mean(1, keepdim=True)
    ref = rs * (gw - a - xh * c)
    ma, mc = gw.abs().mean(1, keepdim=True), (gw.abs() * (xh.abs() + exh)).mean(1, keepdim=True)
    tol = rs * (8 * U * gw.abs() + 64 * U * ma + (64 * U * mc + (gw.abs() * exh).mean(1, keepdim=True)) * (xh.abs() + exh) + exh * mc)
    _close(r["dx"], ref, tol + _half_ulp(ref, dtype) + 1e-30, what + " dx")
    red = [d for d in range(x.dim()) if d != 1]
    terms = (gd.abs() * (xh.abs() + exh)).sum(red)
    _close(r["dweight"], (gd * xh).sum(red), 64 * U * terms + (gd.abs() * exh).sum(red) + 1e-30, what + " dweight")
    _close(r["dbias"], gd.sum(red), 64 * U * gd.abs().sum(red) + 1e-30, what + " dbias")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n", ROWS)
def test_norm_rows(rows, n, dtype):
    x, w, b, dy = _norm_case((rows, n), dtype, 10 + n, 0.5)
    _check_norm(x, w, b, dy, dtype, False, what=f"rows {rows} x {n} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,n,cells", MAPS)
def test_norm_maps(batch, n, cells, dtype):
    x, w, b, dy = _norm_case((batch, n, cells), dtype, 20 + n, -0.25)
    _check_norm(x, w, b, dy, dtype, True, what=f"maps {batch} x {n} x {cells} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_without_weight_and_with_a_large_mean(dtype):
    x, w, b, dy = _norm_case((40, 320), dtype, 3, 1000.0)
    _check_norm(x, None, None, dy, dtype, False, what="rows, no weight")
    x, w, b, dy = _norm_case((2, 96, 40), dtype, 4, 1000.0)
    _check_norm(x, w, None, dy, dtype, True, what="maps, no bias")
    # equal channels: the variance is zero, eps alone is left
    x = torch.full((4, 64), 2.5, device="cuda", dtype=DT[dtype])
    y = pkg.layer_norm_fwd(x)
    assert bool((y == 0).all())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_strided_and_misaligned_views(dtype):
    g = _gen(5)
    wide = torch.randn(50, 400, generator=g, device="cuda").to(DT[dtype])
    w, b = torch.randn(192, generator=g, device="cuda"), torch.randn(192, generator=g, device="cuda")
    for lo in (0, 8, 1, 3):  # rows at a stride of 400, aligned and not
        x = wide[:, lo:lo + 192]
        dy = torch.randn(50, 193, generator=g, device="cuda").to(DT[dtype])[:, 1:]
        _check_norm(x, w, b, dy, dtype, False, what=f"rows view {lo}")
    maps = torch.randn(3, 300, 6, 14, generator=g, device="cuda").to(DT[dtype])
    x = maps[:, 50:242]
    _check_norm(x.flatten(2) if x.is_contiguous() else x, w, b, torch.randn(3, 192, 6, 14, generator=g, device="cuda").to(DT[dtype]), dtype,
                True, what="maps view")
    base = torch.randn(2 * 192 * 77 + 1, generator=g, device="cuda").to(DT[dtype])
    x = base[1:].view(2, 192, 77)
    _check_norm(x, w, b, base[:-1].view(2, 192, 77), dtype, True, what="maps off by one element")
    x = torch.randn(192, 20, generator=g, device="cuda").to(DT[dtype]).t()[:, :, None]  # one cell, channels strided
    _check_norm(x, w, b, x.contiguous(), dtype, True, what="one cell, strided channels")


def test_norm_nan_stays_in_its_row():
    x = torch.randn(9, 512, device="cuda", generator=_gen(6))
    x[4, 100] = float("nan")
    y = pkg.layer_norm_fwd(x)
    bad = torch.isnan(y).any(1)
    assert bad.nonzero().flatten().tolist() == [4]


def test_norm_empty():
    g = {"w": torch.ones(8, device="cuda")}
    y, mean, rstd = pkg.layer_norm_fwd(torch.zeros(0, 8, device="cuda"), g["w"], return_stats=True)
    assert y.shape == (0, 8) and mean.shape == (0,) and rstd.shape == (0,)
    e = torch.zeros(2, 8, 0, device="cuda")
    s = torch.zeros(2, 0, device="cuda")
    r = pkg.layer_norm_bwd(e, g["w"], s, s, e, channels_first=True)
    assert bool((r["dweight"] == 0).all()) and bool((r["dbias"] == 0).all())


def test_norm_gradient_against_differences():
    """dx, dweight and dbias against central differences of the 64-bit formula
    along random directions: the formula itself is right."""
    g = _gen(7)
    x = torch.randn(6, 48, generator=g, device="cuda")
    w, b, dy = (torch.randn(s, generator=g, device="cuda") for s in (48, 48, (6, 48)))
    _, mean, rstd = pkg.layer_norm_fwd(x, w, b, return_stats=True)
    r = pkg.layer_norm_bwd(x, w, mean, rstd, dy)

    def loss(x, w, b):
        mu = x.mean(1, keepdim=True)
        return (((x - mu) / torch.sqrt(((x - mu) ** 2).mean(1, keepdim=True) + 1e-5) * w + b) * dy.double()).sum()

    for k in range(4):
        dirs = [torch.randn(t.shape, generator=g, device="cuda").double() for t in (x, w, b)]
        h = 1e-5
        up = loss(*(t.double() + h * d for t, d in zip((x, w, b), dirs)))
        dn = loss(*(t.double() - h * d for t, d in zip((x, w, b), dirs)))
        want = (up - dn) / (2 * h)
        got = sum((r[n].double() * d).sum() for n, d in zip(("dx", "dweight", "dbias"), dirs))
        # the differences' own error is h^2 of a smooth function (1e-9 here) and 2^-52 / h
        assert abs(float(got - want)) <= 1e-4 * (1 + abs(float(want))), (k, float(got), float(want))


def test_norm_deterministic():
    x, w, b, dy = _norm_case((3000, 96), "f32", 8, 0.0)
    y, mean, rstd = pkg.layer_norm_fwd(x, w, b, return_stats=True)
    r1 = pkg.layer_norm_bwd(x, w, mean, rstd, dy)
    r2 = pkg.layer_norm_bwd(x, w, mean, rstd, dy)
    assert all(torch.equal(r1[k], r2[k]) for k in r1)


def test_norm_on_a_stream_and_in_a_graph():
    s = torch.cuda.Stream()
    x, w, b, dy = _norm_case((2, 96, 196), "bf16", 9, 0.0)
    s.wait_stream(torch.cuda.current_stream())
    y, mean, rstd = pkg.layer_norm_fwd(x, w, b, channels_first=True, return_stats=True, stream=s)
    r = pkg.layer_norm_bwd(x, w, mean, rstd, dy, channels_first=True, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pkg.layer_norm_bwd(x, w, mean, rstd, dy, channels_first=True, out=r)
    for k in range(3):
        dy.copy_(torch.randn(dy.shape, generator=_gen(k), device="cuda"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        e = pkg.layer_norm_bwd(x, w, mean, rstd, dy, channels_first=True)
        assert all(torch.equal(e[n], r[n]) for n in e), k


def test_norm_refusals():
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(8, device="cuda")
    bad = [(ValueError, lambda: pkg.layer_norm_fwd(x, w[:7])),
           (ValueError, lambda: pkg.layer_norm_fwd(x, w.double())),
           (ValueError, lambda: pkg.layer_norm_fwd(x, w.cpu())),
           (ValueError, lambda: pkg.layer_norm_fwd(x.cpu())),
           (TypeError, lambda: pkg.layer_norm_fwd(x.half())),
           (ValueError, lambda: pkg.layer_norm_fwd(x.t())),
           (ValueError, lambda: pkg.layer_norm_fwd(torch.zeros(2, 8, 4, 4, device="cuda").transpose(2, 3)[:, :, :, :3], channels_first=True)),
           (ValueError, lambda: pkg.layer_norm_fwd(x, y=torch.zeros(4, 7, device="cuda"))),
           (pkg.Ssm2dError, lambda: pkg.layer_norm_fwd(torch.zeros(1, 16385, device="cuda"))),
           (ValueError, lambda: pkg.layer_norm_bwd(x, w, torch.zeros(3, device="cuda"), torch.zeros(4, device="cuda"), x)),
           (ValueError, lambda: pkg.layer_norm_bwd(x, w, torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda"), x[:, :7]))]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            pytest.fail(f"case {i} was not refused")


# ------------------------------------------------------------------ rotary positions

def _rope_ref(x, pos, freq, sections, inter, sign):
    axis = sum(([a] * s for a, s in enumerate(sections)), [])
    ang = pos.double()[axis]  # [P, (B,) T]
    ang = (ang * freq.double().view(-1, *([1] * (ang.dim() - 1)))).movedim(0, -1)
    if ang.dim() == 2:
        ang = ang[None]
    c, s = torch.cos(ang)[:, :, None], sign * torch.sin(ang)[:, :, None]
    P, xd = len(axis), x.double()
    out = xd.clone()
    mag = torch.zeros_like(xd)
    i1 = torch.arange(P, device=x.device) * (2 if inter else 1)
    i2 = i1 + (1 if inter else P)
    x1, x2 = xd[..., i1], xd[..., i2]
    out[..., i1], out[..., i2] = x1 * c - x2 * s, x2 * c + x1 * s
    mag[..., i1] = mag[..., i2] = x1.abs() + x2.abs()
    return out, mag


# (batch, tokens, hq, hk, d, sections, interleaved)
ROPE = [(1, 1, 1, 0, 2, (1,), False), (2, 5, 3, 1, 16, (4, 4), False), (1, 9, 2, 2, 16, (3, 5), True), (2, 33, 4, 2, 64, (8, 12, 12), False),
        (1, 7, 5, 1, 72, (8, 14, 14), True), (1, 130, 6, 6, 32, (8, 8), False), (2, 3, 1, 1, 30, (5, 6), False), (1, 4, 2, 1, 10, (2, 2), True),
        (3, 17, 2, 2, 128, (16, 24, 24), False), (1, 2, 1, 1, 1024, (128, 128, 128, 128), False), (1, 6, 3, 3, 40, (4, 0, 8), False),
        (1, 8, 2, 1, 12, (0, 0), True), (1, 300, 1, 1, 7, (2, 1), True), (1, 3136, 6, 6, 32, (8, 8), False)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", ROPE, ids=str)
def test_rope(case, dtype):
    B, T, hq, hk, d, sections, inter = case
    g = _gen(sum(sections) + T)
    P = sum(sections)
    pos = torch.randint(-3, 400, (len(sections), B, T), generator=g, device="cuda", dtype=torch.int32)
    freq = 10000.0 ** (-torch.arange(P, device="cuda").float() / max(P, 1))
    q = torch.randn(B, T, hq, d, generator=g, device="cuda").to(DT[dtype])
    k = torch.randn(B, T, hk, d, generator=g, device="cuda").to(DT[dtype]) if hk else None
    for name, f, sign in (("fwd", pkg.rope_fwd, 1.0), ("bwd", pkg.rope_bwd, -1.0)):
        for p in (pos, pos[:, 0].contiguous()):
            got = f(q, k, p, freq, sections, interleaved=inter)
            assert (got[1] is None) == (k is None)
            for t, o in zip((q, k), got):
                if t is None:
                    continue
                ref, mag = _rope_ref(t, p, freq, sections, inter, sign)
                _close(o, ref, 8 * U * mag + _half_ulp(ref, dtype), f"{name} {case}")


def test_rope_far_positions_and_its_gradient():
    """Angles up to 2^30 keep their digits (exact angles in the reference), and
    the inverse turn undoes the turn."""
    g = _gen(1)
    T = 2000
    pos = torch.randint(-(1 << 30), 1 << 30, (2, T), generator=g, device="cuda", dtype=torch.int32)
    pos[0, :8] = torch.tensor([0, 1, -1, 4095, 4096, -4096, 1 << 20, (1 << 20) + 1], device="cuda", dtype=torch.int32)
    freq = torch.cat([torch.ones(1), 10.0 ** -torch.arange(0, 8).float()]).cuda()
    q = torch.randn(1, T, 2, 18, generator=g, device="cuda")
    o, _ = pkg.rope_fwd(q, None, pos, freq, (4, 5))
    ref, mag = _rope_ref(q, pos, freq, (4, 5), False, 1.0)
    # the reference's angles: 2^30 * 2^-53 in 64 bits
    _close(o, ref, (8 * U + 2.0 ** -22) * mag, "far positions")
    back, _ = pkg.rope_bwd(o, None, pos, freq, (4, 5))
    _close(back, q.double(), 16 * U * (mag + mag), "turned back")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rope_strided_views(dtype):
    g = _gen(2)
    B, T, hq, hk, d = 2, 21, 4, 2, 32
    fused = torch.randn(B, T, (hq + hk) * d + 5, generator=g, device="cuda").to(DT[dtype])
    pos = torch.randint(0, 64, (3, T), generator=g, device="cuda", dtype=torch.int32)
    freq = torch.rand(14, generator=g, device="cuda")
    for lo in (0, 5):
        q = fused[..., lo:lo + hq * d].unflatten(-1, (hq, d))
        k = fused[..., lo + hq * d:lo + (hq + hk) * d].unflatten(-1, (hk, d))
        qt = torch.randn(B, hq, T, d, generator=g, device="cuda").to(DT[dtype]).transpose(1, 2)  # heads before tokens
        for a in (q, qt):
            for inter in (False, True):
                o = pkg.rope_fwd(a, k, pos, freq, (4, 5, 5), interleaved=inter)
                for t, x in zip((a, k), o):
                    ref, mag = _rope_ref(t, pos, freq, (4, 5, 5), inter, 1.0)
                    _close(x, ref, 8 * U * mag + _half_ulp(ref, dtype), f"view {lo} {inter}")


def test_rope_empty_and_refusals():
    f = torch.ones(4, device="cuda")
    pos = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 3, 2, 8, device="cuda")
    e, _ = pkg.rope_fwd(q[:0], None, torch.zeros(2, 0, 3, dtype=torch.int32, device="cuda"), f, (2, 2))
    assert e.shape == (0, 3, 2, 8)
    bad = [(ValueError, lambda: pkg.rope_fwd(q, None, pos.long(), f, (2, 2))),
           (ValueError, lambda: pkg.rope_fwd(q, None, pos[:1], f, (2, 2))),
           (ValueError, lambda: pkg.rope_fwd(q, None, pos, f[:3], (2, 2))),
           (ValueError, lambda: pkg.rope_fwd(q, q.bfloat16(), pos, f, (2, 2))),
           (ValueError, lambda: pkg.rope_fwd(q, q[:, :2], pos, f, (2, 2))),
           (ValueError, lambda: pkg.rope_fwd(q[0], None, pos, f, (2, 2))),
           (ValueError, lambda: pkg.rope_fwd(q[..., ::2], None, pos, f[:2], (1, 1))),
           (pkg.Ssm2dError, lambda: pkg.rope_fwd(q, None, pos, torch.ones(5, device="cuda"), (2, 3))),
           (pkg.Ssm2dError, lambda: pkg.rope_fwd(q, None, pos, f, (5, -1))),
           (ValueError, lambda: pkg.rope_fwd(q, None, torch.zeros(5, 3, dtype=torch.int32, device="cuda"), f, (1, 1, 1, 1, 0))),
           (TypeError, lambda: pkg.rope_fwd(q.half(), None, pos, f, (2, 2)))]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            pytest.fail(f"case {i} was not refused")
