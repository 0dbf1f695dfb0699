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
       (1, 777, 1, 2, 128, 128), (1, 640, 4, 4, 32, 32), (4, 130, 1, 1, 8, 130)]


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
           (ValueError, lambda: S(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], st[:1])),
           (ValueError, lambda: S(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], st.transpose(2, 3))),
           (ValueError, lambda: S(q[:, 0], k[:, 0], v[:, 0], g[:, 0], beta[:, 0], None))]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            pytest.fail(f"case {i} was not refused")
