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
