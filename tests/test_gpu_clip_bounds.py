"""twell_grad_clip where the bound or the norm is zero, infinite or past fp32's range.

Tolerances. A warp's 1024 squares are joined in fp32: chains of 8 fused steps, two
joins and five shuffle steps, 15 roundings, so a sum of squares is off by at most
15 u, u = 2^-24, and a norm by half of that and its own rounding (9 u). Squares
outside fp32's range are summed in 64 bits. A scaled element carries the factor's
error and its own roundings, 11 u in all; bf16 adds half a unit in the last place
(up to 2^-8).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def _clip(ts, max_norm, outs=None):
    norm = torch.full((1,), -1.0, device="cuda")
    ws = torch.empty(tw.twell_grad_clip_workspace_bytes(), dtype=torch.uint8, device="cuda")
    tw.twell_grad_clip(tw.TwellTensorList(ts, outs), max_norm, norm, ws)
    return float(norm)


def _same_bits(a, b):
    kind = torch.int16 if a.dtype is BF else torch.int32
    return torch.equal(a.view(kind), b.view(kind))


@pytest.mark.parametrize("value", [INF, -INF, float("nan"), 1.0])
@pytest.mark.parametrize("in_place", [True, False])
def test_infinite_bound_leaves_the_gradients(value, in_place):
    """INFINITY gives the norm alone, also where it is infinite or NaN."""
    g, h = torch.randn(10_000, device="cuda"), torch.randn(333, device="cuda").to(BF)
    g[5_000] = value
    before = [g.clone(), h.clone()]
    outs = None if in_place else [torch.full_like(g, 5.0), torch.full_like(h, 5.0)]
    norm = _clip([g, h], INF, outs)
    assert math.isnan(norm) if math.isnan(value) else math.isinf(norm) == math.isinf(value)
    for t, b in zip([g, h] if in_place else outs, before):
        assert _same_bits(t, b)


@pytest.mark.parametrize("in_place", [True, False])
def test_zero_bound_and_zero_gradients(in_place):
    """0 is not above a bound of 0: nothing is scaled."""
    ts = [torch.zeros(1000, device="cuda"), torch.zeros(7, device="cuda", dtype=BF)]
    outs = None if in_place else [torch.full_like(t, 5.0) for t in ts]
    assert _clip(ts, 0.0, outs) == 0.0
    assert not any(t.any() for t in (ts if in_place else outs))


@pytest.mark.parametrize("value", [2e38, 3.38e38])
@pytest.mark.parametrize("max_norm", [1.0, 1e30, 3e38, INF])
def test_finite_gradients_whose_norm_passes_32_bits(value, max_norm):
    """The factor comes from the 64-bit norm; the norm itself is reported as infinite."""
    g, h = torch.full((5_000,), value, device="cuda"), torch.full((700,), -value, device="cuda").to(BF)
    g[::7] = 1e30
    before = [g.double().clone(), h.double().clone()]
    assert all(bool(b.isfinite().all()) for b in before)
    ref = math.sqrt(sum(float((b ** 2).sum()) for b in before))
    assert math.isinf(_clip([g, h], max_norm))
    c = min(1.0, max_norm / ref)
    for t, b in ((g, before[0]), (h, before[1])):
        want = b * c
        assert bool(((t.double() - want).abs() <= want.abs() * (11 * 2.0 ** -24 + 2.0 ** -23 + (2.0 ** -8 if t.dtype is BF else 0))
                     + c * 2.0 ** -100).all())
