"""gelu and its derivative relative to their own size, tail included.

The normal distribution function's tail is within 1.2e-4 of its value (fit) and e^(-z^2 / 2) within 13^2 / 2 * 2^-22 for |z| < 13
(an exponent of z^2 / 2 rounded twice): together below 2^-12 of the tail. A value rounded to bf16 is off by 2^-8 more."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
REL = 2.0 ** -12


def _points():
    """Every bf16 number from -12.5 to 12.5 with a magnitude of at least 2^-10."""
    bits = torch.arange(0x3A80, 0x4148, dtype=torch.int32).to(torch.int16)
    z = bits.view(BF)
    return torch.cat([-z, z]).cuda()


def _parts(z):
    """P(z) and z phi(z) in 64 bits."""
    z = z.double()
    return 0.5 * torch.special.erfc(-z / math.sqrt(2)), z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


@pytest.mark.parametrize("M", [1, 7, 100, 300])
@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
def test_value(M, t):
    z = _points()
    N, K = z.numel(), 8
    x, W = torch.zeros(M, K, device="cuda", dtype=BF), torch.zeros(N, K, device="cuda", dtype=BF)
    x[:, 0], W[:, 0] = 1, z  # pre = z
    y, st = torch.empty(M, N, device="cuda", dtype=t), torch.zeros(1, dtype=torch.int32, device="cuda")
    tw.twell_linear_fwd(x, W, False, None, tw.ACT_GELU, None, None, y, st)
    assert tw.twell_check(st) == 0
    want = z.double() * _parts(z)[0]
    bound = (REL + (2.0 ** -8 if t is BF else 0.0)) * want.abs()
    off = (y.double() - want).abs() / bound
    assert float(off.max()) <= 1, (float(off.max()), float(z[off.amax(0).argmax()]))


def test_derivative():
    z = _points()
    N = z.numel()
    pre, dy = z[None].contiguous(), torch.ones(1, N, device="cuda", dtype=BF)
    x, W = torch.zeros(1, 8, device="cuda", dtype=BF), torch.zeros(N, 8, device="cuda", dtype=BF)
    db, st = torch.empty(N, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(tw.twell_linear_bwd_workspace_bytes(1, N, 8), dtype=torch.uint8, device="cuda")
    tw.twell_linear_bwd(dy, x, W, False, tw.ACT_GELU, pre, None, None, False, db, ws, st)
    assert tw.twell_check(st) == 0
    P, zphi = _parts(z)
    off = (db.double() - (P + zphi)).abs() / (REL * (P + zphi.abs()))
    assert float(off.max()) <= 1, (float(off.max()), float(z[off.argmax()]))
