"""bf16 results of long sums: weight gradients of many rows, products of large depth.

The tensor cores' fp32 sums drop what does not fit, towards zero: at most 2^-23 of a sum just above 1 at each step of 16 of
depth. A sum in which that happens at every step: a 1, then products of 3 * 2^-29, 16 of which are 3/4 of that unit, so that a
sum with the 1 in it never grows. They are added up by the tensor cores over at most 16384 of depth (1024 steps), which costs
2^-13 of the result; rounding it once costs 2^-8. Lengths are such that the products add up to 0.0046: 1.0046 rounds to
1.0078, while a sum that loses a quarter of them rounds to 1, further off than both bounds together.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

BF = torch.bfloat16
LONG = 823_040                    # terms
A, B = 3 * 2.0 ** -15, 2.0 ** -14  # a small product's factors
TOTAL = 1 + (LONG - 1) * A * B
LOST, HALF_STEP = 1024 * 2.0 ** -23, 2.0 ** -8


def _ones_then(value, *shape, dim):
    t = torch.full(shape, value, device="cuda", dtype=BF)
    t.select(dim, 0).fill_(1)
    return t


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _close(got, want=TOTAL, terms=1):
    bound = terms * LOST * want + HALF_STEP * (want + terms * LOST)
    assert bool(((got.double() - want).abs() <= bound).all()), (float(got.double().min()), float(got.double().max()), want)


@pytest.mark.parametrize("M", [1, 3, 16, 40, 100, 300, 1100])
def test_linear_forward(M):
    x, W = _ones_then(A, M, LONG, dim=1), _ones_then(B, 24, LONG, dim=1)
    y, st = torch.empty(M, 24, device="cuda", dtype=BF), _status()
    tw.twell_linear_fwd(x, W, False, None, tw.ACT_NONE, None, None, y, st)
    assert tw.twell_check(st) == 0
    _close(y)


@pytest.mark.parametrize("kn", [False, True])
def test_weight_gradient(kn):
    x, dy = _ones_then(A, LONG, 8, dim=0), _ones_then(B, LONG, 16, dim=0)
    W = torch.zeros(*((8, 16) if kn else (16, 8)), device="cuda", dtype=BF)
    dW, dx, st = torch.empty_like(W), torch.empty_like(x), _status()
    ws = torch.empty(tw.twell_linear_bwd_workspace_bytes(LONG, 16, 8), dtype=torch.uint8, device="cuda")
    for out in (None, dx):
        tw.twell_linear_bwd(dy, x, W, kn, tw.ACT_NONE, None, out, dW.fill_(9), False, None, ws, st)
        assert tw.twell_check(st) == 0
        _close(dW)


@pytest.mark.parametrize("M", [1, 5, 40, 100, 300])
def test_gated_forward(M):
    F = 16
    x, W = _ones_then(A, M, LONG, dim=1), _ones_then(B, F, LONG, dim=1)
    Wd = torch.zeros(F, LONG, device="cuda", dtype=BF)
    g, u, h = (torch.empty(M, F, device="cuda", dtype=BF) for _ in range(3))
    y, st = torch.empty(M, LONG, device="cuda", dtype=BF), _status()
    tw.twell_dense_gated_ffn_fwd(x, W, W, None, Wd, tw.ACT_NONE, None, g, u, h, y, st)
    assert tw.twell_check(st) == 0
    _close(g)
    _close(u)
    _close(h, TOTAL * TOTAL, 2)
    assert not bool(y.any())


def test_gated_weight_gradients():
    """dh = dy W_down^T = 1 in row 0, else B; g = u = 1 without an activation: dg = du = dh."""
    F, d = 16, 8
    x = _ones_then(A, LONG, d, dim=0)
    one = torch.ones(LONG, F, device="cuda", dtype=BF)
    h = _ones_then(A, LONG, F, dim=0)
    dy = torch.zeros(LONG, d, device="cuda", dtype=BF)
    dy[:, 0] = B
    dy[0, 0] = 1
    Wd = torch.zeros(F, d, device="cuda", dtype=BF)
    Wd[:, 0] = 1
    W = torch.zeros(F, d, device="cuda", dtype=BF)
    dW, st = [torch.empty(F, d, device="cuda", dtype=BF) for _ in range(3)], _status()
    ws = torch.empty(tw.twell_dense_gated_bwd_workspace_bytes(LONG, d, F), dtype=torch.uint8, device="cuda")
    tw.twell_dense_gated_ffn_bwd(x, W, W, Wd, tw.ACT_NONE, one, one, h, dy, 0.0, None, *dW, False, None, ws, st)
    assert tw.twell_check(st) == 0
    _close(dW[0])
    _close(dW[1])
    _close(dW[2][:, 0])
    assert not bool(dW[2][:, 1:].any())


@pytest.mark.parametrize("M", [40, 300])
def test_gated_input_gradient(M):
    """Two products of depth F in one sum: dg = W_down's column, W_gate = A, and nothing from du."""
    F, d = LONG, 8
    dy = torch.zeros(M, d, device="cuda", dtype=BF)
    dy[:, 0] = 1
    Wd = torch.zeros(F, d, device="cuda", dtype=BF)
    Wd[:, 0] = B
    Wd[0, 0] = 1
    Wg = _ones_then(A, F, d, dim=0)
    Wu = torch.zeros(F, d, device="cuda", dtype=BF)
    g, u = torch.zeros(M, F, device="cuda", dtype=BF), torch.ones(M, F, device="cuda", dtype=BF)
    dx, st = torch.empty(M, d, device="cuda", dtype=BF), _status()
    ws = torch.empty(tw.twell_dense_gated_bwd_workspace_bytes(M, d, F), dtype=torch.uint8, device="cuda")
    tw.twell_dense_gated_ffn_bwd(dy, Wg, Wu, Wd, tw.ACT_NONE, g, u, u, dy, 0.0, dx, None, None, None, False, None, ws, st)
    assert tw.twell_check(st) == 0
    _close(dx)
