"""Derivatives of the activations at the largest pre-activations that bf16 has: 1 above, 0 below."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

BF = torch.bfloat16


@pytest.mark.parametrize("act", [tw.ACT_RELU, tw.ACT_SILU, tw.ACT_GELU, tw.ACT_GELU_TANH], ids=["relu", "silu", "gelu", "gelu_tanh"])
def test_derivative(act):
    z = torch.tensor([100.0, 1e6, 1e13, 1e18, 3e19, 1e25, 3.3e38], device="cuda").to(BF)
    z = torch.cat([z, -z])
    N = z.numel()
    dy = torch.ones(1, N, device="cuda", dtype=BF)
    x, W = torch.ones(1, 8, device="cuda", dtype=BF), torch.eye(N, 8, device="cuda", dtype=BF)
    dx, dW, db = torch.empty_like(x), torch.empty(N, 8, device="cuda"), torch.empty(N, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(tw.twell_linear_bwd_workspace_bytes(1, N, 8), dtype=torch.uint8, device="cuda")
    tw.twell_linear_bwd(dy, x, W, False, act, z[None].contiguous(), dx, dW, False, db, ws, st)
    assert tw.twell_check(st) == 0
    want = (z > 0).float()
    assert torch.equal(db, want) and torch.equal(dW, want[:, None].expand(N, 8)) and torch.equal(dx[0].float(), want[:8])


@pytest.mark.parametrize("act", [tw.ACT_RELU, tw.ACT_SILU, tw.ACT_GELU, tw.ACT_GELU_TANH], ids=["relu", "silu", "gelu", "gelu_tanh"])
def test_gated_layer(act):
    """dg = dh u act'(g) and du = dh act(g) for gates as large as their product with u allows."""
    M, d, F = 16, 8, 8
    g = torch.tensor([1e6, 1e13, 3e19, 1e25, -1e6, -1e13, -3e19, -1e25], device="cuda").to(BF).expand(M, F).contiguous()
    u = torch.full((M, F), 2.0, device="cuda", dtype=BF)
    x, dy = torch.zeros(M, d, device="cuda", dtype=BF), torch.zeros(M, d, device="cuda", dtype=BF)
    x[0, 0] = dy[0, 0] = 1
    W, Wd = torch.zeros(F, d, device="cuda", dtype=BF), torch.zeros(F, d, device="cuda", dtype=BF)
    Wd[:, 0] = 1  # dh = 1 in the first row, else 0
    dW, db, st = [torch.empty(F, d, device="cuda") for _ in range(3)], torch.empty(F, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(tw.twell_dense_gated_bwd_workspace_bytes(M, d, F), dtype=torch.uint8, device="cuda")
    tw.twell_dense_gated_ffn_bwd(x, W, W, Wd, act, g, u, u, dy, 0.0, None, *dW, False, db, ws, st)
    assert tw.twell_check(st) == 0
    open_ = (g[0] > 0).float()
    assert torch.equal(db, 2 * open_) and torch.equal(dW[0][:, 0], 2 * open_) and torch.equal(dW[1][:, 0], g[0].float() * open_)
