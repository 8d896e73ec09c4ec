"""A backward that adds to gradients, with the weights frozen: only the input's and the bias's gradients are asked for."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

BF = torch.bfloat16


@pytest.mark.parametrize("M", [5, 200])
def test_accumulate_without_weight_gradients(M):
    N, K = 72, 64
    x, W, dy = (torch.randn(*s, device="cuda").to(BF) for s in ((M, K), (N, K), (M, N)))
    ws = torch.empty(max(tw.twell_linear_bwd_workspace_bytes(M, N, K), tw.twell_dense_gated_bwd_workspace_bytes(M, K, N)),
                     dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = []
    for accumulate in (False, True):
        dx, db = torch.empty_like(x), torch.empty(N, device="cuda")
        tw.twell_linear_bwd(dy, x, W, False, tw.ACT_SILU, dy, dx, None, accumulate, db, ws, st)
        dx2, db2 = torch.empty_like(x), torch.empty(N, device="cuda")
        tw.twell_dense_gated_ffn_bwd(x, W, W, W, tw.ACT_SILU, dy, dy, dy, x, 0.1, dx2, None, None, None, accumulate, db2, ws, st)
        out.append((dx, db, dx2, db2))
    assert tw.twell_check(st) == 0
    assert all(torch.equal(a, b) for a, b in zip(*out))
