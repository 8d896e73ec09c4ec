"""The gated layer's gradients have the same bits with and without the bias's gradient."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

BF = torch.bfloat16


@pytest.mark.parametrize("M,d,F", [(50, 64, 136), (300, 1000, 264), (777, 1000, 2696), (260, 4096, 2056), (2100, 2056, 520)])
def test_with_and_without(M, d, F):
    g = torch.Generator(device="cuda").manual_seed(2)

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(BF)

    x, Wg, Wu, Wd = rand(M, d), rand(F, d, scale=d ** -0.5), rand(F, d, scale=d ** -0.5), rand(F, d, scale=F ** -0.5)
    gate, up, h, dy = rand(M, F), rand(M, F), rand(M, F), rand(M, d)
    ws = torch.empty(tw.twell_dense_gated_bwd_workspace_bytes(M, d, F), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = []
    for db in (torch.empty(F, device="cuda"), None):
        grads = [torch.empty_like(x), *(torch.empty(F, d, device="cuda") for _ in range(3))]
        tw.twell_dense_gated_ffn_bwd(x, Wg, Wu, Wd, tw.ACT_SILU, gate, up, h, dy, 0.01, *grads, False, db, ws, st)
        out.append(grads)
    assert tw.twell_check(st) == 0
    assert all(torch.equal(a, b) for a, b in zip(*out))
