"""The linear and gated layers' gradients against central differences in 64 bits, along the gradient itself, along its parts and
in random directions, with the bounds of dense_differences (which a gradient of zeros, one that is a quarter too long or one
without a term fails, as test_dense_differences shows)."""
import pytest
import torch

from dense_differences import Gated, Linear, difference, directions

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

BF = torch.bfloat16
CODE = {"silu": tw.ACT_SILU, "gelu": tw.ACT_GELU, "gelu_tanh": tw.ACT_GELU_TANH}


def _bf(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(BF).cuda()


def _check(case, grads, others, gen):
    right = case.gradients()
    for i, name in enumerate(case.names):
        for v in directions([right[i], *(o[i] - right[i] for o in others)], gen):
            off = abs(float((grads[i].double() * v).sum() - difference(case.loss, case.at, i, v)))
            assert off <= float(case.bound(i, v)), (name, off, float(case.bound(i, v)))


@pytest.mark.parametrize("act", list(CODE))
@pytest.mark.parametrize("M,N,K", [(5, 72, 64), (60, 72, 64), (300, 264, 136)])
@pytest.mark.parametrize("kn", [False, True])
def test_linear(act, M, N, K, kn):
    gen = torch.Generator().manual_seed(1)
    x, W, b, dy = _bf(gen, M, K), _bf(gen, N, K, scale=K ** -0.5), torch.randn(N, generator=gen).cuda(), _bf(gen, M, N)
    stored = W.T.contiguous() if kn else W
    y, pre, dx = torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(x)
    dW, db = torch.empty(stored.shape, device="cuda"), torch.empty(N, device="cuda")
    ws = torch.empty(tw.twell_linear_bwd_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tw.twell_linear_fwd(x, stored, kn, b, CODE[act], None, pre, y, st)
    tw.twell_linear_bwd(dy, x, stored, kn, CODE[act], pre, dx, dW, False, db, ws, st)
    assert tw.twell_check(st) == 0
    case = Linear(x, W, b, dy, act)
    _check(case, (dx, dW.T if kn else dW, db), [case.gradients(slope=False)], gen)


@pytest.mark.parametrize("act", list(CODE))
@pytest.mark.parametrize("M,d,F", [(5, 64, 72), (50, 64, 72), (300, 136, 264)])
def test_gated(act, M, d, F):
    gen = torch.Generator().manual_seed(2)
    x, Wg, Wu = _bf(gen, M, d), _bf(gen, F, d, scale=d ** -0.5), _bf(gen, F, d, scale=d ** -0.5)
    Wd, b, dy, l1 = _bf(gen, F, d, scale=F ** -0.5), (0.3 * torch.randn(F, generator=gen)).cuda(), _bf(gen, M, d), 0.3
    g, u, h = (torch.empty(M, F, device="cuda", dtype=BF) for _ in range(3))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dW, db = [torch.empty(F, d, device="cuda") for _ in range(3)], torch.empty(F, device="cuda")
    ws = torch.empty(tw.twell_dense_gated_bwd_workspace_bytes(M, d, F), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tw.twell_dense_gated_ffn_fwd(x, Wg, Wu, b, Wd, CODE[act], None, g, u, h, y, st)
    tw.twell_dense_gated_ffn_bwd(x, Wg, Wu, Wd, CODE[act], g, u, h, dy, l1, dx, *dW, False, db, ws, st)
    assert tw.twell_check(st) == 0
    case = Gated(x, Wg, Wu, Wd, b, dy, act, l1)
    _check(case, (dx, *dW, db), [case.gradients(slope=False), case.gradients(l1=0.0), case.gradients(of_dy=0.0)], gen)
