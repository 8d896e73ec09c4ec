"""A gradient's bits do not depend on which others a call asks for: products that would share a launch are summed in the
same order alone."""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def _rand(g, *shape, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(BF)


def _subsets(n):
    return [w for w in itertools.product((False, True), repeat=n) if any(w)]


@pytest.mark.parametrize("M,N,K", [(100, 264, 1000), (300, 1024, 1024), (1000, 1608, 1000), (2100, 1000, 264), (2048, 2696, 1000),
                                   (777, 5000, 520), (4100, 512, 512)])
@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("dw_type", [BF, F32], ids=["bf16", "f32"])
def test_linear(M, N, K, kn, dw_type):
    g = torch.Generator(device="cuda").manual_seed(1)
    x, W, dy, pre = _rand(g, M, K), _rand(g, *((K, N) if kn else (N, K)), scale=K ** -0.5), _rand(g, M, N), _rand(g, M, N)
    ws = torch.empty(tw.twell_linear_bwd_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(which):
        outs = [t if w else None for w, t in zip(which, (torch.empty_like(x), torch.empty_like(W, dtype=dw_type),
                                                         torch.empty(N, device="cuda")))]
        tw.twell_linear_bwd(dy, x, W, kn, tw.ACT_SILU, pre, outs[0], outs[1], False, outs[2], ws, st)
        return outs

    everything = call((True, True, True))
    for which in _subsets(3):
        got = call(which)
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, everything)), which
    assert tw.twell_check(st) == 0


@pytest.mark.parametrize("M,d,F", [(50, 64, 136), (300, 1000, 264), (777, 1000, 2696), (2048, 1000, 2696), (2100, 2056, 520),
                                   (260, 4096, 2056)])
@pytest.mark.parametrize("dw_type", [BF, F32], ids=["bf16", "f32"])
def test_gated(M, d, F, dw_type):
    g = torch.Generator(device="cuda").manual_seed(2)
    x, Wg, Wu, Wd = _rand(g, M, d), _rand(g, F, d, scale=d ** -0.5), _rand(g, F, d, scale=d ** -0.5), _rand(g, F, d, scale=F ** -0.5)
    gate, up, h, dy = _rand(g, M, F), _rand(g, M, F), _rand(g, M, F), _rand(g, M, d)
    ws = torch.empty(tw.twell_dense_gated_bwd_workspace_bytes(M, d, F), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(which):
        dx = torch.empty_like(x) if which[0] else None
        dW = [torch.empty_like(Wg, dtype=dw_type) if which[1] else None for _ in range(3)]
        db = torch.empty(F, device="cuda") if which[2] else None
        tw.twell_dense_gated_ffn_bwd(x, Wg, Wu, Wd, tw.ACT_SILU, gate, up, h, dy, 0.01, dx, *dW, False, db, ws, st)
        return [dx, *dW, db]

    everything = call((True, True, True))
    for which in _subsets(2):
        got = call((*which, True))
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, everything)), which
    assert tw.twell_check(st) == 0
