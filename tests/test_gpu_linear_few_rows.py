"""fp32 and bf16 results of few rows whose sums have many pieces: with the depth in one CTA (wide outputs) and split over a
cluster (narrow ones), an odd and an even number of pieces, W by rows and by depth, alone and with everything around it. The
errors are bounded as in dense_reference."""
import pytest
import torch

from dense_reference import BF, F32, SLOPE, act64, assert_within, depth_error, half_step

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402


@pytest.mark.parametrize("N,K", [(20008, 1544), (20008, 2048), (20008, 4104), (136, 14400), (264, 8200)])
@pytest.mark.parametrize("M", [5, 16, 20, 32, 50, 61, 64, 100, 128])
@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("t", [F32, BF], ids=["f32", "bf16"])
def test_forward(M, N, K, kn, t):
    if not kn and N > 10000:
        N -= 7  # odd widths too
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    x, W = rand(M, K).to(BF), (rand(*((K, N) if kn else (N, K))) * K ** -0.5).to(BF)
    b, res = rand(N), rand(M, N).to(t)
    y, full, pre = torch.full((M, N), 9.0, device="cuda", dtype=t), torch.full((M, N), 9.0, device="cuda", dtype=t), torch.empty(
        M, N, device="cuda", dtype=BF)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tw.twell_linear_fwd(x, W, kn, None, tw.ACT_NONE, None, None, y, st)
    tw.twell_linear_fwd(x, W, kn, b, tw.ACT_SILU, res, pre, full, st)
    assert tw.twell_check(st) == 0
    Wd = W.double() if kn else W.double().T
    z, tau = x.double() @ Wd, depth_error(256 if t is F32 else K, x.double().abs() @ Wd.abs()) + K / 256 * 2.0 ** -24 * (
        x.double().abs() @ Wd.abs())
    assert_within(y, z, tau + half_step(t) * (z.abs() + tau), "y")
    z = z + b.double()
    tau = tau + 2.0 ** -23 * z.abs()
    assert_within(pre, z, tau + half_step(BF) * (z.abs() + tau), "pre")
    want = act64(z, "silu")[0] + res.double()
    err = SLOPE * tau + 1e-6 * z.abs() + 2.0 ** -23 * want.abs()
    assert_within(full, want, err + half_step(t) * (want.abs() + err), "y with everything")
