"""The last digits of the cross entropy: rows whose loss is near 0, log-sums of exact logits, and deep products.

Tolerances. The sum of a row's exponentials, relative to its maximum, is taken with
exponentials good to 2^-22 each, a second one where tiles are joined, and a
logarithm of it within 2^-23: E = 2^-21 + 2^-23 absolute where one word has nearly
all of the probability. A log-sum adds its own rounding (half a unit in the last
place) and the rounding of log2(e) to fp32 (1.4e-8 of the maximum).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
IGN = -100
E = 2.0 ** -21 + 2.0 ** -23


def _losses(x, W, t, status=None):
    (N, d), V = x.shape, W.shape[0]
    nll, lse, loss = torch.full((N,), 7.0, device="cuda"), torch.full((N,), 7.0, device="cuda"), torch.full((1,), 7.0, device="cuda")
    ws = torch.empty(tw.twell_xent_fwd_workspace_bytes(N, d, V), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
    tw.twell_xent_fwd(x, W, t, IGN, False, nll, lse, loss, ws, st)
    if status is None:
        assert tw.twell_check(st) == 0
    return nll, lse, loss


def _ulp(v):
    return torch.exp2(torch.floor(torch.log2(v.abs())) - 23)


def _exact_rows(N, d, V, seed=0):
    """One word's logit is a product of two bf16 numbers (16 bits), all others are 0: every logit is exact in fp32."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros(N, d, device="cuda", dtype=BF)
    at = torch.randint(0, d, (N,), device="cuda", generator=g)
    x[torch.arange(N, device="cuda"), at] = (4 + 4 * torch.rand(N, device="cuda", generator=g)).to(BF)
    W = torch.zeros(V, d, device="cuda", dtype=BF)
    W[V // 2] = (6 + 6 * torch.rand(d, device="cuda", generator=g)).to(BF)
    t = torch.full((N,), V // 2, device="cuda")
    z = x.double() @ W.double().T
    return x, W, t, z


def _check_log_sums(N, d, V):
    x, W, t, z = _exact_rows(N, d, V)
    _, lse, _ = _losses(x, W, t)
    ref = torch.logsumexp(z, 1)
    assert bool(((lse.double() - ref).abs() <= 0.5 * _ulp(ref) + E + 1.4e-8 * z.amax(1)).all())


@pytest.mark.parametrize("d", [8, 64])
def test_log_sums_of_exact_logits(d):
    """Nothing is lost or counted twice between the maximum, log2 and log."""
    _check_log_sums(2000, d, 300)


def _confident(N, d, V, seed=1):
    """Word 7's logit is between 15 and 60, all others are as far below 0: losses under 1e-11."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    sign = torch.where(torch.rand(d, device="cuda", generator=g) < 0.5, -1.0, 1.0)
    size = 0.5 + torch.rand(N, d, device="cuda", generator=g)
    x = (sign * size * torch.linspace(1, 3.5, N, device="cuda")[:, None]).to(BF)
    W = (-sign * (0.5 + torch.rand(V, d, device="cuda", generator=g)) * (18.0 / d)).to(BF)
    W[7] = -W[7]
    return x, W, torch.full((N,), 7, device="cuda")


@pytest.mark.parametrize("d", [8, 64, 1000, 1024, 4096])
def test_confident_rows_have_no_loss_and_no_gradient(d):
    """The target's logit and the log-sum cancel: a loss is not negative, and its error is that of a sum near 1, not that
    of logits of 60."""
    N, V = 256, 600
    x, W, t = _confident(N, d, V)
    z = x.double() @ W.double().T
    assert 10 < float(z[:, 7].min()) and float(z[:, 7].max()) > 50
    ref = torch.logsumexp(z, 1) - z[:, 7]
    nll, _, loss = _losses(x, W, t)
    assert bool((nll >= 0).all()) and float(loss) >= 0
    assert bool(((nll.double() - ref).abs() <= E).all())
    # the target's gradient expm1(-nll) is not positive: with one word left, dx = dz W has the sign of -W
    dx, dW = torch.empty_like(x), torch.empty(V, d, device="cuda")
    nll, lse, loss = torch.empty(N, device="cuda"), torch.empty(N, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(tw.twell_xent_bwd_workspace_bytes(N, d, V, 0, tw.DTYPE_F32), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tw.twell_xent_fwd_bwd(x, W, t, IGN, False, 1.0, 0, nll, lse, loss, dx, dW, False, ws, st)
    assert tw.twell_check(st) == 0
    assert bool((dx.float() * W[7].float() <= 1e-10).all())
    assert bool((dx.float().abs() <= 1.01 * E * W[7].float().abs() + 1e-10).all())


@pytest.mark.parametrize("V", [300, 5001])
def test_losses_of_likely_targets(V):
    """Losses between 1e-4 and 1 beside logits of 40: relative to 1, no digit is lost to the logits' size."""
    N, d = 512, 64
    x = torch.zeros(N, d, device="cuda", dtype=BF)
    x[:, 0], x[:, 1] = 1.0, torch.linspace(0, 9, N, device="cuda").to(BF)
    W = torch.zeros(V, d, device="cuda", dtype=BF)
    W[:, 0] = 20.0
    W[3, 0], W[V - 2, 0], W[V - 2, 1] = 40.0, 39.0, -1.0   # logits 40, 39 - x, and 20: exact in fp32
    for word in (3, V - 2):
        t = torch.full((N,), word, device="cuda")
        z = x.double() @ W.double().T
        ref = torch.logsumexp(z, 1) - z[:, word]
        nll = _losses(x, W, t)[0].double()
        # log2(e) times the logits' differences (1.4e-8 and two roundings, 2^-23 of them) and the sum near 1
        assert bool(((nll - ref).abs() <= E + (2.0 ** -22 + 1.4e-8) * (1 + ref)).all())


@pytest.mark.parametrize("d", [1024, 4096, 16384])
def test_log_sums_of_exact_logits_of_wide_rows(d):
    """A product of one term is that term, whatever the width."""
    _check_log_sums(300, d, 300)


@pytest.mark.parametrize("d", [512, 2048, 4096, 16384])
def test_deep_sums_of_one_sign(d):
    """With one word a log-sum is its logit. The tensor cores' sums lose up to a unit (2^-23) at each step of 16, towards
    zero; over 512 of depth that is at most 16.5 units of the sum, half of it on average if rounding is as likely to lose
    little as much, and the pieces' sums are joined with nearest rounding (a unit's half each, either way)."""
    N = 512
    g = torch.Generator(device="cuda").manual_seed(2)
    x = (0.5 + torch.rand(N, d, device="cuda", generator=g)).to(BF)
    W = ((0.5 + torch.rand(1, d, device="cuda", generator=g)) * (30.0 / d)).to(BF)
    _, lse, _ = _losses(x, W, torch.zeros(N, dtype=torch.int64, device="cuda"))
    z = (x.double() @ W.double().T)[:, 0]
    rel = (lse.double() - z) / z
    assert float(rel.abs().max()) <= (16.5 + d / 512) * 2.0 ** -23
    assert abs(float(rel.mean())) <= 8.25 * 2.0 ** -23


@pytest.mark.parametrize("N", [100, 2048, 2049, 5000])
@pytest.mark.parametrize("grad", [False, True])
def test_nothing_is_written_after_an_error(N, grad):
    """A status that an earlier kernel set: every later kernel skips its work, whatever the number of rows."""
    d, V = 64, 300
    g = torch.Generator(device="cuda").manual_seed(3)
    x, W = torch.randn(N, d, device="cuda", generator=g).to(BF), torch.randn(V, d, device="cuda", generator=g).to(BF)
    t = torch.randint(0, V, (N,), device="cuda", generator=g)
    t[::3] = IGN
    st = torch.full((1,), 4, dtype=torch.int32, device="cuda")
    if not grad:
        out = _losses(x, W, t, status=st)
    else:
        out = [torch.full((N,), 7.0, device="cuda"), torch.full((N,), 7.0, device="cuda"), torch.full((1,), 7.0, device="cuda"),
               torch.full_like(x, 7.0), torch.full_like(W, 7.0)]
        ws = torch.empty(tw.twell_xent_bwd_workspace_bytes(N, d, V, 0, tw.DTYPE_BF16), dtype=torch.uint8, device="cuda")
        tw.twell_xent_fwd_bwd(x, W, t, IGN, True, 1.0, 0, *out, False, ws, st)
    assert tw.twell_check(st) == 4
    assert all(bool((o == 7.0).all()) for o in out)
