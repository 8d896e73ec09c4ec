"""twell_xent_fwd / twell_xent_fwd_bwd against the definitions in 64 bits.

Tolerances. A logit is a sum of d exact products in fp32 on the tensor cores:
off by at most dz = d 2^-23 sum|x w| (their additions may round towards zero, so
2^-23 a step), which is also the most lse and a loss inherit from it; the
exponentials' sum (V / 32 + 64 steps, and 2^-21 for each exponential) adds
(V / 32 + 64) 2^-24 + 2^-21. In the gradient an exponential is rebuilt from its
code, which is off by half a step of 2^-11 of a power of two (2.0e-4 with the
rounding of the arithmetic around it), logits more than 32 powers of two below
their tile's maximum count as zero, and dz is then rounded to bf16 (8 significant
bits: half a unit in the last place is up to 2^-8 of the value).
The products dx and dW carry these errors with the magnitudes of their terms,
their own fp32 sums (V or N steps of 2^-23), and a bf16 result one more rounding
(2^-8).
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


def _inputs(N, d, V, seed=0, scale=1.5, ignored=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(N, d, device="cuda", generator=g).to(BF)
    W = (torch.randn(V, d, device="cuda", generator=g) * (scale / d ** 0.5)).to(BF)
    t = torch.randint(0, V, (N,), device="cuda", generator=g)
    t[torch.rand(N, device="cuda", generator=g) < ignored] = IGN
    return x, W, t


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _run(x, W, t, mean=True, grad=True, grad_scale=1.0, chunk=0, dw_dtype=BF, ignore=IGN, dW=None, accumulate=False,
         stream=None):
    (N, d), V = x.shape, W.shape[0]
    nll, lse = (torch.full((N,), 7.0, device="cuda") for _ in range(2))
    loss, st = torch.full((1,), 7.0, device="cuda"), _status()
    if not grad:
        ws = torch.empty(tw.twell_xent_fwd_workspace_bytes(N, d, V), dtype=torch.uint8, device="cuda").fill_(0xff)
        tw.twell_xent_fwd(x, W, t, ignore, mean, nll, lse, loss, ws, st, stream=stream)
        assert tw.twell_check(st, stream) == 0
        return nll, lse, loss
    dx = torch.full((N, d), 7.0, device="cuda", dtype=BF)
    dW = torch.full((V, d), 7.0, device="cuda", dtype=dw_dtype) if dW is None else dW
    code = tw.DTYPE_BF16 if dW.dtype is BF else tw.DTYPE_F32
    ws = torch.empty(tw.twell_xent_bwd_workspace_bytes(N, d, V, chunk, code), dtype=torch.uint8, device="cuda").fill_(0xff)
    torch.cuda.synchronize()
    tw.twell_xent_fwd_bwd(x, W, t, ignore, mean, grad_scale, chunk, nll, lse, loss, dx, dW, accumulate, ws, st,
                          stream=stream)
    assert tw.twell_check(st, stream) == 0
    return nll, lse, loss, dx, dW


def _check(x, W, t, out, mean=True, grad_scale=1.0, ignore=IGN, dW0=None):
    (N, d), V = x.shape, W.shape[0]
    rows = torch.nonzero(t != ignore)[:, 0]
    n = len(rows)
    X, Wd = x.double()[rows], W.double()
    z = X @ Wd.T
    lse = torch.logsumexp(z, 1)
    zt = z[torch.arange(n, device="cuda"), t[rows]]
    size = X.abs() @ Wd.abs().T                                  # sum |x w| of each logit
    dz = d * 2.0 ** -23 * size
    e_lse = dz.amax(1) + (V / 32 + 64) * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -23 * (1 + lse.abs() + z.abs().amax(1))
    e_nll = e_lse + dz.amax(1) + 2.0 ** -23 * zt.abs()
    nll_g, lse_g, loss_g = out[:3]
    off = t == ignore
    assert not nll_g[off].any() and not lse_g[off].any()
    assert bool(((lse_g.double()[rows] - lse).abs() <= e_lse).all())
    nll = lse - zt
    assert bool(((nll_g.double()[rows] - nll).abs() <= e_nll).all())
    total = float(nll.sum())
    want = total / n if mean and n else total
    allow = float(e_nll.sum()) / (n if mean and n else 1) + 2.0 ** -23 * abs(want)
    assert abs(float(loss_g) - want) <= allow
    if len(out) == 3:
        return
    dx_g, dW_g = out[3:]
    g = grad_scale / n if mean and n else grad_scale
    p = torch.exp(z - lse[:, None])
    grad = p.clone()
    grad[torch.arange(n, device="cuda"), t[rows]] -= 1.0
    grad *= g
    e_p = abs(g) * p * (2.0e-4 + 2 * (dz + e_lse[:, None])) + abs(g) * 2.0 ** -32
    e_dz = e_p + 2.0 ** -8 * grad.abs() + 2.0 ** -20 * grad.abs()
    # the target's own entry comes from its loss
    at = (torch.arange(n, device="cuda"), t[rows])
    e_dz[at] = abs(g) * (p[at] * 2 * e_nll + 2.0 ** -22) + 2.0 ** -8 * grad[at].abs()
    ref_dx = torch.zeros(N, d, dtype=torch.float64, device="cuda")
    ref_dx[rows] = grad @ Wd
    tol_dx = torch.zeros_like(ref_dx)
    tol_dx[rows] = e_dz @ Wd.abs() + V * 2.0 ** -23 * (grad.abs() @ Wd.abs())
    tol_dx += 2.0 ** -8 * ref_dx.abs() + 1e-38
    assert not dx_g[off].any()
    assert bool(((dx_g.double() - ref_dx).abs() <= tol_dx).all())
    ref_dW = grad.T @ X
    tol_dW = e_dz.T @ X.abs() + max(n, 1) * 2.0 ** -23 * (grad.abs().T @ X.abs())
    if dW0 is not None:
        ref_dW = ref_dW + dW0.double()
        tol_dW = tol_dW + 2.0 ** -22 * dW0.double().abs()
    tol_dW += (2.0 ** -8 if dW_g.dtype is BF else 2.0 ** -22) * ref_dW.abs() + 1e-38
    assert bool(((dW_g.double() - ref_dW).abs() <= tol_dW).all())
    # and as a whole: the bf16 roundings of dz are independent, so norms agree far better than the bounds above
    for got, ref in ((dx_g, ref_dx), (dW_g, ref_dW)):
        if float(ref.norm()) > 0:
            assert float((got.double() - ref).norm() / ref.norm()) < 5e-3


SHAPES = [(1, 8, 1), (1, 8, 2), (1, 64, 1000), (5, 16, 255), (64, 8, 256), (61, 520, 1000), (130, 64, 257), (257, 72, 511),
          (128, 1024, 4096), (300, 1000, 5001), (64, 8, 20000), (513, 264, 777), (1000, 128, 63), (2, 4096, 300),
          (200, 8, 8)]


@pytest.mark.parametrize("N,d,V", SHAPES)
@pytest.mark.parametrize("mean", [True, False])
def test_losses(N, d, V, mean):
    x, W, t = _inputs(N, d, V)
    _check(x, W, t, _run(x, W, t, mean, grad=False), mean)


@pytest.mark.parametrize("N,d,V", SHAPES)
@pytest.mark.parametrize("dw", [BF, F32])
def test_losses_and_gradients(N, d, V, dw):
    x, W, t = _inputs(N, d, V, seed=1)
    _check(x, W, t, _run(x, W, t, dw_dtype=dw))


@pytest.mark.parametrize("chunk", [1, 63, 64, 100, 256, 299, 300, 1000])
@pytest.mark.parametrize("dw", [BF, F32])
def test_rows_in_chunks(chunk, dw):
    x, W, t = _inputs(300, 200, 1333, seed=2)
    if chunk == 1:
        x, t = x[:9].contiguous(), t[:9].contiguous()
    out = _run(x, W, t, chunk=chunk, dw_dtype=dw)
    _check(x, W, t, out)
    whole = _run(x, W, t, dw_dtype=dw)
    assert all(torch.equal(a, b) for a, b in zip(out[:3], whole[:3]))


@pytest.mark.parametrize("chunk", [0, 100])
def test_sum_scale_and_accumulation(chunk):
    x, W, t = _inputs(270, 96, 700, seed=3)
    dW0 = torch.randn(700, 96, device="cuda")
    out = _run(x, W, t, mean=False, grad_scale=0.125, chunk=chunk, dW=dW0.clone(), accumulate=True)
    _check(x, W, t, out, mean=False, grad_scale=0.125, dW0=dW0)


@pytest.mark.parametrize("N", [2047, 2048, 2049, 5000])
@pytest.mark.parametrize("chunk", [0, 700])
def test_many_rows(N, chunk):
    x, W, t = _inputs(N, 72, 333, seed=13, ignored=0.4)
    _check(x, W, t, _run(x, W, t, chunk=chunk, dw_dtype=F32))
    _check(x, W, t, _run(x, W, t, chunk=chunk))


@pytest.mark.parametrize("N,scored", [(600, 1), (600, 255), (600, 257), (3000, 63), (3000, 64), (3000, 65)])
def test_few_of_the_rows_are_scored(N, scored):
    """The vocabulary is split for dx by the rows that are scored, known on the device only."""
    x, W, t = _inputs(N, 136, 9000, seed=14, ignored=0.0)
    order = torch.randperm(N, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    t[order[scored:]] = IGN
    _check(x, W, t, _run(x, W, t))
    _check(x, W, t, _run(x, W, t, chunk=500, dw_dtype=F32))


def test_losses_of_deep_products_are_centred():
    """d = 4096: the mean error of the log-sums. Sums that drop half a unit towards zero at each of 256 steps would be
    9e-6 low on these inputs (logits weighted by their probabilities average 2.2, 4e-6 of each is lost)."""
    x, W, t = _inputs(2048, 4096, 4096, seed=15, ignored=0.0)
    nll, lse, _ = _run(x, W, t, grad=False)
    z = x.double() @ W.double().T
    ref = torch.logsumexp(z, 1)
    assert abs(float((lse.double() - ref).mean())) < 2e-6
    want = ref - z.gather(1, t[:, None])[:, 0]
    assert float((nll.double() - want).norm() / want.norm()) < 1e-6


@pytest.mark.parametrize("dw", [BF, F32])
def test_no_row_is_scored(dw):
    x, W, t = _inputs(70, 64, 300)
    t.fill_(IGN)
    for chunk in (0, 30):
        nll, lse, loss, dx, dW = _run(x, W, t, chunk=chunk, dw_dtype=dw)
        assert not nll.any() and not lse.any() and not loss.any() and not dx.any() and not dW.any()
    dW0 = torch.randn(300, 64, device="cuda")
    out = _run(x, W, t, dW=dW0.clone(), accumulate=True)
    assert torch.equal(out[4], dW0)


@pytest.mark.parametrize("dw", [BF, F32])
def test_no_rows(dw):
    x, W, t = _inputs(0, 64, 300)
    nll, lse, loss, dx, dW = _run(x, W, t, dw_dtype=dw)
    assert float(loss) == 0.0 and not dW.any()
    assert float(_run(x, W, t, grad=False)[2]) == 0.0


def test_rows_that_are_not_scored_may_hold_anything():
    x, W, t = _inputs(333, 128, 900, seed=4, ignored=0.5)
    ref = _run(x, W, t)
    off = t == IGN
    for bad in (float("nan"), float("inf"), -float("inf")):
        y = x.clone()
        y[off] = bad
        out = _run(y, W, t)
        assert all(torch.equal(a, b) for a, b in zip(ref, out))


def test_bad_row_stays_alone():
    """A NaN in a scored row makes that row's loss and gradient NaN (and dW, which sums over the rows), no other row's."""
    x, W, t = _inputs(150, 64, 700, seed=5, ignored=0.0)
    ref = _run(x, W, t, mean=False)
    y = x.clone()
    y[77, 3] = float("nan")
    out = _run(y, W, t, mean=False)
    keep = torch.arange(150, device="cuda") != 77
    assert bool(out[0][77].isnan()) and bool(out[2].isnan().all()) and bool(out[3][77].isnan().all())
    for k in (0, 1, 3):
        assert torch.equal(out[k][keep], ref[k][keep])


def test_words_at_minus_infinity():
    """Words masked by a logit of -inf (whole tiles of them too) add nothing; a target among them has an infinite loss."""
    N, d, V = 70, 64, 900
    x, W, t = _inputs(N, d, V, seed=16, ignored=0.0)
    x[:, 0] = 1.0
    W[:, 0] = 0.0
    masked = torch.zeros(V, dtype=torch.bool, device="cuda")
    masked[:300] = True
    masked[520:650] = True
    masked[::7] = True
    W[masked, 0] = -float("inf")
    allowed = torch.nonzero(~masked)[:, 0]
    t = allowed[t % len(allowed)]
    kept = W[allowed].contiguous()
    place = torch.cumsum(~masked, 0) - 1
    ref = _run(x, kept, place[t], mean=False, grad=False)
    out = _run(x, W, t, mean=False, grad=False)
    for a, b in zip(out, ref):
        assert torch.allclose(a, b, rtol=2e-6, atol=0)
    t[5] = 10
    out = _run(x, W, t, mean=False, grad=False)
    assert float(out[0][5]) == float("inf") and float(out[2]) == float("inf")
    assert bool(out[0][6:].isfinite().all()) and torch.allclose(out[1], ref[1], rtol=2e-6, atol=0)
    W[:, 0] = -float("inf")  # nothing is left
    out = _run(x, W, t, mean=False, grad=False)
    assert bool((out[1] == -float("inf")).all()) and bool(out[0].isnan().all())


def test_ignore_index_may_be_a_word():
    x, W, t = _inputs(100, 64, 50, seed=6, ignored=0.0)
    t[::3] = 0
    _check(x, W, t, _run(x, W, t, ignore=0), ignore=0)


def test_steep_and_flat_rows():
    """Logits up to +-150: probabilities of 1 and below 2^-32, targets with either; and rows of equal logits."""
    N, d, V = 96, 64, 600
    x, W, t = _inputs(N, d, V, seed=7, ignored=0.0)
    x = (x.float() * torch.logspace(-2, 1.5, N, device="cuda")[:, None]).to(BF)
    best = (x.double() @ W.double().T)
    t[::2] = best.argmax(1)[::2]
    t[1::4] = best.argmin(1)[1::4]
    _check(x, W, t, _run(x, W, t))
    x.zero_()
    out = _run(x, W, t)
    _check(x, W, t, out)
    assert torch.allclose(out[1], torch.full((N,), float(torch.tensor(float(V)).log()), device="cuda"), rtol=1e-6)


def test_words_far_below_their_tile():
    """Whole 256-word tiles hundreds of powers of two below the row's maximum, before and after it."""
    N, d, V = 40, 8, 1024
    x = torch.ones(N, d, device="cuda", dtype=BF)
    W = torch.zeros(V, d, device="cuda", dtype=BF)
    W[:256] = -30.0
    W[256:300] = 10.0
    W[300:512] = 9.0
    W[512:] = 5.0
    t = torch.arange(N, device="cuda") * 25
    _check(x, W, t, _run(x, W, t))


def test_gradients_against_differences():
    """Differences of the 64-bit loss along random directions against the kernels' gradients: the directional derivative
    of a bf16 gradient is off by at most the 5e-3 (norm-wise) of its roundings, times both norms."""
    x, W, t = _inputs(60, 48, 301, seed=8)
    _, _, _, dx, dW = _run(x, W, t, dw_dtype=F32)
    rows = t != IGN
    h = 1e-4

    def loss(X, Wd):
        z = X[rows] @ Wd.T
        return float((torch.logsumexp(z, 1) - z.gather(1, t[rows][:, None])[:, 0]).mean())

    X, Wd = x.double(), W.double()
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        vx = torch.randn(X.shape, device="cuda", dtype=torch.float64, generator=g)
        vw = torch.randn(Wd.shape, device="cuda", dtype=torch.float64, generator=g)
        for got, v, slope in ((dx, vx, (loss(X + h * vx, Wd) - loss(X - h * vx, Wd)) / (2 * h)),
                              (dW, vw, (loss(X, Wd + h * vw) - loss(X, Wd - h * vw)) / (2 * h))):
            assert abs(float((got.double() * v).sum()) - slope) <= 5e-3 * float(got.double().norm()) * 6 + 1e-6


def test_same_bits_every_time_and_on_another_stream():
    x, W, t = _inputs(700, 264, 3001, seed=9)
    ref = _run(x, W, t)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.current_stream()):
        out = _run(x, W, t, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, out))


def test_replayed_from_a_graph():
    x, W, t = _inputs(200, 128, 1001, seed=10)
    N, d, V = 200, 128, 1001
    nll, lse, loss = torch.empty(N, device="cuda"), torch.empty(N, device="cuda"), torch.empty(1, device="cuda")
    dx, dW = torch.empty_like(x), torch.empty_like(W)
    ws = torch.empty(tw.twell_xent_bwd_workspace_bytes(N, d, V, 0, tw.DTYPE_BF16), dtype=torch.uint8, device="cuda")
    st = _status()
    args = (x, W, t, IGN, True, 1.0, 0, nll, lse, loss, dx, dW, False, ws, st)
    tw.twell_xent_fwd_bwd(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tw.twell_xent_fwd_bwd(*args)
    x2, _, t2 = _inputs(N, d, V, seed=11, ignored=0.6)
    x.copy_(x2)
    t.copy_(t2)
    graph.replay()
    torch.cuda.synchronize()
    out = _run(x, W, t)
    assert all(torch.equal(a, b) for a, b in zip((nll, lse, loss, dx, dW), out))


def test_target_outside_the_vocabulary_is_reported():
    for bad in (300, -1, 2 ** 40, -2 ** 40):
        x, W, t = _inputs(40, 64, 300, ignored=0.0)
        t[11] = bad
        N, d, V = 40, 64, 300
        nll, lse, loss = torch.empty(N, device="cuda"), torch.empty(N, device="cuda"), torch.empty(1, device="cuda")
        ws = torch.empty(tw.twell_xent_bwd_workspace_bytes(N, d, V, 0, tw.DTYPE_BF16), dtype=torch.uint8, device="cuda")
        st = _status()
        tw.twell_xent_fwd_bwd(x, W, t, IGN, True, 1.0, 0, nll, lse, loss, torch.empty_like(x), torch.empty_like(W), False,
                              ws, st)
        assert tw.twell_check(st) == 1
        st = _status()
        tw.twell_xent_fwd(x, W, t, IGN, True, nll, lse, loss, ws, st)
        assert tw.twell_check(st) == 1


def test_codes_past_32_bit_offsets():
    """2.6e9 codes in one chunk: the last rows against the same rows alone."""
    N, d, V = 40_000, 8, 65_536
    if torch.cuda.mem_get_info()[0] < 20e9:
        pytest.skip("needs 20 GB")
    x, W, t = _inputs(N, d, V, seed=12, ignored=0.0, scale=4.0)
    out = _run(x, W, t, mean=False)
    tail = _run(x[-300:].contiguous(), W, t[-300:].contiguous(), mean=False)
    assert torch.equal(out[0][-300:], tail[0]) and torch.equal(out[1][-300:], tail[1])
    a, b = out[3][-300:].double(), tail[3].double()
    assert float((a - b).norm() / b.norm()) < 3e-3  # the vocabulary is split differently: sums in another order
    _check(x[-300:].contiguous(), W, t[-300:].contiguous(), tail, mean=False)


def test_wrong_arguments_are_refused():
    x, W, t = _inputs(16, 64, 100)
    nll, lse, loss = torch.empty(16, device="cuda"), torch.empty(16, device="cuda"), torch.empty(1, device="cuda")
    dx, dW, st = torch.empty_like(x), torch.empty_like(W), _status()
    ws = torch.empty(tw.twell_xent_bwd_workspace_bytes(16, 64, 100, 0, tw.DTYPE_BF16), dtype=torch.uint8, device="cuda")

    def call(x=x, W=W, t=t, nll=nll, dx=dx, dW=dW, acc=False, ws=ws, chunk=0):
        tw.twell_xent_fwd_bwd(x, W, t, IGN, True, 1.0, chunk, nll, lse, loss, dx, dW, acc, ws, st)

    for bad in (dict(x=x.float()), dict(W=W.float()), dict(t=t.int()), dict(nll=nll[:5]), dict(dx=dx.float()),
                dict(x=x[:, :56]), dict(W=W.cpu()), dict(dW=torch.empty(99, 64, device="cuda")), dict(t=t[:3])):
        with pytest.raises(ValueError):
            call(**bad)
    for bad, status in ((dict(acc=True), 1), (dict(ws=ws[:1024]), 3), (dict(chunk=-1), 1)):
        with pytest.raises(tw.TwellError) as e:
            call(**bad)
        assert e.value.status == status
    with pytest.raises(tw.TwellError) as e:  # a width that is not a multiple of 8
        call(x=x[:, :60].contiguous(), W=W[:, :60].contiguous(), dx=dx[:, :60].contiguous(), dW=dW[:, :60].contiguous())
    assert e.value.status == 1
