"""twell_linear_fwd and twell_linear_bwd against the formulas in 64 bits, with the bounds of dense_reference."""
import pytest
import torch

from dense_reference import ACTS, BF, F32, SLOPE, act64, assert_within, depth_error, half_step

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

CODE = {"none": tw.ACT_NONE, "relu": tw.ACT_RELU, "silu": tw.ACT_SILU, "gelu": tw.ACT_GELU, "gelu_tanh": tw.ACT_GELU_TANH}


def _rand(g, *shape, scale=1.0, t=BF, pad=0, offset=0):
    """A random matrix whose rows lie `pad` elements apart, starting `offset` elements into its memory."""
    base = torch.full((shape[0] * (shape[1] + pad) + offset,), 7.0, device="cuda", dtype=t)
    out = base[offset:].view(shape[0], shape[1] + pad)[:, :shape[1]]
    out.copy_(torch.randn(*shape, device="cuda", generator=g) * scale)
    return out


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _forward(M, N, K, kn, act, y_type, bias, res, save, pad=0, offset=0, seed=0, stream=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = _rand(g, M, K, pad=8 if pad else 0)
    W = _rand(g, *((K, N) if kn else (N, K)), scale=K ** -0.5)
    b = torch.randn(N, device="cuda", generator=g) if bias else None
    r = _rand(g, M, N, t=y_type, pad=pad, offset=offset) if res else None
    y = torch.full((M * (N + pad) + offset,), 9.0, device="cuda", dtype=y_type)
    pre = torch.full((M * (N + pad) + offset,), 9.0, device="cuda", dtype=BF) if save else None
    view = lambda t: None if t is None else t[offset:].view(M, N + pad)[:, :N]  # noqa: E731
    st = _status()
    tw.twell_linear_fwd(x, W, kn, b, CODE[act], r, view(pre), view(y), st, stream=stream)
    assert tw.twell_check(st) == 0
    Wd = W.double() if kn else W.double().T
    z = x.double() @ Wd + (b.double() if bias else 0.0)
    tau = depth_error(K, x.double().abs() @ Wd.abs()) + 2.0 ** -23 * z.abs()
    if save:
        assert_within(view(pre), z, tau + half_step(BF) * (z.abs() + tau), "pre")
        if pad:
            assert bool((pre[offset:].view(M, N + pad)[:, N:] == 9.0).all())
    a = act64(z, act)[0]
    want = a + (r.double() if res else 0.0)
    err = SLOPE * tau + (1e-6 * z.abs() if act not in ("none", "relu") else 0.0) + 2.0 ** -23 * want.abs()
    assert_within(view(y), want, err + half_step(y_type) * (want.abs() + err), "y")
    if pad:
        assert bool((y[offset:].view(M, N + pad)[:, N:] == 9.0).all())
    assert bool((y[:offset] == 9.0).all())


SIZES = [(1, 8, 8), (1, 4096, 4096), (2, 51, 64), (7, 257, 72), (16, 1000, 1032), (17, 130, 2048), (33, 50001, 128),
         (64, 384, 4104), (65, 640, 520), (128, 264, 1000), (129, 1001, 64), (200, 8, 192), (257, 513, 2056), (300, 2048, 24),
         (512, 4096, 1024), (1030, 777, 264)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("y_type", [BF, F32], ids=["bf16", "f32"])
def test_forward_plain(M, N, K, y_type):
    _forward(M, N, K, False, "none", y_type, False, False, False)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward_everything(M, N, K):
    _forward(M, N, K, False, "silu", BF, True, True, True)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 14336), (3, 64, 2696), (33, 1000, 520), (100, 264, 72), (260, 1024, 1000), (600, 520, 64)])
@pytest.mark.parametrize("y_type", [BF, F32], ids=["bf16", "f32"])
def test_forward_of_weights_by_depth(M, N, K, y_type):
    _forward(M, N, K, True, "gelu", y_type, True, True, True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("y_type", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M", [5, 300])
def test_activations(act, y_type, M):
    _forward(M, 264, 136, False, act, y_type, True, False, True)


@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 0), (5, 3), (64, 1)])
@pytest.mark.parametrize("M", [3, 50, 290])
@pytest.mark.parametrize("y_type", [BF, F32], ids=["bf16", "f32"])
def test_strides_and_alignment(pad, offset, M, y_type):
    """Rows that start anywhere; what lies between them stays."""
    for N in (96, 101):
        _forward(M, N, 200, False, "relu", y_type, True, True, True, pad=pad, offset=offset)


@pytest.mark.parametrize("M,N,K,kn", [(65, 20001, 1544, False), (100, 20000, 2048, True), (128, 20001, 4096, False), (127, 1000, 14336, True),
                                      (128, 136, 14400, False), (200, 2048, 8192, False), (1000, 640, 4104, False)])
def test_fp32_results_of_any_depth(M, N, K, kn):
    """fp32 results are summed in pieces of at most 48 steps of the tensor cores (K = 16 each). A step drops at most 2^-23
    of the sum so far, which after s steps is sqrt(s / 48) of the piece's in the mean square: 2/3 of 48 units of 2^-23 of
    a piece, and as much of the result, since the pieces are independent; and half a unit for each piece added."""
    _forward(M, N, K, kn, "gelu", F32, True, True, True)
    g = torch.Generator(device="cuda").manual_seed(7)
    x, W = _rand(g, M, K), _rand(g, *((K, N) if kn else (N, K)), scale=K ** -0.5)
    y, again = (torch.empty(M, N, device="cuda") for _ in range(2))
    st = _status()
    for out in (y, again):
        tw.twell_linear_fwd(x, W, kn, None, tw.ACT_NONE, None, None, out, st)
    assert tw.twell_check(st) == 0 and torch.equal(y, again)
    want = x.double() @ (W.double() if kn else W.double().T)
    assert float((y.double() - want).norm() / want.norm()) <= (2 / 3 * 48 + K / 768) * 2.0 ** -23


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("N,K", [(1, 8), (3, 264), (1000, 520), (130, 8200), (5001, 1288), (8192, 8192)])
@pytest.mark.parametrize("y_type", [BF, F32], ids=["bf16", "f32"])
def test_single_tokens(M, N, K, y_type):
    _forward(M, N, K, False, "gelu", y_type, True, True, True)
    _forward(M, N, K, False, "none", y_type, False, False, False, pad=3, offset=1)


def test_residual_in_place():
    g = torch.Generator(device="cuda").manual_seed(3)
    for M in (1, 40, 300):
        for t in (BF, F32):
            x, W, r = _rand(g, M, 256), _rand(g, 128, 256, scale=1 / 16), _rand(g, M, 128, t=t)
            y = torch.empty_like(r)
            st = _status()
            tw.twell_linear_fwd(x, W, False, None, tw.ACT_NONE, r, None, y, st)
            tw.twell_linear_fwd(x, W, False, None, tw.ACT_NONE, r, None, r, st)
            assert tw.twell_check(st) == 0 and torch.equal(r, y)


@pytest.mark.parametrize("M", [2, 70, 300])
def test_non_finite_values_stay_in_their_rows(M):
    g = torch.Generator(device="cuda").manual_seed(4)
    x, W = _rand(g, M, 200), _rand(g, 150, 200, scale=0.1)
    clean = torch.empty(M, 150, device="cuda", dtype=BF)
    y = torch.empty_like(clean)
    st = _status()
    tw.twell_linear_fwd(x, W, False, None, tw.ACT_NONE, None, None, clean, st)
    x[1, 3], x[0, 5] = float("nan"), float("inf")
    tw.twell_linear_fwd(x, W, False, None, tw.ACT_NONE, None, None, y, st)
    assert tw.twell_check(st) == 0
    assert bool(y[1].isnan().all()) and not bool(y[0].isfinite().any())
    assert torch.equal(y[2:], clean[2:])


def _backward(M, N, K, kn, act, dw_type=BF, accumulate=False, pad=0, offset=0, with_dx=True, with_dw=True, with_db=True, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = _rand(g, M, K, pad=8 if pad else 0)
    W = _rand(g, *((K, N) if kn else (N, K)), scale=K ** -0.5)
    dy = _rand(g, M, N, pad=pad, offset=offset)
    pre = _rand(g, M, N, pad=pad, offset=offset, scale=2.0) if act != "none" else None
    dx = torch.full((M, K), 9.0, device="cuda", dtype=BF) if with_dx else None
    dW0 = torch.randn(W.shape, device="cuda", generator=g) if accumulate else torch.full(W.shape, 9.0, device="cuda")
    dW = dW0.to(dw_type).clone() if with_dw else None
    db = torch.full((N,), 9.0, device="cuda") if with_db else None
    ws = torch.empty(tw.twell_linear_bwd_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda").fill_(255)
    st = _status()
    tw.twell_linear_bwd(dy, x, W, kn, CODE[act], pre, dx, dW, accumulate, db, ws, st)
    assert tw.twell_check(st) == 0
    X, Wm, d = x.double(), (W.double().T if kn else W.double()), dy.double()  # Wm [N, K]
    slip = torch.zeros_like(d)  # error of the dpre that enters the products
    if pre is not None:
        z = pre.double()
        d = d * act64(z, act)[1]
        exact = act == "relu"
        own = 0.0 if exact else 2e-6 * (1 + z.abs()) * dy.double().abs()
        slip = own + (0.0 if exact else half_step(BF)) * (d.abs() + own)
    if with_dx:
        want, mag = d @ Wm, d.abs() @ Wm.abs()
        err = slip @ Wm.abs() + depth_error(N, mag)
        assert_within(dx, want, err + half_step(BF) * (want.abs() + err), "dx")
    if with_dw:
        want, mag = d.T @ X, d.abs().T @ X.abs()
        err = slip.T @ X.abs() + depth_error(M, mag)
        if kn:
            want, err = want.T, err.T
        if accumulate:
            want = want + dW0.double()
            err = err + 2.0 ** -23 * want.abs()
        assert_within(dW, want, err + half_step(dw_type) * (want.abs() + err), "dW")
    if with_db:
        own = 0.0 if pre is None or act == "relu" else 2e-6 * (1 + pre.double().abs()) * dy.double().abs()
        err = ((M / 16 + 64) * 2.0 ** -24 * d.abs() + own).sum(0)
        assert_within(db, d.sum(0), err, "dbias")


BWD = [(1, 8, 8), (7, 264, 72), (63, 51, 64), (130, 1001, 136), (300, 520, 1000), (777, 96, 2048), (2100, 300, 264)]


@pytest.mark.parametrize("M,N,K", BWD)
@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
@pytest.mark.parametrize("dw_type", [BF, F32], ids=["bf16", "f32"])
def test_backward(M, N, K, act, dw_type):
    _backward(M, N, K, False, act, dw_type)


@pytest.mark.parametrize("M,N,K", [(5, 64, 72), (300, 264, 520), (513, 1024, 136)])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("dw_type", [BF, F32], ids=["bf16", "f32"])
def test_backward_of_weights_by_depth(M, N, K, act, dw_type):
    _backward(M, N, K, True, act, dw_type)


@pytest.mark.parametrize("M,N,K", [(300, 1024, 1024), (1000, 4096, 1032), (2000, 2304, 2312), (4100, 1000, 3992)])
@pytest.mark.parametrize("kn", [False, True])
@pytest.mark.parametrize("dw_type,accumulate", [(BF, False), (F32, True)], ids=["bf16", "f32_added"])
def test_backward_of_two_products_in_one_launch(M, N, K, kn, dw_type, accumulate):
    """One or several rounds of tiles in either product, in the last of which some pairs have none."""
    _backward(M, N, K, kn, "relu", dw_type, accumulate)


@pytest.mark.parametrize("act", ACTS)
def test_backward_activations(act):
    _backward(257, 264, 200, False, act)


@pytest.mark.parametrize("kn", [False, True])
def test_backward_adds_to_a_gradient(kn):
    _backward(300, 264, 200, kn, "relu", F32, accumulate=True)


@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 0), (5, 1)])
def test_backward_strides(pad, offset):
    for N in (96, 101):
        for act in ("none", "silu"):
            _backward(70, N, 200, False, act, pad=pad, offset=offset)


@pytest.mark.parametrize("which", [(True, False, False), (False, True, False), (False, False, True), (True, False, True)])
def test_backward_of_some(which):
    for act in ("none", "gelu"):
        _backward(100, 96, 64, False, act, with_dx=which[0], with_dw=which[1], with_db=which[2])


def test_no_rows():
    W = torch.randn(16, 8, device="cuda").to(BF)
    x, y = torch.empty(0, 8, device="cuda", dtype=BF), torch.empty(0, 16, device="cuda", dtype=BF)
    st = _status()
    tw.twell_linear_fwd(x, W, False, None, tw.ACT_NONE, None, None, y, st)
    dW, db = torch.ones(16, 8, device="cuda"), torch.ones(16, device="cuda")
    ws = torch.empty(tw.twell_linear_bwd_workspace_bytes(0, 16, 8), dtype=torch.uint8, device="cuda")
    tw.twell_linear_bwd(y, x, W, False, tw.ACT_NONE, None, torch.empty_like(x), dW, True, db, ws, st)
    assert tw.twell_check(st) == 0 and bool((dW == 1).all()) and not bool(db.any())
    tw.twell_linear_bwd(y, x, W, False, tw.ACT_NONE, None, None, dW, False, None, ws, st)
    assert tw.twell_check(st) == 0 and not bool(dW.any())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gradients_against_differences(act):
    """<gradient, direction> against central differences of L = <dy, y> in 64 bits at the bf16 point. The kept
    pre-activation is rounded (2^-8 of |z|, times a curvature of at most 1.2), dpre and the results too: 4 x 2^-8 of
    the terms' magnitudes."""
    g = torch.Generator(device="cuda").manual_seed(6)
    M, N, K = 60, 72, 64
    x, W, dy = _rand(g, M, K), _rand(g, N, K, scale=K ** -0.5), _rand(g, M, N)
    b = torch.randn(N, device="cuda", generator=g)
    y, pre = torch.empty(M, N, device="cuda", dtype=BF), torch.empty(M, N, device="cuda", dtype=BF)
    dx, dW, db = torch.empty_like(x), torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
    ws = torch.empty(tw.twell_linear_bwd_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
    st = _status()
    tw.twell_linear_fwd(x, W, False, b, CODE[act], None, pre, y, st)
    tw.twell_linear_bwd(dy, x, W, False, CODE[act], pre, dx, dW, False, db, ws, st)
    assert tw.twell_check(st) == 0

    def loss(x, W, b):
        return (dy.double() * act64(x @ W.T + b, act)[0]).sum()

    at = [x.double(), W.double(), b.double()]
    z = at[0] @ at[1].T + at[2]
    size = dy.double().abs() * (1 + z.abs())
    sizes = [size @ at[1].abs(), size.T @ at[0].abs(), size.sum(0)]
    for i, (grad, total) in enumerate(zip((dx, dW, db), sizes)):
        v = torch.randn(at[i].shape, device="cuda", generator=g, dtype=torch.float64)
        eps = 1e-6
        up, down = [list(at) for _ in range(2)]
        up[i], down[i] = at[i] + eps * v, at[i] - eps * v
        want = (loss(*up) - loss(*down)) / (2 * eps)
        # independent errors of the terms: their root of squares, six times over
        bound = 6 * 4 * 2.0 ** -8 * ((total * v.abs()) ** 2).sum().sqrt()
        assert abs(float((grad.double() * v).sum() - want)) <= float(bound)


def test_on_another_stream_and_replayed():
    """A captured forward and backward give an eager call's bits when replayed on new inputs."""
    g = torch.Generator(device="cuda").manual_seed(8)
    for M in (3, 300):
        N, K = 200, 264
        x, W, dy = _rand(g, M, K), _rand(g, N, K, scale=K ** -0.5), _rand(g, M, N)
        y, pre, dx = torch.empty_like(dy), torch.empty_like(dy), torch.empty_like(x)
        dW, db = torch.empty(N, K, device="cuda"), torch.empty(N, device="cuda")
        ws = torch.empty(tw.twell_linear_bwd_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")
        st = _status()

        def step(stream=None):
            tw.twell_linear_fwd(x, W, False, None, tw.ACT_SILU, None, pre, y, st, stream=stream)
            tw.twell_linear_bwd(dy, x, W, False, tw.ACT_SILU, pre, dx, dW, False, db, ws, st, stream=stream)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        x.copy_(torch.randn(M, K, device="cuda", generator=g))
        dy.copy_(torch.randn(M, N, device="cuda", generator=g))
        for t in (y, pre, dx, dW, db):
            t.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in (y, pre, dx, dW, db)]
        for t in (y, pre, dx, dW, db):
            t.fill_(6)
        step()
        assert tw.twell_check(st) == 0
        assert all(torch.equal(a, b) for a, b in zip(replayed, (y, pre, dx, dW, db)))


def test_an_earlier_error_leaves_the_outputs_alone():
    x, W = torch.randn(300, 64, device="cuda").to(BF), torch.randn(72, 64, device="cuda").to(BF)
    for M in (2, 300):
        y = torch.full((M, 72), 5.0, device="cuda", dtype=BF)
        st = torch.full((1,), 4, dtype=torch.int32, device="cuda")
        tw.twell_linear_fwd(x[:M], W, False, None, tw.ACT_NONE, None, None, y, st)
        assert tw.twell_check(st) == 4 and bool((y == 5).all())
