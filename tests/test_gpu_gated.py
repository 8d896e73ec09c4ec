"""twell_dense_gated_ffn_fwd and _bwd against the formulas in 64 bits, with the bounds of dense_reference."""
import pytest
import torch

from dense_reference import ACTS, BF, F32, SLOPE, act64, assert_within, depth_error, half_step

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

CODE = {"none": tw.ACT_NONE, "relu": tw.ACT_RELU, "silu": tw.ACT_SILU, "gelu": tw.ACT_GELU, "gelu_tanh": tw.ACT_GELU_TANH}


def _bf(g, *shape, scale=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(BF)


class Layer:
    def __init__(self, M, d, F, act, bias=True, seed=0):
        g = self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.M, self.d, self.F, self.act = M, d, F, act
        self.x, self.Wg, self.Wu = _bf(g, M, d), _bf(g, F, d, scale=d ** -0.5), _bf(g, F, d, scale=d ** -0.5)
        self.Wd = _bf(g, F, d, scale=F ** -0.5)
        self.b = 0.3 * torch.randn(F, device="cuda", generator=g) if bias else None
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def forward(self, save=True, res=None, y=None, stream=None):
        M, d, F = self.M, self.d, self.F
        self.g, self.u = (torch.full((M, F), 9.0, device="cuda", dtype=BF) for _ in range(2)) if save else (None, None)
        self.h = torch.full((M, F), 9.0, device="cuda", dtype=BF)
        self.y = torch.full((M, d), 9.0, device="cuda", dtype=BF) if y is None else y
        tw.twell_dense_gated_ffn_fwd(self.x, self.Wg, self.Wu, self.b, self.Wd, CODE[self.act], res, self.g, self.u, self.h,
                                     self.y, self.st, stream=stream)
        assert tw.twell_check(self.st) == 0

    def check_forward(self, res=None):
        X, Wg, Wu = self.x.double(), self.Wg.double(), self.Wu.double()
        g, u = X @ Wg.T + (self.b.double() if self.b is not None else 0.0), X @ Wu.T
        tg = depth_error(self.d, X.abs() @ Wg.abs().T) + 2.0 ** -23 * g.abs()
        tu = depth_error(self.d, X.abs() @ Wu.abs().T)
        if self.g is not None:
            assert_within(self.g, g, tg + half_step(BF) * (g.abs() + tg), "g")
            assert_within(self.u, u, tu + half_step(BF) * (u.abs() + tu), "u")
        a = act64(g, self.act)[0]
        ta = SLOPE * tg + 1e-6 * g.abs()
        h = a * u
        th = ta * u.abs() + (a.abs() + ta) * tu + 2.0 ** -23 * h.abs()
        assert_within(self.h, h, th + half_step(BF) * (h.abs() + th), "h")
        # y is defined on h as stored
        H, Wd = self.h.double(), self.Wd.double()
        y = H @ Wd + (res.double() if res is not None else 0.0)
        ty = depth_error(self.F, H.abs() @ Wd.abs()) + 2.0 ** -23 * y.abs()
        assert_within(self.y, y, ty + half_step(BF) * (y.abs() + ty), "y")

    def backward(self, dy, l1, dw_type=BF, accumulate=False, with_dx=True, with_dw=True, with_db=True, stream=None):
        M, d, F = self.M, self.d, self.F
        self.dx = torch.full((M, d), 9.0, device="cuda", dtype=BF) if with_dx else None
        self.before = [torch.randn(F, d, device="cuda", generator=self.gen).to(dw_type) for _ in range(3)]
        self.dW = [t.clone() for t in self.before] if with_dw else [None] * 3
        self.db = torch.full((F,), 9.0, device="cuda") if with_db else None
        ws = torch.empty(tw.twell_dense_gated_bwd_workspace_bytes(M, d, F), dtype=torch.uint8, device="cuda").fill_(255)
        tw.twell_dense_gated_ffn_bwd(self.x, self.Wg, self.Wu, self.Wd, CODE[self.act], self.g, self.u, self.h, dy, l1, self.dx,
                                     *self.dW, accumulate, self.db, ws, self.st, stream=stream)
        assert tw.twell_check(self.st) == 0

    def check_backward(self, dy, l1, dw_type=BF, accumulate=False):
        """Against the gradients at the g, u and h that were kept."""
        X, Wg, Wu, Wd, D = (t.double() for t in (self.x, self.Wg, self.Wu, self.Wd, dy))
        g, u, H = self.g.double(), self.u.double(), self.h.double()
        a, da = act64(g, self.act)
        exact = self.act in ("none", "relu")
        ta, tda = (0.0, 0.0) if exact else (1e-6 * g.abs(), 2e-6 * (1 + g.abs()))
        dh = D @ Wd.T + l1 * torch.sign(a) * torch.sign(u)
        tdh = depth_error(self.d, D.abs() @ Wd.abs().T) + 2.0 ** -23 * dh.abs()
        dg, du = dh * u * da, dh * a
        tdg = (tdh * (da.abs() + tda) + dh.abs() * tda) * u.abs() + 2.0 ** -22 * dg.abs()
        tdu = tdh * (a.abs() + ta) + dh.abs() * ta + 2.0 ** -23 * du.abs()
        if self.db is not None:
            assert_within(self.db, dg.sum(0), (tdg + (self.M / 16 + 64) * 2.0 ** -24 * dg.abs()).sum(0), "db")
        rg, ru = tdg + half_step(BF) * (dg.abs() + tdg), tdu + half_step(BF) * (du.abs() + tdu)  # as operands
        if self.dx is not None:
            want = dg @ Wg + du @ Wu
            err = rg @ Wg.abs() + ru @ Wu.abs() + depth_error(2 * self.F, dg.abs() @ Wg.abs() + du.abs() @ Wu.abs())
            assert_within(self.dx, want, err + half_step(BF) * (want.abs() + err), "dx")
        for got, was, left, slip, right, what in zip(self.dW, self.before, (dg, du, H), (rg, ru, 0 * H), (X, X, D),
                                                     ("dW_gate", "dW_up", "dW_down")):
            if got is None:
                continue
            want = left.T @ right
            err = slip.T @ right.abs() + depth_error(self.M, left.abs().T @ right.abs())
            if accumulate:
                want = want + was.double()
                err = err + 2.0 ** -23 * want.abs()
            assert_within(got, want, err + half_step(dw_type) * (want.abs() + err), what)


SIZES = [(1, 8, 8), (1, 4096, 1000), (2, 64, 136), (9, 1000, 264), (16, 520, 2048), (33, 128, 5000), (64, 2048, 520), (65, 72, 200),
         (128, 256, 1032), (130, 1000, 72), (256, 264, 64), (300, 1024, 1320), (777, 1000, 2696)]


@pytest.mark.parametrize("M,d,F", SIZES)
@pytest.mark.parametrize("save", [False, True])
def test_forward(M, d, F, save):
    layer = Layer(M, d, F, "silu")
    res = _bf(layer.gen, M, d) if M % 2 else None
    layer.forward(save, res)
    layer.check_forward(res)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("d,F", [(8, 8), (264, 40), (520, 5000), (2056, 8200)])
def test_single_tokens(M, d, F):
    layer = Layer(M, d, F, "silu", M % 2 == 0)
    res = _bf(layer.gen, M, d)
    layer.forward(M != 3, res)
    layer.check_forward(res)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 150])
@pytest.mark.parametrize("bias", [False, True])
def test_activations(act, M, bias):
    layer = Layer(M, 136, 264, act, bias)
    layer.forward(True)
    layer.check_forward()
    dy = _bf(layer.gen, M, 136)
    layer.backward(dy, 0.05)
    layer.check_backward(dy, 0.05)


@pytest.mark.parametrize("M,d,F", [(1, 64, 136), (63, 8, 8), (129, 264, 1000), (300, 1032, 520), (777, 136, 2696), (1500, 2056, 264)])
@pytest.mark.parametrize("dw_type", [BF, F32], ids=["bf16", "f32"])
def test_backward(M, d, F, dw_type):
    layer = Layer(M, d, F, "gelu_tanh")
    layer.forward(True)
    dy = _bf(layer.gen, M, d)
    layer.backward(dy, 0.0, dw_type)
    layer.check_backward(dy, 0.0, dw_type)


@pytest.mark.parametrize("M,d,F", [(260, 2048, 2056), (777, 2048, 2816), (2100, 1000, 2696), (4100, 1544, 1032)])
@pytest.mark.parametrize("dw_type,accumulate", [(BF, False), (F32, True)], ids=["bf16", "f32_added"])
def test_backward_of_all_products_in_one_launch(M, d, F, dw_type, accumulate):
    layer = Layer(M, d, F, "silu")
    layer.forward(True)
    dy = _bf(layer.gen, M, d)
    layer.backward(dy, 0.01, dw_type, accumulate=accumulate)
    layer.check_backward(dy, 0.01, dw_type, accumulate=accumulate)


def test_backward_adds_to_gradients():
    layer = Layer(200, 136, 264, "relu")
    layer.forward(True)
    dy = _bf(layer.gen, 200, 136)
    layer.backward(dy, 0.01, F32, accumulate=True)
    layer.check_backward(dy, 0.01, F32, accumulate=True)


@pytest.mark.parametrize("which", [(True, False, False), (False, True, False), (False, False, True)])
def test_backward_of_some(which):
    layer = Layer(100, 72, 136, "silu")
    layer.forward(True)
    dy = _bf(layer.gen, 100, 72)
    layer.backward(dy, 0.01, BF, False, *which)
    layer.check_backward(dy, 0.01)


@pytest.mark.parametrize("M", [3, 64, 200])
def test_residual_in_place(M):
    layer = Layer(M, 264, 136, "silu")
    res = _bf(layer.gen, M, 264)
    layer.forward(False, res)
    want = layer.y
    layer.forward(False, res, y=res)
    assert torch.equal(res, want)


def test_closed_gates_and_zero_rows():
    """A ReLU gate that nothing passes, rows of zeros: y is the residual, all gradients but those of l1 = 0 are 0."""
    for M in (4, 150):
        layer = Layer(M, 64, 136, "relu")
        layer.b.fill_(-1e4)
        res = _bf(layer.gen, M, 64)
        layer.forward(True, res)
        assert not bool(layer.h.any()) and torch.equal(layer.y, res)
        dy = _bf(layer.gen, M, 64)
        layer.backward(dy, 0.1, F32)
        assert not bool(layer.dx.any()) and not bool(layer.db.any()) and not any(bool(t.any()) for t in layer.dW)
        layer = Layer(M, 64, 136, "silu", bias=False)
        layer.x.zero_()
        layer.forward(True)
        assert not bool(layer.h.any()) and not bool(layer.y.any())


def test_no_rows():
    layer = Layer(0, 16, 24, "silu")
    layer.forward(True)
    dy = torch.empty(0, 16, device="cuda", dtype=BF)
    layer.backward(dy, 0.1, F32, accumulate=True)
    assert all(torch.equal(a, b) for a, b in zip(layer.dW, layer.before)) and not bool(layer.db.any())
    layer.backward(dy, 0.1, F32)
    assert not any(bool(t.any()) for t in layer.dW)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_against_differences(act):
    """<gradient, direction> against central differences of L = <dy, y> + l1 sum |h| in 64 bits. What is kept and what
    enters the products is rounded to bf16: 8 x 2^-8 of the terms' magnitudes for each term (g, u, h, the two products,
    the curvature), independent of one another: their root of squares, six times over."""
    M, d, F, l1 = 50, 64, 72, 0.02
    layer = Layer(M, d, F, act)
    layer.forward(True)
    dy = _bf(layer.gen, M, d)
    layer.backward(dy, l1, F32)

    def loss(x, Wg, Wu, Wd, b):
        h = act64(x @ Wg.T + b, act)[0] * (x @ Wu.T)
        return (dy.double() * (h @ Wd)).sum() + l1 * h.abs().sum()

    at = [t.double() for t in (layer.x, layer.Wg, layer.Wu, layer.Wd, layer.b)]
    X, Wg, Wu, Wd, b = at
    g, u = X @ Wg.T + b, X @ Wu.T
    dh = dy.double().abs() @ Wd.abs().T + l1
    mg, mu = dh * u.abs() * (1 + g.abs()), dh * (1 + g.abs())
    sizes = [mg @ Wg.abs() + mu @ Wu.abs(), mg.T @ X.abs(), mu.T @ X.abs(), (g.abs() * u.abs()).T @ dy.double().abs(), mg.sum(0)]
    for i, (grad, total) in enumerate(zip((layer.dx, *layer.dW, layer.db), sizes)):
        v = torch.randn(at[i].shape, device="cuda", generator=layer.gen, dtype=torch.float64)
        # no step passes a kink of |h|: those would be at g = 0 or u = 0, further away than the step for all but few
        eps = 1e-7
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + eps * v, at[i] - eps * v
        want = (loss(*up) - loss(*down)) / (2 * eps)
        assert abs(float((grad.double() * v).sum() - want)) <= float(6 * 8 * 2.0 ** -8 * ((total * v.abs()) ** 2).sum().sqrt())


def test_relu_gate_agrees_with_the_sparse_forward():
    """The weights that this layer trains are what the packed layer serves: h and y of both within a bf16 rounding."""
    M, d, F, T = 40, 256, 512, 8
    layer = Layer(M, d, F, "relu")
    layer.b.sub_(1.5)
    layer.forward(False)
    buf = tw.TwellBuffers(M, F, T, M * F)
    y = torch.empty(M, d, dtype=torch.int16, device="cuda")
    ws = torch.empty(tw.twell_workspace_bytes(tw.OP_GATED_FWD, M, d, F, T, M * F), dtype=torch.uint8, device="cuda")
    tw.twell_ffn_fwd(layer.x, layer.Wu, layer.Wg, layer.b, layer.Wd, T, buf, y, ws, layer.st)
    assert tw.twell_check(layer.st) == 0
    H, Wd = layer.h.double(), layer.Wd.double()
    mag = H.abs() @ Wd.abs()
    bound = 2 * half_step(BF) * mag + depth_error(F, mag) + 2 * half_step(BF) * (H @ Wd).abs() + 1e-5
    assert_within(y.view(BF), layer.y.double(), bound, "y")


def test_replayed_from_a_graph_beside_an_eager_call():
    for M in (3, 200):
        layer = Layer(M, 136, 264, "silu")
        dy = _bf(layer.gen, M, 136)
        g, u, h = (torch.empty(M, 264, device="cuda", dtype=BF) for _ in range(3))
        y, dx = torch.empty(M, 136, device="cuda", dtype=BF), torch.empty(M, 136, device="cuda", dtype=BF)
        dW, db = [torch.empty(264, 136, device="cuda") for _ in range(3)], torch.empty(264, device="cuda")
        ws = torch.empty(tw.twell_dense_gated_bwd_workspace_bytes(M, 136, 264), dtype=torch.uint8, device="cuda")

        def step():
            tw.twell_dense_gated_ffn_fwd(layer.x, layer.Wg, layer.Wu, layer.b, layer.Wd, tw.ACT_SILU, None, g, u, h, y, layer.st)
            tw.twell_dense_gated_ffn_bwd(layer.x, layer.Wg, layer.Wu, layer.Wd, tw.ACT_SILU, g, u, h, dy, 0.01, dx, *dW, False,
                                         db, ws, layer.st)

        outs = (g, u, h, y, dx, *dW, db)
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        layer.x.copy_(torch.randn(M, 136, device="cuda", generator=layer.gen))
        for t in outs:
            t.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in outs]
        for t in outs:
            t.fill_(6)
        step()
        assert tw.twell_check(layer.st) == 0
        assert all(torch.equal(a, b) for a, b in zip(replayed, outs))
