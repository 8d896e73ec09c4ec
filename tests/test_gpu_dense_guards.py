"""The linear and gated layers and the optimiser's step beside other work: rows behind the last one stay as they were, calls
on two streams at once, and two captured graphs that take turns."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def _bf(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(BF)


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _more(M, N, t=BF, rows=300):
    """The first M rows of a matrix that has more of them, all 7."""
    big = torch.full((M + rows, N), 7.0, device="cuda", dtype=t)
    return big, big[:M]


@pytest.mark.parametrize("M", [1, 15, 33, 65, 127, 130, 257, 300])
@pytest.mark.parametrize("N,K", [(40, 64), (51, 520), (520, 2048)])
def test_linear_writes_its_rows_alone(M, N, K):
    x, W, dy = _bf(M, K), _bf(N, K, seed=1, scale=K ** -0.5), _bf(M, N, seed=2)
    for t in (BF, F32):
        (ybig, y), (pbig, pre) = _more(M, N, t), _more(M, N)
        st = _status()
        tw.twell_linear_fwd(x, W, False, None, tw.ACT_SILU, None, pre, y, st)
        assert tw.twell_check(st) == 0
        assert bool((ybig[M:] == 7).all()) and bool((pbig[M:] == 7).all()) and not bool((y == 7).all())
    dbig, dx = _more(M, K)
    wbig, dW = _more(N, K, F32)
    bbig = torch.full((N + 64,), 7.0, device="cuda")
    need = tw.twell_linear_bwd_workspace_bytes(M, N, K)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    tw.twell_linear_bwd(dy, x, W, False, tw.ACT_SILU, pre, dx, dW, False, bbig[:N], ws[:need], st)
    assert tw.twell_check(st) == 0
    assert bool((dbig[M:] == 7).all()) and bool((wbig[N:] == 7).all()) and bool((bbig[N:] == 7).all()) and bool((ws[need:] == 77).all())


@pytest.mark.parametrize("M", [1, 15, 33, 65, 127, 130, 300])
@pytest.mark.parametrize("d,F", [(64, 40), (264, 520)])
def test_gated_layer_writes_its_rows_alone(M, d, F):
    x, Wg, Wu, Wd = _bf(M, d), _bf(F, d, seed=1), _bf(F, d, seed=2), _bf(F, d, seed=3)
    b = torch.zeros(F, device="cuda")
    bigs = [_more(M, F) for _ in range(3)] + [_more(M, d) for _ in range(2)]
    g, u, h, y, dx = (v for _, v in bigs)
    st = _status()
    tw.twell_dense_gated_ffn_fwd(x, Wg, Wu, b, Wd, tw.ACT_GELU, None, g, u, h, y, st)
    grads = [_more(F, d) for _ in range(3)]
    db = torch.full((F + 64,), 7.0, device="cuda")
    need = tw.twell_dense_gated_bwd_workspace_bytes(M, d, F)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    tw.twell_dense_gated_ffn_bwd(x, Wg, Wu, Wd, tw.ACT_GELU, g, u, h, _bf(M, d, seed=4), 0.01, dx, *(v for _, v in grads), False,
                                 db[:F], ws[:need], st)
    assert tw.twell_check(st) == 0
    assert all(bool((big[M:] == 7).all()) for big, _ in bigs) and all(bool((big[F:] == 7).all()) for big, _ in grads)
    assert bool((db[F:] == 7).all()) and bool((ws[need:] == 77).all())


class _Work:
    """One of each call, with buffers of its own."""

    def __init__(self, M, d, F, seed):
        self.M, self.d, self.F = M, d, F
        self.x, self.dy = _bf(M, d, seed=seed), _bf(M, d, seed=seed + 1)
        self.W = [_bf(F, d, seed=seed + 2 + i, scale=d ** -0.5) for i in range(3)]
        self.b = torch.zeros(F, device="cuda")
        self.mid = [torch.empty(M, F, device="cuda", dtype=BF) for _ in range(3)]
        self.y, self.dx, self.z = (torch.empty(M, d, device="cuda", dtype=BF) for _ in range(3))
        self.dW, self.db = [torch.empty(F, d, device="cuda") for _ in range(3)], torch.empty(F, device="cuda")
        self.ws = torch.empty(tw.twell_dense_gated_bwd_workspace_bytes(M, d, F), dtype=torch.uint8, device="cuda")
        self.st = _status()
        self.lr, self.step = torch.full((1,), 1e-3, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
        self.m, self.v = ([torch.zeros(F * d, dtype=torch.uint8, device="cuda") for _ in range(3)] for _ in range(2))
        n = -(-F * d // tw.ADAMW_BLOCK)
        scales = [[torch.zeros(n, device="cuda") for _ in range(3)] for _ in range(2)]
        self.p = [torch.ones(F, d, device="cuda") for _ in range(3)]
        self.list = tw.TwellAdamWList(self.p, self.dW, self.m, self.v, *scales)

    def run(self, stream=None):
        g, u, h = self.mid
        tw.twell_dense_gated_ffn_fwd(self.x, self.W[0], self.W[1], self.b, self.W[2], tw.ACT_SILU, None, g, u, h, self.y, self.st,
                                     stream=stream)
        tw.twell_linear_fwd(h, self.W[2], True, None, tw.ACT_NONE, self.y, None, self.z, self.st, stream=stream)
        tw.twell_dense_gated_ffn_bwd(self.x, *self.W, tw.ACT_SILU, g, u, h, self.dy, 0.01, self.dx, *self.dW, False, self.db, self.ws,
                                     self.st, stream=stream)
        tw.twell_adamw(self.list, self.lr, self.step, 0.9, 0.99, 1e-8, 0.1, None, 1.0, 5, stream=stream)

    def results(self):
        return [t.clone() for t in (*self.mid, self.y, self.z, self.dx, *self.dW, self.db, *self.p, *self.m, *self.v)]

    def reset(self):
        for t in (*self.m, *self.v, *self.list.m_scale, *self.list.v_scale):
            t.zero_()
        for t in self.p:
            t.fill_(1)


SHAPES = [(3, 264, 520), (64, 1024, 2048), (300, 520, 1032), (700, 264, 264)]


def test_two_streams_at_once():
    works = [_Work(*s, seed=20 * i) for i, s in enumerate(SHAPES)]
    want = []
    for w in works:
        w.run()
        torch.cuda.synchronize()
        want.append(w.results())
        w.reset()
    streams = [torch.cuda.Stream() for _ in works]
    torch.cuda.synchronize()
    for _ in range(5):
        for w in works:
            w.reset()
        torch.cuda.synchronize()
        for w, s in zip(works, streams):
            w.run(s)
        torch.cuda.synchronize()
        assert all(tw.twell_check(w.st) == 0 for w in works)
        for w, ref in zip(works, want):
            assert all(torch.equal(a, b) for a, b in zip(w.results(), ref))


def test_two_graphs_take_turns():
    works = [_Work(*s, seed=20 * i) for i, s in enumerate(SHAPES[:3])]
    want, graphs = [], []
    for w in works:
        w.run()
        torch.cuda.synchronize()
        want.append(w.results())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            w.run()
        graphs.append(graph)
    for _ in range(3):
        for w, graph in zip(works, graphs):
            w.reset()
            graph.replay()
        torch.cuda.synchronize()
        for w, ref in zip(works, want):
            assert all(torch.equal(a, b) for a, b in zip(w.results(), ref))
