"""twell_adamw and twell_adamw_values against the formulas.

Bounds. First moments and second moments are three rounded operations each: 4 x 2^-24 of the terms' magnitudes. A step's
quotient is within 2^-20 (fast root and quotient, bias corrections), and the parameter is rounded once more: 2^-24 of it,
2^-8 in bf16, where it is rounded up or down (a whole unit, 2^-7). 8-bit codes: the value is one of the two codes next to the
32-bit one (within 2^-22 of it), 1/8 of the value apart, or one step of the smallest ones.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
B1, B2, EPS, WD = 0.9, 0.99, 1e-8, 0.1


def _blocks(n):
    return -(-n // tw.ADAMW_BLOCK)


class Problem:
    def __init__(self, sizes, p_type=F32, g_type=F32, bits=32, copy=False, shift=0, seed=0, first=False):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def make(n, t, values):
            base = torch.full((n + shift + 5,), 3, device="cuda", dtype=t)
            out = base[shift:shift + n]
            out.copy_(values)
            return base, out

        self.bits, self.guards = bits, []

        def keep(n, t, values):
            base, out = make(n, t, values)
            self.guards.append((base, n))
            return out

        self.shift = shift
        spread = [torch.exp(2 * torch.randn(n, device="cuda", generator=g)) * 1e-3 for n in sizes]
        rand = lambda n: torch.randn(n, device="cuda", generator=g)  # noqa: E731
        self.p = [keep(n, p_type, 0.05 * rand(n)) for n in sizes]
        self.g = [keep(n, g_type, rand(n) * s) for n, s in zip(sizes, spread)]
        self.copy = [keep(n, BF, torch.zeros(n, device="cuda")) for n in sizes] if copy else None
        if bits == 32:
            self.m = [keep(n, F32, rand(n) * s * (0 if first else 0.3)) for n, s in zip(sizes, spread)]
            self.v = [keep(n, F32, s * s * (0 if first else 0.5)) for n, s in zip(sizes, spread)]
            self.ms = self.vs = None
        else:
            u8 = torch.uint8
            codes = lambda n: (torch.randint(0, 256, (n,), device="cuda", generator=g) * (0 if first else 1)).to(u8)  # noqa: E731
            self.m, self.v = ([keep(n, u8, codes(n)) for n in sizes] for _ in range(2))
            scale = lambda n, at: 2.0 ** torch.randint(at - 3, at + 3, (_blocks(n),), device="cuda", generator=g).float()  # noqa: E731
            self.ms = [scale(n, -9) * (0 if first else 1) for n in sizes]
            self.vs = [scale(n, -17) * (0 if first else 1) for n in sizes]
        self.lr = torch.full((1,), 1e-2, device="cuda")
        self.step = torch.ones(1, device="cuda", dtype=torch.int32)
        self.norm = torch.tensor([math.sqrt(sum(float((t.double() ** 2).sum()) for t in self.g))], device="cuda")
        self.list = tw.TwellAdamWList(self.p, self.g, self.m, self.v, self.ms, self.vs, self.copy)

    def values(self):
        """(m, v) in 64 bits."""
        if self.bits == 32:
            return [t.double() for t in self.m], [t.double() for t in self.v]
        return ([_decode(c, s, 4, True) for c, s in zip(self.m, self.ms)], [_decode(c, s, 5, False) for c, s in zip(self.v, self.vs)])

    def run(self, max_norm=float("inf"), norm=True, seed=7, stream=None, wd=WD):
        tw.twell_adamw(self.list, self.lr, self.step, B1, B2, EPS, wd, self.norm if norm else None, max_norm, seed, stream=stream)

    def guards_intact(self):
        return all(bool((b[:self.shift] == 3).all()) and bool((b[self.shift + n:] == 3).all()) for b, n in self.guards)


def _decode(code, scale, E, signed):
    c = code.long()
    size = c & 127 if signed else c
    e, f = size >> 3, (size & 7).double()
    power = torch.tensor([2.0 ** (max(k, 1) - 2 ** E) for k in range(2 ** E)], dtype=torch.float64, device=c.device)[e]
    x = torch.where(e > 0, 1 + f / 8, f / 8) * power  # (torch.ldexp goes through pow, which is off by a unit on the GPU)
    x = x * scale.double().repeat_interleave(tw.ADAMW_BLOCK)[:x.numel()]
    return torch.where(c > 127, -x, x) if signed else x


def _check(pr, max_norm, wd=WD, **kw):
    old = [t.double() for t in pr.p]
    om, ov = pr.values()
    grads = [t.double() for t in pr.g]
    t, lr = int(pr.step), float(pr.lr)
    pr.run(max_norm, wd=wd, **kw)
    torch.cuda.synchronize()
    norm = float(pr.norm)
    c = max_norm / norm if norm > max_norm else 1.0
    nm, nv = pr.values()
    for i, p0 in enumerate(old):
        g = grads[i] * c
        m, v = B1 * om[i] + (1 - B1) * g, B2 * ov[i] + (1 - B2) * g * g
        slip = 4 * 2.0 ** -24 * (B1 * om[i].abs() + (1 - B1) * g.abs())
        to = m / (1 - B1 ** t) / ((v / (1 - B2 ** t)).sqrt() + EPS)
        want = p0 - lr * (to + wd * p0)
        off = lr * (2.0 ** -20 * to.abs() + slip / (1 - B1 ** t) / ((v / (1 - B2 ** t)).sqrt() + EPS)) + 2.0 ** -22 * p0.abs()
        unit = 2.0 ** -7 if pr.p[i].dtype is BF else 2.0 ** -24
        assert bool(((pr.p[i].double() - want).abs() <= off + unit * (want.abs() + off) + 1e-37).all())
        if pr.copy is not None:
            assert torch.equal(pr.copy[i], pr.p[i].to(BF))
        if pr.bits == 32:
            assert bool(((nm[i] - m).abs() <= slip + 1e-37).all())
            assert bool(((nv[i] - v).abs() <= 6 * 2.0 ** -24 * v + 1e-37).all())
        else:
            for new, x, scale, E in ((nm[i], m, pr.ms[i], 4), (nv[i], v, pr.vs[i], 5)):
                s = scale.double().repeat_interleave(tw.ADAMW_BLOCK)[:x.numel()]
                top = torch.nn.functional.pad(x.abs(), (0, -x.numel() % tw.ADAMW_BLOCK)).view(-1, tw.ADAMW_BLOCK).amax(1)
                sc = scale.double()
                assert bool((torch.frexp(sc)[0].eq(0.5) | sc.eq(0)).all())       # powers of two
                assert bool((top <= sc * 15 / 16 * (1 + 2.0 ** -22)).all())      # the smallest that holds the block
                assert bool((top >= sc * 15 / 32 * (1 - 2.0 ** -22)).all())
                apart = torch.maximum(x.abs() / 8 * (1 + 2.0 ** -20), s * 2.0 ** (1 - 2 ** E - 3)) + slip
                assert bool(((new - x).abs() <= apart).all())
                if E == 5:
                    assert bool(((new > 0) | (x == 0)).all())
    assert pr.guards_intact()


SIZES = [[1], [255, 256, 257], [7, 2048, 2049, 1, 100003], [0, 17, 0, 4096], [1 + (i * 37) % 901 for i in range(600)],
         [1_000_001, 3, 2_000_000]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("types", [(F32, F32, True), (F32, BF, False), (BF, BF, False), (BF, F32, False)],
                         ids=["f32_f32_copy", "f32_bf16", "bf16_bf16", "bf16_f32"])
@pytest.mark.parametrize("bits", [32, 8])
def test_step(sizes, types, bits):
    pr = Problem(sizes, types[0], types[1], bits, types[2])
    pr.step.fill_(5)
    _check(pr, 0.3 * float(pr.norm))


@pytest.mark.parametrize("shift", [1, 2, 3, 4])
@pytest.mark.parametrize("bits", [32, 8])
def test_tensors_at_any_offset(shift, bits):
    for p_type, copy in ((F32, True), (BF, False)):
        _check(Problem([1000, 255, 5000], p_type, BF, bits, copy, shift=shift), float("inf"))


@pytest.mark.parametrize("bits", [32, 8])
def test_first_steps_from_nothing(bits):
    pr = Problem([3000, 40], bits=bits, first=True)
    for t in range(1, 4):
        pr.step.fill_(t)
        _check(pr, 1e9, wd=0.0)


@pytest.mark.parametrize("scale", [1e-13, 1e6, 1e12, 1e17])
@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_of_any_magnitude(scale, bits):
    """Scales of codes far from 1, where a factor of the conversion leaves fp32's range and takes two steps."""
    pr = Problem([3000, 255], bits=bits, first=True)
    for g in pr.g:
        g.mul_(scale)
    pr.norm.fill_(math.sqrt(sum(float((t.double() ** 2).sum()) for t in pr.g)))
    for t in (1, 2, 3):
        pr.step.fill_(t)
        _check(pr, 0.5 * float(pr.norm), wd=0.0)


@pytest.mark.parametrize("types", [(F32, F32), (BF, BF), (F32, BF)], ids=["f32", "bf16", "f32_bf16"])
def test_moments_are_single_rounded_operations(types):
    """With 32-bit states, m and v as torch's operations give them, to the bit (the 8-bit codes are formed of them)."""
    pr = Problem([70_000, 1001], *types)
    want = []
    c = torch.where(pr.norm > 0.01, 0.01 / pr.norm, 1.0)
    for g, m, v in zip(pr.g, pr.m, pr.v):
        gs = g.float() * c
        want.append((B1 * m + (1 - B1) * gs, B2 * v + (1 - B2) * (gs * gs)))
    pr.run(0.01)
    assert all(torch.equal(m, a) and torch.equal(v, b) for m, v, (a, b) in zip(pr.m, pr.v, want))


@pytest.mark.parametrize("bits", [32, 8])
def test_late_steps_without_a_norm(bits):
    pr = Problem([3000], bits=bits)
    pr.step.fill_(2_000_000_000)
    _check(pr, float("inf"), norm=False)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_norm_that_is_not_finite_changes_nothing(bad, bits):
    pr = Problem([3000, 7], bits=bits, copy=True)
    before = [t.clone() for t in pr.p + pr.m + pr.v + pr.copy]
    pr.norm.fill_(bad)
    pr.run(1.0)
    pr.norm.fill_(1.0)
    pr.step.fill_(0)
    pr.run(1.0)
    assert all(torch.equal(a, b) for a, b in zip(before, pr.p + pr.m + pr.v + pr.copy))


def test_zero_bound_and_zero_gradients():
    """c = 0, or no gradient: the moments decay, parameters without them only lose their decay."""
    pr = Problem([2000], first=True)
    p0 = pr.p[0].clone()
    pr.run(0.0)
    want = p0.double() - 1e-2 * WD * p0.double()
    assert not bool(pr.m[0].any()) and bool(((pr.p[0].double() - want).abs() <= 2.0 ** -23 * want.abs()).all())


def test_a_gradient_that_is_not_finite_stays_in_its_element_or_block():
    for bits in (32, 8):
        pr = Problem([2000], bits=bits)
        pr.g[0][700] = float("nan")
        pr.run(norm=False)
        m, _ = pr.values()
        bad = m[0].isnan()
        where = torch.zeros_like(bad)
        where[700 if bits == 32 else slice(512, 768)] = True
        assert torch.equal(bad, where)
        assert int(pr.p[0].isnan().sum()) == 1


@pytest.mark.parametrize("E", [4, 5])
def test_codes_keep_the_mean(E):
    """Many steps with other seeds from one state: the mean of the codes is the value. The codes around a value lie a gap
    apart, at most 1/8 of the value, or 2^(1 - 2^E) / 8 of the scale among the smallest ones (the new m can be near 0, where
    gradient and old m cancel). A choice between the two has a spread of half the gap at most, independently from seed to
    seed: the mean of n is within 6 spreads / sqrt(n), and 2^-16 of the gap for the random bits' number."""
    n, size = 400, 4096
    base = Problem([size], bits=8, seed=3)
    base.m[0].copy_(torch.randint(64, 128, (size,), device="cuda"))    # nothing near the smallest codes
    base.v[0].copy_(torch.randint(160, 256, (size,), device="cuda"))
    base.g[0].mul_(0.01)
    keep = [t.clone() for t in (base.p[0], base.m[0], base.v[0], base.ms[0], base.vs[0])]
    total = 0
    for seed in range(n):
        for t, k in zip((base.p[0], base.m[0], base.v[0], base.ms[0], base.vs[0]), keep):
            t.copy_(k)
        base.run(norm=False, seed=seed)
        total = total + base.values()[0 if E == 4 else 1][0]
    g = base.g[0].double()
    if E == 4:
        x = B1 * _decode(keep[1], keep[3], 4, True) + (1 - B1) * g
    else:
        x = B2 * _decode(keep[2], keep[4], 5, False) + (1 - B2) * g * g
    scale = (base.ms if E == 4 else base.vs)[0].double().repeat_interleave(tw.ADAMW_BLOCK)
    gap = torch.maximum(x.abs() / 8, scale * 2.0 ** (1 - 2 ** E) / 8)
    assert bool(((total / n - x).abs() <= (6 / 2 / math.sqrt(n) + 2.0 ** -16) * gap).all())


def test_bf16_parameters_follow_steps_below_their_resolution():
    """10000 parameters of 1, each step 2^-12 (a sixteenth of the unit below 1): on average they move all the same."""
    p = torch.ones(10_000, device="cuda", dtype=BF)
    g = torch.ones_like(p)
    m, v = torch.ones(10_000, device="cuda"), torch.ones(10_000, device="cuda")
    lr, step = torch.full((1,), 2.0 ** -12, device="cuda"), torch.full((1,), 1 << 20, dtype=torch.int32, device="cuda")
    lst = tw.TwellAdamWList([p], [g], [m], [v])
    for t in range(64):
        step += 1
        tw.twell_adamw(lst, lr, step, B1, B2, EPS, 0.0, None, 1.0, 11)
    moved = 1 - float(p.double().mean())
    # 64 steps of 2^-12; a step's spread is at most half a unit (2^-9), over 10000 elements and 64 steps: 6 sigma
    assert abs(moved - 64 * 2.0 ** -12) <= 6 * 2.0 ** -9 * math.sqrt(64 / 10_000) + 64 * 2.0 ** -30


def test_results_are_a_function_of_the_inputs():
    """Twice the same bits, on another stream, and with the list cut in other places but the seed's tensors the same."""
    for bits in (32, 8):
        sizes = [5000, 300, 70_000]
        a, b, c = (Problem(sizes, BF, F32, bits) for _ in range(3))
        a.run(1.0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        b.run(1.0, stream=side)
        side.synchronize()
        c.run(1.0, seed=8)
        assert all(torch.equal(x, y) for x, y in zip(a.p + a.m + a.v, b.p + b.m + b.v))
        assert not all(torch.equal(x, y) for x, y in zip(a.p, c.p))


def test_replayed_from_a_graph():
    """A captured step follows lr, step and norm on the device."""
    for bits in (32, 8):
        a, b = Problem([5000, 300], bits=bits, copy=True), Problem([5000, 300], bits=bits, copy=True)
        warm = Problem([5000, 300], bits=bits, copy=True)
        warm.run(1.0)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a.run(0.01)
        for t in range(1, 5):
            for pr in (a, b):
                pr.step.fill_(t)
                pr.lr.fill_(0.01 / t)
                pr.norm.fill_(0.002 * t * t)
            graph.replay()
            b.run(0.01)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.p + a.m + a.v + a.copy, b.p + b.m + b.v + b.copy))


@pytest.mark.parametrize("t", [BF, F32], ids=["bf16", "f32"])
def test_values(t):
    pr = Problem([1, 255, 256, 70_001], bits=8)
    out = [[torch.full((p.numel() + 3,), 9.0, device="cuda", dtype=t) for p in pr.p] for _ in range(2)]
    for shift in (0, 1):
        lists = [tw.TwellTensorList([o[shift:shift + p.numel()] for o, p in zip(k, pr.p)]) for k in out]
        tw.twell_adamw_values(pr.list, *lists)
        for got, want in zip(lists, pr.values()):
            assert all(torch.equal(a.double(), b) for a, b in zip(got.outs, want))
    assert all(bool((o[-2:] == 9).all()) for k in out for o in k)


def test_lists_are_checked():
    pr = Problem([10, 20])
    with pytest.raises(ValueError):
        tw.TwellAdamWList(pr.p, pr.g[:1], pr.m, pr.v)
    with pytest.raises(ValueError):
        tw.TwellAdamWList(pr.p, pr.g, pr.m, pr.v, pr.m, None)
    with pytest.raises(ValueError):
        tw.TwellAdamWList(pr.p, pr.g, [t.half() for t in pr.m], pr.v)
    with pytest.raises(ValueError):
        tw.TwellAdamWList(pr.p, pr.g[::-1], pr.m, pr.v)
    for p, g, m, v in ((pr.p[:1] * 2, pr.g[:1] * 2, pr.m[:1] * 2, pr.v[:1] * 2), (pr.p, pr.g, pr.m, [pr.v[0], pr.m[1]]),
                       (pr.p, [pr.g[0], pr.m[1]], pr.m, pr.v)):  # tied weights; a state as another; a state as a gradient
        with pytest.raises(ValueError):
            tw.TwellAdamWList(p, g, m, v)
    empty = tw.TwellAdamWList([], [], [], [])
    tw.twell_adamw(empty, pr.lr, pr.step, B1, B2, EPS, WD, None, 1.0, 0)
