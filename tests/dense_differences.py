"""Directional derivatives of the linear and gated layers' losses by central differences in 64 bits, and how far a gradient that
was formed from rounded intermediates may be off along a direction.

Every rounding is a source of its own: an intermediate z that is kept or multiplied in bf16 is off by at most 2^-8 |z|, and a
change of z by dz changes <gradient, v> by c dz with a coefficient c that the formulas give. Independent errors within b_i have
a sum that passes 6 (sum b_i^2)^(1/2) with a probability of 2 exp(-18) at most (Hoeffding). The products' own errors, (depth / 16
+ 8) 2^-23 of their terms' magnitudes, are added up. Everything in 64 bits on the inputs' device.
"""
import torch

from dense_reference import act64

STEP = 2.0 ** -8


def _curvature(z, act):
    """act''(z)."""
    z = z.detach().clone().requires_grad_()
    da = act64(z, act)[1]
    return torch.autograd.grad(da.sum(), z)[0] if da.requires_grad else torch.zeros_like(z)


def difference(loss, at, i, v, eps=1e-6):
    """d/dt loss(at with at[i] + t v) at 0."""
    up, down = list(at), list(at)
    up[i], down[i] = at[i] + eps * v, at[i] - eps * v
    return (loss(*up) - loss(*down)) / (2 * eps)


def directions(gradients, gen, random=2):
    """Unit vectors along the given gradients, and a few random ones."""
    g = gradients[0]
    vs = [*gradients, *(torch.randn(g.shape, generator=gen, dtype=torch.float64).to(g.device) for _ in range(random))]
    return [v / v.norm() for v in vs if float(v.norm()) > 0]


class Linear:
    """L = <dy, act(x W^T + b)>; gradients in the order x, W, b."""
    names = ("dx", "dW", "dbias")

    def __init__(self, x, W, b, dy, act):
        self.at, self.dy, self.act = [x.double(), W.double(), b.double()], dy.double(), act

    def loss(self, x, W, b):
        return (self.dy * act64(x @ W.T + b, self.act)[0]).sum()

    def gradients(self, slope=True):
        """The formulas; slope False: act' left out."""
        x, W, b = self.at
        d = self.dy * (act64(x @ W.T + b, self.act)[1] if slope else 1.0)
        return [d @ W, d.T @ x, d.sum(0)]

    def rounded(self):
        """As the layer forms them, with its roundings (dW and dbias in 32 bits: not rounded here)."""
        x, W, b = self.at
        pre = (x @ W.T + b).bfloat16().double()
        d = self.dy * act64(pre, self.act)[1]
        op = d.bfloat16().double()
        return [(op @ W).bfloat16().double(), op.T @ x, d.sum(0)]

    def bound(self, i, v):
        x, W, b = self.at
        z = x @ W.T + b
        d = self.dy * act64(z, self.act)[1]
        c = v @ W.T if i == 0 else x @ v.T if i == 1 else v.expand_as(z)  # of a change of dpre
        sources = [c * self.dy * _curvature(z, self.act) * z]
        if i < 2:
            sources.append(c * d)
        if i == 0:
            sources.append(v * (d @ W))
        depth = (W.shape[0], x.shape[0], x.shape[0])[i]
        size = d.abs() @ W.abs() if i == 0 else d.abs().T @ x.abs() if i == 1 else d.abs()
        terms = (size * v.abs()).sum()
        return 6 * STEP * sum((s * s).sum() for s in sources).sqrt() + (depth / 16 + 8) * 2.0 ** -23 * terms


class Gated:
    """L = <dy, h W_down> + l1 sum |h|, h = act(x W_gate^T + b) * (x W_up^T); gradients in the order x, W_gate, W_up, W_down, b."""
    names = ("dx", "dW_gate", "dW_up", "dW_down", "db")

    def __init__(self, x, Wg, Wu, Wd, b, dy, act, l1):
        self.at, self.dy, self.act, self.l1 = [t.double() for t in (x, Wg, Wu, Wd, b)], dy.double(), act, l1

    def loss(self, x, Wg, Wu, Wd, b):
        h = act64(x @ Wg.T + b, self.act)[0] * (x @ Wu.T)
        return (self.dy * (h @ Wd)).sum() + self.l1 * h.abs().sum()

    def _hidden(self):
        x, Wg, Wu, Wd, b = self.at
        return x @ Wg.T + b, x @ Wu.T

    def _from(self, g, u, h, l1, slope=True, of_dy=1.0, op=lambda t: t):
        x, Wg, Wu, Wd, _ = self.at
        a, da = act64(g, self.act)
        dh = of_dy * (self.dy @ Wd.T) + l1 * torch.sign(a) * torch.sign(u)
        dg, du = dh * u * (da if slope else 1.0), dh * a
        return [op(dg) @ Wg + op(du) @ Wu, op(dg).T @ x, op(du).T @ x, of_dy * (h.T @ self.dy), dg.sum(0)]

    def gradients(self, l1=None, **kw):
        g, u = self._hidden()
        return self._from(g, u, act64(g, self.act)[0] * u, self.l1 if l1 is None else l1, **kw)

    def rounded(self):
        g, u = self._hidden()
        h = (act64(g, self.act)[0] * u).bfloat16().double()
        bf = lambda t: t.bfloat16().double()  # noqa: E731
        grads = self._from(bf(g), bf(u), h, self.l1, op=bf)
        return [bf(grads[0]), *grads[1:]]

    def bound(self, i, v):
        x, Wg, Wu, Wd, _ = self.at
        g, u = self._hidden()
        a, da = act64(g, self.act)
        dh = self.dy @ Wd.T + self.l1 * torch.sign(a) * torch.sign(u)
        dg, du, h = dh * u * da, dh * a, a * u
        zero = torch.zeros_like(g)
        # of a change of dg, of du, of h
        cg = v @ Wg.T if i == 0 else x @ v.T if i == 1 else v.expand_as(g) if i == 4 else zero
        cu = v @ Wu.T if i == 0 else x @ v.T if i == 2 else zero
        ch = self.dy @ v.T if i == 3 else zero
        sources = [(cg * dh * u * _curvature(g, self.act) + cu * dh * da) * g, cg * dh * da * u, ch * h]
        if i < 3:
            sources += [cg * dg, cu * du]
        if i == 0:
            sources.append(v * (dg @ Wg + du @ Wu))
        M, d, F = x.shape[0], x.shape[1], g.shape[1]
        if i == 0:
            size = dg.abs() @ Wg.abs() + du.abs() @ Wu.abs()
        elif i == 4:
            size = dg.abs()
        else:
            size = (dg, du, h)[i - 1].abs().T @ (self.dy if i == 3 else x).abs()
        terms = (size * v.abs()).sum()
        return 6 * STEP * sum((s * s).sum() for s in sources).sqrt() + ((2 * F + M + d) / 16 + 16) * 2.0 ** -23 * terms
