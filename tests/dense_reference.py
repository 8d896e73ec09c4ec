"""What the tests of the linear and gated layers share: activations and their derivatives in 64 bits, and error bounds.

Bounds. A product of depth K on the tensor cores drops at each of its K / 16 steps at most 2^-23 of the sum of the
magnitudes, and the pieces that are added up afterwards round by half of that: `depth_error` takes (K / 16 + 8) 2^-23 of
the products' magnitudes. An activation's slope is at most 1.13, and its own evaluation (fast exponential and quotient,
erf) is within 1e-6 of |z|, its derivative's within 2e-6 (1 + |z|). A rounding to bf16 is off by 2^-8 of the value at
most, one to fp32 by 2^-24.
"""
import math

import torch

BF, F32 = torch.bfloat16, torch.float32
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
SLOPE = 1.13


def half_step(t):
    return torch.finfo(t).eps / 2


def act64(z, kind):
    """(act(z), act'(z)) in 64 bits."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp(min=0), (z > 0).double()
    if kind == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if kind == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(8 / math.pi)
    s = torch.sigmoid(k * (z + 0.044715 * z ** 3))
    return z * s, s + z * s * (1 - s) * k * (1 + 0.134145 * z ** 2)


def depth_error(K, magnitudes):
    return (K / 16 + 8) * 2.0 ** -23 * magnitudes


def assert_within(got, want, bound, what):
    got, bad = got.double(), None
    assert got.shape == want.shape, what
    off = (got - want).abs()
    bad = ~(off <= bound + 1e-30)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((off / (bound + 1e-30)).max()):.3g} "
                                 f"times its bound, first at {bad.nonzero()[0].tolist()}")
