"""The gradients' tests by differences can tell: on the CPU, with gradients as the layers round them, and with wrong ones."""
import pytest
import torch

from dense_differences import Gated, Linear, difference, directions

ACTS = ("silu", "gelu", "gelu_tanh")


def _off(case, i, grad, v):
    """Difference along v in units of the bound."""
    return abs(float((grad * v).sum() - difference(case.loss, case.at, i, v))) / float(case.bound(i, v))


def _bf(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).bfloat16()


def _linear(act, seed):
    gen = torch.Generator().manual_seed(seed)
    M, N, K = 60, 72, 64
    return gen, Linear(_bf(gen, M, K), _bf(gen, N, K, scale=K ** -0.5), torch.randn(N, generator=gen), _bf(gen, M, N), act)


def _gated(act, seed):
    gen = torch.Generator().manual_seed(seed)
    M, d, F = 50, 64, 72
    return gen, Gated(_bf(gen, M, d), _bf(gen, F, d, scale=d ** -0.5), _bf(gen, F, d, scale=d ** -0.5), _bf(gen, F, d, scale=F ** -0.5),
                      0.3 * torch.randn(F, generator=gen), _bf(gen, M, d), act, 0.3)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("make", [_linear, _gated])
def test_rounded_gradients_pass_and_wrong_ones_do_not(make, act):
    for seed in range(3):
        gen, case = make(act, seed)
        right, rounded = case.gradients(), case.rounded()
        wrong = [case.gradients(slope=False)]
        if make is _gated:
            wrong += [case.gradients(l1=0.0), case.gradients(of_dy=0.0)]
        for i, name in enumerate(case.names):
            along = [right[i], *(w[i] - right[i] for w in wrong)]
            vs = directions(along, gen)
            assert max(_off(case, i, right[i], v) for v in vs) < 0.01, name
            assert max(_off(case, i, rounded[i], v) for v in vs) <= 1, name
            for bad in (torch.zeros_like(right[i]), 2 * right[i], -right[i], 1.25 * right[i],
                        *(w[i] for w in wrong if float((w[i] - right[i]).norm()) > 1e-9)):
                assert max(_off(case, i, bad, v) for v in vs) > 2, name
