"""twell_adamw's random bits: a function of (seed, step, place in the list, element) alone. Codes and bf16 parameters to the bit
as splitmix64 and the rounding that twell.h describes give them, for lists that take several launches, at every alignment,
and with the other tensors of the list exchanged."""
import pytest
import torch

from test_gpu_adamw import Problem

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
B1, B2 = 0.9, 0.99
MASK = (1 << 64) - 1
GAMMA = 0x9E3779B97F4A7C15


def _signed(k):
    k &= MASK
    return k - (1 << 64) if k >> 63 else k


def _mix_int(z):
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & MASK
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & MASK
    return z ^ (z >> 31)


def _mix(z):
    """The same of an int64 tensor (which wraps around)."""
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * _signed(0xBF58476D1CE4E5B9)
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * _signed(0x94D049BB133111EB)
    return z ^ ((z >> 31) & ((1 << 33) - 1))


def _bits(seed, step, place, n, stream):
    """stream 0: 32 bits an element, m's 16 low, v's high; 1: 16 bits of a bf16 parameter."""
    base = _mix_int((seed + step * GAMMA) & MASK)
    key = _mix_int((base + (2 * place + 1 + stream) * GAMMA) & MASK)
    e, per = torch.arange(n, device="cuda"), 4 if stream else 2
    word = _mix((e // per + 1) * _signed(GAMMA) + _signed(key))
    return (word >> (e % per * (64 // per))) & ((1 << (64 // per)) - 1)


def _codes(x, random, E):
    """(codes, scales) of fp32 values x."""
    n = x.numel()
    blocks = torch.nn.functional.pad(x, (0, -n % tw.ADAMW_BLOCK)).view(-1, tw.ADAMW_BLOCK)
    frac, power = torch.frexp(blocks.abs().amax(1).double())
    power = power + (frac > 15 / 16).int()
    scale = torch.where(frac > 0, torch.ldexp(torch.ones_like(frac), power), 0.0)
    # as an fp32 number whose exponent and first three bits of fraction are the code (2^(2^E - 127) for a whole scale)
    small = torch.where(scale > 0, blocks.abs().double().T / scale * 2.0 ** (2 ** E - 127), 0.0).T.float()
    code = (small.contiguous().view(torch.int32).view(-1)[:n].long() + random * 16) >> 20
    if E == 5:
        code = torch.where((code == 0) & (x > 0), 1, code)
    else:
        code = code | torch.where(torch.signbit(x), 128, 0)
    return code.to(torch.uint8), scale.float()


def _values(code, scale, E):
    size = (code & 127 if E == 4 else code).to(torch.int32) << 20
    x = size.view(F32) * 2.0 ** (127 - 2 ** E) * scale.repeat_interleave(tw.ADAMW_BLOCK)[:code.numel()]
    return torch.where(code > 127, -x, x) if E == 4 else x


MANY = [1 + (i * 37) % 901 for i in range(1100)]


@pytest.mark.parametrize("sizes", [[70_001, 255], MANY], ids=["two", "many"])
@pytest.mark.parametrize("p_type,g_type", [(F32, F32), (BF, BF)], ids=["f32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1])
def test_codes_to_the_bit(sizes, p_type, g_type, shift):
    pr = Problem(sizes, p_type, g_type, bits=8, shift=shift, seed=4)
    pr.step.fill_(12)
    c = torch.where(pr.norm > 0.01, 0.01 / pr.norm, 1.0)
    want = []
    for i, (g, m, v, ms, vs) in enumerate(zip(pr.g, pr.m, pr.v, pr.ms, pr.vs)):
        gs = g.float() * c
        new_m = B1 * _values(m, ms, 4) + (1 - B1) * gs
        new_v = B2 * _values(v, vs, 5) + (1 - B2) * (gs * gs)
        r = _bits(77, 12, i, g.numel(), 0)
        want.append((*_codes(new_m, r & 0xffff, 4), *_codes(new_v, r >> 16, 5)))
    pr.run(0.01, seed=77)
    for i, (m, ms, v, vs) in enumerate(want):
        assert torch.equal(pr.ms[i], ms) and torch.equal(pr.vs[i], vs), i
        assert torch.equal(pr.m[i], m) and torch.equal(pr.v[i], v), i


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[70_001, 255], MANY], ids=["two", "many"])
@pytest.mark.parametrize("shift", [0, 1])
def test_bf16_parameters_to_the_bit(bits, sizes, shift):
    """No gradient, no moments, beta1 = 0: a step of lr weight_decay p = 2^-12 p, exact in fp32."""
    pr = Problem(sizes, BF, BF, bits, shift=shift, seed=5, first=True)
    for g in pr.g:
        g.zero_()
    pr.lr.fill_(2.0 ** -9)
    pr.step.fill_(3)
    want = []
    for i, p in enumerate(pr.p):
        x = (p.double() * (1 - 2.0 ** -12)).float()
        raised = x.view(torch.int32).long() + _bits(78, 3, i, p.numel(), 1)
        want.append((raised >> 16 << 16).to(torch.int32).view(F32).to(BF))
    tw.twell_adamw(pr.list, pr.lr, pr.step, 0.0, B2, 1e-8, 2.0 ** -3, None, 1.0, 78)
    moved = 0
    for i, p in enumerate(want):
        assert torch.equal(pr.p[i], p), i
        moved += p.numel()
    assert moved == sum(sizes)


@pytest.mark.parametrize("bits", [32, 8])
def test_other_tensors_of_the_list_change_nothing(bits):
    """A tensor at its place with the others there and with the others empty, which leaves it in the first launch."""
    for place in (0, 3, 450, 550, 1050):
        alone = [n if i == place else 0 for i, n in enumerate(MANY)]
        a, b = Problem(MANY, BF, F32, bits, seed=6), Problem(alone, BF, F32, bits, seed=6)
        for key in ("p", "g", "m", "v") + (("ms", "vs") if bits == 8 else ()):
            getattr(b, key)[place].copy_(getattr(a, key)[place])
        b.norm.copy_(a.norm)
        for pr in (a, b):
            pr.run(0.1 * float(a.norm))
        for key in ("p", "m", "v") + (("ms", "vs") if bits == 8 else ()):
            assert torch.equal(getattr(a, key)[place], getattr(b, key)[place]), (place, key)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_type", [F32, BF], ids=["f32", "bf16"])
def test_alignment_changes_nothing(bits, p_type):
    runs = []
    for shift in (0, 1, 2, 4):
        pr = Problem([5000, 255, 70_000], p_type, F32, bits, copy=p_type is F32, shift=shift, seed=8)
        pr.run(0.1 * float(pr.norm))
        runs.append(pr)
    for pr in runs[1:]:
        for key in ("p", "m", "v") + (("ms", "vs") if bits == 8 else ()) + (("copy",) if p_type is F32 else ()):
            assert all(torch.equal(x, y) for x, y in zip(getattr(pr, key), getattr(runs[0], key))), (pr.shift, key)
