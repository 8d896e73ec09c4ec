"""twell_grad_clip against 64-bit norms.

Tolerances. The norm's squares are summed in at least 32 bits per thread over at
most a few hundred elements and in 64 bits beyond, so it is within 2e-5 of the
exact norm, whatever the sizes (bound: 256 u / 2 plus its own rounding). A scaled
element carries the factor's error and two roundings: 2e-5 + 2 u relative, and
half a unit in the last place (up to 2^-8) more in bf16.
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


def _grads(sizes, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, device="cuda", generator=g) * scale).to(BF if i % 2 else F32) for i, n in enumerate(sizes)]


def _norm(ts):
    return math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in ts))


def _clip(ts, max_norm, outs=None, stream=None):
    norm = torch.full((1,), -1.0, device="cuda")
    ws = torch.empty(tw.twell_grad_clip_workspace_bytes(), dtype=torch.uint8, device="cuda")
    tw.twell_grad_clip(tw.TwellTensorList(ts, outs), max_norm, norm, ws, stream=stream)
    return norm


def _check(before, after, norm, max_norm):
    ref = _norm(before)
    assert abs(float(norm) - ref) <= 2e-5 * ref
    c = min(1.0, max_norm / ref) if ref > 0 else 1.0
    for b, a in zip(before, after):
        want = b.double() * c
        assert bool(((a.double() - want).abs() <= want.abs() * (2e-5 + (2.0 ** -8 if b.dtype is BF else 2.0 ** -23))
                     + 1e-38).all())


SIZES = [[1], [7], [4096], [8191, 8192, 8193], [1, 2, 3, 5, 100003], [0, 17, 0, 1000, 0], [65536 * 3 + 1, 33],
         [2_000_003, 1_000_001, 5], [1 + (i * 37) % 501 for i in range(700)], [4_194_304, 4096, 4_194_304]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("ratio", [0.1, 0.999, 1.5])
@pytest.mark.parametrize("in_place", [True, False])
def test_norm_and_scaled_tensors(sizes, ratio, in_place):
    ts = _grads(sizes)
    before = [t.clone() for t in ts]
    bound = ratio * _norm(ts)
    outs = None if in_place else [torch.full_like(t, 5.0) for t in ts]
    norm = _clip(ts, bound, outs)
    _check(before, ts if in_place else outs, norm, bound)
    if not in_place:
        assert all(torch.equal(a, b) for a, b in zip(ts, before))
    if ratio > 1:  # under the bound: every bit stays
        assert all(torch.equal(a, b) for a, b in zip(ts if in_place else outs, before))


def test_slices_at_any_offset():
    """Slices of flat buffers that start anywhere, beside elements that are not theirs."""
    for dtype in (BF, F32):
        base = torch.randn(300_000, device="cuda").to(dtype)
        out = torch.full_like(base, 9.0)
        cuts = [1, 2, 6, 13, 4109, 12302, 12303, 100_002, 250_001]
        ts = [base[a:b - 1] for a, b in zip(cuts, cuts[1:])]
        for shift in (0, 1, 3):
            out.fill_(9.0)
            outs = [out[a + shift:b - 1 + shift] for a, b in zip(cuts, cuts[1:])]
            norm = _clip(ts, 1.0, outs)
            _check(ts, outs, norm, 1.0)
            used = torch.zeros(300_000, dtype=torch.bool, device="cuda")
            for a, b in zip(cuts, cuts[1:]):
                used[a + shift:b - 1 + shift] = True
            assert bool((out[~used] == 9.0).all())


def test_no_tensors_and_only_empty_ones():
    assert float(_clip([], 1.0)) == 0.0
    assert float(_clip([torch.empty(0, device="cuda"), torch.empty(0, device="cuda", dtype=BF)], 1.0)) == 0.0


def test_zero_gradients_and_bounds():
    z = torch.zeros(1000, device="cuda")
    assert float(_clip([z], 1.0)) == 0.0 and not z.any()
    g = torch.randn(1000, device="cuda")
    assert float(_clip([g], 0.0)) > 0 and not g.any()
    g = torch.randn(1000, device="cuda")
    before = g.clone()
    norm = _clip([g], float("inf"))
    assert torch.equal(g, before) and abs(float(norm) - _norm([g])) <= 2e-5 * _norm([g])


@pytest.mark.parametrize("scale", [1e-30, 1e-25, 1e15, 1e25, 1e30])
def test_squares_outside_the_range_of_32_bits(scale):
    """Elements whose squares under- or overflow fp32 still have a norm."""
    g = torch.randn(50_001, device="cuda") * scale
    before = g.clone()
    bound = 0.5 * _norm([g])
    norm = _clip([g], bound)
    _check([before], [g], norm, bound)


def test_one_huge_element_among_small_ones():
    g = torch.full((100_000,), 1e-3, device="cuda")
    g[77_777] = 3e30
    before = g.clone()
    norm = _clip([g], 1.0)
    assert abs(float(norm) / 3e30 - 1) < 1e-6
    assert abs(float(g[77_777]) - 1.0) < 1e-5 and float(g[0]) == float(before[0] * (1.0 / norm[0]))


def test_infinities_and_nan():
    g = torch.randn(10_000, device="cuda")
    g[5_000] = float("inf")
    h = torch.randn(300, device="cuda").to(BF)
    norm = _clip([g, h], 1.0)
    assert math.isinf(float(norm)) and bool(g[5_000].isnan()) and not g[:5_000].any() and not h.any()
    g = torch.randn(10_000, device="cuda")
    g[3] = float("nan")
    norm = _clip([g, h], 1.0)
    assert math.isnan(float(norm)) and bool(g.isnan().all()) and bool(h.isnan().all())


def test_same_bits_every_time_and_on_another_stream():
    ts = _grads([1_000_003, 5, 77_777])
    ref = None
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        outs = [torch.empty_like(t) for t in ts]
        torch.cuda.synchronize()
        norm = _clip(ts, 0.3, outs, stream=stream)
        stream.synchronize()
        torch.cuda.synchronize()
        got = [norm] + outs
        if ref is None:
            ref = got
        assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_tensor_past_32_bit_offsets():
    n = 2 ** 31 + 12_345
    if torch.cuda.mem_get_info()[0] < 20e9:
        pytest.skip("needs 20 GB")
    g = torch.zeros(n, device="cuda", dtype=BF)
    g[-3:] = 3.0
    g[0] = 3.0
    norm = _clip([g], 3.0)
    assert abs(float(norm) - 6.0) < 1e-5
    assert [float(v) for v in g[-4:]] == [0.0, 1.5, 1.5, 1.5] and float(g[0]) == 1.5


def test_wrong_arguments_are_refused():
    g, norm = torch.randn(64, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(tw.twell_grad_clip_workspace_bytes(), dtype=torch.uint8, device="cuda")
    for make in (lambda: tw.TwellTensorList([g.cpu()]), lambda: tw.TwellTensorList([g.half()]),
                 lambda: tw.TwellTensorList([g.view(8, 8).t()]), lambda: tw.TwellTensorList([g], [g.to(BF)]),
                 lambda: tw.TwellTensorList([g], [g[:5]]), lambda: tw.TwellTensorList([g], [])):
        with pytest.raises(ValueError):
            make()
    lst = tw.TwellTensorList([g])
    for bad in (-1.0, float("nan")):
        with pytest.raises(tw.TwellError) as e:
            tw.twell_grad_clip(lst, bad, norm, ws)
        assert e.value.status == 1
    with pytest.raises(tw.TwellError) as e:
        tw.twell_grad_clip(lst, 1.0, norm, ws[:256])
    assert e.value.status == 3
    many = tw.TwellTensorList([g[:1]] * 32769)
    with pytest.raises(tw.TwellError) as e:
        tw.twell_grad_clip(many, 1.0, norm, ws)
    assert e.value.status == 2
