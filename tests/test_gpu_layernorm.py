"""twell_layernorm_fwd / _bwd against the definitions in 64 bits.

Tolerances. A sum of n fp32 terms added by threads and then a tree is off by at
most k u times the sum of magnitudes, u = 2^-24, with k the longest chain: at
most d / 32 + 64 along a row, N + 64 down a column. That bounds the error of the
mean by k u mean|x| and, through it and the variance, the error of a normalised
value by E = 4 k u (max|x| rstd + 1)(1 + |hat|); outputs then follow from the
formulas, and a bf16 output (8 significant bits) may be off by half a unit in the
last place more (up to 2^-8 of itself).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def _rand(shape, dtype, seed, scale=1.0, offset=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * scale + offset).to(dtype)


def _out_tol(ref, dtype):
    # bf16: half a unit in the last place, up to 2^-8 relative
    return ref.abs() * (2.0 ** -8 if dtype is BF else 2 * U) + 1e-37


def _fwd_ref(x, res, w, b, eps):
    s = x if res is None else (x.double() + res.double()).to(x.dtype)
    v = s.double()
    mean = v.mean(1)
    rstd = 1.0 / torch.sqrt(((v - mean[:, None]) ** 2).mean(1) + eps)
    hat = (v - mean[:, None]) * rstd[:, None]
    wd = torch.ones(x.shape[1], dtype=torch.float64, device=x.device) if w is None else w.double()
    bd = torch.zeros_like(wd) if b is None else b.double()
    return s, mean, rstd, hat, hat * wd + bd, wd


def _hat_err(v, rstd, hat, d):
    k = d / 32 + 64
    return 4 * k * U * (v.abs().amax(1) * rstd + 1)[:, None] * (1 + hat.abs())


def _check_fwd(x, res, w, b, y_dtype, eps=1e-5, make=torch.empty):
    N, d = x.shape
    y = make(N, d, device="cuda", dtype=y_dtype)
    sum_out = make(N, d, device="cuda", dtype=x.dtype) if res is not None else None
    mean, rstd = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    tw.twell_layernorm_fwd(x, res, w, b, eps, sum_out, y, mean, rstd)
    s, m, r, hat, ref, wd = _fwd_ref(x, res, w, b, eps)
    if res is not None:
        # the sum is one fp32 addition rounded once more for bf16
        assert bool(((sum_out.double() - (x.double() + res.double())).abs()
                     <= (x.double() + res.double()).abs() * (2.0 ** -8 if x.dtype is BF else U) + 1e-37).all())
        s = sum_out
        _, m, r, hat, ref, wd = _fwd_ref(s, None, w, b, eps)
    v = s.double()
    k = d / 32 + 64
    assert bool(((mean.double() - m).abs() <= k * U * v.abs().mean(1) + 1e-37).all())
    e = _hat_err(v, r, hat, d)
    assert bool(((rstd.double() - r).abs() <= r * e.amax(1)).all())
    assert bool(((y.double() - ref).abs() <= e * wd.abs() + _out_tol(ref, y_dtype)).all())
    return y, sum_out, mean, rstd


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 33), (2, 1000), (129, 257), (33, 24), (64, 4096), (300, 512), (7, 8192), (700, 2048),
          (3, 12345), (4, 16384), (2, 40000), (1000, 96)]


@pytest.mark.parametrize("N,d", SHAPES)
@pytest.mark.parametrize("types", [(BF, BF, F32), (F32, BF, F32), (F32, F32, BF), (BF, F32, BF)])
@pytest.mark.parametrize("res", [False, True])
def test_forward(N, d, types, res):
    tx, ty, tp = types
    x = _rand((N, d), tx, 1, 2.0, 0.3)
    r = _rand((N, d), tx, 2) if res else None
    _check_fwd(x, r, _rand((d,), tp, 3, 0.2, 1.0), _rand((d,), tp, 4, 0.3), ty)


def _check_bwd(dy, x, w, dres, mean, rstd, make=torch.empty, grads=True):
    N, d = x.shape
    dx = make(N, d, device="cuda", dtype=x.dtype)
    dw, db = (torch.full((d,), 7.0, device="cuda") for _ in range(2)) if grads else (None, None)
    ws = torch.empty(tw.twell_layernorm_bwd_workspace_bytes(N, d), dtype=torch.uint8, device="cuda")
    tw.twell_layernorm_bwd(dy, x, w, mean, rstd, dres, dx, dw, db, ws)
    hat = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    wd = torch.ones(d, dtype=torch.float64, device="cuda") if w is None else w.double()
    v = dy.double() * wd
    r = rstd.double()[:, None]
    ref = r * (v - v.mean(1, keepdim=True) - hat * (v * hat).mean(1, keepdim=True))
    # hat here is one fp32 subtraction and product from exact inputs: 3 u of (|x| + |mean|) rstd
    h = hat.abs() + 3 * U * (x.double().abs() + mean.double().abs()[:, None]) * r
    dh = 3 * U * (x.double().abs() + mean.double().abs()[:, None]) * r
    k = (d / 32 + 64) * U
    tol = r * (8 * U * v.abs() + k * v.abs().mean(1, keepdim=True) + h * (k * (v.abs() * h).mean(1, keepdim=True))
               + dh * (v.abs() * h).mean(1, keepdim=True) + h * (v.abs() * dh).mean(1, keepdim=True)
               + 8 * U * h * (v.abs() * h).mean(1, keepdim=True))
    if dres is not None:
        ref = ref + dres.double()
        tol = tol + 2 * U * ref.abs() + 2 * U * dres.double().abs()
    assert bool(((dx.double() - ref).abs() <= tol + _out_tol(ref, x.dtype)).all())
    if grads:
        kn = (min(N, 20000) + 64) * U
        g = dy.double()
        assert bool(((dw.double() - (g * hat).sum(0)).abs() <= kn * (g.abs() * h).sum(0) + (g.abs() * dh).sum(0) + 1e-37).all())
        assert bool(((db.double() - g.sum(0)).abs() <= kn * g.abs().sum(0) + 1e-37).all())
    return dx, dw, db


def _stats(x, eps=1e-5):
    v = x.float()
    mean = v.mean(1)
    return mean, 1.0 / torch.sqrt(((v - mean[:, None]) ** 2).mean(1) + eps)


@pytest.mark.parametrize("N,d", SHAPES + [(5000, 40), (3000, 257)])
@pytest.mark.parametrize("types", [(BF, BF, F32), (F32, BF, F32), (F32, F32, BF), (BF, F32, BF)])
@pytest.mark.parametrize("dres", [False, True])
def test_backward(N, d, types, dres):
    tx, ty, tp = types
    x = _rand((N, d), tx, 1, 2.0, 0.3)
    mean, rstd = _stats(x)
    _check_bwd(_rand((N, d), ty, 2), x, _rand((d,), tp, 3, 0.2, 1.0), _rand((N, d), tx, 5) if dres else None, mean, rstd)


@pytest.mark.parametrize("w,b", [(False, False), (True, False), (False, True)])
def test_without_weight_or_bias(w, b):
    x = _rand((37, 520), BF, 1)
    wt = _rand((520,), F32, 2, 0.1, 1.0) if w else None
    bt = _rand((520,), F32, 3) if b else None
    _, _, mean, rstd = _check_fwd(x, None, wt, bt, BF)
    _check_bwd(_rand((37, 520), BF, 4), x, wt, None, mean, rstd)
    _check_bwd(_rand((37, 520), BF, 4), x, wt, None, mean, rstd, grads=False)


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (16, 8), (5, 1), (0, 1), (7, 3)])
@pytest.mark.parametrize("d", [256, 1000, 4096])
def test_strided_and_misaligned_rows(pad, shift, d):
    """Rows of a wider matrix that start anywhere; what lies between the rows of the outputs stays."""
    N = 21
    made = []

    def make(n, dd, device, dtype):
        base = torch.full((n * (dd + pad) + shift,), 9.0, device=device, dtype=dtype)
        view = base[shift:].view(n, dd + pad)[:, :dd] if pad else base[shift:].view(n, dd)
        made.append((base, view, shift, pad))
        return view

    def strided(t):
        v = make(t.shape[0], t.shape[1], "cuda", t.dtype)
        v.copy_(t)
        made.pop()
        return v

    for tx, ty in ((BF, BF), (F32, BF)):
        x, res = strided(_rand((N, d), tx, 1)), strided(_rand((N, d), tx, 2))
        w, b = _rand((d,), F32, 3, 0.1, 1.0), _rand((d,), F32, 4)
        _, s, mean, rstd = _check_fwd(x, res, w, b, ty, make=make)
        _check_bwd(strided(_rand((N, d), ty, 5)), s, w, strided(_rand((N, d), tx, 6)), mean, rstd, make=make)
    for base, view, sh, pd in made:
        outside = torch.ones_like(base, dtype=torch.bool)
        outside[sh:].view(N, -1)[:, :d] = False
        assert bool((base[outside] == 9.0).all())


def test_large_offset_keeps_its_variance():
    """Rows whose mean is 10^4 times their deviation: a one-pass variance of squares would lose it."""
    x = _rand((50, 1024), F32, 1, 1.0, 1e4)
    _check_fwd(x, None, None, None, F32)
    _check_fwd(_rand((9, 777), F32, 1, 1.0, -3e4), None, None, None, F32)


def test_constant_rows_and_single_elements():
    x = torch.full((3, 640), 2.5, device="cuda", dtype=BF)
    y, _, mean, rstd = _check_fwd(x, None, None, _rand((640,), F32, 1), BF)
    assert bool((mean == 2.5).all())
    assert torch.allclose(rstd, torch.full((3,), 1e-5 ** -0.5, device="cuda"), rtol=1e-6)


def test_one_bad_row_leaves_the_others():
    for d in (64, 1001, 4096):
        x = _rand((40, d), F32, 1)
        y0, _, m0, r0 = _check_fwd(x, None, None, None, F32)
        for bad in (float("nan"), float("inf")):
            z = x.clone()
            z[17, d // 2] = bad
            y = torch.empty_like(y0)
            mean, rstd = torch.empty_like(m0), torch.empty_like(r0)
            tw.twell_layernorm_fwd(z, None, None, None, 1e-5, None, y, mean, rstd)
            keep = torch.arange(40, device="cuda") != 17
            assert torch.equal(y[keep], y0[keep]) and torch.equal(mean[keep], m0[keep])
            assert bool(y[17].isnan().all())


def test_no_rows():
    d = 96
    e = torch.empty(0, d, device="cuda", dtype=BF)
    w, b = torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")
    st = torch.empty(0, device="cuda")
    tw.twell_layernorm_fwd(e, None, w, b, 1e-5, None, e.clone(), st, st)
    dw, db = torch.full((d,), 3.0, device="cuda"), torch.full((d,), 3.0, device="cuda")
    ws = torch.empty(tw.twell_layernorm_bwd_workspace_bytes(0, d), dtype=torch.uint8, device="cuda")
    tw.twell_layernorm_bwd(e, e, w, st, st, None, e.clone(), dw, db, ws)
    assert not dw.any() and not db.any()


def test_same_bits_every_time_and_on_another_stream():
    x, dy = _rand((3001, 520), BF, 1), _rand((3001, 520), BF, 2)
    w, b = _rand((520,), F32, 3), _rand((520,), F32, 4)
    ref = None
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        stream.wait_stream(torch.cuda.current_stream())
        y, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd, dw, db = (torch.empty(n, device="cuda") for n in (3001, 3001, 520, 520))
        ws = torch.empty(tw.twell_layernorm_bwd_workspace_bytes(3001, 520), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        tw.twell_layernorm_fwd(x, None, w, b, 1e-5, None, y, mean, rstd, stream=stream)
        tw.twell_layernorm_bwd(dy, x, w, mean, rstd, None, dx, dw, db, ws, stream=stream)
        stream.synchronize()
        out = (y, dx, mean, rstd, dw, db)
        if ref is None:
            ref = out
        assert all(torch.equal(a, c) for a, c in zip(ref, out))


def test_gradients_against_differences():
    """Central differences of sum(c * LN(x)) in 64 bits along random directions, against the kernels' fp32 gradients.
    Truncation is h^2 times the third derivative (h = 1e-4: ~1e-7), the kernels' own error a few times 1e-6 of the
    magnitudes summed."""
    N, d, h = 11, 200, 1e-4
    x, c = _rand((N, d), F32, 1), _rand((N, d), F32, 2)
    w, b = _rand((d,), F32, 3, 0.2, 1.0), _rand((d,), F32, 4)
    mean, rstd = _stats(x)
    dx, dw, db = _check_bwd(c, x, w, None, mean, rstd)

    def loss(xx, ww, bb):
        m = xx.mean(1, keepdim=True)
        hat = (xx - m) / torch.sqrt(((xx - m) ** 2).mean(1, keepdim=True) + 1e-5)
        return float((c.double() * (hat * ww + bb)).sum())

    X, Wd, Bd = x.double(), w.double(), b.double()
    for seed in range(3):
        vx, vw, vb = (_rand(t.shape, F32, 10 + seed).double() for t in (x, w, b))
        for got, v, up, down in ((dx, vx, loss(X + h * vx, Wd, Bd), loss(X - h * vx, Wd, Bd)),
                                 (dw, vw, loss(X, Wd + h * vw, Bd), loss(X, Wd - h * vw, Bd)),
                                 (db, vb, loss(X, Wd, Bd + h * vb), loss(X, Wd, Bd - h * vb))):
            along = float((got.double() * v).sum())
            size = float((got.double() * v).abs().sum())
            assert abs(along - (up - down) / (2 * h)) <= 1e-5 * size + 1e-5


def test_offsets_past_32_bits():
    """2.5e9 elements: the last rows are where a 32-bit offset would wrap."""
    N, d = 600_000, 4096
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB")
    x = torch.zeros(N, d, device="cuda", dtype=BF)
    dy = torch.zeros(N, d, device="cuda", dtype=BF)
    tail = _rand((5, d), BF, 1)
    x[-5:] = tail
    dy[-5:] = tail.flip(0)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    tw.twell_layernorm_fwd(x, None, None, None, 1e-5, None, y, mean, rstd)
    dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(tw.twell_layernorm_bwd_workspace_bytes(N, d), dtype=torch.uint8, device="cuda")
    tw.twell_layernorm_bwd(dy, x, None, mean, rstd, None, dx, dw, db, ws)
    small = torch.empty_like(tail)
    m5, r5 = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    tw.twell_layernorm_fwd(tail, None, None, None, 1e-5, None, small, m5, r5)
    assert torch.equal(y[-5:], small) and torch.equal(mean[-5:], m5)
    assert not y[:-5].any()
    dx5, dw5, db5 = _check_bwd(tail.flip(0).contiguous(), tail, None, None, m5, r5)
    assert torch.equal(dx[-5:], dx5)
    assert torch.allclose(dw, dw5, rtol=1e-5, atol=1e-5) and torch.allclose(db, db5, rtol=1e-5, atol=1e-5)


def test_wrong_arguments_are_refused():
    x = _rand((4, 64), BF, 1)
    y, w = torch.empty_like(x), torch.ones(64, device="cuda")
    m, r = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    with pytest.raises(ValueError):
        tw.twell_layernorm_fwd(x.cpu(), None, w, None, 1e-5, None, y, m, r)
    with pytest.raises(ValueError):
        tw.twell_layernorm_fwd(x, None, w[:63], None, 1e-5, None, y, m, r)
    with pytest.raises(ValueError):
        tw.twell_layernorm_fwd(x, x.float(), w, None, 1e-5, torch.empty_like(x), y, m, r)
    with pytest.raises(ValueError):
        tw.twell_layernorm_fwd(x.half(), None, w, None, 1e-5, None, y, m, r)
    with pytest.raises(ValueError):
        tw.twell_layernorm_fwd(x.t().contiguous().t(), None, w, None, 1e-5, None, y, m, r)
    for bad in (lambda: tw.twell_layernorm_fwd(x, x, w, None, 1e-5, None, y, m, r),         # res without sum
                lambda: tw.twell_layernorm_fwd(x, None, w, None, 1e-5, None, x, m, r),      # y on x
                lambda: tw.twell_layernorm_fwd(x, None, w, None, -1.0, None, y, m, r),
                lambda: tw.twell_layernorm_fwd(x, None, w, None, float("nan"), None, y, m, r)):
        with pytest.raises(tw.TwellError) as e:
            bad()
        assert e.value.status == 1
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(tw.TwellError) as e:
        tw.twell_layernorm_bwd(x, y, w, m, r, None, torch.empty_like(x), torch.empty(64, device="cuda"),
                               torch.empty(64, device="cuda"), ws)
    assert e.value.status == 3
    assert np.isfinite(float(w.sum()))


@pytest.mark.parametrize("N,d", [(9, 2), (50, 1002), (700, 130), (33, 4094), (5, 8190), (3000, 34)])
@pytest.mark.parametrize("types", [(BF, BF, F32), (F32, BF, BF), (F32, F32, F32), (BF, F32, F32)])
@pytest.mark.parametrize("res", [False, True])
def test_even_widths(N, d, types, res):
    """Rows of an even number of elements that is no multiple of 4 start on a pair's boundary only."""
    tx, ty, tp = types
    x, r = _rand((N, d), tx, 1, 2.0, 0.3), _rand((N, d), tx, 2) if res else None
    w, b = _rand((d,), tp, 3, 0.2, 1.0), _rand((d,), tp, 4, 0.3)
    _, s, mean, rstd = _check_fwd(x, r, w, b, ty)
    _check_bwd(_rand((N, d), ty, 5), x if s is None else s, w, _rand((N, d), tx, 6) if res else None, mean, rstd)


@pytest.mark.parametrize("N", [1, 2, 151, 152, 153, 303, 304, 305, 608, 609, 896, 897, 1216, 1217, 3000])
def test_rows_around_a_full_gpu(N):
    """Fewer rows than resident blocks, exactly as many, one more: groups with no row, one row, several."""
    for d in (24, 512, 1001):
        x = _rand((N, d), BF, 1, 2.0, 0.3)
        w = _rand((d,), F32, 3, 0.2, 1.0)
        _, _, mean, rstd = _check_fwd(x, None, w, None, BF)
        _check_bwd(_rand((N, d), BF, 5), x, w, None, mean, rstd)
