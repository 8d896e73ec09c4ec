"""Layer norm with weights that start anywhere in a flat buffer."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from activation_sparse_transformer_tcgen05_gb300 import build as _build
    _build.build()
import activation_sparse_transformer_tcgen05_gb300 as tw  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def _at(v, offset):
    """A copy of v that starts `offset` elements into a buffer."""
    flat = torch.empty(v.numel() + 64, device="cuda", dtype=v.dtype)
    assert flat.data_ptr() % 256 == 0
    out = flat[offset:offset + v.numel()]
    out.copy_(v)
    return out


def _forward_backward(x, w, b, dy):
    N, d = x.shape
    y, dx = torch.empty(N, d, device="cuda", dtype=dy.dtype), torch.empty_like(x)
    mean, rstd = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(tw.twell_layernorm_bwd_workspace_bytes(N, d), dtype=torch.uint8, device="cuda")
    tw.twell_layernorm_fwd(x, None, w, b, 1e-5, None, y, mean, rstd)
    tw.twell_layernorm_bwd(dy, x, w, mean, rstd, None, dx, dw, db, ws)
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("types,w_type", [((BF, BF), F32), ((BF, BF), BF), ((F32, BF), F32), ((F32, F32), F32), ((BF, F32), F32)])
@pytest.mark.parametrize("N,d", [(300, 4096), (1500, 1024)])
def test_weights_on_16_byte_boundaries_are_as_good_as_any(types, w_type, N, d):
    """16-byte loads are all that is asked of the weights: on any such boundary the rows are read in the same pieces, so
    that every sum has the same order and the same bits."""
    g = torch.Generator(device="cuda").manual_seed(0)
    x = (3 * torch.randn(N, d, device="cuda", generator=g) + 0.5).to(types[0])
    dy = torch.randn(N, d, device="cuda", generator=g).to(types[1])
    w = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(w_type)
    b = (0.1 * torch.randn(d, device="cuda", generator=g)).to(w_type)
    step = 4 if w_type is F32 else 8
    ref = _forward_backward(x, _at(w, 0), _at(b, 0), dy)
    for ow, ob in ((step, 0), (0, step), (step, 3 * step)):
        out = _forward_backward(x, _at(w, ow), _at(b, ob), dy)
        assert all(torch.equal(p, q) for p, q in zip(ref, out))


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_weights_on_other_boundaries(offset):
    N, d = 64, 1024
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(N, d, device="cuda", generator=g).to(BF)
    dy = torch.randn(N, d, device="cuda", generator=g).to(BF)
    w, b = 1 + 0.1 * torch.randn(d, device="cuda", generator=g), 0.1 * torch.randn(d, device="cuda", generator=g)
    ref = _forward_backward(x, w, b, dy)
    out = _forward_backward(x, _at(w, offset), _at(b, offset), dy)
    for p, q in zip(ref, out):  # sums in another order: fp32 to a few hundred of its roundings, bf16 to one of its own
        tol = 2.0 ** -7 if p.dtype is BF else 2.0 ** -15
        assert bool(((p.double() - q.double()).abs() <= tol * p.double().abs() + 2.0 ** -14).all())
