"""Shapes that the gated layer's functions refuse: matrices of the right size but another layout would be read as if they
were [d_ff, d_model]. CPU tensors, which are refused after their shapes are looked at."""
import pytest
import torch

from activation_sparse_transformer_tcgen05_gb300 import build as tbuild
from activation_sparse_transformer_tcgen05_gb300 import twell as tw

M, D, F = 6, 16, 24


@pytest.fixture(scope="module", autouse=True)
def _library():
    tbuild.build()


def _mat(*shape, t=torch.bfloat16):
    return torch.zeros(*shape, dtype=t)


def _forward(**other):
    t = dict(x=_mat(M, D), W_gate=_mat(F, D), W_up=_mat(F, D), b=_mat(F, t=torch.float32), W_down=_mat(F, D), act=tw.ACT_SILU,
             res=_mat(M, D), g=_mat(M, F), u=_mat(M, F), h=_mat(M, F), y=_mat(M, D), status=torch.zeros(1, dtype=torch.int32))
    tw.twell_dense_gated_ffn_fwd(**{**t, **other})


def _backward(**other):
    t = dict(x=_mat(M, D), W_gate=_mat(F, D), W_up=_mat(F, D), W_down=_mat(F, D), act=tw.ACT_SILU, g=_mat(M, F), u=_mat(M, F),
             h=_mat(M, F), dy=_mat(M, D), l1=0.0, dx=_mat(M, D), dW_gate=_mat(F, D), dW_up=_mat(F, D), dW_down=_mat(F, D),
             accumulate=False, db=_mat(F, t=torch.float32), ws=torch.zeros(1 << 16, dtype=torch.uint8),
             status=torch.zeros(1, dtype=torch.int32))
    tw.twell_dense_gated_ffn_bwd(**{**t, **other})


def test_right_shapes_get_as_far_as_the_device():
    for call in (_forward, _backward):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("name", ["W_gate", "W_up", "W_down", "g", "u", "h", "res", "y"])
def test_forward(name):
    shape = (D, F) if name[0] == "W" else (F, M) if name in "guh" else (D, M)
    for bad in (_mat(*shape), _mat(shape[0] * shape[1])):
        with pytest.raises(ValueError, match=rf"{name} must be a \["):
            _forward(**{name: bad})


@pytest.mark.parametrize("name", ["W_gate", "W_up", "W_down", "dW_gate", "dW_up", "dW_down", "g", "u", "h", "dy", "dx"])
def test_backward(name):
    shape = (D, F) if "W" in name else (F, M) if name in "guh" else (D, M)
    for bad in (_mat(*shape), _mat(shape[0] * shape[1])):
        with pytest.raises(ValueError, match=rf"{name} must be a \["):
            _backward(**{name: bad})


def test_rows_that_are_no_matrix():
    for call in (_forward, _backward):
        with pytest.raises(ValueError, match="x must be a matrix"):
            call(x=_mat(M * D))
