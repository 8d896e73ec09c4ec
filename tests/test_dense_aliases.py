"""Buffers that the linear and gated layers refuse to share, on the host: no call below reaches a GPU."""
import ctypes
import itertools

import pytest

from activation_sparse_transformer_tcgen05_gb300 import build as tbuild
from activation_sparse_transformer_tcgen05_gb300 import twell as tw

INVALID = 1


@pytest.fixture(scope="module")
def lib():
    tbuild.build()
    return tw.load_library()


def _at(names):
    return {k: ctypes.c_void_p((i + 1) << 20) for i, k in enumerate(names)}


def _refused(call, names, outputs, inputs):
    """Every output as every input and as every other output."""
    for out, other in [*itertools.product(outputs, inputs), *itertools.combinations(outputs, 2)]:
        at = _at(names)
        at[out] = at[other]
        assert call(**at) == INVALID, (out, other)


def test_linear_forward(lib):
    names = ("x", "W", "bias", "res", "pre", "y", "st")

    def call(x, W, bias, res, pre, y, st, ldres=24, ldy=24):
        return lib.twell_linear_fwd(x, 64, W, 0, bias, 0, res, ldres, 4, 24, 64, pre, 24, y, ldy, 1, st, None)

    _refused(call, names, ("pre", "y"), ("x", "W", "bias"))
    at = _at(names)
    assert call(**{**at, "pre": at["res"]}) == INVALID
    # in place: rows of the sum that lie elsewhere than the residual's would replace rows that are not read yet
    in_place = {**at, "y": at["res"]}
    assert call(**in_place, ldres=32) == call(**in_place, ldy=32) == INVALID


def test_linear_backward(lib):
    need = lib.twell_linear_bwd_workspace_bytes(100, 24, 64)

    def call(dy, x, W, pre, dx, dW, db, ws, st):
        return lib.twell_linear_bwd(dy, 24, x, 64, W, 0, 1, pre, 24, 100, 24, 64, dx, 64, dW, 1, 0, db, ws, need, st, None)

    _refused(call, ("dy", "x", "W", "pre", "dx", "dW", "db", "ws", "st"), ("dx", "dW", "db", "ws"), ("dy", "x", "W", "pre"))


def test_gated_forward(lib):
    names = ("x", "Wg", "Wu", "b", "Wd", "res", "g", "u", "h", "y", "st")

    def call(x, Wg, Wu, b, Wd, res, g, u, h, y, st):
        return lib.twell_dense_gated_ffn_fwd(x, Wg, Wu, b, Wd, 1, res, 4, 64, 24, g, u, h, y, st, None)

    _refused(call, names, ("g", "u", "h", "y"), ("x", "Wg", "Wu", "b", "Wd"))
    at = _at(names)
    for k in ("g", "u", "h"):  # written before the residual is read
        assert call(**{**at, "res": at[k]}) == INVALID, k


def test_gated_backward(lib):
    need = lib.twell_dense_gated_bwd_workspace_bytes(100, 64, 24)

    def call(x, Wg, Wu, Wd, g, u, h, dy, dx, dWg, dWu, dWd, db, ws, st):
        return lib.twell_dense_gated_ffn_bwd(x, Wg, Wu, Wd, 1, g, u, h, dy, 0.0, 100, 64, 24, dx, dWg, dWu, dWd, 1, 0, db, ws, need, st,
                                             None)

    inputs = ("x", "Wg", "Wu", "Wd", "g", "u", "h", "dy")
    outputs = ("dx", "dWg", "dWu", "dWd", "db", "ws")
    _refused(call, (*inputs, *outputs, "st"), outputs, inputs)
