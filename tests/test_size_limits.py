"""Sizes next to the range of int are refused on the host."""
import subprocess
import sys

import pytest

CALL = """
import ctypes
import activation_sparse_transformer_tcgen05_gb300 as tw
lib = tw.load_library()
a, b, c = (ctypes.c_void_p(k << 40) for k in (1, 2, 3))  # never dereferenced: the calls below are refused on the host
for d in ({sizes}):
    print(lib.twell_layernorm_bwd_workspace_bytes(3, d),
          lib.twell_layernorm_fwd(a, d, None, 0, None, None, 1, d, 1e-5, 0, 0, 1, None, 0, b, d, None, None, None),
          lib.twell_layernorm_bwd(a, d, b, d, None, a, a, None, 0, 1, d, 0, 0, 1, c, d, None, None, a, 1 << 60, None))
"""


@pytest.mark.parametrize("sizes", ["2**29 + 1, 2**30", "2**30 + 1, 2**31 - 1"])
def test_layer_norm_rows_past_the_limit(sizes):
    from activation_sparse_transformer_tcgen05_gb300 import build
    build.build()
    out = subprocess.run([sys.executable, "-c", CALL.format(sizes=sizes)], capture_output=True, text=True, timeout=300,
                         check=True).stdout
    assert out.split("\n")[:2] == ["0 2 2"] * 2


XENT = """
import ctypes
import activation_sparse_transformer_tcgen05_gb300 as tw
lib = tw.load_library()
a = ctypes.c_void_p(1 << 40)
for N, d, V in ((1, 8, 2**30 + 1), (1, 8, 2**31 - 1), (2**31 - 1, 8, 5), (1, 2**31 - 8, 5)):
    print(lib.twell_xent_fwd_workspace_bytes(N, d, V), lib.twell_xent_bwd_workspace_bytes(N, d, V, 1, 0),
          lib.twell_xent_fwd(a, a, a, N, d, V, -100, 1, a, a, a, a, 1 << 63, a, None),
          lib.twell_xent_fwd_bwd(a, a, a, N, d, V, -100, 1, 1.0, 1, a, a, a, a, a, 0, 0, a, 1 << 63, a, None))
"""


def test_cross_entropy_sizes_past_the_limit():
    from activation_sparse_transformer_tcgen05_gb300 import build
    build.build()
    out = subprocess.run([sys.executable, "-c", XENT], capture_output=True, text=True, timeout=300, check=True).stdout
    assert out.split("\n")[:4] == ["0 0 2 2"] * 4
