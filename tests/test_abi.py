"""CPU-only checks of the C ABI: the library builds, loads, exports every
symbol include/twell.h declares, and its host-side logic (sizes, argument
checks, status strings) answers without touching a GPU."""
import ctypes
import os
import re

import pytest

from activation_sparse_transformer_tcgen05_gb300 import build as tbuild
from activation_sparse_transformer_tcgen05_gb300 import twell as tw

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    tbuild.build()
    return tw.load_library()


def _declared_functions():
    src = open(os.path.join(ROOT, "include", "twell.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(twell_[a-z0-9_]+)\s*\(", src)))


def test_every_declared_symbol_is_exported(lib):
    names = _declared_functions()
    assert len(names) >= 10
    for n in names:
        assert hasattr(lib, n), f"{n} declared in twell.h but not exported"
    assert set(names) == set(tw.EXPORTED_SYMBOLS)


def test_status_strings(lib):
    assert tw.twell_status_string(0) == "ok"
    assert "capacity" in tw.twell_status_string(4)
    assert tw.twell_status_string(99) == "unknown status"


def test_slot_bound_and_workspace_sizes(lib):
    assert tw.twell_buf_slots_bound(4096, 8192, 128) == 4096 * 8192
    assert tw.twell_buf_slots_bound(0, 8, 1) == -1
    fwd = tw.twell_workspace_bytes(tw.OP_FFN_FWD, 4096, 2048, 8192, 128)
    # staging: one 32-bit entry per (row, column) plus a count per (row, 256-column block)
    assert fwd >= 4096 * 8192 * 4 + 4096 * 32 * 4
    assert tw.twell_workspace_bytes(tw.OP_PACK, 64, 128, 512, 16) == 0
    bwd_small = tw.twell_workspace_bytes(tw.OP_FFN_BWD, 4096, 2048, 8192, 128, 10_000)
    bwd_big = tw.twell_workspace_bytes(tw.OP_FFN_BWD, 4096, 2048, 8192, 128, 1_000_000)
    assert bwd_big - bwd_small >= 3 * 4 * 990_000 - 3 * 256  # dpre, row and slot per stored entry
    assert tw.twell_workspace_bytes(tw.OP_FFN_FWD, 0, 2048, 8192, 128) == 0
    # union down-projection: per group a list of F unit ids, plus one word per stored entry
    u_small = tw.twell_spmm_down_tc_workspace_bytes(4096, 8192, 10_000)
    u_big = tw.twell_spmm_down_tc_workspace_bytes(4096, 8192, 1_000_000)
    assert u_small >= 32 * 8192 * 4 and u_big - u_small >= 4 * 990_000 - 256
    assert tw.twell_spmm_down_tc_workspace_bytes(4096, 65544, 10) == 0
    assert tw.twell_spmm_down_tc_workspace_bytes(4096, 100, 10) == 0  # F % 8 != 0


def test_host_argument_errors_need_no_gpu(lib):
    buf = tw._TwellBuf(64, 512, 16, 4, 0, None, None, None, None, None)
    rc = lib.twell_ffn_fwd(None, None, None, None, None, 64, 128, 512, 16, ctypes.byref(buf),
                           None, None, 0, None, None)
    assert rc == 1  # TWELL_ERR_INVALID_ARG
    rc = lib.twell_pack(None, 64, 512, 512, 16, ctypes.byref(buf), None, None)
    assert rc == 1
    rc = lib.twell_spmm_down(None, None, 128, None, None, None)
    assert rc == 1
    rc = lib.twell_ffn_bwd(None, None, None, None, None, 128, 0.0, None, None, None, None, None, 0, None, None)
    assert rc == 1
    rc = lib.twell_check(None, None, None)
    assert rc == 1
    rc = lib.twell_dense_ffn_fwd(None, None, None, None, 64, 128, 512, None, None, None, None)
    assert rc == 1
    rc = lib.twell_dense_ffn_bwd(None, None, None, None, None, 64, 128, 512, 0.0, None, None, None, None, None, 0,
                                 None, None)
    assert rc == 1
    fake = ctypes.c_void_p(256)  # never dereferenced: d % 8 != 0 is rejected first
    rc = lib.twell_dense_ffn_bwd(fake, fake, fake, fake, fake, 64, 124, 512, 0.0, fake, fake, fake, fake, fake,
                                 1 << 20, fake, None)
    assert rc == 1
    assert lib.twell_dense_bwd_workspace_bytes(64, 124, 512) == 0
    assert lib.twell_dense_bwd_workspace_bytes(256, 128, 512) == 256 * 512 * 2 + 2 * 512 * 4
    assert lib.twell_set_kernel_timer(11, None, None) == 1  # no such call site
    rc = lib.twell_spmm_down_tc(None, None, 128, None, None, 0, None, None)
    assert rc == 1
    big = tw._TwellBuf(64, 65544, 16, 4, 0, fake, fake, fake, None, None)  # F above the union kernel's limit
    rc = lib.twell_spmm_down_tc(ctypes.byref(big), fake, 128, fake, fake, 1 << 20, fake, None)
    assert rc == 2  # TWELL_ERR_UNSUPPORTED
    assert lib.twell_wait_selftest(2, fake, fake, None) == 1  # no such wait
    assert lib.twell_wait_selftest(0, None, None, None) == 1


def test_ops_fail_loudly_without_library(tmp_path):
    with pytest.raises(RuntimeError, match="not found"):
        tw.load_library(str(tmp_path / "missing.so"))


def test_training_step_operators_refuse_wrong_arguments_without_a_gpu(lib):
    fake = ctypes.c_void_p(256)  # never dereferenced: each call below is refused on the host
    odd = ctypes.c_void_p(257)
    inf = float("inf")

    def ln(x=fake, ldx=64, res=None, N=4, d=64, eps=1e-5, tx=0, ty=0, sum_=None, y=ctypes.c_void_p(512), ldy=64):
        return lib.twell_layernorm_fwd(x, ldx, res, 64, None, None, N, d, eps, tx, ty, 1, sum_, 64, y, ldy, None, None, None)

    assert ln(x=None) == 1 and ln(y=None) == 1 and ln(N=-1) == 1 and ln(d=0) == 1 and ln(eps=-1.0) == 1
    assert ln(ldx=63) == 1 and ln(ldy=63) == 1 and ln(tx=2) == 1 and ln(ty=-1) == 1
    assert ln(res=fake) == 1 and ln(sum_=fake) == 1 and ln(y=fake) == 1 and ln(x=odd) == 1
    assert ln(N=0, x=None, y=None) == 0  # no rows: nothing to do
    assert lib.twell_layernorm_bwd_workspace_bytes(-1, 64) == 0 and lib.twell_layernorm_bwd_workspace_bytes(4, 0) == 0
    need = lib.twell_layernorm_bwd_workspace_bytes(4096, 2048)
    assert need >= 2 * 2048 * 4
    y = ctypes.c_void_p(512)
    assert lib.twell_layernorm_bwd(fake, 2048, fake, 2048, None, fake, fake, None, 0, 4096, 2048, 0, 0, 1, y, 2048, fake,
                                   fake, fake, need - 1, None) == 3
    assert lib.twell_layernorm_bwd(fake, 2048, fake, 2048, None, fake, fake, None, 0, 4096, 2048, 0, 0, 1, y, 2048, fake,
                                   None, fake, need, None) == 1  # dw without db

    fwd, bwd = lib.twell_xent_fwd_workspace_bytes, lib.twell_xent_bwd_workspace_bytes
    assert fwd(-1, 64, 10) == 0 and fwd(4, 60, 10) == 0 and fwd(4, 64, 0) == 0 and bwd(4, 64, 10, -1, 0) == 0
    assert bwd(4, 64, 10, 0, 2) == 0
    assert bwd(8192, 4096, 65536, 8192, 0) >= 8192 * 65536 * 2          # two bytes a logit of the chunk
    assert bwd(8192, 4096, 65536, 1024, 1) < 8192 * 65536               # fewer rows at a time: less
    assert bwd(8192, 4096, 65536, 1024, 0) - bwd(8192, 4096, 65536, 1024, 1) == 65536 * 4096 * 4  # bf16 dW: fp32 sums
    big = 1 << 40

    def xe(x=fake, N=4, d=64, V=10, ws=fake, n=big, dx=fake, dW=fake, tw_=0, acc=0, chunk=0, status=fake):
        return lib.twell_xent_fwd_bwd(x, fake, fake, N, d, V, -100, 1, 1.0, chunk, fake, fake, fake, dx, dW, tw_, acc, ws, n,
                                      status, None)

    assert xe(x=None) == 1 and xe(dx=None) == 1 and xe(dW=None) == 1 and xe(status=None) == 1 and xe(d=60) == 1
    assert xe(N=-1) == 1 and xe(V=0) == 1 and xe(tw_=3) == 1 and xe(acc=1) == 1 and xe(chunk=-2) == 1
    assert xe(x=ctypes.c_void_p(264)) == 1 and xe(ws=None) == 3 and xe(n=16) == 3 and xe(ws=ctypes.c_void_p(128)) == 1
    assert lib.twell_xent_fwd(fake, fake, fake, 4, 64, 10, -100, 1, fake, fake, None, fake, big, fake, None) == 1
    assert lib.twell_xent_fwd(fake, fake, fake, 4, 64, 10, -100, 1, fake, fake, fake, fake, 16, fake, None) == 3

    def clip(n=1, numel=4, type_=1, addr=256, max_norm=1.0, ws=fake, nb=big, norm=fake):
        a, o = (ctypes.c_void_p * 1)(addr), (ctypes.c_void_p * 1)(addr)
        m, t = (ctypes.c_int64 * 1)(numel), (ctypes.c_int32 * 1)(type_)
        st = tw._TwellTensorList(n, ctypes.addressof(a), ctypes.addressof(o), ctypes.addressof(m), ctypes.addressof(t))
        return lib.twell_grad_clip(ctypes.byref(st), max_norm, norm, ws, nb, None)

    assert lib.twell_grad_clip(None, 1.0, fake, fake, big, None) == 1
    assert clip(n=-1) == 1 and clip(numel=-1) == 1 and clip(type_=2) == 1 and clip(addr=0) == 1 and clip(addr=258) == 1
    assert clip(max_norm=-1.0) == 1 and clip(max_norm=float("nan")) == 1 and clip(norm=None) == 1
    assert clip(ws=None) == 3 and clip(nb=16) == 3 and clip(ws=ctypes.c_void_p(128)) == 1
    assert clip(numel=1 << 60, max_norm=inf) == 2
