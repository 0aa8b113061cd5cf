"""Host-side checks of the operators over point features that need no GPU:
argument validation of the C ABI and of the binding."""
import ctypes

import pytest
import torch

import point_cloud_neighbor_gb300 as pc
from point_cloud_neighbor_gb300 import binding, build
from point_cloud_neighbor_gb300.binding import lib

FAKE = ctypes.c_void_p(0x1000)   # never read: the checks come first


@pytest.fixture(scope="module")
def L():
    build.build()
    return lib()


def _msg(L):
    return L.pc_last_error_message().decode()


def gn(L, dtype=0, B=1, L_=4, C=8, G=2, p=0, eps=1e-5, act=1, mean=None, rstd=None):
    return L.pc_group_norm(FAKE, dtype, B, L_, C, G, None, None, p, eps, act, None, FAKE, mean,
                           rstd, None)


def test_group_norm_validation(L):
    assert gn(L, dtype=2) == 1
    assert gn(L, B=-1) == 1
    assert gn(L, p=1) == 1
    assert gn(L, G=0) == 1
    assert gn(L, G=3) == 1 and "divide" in _msg(L)
    assert gn(L, act=5) == 1 and gn(L, act=-1) == 1
    assert gn(L, eps=float("nan")) == 1 and gn(L, eps=-1e-9) == 1
    assert gn(L, mean=FAKE) == 1 and "go together" in _msg(L)
    assert gn(L, C=16386) == 2
    assert gn(L, L_=2 ** 31) == 2
    assert gn(L, B=2 ** 28) == 2
    assert gn(L, B=0) == 0 and gn(L, L_=0) == 0

    def back(dtype=0, B=1, G=2, act=1, dx=FAKE):
        return L.pc_group_norm_backward(FAKE, FAKE, dtype, B, 4, 8, G, FAKE, FAKE, None, None, 0,
                                        act, None, dx, None, None, None)
    assert back(dtype=7) == 1 and back(G=5) == 1 and back(act=9) == 1 and back(B=-2) == 1
    assert back(dx=None) == 0


def test_gated_linear_validation(L):
    def call(dtype=0, rows=4, C=8, F=8, bg=None, bu=None, act=1):
        return L.pc_gated_linear(FAKE, dtype, rows, C, F, FAKE, FAKE, bg, bu, act, FAKE, None, 0,
                                 None)
    assert call(dtype=3) == 1
    assert call(rows=-1) == 1 and call(F=-1) == 1 and call(C=0) == 1
    assert call(bg=FAKE) == 1 and "go together" in _msg(L)
    assert call(act=6) == 1
    assert call(C=16385) == 2 and call(F=65537) == 2 and call(rows=2 ** 30 + 1) == 2
    assert call(rows=0) == 0 and call(F=0) == 0

    def back(dwg=FAKE, dwu=FAKE, dbg=None, dbu=None, dx=FAKE, dtype=0):
        return L.pc_gated_linear_backward(FAKE, FAKE, dtype, 4, 8, 8, FAKE, FAKE, None, None, 1,
                                          dx, dwg, dwu, dbg, dbu, None, 0, None)
    assert back(dwu=None) == 1 and back(dbg=FAKE) == 1 and back(dtype=-1) == 1
    assert back(dwg=None, dwu=None, dx=None) == 0


def test_embedding_validation(L):
    def call(dtype=0, B=1, V=5, C=8, T=3, scale=1.0):
        return L.pc_embedding(FAKE, dtype, B, V, C, FAKE, T, scale, FAKE, None)
    assert call(dtype=2) == 1
    assert call(B=-1) == 1 and call(V=-1) == 1 and call(T=-1) == 1
    assert call(scale=float("inf")) == 1 and call(scale=float("nan")) == 1
    assert call(C=65537) == 2 and call(B=2 ** 21, T=2 ** 21) == 2
    assert call(B=0) == 0 and call(T=0) == 0 and call(C=0) == 0

    def back(B=1, V=5, T=3, dtype=0, scale=1.0):
        return L.pc_embedding_backward(FAKE, dtype, B, V, 8, FAKE, T, scale, FAKE, None)
    assert back(V=2 ** 31) == 2 and back(T=2 ** 31) == 2 and back(B=2 ** 16, V=2 ** 16) == 2
    assert back(dtype=4) == 1 and back(scale=float("nan")) == 1
    assert back(V=0) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_feature_operators_report_no_device(L):
    assert gn(L) == binding.PC_ERR_NO_DEVICE
    assert L.pc_gated_linear(FAKE, 0, 4, 8, 8, FAKE, FAKE, None, None, 1, FAKE, None, 0,
                             None) == binding.PC_ERR_NO_DEVICE
    assert L.pc_gated_linear_workspace_bytes(0, 4, 8, 8, 7) == 0
    assert L.pc_embedding(FAKE, 0, 1, 5, 8, FAKE, 3, 1.0, FAKE, None) == binding.PC_ERR_NO_DEVICE
    assert L.pc_embedding_backward(FAKE, 0, 1, 5, 8, FAKE, 3, 1.0, FAKE,
                                   None) == binding.PC_ERR_NO_DEVICE


def test_feature_operators_reject_cpu_tensors():
    x = torch.zeros(1, 4, 8)
    i = torch.zeros(1, 4, dtype=torch.int64)
    for call in (lambda: pc.pc_group_norm(x, 2), lambda: pc.pc_gated_linear(x, x[0], x[0]),
                 lambda: pc.pc_embedding(x, i), lambda: pc.pc_embedding_backward(x, i, (5, 8))):
        with pytest.raises(ValueError, match="no CPU path"):
            call()
