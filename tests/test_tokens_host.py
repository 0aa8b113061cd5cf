"""Host-side checks of the point-token operators that need no GPU: argument
validation of the C ABI, and the autograd rules over stand-ins of the calls."""
import ctypes

import pytest

from point_cloud_neighbor_gb300 import build
from point_cloud_neighbor_gb300.binding import lib

FAKE = ctypes.c_void_p(0x1000)   # never read: the checks come first


@pytest.fixture(scope="module")
def L():
    build.build()
    return lib()


def test_the_output_s_low_part_is_bfloat16_s(L):
    def forward(dtype, low, B=0):
        return L.pc_attention_ex(FAKE, FAKE, FAKE, dtype, B, 4, 4, 2, 1, 64, None, None, None,
                                 0.125, None, None, None, None, None, FAKE, low, None, None)

    def backward(dtype, low):
        return L.pc_attention_backward_ex(FAKE, FAKE, FAKE, FAKE, FAKE, low, FAKE, dtype, 0, 4, 4,
                                          2, 1, 64, None, None, None, 0.125, None, None, None,
                                          None, None, FAKE, FAKE, FAKE, None, None)
    for call in (forward, backward):
        assert call(1, FAKE) == 0 and call(0, None) == 0
        assert call(0, FAKE) == 1
        assert "out_low" in L.pc_last_error_message().decode()
