"""More of what the entry points of the short convolution and the selective scan take and refuse (nothing
is launched)."""
import ctypes

import pytest

from adjoint_gradients_long_gb300 import build as adj_build, lib


@pytest.fixture(scope="module")
def L():
    adj_build.build()
    return lib.load()


A0, A1, A2 = (1 << 40) + (1 << 30), (1 << 40) + (2 << 30), (1 << 40) + (3 << 30)    # never dereferenced


def test_steps_read_neither_length_nor_packing(L):
    """One token a sequence: T and packed may hold anything."""
    for T, packed in ((0, 0), (-5, 1), (1 << 40, -3), (16, 77)):
        conv = ctypes.byref(lib.conv_dims(0, T, 16, 4, lib.BF16, packed))
        assert L.adj_conv_step(conv, A0, A0, None, A1, 4, None, A2, None) == 0
        scan = ctypes.byref(lib.ssm_dims(0, T, 16, 16, lib.BF16, packed))
        assert L.adj_ssm_step(scan, A0, A0, A0, A0, A0, None, None, None, A1, 4, None, A2, None) == 0
        assert packed in (0, 1) or L.adj_conv_workspace_bytes(conv) == 0
        assert packed in (0, 1) or L.adj_ssm_workspace_bytes(scan, lib.OP_SSM_FWD) == 0
