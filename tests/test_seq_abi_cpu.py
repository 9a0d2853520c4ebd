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


def test_offsets_are_no_output(L):
    """The address of the offsets as an output is refused, as any other input's."""
    conv, scan = lib.conv_dims(0, 16, 16, 4, lib.BF16, 1), lib.ssm_dims(0, 16, 16, 16, lib.BF16, 1)
    for y, s1 in ((A1, None), (A2, A1)):
        assert L.adj_conv_fwd(ctypes.byref(conv), A0, A0, None, None, A1, y, s1, None) == 1
        assert L.adj_ssm_fwd(ctypes.byref(scan), *[A0] * 5, None, None, None, None, A1, y, s1, A0, 1 << 50, None) == 1
    for i in range(4):
        outs = [A2, A2 + 64, A2 + 128, A2 + 192]
        outs[i] = A1
        assert L.adj_conv_bwd(ctypes.byref(conv), A0, A0, None, None, A1, A0, None, *outs, A0, 1 << 50, None) == 1
    for i in (0, 1, 2, 3, 4, 5, 7, 8):                      # dx ddt dA dB dC dD (dz) ddt_bias ds0
        outs = [A2 + 64 * k for k in range(9)]
        outs[6] = None
        outs[i] = A1
        assert L.adj_ssm_bwd(ctypes.byref(scan), *[A0] * 5, None, None, None, None, A1, A0, None, *outs, A0, 1 << 50, None) == 1
