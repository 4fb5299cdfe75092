"""What the layer operators refuse beyond test_layer_abi_cpu.py, without a GPU."""
import ctypes

import pytest

from gated_deltanet_chunked_rule_b200 import _binding as B

INV = B.GDN_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def L():
    from gated_deltanet_chunked_rule_b200 import build
    build.build()
    return B.lib()


def q(i):
    return ctypes.c_void_p((1 << 20) + (i << 12))


def test_token_updates_refuse_outputs_over_inputs(L):
    """Each output given another buffer's place, everything else distinct; the states in place stay allowed
    (that they run is test_conv_gpu.py's and test_scan_gpu.py's)."""
    p = ctypes.byref(B.gdn_conv_problem(2, 1, 64, 4, 0, None, 1, 1, 64))
    for out in (3, 4):  # state (in place), y
        for i in range(5):
            if i != out:
                a = [q(k) for k in range(5)]  # x, weight, bias, state, y
                a[out] = q(i)
                assert L.gdn_conv_update(p, *a, None) == INV, (out, i)
    p = ctypes.byref(B.gdn_scan_problem(2, 1, 1, 2, 128, 64, 0, None, 1, 0, 1, 128, 128, 128, 2))
    for out in (8, 9):  # y, final state
        for i in range(10):
            if i != out and (out, i) != (9, 7):  # h0 may be updated in place
                a = [q(k) for k in range(10)]  # x, dt, A, B, C, D, dt_bias, h0, y, final
                a[out] = q(i)
                assert L.gdn_scan_step(p, *a, None) == INV, (out, i)
