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


def test_switches_of_the_prompts_paths(L, monkeypatch):
    # sizes are those of the path that the environment chooses; 8192 tokens of 64 heads go by segments anyhow
    def sizes(T, H, dtype=1):
        p = ctypes.byref(B.gdn_scan_problem(1, T, 1, H, 128, 64, 0, None, dtype, 0, 1, H * 64, 128, 128, H))
        return L.gdn_scan_fwd_workspace_size(p), L.gdn_scan_bwd_workspace_size(p), L.gdn_scan_saved_size(p)

    for name in ("GDN_IMPL", "GDN_SCAN_SPLIT"):
        monkeypatch.delenv(name, raising=False)
    small, large, fp32 = sizes(1024, 4), sizes(8192, 64), sizes(1024, 4, 0)
    assert small[2] > 0 and fp32[2] == 0
    monkeypatch.setenv("GDN_SCAN_SPLIT", "segments")
    assert sizes(1024, 4) != small and sizes(1024, 4)[2] == small[2]
    assert sizes(8192, 64) == large and sizes(1024, 4, 0) == fp32
    monkeypatch.setenv("GDN_IMPL", "simt")
    assert sizes(1024, 4) == fp32


def test_backward_workspace_with_kept_states(L, monkeypatch):
    # refused below what is needed; that this is enough is test_scan_paths_gpu.py's
    for name in ("GDN_IMPL", "GDN_SCAN_SPLIT"):
        monkeypatch.delenv(name, raising=False)
    for dtype in (0, 1):
        p = ctypes.byref(B.gdn_scan_problem(1, 700, 1, 2, 128, 64, 0, None, dtype, 0, 1, 128, 128, 128, 2))
        full, kept = L.gdn_scan_bwd_workspace_size(p), L.gdn_scan_saved_size(p)
        a = [q(k) for k in range(8)]
        out = [q(20 + k) for k in range(8)]
        for saved, need in ((q(10), full - kept), (None, full)):
            assert L.gdn_scan_bwd(p, *a, saved, q(11), q(12), *out, q(40), need - 1, None) == B.GDN_ERR_WORKSPACE


@pytest.mark.parametrize("seqs", [(1 << 30) + 1, (1 << 31) - 1])
def test_more_sequences_than_counts_hold(L, seqs):
    # slots (tokens / length + sequences) stay in 32 bits; refused before anything is read
    a = [q(k) for k in range(30)]
    p = ctypes.byref(B.gdn_conv_problem(1, 1 << 30, 64, 4, seqs, 1 << 20, 1, 1, 64))
    assert L.gdn_conv_bwd_workspace_size(p) == 0 and L.gdn_conv_fwd(p, *a[:6], None) == INV
    p = ctypes.byref(B.gdn_scan_problem(1, 1 << 30, 1, 2, 128, 64, seqs, 1 << 20, 1, 0, 1, 128, 128, 128, 2))
    assert L.gdn_scan_fwd_workspace_size(p) == 0 and L.gdn_scan_step(p, *a[:10], None) == INV
