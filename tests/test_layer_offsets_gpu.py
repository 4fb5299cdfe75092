"""Packed offsets that do not fit their tokens, in the gradients: nothing outside the tensors is read, the
status word says so, and the next call is right."""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
BAD = 6  # GDN_ERR_DEVICE_ARG


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_rule_b200 import build
    build.build()
    import gated_deltanet_chunked_rule_b200 as g
    return g


def offsets(*cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("C", [40, 37])
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("T,cu", [(71, (0, 30, 60)), (71, (0, 0, 0)), (71, (0, 70)), (4096, (0, 30, 60)), (4096, (0, 0))])
def test_convolution_padded_at_its_end(gdn, dtype, C, W, T, cu):
    # the last offset below the token count; behind dfinal's rows lie NaN
    g = torch.Generator().manual_seed(T + W)

    def r(*s):
        return torch.randn(s, generator=g).to(DT[dtype]).cuda()

    N = len(cu) - 1
    wide = torch.full((N + T, W - 1, C), float("nan"), dtype=DT[dtype], device="cuda")
    wide[:N] = r(N, W - 1, C)
    x, weight, bias, state, dy = r(1, T, C), r(C, W), r(C), r(N, W - 1, C), r(1, T, C)
    args = (x, weight, bias, dy, wide[:N], "silu", state)
    dx, dw, db, ds = gdn.causal_conv1d_bwd(*args, offsets(*cu))
    assert gdn.device_status() == BAD
    for t in (dx, dw, db, ds):
        assert torch.isfinite(t).all()
    # and with an end that fits
    lens = [b - a for a, b in zip(cu, cu[1:-1] + (T,))]
    dx, dw, db, ds = gdn.causal_conv1d_bwd(*args, offsets(*cu[:-1], T))
    assert gdn.device_status() == 0
    if T > 100:
        return
    a = (x[0], weight, bias, state, True, lens, dy[0], wide[:N])
    ref, mass = R.conv(*a), R.conv(*a, mass=True)
    # as in test_conv_gpu.py: the fp32 operations in sequence, and the fast exponential's error
    base = 2.0 ** -18 if dtype == "bf16" else 0
    for name, got, ops in (("dx", dx[0], 16), ("dweight", dw, T), ("dbias", db, T), ("dstate", ds, 16)):
        R.close(name, got, ref[name], mass[name], base + (16 + ops) * 2.0 ** -24)


def scan_inputs(T, N, dtype, seed):
    g = torch.Generator().manual_seed(seed)

    def r(*s, dt=dtype):
        return torch.randn(s, generator=g).to(dt).cuda()

    f = torch.float32
    a = (r(1, T, 2, 64), r(1, T, 2), -r(2, dt=f).abs() - 0.1, r(1, T, 1, 128), r(1, T, 1, 128), r(2, dt=f), r(2, dt=f), True)
    return a, r(N, 2, 128, 64, dt=f), r(1, T, 2, 64), r(N, 2, 128, 64, dt=f)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("T,good", [(171, (0, 100, 171)), (1400, (0, 100, 1400))])
def test_scan_gradients_report_offsets(gdn, dtype, keep, T, good):
    # each call by itself: a forward on good offsets says nothing for the backward, whose offsets went bad
    # after it (whole sequences, and sequences in segments)
    a, h0, dy, dht = scan_inputs(T, 2, DT[dtype], T)
    _, _, saved = gdn.chunk_selective_scan_fwd(*a, h0, True, offsets(*good), save_for_backward=keep)
    want = gdn.chunk_selective_scan_bwd(*a, saved, dy, dht, h0, offsets(*good))
    assert gdn.device_status() == 0
    for cu in ((0, T + 9, T), (0, 100, T - 11), (0, -5, T), (3, 100, T)):
        gdn.chunk_selective_scan_bwd(*a, saved, dy, dht, h0, offsets(*cu))
        assert gdn.device_status() == BAD, cu
        gdn.chunk_selective_scan_fwd(*a, h0, True, offsets(*cu))
        assert gdn.device_status() == BAD, cu
    again = gdn.chunk_selective_scan_bwd(*a, saved, dy, dht, h0, offsets(*good))
    assert gdn.device_status() == 0
    for p, q in zip(again, want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_no_tokens_report_offsets(gdn, dtype):
    x, w = torch.empty(1, 0, 40, dtype=DT[dtype], device="cuda"), torch.zeros(40, 4, dtype=DT[dtype], device="cuda")
    a, h0, dy, dht = scan_inputs(0, 2, DT[dtype], 1)
    for cu, status in ((offsets(0, 5, 0), BAD), (offsets(0, 0, 0), 0)):
        for final in (True, False):
            gdn.causal_conv1d_fwd(x, w, None, None, None, final, cu)
            assert gdn.device_status() == status
        gdn.causal_conv1d_bwd(x, w, None, x, None, None, None, cu)
        assert gdn.device_status() == status
        _, _, saved = gdn.chunk_selective_scan_fwd(*a, h0, True, cu, save_for_backward=True)
        assert gdn.device_status() == status
        for kept in (saved, None):
            gdn.chunk_selective_scan_bwd(*a, kept, dy, dht, h0, cu)
            assert gdn.device_status() == status
