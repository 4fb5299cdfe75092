"""The operators around the gated delta rule, without a GPU: the C entry points refuse bad
problems and pointers before anything is enqueued, the binding refuses CPU tensors and finds
token strides and packed batches."""
import ctypes

import pytest
import torch

import gated_deltanet_chunked_rule_b200 as gdn
from gated_deltanet_chunked_rule_b200 import _binding as B
from gated_deltanet_chunked_rule_b200 import layer_ops as ops

d = ctypes.c_void_p(1 << 20)
bad = ctypes.c_void_p((1 << 20) + 2)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from gated_deltanet_chunked_rule_b200 import build
    build.build()
    return B.lib()


def conv(**kw):
    f = dict(B=1, T=100, C=64, W=4, num_seqs=0, cu_seqlens=None, dtype=1, silu=1, x_stride=64)
    f.update(kw)
    return B.gdn_conv_problem(*f.values())


def scan(**kw):
    f = dict(B=1, T=100, Hq=1, Hv=2, K=128, V=64, num_seqs=0, cu_seqlens=None, dtype=1, dt_dtype=0, dt_softplus=1,
             x_stride=128, b_stride=128, c_stride=128, dt_stride=2)
    f.update(kw)
    return B.gdn_scan_problem(*f.values())


def norm(**kw):
    f = dict(rows=10, D=64, dtype=1, weight_dtype=0, center=1, gate_first=0, eps=1e-5)
    f.update(kw)
    return B.gdn_norm_problem(*f.values())


INV, UNS, WS = B.GDN_ERR_INVALID_ARG, B.GDN_ERR_UNSUPPORTED, B.GDN_ERR_WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INV), (dict(T=-1), INV), (dict(C=0), INV), (dict(W=0), INV), (dict(W=1), UNS), (dict(W=5), UNS),
    (dict(dtype=2), UNS), (dict(x_stride=63), INV), (dict(num_seqs=-1), INV), (dict(num_seqs=2), INV),
    (dict(num_seqs=2, cu_seqlens=1 << 20, B=2), INV), (dict(B=1 << 16, T=1 << 16), INV), (dict(C=1 << 21, x_stride=1 << 21), UNS),
])
def test_conv_problems_refused(L, kw, code):
    p = ctypes.byref(conv(**kw))
    assert L.gdn_conv_bwd_workspace_size(p) == 0
    assert L.gdn_conv_fwd(p, d, d, None, None, d, None, None) == code
    assert L.gdn_conv_bwd(p, d, d, None, None, d, None, d, d, None, None, d, BIG, None) == code
    assert L.gdn_conv_update(p, d, d, None, d, d, None) == code


def test_conv_pointers_refused(L):
    p = ctypes.byref(conv())
    assert L.gdn_conv_fwd(None, d, d, None, None, d, None, None) == INV
    assert L.gdn_conv_fwd(p, None, d, None, None, d, None, None) == INV
    assert L.gdn_conv_fwd(p, d, None, None, None, d, None, None) == INV
    assert L.gdn_conv_fwd(p, bad, d, None, None, d, None, None) == INV
    assert L.gdn_conv_fwd(p, d, d, None, d, d, d, None) == INV  # final over initial
    need = L.gdn_conv_bwd_workspace_size(p)
    assert need >= 5 * 64 * 4
    assert L.gdn_conv_bwd(p, d, d, None, None, d, None, d, d, None, None, d, 5 * 64 * 4 - 1, None) == WS
    assert L.gdn_conv_bwd(p, d, d, None, None, d, None, d, d, None, None, ctypes.c_void_p((1 << 20) + 16), need, None) == WS
    assert L.gdn_conv_bwd(p, d, d, None, None, d, None, None, d, None, None, d, need, None) == INV
    cu = ctypes.byref(conv(num_seqs=2, cu_seqlens=1 << 20))
    assert L.gdn_conv_update(cu, d, d, None, d, d, None) == INV
    assert L.gdn_conv_update(p, d, d, None, None, d, None) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), INV), (dict(T=-1), INV), (dict(Hq=0), INV), (dict(Hv=3, Hq=2), INV), (dict(K=96), UNS), (dict(V=32), UNS),
    (dict(dtype=3), UNS), (dict(dt_dtype=5), UNS), (dict(dtype=0, dt_dtype=1, x_stride=128), UNS), (dict(x_stride=120), INV),
    (dict(x_stride=132), INV), (dict(b_stride=64), INV), (dict(c_stride=129), INV), (dict(dt_stride=1), INV),
    (dict(num_seqs=1), INV), (dict(Hv=2048, x_stride=2048 * 64, dt_stride=2048), UNS),
])
def test_scan_problems_refused(L, kw, code):
    p = ctypes.byref(scan(**kw))
    assert L.gdn_scan_bwd_workspace_size(p) == 0
    assert L.gdn_scan_fwd_workspace_size(p) == 0 and L.gdn_scan_saved_size(p) == 0
    assert L.gdn_scan_fwd(p, d, d, d, d, d, None, None, None, d, None, None, d, BIG, None) == code
    assert L.gdn_scan_step(p, d, d, d, d, d, None, None, None, d, None, None) == code
    assert L.gdn_scan_bwd(p, d, d, d, d, d, None, None, None, None, d, None, d, d, d, d, d, None, None, None, d, BIG, None) == code


@pytest.mark.parametrize("dtype,K", [(1, 128), (0, 128), (1, 64)])
def test_scan_pointers_refused(L, dtype, K):
    pr = scan(dtype=dtype, K=K)
    p = ctypes.byref(pr)
    assert L.gdn_scan_fwd(None, d, d, d, d, d, None, None, None, d, None, None, d, BIG, None) == INV
    ok = [d, d, d, d, d, None, None, None]
    for i in range(5):
        a = list(ok)
        a[i] = None
        assert L.gdn_scan_fwd(p, *a, d, None, None, d, BIG, None) == INV
        if i != 1:  # dt needs its own alignment only
            a[i] = bad
            assert L.gdn_scan_fwd(p, *a, d, None, None, d, BIG, None) == INV
            assert L.gdn_scan_step(p, *a, d, None, None) == INV
    assert L.gdn_scan_fwd(p, *ok, None, None, None, d, BIG, None) == INV
    assert L.gdn_scan_fwd(p, *ok, d, None, ctypes.c_void_p((1 << 20) + 16), d, BIG, None) == INV  # saved off 256
    n = L.gdn_scan_fwd_workspace_size(p)
    if n:
        assert L.gdn_scan_fwd(p, *ok, d, None, None, d, n - 1, None) == WS
        assert L.gdn_scan_fwd(p, *ok, d, None, None, None, n, None) == WS
    n = L.gdn_scan_bwd_workspace_size(p)
    assert n > 0
    out = [d, d, d, d, d, None, None, None]
    assert L.gdn_scan_bwd(p, *ok, None, d, None, *out, d, n - 1, None) == WS
    for i in range(5):
        o = list(out)
        o[i] = None
        assert L.gdn_scan_bwd(p, *ok, None, d, None, *o, d, n, None) == INV
    assert L.gdn_scan_bwd(p, *ok, None, None, None, *out, d, n, None) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INV), (dict(D=0), INV), (dict(dtype=9), UNS), (dict(weight_dtype=9), UNS), (dict(eps=-1.0), INV),
    (dict(eps=float("nan")), INV), (dict(eps=float("inf")), INV), (dict(dtype=0, weight_dtype=1), UNS), (dict(D=1 << 21), UNS),
])
def test_norm_problems_refused(L, kw, code):
    p = ctypes.byref(norm(**kw))
    assert L.gdn_norm_bwd_workspace_size(p) == 0
    assert L.gdn_norm_fwd(p, d, d, None, None, d, None, None) == code
    assert L.gdn_norm_bwd(p, d, d, None, None, d, d, d, d, None, None, d, BIG, None) == code


def test_norm_pointers_refused(L):
    p = ctypes.byref(norm())
    assert L.gdn_norm_fwd(None, d, d, None, None, d, None, None) == INV
    assert L.gdn_norm_fwd(p, bad, d, None, None, d, None, None) == INV
    assert L.gdn_norm_fwd(p, d, None, None, None, d, None, None) == INV
    n = L.gdn_norm_bwd_workspace_size(p)
    assert n > 0
    assert L.gdn_norm_bwd(p, d, d, None, None, d, d, d, d, None, None, d, 16, None) == WS
    assert L.gdn_norm_bwd(p, d, d, None, d, d, d, d, d, None, None, d, n, None) == INV  # a gate without dgate
    assert L.gdn_norm_bwd(p, d, d, None, None, d, None, d, d, None, None, d, n, None) == INV


def test_cpu_tensors_refused():
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.causal_conv1d(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.causal_conv1d_update(x, torch.zeros(1, 3, 8), torch.zeros(8, 4))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.layer_norm(x, torch.ones(8))
    s = torch.zeros(1, 4, 2, 64)
    for f in (gdn.chunk_selective_scan, gdn.recurrent_selective_scan):
        with pytest.raises(ValueError, match="CUDA"):
            f(s, torch.zeros(1, 4, 2), torch.zeros(2), s, s)


def test_token_strides():
    w = torch.zeros(2, 5, 3, 8)
    t, st = ops._tokens(w, 24)
    assert t is w and st == 24
    wide = torch.zeros(2, 5, 40)
    t, st = ops._tokens(wide[..., 8:32].unflatten(-1, (3, 8)), 24)
    assert st == 40 and t.data_ptr() == wide.data_ptr() + 32
    for view in (wide[..., 1:25], wide[:, ::2, :24].expand(2, 3, 24)[:, :, :24], wide[:, :, ::2][..., :20], wide.transpose(0, 1)):
        t, st = ops._tokens(view, view.shape[2])
        if t.data_ptr() != view.data_ptr():
            assert st == view.shape[2] and t.is_contiguous() and t.data_ptr() % 16 == 0
        else:  # every token where the stride says
            B, T = view.shape[:2]
            for b in range(B):
                for s in range(T):
                    assert view[b, s].data_ptr() == t.data_ptr() + 4 * (b * T + s) * st
    one = torch.zeros(1, 1, 24).expand(1, 7, 24)  # a token stride of 0
    t, st = ops._tokens(one, 24)
    assert st == 24 and t.is_contiguous()
    odd = torch.zeros(1, 5, 25)[..., :24]
    assert ops._tokens(odd, 24, 1)[1] == 25 and ops._tokens(odd, 24, 4)[1] == 24
    assert ops._tokens(torch.zeros(3, 1, 50)[..., :24], 24)[1] == 50
    assert ops._tokens(torch.zeros(0, 4, 24), 24)[1] == 24


def test_packed_offsets():
    cpu = torch.device("cpu")
    assert ops._packed(None, 3, cpu) == (None, 0, 3)
    cu, ns, n = ops._packed(torch.tensor([0, 2, 5]), 1, cpu)
    assert cu.dtype == torch.int32 and ns == n == 2
    for c, b in ((torch.tensor([0]), 1), (torch.tensor([[0, 1]]), 1), (torch.tensor([0.0, 1.0]), 1), (torch.tensor([0, 1]), 2)):
        with pytest.raises(ValueError):
            ops._packed(c, b, cpu)


def test_outputs_over_inputs_refused(L):
    """Each output given one of the inputs' buffers, everything else distinct."""
    def q(i):
        return ctypes.c_void_p((1 << 20) + (i << 12))

    ws = q(40)
    p = ctypes.byref(conv())
    for out in range(2):
        for i in range(4):
            o = [q(10), q(11)]
            o[out] = q(i)
            assert L.gdn_conv_fwd(p, q(0), q(1), q(2), q(3), *o, None) == INV
    for out in range(4):
        for i in range(6):
            o = [q(10 + k) for k in range(4)]
            o[out] = q(i)
            assert L.gdn_conv_bwd(p, *(q(k) for k in range(6)), *o, ws, BIG, None) == INV
    p = ctypes.byref(scan())
    for out in range(2):
        for i in range(8):
            o = [q(10), q(11)]
            o[out] = q(i)
            assert L.gdn_scan_fwd(p, *(q(k) for k in range(8)), *o, None, ws, BIG, None) == INV
    for out in range(8):
        for i in range(11):
            o = [q(20 + k) for k in range(8)]
            o[out] = q(i)
            assert L.gdn_scan_bwd(p, *(q(k) for k in range(11)), *o, ws, BIG, None) == INV
    p = ctypes.byref(norm())
    for out in range(2):
        for i in range(4):
            o = [q(10), q(11)]
            o[out] = q(i)
            assert L.gdn_norm_fwd(p, *(q(k) for k in range(4)), *o, None) == INV
    for out in range(4):
        for i in range(6):
            o = [q(20 + k) for k in range(4)]
            o[out] = q(i)
            assert L.gdn_norm_bwd(p, *(q(k) for k in range(6)), *o, ws, BIG, None) == INV
