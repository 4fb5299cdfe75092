"""The scan's CUDA-core path for both types, judged by the stretches of tokens that it sums over; long
sequences; and calls in a row.

Tolerances as in test_scan_gpu.py: of the terms' mass, every fp32 operation in sequence, (T + 512 + 17 * 128)
2^-24, and a sum over T tokens T 2^-24 more. The CUDA-core kernels round nothing to bf16 but the results, for
bf16 tensors too, and start the sum behind the gates' gradients anew every 16 tokens: the masses are those of
16 tokens."""
import pytest
import torch

import layer_ref as R
import test_scan_gpu as S

pytestmark = pytest.mark.gpu
DT = S.DT


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_rule_b200 import build
    build.build()
    import gated_deltanet_chunked_rule_b200 as g
    return g


def verify(v, lens, softplus, got):
    ref, mass = S.reference(v, lens, softplus, keep=16)
    base = (max(lens, default=0) + 512 + 17 * 128) * 2.0 ** -24
    for k, t in got.items():
        if t is not None:
            R.close(k, t.reshape(ref[k].shape), ref[k], mass[k], base + (sum(lens) * 2.0 ** -24 if k in ("dA", "dD", "ddt_bias") else 0))


FORMS = [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16")]


@pytest.mark.parametrize("dtype,dt_dtype", FORMS)
@pytest.mark.parametrize("K,P", [(64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("lens", [[1], [16, 17], [0, 5, 0, 130, 1, 0], [300], [700]])
def test_on_cuda_cores(gdn, monkeypatch, dtype, dt_dtype, K, P, lens):
    monkeypatch.setenv("GDN_IMPL", "simt")
    v = S.make(lens, 4, 2, K, P, DT[dtype], DT[dt_dtype], seed=K + sum(lens))
    got = S.train(gdn, v)
    verify(v, lens, True, got)
    again = S.train(gdn, v, save=False)
    for k in got:
        assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("dtype,dt_dtype", FORMS)
@pytest.mark.parametrize("form", ["bare", "D", "bias", "h0", "linear"])
def test_forms_on_cuda_cores(gdn, monkeypatch, dtype, dt_dtype, form):
    monkeypatch.setenv("GDN_IMPL", "simt")
    v = S.make([200, 70], 2, 1, 128, 64, DT[dtype], DT[dt_dtype], 7, D=form == "D", bias=form in ("bias", "linear"), h0=form == "h0",
               slices=True)
    if form == "linear":
        v["dt"] = (v["dt"] * 0.05).to(v["dt"].dtype)
        v["dt_bias"] = v["dt_bias"].abs() * 0 + 0.3
    verify(v, [200, 70], form != "linear", S.train(gdn, v, form != "linear"))


def test_kept_states_are_those_of_the_path(gdn, monkeypatch):
    # what one path kept is nothing to the other: refused where too short, recomputed where not needed
    v = S.make([150], 2, 1, 64, 64, torch.bfloat16, seed=3)
    a, rest = (*S.args(v), True), (v["dy"], v["dht"], v["h0"], v["cu"])
    _, _, tc = gdn.chunk_selective_scan_fwd(*a, v["h0"], True, v["cu"], save_for_backward=True)
    monkeypatch.setenv("GDN_IMPL", "simt")
    _, _, simt = gdn.chunk_selective_scan_fwd(*a, v["h0"], True, v["cu"], save_for_backward=True)
    assert simt.numel() == 0
    for p, q in zip(gdn.chunk_selective_scan_bwd(*a, tc, *rest), gdn.chunk_selective_scan_bwd(*a, simt, *rest)):
        assert torch.equal(p, q)
    monkeypatch.delenv("GDN_IMPL")
    with pytest.raises(ValueError, match="saved holds"):
        gdn.chunk_selective_scan_bwd(*a, simt, *rest)


@pytest.mark.parametrize("T", [0, 150, 1400])
def test_workspace_with_kept_states(gdn, T):
    # with what the forward kept, the backward's workspace has no room for it; the bytes behind stay as they were
    from gated_deltanet_chunked_rule_b200 import _binding as B
    from gated_deltanet_chunked_rule_b200 import layer_ops as ops
    v = S.make([T], 2, 1, 128, 64, torch.bfloat16, seed=T)
    want = S.train(gdn, v)
    _, _, saved = gdn.chunk_selective_scan_fwd(*S.args(v), True, v["h0"], True, v["cu"], save_for_backward=True)
    s = ops._Scan(*S.args(v), True, v["h0"], v["cu"])
    P = ops.byref(s.P)
    n = B.lib().gdn_scan_bwd_workspace_size(P) - B.lib().gdn_scan_saved_size(P)
    ws = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0")
    out = [torch.empty_like(want[k]) for k in names]
    ops._call(s.dev, "gdn_scan_bwd", *s.inputs(), saved.data_ptr(), v["dy"].data_ptr(), v["dht"].data_ptr(),
              *(t.data_ptr() for t in out), ws.data_ptr(), n)
    torch.cuda.synchronize()
    assert gdn.device_status() == 0 and (ws[n:] == 77).all()
    for k, t in zip(names, out):
        assert torch.equal(t, want[k]), k


@pytest.mark.parametrize("H,G,K,P,lens", [(4, 1, 128, 64, [128]), (8, 2, 64, 64, [128, 100]), (6, 2, 128, 128, [128]), (1, 1, 128, 64, [127, 1])])
def test_shared_gradients_round_once(gdn, H, G, K, P, lens):
    """dB and dC of sequences within a chunk, without states before or gradients behind: one product with the summed
    masked scores, which it takes in two bf16 parts (2^-16), in fp32 otherwise: 2^-16 and sqrt(T + 512 + 17 * 128) 2^-24,
    independent roundings, against 2^-8 / sqrt(3) of the result's own. So the error's norm is that of rounding the
    64-bit result, up to a hundredth, and 5 / sqrt(n) for its scatter over n values."""
    v = S.make(lens, H, G, K, P, torch.bfloat16, torch.float32, seed=H + K, h0=False, slow=True)
    v["dht"].zero_()
    got = S.train(gdn, v)
    ref, _ = S.reference(v, lens, True)
    for k in ("dB", "dC"):
        want = ref[k].reshape(got[k].shape)
        mine, best = ((t.cpu().double() - want).norm() / want.norm() for t in (got[k], want.to(torch.bfloat16)))
        print(k, f"{mine:.2e} of {best:.2e}")
        assert mine <= best * (1.01 + 5 / want.numel() ** 0.5), k


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("A,small", [(-1e6, 1e-6), (-3e4, 1e-5), (float("-inf"), 0.02)])
def test_tokens_that_clear_the_state(gdn, dtype, A, small):
    # one step in nine decays by e^A (to 0), the others slowly: what comes behind it in its block is as exact as
    # elsewhere. The clearing steps alone where A is infinite (0 times it is no number)
    v = S.make([200, 40], 2, 1, 128, 64, DT[dtype], torch.float32, seed=13, bias=False)
    g = torch.Generator().manual_seed(14)
    v["dt"] = (small * (0.5 + torch.rand(v["dt"].shape, generator=g))).cuda()
    v["dt"][:, 4::9] = 1.0
    v["A"].fill_(A)
    if A == float("-inf"):
        y, fin, _ = gdn.chunk_selective_scan_fwd(*S.args(v), False, v["h0"], True, v["cu"])
        S.verify(v, [200, 40], False, {"y": y, "final": fin})
    else:
        S.verify(v, [200, 40], False, S.train(gdn, v, False))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.float32).min])
def test_tokens_masked_by_their_step(gdn, dtype, low):
    # a step of the lowest value is one of 0: the token leaves the state as it is and gets no gradient of its step
    v = S.make([150, 70], 2, 1, 128, 64, DT[dtype], torch.float32, seed=15)
    off = torch.zeros(220, dtype=torch.bool)
    off[[0, 3, 31, 32, 127, 128, 149, 150, 219]] = True
    w = dict(v, dt=v["dt"].clone())
    w["dt"][:, off] = low
    got = S.train(gdn, w)
    assert not got["ddt"][:, off].any()
    w["dt"] = w["dt"].clamp(min=-200)  # the reference's 64 bits know no lowest value of 32: softplus is 0 here too
    S.verify(w, [150, 70], True, got)


@pytest.mark.parametrize("dtype,impl", [("fp32", ""), ("bf16", "simt")])
@pytest.mark.parametrize("lens", [[300], [7] * 20, [16, 17, 1, 120]])
def test_gate_gradients_on_cuda_cores_add_up(gdn, monkeypatch, dtype, impl, lens):
    """Norms over 32 heads of dA and ddt_bias, sums over the tokens of terms of either sign, as large as the root of
    the sum of their squares. A term is off by at most about 6 2^-24: the products over K and P in up to 32 roundings in
    sequence, independent ones (sqrt(32 / 3)), as many again for the states' own over the tokens that they remember, the
    decays' exponentials; the 16 tokens of a tile may share them (sqrt(16)). 24 2^-24; bf16 results' inputs are exact."""
    if impl:
        monkeypatch.setenv("GDN_IMPL", impl)
    v = S.make(lens, 32, 4, 64, 64, DT[dtype], torch.float32, seed=len(lens))
    g = torch.Generator().manual_seed(5)
    v["A"] = -(1 + 15 * torch.rand(32, generator=g)).cuda()
    v["dt_bias"] = (-7 + 5 * torch.rand(32, generator=g)).cuda()
    v["h0"], v["dht"] = 0.1 * v["h0"], 0.1 * v["dht"]
    got = S.train(gdn, v)
    ref, _ = S.reference(v, lens, True)
    for k in ("dA", "ddt_bias"):
        off = ((got[k].cpu().double() - ref[k]).norm() / ref[k].norm()).item()
        print(k, f"{off:.2e}")
        assert off <= 24 * 2.0 ** -24, k


@pytest.mark.parametrize("K,P", [(128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("lens", [[2] * 12, [40, 60], [300, 128], [1500]])
def test_gate_gradients_on_tensor_cores_add_up(gdn, K, P, lens):
    """The same of the tensor-core kernels, between states as large as the tokens' own: their products are exact ones of
    bf16 values and of states in 24 bits, summed in fp32. 24 2^-24 as above, and three decays by exponentials of 2^-22
    each in a term."""
    v = S.make(lens, 32, 4, K, P, torch.bfloat16, torch.float32, seed=len(lens) + K)
    g = torch.Generator().manual_seed(5)
    v["A"] = -(1 + 15 * torch.rand(32, generator=g)).cuda()
    v["dt_bias"] = (-7 + 5 * torch.rand(32, generator=g)).cuda()
    ref, _ = S.reference(v, lens, True)
    for save in (True, False):
        got = S.train(gdn, v, save=save)
        for k in ("dA", "ddt_bias"):
            off = ((got[k].cpu().double() - ref[k]).norm() / ref[k].norm()).item()
            print(k, f"{off:.2e}")
            assert off <= (24 + 12) * 2.0 ** -24, k


def chunked(v, lens):
    """The scan in 64 bits on the GPU in chunks of 64 tokens, the state carried from chunk to chunk."""
    x, dt, A, B, C, D, bias = (t.double() if t is not None else None for t in S.args(v))
    H, G = x.shape[2], B.shape[2]
    h = v["h0"].double()[0]
    raw = dt[0] + bias
    delta = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    mask = torch.ones(64, 64, dtype=torch.bool, device="cuda").tril()
    ys = []
    for t in range(0, lens[0], 64):
        xs, dl = x[0, t:t + 64], delta[t:t + 64]
        bs, cs = (w[0, t:t + 64].repeat_interleave(H // G, 1) for w in (B, C))
        n = xs.shape[0]
        gam = torch.cumsum(dl * A, 0).t()
        L = torch.exp((gam[:, :, None] - gam[:, None]).masked_fill(~mask[:n, :n], -float("inf")))
        w = xs * dl[..., None]
        y = torch.einsum("hqs,shp->qhp", torch.einsum("qhk,shk->hqs", cs, bs) * L, w)
        y = y + torch.einsum("qhk,hkp->qhp", cs, h) * torch.exp(gam).t()[..., None] + D[:, None] * xs
        h = torch.exp(gam[:, -1])[:, None, None] * h + torch.einsum("shk,shp->hkp", bs * torch.exp(gam[:, -1:] - gam).t()[..., None], w)
        ys.append(y)
    return torch.cat(ys)[None], h[None]


@pytest.mark.parametrize("dtype,T,H,split", [("bf16", 8229, 3, ""), ("bf16", 8229, 3, "segments"), ("bf16", 65536, 8, ""),
                                             ("fp32", 8229, 2, "")])
def test_long_sequences(gdn, monkeypatch, dtype, T, H, split):
    """Of norms. bf16 results: half a step, 2^-8, for the rounding of the result and of one operand in each of its
    two terms. fp32 results: the operations in sequence, whose roundings are independent, sqrt(T + 512 + 17 * 128)
    2^-24, and 2^-16 for operands cut into bf16 parts (two at least); the gates' gradients pass through four such results
    (kept states, exit gradients, their product, the sum)."""
    if split:
        monkeypatch.setenv("GDN_SCAN_SPLIT", split)
    v = S.make([T], H, 1, 128, 64, DT[dtype], torch.float32, seed=T + H, slow=True)
    got = S.train(gdn, v)
    names = ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")
    leaves = {k: v[k].double().requires_grad_() for k in names}
    y, fin = chunked({**v, **leaves}, [T])
    want = dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"),
                    torch.autograd.grad([y, fin], [leaves[k] for k in names], [v["dy"].double(), v["dht"].double()])))
    want |= {"y": y.detach(), "final": fin.detach()}
    fp32 = (T + 512 + 17 * 128) ** 0.5 * 2.0 ** -24 + (2.0 ** -16 if dtype == "bf16" else 0)
    for k, t in got.items():
        tol = 3 * 2.0 ** -8 if t.dtype == torch.bfloat16 else 4 * fp32
        off = ((t.double() - want[k]).norm() / want[k].norm()).item()
        print(k, f"{off:.2e} of {tol:.2e}")
        assert off <= tol, (k, off, tol)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("H,lens", [(2, [2100]), (2, [700, 0, 1400]), (96, [130])])
def test_backward_calls_in_a_row(gdn, dtype, H, lens):
    # forward and backward after one another with no wait between, on the same memory
    both = [S.make(lens, H, 1, 64, 64, DT[dtype], seed=s) for s in (41, 42)]

    def call(v, save):
        _, _, saved = gdn.chunk_selective_scan_fwd(*S.args(v), True, v["h0"], True, v["cu"], save_for_backward=save)
        return gdn.chunk_selective_scan_bwd(*S.args(v), True, saved, v["dy"], v["dht"], v["h0"], v["cu"])

    alone = []
    for v in both:
        alone.append(call(v, True))
        torch.cuda.synchronize()
    got = [call(both[i % 2], i % 3 > 0) for i in range(12)]
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    for i, g in enumerate(got):
        for p, q in zip(g, alone[i % 2]):
            assert torch.equal(p, q), i
