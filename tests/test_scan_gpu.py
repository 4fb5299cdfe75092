"""Selective state space scan on the GPU (prompts, their gradients, the token step) against
its plain 64-bit form, element by element.

Tolerances (layer_ref.close): the output's rounding, and of the terms' mass
  - every fp32 operation in sequence: a state takes one per token (T), a product over K or P
    or a group's heads another (256 at most here), exponentials and softplus a few: (T + 512)
    2^-24; a decay is the exponential of a running sum of up to 128 logs, of magnitude up to
    the largest sum M that still matters (e^-M below 2^-24: M = 17): 17 * 128 * 2^-24;
  - where bf16 tensor-core products are formed, 2^-8 for the one operand of a product that is
    rounded to bf16 on the way to a bf16 result (decay-masked scores, kept states, scaled
    rows), and 2^-16 for the two-part operands of fp32 results."""
import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_rule_b200 import build
    build.build()
    import gated_deltanet_chunked_rule_b200 as g
    return g


def make(lens, H=2, G=1, K=64, P=64, dtype=torch.float32, dt_dtype=None, seed=0, packed=True, D=True, bias=True, h0=True,
         slices=False, slow=False):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    B = 1 if packed else N

    def r(*s, std=1.0, dt=dtype):
        return (torch.randn(s, generator=g) * std).to(dt).cuda()

    n = T // B
    xbc = r(B, n, H * P + 2 * G * K + (16 if slices else 0))
    x, b, c = xbc[..., :H * P], xbc[..., H * P:H * P + G * K], xbc[..., H * P + G * K:H * P + 2 * G * K]
    x, b, c = x.unflatten(-1, (H, P)), b.unflatten(-1, (G, K)), c.unflatten(-1, (G, K))
    if not slices:
        x, b, c = x.contiguous(), b.contiguous(), c.contiguous()
    f = torch.float32
    A = -(torch.rand(H, generator=g) * (0.05 if slow else 4) + (0.001 if slow else 0.2)).cuda()
    return dict(x=x, dt=r(B, n, H, dt=dt_dtype or dtype), A=A, B=b, C=c, D=r(H, dt=f) if D else None,
                dt_bias=r(H, std=0.5, dt=f) - 1 if bias else None, h0=r(N, H, K, P, dt=f) if h0 else None,
                dy=r(B, n, H, P), dht=r(N, H, K, P, dt=f),
                cu=torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() if packed else None)


def args(v):
    return v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["dt_bias"]


def reference(v, lens, softplus, **kw):
    x, dt, B, C, dy = (v[k].flatten(0, 1) for k in ("x", "dt", "B", "C", "dy"))
    both = []
    for mass in (False, True):
        both.append(R.scan(x, dt, v["A"], B, C, v["D"], v["dt_bias"], softplus, v["h0"], lens, dy, v["dht"], mass=mass, **kw))
    return both


def rels(v, lens):
    base = (max(lens, default=0) + 512 + 17 * 128) * 2.0 ** -24
    if v["x"].dtype == torch.float32:
        return base, base
    return base + 2.0 ** -8 + 2.0 ** -16, base + 2.0 ** -16  # of bf16 and of fp32 results


def verify(v, lens, softplus, got, label=""):
    ref, mass = reference(v, lens, softplus)
    low, high = rels(v, lens)
    T = sum(lens)
    worst = {}
    for k, t in got.items():
        if t is None:
            continue
        want = ref[k]
        t = t.reshape(want.shape)
        e = low if t.dtype == torch.bfloat16 else high
        if k in ("dA", "dD", "ddt_bias"):
            e += T * 2.0 ** -24
        worst[k] = R.close(label + k, t, want, mass[k], e)
    print(label, {k: f"{w:.2g}" for k, w in worst.items()})


def train(gdn, v, softplus=True, save=True, **kw):
    y, fin, saved = gdn.chunk_selective_scan_fwd(*args(v), softplus, v["h0"], True, v["cu"], save_for_backward=save)
    g = gdn.chunk_selective_scan_bwd(*args(v), softplus, saved, v["dy"], v["dht"], v["h0"], v["cu"])
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    return dict(zip(("y", "final", "dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"), (y, fin, *g)))


LENS = [[1], [2], [63], [64], [65], [127], [128], [129], [300], [0, 5, 0, 130, 1, 0], [17, 128, 64, 90], [256, 128]]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("K,P", [(64, 64), (128, 64), (128, 128), (64, 128)])
@pytest.mark.parametrize("lens", LENS)
def test_packed_prompts_and_gradients(gdn, dtype, K, P, lens):
    v = make(lens, 2, 1, K, P, DT[dtype], seed=K + P + sum(lens))
    verify(v, lens, True, train(gdn, v))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (4, 2), (5, 5), (12, 2)])
def test_heads_and_groups(gdn, dtype, H, G):
    v = make([150, 40], H, G, 128, 64, DT[dtype], seed=H)
    verify(v, [150, 40], True, train(gdn, v))


@pytest.mark.parametrize("dtype,dt_dtype", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16")])
@pytest.mark.parametrize("form", ["bare", "D", "bias", "h0", "linear"])
def test_forms(gdn, dtype, dt_dtype, form):
    # each optional input by itself; delta without softplus (made positive by its bias)
    v = make([200, 70], 2, 1, 128, 64, DT[dtype], DT[dt_dtype], 7, D=form == "D", bias=form in ("bias", "linear"),
             h0=form == "h0")
    if form == "linear":
        v["dt"] = (v["dt"] * 0.05).to(v["dt"].dtype)
        v["dt_bias"] = v["dt_bias"].abs() * 0 + 0.3
    got = train(gdn, v, form != "linear")
    for k, there in (("dD", v["D"] is not None), ("ddt_bias", v["dt_bias"] is not None)):
        assert (got[k] is not None) == there
    verify(v, [200, 70], form != "linear", got)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("slow", [True, False])
def test_batch_of_slices_without_saved(gdn, dtype, slow):
    # rows of a batch, x, B, C slices of one tensor; states recomputed in the backward; decays
    # that keep the whole sequence, or forget it within tokens
    v = make([333] * 2, 4, 2, 128, 64, DT[dtype], seed=9, packed=False, slices=True, slow=slow)
    got = train(gdn, v, save=False)
    verify(v, [333] * 2, True, got)
    kept = train(gdn, v, save=True)
    for k in got:
        assert torch.equal(got[k], kept[k]), k


SEGMENTED = [([1100], False), ([1025, 1, 0, 70, 1300], True), ([640] * 2, False), ([1536], True)]


@pytest.mark.parametrize("lens,packed", SEGMENTED)
@pytest.mark.parametrize("K,P,H", [(128, 64, 1), (64, 128, 2)])
def test_sequences_cut_into_segments(gdn, monkeypatch, lens, packed, K, P, H):
    # few heads and many chunks: state passes over segments of a sequence; ends on and off the
    # segments' borders, beside short and empty sequences. bf16 in every way the segments are joined:
    # from the chunks' products, from the segments' ends in two passes (something kept), in one (nothing)
    for dtype in (torch.bfloat16, torch.float32):
        v = make(lens, H, 1, K, P, dtype, seed=21, packed=packed, slow=True)
        got = train(gdn, v)
        verify(v, lens, True, got)
        if dtype == torch.float32:
            continue
        once = gdn.chunk_selective_scan_fwd(*args(v), True, v["h0"], True, v["cu"])
        assert torch.equal(once[0], got["y"]) and torch.equal(once[1], got["final"])
        monkeypatch.setenv("GDN_SCAN_SPLIT", "segments")
        verify(v, lens, True, train(gdn, v), "two passes ")
        bare = train(gdn, v, save=False)
        verify(v, lens, True, bare, "one pass ")
        v["h0"] = None
        y, fin, _ = gdn.chunk_selective_scan_fwd(*args(v), True, None, True, v["cu"])
        verify(v, lens, True, {"y": y, "final": fin}, "one pass, no start ")
        monkeypatch.delenv("GDN_SCAN_SPLIT")


@pytest.mark.parametrize("H,G,P,lens", [(24, 1, 128, [300]), (40, 1, 64, [128, 200]), (48, 2, 128, [129]), (7, 1, 128, [256])])
def test_many_heads_of_one_group(gdn, H, G, P, lens):
    # long runs of heads in one block of the output and gradient kernels
    v = make(lens, H, G, 128, P, torch.bfloat16, seed=H)
    for _ in range(3):
        got = train(gdn, v)
    verify(v, lens, True, got)


def test_large_and_small_steps(gdn):
    # delta near 0 and above softplus's switch; decays that underflow to 0
    for dtype in (torch.float32, torch.bfloat16):
        v = make([140], 2, 1, 128, 64, dtype, torch.float32, seed=11)
        v["dt"][0, ::3] = -30
        v["dt"][0, 1::7] = 25
        v["dt"][0, 100] = 60
        verify(v, [140], True, train(gdn, v))


def test_only_final_state_gradient_and_only_outputs(gdn):
    for dtype in (torch.float32, torch.bfloat16):
        v = make([200], 2, 1, 128, 64, dtype, seed=12)
        a = gdn.chunk_selective_scan_bwd(*args(v), True, None, v["dy"], None, v["h0"], v["cu"])
        zero = dict(v, dht=torch.zeros_like(v["dht"]))
        b = gdn.chunk_selective_scan_bwd(*args(v), True, None, v["dy"], zero["dht"], v["h0"], v["cu"])
        for p, q in zip(a, b):
            assert torch.equal(p, q)
        w = dict(v, dy=torch.zeros_like(v["dy"]))
        verify(w, [200], True, train(gdn, w))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("K,P", [(64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [1, 2, 19])
def test_token_step(gdn, dtype, K, P, T):
    v = make([T] * 3, 4, 2, K, P, DT[dtype], torch.float32, seed=T, packed=False)
    y, fin = gdn.recurrent_selective_scan(*args(v), True, v["h0"])
    assert gdn.device_status() == 0
    verify(v, [T] * 3, True, {"y": y, "final": fin})
    state = v["h0"].clone()
    outs = []
    for t in range(T):  # one by one, in place
        one = [a[:, t:t + 1] if a is not None and a.dim() > 1 else a for a in args(v)]
        o, s = gdn.recurrent_selective_scan(*one, True, state, state)
        assert s is state
        outs.append(o)
    assert torch.equal(torch.cat(outs, 1), y) and torch.equal(state, fin)


def test_step_packed_and_empty(gdn):
    lens = [0, 1, 4, 0]
    v = make(lens, 2, 1, 128, 64, torch.bfloat16, seed=5)
    y, fin = gdn.recurrent_selective_scan(*args(v), True, v["h0"], None, v["cu"])
    verify(v, lens, True, {"y": y, "final": fin})
    assert torch.equal(fin[0], v["h0"][0]) and torch.equal(fin[3], v["h0"][3])
    v = make([0, 0], 2, 1, 128, 64, torch.bfloat16, seed=6)
    got = train(gdn, v)
    assert torch.equal(got["final"], v["h0"]) and torch.equal(got["dh0"], v["dht"])
    assert not got["dA"].any() and not got["dD"].any()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_prompt_then_steps(gdn, dtype):
    # a prompt's final state continued token by token equals the prompt over everything
    v = make([140] * 2, 2, 1, 128, 64, DT[dtype], seed=14, packed=False)
    cut = lambda a, b: [t[:, a:b] if t is not None and t.dim() > 1 else t for t in args(v)]  # noqa: E731
    y0, st, _ = gdn.chunk_selective_scan_fwd(*cut(0, 130), True, v["h0"])
    y1, fin = gdn.recurrent_selective_scan(*cut(130, 140), True, st, st)
    verify(v, [140] * 2, True, {"y": torch.cat([y0, y1], 1), "final": fin})


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_packed_sequences_do_not_touch(gdn, dtype):
    lens = [100, 60, 170]
    v = make(lens, 2, 1, 128, 64, DT[dtype], seed=15)
    clean = train(gdn, v)
    for bad in (float("nan"), float("inf")):
        w = {k: (t.clone() if t is not None else None) for k, t in v.items()}
        for k in ("x", "B", "C", "dy", "dt"):
            w[k][:, 100:160] = bad
        w["h0"][1], w["dht"][1] = bad, bad
        got = train(gdn, w)
        for k in ("y", "dx", "ddt", "dB", "dC"):
            assert torch.equal(got[k][:, :100], clean[k][:, :100]) and torch.equal(got[k][:, 160:], clean[k][:, 160:]), (k, bad)
        for k in ("final", "dh0"):
            assert torch.equal(got[k][0], clean[k][0]) and torch.equal(got[k][2], clean[k][2]), (k, bad)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_autograd_repeat_and_other_stream(gdn, dtype):
    v = make([150, 90], 4, 2, 128, 64, DT[dtype], seed=16)
    want = train(gdn, v)
    names = ("x", "dt", "A", "B", "C", "D", "dt_bias", "h0")
    leaves = {k: v[k].clone().requires_grad_() for k in names}
    y, fin = gdn.chunk_selective_scan(*(leaves[k] for k in names[:7]), True, leaves["h0"], True, v["cu"])
    got = torch.autograd.grad([y, fin], [leaves[k] for k in names], [v["dy"], v["dht"]])
    for k, g in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"), got):
        assert torch.equal(g, want[k]), k
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = train(gdn, v)
    for k in want:
        assert torch.equal(again[k], want[k]), k


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("H,lens", [(2, [2100]), (2, [700, 0, 1400]), (192, [130])])
def test_calls_in_a_row(gdn, dtype, H, lens):
    # nothing between the calls, whose kernels come up early and whose workspaces are the same memory:
    # each call's results are those of the call by itself
    both = [make(lens, H, 1, 64, 64, DT[dtype], seed=s) for s in (31, 32)]

    def call(v):
        y, fin, _ = gdn.chunk_selective_scan_fwd(*args(v), True, v["h0"], True, v["cu"])
        return y, fin

    alone = []
    for v in both:
        alone.append(call(v))
        torch.cuda.synchronize()
    got = [call(both[i % 2]) for i in range(24)]
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    for i, (y, fin) in enumerate(got):
        assert torch.equal(y, alone[i % 2][0]) and torch.equal(fin, alone[i % 2][1]), i


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_captured_graph(gdn, dtype):
    v = make([150, 90], 4, 2, 128, 64, DT[dtype], seed=17)
    want = train(gdn, v)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, fin, saved = gdn.chunk_selective_scan_fwd(*args(v), True, v["h0"], True, v["cu"], save_for_backward=True)
        grads = gdn.chunk_selective_scan_bwd(*args(v), True, saved, v["dy"], v["dht"], v["h0"], v["cu"])
    v2 = make([150, 90], 4, 2, 128, 64, DT[dtype], seed=18)
    want2 = train(gdn, v2)
    for src, exp in ((v2, want2), (make([150, 90], 4, 2, 128, 64, DT[dtype], seed=17), want)):
        for k in v:
            if v[k] is not None:
                v[k].copy_(src[k])
        g.replay()
        torch.cuda.synchronize()
        got = dict(zip(("y", "final", "dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"), (y, fin, *grads)))
        for k in got:
            assert torch.equal(got[k], exp[k]), k


def test_bad_offsets_are_reported(gdn):
    for dtype in (torch.float32, torch.bfloat16):
        v = make([100, 71], 2, 1, 128, 64, dtype, seed=18)
        for cu in ([0, 180, 171], [0, 100, 160], [0, -5, 171], [3, 100, 171]):
            bad = dict(v, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"))
            y, fin, _ = gdn.chunk_selective_scan_fwd(*args(bad), True, bad["h0"], True, bad["cu"])
            gdn.chunk_selective_scan_bwd(*args(bad), True, None, bad["dy"], bad["dht"], bad["h0"], bad["cu"])
            assert gdn.device_status() == 6
        verify(v, [100, 71], True, train(gdn, v))


def test_refusals(gdn):
    v = make([100], 2, 1, 128, 64, torch.bfloat16, seed=19)
    a = list(args(v))

    def f(i, t, **kw):
        b = list(a)
        b[i] = t
        return gdn.chunk_selective_scan_fwd(*b, True, **kw)

    with pytest.raises(TypeError, match="dt has dtype"):
        f(1, v["dt"].double())
    with pytest.raises(ValueError, match="dt"):
        f(1, v["dt"][..., :1])
    with pytest.raises(TypeError, match="A has dtype"):
        f(2, v["A"].bfloat16())
    with pytest.raises(ValueError, match="C has shape"):
        f(4, v["C"][..., :64])
    with pytest.raises(TypeError, match="B has dtype"):
        f(3, v["B"].float())
    with pytest.raises(ValueError, match="D has shape"):
        f(5, v["D"][:1])
    with pytest.raises(ValueError, match="initial_state"):
        f(0, v["x"], initial_state=v["h0"][:, :1])
    with pytest.raises(ValueError, match="x and B"):
        f(0, v["x"][0])
    with pytest.raises(gdn.GdnError):
        gdn.chunk_selective_scan_fwd(v["x"][..., :32].contiguous(), *a[1:], True)
    with pytest.raises(ValueError, match="in place"):
        gdn.recurrent_selective_scan(*a, True, v["h0"], v["h0"].transpose(2, 3).contiguous().transpose(2, 3))
