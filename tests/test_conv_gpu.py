"""Short causal convolution on the GPU against its plain 64-bit form, element by element.

Tolerances (layer_ref.close): the output's rounding, and of the terms' mass the fp32
operations in sequence (taps, bias and silu: under 16; a sum over tokens: that many more) and,
for bf16, the fast exponential's 2^-18."""
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


def rel(dtype, ops):
    return (16 + ops) * 2.0 ** -24 + (2.0 ** -18 if dtype == torch.bfloat16 else 0)


def make(lens, C, W, dtype, seed, bias=True, state=True, packed=True, wide=0):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)

    def r(*s, std=1.0):
        return (torch.randn(s, generator=g) * std).to(dtype).cuda()

    B = 1 if packed else N
    x = r(B, T // B, C + wide)[..., wide // 2:wide // 2 + C]
    return dict(x=x, weight=r(C, W, std=0.5), bias=r(C) if bias else None, state=r(N, W - 1, C) if state else None,
                dy=r(B, T // B, C), dfinal=r(N, W - 1, C),
                cu=torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() if packed else None)


def check(gdn, v, lens, silu, label=""):
    C, W = v["weight"].shape
    dtype = v["x"].dtype
    act = "silu" if silu else None
    y, fin = gdn.causal_conv1d_fwd(v["x"], v["weight"], v["bias"], act, v["state"], True, v["cu"])
    dx, dw, db, ds = gdn.causal_conv1d_bwd(v["x"], v["weight"], v["bias"], v["dy"], v["dfinal"], act, v["state"], v["cu"])
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    assert (db is None) == (v["bias"] is None) and (ds is None) == (v["state"] is None)
    flat = lambda t: t.reshape(-1, C)  # noqa: E731
    args = (flat(v["x"]), v["weight"], v["bias"], v["state"], silu, lens, flat(v["dy"]), v["dfinal"])
    ref, mass = R.conv(*args), R.conv(*args, mass=True)
    T = sum(lens)
    R.close(label + "y", flat(y), ref["y"], mass["y"], rel(dtype, 0))
    assert torch.equal(R.f64(fin), ref["final"]), label + "final"
    R.close(label + "dx", flat(dx), ref["dx"], mass["dx"], rel(dtype, 16))
    R.close(label + "dweight", dw, ref["dweight"], mass["dweight"], rel(dtype, T))
    if db is not None:
        R.close(label + "dbias", db, ref["dbias"], mass["dbias"], rel(dtype, T))
    if ds is not None:
        R.close(label + "dstate", ds, ref["dstate"], mass["dstate"], rel(dtype, 16))


# lengths around the runs of 32 and 64 tokens, the taps, empty sequences first, last and in a row
LENS = [[1], [2], [70], [0, 3, 0, 0, 1, 65, 0], [31, 1, 32, 33, 2, 64, 129], [200]]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("lens", LENS)
def test_packed(gdn, dtype, W, lens):
    check(gdn, make(lens, 264, W, DT[dtype], 10 * W + len(lens)), lens, True)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("C", [1, 7, 201, 512])
def test_widths_and_forms(gdn, dtype, silu, C):
    check(gdn, make([40, 5], C, 4, DT[dtype], C, bias=silu, state=not silu), [40, 5], silu)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_batch_and_slices(gdn, dtype):
    # a batch without packing; x a slice of a wider tensor, on and off 16-byte boundaries
    check(gdn, make([90] * 3, 72, 4, DT[dtype], 5, packed=False), [90] * 3, True)
    for wide in (32, 6, 3):
        check(gdn, make([90] * 2, 72, 3, DT[dtype], 6, packed=False, wide=wide), [90] * 2, True, f"wide {wide} ")


def test_many_packed_sequences(gdn):
    lens = [(7 * i) % 5 for i in range(300)]
    check(gdn, make(lens, 16, 4, torch.float32, 8), lens, True)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_long_runs(gdn, dtype):
    # so many channels that a warp's run spans tens of tokens, with sequences' borders inside
    lens = [500, 1, 0, 2, 37, 300, 3, 0, 163, 8, 486]
    check(gdn, make(lens, 8192, 4, DT[dtype], 12), lens, True)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_empty_batch(gdn, dtype):
    v = make([0, 0], 24, 4, DT[dtype], 9)
    check(gdn, v, [0, 0], True)  # final = initial, dstate = dfinal, dweight = 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("C", [8, 37, 2056])
def test_update_continues_a_prompt(gdn, dtype, C):
    # a prompt, then single tokens and a few at once, equal the convolution of the whole, bit for bit
    v = make([60] * 3, C, 4, DT[dtype], C, packed=False)
    y, fin = gdn.causal_conv1d_fwd(v["x"], v["weight"], v["bias"], "silu", v["state"], True)
    x = v["x"]
    _, st = gdn.causal_conv1d_fwd(x[:, :50], v["weight"], v["bias"], "silu", v["state"], True)
    at, out = 50, []
    for n in (1, 1, 2, 5, 1):
        out.append(gdn.causal_conv1d_update(x[:, at:at + n], st, v["weight"], v["bias"], "silu"))
        at += n
    assert torch.equal(torch.cat(out, 1), y[:, 50:]) and torch.equal(st, fin)


def test_packed_sequences_do_not_touch(gdn):
    lens = [33, 40, 20]
    v = make(lens, 64, 4, torch.bfloat16, 12)
    clean = gdn.causal_conv1d_fwd(v["x"], v["weight"], v["bias"], "silu", v["state"], True, v["cu"])
    gclean = gdn.causal_conv1d_bwd(v["x"], v["weight"], v["bias"], v["dy"], v["dfinal"], "silu", v["state"], v["cu"])
    for bad in (float("nan"), float("inf")):
        w = {k: (t.clone() if t is not None else None) for k, t in v.items()}
        w["x"][:, 33:73], w["dy"][:, 33:73], w["state"][1], w["dfinal"][1] = bad, bad, bad, bad
        y, fin = gdn.causal_conv1d_fwd(w["x"], w["weight"], w["bias"], "silu", w["state"], True, w["cu"])
        dx, _, _, ds = gdn.causal_conv1d_bwd(w["x"], w["weight"], w["bias"], w["dy"], w["dfinal"], "silu", w["state"], w["cu"])
        for got, want, ax in ((y, clean[0], 1), (dx, gclean[0], 1)):
            assert torch.equal(got[:, :33], want[:, :33]) and torch.equal(got[:, 73:], want[:, 73:])
        for got, want in ((fin, clean[1]), (ds, gclean[3])):
            assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


def test_autograd_and_repeat(gdn):
    v = make([30, 41], 40, 4, torch.float32, 13)
    leaves = [v[k].clone().requires_grad_() for k in ("x", "weight", "bias", "state")]
    y, fin = gdn.causal_conv1d(leaves[0], leaves[1], leaves[2], "silu", leaves[3], True, v["cu"])
    got = torch.autograd.grad([y, fin], leaves, [v["dy"], v["dfinal"]])
    want = gdn.causal_conv1d_bwd(v["x"], v["weight"], v["bias"], v["dy"], v["dfinal"], "silu", v["state"], v["cu"])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    y, fin = gdn.causal_conv1d(leaves[0], leaves[1], None, None)
    assert fin is None
    y.sum().backward()  # an expanded gradient, no final state
    assert torch.isfinite(leaves[0].grad).all()


def test_bad_offsets_are_reported(gdn):
    v = make([30, 41], 40, 4, torch.float32, 14)
    for cu in ([0, 80, 71], [0, 30, 60], [0, -5, 71], [3, 30, 71]):
        gdn.causal_conv1d_fwd(v["x"], v["weight"], v["bias"], None, None, True,
                              torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert gdn.device_status() == 6
    check(gdn, v, [30, 41], True)


def test_refusals(gdn):
    v = make([30, 41], 40, 4, torch.bfloat16, 15)
    f = gdn.causal_conv1d_fwd
    with pytest.raises(TypeError, match="weight"):
        f(v["x"], v["weight"].float())
    with pytest.raises(ValueError, match="weight"):
        f(v["x"], v["weight"][:20])
    with pytest.raises(ValueError, match="W in 2..4"):
        f(v["x"], v["weight"][:, :1])
    with pytest.raises(ValueError, match="bias"):
        f(v["x"], v["weight"], v["bias"][:3])
    with pytest.raises(ValueError, match="activation"):
        f(v["x"], v["weight"], None, "gelu")
    with pytest.raises(ValueError, match="initial_state"):
        f(v["x"], v["weight"], None, None, v["state"])  # two states, one sequence
    with pytest.raises(ValueError, match="B == 1"):
        f(v["x"].view(71, 1, 40), v["weight"], cu_seqlens=v["cu"])
    with pytest.raises(ValueError, match="x must be"):
        f(v["x"][0], v["weight"])
    with pytest.raises(TypeError, match="unsupported dtype"):
        f(v["x"].half(), v["weight"].half())
    with pytest.raises(ValueError, match="expected cuda"):
        f(v["x"], v["weight"].cpu())
    with pytest.raises(ValueError, match="in place"):
        gdn.causal_conv1d_update(v["x"], torch.zeros(1, 40, 3, dtype=torch.bfloat16, device="cuda").transpose(1, 2),
                                 v["weight"])
