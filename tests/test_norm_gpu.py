"""Layer norm, centred or not, with and without a silu gate, on the GPU against its plain
64-bit form, element by element.

Tolerances: the output's rounding, and of the terms' magnitudes the fp32 operations in
sequence (a row's sums: a thread's own elements and a tree, under 100 for the widths here
up to 8192, under 200 for the widest; a column's sum: that many rows) plus, for a gate in
bf16, the fast exponential's 2^-18."""
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


def make(rows, D, dtype, wdtype, seed, bias, gate, mean=0.0):
    g = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=g)

    x = (r(rows, D) + mean * r(rows, 1)).to(dtype).cuda()
    return dict(x=x, weight=(1 + 0.1 * r(D)).to(wdtype).cuda(), bias=r(D).to(wdtype).cuda() if bias else None,
                gate=r(rows, D).to(dtype).cuda() if gate else None, dy=r(rows, D).to(dtype).cuda())


def check(gdn, v, center, first, eps=1e-5):
    a = (v["x"], v["weight"], v["bias"], v["gate"])
    y, stats = gdn.layer_norm_fwd(*a, eps, center, first)
    dx, dw, db, dg = gdn.layer_norm_bwd(*a, v["dy"], stats, eps, center, first)
    torch.cuda.synchronize()
    assert (db is None) == (v["bias"] is None) and (dg is None) == (v["gate"] is None)
    ref = R.norm(*a, eps, center, first, v["dy"])
    x, w, b, z, d = (R.f64(t) for t in (*a, v["dy"]))
    rows, D = x.shape
    e = 200 * 2.0 ** -24 + (2.0 ** -18 if z is not None and v["x"].dtype == torch.bfloat16 else 0)
    s = R.sigm(z) if z is not None else None
    gf = (z * s).abs() if z is not None else torch.ones_like(x)
    dgf = (s * (1 + z * (1 - s))).abs() + (s.abs() + gf) if z is not None else None
    u = x.abs() * (gf if first else 1)
    mu = u.mean(1, keepdim=True) if center else 0
    n = (u + mu) * ref["rstd"]                      # magnitude of the normalised value's terms
    n = n + ref["n"].abs() * (n * n).mean(1, keepdim=True)  # and through the variance
    lin = n * w.abs() + (b.abs() if b is not None else 0)
    last = z is not None and not first
    R.close("y", y, ref["y"], lin * gf if last else lin, e)
    dl = d.abs() * gf if last else d.abs()
    dn = dl * w.abs()
    du = ref["rstd"] * (dn + n * (dn * n).mean(1, keepdim=True) + dn.mean(1, keepdim=True))
    du = du + du * (n * n).mean(1, keepdim=True)    # rstd's own error
    R.close("dx", dx, ref["dx"], du * gf if first else du, 2 * e)
    R.close("dweight", dw, ref["dweight"], (dl * n).sum(0), e + (rows + 64) * 2.0 ** -24)
    if b is not None:
        R.close("dbias", db, ref["dbias"], dl.sum(0), e + (rows + 64) * 2.0 ** -24)
    if z is not None:
        R.close("dgate", dg, ref["dgate"], (du * x.abs() if first else d.abs() * lin) * dgf, 2 * e)


# every way a row is held: 8, 16, 32 threads, one to four accesses, a block, and the widths and
# alignments that read a row once per pass
WIDTHS = [1, 3, 8, 40, 64, 128, 200, 256, 320, 512, 777, 1024, 1096, 2048, 2304, 4096, 8192, 8200, 20000]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("form", ["plain", "first", "last"])
def test_widths(gdn, D, dtype, form):
    v = make(37, D, DT[dtype], torch.float32, D, True, form != "plain")
    check(gdn, v, form != "last", form == "first")


@pytest.mark.parametrize("rows", [1, 2, 16, 17, 5000])
@pytest.mark.parametrize("D", [64, 128, 2048, 33])
def test_rows(gdn, rows, D):
    check(gdn, make(rows, D, torch.bfloat16, torch.bfloat16, rows, False, True), False, False)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("wdtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gate", ["none", "first", "last"])
def test_forms(gdn, center, bias, wdtype, gate):
    check(gdn, make(70, 128, torch.bfloat16, DT[wdtype], 3, bias, gate != "none", mean=3.0), center, gate == "first")


@pytest.mark.parametrize("D", [96, 4096, 55])
def test_constant_and_zero_rows(gdn, D):
    # variance 0: eps alone; with a far mean the centred value keeps its precision
    v = make(6, D, torch.float32, torch.float32, 7, True, False)
    v["x"][0] = 0
    v["x"][1] = 2.5
    y, _ = gdn.layer_norm_fwd(v["x"], v["weight"], v["bias"], None, 1e-5, True)
    assert torch.equal(y[0], v["bias"])
    torch.testing.assert_close(y[1], v["bias"], rtol=0, atol=2.5 * 2 ** -22 / 1e-5 ** 0.5 * 2)
    v["x"][0] = torch.randn(D, device="cuda")
    v["x"][1] = 100 + torch.randn(D, device="cuda")
    check(gdn, v, True, False)


def test_a_bad_row_stays_alone(gdn):
    for D in (128, 4096, 33):
        v = make(40, D, torch.bfloat16, torch.float32, 8, True, True)
        a, st = gdn.layer_norm_fwd(v["x"], v["weight"], v["bias"], v["gate"])
        ga = gdn.layer_norm_bwd(v["x"], v["weight"], v["bias"], v["gate"], v["dy"], st)[0]
        v["x"][7] = float("inf")
        b, st = gdn.layer_norm_fwd(v["x"], v["weight"], v["bias"], v["gate"])
        gb = gdn.layer_norm_bwd(v["x"], v["weight"], v["bias"], v["gate"], v["dy"], st)[0]
        keep = [i for i in range(40) if i != 7]
        assert torch.equal(a[keep], b[keep]) and torch.equal(ga[keep], gb[keep])


def test_shapes_views_and_autograd(gdn):
    # [.., D] of any rank, a strided view, no rows at all; the same results by autograd, twice
    v = make(60, 64, torch.float32, torch.float32, 9, True, True)
    y, st = gdn.layer_norm_fwd(v["x"], v["weight"], v["bias"], v["gate"])
    y3, _ = gdn.layer_norm_fwd(v["x"].view(3, 4, 5, 64), v["weight"], v["bias"], v["gate"].view(3, 4, 5, 64))
    assert torch.equal(y3.view(60, 64), y)
    wide = torch.empty(60, 130, device="cuda")
    wide[:, 1:65] = v["x"]
    yw, _ = gdn.layer_norm_fwd(wide[:, 1:65], v["weight"], v["bias"], v["gate"])
    assert torch.equal(yw, y)
    leaves = [v[k].clone().requires_grad_() for k in ("x", "weight", "bias", "gate")]
    for _ in range(2):
        got = torch.autograd.grad(gdn.layer_norm(*leaves), leaves, v["dy"])
        for p, q in zip(got, gdn.layer_norm_bwd(v["x"], v["weight"], v["bias"], v["gate"], v["dy"], st)):
            assert torch.equal(p, q)
    for D in (64, 33):
        w = torch.ones(D, device="cuda")
        e = torch.empty(0, D, device="cuda")
        y, st = gdn.layer_norm_fwd(e, w, w)
        dx, dw, db, _ = gdn.layer_norm_bwd(e, w, w, None, e, st)
        assert y.shape == (0, D) and dx.shape == (0, D) and not dw.any() and not db.any()


def test_refusals(gdn):
    v = make(5, 64, torch.bfloat16, torch.float32, 10, True, True)
    f = gdn.layer_norm_fwd
    with pytest.raises(ValueError, match="weight"):
        f(v["x"], v["weight"][:32])
    with pytest.raises(TypeError, match="weight"):
        f(v["x"], v["weight"].double())
    with pytest.raises(TypeError, match="bias"):
        f(v["x"], v["weight"], v["bias"].bfloat16())
    with pytest.raises(ValueError, match="gate"):
        f(v["x"], v["weight"], None, v["gate"][:3])
    with pytest.raises(ValueError, match="gate_first"):
        f(v["x"], v["weight"], gate_first=True)
    with pytest.raises(gdn.GdnError):
        f(v["x"], v["weight"], eps=-1.0)
    with pytest.raises(ValueError, match="stats"):
        gdn.layer_norm_bwd(v["x"], v["weight"], None, None, v["dy"], torch.zeros(4, 2, device="cuda"))
