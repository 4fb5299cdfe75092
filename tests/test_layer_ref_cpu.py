"""The plain 64-bit forms that the operators' GPU tests compare with (layer_ref.py) are
themselves checked here, on the CPU: values against automatic differentiation of independent
forms, gradients against central differences, packed sequences against separate calls."""
import pytest
import torch

import layer_ref as R

torch.manual_seed(0)


def rnd(*s, g):
    return torch.randn(s, generator=g, dtype=torch.float64)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def differences(f, args, names, grads, seed, eps=1e-5):
    """Central differences of the scalar f along a random direction of each argument."""
    g = gen(seed)
    for n in names:
        if args[n] is None:
            continue
        d = torch.randn(args[n].shape, generator=g, dtype=torch.float64)
        up, down = dict(args), dict(args)
        up[n], down[n] = args[n] + eps * d, args[n] - eps * d
        num = (f(up) - f(down)) / (2 * eps)
        ana = float((grads[n] * d).sum())
        assert abs(num - ana) <= 1e-7 * (1 + abs(ana)), (n, num, ana)


@pytest.mark.parametrize("silu,W,lens", [(True, 4, [5, 0, 1, 9]), (False, 3, [7]), (True, 2, [1, 2])])
def test_conv(silu, W, lens):
    g = gen(1)
    T, C, N = sum(lens), 3, len(lens)
    a = {"x": rnd(T, C, g=g), "w": rnd(C, W, g=g), "b": rnd(C, g=g), "s": rnd(N, W - 1, C, g=g)}
    dy, df = rnd(T, C, g=g), rnd(N, W - 1, C, g=g)
    r = R.conv(a["x"], a["w"], a["b"], a["s"], silu, lens, dy, df)

    def loss(v):
        o = R.conv(v["x"], v["w"], v["b"], v["s"], silu, lens)
        return float((o["y"] * dy).sum() + (o["final"] * df).sum())

    differences(loss, a, "xwbs", {"x": r["dx"], "w": r["dweight"], "b": r["dbias"], "s": r["dstate"]}, 2)
    # the library's own convolution, one sequence at a time
    at = 0
    for n, ln in enumerate(lens):
        seen = torch.cat([a["s"][n], a["x"][at:at + ln]]).T[None]
        if ln:
            ref = torch.nn.functional.conv1d(seen, a["w"][:, None], a["b"], groups=C)[0].T
            ref = torch.nn.functional.silu(ref) if silu else ref
            torch.testing.assert_close(r["y"][at:at + ln], ref)
        at += ln


@pytest.mark.parametrize("softplus,lens,h0,D", [(True, [6, 0, 3], True, True), (False, [8], False, False)])
def test_scan(softplus, lens, h0, D):
    g = gen(3)
    T, N, H, G, K, P = sum(lens), len(lens), 4, 2, 3, 2
    a = {"x": rnd(T, H, P, g=g), "dt": rnd(T, H, g=g), "A": -rnd(H, g=g).abs(), "B": rnd(T, G, K, g=g),
         "C": rnd(T, G, K, g=g), "D": rnd(H, g=g) if D else None, "bias": rnd(H, g=g),
         "h0": rnd(N, H, K, P, g=g) if h0 else None}
    dy, dht = rnd(T, H, P, g=g), rnd(N, H, K, P, g=g)

    def call(v, **kw):
        return R.scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["bias"], softplus, v["h0"], lens, **kw)

    r = call(a, dy=dy, dht=dht)

    def loss(v):
        o = call(v)
        return float((o["y"] * dy).sum() + (o["final"] * dht).sum())

    grads = {"x": r["dx"], "dt": r["ddt"], "A": r["dA"], "B": r["dB"], "C": r["dC"], "D": r["dD"], "bias": r["ddt_bias"],
             "h0": r["dh0"]}
    differences(loss, a, list(a), grads, 4)
    # the unrolled sum: y_t = C_t . (sum_s decay(s, t) delta_s B_s x_s + decay h0)
    raw = a["dt"] + a["bias"]
    dl = torch.nn.functional.softplus(raw) if softplus else raw
    at = 0
    for n, ln in enumerate(lens):
        for t in range(at, at + ln):
            for h in range(H):
                v = torch.zeros(P, dtype=torch.float64)
                for s in range(at, t + 1):
                    dec = torch.exp((dl[s + 1:t + 1, h] * a["A"][h]).sum())
                    v = v + dec * dl[s, h] * (a["C"][t, h // 2] @ a["B"][s, h // 2]) * a["x"][s, h]
                if a["h0"] is not None:
                    v = v + torch.exp((dl[at:t + 1, h] * a["A"][h]).sum()) * (a["C"][t, h // 2] @ a["h0"][n, h])
                if D:
                    v = v + a["D"][h] * a["x"][t, h]
                torch.testing.assert_close(r["y"][t, h], v)
        at += ln
    # a mass is never smaller than the value
    m = call(a, dy=dy, dht=dht, mass=True)
    for k in ("y", "final", "dx", "dB", "dC", "dA", "dD", "dh0"):
        assert (m[k] >= r[k].abs() - 1e-12).all(), k


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("gate", [None, "first", "last"])
def test_norm(center, gate):
    g = gen(5)
    a = {"x": rnd(4, 6, g=g), "w": rnd(6, g=g), "b": rnd(6, g=g), "z": rnd(4, 6, g=g) if gate else None}
    dy = rnd(4, 6, g=g)
    r = R.norm(a["x"], a["w"], a["b"], a["z"], 1e-3, center, gate == "first", dy)

    def loss(v):
        return float((R.norm(v["x"], v["w"], v["b"], v["z"], 1e-3, center, gate == "first")["y"] * dy).sum())

    differences(loss, a, "xwbz", {"x": r["dx"], "w": r["dweight"], "b": r["dbias"], "z": r.get("dgate")}, 6)
    if center and gate is None:
        torch.testing.assert_close(r["y"], torch.nn.functional.layer_norm(a["x"], (6,), a["w"], a["b"], 1e-3))
