"""Plain 64-bit forms of the operators around the gated delta rule, written from their
definitions (sequence by sequence, token by token), and the tolerances their tests use.

Every function also runs with `mass=True`: the same sums over the absolute values of their
terms (inputs made positive, differences turned into sums, decays and derivative factors
kept). A computed value's error is bounded by its mass times the relative error of its
terms, whatever cancels in the value itself, so a tolerance is

    |got - ref| <= half(out) |ref| + rel * mass(ref)

with half(t) = eps(t)/2, the rounding of the output, and rel the sum of the relative errors
that the terms can take: 2^-24 for each fp32 operation in sequence (n of them: n 2^-24), and
half(bf16) = 2^-8 for each operand that a kernel rounds to bf16.
"""
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return None if t is None else t.detach().to("cpu").double()


def sigm(v):
    return 1 / (1 + torch.exp(-v))


def close(name, got, ref, mass, rel):
    """Asserts |got - ref| <= half(out) |ref| + rel * mass element by element."""
    g = f64(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    if not g.numel():
        return 0.0
    tol = HALF[got.dtype] * ref.abs() * (1 + rel) + rel * mass.abs() + 1e-37
    bad = (g - ref).abs() > tol
    worst = float(((g - ref).abs() / tol).max())
    assert not bad.any() and torch.isfinite(g).all(), (
        name, f"{int(bad.sum())} of {bad.numel()} values off, worst {worst:.3g} tolerances", got.dtype)
    return worst


def spans(total, lens):
    at = 0
    for n in lens:
        yield at, at + n
        at += n
    assert at == total


# ------------------------------------------------------------------ convolution
def conv(x, weight, bias, state, silu, lens, dy=None, dfinal=None, mass=False):
    """x [total, C]; state [N, W-1, C] or None. Returns a dict of y, final and the gradients."""
    C, W = weight.shape
    pick = (lambda t: None if t is None else f64(t).abs()) if mass else f64
    xs, w, b, st, d_y, d_f = (pick(t) for t in (x, weight, bias, state, dy, dfinal))
    tx, tw, tb, ts = f64(x), f64(weight), f64(bias), f64(state)  # the true values, for the factors
    out = {"y": torch.zeros_like(xs), "final": torch.zeros((len(lens), W - 1, C), dtype=torch.float64)}
    g = {"dx": torch.zeros_like(xs), "dweight": torch.zeros_like(w), "dbias": torch.zeros(C, dtype=torch.float64),
         "dstate": torch.zeros((len(lens), W - 1, C), dtype=torch.float64)}
    for n, (a, e) in enumerate(spans(x.shape[0], lens)):
        zero = torch.zeros((W - 1, C), dtype=torch.float64)
        seen = torch.cat([st[n] if st is not None else zero, xs[a:e]])
        true = torch.cat([ts[n] if ts is not None else zero, tx[a:e]])
        out["final"][n] = seen[e - a:]
        dseen = torch.zeros_like(seen)
        if d_f is not None:
            dseen[e - a:] += d_f[n]
        for t in range(e - a):
            pre = (seen[t:t + W] * w.T).sum(0) + (b if b is not None else 0)
            tp = (true[t:t + W] * tw.T).sum(0) + (tb if tb is not None else 0)
            s = sigm(tp)
            # d silu / d pre <= 1.1: an error of pre moves the output by at most that much of it
            out["y"][a + t] = (pre * 1.1 if mass else pre * s) if silu else pre
            if d_y is None:
                continue
            factor = s * (1 + tp * (1 - s)) if silu else torch.ones_like(s)
            d = d_y[a + t] * factor
            if mass:  # the factor's own error: |silu''| <= 0.5, by pre's mass
                d = d_y[a + t] * (factor.abs() + (0.5 * pre if silu else 0))
            dseen[t:t + W] += w.T * d
            g["dweight"] += (seen[t:t + W] * d).T
            g["dbias"] += d
        g["dx"][a:e] = dseen[W - 1:]
        g["dstate"][n] = dseen[:W - 1]
    if dy is not None:
        out.update(g)
    return out


# ------------------------------------------------------------------------- scan
def scan(x, dt, A, B, C, D, dt_bias, softplus, h0, lens, dy=None, dht=None, mass=False, keep=128):
    """x [total, H, P], dt [total, H], B, C [total, G, K]; h0 [N, H, K, P] or None. Returns y,
    final and, with dy, every gradient. The gradient of the log decay is a_t <h_{t-1}, g_t>, g_t
    being the state's gradient; its mass is that of the kernels' sum, backwards over the
    token's stretch of `keep` tokens from <h, g> at the stretch's end."""
    H, P = x.shape[1], x.shape[2]
    G, K = B.shape[1], B.shape[2]
    r = H // G
    pick = (lambda t: None if t is None else f64(t).abs()) if mass else f64
    xs, Bs, Cs, d_y, g0, gT = (pick(t) for t in (x, B, C, dy, h0, dht))
    Ds = pick(D)
    Bs, Cs = Bs.repeat_interleave(r, 1), Cs.repeat_interleave(r, 1)
    At = f64(A)
    As = At.abs() if mass else At
    raw = f64(dt) + (f64(dt_bias) if dt_bias is not None else 0)
    delta = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw.clamp(max=30)))) if softplus else raw
    a = torch.exp(delta * At)
    dl = delta.abs() if mass else delta
    draw = sigm(raw) if softplus else torch.ones_like(raw)
    N = len(lens)
    out = {"y": torch.zeros_like(xs), "final": torch.zeros((N, H, K, P), dtype=torch.float64)}
    for nm, like in (("dx", xs), ("dB_", Bs), ("dC_", Cs), ("ddt", raw)):
        out[nm] = torch.zeros_like(like)
    for nm in ("dA", "dD", "ddt_bias"):
        out[nm] = torch.zeros(H, dtype=torch.float64)
    out["dh0"] = torch.zeros((N, H, K, P), dtype=torch.float64)
    for n, (s, e) in enumerate(spans(x.shape[0], lens)):
        h = g0[n].clone() if g0 is not None else torch.zeros((H, K, P), dtype=torch.float64)
        ends, before = {}, {}
        for t in range(s, e):
            before[t] = h
            h = a[t][:, None, None] * h + (dl[t][:, None] * Bs[t])[:, :, None] * xs[t][:, None, :]
            out["y"][t] = (Cs[t][:, :, None] * h).sum(1)
            if Ds is not None:
                out["y"][t] += Ds[:, None] * xs[t]
            if d_y is not None:
                out["dC_"][t] = (h * d_y[t][:, None, :]).sum(2)
                if (t - s + 1) % keep == 0 or t == e - 1:
                    ends[t] = h.clone()
        out["final"][n] = h
        if d_y is None:
            continue
        g = gT[n].clone() if gT is not None else torch.zeros((H, K, P), dtype=torch.float64)
        carry = torch.zeros(H, dtype=torch.float64)
        for t in range(e - 1, s - 1, -1):
            if mass and t in ends:
                carry = (ends[t] * g).sum((1, 2))
            g = g + Cs[t][:, :, None] * d_y[t][:, None, :]
            u = (Bs[t][:, :, None] * g).sum(1)
            w = (u * xs[t]).sum(1)
            out["dx"][t] = dl[t][:, None] * u + (Ds[:, None] * d_y[t] if Ds is not None else 0)
            out["dB_"][t] = (g * (dl[t][:, None] * xs[t])[:, None, :]).sum(2)
            if mass:
                carry = carry + (Cs[t] * out["dC_"][t]).sum(1) + dl[t] * w
            else:
                carry = a[t] * (before[t] * g).sum((1, 2))
            out["ddt"][t] = (As * carry + w) * draw[t]
            out["dA"] += dl[t] * carry
            out["ddt_bias"] += out["ddt"][t]
            out["dD"] += (xs[t] * d_y[t]).sum(1)
            g = a[t][:, None, None] * g
        out["dh0"][n] = g
    out["dB"] = out.pop("dB_").unflatten(1, (G, r)).sum(2)
    out["dC"] = out.pop("dC_").unflatten(1, (G, r)).sum(2)
    return out


# ------------------------------------------------------------------- layer norm
def norm(x, weight, bias, gate, eps, center, gate_first, dy=None):
    """[R, D]; values only (the tests bound errors row by row)."""
    x, w, b, z, d = (f64(t) for t in (x, weight, bias, gate, dy))
    s = sigm(z) if z is not None else None
    first, last = z is not None and gate_first, z is not None and not gate_first
    u = x * z * s if first else x
    mean = u.mean(1, keepdim=True) if center else torch.zeros((x.shape[0], 1), dtype=torch.float64)
    rstd = 1 / torch.sqrt(((u - mean) ** 2).mean(1, keepdim=True) + eps)
    n = (u - mean) * rstd
    lin = n * w + (b if b is not None else 0)
    out = {"y": lin * z * s if last else lin, "rstd": rstd, "n": n}
    if d is None:
        return out
    dl = d * z * s if last else d
    dn = dl * w
    du = rstd * (dn - n * (dn * n).mean(1, keepdim=True) - (dn.mean(1, keepdim=True) if center else 0))
    out["dweight"], out["dbias"] = (dl * n).sum(0), dl.sum(0)
    out["dx"] = du * z * s if first else du
    if z is not None:
        ds = s * (1 + z * (1 - s))
        out["dgate"] = (du * x if first else d * lin) * ds
    return out
