"""Workloads of the operators around the gated delta rule: the short causal
convolution, the selective state space scan and the (gated) layer norm.

A case is one call, or one forward and backward pass, of one operator:

  conv   y_t = act(bias + sum_j weight_j x_{t-W+1+j}) per channel, sequences packed
         or in a batch, the W-1 inputs before each sequence in a state; "step" takes
         one token per sequence and updates the state in place
  scan   h_t = exp(D_t A) h_{t-1} + D_t B_t x_t^T,  y_t = C_t h_t + skip x_t, with
         D_t = softplus(dt_t + dt_bias); "step" takes one token per sequence
  norm   x^ = (x - mean) rstd (mean 0 where not centred), y = x^ weight + bias, with
         a gate silu(z) multiplied before or after the normalisation

`run` computes a case in plain torch operations in 32 bits (64 for the running sums
of the log decay), or, where `own` is true, by the framework's calls.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # q, k, v of one Gated DeltaNet layer (16 q/k heads, 32 value heads of 128) through the short
        # convolution in a long prefill, its last inputs kept for decoding
        {"name": "conv_prompt_t8192", "op": "conv", "mode": "prompt", "B": 1, "T": 8192, "C": 8192, "W": 4, "lens": "",
         "act": True, "bias": False, "state": False, "dtype": "bf16"},
        # a training step's packed documents through the convolution of a state space layer
        # (64 heads of 64 and one B, C group of 128)
        {"name": "conv_train_packed", "op": "conv", "mode": "train", "B": 1, "T": 8192, "C": 4352, "W": 4,
         "lens": "1,2047,130,3000,0,513,2501", "act": True, "bias": True, "state": True, "dtype": "bf16"},
        # single precision at odd sizes, as a gradient check runs it
        {"name": "conv_train_fp32_odd", "op": "conv", "mode": "train", "B": 2, "T": 333, "C": 201, "W": 3, "lens": "",
         "act": False, "bias": True, "state": False, "dtype": "fp32"},
        # one decoding step of 256 sequences
        {"name": "conv_step_b256", "op": "conv", "mode": "step", "B": 256, "T": 1, "C": 8192, "W": 4, "lens": "",
         "act": True, "bias": True, "state": True, "dtype": "bf16"},
        # long prefill of one sequence
        {"name": "scan_prompt_t8192_h64", "op": "scan", "mode": "prompt", "B": 1, "T": 8192, "H": 64, "G": 1, "K": 128,
         "P": 64, "lens": "", "state": False, "skip": True, "dtype": "bf16", "dt": "bf16"},
        # prefill of a packed batch with lengths from 64 to 8192, continued from kept states
        {"name": "scan_prompt_packed_32k", "op": "scan", "mode": "prompt", "B": 1, "T": 32768, "H": 32, "G": 4, "K": 128,
         "P": 64, "lens": "8192,64,5003,731,4099,97,2048,6001,311,129,1777,512,1300,1000,904,600", "state": True,
         "skip": True, "dtype": "bf16", "dt": "fp32"},
        # a training step: forward and every gradient
        {"name": "scan_train_b2_t4096_h16", "op": "scan", "mode": "train", "B": 2, "T": 4096, "H": 16, "G": 2, "K": 128,
         "P": 128, "lens": "", "state": True, "skip": True, "dtype": "bf16", "dt": "bf16"},
        # single precision at an odd length, as a gradient check runs it
        {"name": "scan_train_fp32_t1000", "op": "scan", "mode": "train", "B": 1, "T": 1000, "H": 4, "G": 2, "K": 64,
         "P": 64, "lens": "", "state": True, "skip": True, "dtype": "fp32", "dt": "fp32"},
        # one decoding step of 256 sequences, and of one
        {"name": "scan_step_b256_h64", "op": "scan", "mode": "step", "B": 256, "T": 1, "H": 64, "G": 1, "K": 128, "P": 64,
         "lens": "", "state": True, "skip": True, "dtype": "bf16", "dt": "bf16"},
        {"name": "scan_step_b1_h64", "op": "scan", "mode": "step", "B": 1, "T": 1, "H": 64, "G": 1, "K": 128, "P": 64,
         "lens": "", "state": True, "skip": True, "dtype": "bf16", "dt": "bf16"},
        # the gated norm on the recurrence's output, per head of 128 (8192 tokens, 32 heads), trained
        {"name": "norm_train_heads_d128", "op": "norm", "mode": "train", "R": 262144, "D": 128, "center": False,
         "bias": False, "gate": "after", "dtype": "bf16", "wdtype": "fp32"},
        # layer norm over a layer's width, trained
        {"name": "norm_train_layer_d4096", "op": "norm", "mode": "train", "R": 4096, "D": 4096, "center": True,
         "bias": True, "gate": "", "dtype": "bf16", "wdtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total):
    """A few sequence lengths that add up to `total`; now and then an empty one."""
    n = rng.randint(2, 12)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    op = rng.choice(["conv", "conv", "scan", "scan", "scan", "norm"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op == "conv":
        mode = rng.choice(["prompt", "train", "step"])
        c = {"op": "conv", "mode": mode, "B": 1, "T": 1, "C": _log(rng, 64, 8192), "W": rng.choice([2, 3, 4, 4]),
             "lens": "", "act": rng.random() < 0.7, "bias": rng.random() < 0.5, "state": rng.random() < 0.5, "dtype": dtype}
        if mode == "step":
            c["B"], c["state"] = _log(rng, 1, 256), True
        elif rng.random() < 0.5:
            c["T"] = _log(rng, 1, 8192)
            c["lens"] = _lens(rng, c["T"])
        else:
            c["B"] = rng.randint(1, 4)
            c["T"] = _log(rng, 1, 8192 // c["B"])
        return c
    if op == "scan":
        mode = rng.choice(["prompt", "prompt", "train", "train", "step"])
        G = rng.choice([1, 1, 2, 4])
        c = {"op": "scan", "mode": mode, "B": 1, "T": 1, "H": G * rng.randint(1, 8), "G": G,
             "K": rng.choice([128, 128, 64]), "P": rng.choice([64, 64, 128]), "lens": "", "state": rng.random() < 0.6,
             "skip": rng.random() < 0.8, "dtype": dtype, "dt": rng.choice([dtype, "fp32"])}
        most = 8192 if dtype == "bf16" else 2048
        if mode == "step":
            c["B"], c["state"] = _log(rng, 1, 256), True
        elif rng.random() < 0.5:
            c["T"] = _log(rng, 1, most)
            c["lens"] = _lens(rng, c["T"])
        else:
            c["B"] = rng.randint(1, 3)
            c["T"] = _log(rng, 1, most // c["B"])
        return c
    D = _log(rng, 32, 8192)
    gate = rng.choice(["", "before", "after"])
    return {"op": "norm", "mode": rng.choice(["prompt", "train"]), "R": _log(rng, 1, max(2, (1 << 24) // D)), "D": D,
            "center": rng.random() < 0.5, "bias": rng.random() < 0.5, "gate": gate, "dtype": dtype,
            "wdtype": rng.choice([dtype, "fp32"])}


def _lengths(c):
    return [int(v) for v in c["lens"].split(",")] if c["lens"] else [c["T"]] * c["B"]


# ----------------------------------------------------------------------- inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = _DT[c["dtype"]]

    def randn(*shape, std=1.0, dtype=d):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    s = {"case": c}
    train = c["mode"] == "train"
    if c["op"] == "norm":
        w = _DT[c["wdtype"]]
        s["x"] = randn(c["R"], c["D"])
        if c["center"]:  # a mean of its own in every row
            s["x"] = (s["x"].float() + torch.randn((c["R"], 1), generator=g, device="cuda")).to(d)
        s["weight"] = (1 + randn(c["D"], std=0.1, dtype=torch.float32)).to(w)
        s["bias"] = randn(c["D"], std=0.1, dtype=w) if c["bias"] else None
        s["gate"] = randn(c["R"], c["D"]) if c["gate"] else None
        s["dy"] = randn(c["R"], c["D"]) if train else None
        return s
    lens = _lengths(c)
    N = len(lens)
    s["lens"] = lens
    s["cu"] = None
    if c["lens"]:
        s["cu"] = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    if c["op"] == "conv":
        s["x"] = randn(c["B"], c["T"], c["C"])
        s["weight"] = randn(c["C"], c["W"], std=c["W"] ** -0.5)
        s["bias"] = randn(c["C"], std=0.1) if c["bias"] else None
        s["state"] = randn(N, c["W"] - 1, c["C"]) if c["state"] else None
        if train:
            s["dy"] = randn(c["B"], c["T"], c["C"])
            s["dfinal"] = randn(N, c["W"] - 1, c["C"])
        return s
    H, G, K, P = c["H"], c["G"], c["K"], c["P"]
    # x, B and C are slices of one convolution's output, as a layer has them
    xbc = randn(c["B"], c["T"], H * P + 2 * G * K)
    s["x"] = xbc[..., :H * P].unflatten(-1, (H, P))
    s["Bm"] = xbc[..., H * P:H * P + G * K].unflatten(-1, (G, K))
    s["Cm"] = xbc[..., H * P + G * K:].unflatten(-1, (G, K))
    s["dt"] = randn(c["B"], c["T"], H, dtype=_DT[c["dt"]])
    s["A"] = -(1 + 15 * rand(H))
    step = torch.exp(math.log(1e-3) + rand(H) * (math.log(1e-1) - math.log(1e-3)))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["D"] = 1 + randn(H, std=0.1, dtype=torch.float32) if c["skip"] else None
    s["h0"] = randn(N, H, K, P, std=0.1, dtype=torch.float32) if c["state"] else None
    if train:
        s["dy"] = randn(c["B"], c["T"], H, P)
        s["dht"] = randn(N, H, K, P, std=0.1, dtype=torch.float32)
    return s


# -------------------------------------------------------------------------- run
def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    if c["op"] == "norm":
        return _plain_norm(c, state)
    if c["op"] == "conv":
        return _plain_conv_step(c, state) if c["mode"] == "step" else _plain_conv(c, state)
    return _plain_scan_step(c, state) if c["mode"] == "step" else _plain_scan(c, state)


def _own(c, s):
    import gated_deltanet_chunked_rule_b200 as gdn

    if c["op"] == "norm":
        kw = {"center": c["center"], "gate_first": c["gate"] == "before"}
        y, stats = gdn.layer_norm_fwd(s["x"], s["weight"], s["bias"], s["gate"], 1e-5, **kw)
        out = {"y": y}
        if c["mode"] == "train":
            dx, dw, db, dg = gdn.layer_norm_bwd(s["x"], s["weight"], s["bias"], s["gate"], s["dy"], stats, 1e-5, **kw)
            out.update(dx=dx, dweight=dw, dbias=db, dgate=dg)
        return out
    if c["op"] == "conv":
        act = "silu" if c["act"] else None
        if c["mode"] == "step":
            y = gdn.causal_conv1d_update(s["x"], s["state"], s["weight"], s["bias"], act)
            return {"y": y, "state": s["state"]}
        y, fin = gdn.causal_conv1d_fwd(s["x"], s["weight"], s["bias"], act, s["state"], True, s["cu"])
        out = {"y": y, "final": fin}
        if c["mode"] == "train":
            dx, dw, db, ds = gdn.causal_conv1d_bwd(s["x"], s["weight"], s["bias"], s["dy"], s["dfinal"], act, s["state"],
                                                   s["cu"])
            out.update(dx=dx, dweight=dw, dbias=db, dstate=ds)
        return out
    a = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["D"], s["dt_bias"], True)
    if c["mode"] == "step":
        y, fin = gdn.recurrent_selective_scan(*a, s["h0"], final_state=s["h0"])
        return {"y": y, "state": fin}
    train = c["mode"] == "train"
    y, fin, saved = gdn.chunk_selective_scan_fwd(*a, s["h0"], True, s["cu"], save_for_backward=train)
    out = {"y": y, "final": fin}
    if train:
        g = gdn.chunk_selective_scan_bwd(*a, saved, s["dy"], s["dht"], s["h0"], s["cu"])
        out.update(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"), g))
        if s["h0"] is None:
            out["dh0"] = None
    return out


# ------------------------------------------------------------------ plain: norm
def _plain_norm(c, s):
    x, w = s["x"].float(), s["weight"].float()
    z = s["gate"].float() if c["gate"] else None
    sig = torch.sigmoid(z) if c["gate"] else None
    u = x * z * sig if c["gate"] == "before" else x
    if c["center"]:
        u = u - u.mean(-1, keepdim=True)
    rstd = torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-5)
    n = u * rstd
    lin = n * w + s["bias"].float() if c["bias"] else n * w
    y = lin * z * sig if c["gate"] == "after" else lin
    out = {"y": y.to(s["x"].dtype)}
    if c["mode"] != "train":
        return out
    dy = s["dy"].float()
    dlin = dy * z * sig if c["gate"] == "after" else dy
    out["dweight"] = (dlin * n).sum(0).to(s["weight"].dtype)
    out["dbias"] = dlin.sum(0).to(s["weight"].dtype) if c["bias"] else None
    dn = dlin * w
    du = dn - n * (dn * n).mean(-1, keepdim=True)
    if c["center"]:
        du = du - dn.mean(-1, keepdim=True)
    du = du * rstd
    out["dgate"] = None
    if c["gate"]:
        dsilu = sig * (1 + z * (1 - sig))
        out["dgate"] = ((dy * lin if c["gate"] == "after" else du * x) * dsilu).to(s["x"].dtype)
        if c["gate"] == "before":
            du = du * z * sig
    out["dx"] = du.to(s["x"].dtype)
    return out


# ------------------------------------------------------------------ plain: conv
def _plain_conv(c, s):
    """Every sequence's W-1 state rows and its inputs one after another on one axis:
    there the convolution is a sum of W shifted slices."""
    x, W, C = s["x"], c["W"], c["C"]
    w = s["weight"].float()
    dev, N = x.device, len(s["lens"])
    lens = torch.tensor(s["lens"], device=dev)
    end = torch.cumsum(lens + W - 1, 0)  # of each sequence on the joint axis
    total = x.shape[0] * x.shape[1]
    seq = torch.repeat_interleave(torch.arange(N, device=dev), lens, output_size=total)
    rows = torch.arange(total, device=dev) + (seq + 1) * (W - 1)  # each input's row
    last = end[:, None] - (W - 1) + torch.arange(W - 1, device=dev)  # each sequence's last W-1 rows
    head = (end - lens - (W - 1))[:, None] + torch.arange(W - 1, device=dev)
    buf = torch.zeros((total + N * (W - 1), C), device=dev)
    buf[rows] = x.reshape(-1, C).float()
    if s["state"] is not None:
        buf[head.reshape(-1)] = s["state"].reshape(-1, C).float()
    n = buf.shape[0]
    pre = sum(buf[j:n - (W - 1) + j] * w[:, j] for j in range(W))[rows - (W - 1)]
    if s["bias"] is not None:
        pre = pre + s["bias"].float()
    sig = torch.sigmoid(pre) if c["act"] else None
    y = pre * sig if c["act"] else pre
    out = {"y": y.to(x.dtype).view_as(x), "final": buf[last].to(x.dtype)}
    if c["mode"] != "train":
        return out
    dpre = s["dy"].reshape(-1, C).float()
    if c["act"]:
        dpre = dpre * sig * (1 + pre * (1 - sig))
    full = torch.zeros_like(buf)
    full[rows] = dpre
    out["dweight"] = torch.stack([(full[W - 1:] * buf[j:n - (W - 1) + j]).sum(0) for j in range(W)], 1).to(s["weight"].dtype)
    out["dbias"] = dpre.sum(0).to(x.dtype) if s["bias"] is not None else None
    tail = torch.cat([full, torch.zeros((W - 1, C), device=dev)])
    dbuf = sum(tail[W - 1 - j:n + W - 1 - j] * w[:, j] for j in range(W))
    dbuf = dbuf.index_add(0, last.reshape(-1), s["dfinal"].reshape(-1, C).float())
    out["dx"] = dbuf[rows].to(x.dtype).view_as(x)
    out["dstate"] = dbuf[head].to(x.dtype) if s["state"] is not None else None
    return out


def _plain_conv_step(c, s):
    joint = torch.cat([s["state"].float(), s["x"].float()], 1)
    y = (joint * s["weight"].float().t()).sum(1, keepdim=True)
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if c["act"]:
        y = y * torch.sigmoid(y)
    s["state"].copy_(joint[:, 1:])
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


# ------------------------------------------------------------------ plain: scan
_Q = 64  # tokens of a chunk


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(torch.clamp(v, max=20))))


def _plain_scan(c, s):
    train = c["mode"] == "train"
    names = [n for n in ("x", "dt", "A", "Bm", "Cm", "D", "dt_bias", "h0") if s[n] is not None]
    v = {n: s[n].float() for n in names}
    if train:
        v = {n: t.detach().requires_grad_() for n, t in v.items()}
    with torch.set_grad_enabled(train):
        y, fin = _chunked(c, s["lens"], v["x"], v["dt"], v["A"], v["Bm"], v["Cm"], v.get("D"), v["dt_bias"], v.get("h0"))
    out = {"y": y.detach().to(s["x"].dtype), "final": fin.detach()}
    if train:
        grads = torch.autograd.grad([y, fin], [v[n] for n in names], [s["dy"].float(), s["dht"]])
        got = {n: t.to(s[n].dtype) for n, t in zip(names, grads)}
        keys = {"x": "dx", "dt": "ddt", "A": "dA", "Bm": "dB", "Cm": "dC", "D": "dD", "dt_bias": "ddt_bias", "h0": "dh0"}
        out.update({o: got.get(n) for n, o in keys.items()})
    return out


def _chunked(c, lens, x, dt, A, Bm, Cm, D, dt_bias, h0):
    """The scan in chunks of 64 tokens, all chunks at once: products within a chunk, each
    chunk's own state, and the states carried from chunk to chunk by one matrix of decays."""
    H, G, K, P = c["H"], c["G"], c["K"], c["P"]
    dev, N = x.device, len(lens)
    ln = torch.tensor(lens, device=dev)
    start = torch.cumsum(ln, 0) - ln
    per = (ln + _Q - 1) // _Q
    nc = sum((v + _Q - 1) // _Q for v in lens)
    cseq = torch.repeat_interleave(torch.arange(N, device=dev), per, output_size=nc)
    local = torch.arange(nc, device=dev) - (torch.cumsum(per, 0) - per)[cseq]
    pos = local[:, None] * _Q + torch.arange(_Q, device=dev)
    live = pos < ln[cseq][:, None]
    tok = torch.where(live, start[cseq][:, None] + pos, 0)
    delta = _softplus(dt.reshape(-1, H) + dt_bias)
    dl = torch.where(live[..., None], delta[tok], 0.0)  # [nc, Q, H]
    xs = torch.where(live[..., None, None], x.reshape(-1, H, P)[tok], 0.0)
    bs = torch.where(live[..., None, None], Bm.reshape(-1, G, K)[tok], 0.0)
    cs = torch.where(live[..., None, None], Cm.reshape(-1, G, K)[tok], 0.0)
    gam = torch.cumsum(dl.double() * A.double(), 1).transpose(1, 2)  # [nc, H, Q]
    gap = (gam[..., :, None] - gam[..., None, :]).masked_fill(
        ~torch.ones((_Q, _Q), dtype=torch.bool, device=dev).tril(), -math.inf)
    S = torch.einsum("cqgk,csgk->cgqs", cs, bs).repeat_interleave(H // G, 1)
    w = xs * dl[..., None]  # D_s x_s
    y = torch.einsum("chqs,cshp->cqhp", S * torch.exp(gap).float(), w)
    tail = torch.exp(gam[..., -1:] - gam).float().transpose(1, 2)  # decay to the chunk's end
    bh = bs.repeat_interleave(H // G, 2)
    ch = cs.repeat_interleave(H // G, 2)
    own_state = torch.einsum("cshk,cshp->chkp", bh, w * tail[..., None]).flatten(2)
    # decay over the chunks between: total log decay before each chunk, within its sequence
    tot = gam[..., -1]  # [nc, H]
    upto = torch.cumsum(tot, 0)
    at = torch.cat([upto - tot, upto[-1:] if nc else upto.new_zeros((1, H))])  # before chunk c (and after the last)
    first = torch.cumsum(per, 0) - per
    ends = torch.cumsum(per, 0)
    rows = torch.cat([at[:nc], at[ends]])  # where states are wanted: each chunk's start, each sequence's end
    rseq = torch.cat([cseq, torch.arange(N, device=dev)])
    rpos = torch.cat([torch.arange(nc, device=dev), ends])
    ok = (rseq[:, None] == cseq[None, :]) & (torch.arange(nc, device=dev)[None, :] < rpos[:, None])
    M = torch.exp((rows[:, None] - upto[None]).masked_fill(~ok[..., None], -math.inf)).float()
    h = torch.einsum("rch,chf->rhf", M, own_state).view(nc + N, H, K, P)
    if h0 is not None:
        h = h + torch.exp(rows - at[first][rseq]).float()[..., None, None] * h0[rseq]
    y = y + torch.einsum("cqhk,chkp->cqhp", ch, h[:nc]) * torch.exp(gam).float().transpose(1, 2)[..., None]
    if D is not None:
        y = y + xs * D[:, None]
    return y.flatten(0, 1)[live.reshape(-1)].view(x.shape), h[nc:]


def _plain_scan_step(c, s):
    r = c["H"] // c["G"]
    delta = _softplus(s["dt"][:, 0].float() + s["dt_bias"])  # [B, H]
    b = s["Bm"][:, 0].float().repeat_interleave(r, 1)
    q = s["Cm"][:, 0].float().repeat_interleave(r, 1)
    x = s["x"][:, 0].float()
    h = torch.exp(delta * s["A"])[..., None, None] * s["h0"] + (delta[..., None] * b)[..., None] * x[:, :, None]
    y = (q[..., None] * h).sum(2)
    if s["D"] is not None:
        y = y + s["D"][:, None] * x
    s["h0"].copy_(h)
    return {"y": y[:, None].to(s["x"].dtype), "state": s["h0"]}


# ------------------------------------------------------------------------ exact
def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "norm":
        return _exact_norm(c, s)
    return _exact_conv(c, s) if c["op"] == "conv" else _exact_scan(c, s)


def _f64(t):
    return None if t is None else t.double()


def _exact_norm(c, s):
    names = [n for n in ("x", "weight", "bias", "gate") if s[n] is not None]
    v = {n: s[n].double().requires_grad_() for n in names}

    def silu(t):
        return t / (1 + torch.exp(-t))

    u = v["x"] * silu(v["gate"]) if c["gate"] == "before" else v["x"]
    mean = u.sum(-1, keepdim=True) / c["D"] if c["center"] else 0.0
    var = ((u - mean) ** 2).sum(-1, keepdim=True) / c["D"]
    y = (u - mean) / torch.sqrt(var + 1e-5) * v["weight"]
    if c["bias"]:
        y = y + v["bias"]
    if c["gate"] == "after":
        y = y * silu(v["gate"])
    out = {"y": y.detach()}
    if c["mode"] == "train":
        g = dict(zip(names, torch.autograd.grad(y, [v[n] for n in names], s["dy"].double())))
        out.update(dx=g["x"], dweight=g["weight"], dbias=g.get("bias"), dgate=g.get("gate"))
    return out


def _exact_conv(c, s):
    """Sequence by sequence, tap by tap."""
    W, C = c["W"], c["C"]
    w, b = s["weight"].double(), _f64(s["bias"])
    lens = s["lens"] if c["mode"] != "step" else [1] * c["B"]
    x = s["x"].reshape(-1, C).double()
    y, fin = torch.empty_like(x), []
    dx, dstate = torch.zeros_like(x), []
    dw, db = torch.zeros_like(w), torch.zeros(C, dtype=torch.float64, device=x.device)
    at = 0
    for n, ln in enumerate(lens):
        past = s["state"][n].double() if s["state"] is not None else torch.zeros((W - 1, C), dtype=torch.float64, device=x.device)
        seen = torch.cat([past, x[at:at + ln]])
        pre = torch.zeros((ln, C), dtype=torch.float64, device=x.device)
        for j in range(W):
            pre += w[:, j] * seen[j:j + ln]
        if b is not None:
            pre += b
        y[at:at + ln] = pre / (1 + torch.exp(-pre)) if c["act"] else pre
        fin.append(seen[ln:])
        if c["mode"] == "train":
            d = s["dy"].reshape(-1, C)[at:at + ln].double()
            if c["act"]:
                e = 1 / (1 + torch.exp(-pre))
                d = d * (e + pre * e * (1 - e))
            dseen = torch.zeros_like(seen)
            dseen[ln:] += s["dfinal"][n].double()
            for j in range(W):
                dseen[j:j + ln] += w[:, j] * d
                dw[:, j] += (d * seen[j:j + ln]).sum(0)
            db += d.sum(0)
            dx[at:at + ln] = dseen[W - 1:]
            dstate.append(dseen[:W - 1])
        at += ln
    out = {"y": y.view(s["x"].shape), ("state" if c["mode"] == "step" else "final"): torch.stack(fin)}
    if c["mode"] == "train":
        out.update(dx=dx.view(s["x"].shape), dweight=dw, dbias=db if b is not None else None,
                   dstate=torch.stack(dstate) if s["state"] is not None else None)
    return out


def _exact_scan(c, s):
    """Token by token, every sequence at once; the gradients by the reverse recurrence."""
    H, G, K, P = c["H"], c["G"], c["K"], c["P"]
    lens = s["lens"] if c["mode"] != "step" else [1] * c["B"]
    N, L = len(lens), max(lens)
    dev = s["x"].device
    ln = torch.tensor(lens, device=dev)
    pos = torch.arange(L, device=dev)
    live = pos[None] < ln[:, None]  # [N, L]
    tok = (torch.cumsum(ln, 0) - ln)[:, None] + pos
    flat = tok[live]

    def padded(t, *shape):
        o = torch.zeros((N, L) + shape, dtype=torch.float64, device=dev)
        o[live] = t.reshape((-1,) + shape).double()[flat]
        return o.transpose(0, 1).contiguous()

    x, q, b = padded(s["x"], H, P), padded(s["Cm"], G, K), padded(s["Bm"], G, K)
    raw = padded(s["dt"], H) + s["dt_bias"].double()
    delta = torch.where(live.t()[..., None], torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())), 0.0)
    A = s["A"].double()
    a = torch.exp(delta * A)
    r = H // G
    D = _f64(s["D"])
    zero = torch.zeros((N, H, K, P), dtype=torch.float64, device=dev)
    h = zero.clone() if s["h0"] is None else s["h0"].double()
    train = c["mode"] == "train"
    dy = padded(s["dy"], H, P) if train else None
    y, dq = torch.empty_like(x), torch.zeros((L, N, H, K), dtype=torch.float64, device=dev)
    dx_ = delta[..., None] * x
    for t in range(L):
        bt = b[t].repeat_interleave(r, 1)
        h = a[t][..., None, None] * h + bt[..., None] * dx_[t][:, :, None]
        y[t] = torch.matmul(q[t].repeat_interleave(r, 1)[:, :, None], h)[:, :, 0]
        if train:
            dq[t] = torch.matmul(h, dy[t][..., None])[..., 0]

    def back(t):
        o = torch.empty((sum(lens),) + t.shape[2:], dtype=torch.float64, device=dev)
        o[flat] = t.transpose(0, 1)[live]
        return o

    ys = y if D is None else y + D[:, None] * x
    out = {"y": back(ys).view(s["x"].shape), ("state" if c["mode"] == "step" else "final"): h}
    if not train:
        return out
    g = s["dht"].double()
    # log-decay gradients: with r_t = C_t.dC_t and w_t = B_t.dB_t (each head's own), dg_t = dg_{t+1} + r_t - w_t
    carry = (h * g).sum((-1, -2))
    db, dx, ddl = torch.zeros_like(dq), torch.empty_like(x), torch.empty_like(delta)
    for t in range(L - 1, -1, -1):
        # a sequence's state gradient only begins at its own last token; beyond it a = 1 and dy = 0
        qt, bt = q[t].repeat_interleave(r, 1), b[t].repeat_interleave(r, 1)
        g = g + qt[..., None] * dy[t][:, :, None]
        u = torch.matmul(bt[:, :, None], g)[:, :, 0]
        direct = (u * x[t]).sum(-1)
        dx[t] = delta[t][..., None] * u
        db[t] = torch.matmul(g, dx_[t][..., None])[..., 0]
        carry = carry + (qt * dq[t]).sum(-1) - delta[t] * direct
        ddl[t] = A * carry + direct
        raw[t] = carry * delta[t]  # now delta_t dg_t, for dA
        g = a[t][..., None, None] * g
    m = live.t()[..., None]
    rawdt = padded(s["dt"], H) + s["dt_bias"].double()
    ddt = torch.where(m, ddl / (1 + torch.exp(-rawdt)), 0.0)
    out["dA"] = torch.where(m, raw, 0.0).sum((0, 1))
    out["ddt"] = back(ddt).view(s["dt"].shape)
    out["ddt_bias"] = ddt.sum((0, 1))
    out["dx"] = back(dx if D is None else dx + D[:, None] * dy).view(s["x"].shape)
    out["dB"] = back(db.unflatten(2, (G, r)).sum(3)).view(s["Bm"].shape)
    out["dC"] = back(dq.unflatten(2, (G, r)).sum(3)).view(s["Cm"].shape)
    out["dD"] = (x * dy).sum((0, 1, 3)) if D is not None else None
    out["dh0"] = g if s["h0"] is not None else None
    return out


# ------------------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once; the recurrences' own operations."""
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    train = c["mode"] == "train"
    if c["op"] == "norm":
        el = c["R"] * c["D"]
        tensors = 2 + (1 if c["gate"] else 0) + ((2 + (1 if c["gate"] else 0)) if train else 0)
        return {"bytes": tensors * el * e, "flops": el * (8 + (20 if train else 0))}
    N = len(_lengths(c))
    tokens = c["B"] * c["T"]
    if c["op"] == "conv":
        el, st = tokens * c["C"], N * (c["W"] - 1) * c["C"]
        states = (1 if c["state"] else 0) + 1 + ((1 + (1 if c["state"] else 0)) if train else 0)
        by = (2 + (2 if train else 0)) * el * e + states * st * e + c["C"] * c["W"] * e * (2 if train else 1)
        return {"bytes": by, "flops": el * (2 * c["W"] + 6) * (3 if train else 1)}
    H, G, K, P = c["H"], c["G"], c["K"], c["P"]
    ed = 2 if c["dt"] == "bf16" else 4
    row = H * P * e + 2 * G * K * e + H * ed  # x, B, C, dt of a token
    st = N * H * K * P * 4
    states = (1 if c["state"] else 0) + 1 + ((1 + (1 if c["state"] else 0)) if train else 0)
    by = tokens * (row + H * P * e) + states * st
    if train:
        by += tokens * (H * P * e + row)  # dy in; dx, dB, dC, ddt out
    return {"bytes": by, "flops": tokens * H * K * P * (5 + (10 if train else 0))}
