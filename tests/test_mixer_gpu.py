"""The operators together, as a layer runs them: the short convolution in front of a recurrence
(the selective scan, or the gated delta rule), the gated norm behind it; prompts with every
gradient, then single tokens on the states that the prompt left, captured into a graph.

Tolerances are of norms (|got - ref| / |ref|), against the same chain in 64 bits:
  - fp32: an operator's results are within (T + 512 + 17 * 128) 2^-24 of their terms' mass (the
    operators' own tests), at most 1.7e-4 here; three operators forward and three back, and a sum
    of n terms of random sign has a mass of about sqrt(n) times its size, n <= 256: 16 * 6 * 1.7e-4;
  - bf16: half a step, 2^-8, for each result that is rounded (the convolution's, one operand of the
    recurrence's products, its output, the norm's output, and the same four of the gradients on the
    way back), each amplified at most twice (silu, norm and gate; the recurrence decays)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
F = torch.nn.functional
TOL = {torch.float32: 16 * 6 * 1.7e-4, torch.bfloat16: 2 * 8 * 2.0 ** -8}


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_rule_b200 import build
    build.build()
    import gated_deltanet_chunked_rule_b200 as g
    return g


H, G, K, V, W = 4, 2, 64, 64, 4


def params(kind, T, dtype, seed=0):
    """Leaves on the CPU in 64 bits, at values that `dtype` holds."""
    g = torch.Generator().manual_seed(seed)

    def r(*s, std=1.0, dt=dtype):
        return (torch.randn(s, generator=g) * std).to(dt).double()

    C = H * V + 2 * G * K
    p = dict(u=r(1, T, C), cw=r(C, W, std=0.5), cb=r(C, std=0.1), z=r(1, T, H, V), nw=1 + r(V, std=0.1, dt=torch.float32),
             a=r(1, T, H), A=-(torch.rand(H, generator=g) + 0.5).double().float().double())
    if kind == "scan":
        p |= dict(D=r(H, dt=torch.float32), bias=r(H, std=0.3, dt=torch.float32))
    else:
        p |= dict(b=r(1, T, H))
    return p


def split(c):
    q, k, v = c.split([G * K, G * K, H * V], -1)
    return q.unflatten(-1, (G, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (H, V))


def chain(gdn, kind, p, cu=None):
    """The layer on the GPU: its output."""
    c, _ = gdn.causal_conv1d(p["u"], p["cw"], p["cb"], "silu", cu_seqlens=cu)
    q, k, v = split(c)
    if kind == "scan":
        o, _ = gdn.chunk_selective_scan(v, p["a"], p["A"], k, q, p["D"], p["bias"], True, cu_seqlens=cu)
    else:
        q, k = F.normalize(q, dim=-1), F.normalize(k, dim=-1)
        o, _ = gdn.chunk_gated_delta_rule(q, k, v, F.softplus(p["a"].float()) * p["A"], torch.sigmoid(p["b"]).float(), cu_seqlens=cu)
    return gdn.layer_norm(o, p["nw"], gate=p["z"], center=False)


def plain(kind, p, lens):
    """The same in plain operations, token by token."""
    out = []
    t0 = 0
    for n in lens:
        u = F.pad(p["u"][0, t0:t0 + n], (0, 0, W - 1, 0))
        pre = p["cb"] + sum(u[j:j + n] * p["cw"][:, j] for j in range(W))
        q, k, v = split(F.silu(pre))
        a = p["a"][0, t0:t0 + n]
        S, rows = torch.zeros(H, K, V, dtype=torch.float64), []
        q, k = (t.repeat_interleave(H // G, 1) for t in (q, k))
        if kind == "scan":
            dt = F.softplus(a + p["bias"])
            for t in range(n):
                S = torch.exp(dt[t] * p["A"])[:, None, None] * S + k[t][:, :, None] * (dt[t][:, None] * v[t])[:, None]
                rows.append(torch.einsum("hk,hkv->hv", q[t], S) + p["D"][:, None] * v[t])
        else:
            q, k = F.normalize(q, dim=-1), F.normalize(k, dim=-1)
            g, beta = F.softplus(a) * p["A"], torch.sigmoid(p["b"][0, t0:t0 + n])
            for t in range(n):
                S = torch.exp(g[t])[:, None, None] * S
                d = beta[t][:, None] * (v[t] - torch.einsum("hk,hkv->hv", k[t], S))
                S = S + k[t][:, :, None] * d[:, None]
                rows.append(torch.einsum("hk,hkv->hv", q[t], S) * K ** -0.5)
        if n:
            o = torch.stack(rows)
            y = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + 1e-5) * p["nw"]
            out.append(y * F.silu(p["z"][0, t0:t0 + n]))
        t0 += n
    return torch.cat(out)[None]


def off(got, ref):
    return ((got.detach().cpu().double() - ref).norm() / ref.norm()).item()


def on_gpu(p, dtype, grad):
    f32 = ("A", "D", "bias", "nw")
    return {k: v.to(torch.float32 if k in f32 else dtype).cuda().requires_grad_(grad) for k, v in p.items()}


@pytest.mark.parametrize("kind", ["scan", "delta"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens", [[70], [1, 33, 0, 130, 5]])
def test_layer_and_gradients(gdn, kind, dtype, lens):
    p = params(kind, sum(lens), dtype)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() if len(lens) > 1 else None
    leaves = on_gpu(p, dtype, True)
    out = chain(gdn, kind, leaves, cu)
    w = torch.randn(out.shape, generator=torch.Generator().manual_seed(1)).to(dtype).double()
    out.backward(w.to(dtype).cuda())
    ref = {k: v.clone().requires_grad_(True) for k, v in p.items()}
    want = plain(kind, ref, lens)
    want.backward(w)
    assert off(out, want.detach()) <= TOL[dtype]
    # the gates' gradients are sums over whole rows of terms of either sign: in fp32 only
    for k in p if dtype == torch.float32 else ("u", "cw", "cb", "z", "nw"):
        assert off(leaves[k].grad, ref[k].grad) <= TOL[dtype], k


@pytest.mark.parametrize("kind", ["scan", "delta"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens_after_a_prompt(gdn, kind, dtype):
    """A prompt, then single tokens by one captured step, equal the prompt of them all."""
    T, n = 37, 6
    p = on_gpu(params(kind, T + n, dtype), dtype, False)
    want = chain(gdn, kind, p)
    head = {k: v[:, :T].contiguous() if v.dim() >= 3 else v for k, v in p.items()}
    c, conv_state = gdn.causal_conv1d(head["u"], p["cw"], p["cb"], "silu", output_final_state=True)
    q, k, v = split(c)

    def gates(x):
        return F.softplus(x["a"].float()) * p["A"], torch.sigmoid(x["b"]).float()

    if kind == "scan":
        _, state = gdn.chunk_selective_scan(v, head["a"], p["A"], k, q, p["D"], p["bias"], True, output_final_state=True)
    else:
        _, state = gdn.chunk_gated_delta_rule(F.normalize(q, dim=-1), F.normalize(k, dim=-1), v, *gates(head),
                                              output_final_state=True)
    tok = {k: v[:, :1].clone() for k, v in p.items() if v.dim() >= 3}

    def step():
        c = gdn.causal_conv1d_update(tok["u"], conv_state, p["cw"], p["cb"], "silu")
        q, k, v = split(c)
        if kind == "scan":
            o, _ = gdn.recurrent_selective_scan(v, tok["a"], p["A"], k, q, p["D"], p["bias"], True, state, final_state=state)
        else:
            o, _ = gdn.recurrent_gated_delta_rule(F.normalize(q, dim=-1), F.normalize(k, dim=-1), v, *gates(tok),
                                                  initial_state=state, final_state=state)
        return gdn.layer_norm(o, p["nw"], gate=tok["z"], center=False)

    kept = conv_state.clone(), state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    conv_state.copy_(kept[0])
    state.copy_(kept[1])
    for t in range(T, T + n):
        for name in tok:
            tok[name].copy_(p[name][:, t:t + 1])
        graph.replay()
        assert off(out, want[:, t:t + 1].cpu().double()) <= TOL[dtype], t
