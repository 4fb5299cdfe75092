"""What the high-level calls do where autograd could be passed by: forward-mode tangents, and states written
in place."""
import pytest
import torch
import torch.autograd.forward_ad as fwad

import test_mixer_gpu as M
import test_scan_gpu as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_rule_b200 import build
    build.build()
    import gated_deltanet_chunked_rule_b200 as g
    return g


def calls(gdn):
    """The high-level calls, each a function of one tensor of its inputs."""
    p = M.on_gpu(M.params("delta", 40, torch.float32), torch.float32, False)
    v = S.make([40], 2, 1, 64, 64, torch.float32, seed=2)
    q, k, w = M.split(p["u"])
    g, beta = torch.nn.functional.softplus(p["a"]) * p["A"], torch.sigmoid(p["b"])
    return {
        "conv": (lambda t: gdn.causal_conv1d(p["u"], t, p["cb"], "silu")[0], p["cw"]),
        "scan": (lambda t: gdn.chunk_selective_scan(v["x"], v["dt"], t, v["B"], v["C"], v["D"], v["dt_bias"], True)[0], v["A"]),
        "norm": (lambda t: gdn.layer_norm(p["z"], t, gate=w, center=False), p["nw"]),
        "delta": (lambda t: gdn.chunk_gated_delta_rule(q.contiguous(), k.contiguous(), t, g, beta)[0], w.contiguous()),
    }


@pytest.mark.parametrize("name", ["conv", "scan", "norm", "delta"])
def test_tangents_are_refused(gdn, name):
    f, t = calls(gdn)[name]
    want = f(t)
    with fwad.dual_level():
        assert torch.equal(f(t), want)  # no tangent: as ever
        for grad in (True, False):
            with torch.set_grad_enabled(grad), pytest.raises(NotImplementedError, match="jvp"):
                f(fwad.make_dual(t, torch.ones_like(t)))
    assert torch.equal(f(t), want)


def graph_and_step(gdn, name):
    """(a graph that saved a state, a step that writes that state)."""
    p = M.on_gpu(M.params("delta", 9, torch.float32), torch.float32, False)
    v = S.make([9], 2, 1, 64, 64, torch.float32, seed=2, packed=False)
    if name == "conv":
        state = torch.zeros(1, M.W - 1, p["u"].shape[2], device="cuda")
        u = p["u"].clone().requires_grad_()
        out = gdn.causal_conv1d(u, p["cw"], p["cb"], "silu", state)[0]
        return out, u, lambda: gdn.causal_conv1d_update(p["u"][:, :1].contiguous(), state, p["cw"], p["cb"], "silu")
    if name == "scan":
        state, x = v["h0"].clone(), v["x"].clone().requires_grad_()
        a = S.args(v)
        out = gdn.chunk_selective_scan(x, *a[1:], True, state)[0]
        one = [t[:, :1] if t is not None and t.dim() > 1 else t for t in a]
        return out, x, lambda: gdn.recurrent_selective_scan(*one, True, state, state)
    q, k, w = (t.contiguous() for t in M.split(p["u"]))
    g, beta = torch.nn.functional.softplus(p["a"]) * p["A"], torch.sigmoid(p["b"])
    state, x = torch.zeros(1, M.H, M.K, M.V, device="cuda"), w.clone().requires_grad_()
    out = gdn.chunk_gated_delta_rule(q, k, x, g, beta, initial_state=state)[0]
    one = [t[:, :1].contiguous() for t in (q, k, w, g, beta)]
    if name == "delta":
        return out, x, lambda: gdn.recurrent_gated_delta_rule(*one, initial_state=state, final_state=state)
    # an output of the caller's own: the memory of v, which the graph saved, given back to another call
    other = torch.randn_like(w)
    if name == "step's out":
        return out, x, lambda: gdn.recurrent_gated_delta_rule(q, k, other, g, beta, out=x.detach())
    return out, x, lambda: gdn.chunk_gated_delta_rule_fwd(q, k, other, g, beta, 1.0, out=x.detach())


@pytest.mark.parametrize("name", ["conv", "scan", "delta", "step's out", "prompt's out"])
@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_states_written_in_place_are_noticed(gdn, name, mode):
    out, x, step = graph_and_step(gdn, name)
    torch.autograd.grad(out.sum(), x, retain_graph=True)
    with mode():
        step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(out.sum(), x)
