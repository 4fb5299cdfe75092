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
