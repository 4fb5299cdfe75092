"""Convolution and norm gradients in calls in a row, whose second kernels come up while the first ones run, and
the layers' fp32 precision."""
import pytest
import torch

import test_mixer_gpu as M

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


def in_a_row(call, inputs, n=24):
    alone = []
    for v in inputs:
        alone.append(call(v))
        torch.cuda.synchronize()
    got = [call(inputs[i % len(inputs)]) for i in range(n)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for p, q in zip(g, alone[i % len(inputs)]):
            assert (p is None and q is None) or torch.equal(p, q), i


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,C", [(300, 40), (2000, 2056), (40, 37)])
def test_convolution_gradients_in_a_row(gdn, dtype, T, C):
    g = torch.Generator().manual_seed(C)

    def r(*s):
        return torch.randn(s, generator=g).to(DT[dtype]).cuda()

    inputs = [(r(2, T, C), r(C, 4), r(C), r(2, T, C), r(2, 3, C), "silu", r(2, 3, C)) for _ in range(2)]
    in_a_row(lambda v: gdn.causal_conv1d_bwd(*v), inputs)
    assert gdn.device_status() == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,D", [(5000, 128), (700, 4096), (300, 33)])
@pytest.mark.parametrize("form", ["none", "first", "last"])
def test_norm_gradients_in_a_row(gdn, dtype, rows, D, form):
    g = torch.Generator().manual_seed(D)

    def r(*s):
        return torch.randn(s, generator=g).to(DT[dtype]).cuda()

    inputs = [(r(rows, D), r(D), r(D), r(rows, D) if form != "none" else None, r(rows, D)) for _ in range(2)]

    def call(v):
        x, w, b, z, dy = v
        y, st = gdn.layer_norm_fwd(x, w, b, z, 1e-5, True, form == "first")
        return y, *gdn.layer_norm_bwd(x, w, b, z, dy, st, 1e-5, True, form == "first")

    in_a_row(call, inputs)


@pytest.mark.parametrize("kind", ["scan", "delta"])
@pytest.mark.parametrize("lens", [[70], [1, 33, 0, 130, 5]])
def test_layer_keeps_fp32(gdn, kind, lens):
    """Norms of test_mixer_gpu.py's chain in fp32 against 64 bits. An operator rounds each term up to
    T + 512 + 17 * 128 times in sequence, independently, so by sqrt of that 2^-24; the terms' signs are as random
    as the errors', so a sum's relative error is no larger than its terms'; three operators forward and three
    back amplify it at most twice each. That is 4e-5: an operand rounded to bf16 (2^-9 / sqrt(3) rms) or
    to 11 bits (2^-12 / sqrt(3)) does not pass."""
    tol = 6 * 2 * (sum(lens) + 512 + 17 * 128) ** 0.5 * 2.0 ** -24
    assert tol < 2.0 ** -12 / 3 ** 0.5
    p = M.params(kind, sum(lens), torch.float32, seed=5)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() if len(lens) > 1 else None
    leaves = M.on_gpu(p, torch.float32, True)
    out = M.chain(gdn, kind, leaves, cu)
    w = torch.randn(out.shape, generator=torch.Generator().manual_seed(6)).double()
    w = w.float().double()
    out.backward(w.float().cuda())
    ref = {k: t.clone().requires_grad_(True) for k, t in p.items()}
    want = M.plain(kind, ref, lens)
    want.backward(w)
    offs = {"out": M.off(out, want.detach()), **{k: M.off(leaves[k].grad, ref[k].grad) for k in p}}
    print({k: f"{e:.1e}" for k, e in offs.items()}, f"of {tol:.1e}")
    for k, e in offs.items():
        assert e <= tol, (k, e)
