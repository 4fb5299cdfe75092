"""The layer operators where calls meet: on two streams at once, in graphs that are captured through autograd and
replayed in turn, and beside each other's workspaces."""
import pytest
import torch

import test_mixer_gpu as M
import test_scan_gpu as S

pytestmark = pytest.mark.gpu
DT = S.DT


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_rule_b200 import build
    build.build()
    import gated_deltanet_chunked_rule_b200 as g
    return g


def layer(gdn, p, cu):
    """Output and gradients of every leaf."""
    out = M.chain(gdn, "scan", p, cu)
    names = list(p)
    return [out.detach(), *torch.autograd.grad(out.float().square().sum(), [p[k] for k in names])]


def leaves(lens, dtype, seed):
    p = M.on_gpu(M.params("scan", sum(lens), dtype, seed), dtype, True)
    return p, torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_two_streams_at_once(gdn, dtype):
    work = [leaves([700, 0, 333, 5], dtype, 1), leaves([129, 640], dtype, 2)]
    want = [layer(gdn, *w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = [[] for _ in work]
    for _ in range(6):  # the calls of both in turn, nothing waits
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(layer(gdn, *work[i]))
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    for i, runs in enumerate(got):
        for run in runs:
            for p, q in zip(run, want[i]):
                assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_two_captured_layers(gdn, dtype):
    # forward and gradients captured through autograd, two graphs on one memory pool, replayed in turn; the
    # second's results are read before the first, which shares its pool, runs again
    lens = [300, 0, 77]
    work = [leaves(lens, dtype, s) for s in (3, 4)]
    want = [layer(gdn, *w) for w in work]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for w in work:
            layer(gdn, *w)
    torch.cuda.current_stream().wait_stream(side)
    pool = torch.cuda.graph_pool_handle()
    graphs, outs = [], []
    for w in work:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(layer(gdn, *w))
        graphs.append(g)
    for _ in range(3):
        for g, out, exp in zip(graphs, outs, want):
            for t in out:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            for p, q in zip(out, exp):
                assert torch.equal(p, q)
    assert gdn.device_status() == 0


def test_beside_the_delta_rule(gdn):
    # the delta rule's tensor-core kernels on one stream, the scan's on another
    p, cu = leaves([900, 124], torch.bfloat16, 5)
    g = torch.Generator().manual_seed(6)
    r = lambda *s, d=torch.bfloat16: torch.randn(s, generator=g).to(d).cuda()  # noqa: E731
    q, k, v = r(1, 1024, 2, 128), torch.nn.functional.normalize(r(1, 1024, 2, 128), dim=-1), r(1, 1024, 4, 128)
    gate, beta = -r(1, 1024, 4, d=torch.float32).abs(), torch.sigmoid(r(1, 1024, 4, d=torch.float32))
    cu_host = cu.cpu()

    def delta():
        o, fin, saved = gdn.chunk_gated_delta_rule_fwd(q, k, v, gate, beta, 0.1, None, True, cu, cu_host, True)
        return [o, fin, *gdn.chunk_gated_delta_rule_bwd(q, k, v, gate, beta, saved, o, fin, 0.1, None, cu, cu_host)]

    calls = [delta, lambda: layer(gdn, p, cu)]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(calls[i]())
    torch.cuda.synchronize()
    assert gdn.device_status() == 0
    for i, runs in enumerate(got):
        for run in runs:
            for a, b in zip(run, want[i]):
                assert torch.equal(a, b), i
