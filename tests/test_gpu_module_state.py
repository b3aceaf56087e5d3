"""What the modules keep between calls: AWQLinear's bf16 copy of its bias (a first call
that is captured, a bias changed under a captured call, first calls on two streams
at once) and SVDQLinear's workspace; and two host threads at once."""

import threading

import pytest
import torch

from tests.test_gpu_w4a16_modules import linear
from w4a4_quantized_diffusion_amd import linear as L

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
N, K = 256, 128


def layer():
    """(a biased layer, its values on x, x); the library is loaded and warm."""
    mod = L.AWQLinear.from_linear(linear(K, N, 1))
    warm = L.AWQLinear.from_linear(linear(K, N, 1))
    x = torch.randn(4, K, device="cuda").to(BF)
    y = warm(x)
    torch.cuda.synchronize()
    return mod, y, x


def test_first_call_captured():
    """A layer whose first call is captured gives an eager call, before any replay,
    its own bias, and follows a bias changed between replays."""
    mod, y, x = layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mod(x)
    assert torch.equal(mod(x), y)
    for i in range(3):
        with torch.no_grad():
            mod.bias.mul_(0.5 if i else 1.0)
        eager = mod(x)
        fill = [torch.full((N,), 9.0, dtype=BF, device="cuda") for _ in range(16)]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), i
        del fill


def test_a_captured_call_after_an_eager_one():
    """The same with an eager call in front, which has left a copy of the bias."""
    mod, y, x = layer()
    assert torch.equal(mod(x), y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mod(x)
    for i in range(3):
        with torch.no_grad():
            mod.bias.add_(1.0)
        eager = mod(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and not torch.equal(eager, y), i


def test_first_calls_on_two_streams():
    """The second stream does not read a copy that the first has yet to write."""
    mod, y, x = layer()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(a):
        torch.cuda._sleep(20_000_000)            # some ms in front of the first call
        ya = mod(x)
    with torch.cuda.stream(b):
        yb = mod(x)
    torch.cuda.synchronize()
    assert torch.equal(ya, y) and torch.equal(yb, y)


@pytest.mark.parametrize("first", ["eager", "captured"])
@pytest.mark.parametrize("gelu", [False, True])
def test_captured_svdq_calls_share_nothing(first, gelu):
    """Two captured calls of one SVDQLinear, replayed beside eager calls on more rows:
    they keep their own workspaces, and write to nothing else."""
    a = L.SVDQLinear.from_linear(linear(512, 272, 9), rank=16, gelu_input=gelu)
    ref = L.SVDQLinear.from_linear(linear(512, 272, 9), rank=16, gelu_input=gelu)
    xs = [torch.randn(m, 512, device="cuda").to(BF) for m in (100, 200)]
    big = torch.randn(900, 512, device="cuda").to(BF)
    want = [ref(x) for x in xs + [big]]
    if first == "eager":
        assert torch.equal(a(xs[0]), want[0])
    torch.cuda.synchronize()
    outs, graphs = [], [torch.cuda.CUDAGraph() for _ in xs]
    for g, x in zip(graphs, xs):
        with torch.cuda.graph(g):
            outs.append(a(x))
    yb = a(big)
    assert torch.equal(yb, want[2])
    fill = [torch.full((n,), 5.0, device="cuda") for n in (64, 1024, 4096, 16384, 1 << 18) * 4]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(3):
        for y in outs:
            y.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        assert torch.equal(a(big), want[2])
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(outs, want))
    assert all((t == 5.0).all() for t in fill)


def test_two_host_threads():
    """Calls of two host threads on streams of their own: the same kernels with more
    and with less LDS at once."""
    from tests.test_gpu_w4a16 import awq_layer, bf, svdq_layer
    from w4a4_quantized_diffusion_amd import svdq

    d, _ = svdq_layer(256, 4096, 16, "int4", 61)
    lay, _ = awq_layer(4096, 512, 62)
    jobs = []
    for m in (49, 64):
        x, dy = bf((m, 4096), 63), bf((m, 4096), 64)
        jobs.append(lambda x=x, dy=dy: (svdq.svdq_linear_w4a16(x, d), svdq.awq_linear_w4a16_grad(dy, lay)))
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    bad = []

    def work(job, ref):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    out = job()
                torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(out, ref)):
                bad.append("differs")
        except Exception as e:                   # a thread's failure is the test's
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(jobs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
