"""The modules around a block's 4-bit layers as they are used together: a modulated
transformer block trained in front of frozen AWQ layers, and a layer of experts, against
the same formulas in float64 on the layers' own weights.

Tolerance of a chain: every bf16 rounding between two layers (at most eight on any path
here, forward and backward together) is off by 2^-8 of a value at most, and enters the
result with a gain of the order of one (weights of standard deviation 1 / sqrt(K), norms,
slopes up to 1.13): 16 x 2^-8 in relative norm.  A missing or wrong term is of the order
of one."""

import pytest
import torch
from torch import nn

from w4a4_quantized_diffusion_amd import linear as L
from w4a4_quantized_diffusion_amd import svdq
from tests.test_gpu_moe import experts, weight

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
CHAIN = 16 * 2.0 ** -8


def randn(*shape, seed, std=1.0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def linear(k, n, seed, bias=True):
    lin = nn.Linear(k, n, bias=bias, device="cuda")
    with torch.no_grad():
        lin.weight.copy_(randn(n, k, seed=seed, std=k ** -0.5))
        if bias:
            lin.bias.copy_(randn(n, seed=seed + 1, std=0.1))
    return lin


def weight64(m):
    lay = dict(E=1, N=m.out_features, K=m.in_features, group=64, q=m.q[None], scales=m.scales[None],
               zeros=m.zeros[None])
    return weight(lay, 0)


def close(got, ref, what, tol=CHAIN):
    err = float((got.detach().double() - ref.detach()).norm() / ref.detach().norm())
    assert err <= tol, (what, err)


class Block(nn.Module):
    def __init__(self, d, hidden, seed):
        super().__init__()
        self.norm1 = L.BlockNorm(d, "layer")
        self.norm2 = L.BlockNorm(d, "layer", post=randn(d, seed=seed + 9, std=0.2) + 1)
        self.attn = L.AWQLinear.from_linear(linear(d, d, seed))
        self.up = L.AWQLinear.from_linear(linear(d, hidden, seed + 2))
        self.down = L.AWQLinear.from_linear(linear(hidden, d, seed + 4, bias=False))

    def forward(self, x, mod):
        m = mod.chunk(6, dim=-1)
        a = self.attn(self.norm1(x, scale=m[0], shift=m[1]))
        x, y = self.norm2(x, a, gate=m[2], scale=m[3], shift=m[4])
        return self.down(self.up(y, act="gelu"), gate=m[5], residual=x)

    def reference(self, x, mod, post):
        m = [v.unsqueeze(1) for v in mod.chunk(6, dim=-1)]
        ln = lambda v: nn.functional.layer_norm(v, v.shape[-1:], eps=1e-6)  # noqa: E731
        lin = lambda l, v: v @ weight64(l).t() + (  # noqa: E731
            0 if l.bias is None else l.bias.to(BF).double())
        a = lin(self.attn, ln(x) * (1 + m[0]) + m[1])
        x = x + m[2] * (ln(a) * post)
        u = nn.functional.gelu(lin(self.up, ln(x) * (1 + m[3]) + m[4]), approximate="tanh")
        return x + m[5] * lin(self.down, u)


@pytest.mark.parametrize("images,tokens,xt", [(1, 1, F32), (2, 30, F32), (3, 120, BF), (2, 700, F32)])
def test_block(images, tokens, xt):
    d = 256
    net = Block(d, 1024, 5)
    x = randn(images, tokens, d, seed=1).to(xt).requires_grad_()
    mod = randn(images, 6 * d, seed=2, std=0.5).requires_grad_()
    v = randn(images, tokens, d, seed=3)
    y = net(x, mod)
    assert y.dtype == xt and y.shape == x.shape
    got = torch.autograd.grad((y.float() * v).sum(), [x, mod, net.norm2.post])
    x64, mod64, post64 = (t.detach().double().requires_grad_() for t in (x, mod, net.norm2.post))
    ref = net.reference(x64, mod64, post64)
    want = torch.autograd.grad((ref * v.double()).sum(), [x64, mod64, post64])
    close(y, ref, "y")
    for g, w, p, n in zip(got, want, (x, mod, net.norm2.post), ("x", "mod", "post")):
        assert g.dtype == p.dtype and g.shape == p.shape
        close(g, w, n)
    with torch.no_grad():
        assert torch.equal(net(x, mod), y)


def test_block_gradients_by_differences():
    """The loss's change along the gradient's direction, by central differences of the
    float64 reference."""
    d = 128
    net = Block(d, 256, 8)
    x, mod = randn(2, 9, d, seed=1), randn(2, 6 * d, seed=2, std=0.5).requires_grad_()
    v = randn(2, 9, d, seed=3)
    g, = torch.autograd.grad((net(x, mod) * v).sum(), mod)
    step = 1e-5 * g.double() / g.double().norm()
    post = net.norm2.post.detach().double()
    with torch.no_grad():
        hi, lo = (float((net.reference(x.double(), mod.double() + s * step, post) * v).sum())
                  for s in (1, -1))
    assert abs((hi - lo) / 2e-5 / float(g.double().norm()) - 1) <= CHAIN


def test_gradients_of_single_inputs():
    """Each input alone: the others get none, and the values do not change."""
    d = 128
    net = Block(d, 256, 11)
    x, mod = randn(2, 5, d, seed=1), randn(2, 6 * d, seed=2, std=0.5)
    v = randn(2, 5, d, seed=3)
    want = torch.autograd.grad((net(x.requires_grad_(), mod.requires_grad_()) * v).sum(), [x, mod])
    x, mod = x.detach(), mod.detach()
    xr = x.clone().requires_grad_()
    a, = torch.autograd.grad((net(xr, mod) * v).sum(), [xr])
    mr = mod.clone().requires_grad_()
    b, = torch.autograd.grad((net(x, mr) * v).sum(), [mr])
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("rt", [F32, BF])
def test_linear_epilogue_gradients(act, rt):
    m = L.AWQLinear.from_linear(linear(128, 192, 21))
    w = weight64(m)
    x = randn(2, 7, 128, seed=1, dtype=BF).requires_grad_()
    gate = randn(2, 1, 192, seed=2, dtype=BF).requires_grad_()
    res = randn(2, 7, 192, seed=3).to(rt).requires_grad_()
    v = randn(2, 7, 192, seed=4)
    for use_gate, use_res in ((True, True), (True, False), (False, True), (False, False)):
        ins = [x] + [gate] * use_gate + [res] * use_res
        y = m(x, act, gate if use_gate else None, res if use_res else None)
        assert y.dtype == (rt if use_res else BF)
        got = torch.autograd.grad((y.float() * v).sum(), ins)
        x64, g64, r64 = (t.detach().double().requires_grad_() for t in (x, gate, res))
        z = x64 @ w.t() + m.bias.to(BF).double()
        z = nn.functional.silu(z) if act else z
        ref = (z * g64 if use_gate else z) + (r64 if use_res else 0)
        want = torch.autograd.grad((ref * v.double()).sum(),
                                   [x64] + [g64] * use_gate + [r64] * use_res)
        close(y, ref.detach(), "y")
        for g, t, p in zip(got, want, ins):
            assert g.dtype == p.dtype and g.shape == p.shape
            close(g, t, tuple(p.shape))


def test_views_and_broadcasts():
    """Slices, broadcast vectors and rows between 16-byte addresses."""
    n = L.BlockNorm(96, "rms", weight=torch.ones(96, device="cuda"))
    big = randn(2, 10, 200, seed=1)
    x = big[:, 1:9, 3:99]
    h = randn(2, 8, 96, seed=2, dtype=BF)
    scale = randn(1, 96, seed=3).expand(2, 96)
    gate = randn(96, 2, seed=4).t()
    a = n(x, h, gate=gate, scale=scale)
    b = n(x.contiguous(), h, gate=gate.contiguous(), scale=scale.contiguous())
    c = n(x.contiguous(), h, gate=gate.contiguous(), scale=scale[0].contiguous())
    for i in range(2):
        assert torch.equal(a[i], b[i]) and torch.equal(a[i], c[i])
    s = scale[:1].clone().requires_grad_()
    g, = torch.autograd.grad(n(x, h, scale=s.expand(2, 96))[1].float().sum(), s)
    y = n(x.double().float(), h)[1]
    assert torch.allclose(g[0], y.float().sum((0, 1)), rtol=2e-2, atol=0.5)


def test_captured_block():
    """Forward and backward in one graph, replayed on new inputs with eager work between."""
    d = 128
    net = Block(d, 256, 31)
    x = randn(2, 40, d, seed=1).requires_grad_()
    mod = randn(2, 6 * d, seed=2, std=0.5).requires_grad_()
    v = randn(2, 40, d, seed=3)

    def run(x, mod):
        y = net(x, mod)
        return [y.detach()] + list(torch.autograd.grad((y * v).sum(), [x, mod]))

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        run(x, mod)
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(x, mod)
    for i in range(3):
        with torch.no_grad():
            x.copy_(torch.roll(x, 1, 1))
            mod.mul_(0.9)
        graph.replay()
        want = run(x.detach().clone().requires_grad_(), mod.detach().clone().requires_grad_())
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b), i


def test_two_streams():
    net = Block(256, 512, 41)
    xs = [randn(1, 300, 256, seed=s) for s in range(2)]
    mods = [randn(1, 6 * 256, seed=s + 5, std=0.5) for s in range(2)]
    with torch.no_grad():
        want = [net(x, m) for x, m in zip(xs, mods)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = [None, None]
        for _ in range(5):
            for i, st in enumerate(streams):
                with torch.cuda.stream(st):
                    got[i] = net(xs[i], mods[i])
        torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_inference_mode_and_frozen():
    with torch.inference_mode():
        net = Block(128, 256, 51)
        x, mod = randn(1, 4, 128, seed=1), randn(1, 768, seed=2)
        y = net(x, mod)
    assert torch.isfinite(y).all()
    m = L.AWQLinear.from_linear(linear(128, 64, 53))
    m.bias.requires_grad_()
    x = randn(3, 128, seed=1, dtype=BF)
    with pytest.raises(RuntimeError, match="frozen"):
        m(x.clone().requires_grad_(), residual=randn(3, 64, seed=2))
    with pytest.raises(RuntimeError, match="frozen"):
        m(x, act="silu").float().sum().backward()


def test_moe_against_single_experts():
    """AWQMoE against its experts as AWQGatedLinear and AWQLinear one by one."""
    e, k, n = 6, 128, 192
    lins = [[linear(*s, 100 + 10 * i + j, bias=False) for i in range(e)]
            for j, s in enumerate(((k, n), (k, n), (n, k)))]
    moe = L.AWQMoE.from_linears(*lins, top=2)
    pairs = [L.AWQGatedLinear.from_linears(a, b) for a, b in zip(*lins[:2])]
    downs = [L.AWQLinear.from_linear(c) for c in lins[2]]
    router = linear(k, e, 99)
    for shape in ((1, k), (64, k), (3, 50, k)):
        x = randn(*shape, seed=7, dtype=BF)
        logits = router(x.float())
        y = moe(x, logits)
        p, ids = torch.softmax(logits.double(), -1).topk(2)
        p = p / p.sum(-1, keepdim=True)
        ref = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        with torch.no_grad():
            for i in range(e):
                w = (p * (ids == i)).sum(-1, keepdim=True)
                ref += w * downs[i](pairs[i](x)).double()
        assert y.shape == x.shape
        close(y, ref, shape, 4 * 2.0 ** -8)        # both round H and Y; the experts' Y too
    assert moe(x[:0], logits[:0]).shape == (0, 50, k)
    with pytest.raises(RuntimeError, match="no backward"):
        moe(x, logits).float().sum().backward()


def test_moe_of_stacked_weights():
    parts = [experts(5, 192, 128, 1), experts(5, 192, 128, 2), experts(5, 128, 192, 3)]
    moe = L.AWQMoE(*parts, 3, "gelu", False)
    x, logits = randn(20, 128, seed=3, dtype=BF), randn(20, 5, seed=4, dtype=BF)
    assert torch.equal(moe(x, logits), svdq.awq_moe_w4a16(x, logits, *parts, 3, "gelu", False))
