"""The weight-only operators through the modules: a gated feed-forward block
forward and backward against a float64 block on its own quantized weights, its
single-token form, autograd's odd gradients, graph capture, another stream, and
SVDQLinear's few-row form."""

import pytest
import torch
from torch import nn

from w4a4_quantized_diffusion_amd import linear as L
from w4a4_quantized_diffusion_amd import svdq

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def linear(k, n, seed, bias=True):
    g = torch.Generator("cuda").manual_seed(seed)
    lin = nn.Linear(k, n, bias=bias, device="cuda")
    with torch.no_grad():
        lin.weight.copy_(torch.randn(n, k, generator=g, device="cuda") / k ** 0.5)
        if bias:
            lin.bias.copy_(torch.randn(n, generator=g, device="cuda") * 0.1)
    return lin.requires_grad_(False)


def block(k, n, act="silu", bias=True, seed=0):
    gated = L.AWQGatedLinear.from_linears(linear(k, n, seed, bias), linear(k, n, seed + 1, bias), act)
    return nn.Sequential(gated, L.AWQLinear.from_linear(linear(n, k, seed + 2, bias)))


def weight(mod, prefix=""):
    q, s, z = (getattr(mod, prefix + f) for f in ("q", "scales", "zeros"))
    g, n, _ = q.shape
    c = torch.stack((q & 15, q >> 4), -1).reshape(g, n, 64).double()
    w = (c - z.view(BF).double().unsqueeze(-1)) * s.view(BF).double().unsqueeze(-1)
    return w.to(BF).double().permute(1, 0, 2).reshape(n, g * 64)


def reference(b, x, dy):
    """float64 block and input gradient on the quantized weights; tolerances
    relative to the sums of magnitudes: each of H, G, U, dH, dG, dU is rounded to
    bf16 once on the way (2^-8 relative, taken as 2^-7 for two neighbours)."""
    gated, down = b
    wg, wu, wd = weight(gated, "gate_"), weight(gated, "up_"), weight(down)
    bias = [0 if t is None else t.to(BF).double()
            for t in (gated.bias_gate, gated.bias_up, down.bias)]
    x = x.double().requires_grad_()
    g, u = x @ wg.t() + bias[0], x @ wu.t() + bias[1]
    a = nn.functional.silu(g) if gated.act == "silu" else nn.functional.gelu(g, approximate="tanh")
    h = a * u
    y = h @ wd.t() + bias[2]
    (dx,) = torch.autograd.grad(y, x, dy.double())
    with torch.no_grad():
        ytol = 2.0 ** -7 * (h.abs() @ wd.abs().t() + y.abs())
        dh = dy.double() @ wd
        dha = dy.double().abs() @ wd.abs()
        # act' <= 1.13 and |act''| <= 0.8: a step 2^-8 |G| in G moves act' by 2^-8 |G|
        dxtol = 2.0 ** -7 * ((dha * u.abs() * (1.13 + g.abs())) @ wg.abs()
                             + (dha * (a.abs() + 1.13 * g.abs())) @ wu.abs() + dx.abs())
    return y.detach(), dx, ytol, dxtol


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("lead,bias", [((1,), True), ((2, 9), False), ((3, 50), True), ((700,), False)])
def test_block(lead, bias, act):
    print(f"block {lead} {bias} {act}", flush=True)
    k, n = 256, 448
    b = block(k, n, act, bias)
    x = torch.randn(*lead, k, device="cuda").to(BF)
    dy = torch.randn(*lead, k, device="cuda").to(BF)
    with torch.no_grad():
        y0 = b(x)
    assert not y0.requires_grad
    xg = x.clone().requires_grad_()
    y = b(xg)
    assert y.shape == x.shape and torch.equal(y, y0)
    y.backward(dy)
    ry, rdx, ytol, dxtol = reference(b, x.reshape(-1, k), dy.reshape(-1, k))
    assert ((y.reshape(-1, k).double() - ry).abs() <= ytol).all()
    assert ((xg.grad.reshape(-1, k).double() - rdx).abs() <= dxtol).all()


def test_single_tokens_give_the_rows_of_a_prompt():
    """Each row alone and all together: the same sums in another order."""
    k, n, m = 256, 320, 70
    b = block(k, n)
    x = torch.randn(m, k, device="cuda").to(BF)
    with torch.no_grad():
        y = b(x)
        rows = torch.cat([b(x[i:i + 1]) for i in range(0, m, 7)])
    _, _, ytol, _ = reference(b, x, torch.zeros_like(x))
    assert ((y[::7].double() - rows.double()).abs() <= ytol[::7]).all()


def test_odd_gradients():
    """Expanded, transposed and zero-row gradients, a module used twice, and a
    second derivative refused."""
    k, n = 128, 192
    b = block(k, n)
    x = torch.randn(6, k, device="cuda").to(BF)
    xg = x.clone().requires_grad_()
    b(xg).sum().backward()                                    # expanded ones
    ones = torch.ones(6, k, device="cuda", dtype=BF)
    (ref,) = torch.autograd.grad(b(xg), xg, ones)
    assert torch.equal(xg.grad, ref)
    dyt = torch.randn(k, 6, device="cuda").to(BF)
    (a,) = torch.autograd.grad(b(xg), xg, dyt.t())            # strided
    (c,) = torch.autograd.grad(b(xg), xg, dyt.t().contiguous())
    assert torch.equal(a, c)
    (twice,) = torch.autograd.grad(b(xg) + b(xg), xg, ones)   # both uses add up
    assert torch.equal(twice, ref + ref)
    e = torch.empty(0, k, device="cuda", dtype=BF, requires_grad=True)
    (z,) = torch.autograd.grad(b(e), e, torch.empty(0, k, device="cuda", dtype=BF))
    assert z.shape == (0, k)
    (gx,) = torch.autograd.grad(b(xg), xg, ones.requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError):
        gx.sum().backward()


def test_block_in_a_graph():
    """Forward and backward captured together and replayed on new inputs, with
    eager steps on other leaves between the replays."""
    k, n, m = 256, 320, 90
    b = block(k, n)
    x = torch.randn(m, k, device="cuda").to(BF).requires_grad_()
    dy = torch.randn(m, k, device="cuda").to(BF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            torch.autograd.grad(b(x), x, dy)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = b(x)
        (dx,) = torch.autograd.grad(y, x, dy)
    for i in range(3):
        new = torch.randn(m, k, device="cuda").to(BF)
        with torch.no_grad():
            x.copy_(new)
        leaf = new.clone().requires_grad_()
        ey = b(leaf)
        (edx,) = torch.autograd.grad(ey, leaf, dy)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ey) and torch.equal(dx, edx), i


def test_two_streams_at_once():
    """One module's calls on two streams: the operators share nothing."""
    k, n = 256, 320
    b = block(k, n)
    xs = [torch.randn(m, k, device="cuda").to(BF) for m in (3, 200)]
    with torch.no_grad():
        ref = [b(x) for x in xs]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in xs]
        out = [[], []]
        for _ in range(5):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    out[i].append(b(xs[i]))
    torch.cuda.synchronize()
    for r, o in zip(ref, out):
        assert all(torch.equal(r, y) for y in o)


@pytest.mark.parametrize("prec", ["int4", "nvfp4"])
def test_svdq_linear_few_rows(prec):
    """SVDQLinear with a16_rows: few rows take svdq_linear_w4a16 and come closer
    to the unquantized layer, more rows stay bit for bit as they were."""
    lin = linear(512, 272, 7)
    x = torch.randn(200, 512, device="cuda").to(BF)
    amax = svdq.svdq_act_absmax(x)
    a = L.SVDQLinear.from_linear(lin, amax, rank=16, prec=prec)
    b = L.SVDQLinear.from_linear(lin, amax, rank=16, prec=prec, a16_rows=12)
    assert torch.equal(a(x), b(x)) and torch.equal(a(x[:13]), b(x[:13]))
    y = b(x[:12])
    assert torch.equal(y, svdq.svdq_linear_w4a16(x[:12], b.layer(), b.bias, y_dtype=BF))
    ref = x[:12].double() @ lin.weight.double().t() + lin.bias.double()
    assert (y.double() - ref).norm() < (a(x[:12]).double() - ref).norm()
    assert b(x[:0]).shape == (0, 272)
    # alternating sizes
    assert torch.equal(b(x[:12]), y) and torch.equal(b(x), a(x)) and torch.equal(b(x[:12]), y)


def test_shim_hands_a16_rows_on():
    """quantize_linears(a16_rows=...) reaches the layers without gelu_input."""
    b = nn.Sequential(linear(128, 256, 8), nn.Linear(256, 128, device="cuda"))
    done = L.quantize_linears(b, rank=16, gelu_input=("1",), a16_rows=5)
    assert done == {"0": "svdq", "1": "svdq"}
    assert b[0].a16_rows == 5 and b[1].a16_rows == 0 and b[1].gelu_input
    x = torch.randn(4, 128, device="cuda").to(BF)
    assert torch.equal(b[0](x), svdq.svdq_linear_w4a16(x, b[0].layer(), b[0].bias, y_dtype=BF))


def test_captured_few_rows_outlive_a_larger_call():
    """A captured call on few rows replays right after eager calls on more rows,
    and writes to nothing but its own memory."""
    a = L.SVDQLinear.from_linear(linear(512, 272, 9), rank=16, a16_rows=64)
    x = torch.randn(2, 512, device="cuda").to(BF)
    ref = a(x)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        y = a(x)
    big = torch.randn(700, 512, device="cuda").to(BF)
    yb = a(big)
    fill = [torch.full((n,), 5.0, device="cuda") for n in (64, 1024, 4096, 16384, 1 << 18) * 4]
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(a(big), yb)
    assert all((t == 5.0).all() for t in fill)
