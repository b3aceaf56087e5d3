"""The modules of the weight-only operators under autograd, without a GPU: the
binding's calls are replaced by the same mathematics in torch on detached values
(the kernels read raw memory, so nothing of autograd passes through them)."""

import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fwAD
from torch import nn

from w4a4_quantized_diffusion_amd import linear as L
from w4a4_quantized_diffusion_amd import svdq

BF = torch.bfloat16
N, K = 64, 128


def awq_layer(n, k, seed):
    g = torch.Generator().manual_seed(seed)
    bits = lambda t: t.to(BF).view(torch.int16)  # noqa: E731
    return dict(N=n, K=k, group=64, q=torch.randint(0, 256, (k // 64, n, 32), generator=g, dtype=torch.uint8),
                scales=bits(torch.rand(k // 64, n, generator=g) / 50 + 0.01),
                zeros=bits(torch.randint(6, 10, (k // 64, n), generator=g).float()))


def weight(lay):
    n, k = lay["N"], lay["K"]
    q = torch.stack((lay["q"] & 15, lay["q"] >> 4), -1).reshape(k // 64, n, 64).float()
    s, z = (lay[f].detach().view(BF).float().unsqueeze(-1) for f in ("scales", "zeros"))
    return ((q - z) * s).to(BF).float().permute(1, 0, 2).reshape(n, k)


def raw(t):
    """What a kernel sees of a tensor, checked as the library checks it."""
    if t is None:
        return 0.0
    t = fwAD.unpack_dual(t).primal.detach()
    assert t.is_contiguous() and t.data_ptr() % 16 == 0
    return t.float()


@pytest.fixture(autouse=True)
def kernels(monkeypatch):
    def linear(x, lay, bias=None):
        return (raw(x) @ weight(lay).t() + raw(bias)).to(BF)

    def linear_grad(dy, lay):
        return (raw(dy) @ weight(lay)).to(BF)

    def gated(x, gate, up, act="silu", bg=None, bu=None, save=False):
        g, u = raw(x) @ weight(gate).t() + raw(bg), raw(x) @ weight(up).t() + raw(bu)
        h = (nn.functional.silu(g) * u).to(BF)
        return (h, g.to(BF), u.to(BF)) if save else h

    def gated_grad(dh, g, u, gate, up, act="silu"):
        g, u, d = raw(g), raw(u), raw(dh)
        s = torch.sigmoid(g)
        dg, du = (d * u * (s + g * s * (1 - s))).to(BF), (d * g * s).to(BF)
        return (dg.float() @ weight(gate) + du.float() @ weight(up)).to(BF), dg, du

    for name, f in (("awq_linear_w4a16", linear), ("awq_linear_w4a16_grad", linear_grad),
                    ("awq_gated_w4a16", gated), ("awq_gated_w4a16_grad", gated_grad)):
        monkeypatch.setattr(svdq, name, torch.no_grad()(f))


def modules(bias=None):
    b = None if bias is None else torch.full((N,), float(bias))
    return [L.AWQLinear(awq_layer(N, K, 1), b),
            L.AWQGatedLinear(awq_layer(N, K, 1), awq_layer(N, K, 2), b, b)]


def rows(m=3, seed=3):
    return torch.randn(m, K, generator=torch.Generator().manual_seed(seed)).to(BF)


@pytest.mark.parametrize("which", [0, 1])
def test_forward_mode_is_refused(which):
    """A tangent of the input is refused, with or without reverse mode beside it, and
    no call outside forward mode is."""
    mod, x = modules(0.5)[which], rows()
    y = mod(x)
    for leaf in (x, x.clone().requires_grad_()):
        with fwAD.dual_level():
            with pytest.raises(RuntimeError, match="forward-mode"):
                mod(fwAD.make_dual(leaf, torch.ones_like(x)))
            assert torch.equal(mod(leaf), y)                  # no tangent: as ever
    with pytest.raises(RuntimeError, match="forward-mode"):
        torch.func.jvp(mod, (x,), (torch.ones_like(x),))
    with torch.no_grad():
        assert torch.equal(mod(x), y)
    with torch.inference_mode():
        assert torch.equal(mod(x), y)


@pytest.mark.parametrize("names", [("bias",), ("bias_gate",), ("bias_up",), ("bias_gate", "bias_up")])
def test_a_bias_that_requires_a_gradient(names):
    """Biases are frozen.  The call on an input without a gradient runs, and a
    gradient asked of the bias raises instead of staying away; the values are those
    of the frozen module, also where they are used in place."""
    mod, x = modules(0.5)[len(names[0]) > 4], rows()
    y = mod(x)
    assert not y.requires_grad
    for n in names:
        getattr(mod, n).requires_grad_()
    for _ in range(2):
        out = mod(x)
        assert torch.equal(out, y) and out.requires_grad
        with pytest.raises(RuntimeError, match="frozen"):
            out.sum().backward()
        assert all(getattr(mod, n).grad is None for n in names)
    out = mod(x)
    out.add_(1)
    w = torch.ones(N, requires_grad=True)
    with pytest.raises(RuntimeError, match="frozen"):
        (out.float() * w).sum().backward()
    (g,) = torch.autograd.grad((mod(x).float() * w).sum(), w)        # nothing asked of the bias
    assert torch.equal(g, y.float().sum(0))
    with torch.no_grad():
        assert torch.equal(mod(x), y) and not mod(x).requires_grad
    with pytest.raises(RuntimeError, match="frozen"):
        mod(x.clone().requires_grad_())
    for n in names:
        getattr(mod, n).requires_grad_(False)
    assert torch.equal(mod(x), y) and not mod(x).requires_grad


@pytest.mark.parametrize("which", [0, 1])
def test_layers_made_under_inference_mode(which):
    """Layers quantized or loaded under inference mode run outside it, with and
    without a gradient of the input, and give what other layers give."""
    ref, x = modules(0.5)[which], rows()
    with torch.inference_mode():
        mod = modules(0.5)[which]
        assert all(b.is_inference() for b in mod.buffers())
    y = ref(x)
    with torch.no_grad():
        assert torch.equal(mod(x), y)
    assert torch.equal(mod(x), y)
    a, b = x.clone().requires_grad_(), x.clone().requires_grad_()
    ref(a).float().square().sum().backward()
    mod(b).float().square().sum().backward()
    assert torch.equal(a.grad, b.grad) and a.grad.any()


@pytest.mark.parametrize("which", [0, 1])
def test_weights_changed_before_the_backward_pass(which):
    """New weights copied into a layer between a forward pass and its backward pass
    are noticed, as torch's own layers notice them."""
    mod, x = modules()[which], rows().requires_grad_()
    y = mod(x)
    other = {k: v.clone() for k, v in mod.state_dict().items()}
    mod.load_state_dict(other)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_a_new_bias_at_an_old_address():
    """The bf16 copy of the bias that AWQLinear keeps belongs to one tensor, not to
    its address: another tensor that took the freed one's place is read anew."""
    mod, x = modules(0.0)[0], rows()
    store = np.zeros(N + 4, dtype=np.float32)
    store = store[-store.ctypes.data % 16 // 4:][:N]
    zero = mod(x).float()
    for v in (4.0, 8.0):
        store[:] = v
        mod.bias = torch.from_numpy(store)       # same address and version every time
        assert torch.equal(mod(x), (raw(x) @ weight(awq_layer(N, K, 1)).t() + v).to(BF))
        assert torch.equal(mod(x), (raw(x) @ weight(awq_layer(N, K, 1)).t() + v).to(BF))
    with torch.no_grad():
        mod.bias.zero_()                         # in place: seen by its version
    assert torch.equal(mod(x).float(), zero)


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("pad", [1, 8])
def test_rows_at_odd_addresses(which, pad):
    """Contiguous views that start between 16-byte addresses, as the input (a slice of
    a flat buffer) and as the gradient (of a concatenation behind an odd number of
    elements): the library takes aligned rows only, so the modules copy them."""
    mod, x = modules(0.5)[which], rows()
    flat = torch.zeros(pad + x.numel(), dtype=BF)
    flat[pad:] = x.flatten()
    view = flat[pad:].view_as(x)
    assert torch.equal(mod(view), mod(x))
    a, b = x.clone().requires_grad_(), flat.clone().requires_grad_()
    dy = torch.randn(3, N, generator=torch.Generator().manual_seed(9)).to(BF)
    mod(a).backward(dy)
    y = mod(b[pad:].view_as(x))
    torch.cat((torch.zeros(pad, dtype=BF), y.flatten())).backward(
        torch.cat((torch.zeros(pad, dtype=BF), dy.flatten())))
    assert torch.equal(b.grad[pad:].view_as(x), a.grad)
