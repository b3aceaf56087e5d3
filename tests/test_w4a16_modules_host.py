"""Modules of the weight-only operators, without a GPU: the gated module and
a16_rows survive save_quantized / load_quantized, and what they refuse."""

import pytest
import torch
from torch import nn

from w4a4_quantized_diffusion_amd import linear as L
from w4a4_quantized_diffusion_amd import svdq
from tests.test_linear_format import _awq_layer, _svdq_layer


class Block(nn.Module):
    def __init__(self):
        super().__init__()
        self.mod = nn.Linear(128, 256)
        self.ff = nn.Sequential(nn.Identity(), nn.Linear(256, 128))


@pytest.mark.parametrize("biases", [(), ("gate",), ("gate", "up")])
def test_save_load_gated(tmp_path, biases):
    g = torch.Generator().manual_seed(3)
    q = Block()
    q.mod = L.SVDQLinear(_svdq_layer(256, 128, 16, svdq.INT4, g), None, a16_rows=9)
    kw = {f"bias_{b}": torch.randn(256, generator=g) for b in biases}
    q.ff[0] = L.AWQGatedLinear(_awq_layer(256, 128, g), _awq_layer(256, 128, g), act="gelu", **kw)
    q.ff[1] = L.AWQLinear(_awq_layer(128, 256, g), None)
    path = str(tmp_path / "b.safetensors")
    assert sorted(L.save_quantized(q, path)) == ["ff.0", "ff.1", "mod"]
    fresh = Block()
    assert sorted(L.load_quantized(fresh, path)) == ["ff.0", "ff.1", "mod"]
    for name in ("mod", "ff.0", "ff.1"):
        a, b = q.get_submodule(name), fresh.get_submodule(name)
        assert type(a) is type(b) and a.extra_repr() == b.extra_repr()
        for buf, t in a.named_buffers():
            assert torch.equal(t, getattr(b, buf)), (name, buf)
    assert fresh.mod.a16_rows == 9 and fresh.ff[0].act == "gelu"
    assert (fresh.ff[0].bias_up is None) == ("up" not in biases)


def test_refusals():
    g = torch.Generator().manual_seed(4)
    lay = _svdq_layer(64, 128, 16, svdq.INT4, g)
    for rows in (-1, 65):
        with pytest.raises(ValueError, match="a16_rows"):
            L.SVDQLinear(lay, a16_rows=rows)
    with pytest.raises(ValueError, match="gelu_input"):
        L.SVDQLinear(lay, gelu_input=True, a16_rows=4)
    a, b = _awq_layer(64, 128, g), _awq_layer(64, 192, g)
    with pytest.raises(ValueError, match="one shape"):
        L.AWQGatedLinear(a, b)
    with pytest.raises(ValueError, match="act must"):
        L.AWQGatedLinear(a, a, act="relu")
    bad = dict(a, zeros=a["zeros"].float())
    with pytest.raises(ValueError, match="up_zeros"):
        L.AWQGatedLinear(a, bad)
    m = L.AWQGatedLinear(a, a)
    with pytest.raises(TypeError, match="bf16"):
        m(torch.zeros(2, 128))
    with pytest.raises(ValueError, match="input"):
        m(torch.zeros(2, 64, dtype=torch.bfloat16))
    lin = L.AWQLinear(a, torch.zeros(64))
    lin.bias.requires_grad_()
    with pytest.raises(RuntimeError, match="frozen"):
        lin(torch.zeros(2, 128, dtype=torch.bfloat16, requires_grad=True))


def test_layers_pickled_before_a16_rows():
    """An SVDQLinear pickled whole by a version without a16_rows is one with none."""
    g = torch.Generator().manual_seed(5)
    m = L.SVDQLinear(_svdq_layer(64, 128, 16, svdq.INT4, g))
    state = m.__getstate__() if hasattr(m, "__getstate__") else m.__dict__
    old = {k: v for k, v in dict(state).items() if k != "a16_rows"}
    new = L.SVDQLinear.__new__(L.SVDQLinear)
    new.__setstate__(old)
    assert new.a16_rows == 0 and "a16_rows" not in new.extra_repr()
    with pytest.raises(ValueError, match="device tensor"):          # as far as a host goes
        new(torch.zeros(2, 128))


def test_shim_checks_a16_rows_first(monkeypatch):
    """quantize_linears refuses its arguments before it swaps anything."""
    g = torch.Generator().manual_seed(6)
    monkeypatch.setattr(L.AWQLinear, "from_linear",
                        classmethod(lambda cls, lin: cls(_awq_layer(256, 128, g))))
    monkeypatch.setattr(svdq, "svdq_quantize_weights",
                        lambda w, a, r, p: _svdq_layer(w.shape[0], w.shape[1], r, svdq._PREC[p], g))
    for rows in (-1, 65):
        b = Block()
        with pytest.raises(ValueError, match="a16_rows"):
            L.quantize_linears(b, rank=16, awq=("mod",), a16_rows=rows)
        assert type(b.mod) is nn.Linear and type(b.ff[1]) is nn.Linear
    assert L.quantize_linears(Block(), rank=16, awq=("mod",), a16_rows=64) == {"mod": "awq", "ff.1": "svdq"}
