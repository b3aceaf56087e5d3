"""Refusals of the operators around a block (norms, AWQ product with an epilogue,
mixture of experts), without GPU work: the library rejects bad arguments before any HIP
call (fake pointers are never touched), and the binding rejects tensors that do not
match the call."""

import ctypes
import os

import pytest
import torch

from w4a4_quantized_diffusion_amd import linear as L
from w4a4_quantized_diffusion_amd import svdq

INVALID, UNSUPPORTED = 1, 2
BIG = 1 << 40
BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(svdq.LIB_PATH):
        pytest.fail("libsvdq.so is not built (run __graft_entry__.build())")
    return svdq.lib()


def at(i):
    """Distinct 256-byte aligned fake addresses, 2^36 apart."""
    return (i + 1) << 36


def vec(i, dtype=1, ld=0):
    return svdq.Vec(at(i), dtype, ld)


def _call(fn, a, kw):
    a.update(kw)
    return fn(*(ctypes.byref(v) if isinstance(v, svdq.Vec) else v for v in a.values()))


def norm(lib, **kw):
    return _call(lib.svdq_block_norm,
                 dict(X=at(0), xt=1, H=at(1), ht=1, M=6, D=128, images=2, kind=0, eps=1e-6, post=None,
                      gate=None, weight=None, scale=None, shift=None, X_out=at(2), Y=at(3), yt=1,
                      stream=None), kw)


def norm_grad(lib, **kw):
    return _call(lib.svdq_block_norm_grad,
                 dict(dY=at(0), yt=1, dX_out=at(1), X=at(2), xt=1, H=at(3), ht=1, M=6, D=128,
                      images=2, kind=0, eps=1e-6, post=None, gate=None, weight=None, scale=None,
                      shift=None, dX=at(4), dH=at(5), dpost=None, dgate=None, dweight=None,
                      dscale=None, dshift=None, ws=at(6), nws=BIG, stream=None), kw)


def res(lib, **kw):
    return _call(lib.awq_linear_w4a16_res,
                 dict(X=at(0), M=6, K=128, N=64, group=64, q=at(1), s=at(2), z=at(3), bias=None,
                      act=2, gate=None, images=2, R=None, rt=1, Y=at(4), yt=1, Z=None, ws=at(5),
                      nws=BIG, stream=None), kw)


def res_grad(lib, **kw):
    return _call(lib.awq_linear_w4a16_res_grad,
                 dict(dY=at(0), dt=1, Z=at(1), M=6, K=128, N=64, group=64, q=at(2), s=at(3), z=at(4),
                      act=0, gate=None, images=2, dX=at(5), dZ=at(6), dgate=None, ws=at(7), nws=BIG,
                      stream=None), kw)


def moe(lib, **kw):
    return _call(lib.awq_moe_w4a16,
                 dict(X=at(0), logits=at(1), lt=0, T=6, E=8, top=2, K=128, N=64, group=64, qg=at(2),
                      sg=at(3), zg=at(4), qu=at(5), su=at(6), zu=at(7), qd=at(8), sd=at(9),
                      zd=at(10), act=0, renorm=1, Y=at(11), ids=None, w=None, ws=at(12), nws=BIG,
                      stream=None), kw)


def refused(status, text, want=INVALID):
    assert status == want, svdq.svdq_last_error()
    assert text in svdq.svdq_last_error(), svdq.svdq_last_error()


@pytest.mark.parametrize("call", [norm, norm_grad])
def test_norm_sizes_and_enums(lib, call):
    refused(call(lib, M=-1), "M out of range")
    refused(call(lib, M=1 << 27, images=1), "M out of range")
    refused(call(lib, D=0), "D must")
    refused(call(lib, D=16385), "16384", UNSUPPORTED)
    for images in (0, -2, 4, (1 << 20) + 1):
        refused(call(lib, images=images), "images")
    refused(call(lib, kind=2), "norm")
    for eps in (-1e-6, float("nan"), float("inf")):
        refused(call(lib, eps=eps), "eps")
    for f in ("xt", "ht", "yt"):
        refused(call(lib, **{f: 2}), "dtype")


@pytest.mark.parametrize("call,names", [(norm, ("X", "X_out", "H", "Y")),
                                        (norm_grad, ("dY", "X", "H", "dX", "dH"))])
def test_norm_pointers(lib, call, names):
    for n in names:
        refused(call(lib, **{n: at(30) + 1}), "aligned")
        status = call(lib, **{n: None})
        assert status == INVALID
        text = svdq.svdq_last_error()
        assert "NULL" in text or "together" in text
    refused(norm_grad(lib, dX_out=at(30) + 1), "aligned")


@pytest.mark.parametrize("call", [norm, norm_grad])
@pytest.mark.parametrize("name", ["post", "gate", "weight", "scale", "shift"])
def test_norm_vectors(lib, call, name):
    refused(call(lib, **{name: svdq.Vec(None, 1, 0)}), "NULL")
    refused(call(lib, **{name: svdq.Vec(at(20) + 1, 1, 0)}), "aligned")
    refused(call(lib, **{name: svdq.Vec(at(20) + 2, 0, 0)}), "aligned")
    refused(call(lib, **{name: svdq.Vec(at(20), 3, 0)}), "dtype")
    for ld in (-1, 1, 127, 1 << 40):
        refused(call(lib, **{name: svdq.Vec(at(20), 1, ld)}), "ld")
    # the vector's second row inside an output
    out = "Y" if call is norm else "dX"
    refused(call(lib, **{name: svdq.Vec(at(20), 1, 4096), out: at(20) + 8192}), "overlap")
    if call is norm_grad:
        refused(call(lib, **{"d" + name: at(25)}), "without " + name)
        refused(call(lib, **{name: vec(20), "d" + name: at(25) + 8}), "aligned")


def test_norm_gate_and_post_need_h(lib):
    for n in ("gate", "post"):
        refused(norm(lib, H=None, X_out=None, **{n: vec(20)}), "go with H")
        refused(norm_grad(lib, H=None, dH=None, **{n: vec(20)}), "go with H")


@pytest.mark.parametrize("call,ins,outs", [
    (norm, ("X", "H"), ("X_out", "Y")),
    (norm_grad, ("dY", "dX_out", "X", "H"), ("dX", "dH", "dweight", "ws")),
    (res, ("X", "q", "s", "z", "bias", "R"), ("Y", "Z")),
    (res_grad, ("dY", "Z", "q", "s", "z"), ("dX", "dZ", "dgate")),
    (moe, ("X", "logits", "qg", "sg", "zg", "qu", "su", "zu", "qd", "sd", "zd"),
     ("Y", "ids", "w", "ws"))])
def test_overlap(lib, call, ins, outs):
    base = {norm_grad: dict(weight=vec(40)), res_grad: dict(gate=vec(40))}.get(call, {})
    for o in outs:
        for i in ins + tuple(p for p in outs if p != o):
            refused(call(lib, **{**base, o: at(30), i: at(30)}), "overlap")


@pytest.mark.parametrize("call", [res, res_grad])
def test_res_sizes(lib, call):
    for kw, msg in ((dict(K=100), "K must"), (dict(N=40), "N must"), (dict(M=-1), "M out of range"),
                    (dict(K=(1 << 22) + 64), "2^22"), (dict(images=4), "images"),
                    (dict(images=0), "images"), (dict(act=3), "activation"),
                    (dict(gate=svdq.Vec(at(20), 1, 63)), "ld"),
                    (dict(gate=svdq.Vec(at(20) + 1, 1, 0)), "aligned")):
        refused(call(lib, **kw), msg)
    refused(call(lib, group=128), "group", UNSUPPORTED)


def test_res_pointers(lib):
    for n in ("X", "q", "s", "z", "Y"):
        refused(res(lib, **{n: None}), "NULL")
        refused(res(lib, **{n: at(30) + 8}), "aligned")
    for n in ("R", "Z"):
        refused(res(lib, **{n: at(30) + 8}), "aligned")
    refused(res(lib, bias=at(30) + 1), "aligned")
    refused(res(lib, yt=2), "dtype")
    refused(res(lib, R=at(30), rt=2), "dtype")
    for n in ("dY", "Z", "q", "s", "z", "dX", "dZ"):
        refused(res_grad(lib, **{n: None}), "NULL")
        refused(res_grad(lib, **{n: at(30) + 8}), "aligned")
    refused(res_grad(lib, dt=2), "dtype")
    refused(res_grad(lib, dgate=at(30)), "without gate")
    refused(res_grad(lib, act=2, Z=None, gate=vec(20), dgate=at(30)), "NULL")


def test_moe_sizes(lib):
    for kw, msg in ((dict(K=100), "K must"), (dict(N=80), "N must"), (dict(T=-1), "M out of range"),
                    (dict(E=0), "E must"), (dict(top=0), "top"), (dict(top=9), "top"),
                    (dict(act=2), "activation"), (dict(lt=2), "dtype")):
        refused(moe(lib, **kw), msg)
    for kw, msg in ((dict(T=65), "64 tokens"), (dict(E=257), "256"), (dict(E=32, top=17), "16"),
                    (dict(group=32), "group")):
        refused(moe(lib, **kw), msg, UNSUPPORTED)
    for n in ("X", "logits", "qg", "sg", "zg", "qu", "su", "zu", "qd", "sd", "zd", "Y"):
        refused(moe(lib, **{n: None}), "NULL")
        refused(moe(lib, **{n: at(30) + 2}), "aligned")
    refused(moe(lib, ids=at(30) + 2), "aligned")
    refused(moe(lib, w=at(30) + 2), "aligned")


def test_workspaces(lib):
    for m, d, images in ((1, 64, 1), (600, 1000, 3), (9216, 4096, 2), (1030, 264, 1030)):
        need = svdq.svdq_block_norm_grad_workspace_bytes(m, d, images)
        assert need > 0 and need % 256 == 0
    need = svdq.svdq_block_norm_grad_workspace_bytes(6, 128, 2)
    refused(norm_grad(lib, nws=need - 1), "too small")
    refused(norm_grad(lib, ws=at(30) + 16), "aligned")
    refused(norm_grad(lib, ws=None), "NULL")
    assert svdq.svdq_block_norm_grad_workspace_bytes(6, 128, 4) == 0
    assert svdq.svdq_block_norm_grad_workspace_bytes(0, 128, 1) == 0
    for m, k, n in ((1, 64, 16), (64, 4096, 8208), (333, 2048, 4112), (4608, 4096, 12288)):
        for need in (svdq.awq_linear_w4a16_res_workspace_bytes(m, k, n),
                     svdq.awq_linear_w4a16_res_grad_workspace_bytes(m, k, n, 1)):
            assert need % 256 == 0
    for args in ((4, 100, 64), (4, 128, 40), (-1, 128, 64)):
        assert svdq.awq_linear_w4a16_res_workspace_bytes(*args) == 0
        assert svdq.awq_linear_w4a16_res_grad_workspace_bytes(*args, 1) == 0
    assert svdq.awq_linear_w4a16_res_grad_workspace_bytes(4, 128, 64, 3) == 0
    need = svdq.awq_linear_w4a16_res_workspace_bytes(300, 2048, 256)
    assert need > 0
    refused(res(lib, M=300, K=2048, N=256, nws=need - 1), "too small")
    need = svdq.awq_linear_w4a16_res_grad_workspace_bytes(300, 256, 2048, 2)
    assert need > 0
    refused(res_grad(lib, M=300, K=256, N=2048, nws=need - 1), "too small")
    for args in ((65, 8, 2, 128, 64), (6, 8, 9, 128, 64), (6, 257, 2, 128, 64), (6, 8, 2, 128, 80)):
        assert svdq.awq_moe_w4a16_workspace_bytes(*args) == 0
    need = svdq.awq_moe_w4a16_workspace_bytes(6, 8, 2, 128, 64)
    assert need > 0 and need % 256 == 0
    refused(moe(lib, nws=need - 1), "too small")


def test_zero_rows_need_nothing(lib):
    assert norm(lib, M=0, images=1, X=None, H=None, X_out=None, Y=None) == 0
    assert norm_grad(lib, M=0, images=1, dY=None, dX_out=None, X=None, H=None, dX=None, dH=None,
                     ws=None, nws=0) == 0
    assert res(lib, M=0, images=1, X=None, q=None, s=None, z=None, Y=None, ws=None, nws=0) == 0
    assert res_grad(lib, M=0, images=1, dY=None, Z=None, q=None, s=None, z=None, dX=None, dZ=None,
                    ws=None, nws=0) == 0
    none = {n: None for n in ("X", "logits", "qg", "sg", "zg", "qu", "su", "zu", "qd", "sd", "zd",
                              "Y", "ws")}
    assert moe(lib, T=0, nws=0, **none) == 0


# ------------------------------------------------------------- the binding

def test_vectors_of_the_binding():
    t = lambda *s: torch.zeros(s, dtype=BF)  # noqa: E731
    one = lambda v, m=12: svdq._vecs((v,), m, 8, -1, ("gate",))  # noqa: E731
    assert one(t(8))[0] == 1 and one(t(8))[1][0].ld == 0
    assert one(t(1, 8))[0] == 1 and one(t(1, 8))[1][0].ld == 0
    images, (v,) = one(t(3, 24)[:, 8:16])
    assert images == 3 and v.ld == 24 and v.dtype == svdq.BF16
    for bad in (t(7), t(3, 7), t(0, 8), t(2, 3, 8), t()):
        with pytest.raises(ValueError, match="gate must have shape"):
            one(bad)
    with pytest.raises(TypeError, match="gate must be"):
        one(t(8).half())
    with pytest.raises(ValueError, match="divide"):
        one(t(5, 8))
    with pytest.raises(ValueError, match="adjacent"):
        one(t(8, 3).t())
    with pytest.raises(ValueError, match="overlap"):
        one(t(1, 8).expand(3, 8))
    with pytest.raises(ValueError, match="another vector"):
        svdq._vecs((t(3, 8), t(4, 8)), 12, 8, -1, ("gate", "scale"))


def test_binding_rejects_host_tensors():
    x = torch.zeros(4, 64, dtype=BF)
    lay = dict(N=64, K=64, group=64)
    for f in (lambda: svdq.svdq_block_norm(x), lambda: svdq.svdq_block_norm_grad(x, x),
              lambda: svdq.awq_linear_w4a16_res(x, lay),
              lambda: svdq.awq_linear_w4a16_res_grad(x, x, lay),
              lambda: svdq.awq_moe_w4a16(x, x, dict(lay, E=2), dict(lay, E=2), dict(lay, E=2), 1)):
        with pytest.raises(ValueError, match="device tensor"):
            f()
    for f in (lambda: svdq.svdq_block_norm(x[0]), lambda: svdq.svdq_block_norm_grad(x[0], x[0]),
              lambda: svdq.awq_linear_w4a16_res(x[0], lay)):
        with pytest.raises(ValueError, match="shape"):
            f()


# ------------------------------------------------------------- the modules

def test_modules_reject():
    x = torch.zeros(2, 3, 64, dtype=BF)
    with pytest.raises(ValueError, match="kind"):
        L.BlockNorm(64, "batch")
    with pytest.raises(ValueError, match="dim"):
        L.BlockNorm(16385)
    with pytest.raises(ValueError, match="weight"):
        L.BlockNorm(64, weight=torch.ones(63))
    with pytest.raises(ValueError, match="expected"):
        L.BlockNorm(32)(x)
    with pytest.raises(ValueError, match="go with h"):
        L.BlockNorm(64)(x, gate=torch.ones(64))
    with pytest.raises(ValueError, match="go with h"):
        L.BlockNorm(64, post=torch.ones(64))(x)
    with pytest.raises(ValueError, match="h: expected"):
        L.BlockNorm(64)(x, x[:1])
    with pytest.raises(ValueError, match="scale: expected"):
        L.BlockNorm(64)(x, scale=torch.ones(2, 63))
    m = L.BlockNorm(64, "rms", weight=torch.ones(64), post=nnp(torch.ones(64)))
    assert {n for n, _ in m.named_parameters()} == {"weight", "post"}
    awq = L.AWQLinear(awq_layer(64, 64))
    with pytest.raises(ValueError, match="act"):
        awq(x, act="relu")
    with pytest.raises(ValueError, match="residual: expected"):
        awq(x, residual=x[:1])
    with pytest.raises(ValueError, match="gate: expected"):
        awq(x, gate=torch.ones(63))


def nnp(t):
    return torch.nn.Parameter(t)


def awq_layer(n, k, e=None):
    lead = () if e is None else (e,)
    lay = dict(N=n, K=k, group=64, q=torch.zeros(*lead, k // 64, n, 32, dtype=torch.uint8),
               scales=torch.zeros(*lead, k // 64, n, dtype=torch.int16),
               zeros=torch.zeros(*lead, k // 64, n, dtype=torch.int16))
    return lay if e is None else dict(lay, E=e)


def test_moe_module():
    parts = [awq_layer(128, 64, 4), awq_layer(128, 64, 4), awq_layer(64, 128, 4)]
    m = L.AWQMoE(*parts, 2)
    assert "experts=4" in repr(m) and m.layer("down")["N"] == 64
    x, logits = torch.zeros(2, 3, 64, dtype=BF), torch.zeros(2, 3, 4)
    with pytest.raises(TypeError, match="bf16"):
        m(x.float(), logits)
    with pytest.raises(ValueError, match="logits"):
        m(x, logits[..., :3])
    with pytest.raises(ValueError, match="input"):
        m(x[..., :32], logits)
    for top in (0, 5):
        with pytest.raises(ValueError, match="top"):
            L.AWQMoE(*parts, top)
    with pytest.raises(ValueError, match="act"):
        L.AWQMoE(*parts, 2, "none")
    with pytest.raises(ValueError, match="down"):
        L.AWQMoE(*parts[:2], awq_layer(128, 64, 4), 2)
    with pytest.raises(ValueError, match="up_q"):
        L.AWQMoE(parts[0], dict(parts[1], q=parts[1]["q"][:2]), parts[2], 2)


def test_moe_save_and_load(tmp_path):
    parts = [awq_layer(128, 64, 3), awq_layer(128, 64, 3), awq_layer(64, 128, 3)]
    for i, p in enumerate(parts):
        p["q"] += i + 1
    net = torch.nn.Sequential(L.AWQMoE(*parts, 2, "gelu", False))
    path = str(tmp_path / "m.safetensors")
    assert L.save_quantized(net, path) == ["0"]
    other = torch.nn.Sequential(torch.nn.Identity())
    assert L.load_quantized(other, path) == ["0"]
    m = other[0]
    assert (m.top, m.act, m.renorm, m.experts) == (2, "gelu", False, 3)
    for f in L._MOE_FIELDS:
        assert torch.equal(getattr(m, f), getattr(net[0], f))
