"""Refusals of the weight-only operators (no GPU work): the library rejects
bad arguments before any HIP call (fake pointers are never touched), and the
binding rejects tensors that do not match the call."""

import ctypes
import os

import pytest
import torch

from w4a4_quantized_diffusion_amd import svdq

INVALID, UNSUPPORTED = 1, 2
P = ctypes.c_void_p
BIG = 1 << 40                      # a workspace size no check exceeds


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(svdq.LIB_PATH):
        pytest.fail("libsvdq.so is not built (run __graft_entry__.build())")
    return svdq.lib()


def at(i):
    """Distinct 256-byte aligned fake addresses, 2^36 apart."""
    return (i + 1) << 36


def a16(lib, **kw):
    a = dict(X=at(0), x_dtype=1, M=4, K=128, N=64, rank=16, prec=0, smooth=at(1), down=at(2),
             up=at(3), wcodes=at(4), wscales=at(5), ts=at(6), bias=at(7), bias_dtype=0, Y=at(8),
             y_dtype=1, ws=at(9), nws=BIG, stream=None)
    a.update(kw)
    return lib.svdq_linear_w4a16(*a.values())


def gated(lib, **kw):
    a = dict(X=at(0), M=4, K=128, N=64, group=64, qg=at(1), sg=at(2), zg=at(3), bg=None, qu=at(4),
             su=at(5), zu=at(6), bu=None, act=0, H=at(7), h_dtype=1, G=None, U=None, ws=at(8),
             nws=BIG, stream=None)
    a.update(kw)
    return lib.awq_gated_w4a16(*a.values())


def gated_grad(lib, **kw):
    a = dict(dH=at(0), G=at(1), U=at(2), M=4, K=128, N=64, group=64, qg=at(3), sg=at(4), zg=at(5),
             qu=at(6), su=at(7), zu=at(8), act=0, dX=at(9), dG=at(10), dU=at(11), ws=at(12),
             nws=BIG, stream=None)
    a.update(kw)
    return lib.awq_gated_w4a16_grad(*a.values())


def linear_grad(lib, **kw):
    a = dict(dY=at(0), M=4, K=128, N=64, group=64, q=at(1), s=at(2), z=at(3), dX=at(4), dx_dtype=1,
             ws=at(5), nws=BIG, stream=None)
    a.update(kw)
    return lib.awq_linear_w4a16_grad(*a.values())


ALL = [a16, gated, gated_grad, linear_grad]


@pytest.mark.parametrize("call", ALL)
def test_sizes(lib, call):
    for kw, msg in ((dict(K=100), "K must"), (dict(K=0), "K must"), (dict(N=40), "N must"),
                    (dict(N=0), "N must"), (dict(N=-16), "N must"), (dict(M=-1), "M out of range"),
                    (dict(M=1 << 27), "M out of range"), (dict(K=1 << 27), "K must"),
                    (dict(K=(1 << 22) + 64), "2^22"), (dict(N=(1 << 22) + 16), "2^22"),
                    (dict(K=1 << 22, N=1 << 22), "2^40")):
        assert call(lib, **kw) == INVALID, kw
        assert msg in svdq.svdq_last_error(), (kw, svdq.svdq_last_error())


@pytest.mark.parametrize("call", [gated, gated_grad, linear_grad])
def test_group_and_large_sizes(lib, call):
    assert call(lib, group=128) == UNSUPPORTED
    assert call(lib, M=(1 << 27) - 1, N=1 << 22) == INVALID
    assert "2^40" in svdq.svdq_last_error()


def test_enums(lib):
    assert a16(lib, x_dtype=7) == INVALID and "x_dtype" in svdq.svdq_last_error()
    assert a16(lib, y_dtype=2) == INVALID and "y_dtype" in svdq.svdq_last_error()
    assert a16(lib, bias_dtype=5) == INVALID and "bias_dtype" in svdq.svdq_last_error()
    assert a16(lib, prec=3) == INVALID and "precision" in svdq.svdq_last_error()
    for call in (gated, gated_grad):
        assert call(lib, act=2) == INVALID and "activation" in svdq.svdq_last_error()
    assert gated(lib, h_dtype=3) == INVALID
    assert linear_grad(lib, dx_dtype=3) == INVALID


def test_a16_rows_and_rank(lib):
    assert a16(lib, M=65) == UNSUPPORTED and "64 rows" in svdq.svdq_last_error()
    for r in (8, -16, 272):
        assert a16(lib, rank=r) == INVALID and "rank" in svdq.svdq_last_error()


@pytest.mark.parametrize("call,names", [
    (a16, ("X", "smooth", "down", "up", "wcodes", "wscales", "Y")),
    (gated, ("X", "qg", "sg", "zg", "qu", "su", "zu", "H")),
    (gated_grad, ("dH", "G", "U", "qg", "sg", "zg", "qu", "su", "zu", "dX", "dG", "dU")),
    (linear_grad, ("dY", "q", "s", "z", "dX"))])
def test_null_and_misaligned(lib, call, names):
    for n in names:
        assert call(lib, **{n: None}) == INVALID, n
        assert "NULL" in svdq.svdq_last_error(), n
        assert call(lib, **{n: at(40) + 8}) == INVALID, n
        assert "aligned" in svdq.svdq_last_error(), n
    assert a16(lib, prec=1, ts=None) == INVALID and "w_tensor_scale" in svdq.svdq_last_error()
    assert a16(lib, bias=at(40) + 2) == INVALID and "aligned" in svdq.svdq_last_error()
    assert gated(lib, G=at(20)) == INVALID and "together" in svdq.svdq_last_error()
    assert gated(lib, U=at(20)) == INVALID and "together" in svdq.svdq_last_error()


@pytest.mark.parametrize("call,ins,outs", [
    (a16, ("X", "smooth", "down", "up", "wcodes", "wscales", "bias"), ("Y", "ws")),
    (gated, ("X", "qg", "sg", "zg", "qu", "su", "zu"), ("H", "G", "U")),
    (gated_grad, ("dH", "G", "U", "qg", "sg", "zg", "qu", "su", "zu"), ("dX", "dG", "dU", "ws")),
    (linear_grad, ("dY", "q", "s", "z"), ("dX",))])
def test_overlap(lib, call, ins, outs):
    base = dict(G=at(20), U=at(21)) if call is gated else {}
    if "ws" in outs and call is gated_grad:
        base = dict(M=20, N=1024)               # a size that needs a workspace
    for o in outs:
        for i in ins + tuple(p for p in outs if p != o):
            assert call(lib, **{**base, o: at(30), i: at(30)}) == INVALID, (o, i)
            assert "overlap" in svdq.svdq_last_error(), (o, i)


def test_workspaces(lib):
    sizes = [(1, 64, 16), (64, 128, 64), (65, 1024, 272), (4096, 4096, 12288), (100000, 512, 1024)]
    for m, k, n in sizes:
        for need in (svdq.awq_gated_w4a16_workspace_bytes(m, k, n),
                     svdq.awq_gated_w4a16_grad_workspace_bytes(m, k, n),
                     svdq.awq_linear_w4a16_grad_workspace_bytes(m, k, n)):
            assert need % 256 == 0
    assert svdq.svdq_linear_w4a16_workspace_bytes(64, 128, 64, 32) % 256 == 0
    assert svdq.svdq_linear_w4a16_workspace_bytes(65, 128, 64, 32) == 0
    for f in (svdq.awq_gated_w4a16_workspace_bytes, svdq.awq_gated_w4a16_grad_workspace_bytes,
              svdq.awq_linear_w4a16_grad_workspace_bytes):
        assert f(4, 100, 64) == 0 and f(4, 128, 40) == 0 and f(-1, 128, 64) == 0
    need = svdq.awq_gated_w4a16_grad_workspace_bytes(20, 128, 1024)
    big = dict(M=20, N=1024)
    assert need > 0
    assert gated_grad(lib, **big, nws=need - 1) == INVALID
    assert "too small" in svdq.svdq_last_error()
    assert gated_grad(lib, **big, ws=at(12) + 16) == INVALID and "aligned" in svdq.svdq_last_error()
    assert gated_grad(lib, **big, ws=None) == INVALID and "NULL" in svdq.svdq_last_error()
    need = svdq.svdq_linear_w4a16_workspace_bytes(4, 128, 64, 16)
    assert a16(lib, nws=need - 1) == INVALID and "too small" in svdq.svdq_last_error()


@pytest.mark.parametrize("call", ALL)
def test_zero_rows_need_nothing(lib, call):
    ptrs = ("X", "smooth", "down", "up", "wcodes", "wscales", "ts", "bias", "Y", "ws") \
        if call is a16 else ("X", "qg", "sg", "zg", "qu", "su", "zu", "H", "ws") \
        if call is gated else ("dH", "G", "U", "qg", "sg", "zg", "qu", "su", "zu", "dX", "dG", "dU",
                               "ws") if call is gated_grad else ("dY", "q", "s", "z", "dX", "ws")
    assert call(lib, M=0, nws=0, **{p: None for p in ptrs}) == 0


# ------------------------------------------------------------- the binding

def _awq(n, k):
    return dict(N=n, K=k, group=64, q=torch.zeros(k // 64, n, 32, dtype=torch.uint8),
                scales=torch.zeros(k // 64, n, dtype=torch.int16),
                zeros=torch.zeros(k // 64, n, dtype=torch.int16))


def test_binding_rejects_host_tensors_and_wrong_shapes(lib):
    bf = torch.bfloat16
    x = torch.zeros(4, 128, dtype=bf)
    lay = _awq(64, 128)
    for f in (lambda: svdq.awq_gated_w4a16(x, lay, lay),
              lambda: svdq.awq_linear_w4a16_grad(torch.zeros(4, 64, dtype=bf), lay),
              lambda: svdq.awq_gated_w4a16_grad(*[torch.zeros(4, 64, dtype=bf)] * 3, lay, lay)):
        with pytest.raises(ValueError, match="device tensor"):
            f()
    with pytest.raises(ValueError, match="shape"):
        svdq.awq_gated_w4a16(torch.zeros(4, 64, dtype=bf), lay, lay)
    with pytest.raises(ValueError, match="shape"):
        svdq.awq_linear_w4a16_grad(torch.zeros(64, dtype=bf), lay)


def test_argument_check():
    t = torch.zeros(4, 6)
    assert svdq._arg(t, "t", (4, 6), torch.float32, -1) == t.data_ptr()
    with pytest.raises(TypeError, match="t must be"):
        svdq._arg(t, "t", (4, 6), torch.bfloat16, -1)
    with pytest.raises(ValueError, match="shape"):
        svdq._arg(t, "t", (4, 7), torch.float32, -1)
    with pytest.raises(ValueError, match="contiguous"):
        svdq._arg(t.t(), "t", (6, 4), torch.float32, -1)
    with pytest.raises(ValueError, match="is on cpu"):
        svdq._arg(t, "t", (4, 6), torch.float32, 0)
    with pytest.raises(ValueError, match="layer_up is 64 x 128"):
        svdq._awq_args(_awq(64, 128), 192, 64, -1, "_up")
