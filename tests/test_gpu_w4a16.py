"""GPU parity of the weight-only operators with plain float64 forms, through
the C ABI: svdq_linear_w4a16, awq_gated_w4a16 with its backward pass and
awq_linear_w4a16_grad.

Tolerances, per element, from the operators' roundings:
  * an output rounded to bf16 is off by at most 2^-8 |v| in either direction of
    a slightly different fp32 value (half a step is 2^-9 of the next power of
    two, so 2^-8 |v| is one full half step relative to v);
  * an fp32 sum of L exact products in any order is off by at most
    L 2^-24 sum |terms|; the longest chain of roundings here is far shorter
    (blocks of 16 or 32 inside the matrix unit, partial sums outside), but the
    bound is used as it stands with L the length of the reduction;
  * exp, reciprocal and the activation's few products: 2^-20 relative to the
    factors' magnitudes (a dozen roundings of 2^-24);
  * a bf16 intermediate (dG, dU) adds 2^-8 sum |dG wd| through the product.
"""

import functools

import numpy as np
import pytest
import torch

from oracle import awq as OA
from oracle import formats as F
from oracle import nvfp4 as ON
from oracle import svdq as O
from w4a4_quantized_diffusion_amd import svdq, synth
from tests.gpu_helpers import t_u8, t_f32, t_bf16_bits, gm_codes, layer_to_device

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------- references

@functools.lru_cache(maxsize=16)
def awq_layer(n, k, seed):
    """(device layer, float64 weights bf16((q - z) s) on the device)."""
    g = np.random.default_rng([seed, n, k])
    q = g.integers(0, 16, (n, k)).astype(np.uint8)
    z = g.integers(0, 16, (n, k // 64)).astype(np.float64)
    s = F.bf16((g.uniform(0.5, 1.5, (n, k // 64)) / (4.6 * np.sqrt(k))).astype(np.float32))
    lay = dict(N=n, K=k, group=64, q=t_u8(gm_codes(OA.pack_nibbles(q))),
               scales=t_bf16_bits(np.ascontiguousarray(s.T)),
               zeros=t_bf16_bits(np.ascontiguousarray(z.T)))
    return lay, torch.from_numpy(OA.dequantize_bf16(q, s, z)).cuda()


def bf(shape, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def act64(x, act):
    if act == "silu":
        s = torch.sigmoid(x)
        return x * s, s + x * s * (1 - s)
    c = np.sqrt(8 / np.pi)
    s = torch.sigmoid(c * (x + 0.044715 * x ** 3))
    return x * s, s + x * s * (1 - s) * c * (1 + 0.134145 * x ** 2)


def check(got, ref, tol, what):
    assert torch.isfinite(got).all(), f"{what}: not finite"
    err = (got.double() - ref).abs()
    bad = err > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance, worst "
                           f"{float((err / tol.clamp_min(1e-300)).max()):.2f} times it")


def round_tol(ref, dtype):
    return ref.abs() * 2.0 ** (-8 if dtype is BF else -24)


# ------------------------------------------------------------- gated pair

def gated_ref(x, wg, wu, bg, bu, act):
    """float64 G, U, H and the tolerances of their fp32 values."""
    x = x.double()
    k = x.shape[1]
    out = []
    for w, b in ((wg, bg), (wu, bu)):
        v = x @ w.t()
        t = (x.abs() @ w.abs().t())
        if b is not None:
            v, t = v + b.double(), t + b.double().abs()
        out.append((v, t * k * 2.0 ** -24))
    (g, tg), (u, tu) = out
    a, da = act64(g, act)
    # |act'| <= 1.13 for both activations
    th = 1.13 * tg * u.abs() + (a.abs() + 1.13 * tg) * tu + 2.0 ** -20 * g.abs() * u.abs()
    return (g, tg), (u, tu), (a * u, th)


GATED = [(1, 64, 16), (1, 1024, 2736), (2, 192, 48), (17, 320, 112), (33, 128, 80), (64, 1024, 272),
         (65, 64, 16), (100, 640, 400), (17, 4096, 16), (33, 8192, 272), (64, 4160, 1008), (130, 256, 144), (257, 448, 528), (300, 1088, 272),
         (1030, 512, 768), (2050, 320, 336)]


@pytest.mark.parametrize("m,k,n", GATED)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_forward(m, k, n, act):
    print(f"gated {m} {k} {n} {act}", flush=True)
    gate, wg = awq_layer(n, k, 1)
    up, wu = awq_layer(n, k, 2)
    x = bf((m, k), 3)
    bg, bu = bf((n,), 4, 0.3), bf((n,), 5, 0.3)
    (g, tg), (u, tu), (h, th) = gated_ref(x, wg, wu, bg, bu, act)
    H, G, U = svdq.awq_gated_w4a16(x, gate, up, act, bg, bu, save=True)
    check(H, h, th + round_tol(h, BF) + 1e-30, "H bf16")
    check(G, g, tg + round_tol(g, BF) + 1e-30, "G")
    check(U, u, tu + round_tol(u, BF) + 1e-30, "U")
    # without biases, fp32, into a given tensor whose surroundings stay
    (g, tg), (u, tu), (h, th) = gated_ref(x, wg, wu, None, None, act)
    buf = torch.full((m * n + 512,), float("nan"), device="cuda")
    H32 = svdq.awq_gated_w4a16(x, gate, up, act, H=buf[256:256 + m * n].view(m, n))
    check(H32, h, th + round_tol(h, F32) + 1e-30, "H fp32")
    assert torch.isnan(buf[:256]).all() and torch.isnan(buf[256 + m * n:]).all()
    # the same call gives the same bits, with and without G and U
    assert torch.equal(H32, svdq.awq_gated_w4a16(x, gate, up, act, h_dtype=F32))
    assert torch.equal(H, svdq.awq_gated_w4a16(x, gate, up, act, bg, bu))


@pytest.mark.parametrize("m", [3, 70, 300, 1100])
def test_gated_large_and_zero_gates(m):
    """Pre-activations from -3e4 to 3e4 and exact zeros: the gate saturates to
    0 or passes U through, and nothing becomes NaN."""
    k, n = 128, 64
    gate, wg = awq_layer(n, k, 6)
    up, wu = awq_layer(n, k, 7)
    x = bf((m, k), 8)
    x[0] = 0
    x[1] *= 3e4
    x[2] *= -3e4
    for act in ("silu", "gelu"):
        H, G, U = svdq.awq_gated_w4a16(x, gate, up, act, save=True)
        (g, tg), (u, tu), (h, th) = gated_ref(x, wg, wu, None, None, act)
        check(H, h, th + round_tol(h, BF) + 1e-30, act)
        assert (H[0] == 0).all()
        dh = bf((m, n), 9)
        dX, dG, dU = svdq.awq_gated_w4a16_grad(dh, G, U, gate, up, act)
        assert torch.isfinite(dX).all() and torch.isfinite(dG).all() and torch.isfinite(dU).all()


# ------------------------------------------------------- backward passes

def grad_tol(d, w):
    """fp32 sum over n of |d wd|."""
    return d.abs() @ w.abs() * (d.shape[1] * 2.0 ** -24)


@pytest.mark.parametrize("m,k,n", GATED)
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_backward(m, k, n, act):
    print(f"gated_grad {m} {k} {n} {act}", flush=True)
    gate, wg = awq_layer(n, k, 11)
    up, wu = awq_layer(n, k, 12)
    dh, G, U = bf((m, n), 13), bf((m, n), 14, 2.0), bf((m, n), 15, 2.0)
    dX, dG, dU = svdq.awq_gated_w4a16_grad(dh, G, U, gate, up, act)
    h, g, u = dh.double(), G.double(), U.double()
    a, da = act64(g, act)
    dg, du = h * u * da, h * a
    # act' has terms of size 1 + |g act'|; 2^-20 of them
    check(dG, dg, round_tol(dg, BF) + 2.0 ** -20 * (h * u).abs() * (1 + g.abs()) + 1e-30, "dG")
    check(dU, du, round_tol(du, BF) + 2.0 ** -20 * (h * g).abs() + 1e-30, "dU")
    dx = dG.double() @ wg + dU.double() @ wu
    tol = 2 * (grad_tol(dG.double(), wg) + grad_tol(dU.double(), wu)) + round_tol(dx, BF) + 1e-30
    check(dX, dx, tol, "dX of the returned dG and dU")
    again = svdq.awq_gated_w4a16_grad(dh, G, U, gate, up, act)
    assert all(torch.equal(p, q) for p, q in zip((dX, dG, dU), again))


@pytest.mark.parametrize("m,k,n", GATED)
def test_linear_backward(m, k, n):
    print(f"linear_grad {m} {k} {n}", flush=True)
    lay, w = awq_layer(n, k, 21)
    dy = bf((m, n), 22)
    ref, tol = dy.double() @ w, grad_tol(dy.double(), w)
    dX = svdq.awq_linear_w4a16_grad(dy, lay)
    check(dX, ref, tol + round_tol(ref, BF) + 1e-30, "dX bf16")
    buf = torch.full((m * k + 512,), float("nan"), device="cuda")
    d32 = svdq.awq_linear_w4a16_grad(dy, lay, dX=buf[256:256 + m * k].view(m, k))
    check(d32, ref, tol + round_tol(ref, F32) + 1e-30, "dX fp32")
    assert torch.isnan(buf[:256]).all() and torch.isnan(buf[256 + m * k:]).all()
    assert torch.equal(d32, svdq.awq_linear_w4a16_grad(dy, lay, dx_dtype=F32))


def test_linear_backward_is_the_transpose_of_the_forward():
    """<dY, X W^T> = <dY W, X> with the library's own forward product."""
    m, k, n = 37, 512, 272
    lay, w = awq_layer(n, k, 23)
    x, dy = bf((m, k), 24), bf((m, n), 25)
    y = svdq.awq_linear_w4a16(x, lay, y_dtype=F32)
    dx = svdq.awq_linear_w4a16_grad(dy, lay, dx_dtype=F32)
    a, b = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    size = (dy.double().abs() * (x.double().abs() @ w.abs().t())).sum()
    assert abs(float(a - b)) <= float(size) * (k + n) * 2.0 ** -24


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_gradient_against_differences(act):
    """dG, dU and dX against central differences of the float64 block."""
    m, k, n = 5, 128, 48
    gate, wg = awq_layer(n, k, 26)
    up, wu = awq_layer(n, k, 27)
    x, dh = bf((m, k), 28), bf((m, n), 29)
    _, G, U = svdq.awq_gated_w4a16(x, gate, up, act, save=True)
    dX, dG, dU = svdq.awq_gated_w4a16_grad(dh, G, U, gate, up, act)

    def loss(x):
        return (act64(x @ wg.t(), act)[0] * (x @ wu.t()) * dh.double()).sum()

    d = torch.randn(m, k, dtype=torch.float64, device="cuda",
                    generator=torch.Generator("cuda").manual_seed(30))
    e = 1e-5
    num = float((loss(x.double() + e * d) - loss(x.double() - e * d)) / (2 * e))
    got = float((dX.double() * d).sum())
    # G and U (2^-9 relative each), dG, dU and dX rounded to bf16
    xd = x.double()
    a, da = act64(xd @ wg.t(), act)
    scale = (((dh.double() * (xd @ wu.t())).abs() * 1.13) @ wg.abs()
             + (dh.double() * a).abs() @ wu.abs()) * d.abs()
    # act'' is at most 0.8 in size: a step of 2^-9 |G| in G moves act' by 0.8 2^-9 |G|
    more = (((dh.double() * (xd @ wu.t()) * (xd @ wg.t())).abs()) @ wg.abs()) * d.abs()
    assert abs(num - got) <= float(scale.sum() * 4 * 2.0 ** -8 + more.sum() * 2.0 ** -9)


# several rounds of large tiles, with the rows behind the last full round taken
# by the few-row form (4099) or the smaller tiles (4300, 4396)
MANY = [(4099, 2048, 4112), (4396, 4096, 2064), (4099, 4096, 1040), (4300, 4096, 1040)]


@pytest.mark.parametrize("m,k,n", MANY)
def test_many_rows(m, k, n):
    print(f"many rows {m} {k} {n}", flush=True)
    gate, wg = awq_layer(n, k, 71)
    up, wu = awq_layer(n, k, 72)
    x, bg, bu = bf((m, k), 73), bf((n,), 74, 0.3), bf((n,), 75, 0.3)
    (g, tg), (u, tu), (h, th) = gated_ref(x, wg, wu, bg, bu, "gelu")
    H, G, U = svdq.awq_gated_w4a16(x, gate, up, "gelu", bg, bu, save=True)
    check(H, h, th + round_tol(h, BF) + 1e-30, "H")
    check(G, g, tg + round_tol(g, BF) + 1e-30, "G")
    check(U, u, tu + round_tol(u, BF) + 1e-30, "U")
    buf = torch.full((m * n + 512,), float("nan"), device="cuda")
    H32 = svdq.awq_gated_w4a16(x, gate, up, "gelu", bg, bu, H=buf[256:256 + m * n].view(m, n))
    check(H32, h, th + round_tol(h, F32) + 1e-30, "H fp32")
    assert torch.isnan(buf[:256]).all() and torch.isnan(buf[256 + m * n:]).all()
    dh = bf((m, n), 76)
    dX, dG, dU = svdq.awq_gated_w4a16_grad(dh, G, U, gate, up, "gelu")
    hd, gd, ud = dh.double(), G.double(), U.double()
    a, da = act64(gd, "gelu")
    check(dG, hd * ud * da, round_tol(hd * ud * da, BF)
          + 2.0 ** -20 * (hd * ud).abs() * (1 + gd.abs()) + 1e-30, "dG")
    check(dU, hd * a, round_tol(hd * a, BF) + 2.0 ** -20 * (hd * gd).abs() + 1e-30, "dU")
    dx = dG.double() @ wg + dU.double() @ wu
    check(dX, dx, 2 * (grad_tol(dG.double(), wg) + grad_tol(dU.double(), wu)) + round_tol(dx, BF)
          + 1e-30, "dX")
    ref = dh.double() @ wg
    buf = torch.full((m * k + 512,), float("nan"), device="cuda")
    d32 = svdq.awq_linear_w4a16_grad(dh, gate, dX=buf[256:256 + m * k].view(m, k))
    check(d32, ref, grad_tol(dh.double(), wg) + round_tol(ref, F32) + 1e-30, "linear dX")
    assert torch.isnan(buf[:256]).all() and torch.isnan(buf[256 + m * k:]).all()
    again = svdq.awq_gated_w4a16_grad(dh, G, U, gate, up, "gelu")
    assert all(torch.equal(p, q) for p, q in zip((dX, dG, dU), again))
    assert torch.equal(H32, svdq.awq_gated_w4a16(x, gate, up, "gelu", bg, bu, h_dtype=F32))


# --------------------------------------------------- SVDQ layer, few rows

def svdq_layer(n, k, rank, prec, seed):
    """(device layer, float64 dense parts: smooth, W [N, K], down, up)."""
    g = np.random.default_rng([seed, n, k, rank])
    if prec == "int4":
        r = synth.random_int4_layer(n, k, rank, seed, "small")
        q = O.unpack_int4(r["wcodes"]).astype(np.float64)
        lay = dict(sW=r["sW"], wcodes=r["wcodes"], smooth=r["smooth"],
                   lora_down=F.bf16_to_f32(r["lora_down_bits"]).astype(np.float64),
                   lora_up=F.bf16_to_f32(r["lora_up_bits"]).astype(np.float64))
        d = layer_to_device(lay, rank, n, k)
        w = (q.reshape(n, k // 64, 64) * r["sW"].astype(np.float64)[:, :, None]).reshape(n, k)
        parts = (r["smooth"].astype(np.float64), w, lay["lora_down"], lay["lora_up"])
    else:
        codes = g.integers(0, 256, (n, k // 2)).astype(np.uint8)
        sb = g.integers(1, 0x7F, (n, k // 16)).astype(np.uint8)
        tw = np.float32(1.5e-5)
        smooth = g.uniform(0.05, 0.5, k).astype(np.float32)
        down = F.bf16((g.standard_normal((rank, k)) * 0.05).astype(np.float32))
        up = F.bf16((g.standard_normal((n, rank)) * 0.02).astype(np.float32))
        nib = np.stack((codes & 15, codes >> 4), -1).reshape(n, k)
        val = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])[nib & 7] * np.where(nib & 8, -1.0, 1.0)
        sv = torch.from_numpy(sb).view(torch.float8_e4m3fn).to(torch.float64).numpy()
        w = (val.reshape(n, k // 16, 16) * sv[:, :, None]).reshape(n, k) * np.float64(tw)
        one = torch.ones(1, device="cuda")
        d = dict(rank=rank, prec=1, N=n, K=k, smooth=t_f32(smooth), wcodes=t_u8(gm_codes(codes)),
                 wscales=t_u8(sb.reshape(n, k // 64, 4).transpose(1, 0, 2)),
                 w_tensor_scale=one * float(tw), x_tensor_scale=one,
                 lora_down=t_bf16_bits(down) if rank else torch.zeros(1, dtype=torch.int16, device="cuda"),
                 lora_up=t_bf16_bits(up) if rank else torch.zeros(1, dtype=torch.int16, device="cuda"))
        parts = (smooth.astype(np.float64), w, down, up)
    return d, [torch.from_numpy(np.ascontiguousarray(p)).double().cuda() for p in parts]


def a16_ref(x, parts, bias, split):
    """float64 Y and the tolerance of its fp32 value: the smoothing's rounding
    (2^-24), the bf16 split of Xh (`split`), and the sums over K and rank."""
    smooth, w, down, up = parts
    x = x.double()
    k = x.shape[1]
    xh = x * smooth
    y, t = xh @ w.t(), (xh.abs() @ w.abs().t()) * (k * 2.0 ** -24 + split + 2.0 ** -22)
    if down.shape[0]:
        lr = x @ down.t()
        y = y + lr @ up.t()
        t = t + ((x.abs() @ down.abs().t()) @ up.abs().t()) * ((k + down.shape[0]) * 2.0 ** -24)
    if bias is not None:
        y, t = y + bias.double(), t + bias.double().abs() * 2.0 ** -23
    return y, t


A16 = [(1, 64, 16, 0), (1, 1024, 1024, 16), (2, 128, 48, 32), (3, 1088, 208, 48), (16, 512, 272, 32),
       (17, 640, 400, 0), (33, 192, 144, 256), (48, 2048, 96, 64), (64, 1024, 528, 32),
       (17, 8256, 16, 16), (54, 7424, 256, 48)]


@pytest.mark.parametrize("m,k,n,rank", A16)
@pytest.mark.parametrize("prec", ["int4", "nvfp4"])
def test_linear_a16(m, k, n, rank, prec):
    print(f"a16 {m} {k} {n} {rank} {prec}", flush=True)
    d, parts = svdq_layer(n, k, rank, prec, 31)
    x32 = torch.from_numpy(synth.activations(m, k, 3, 0, 0, bf16=False)).cuda()
    bias = bf((n,), 33)
    for x, b, yt in ((x32, bias.float(), F32), (x32.to(BF), bias, BF), (x32.to(BF), None, F32),
                     (x32, None, BF)):
        y, tol = a16_ref(x, parts, b, 2.0 ** -17 if yt is BF else 2.0 ** -24)
        Y = svdq.svdq_linear_w4a16(x, d, b, y_dtype=yt)
        check(Y, y, tol + round_tol(y, yt) + 1e-30, f"{x.dtype} -> {yt}")
        assert torch.equal(Y, svdq.svdq_linear_w4a16(x, d, b, y_dtype=yt))
    buf = torch.full((m * n + 512,), float("nan"), device="cuda")
    Y = svdq.svdq_linear_w4a16(x32, d, Y=buf[256:256 + m * n].view(m, n))
    y, tol = a16_ref(x32, parts, None, 2.0 ** -24)
    check(Y, y, tol + round_tol(y, F32) + 1e-30, "given Y")
    assert torch.isnan(buf[:256]).all() and torch.isnan(buf[256 + m * n:]).all()


@pytest.mark.parametrize("prec", ["int4", "nvfp4"])
def test_linear_a16_exact_integers(prec):
    """Codes, unit scales and small integers: every product and sum is exact
    in fp32, so Y is too."""
    m, k, n = 11, 512, 176
    d, parts = svdq_layer(n, k, 0, prec, 35)
    x = torch.randint(-8, 9, (m, k), device="cuda").float()
    d["smooth"] = torch.ones(k, device="cuda")
    if prec == "int4":
        w = parts[1] / d["wscales"].double().t().repeat_interleave(64, 1)
        d["wscales"] = torch.ones_like(d["wscales"])
        w = w.round()
    else:
        d["wscales"] = torch.full_like(d["wscales"], 0x38)          # 1.0
        d["w_tensor_scale"] = torch.ones(1, device="cuda")
        q = d["wcodes"].long()
        nib = torch.stack((q & 15, q >> 4), -1).reshape(k // 64, n, 64).transpose(0, 1).reshape(n, k)
        tab = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        w = tab[nib & 7] * torch.where(nib >= 8, -1.0, 1.0).double()
    for xx in (x, x.to(BF)):
        assert torch.equal(svdq.svdq_linear_w4a16(xx, d).double(), x.double() @ w.t())


def test_a16_agrees_with_the_quantized_layer():
    """On rows that the 4-bit activation quantizer represents exactly (integers
    up to 7 with a 7 in each group, unit smoothing), both forms of the layer
    compute the same sums."""
    m, k, n = 8, 256, 96
    d, parts = svdq_layer(n, k, 16, "int4", 36)
    d["smooth"] = torch.ones(k, device="cuda")
    x = torch.randint(-7, 8, (m, k), device="cuda").float()
    x[:, ::64] = 7
    y4, y16 = svdq.svdq_linear_w4a4(x, d), svdq.svdq_linear_w4a16(x, d)
    parts[0] = torch.ones_like(parts[0])
    y, tol = a16_ref(x, parts, None, 2.0 ** -24)
    check(y16, y, tol + round_tol(y, F32), "a16")
    # the quantized layer rounds LR to bf16
    lr = (x.double() @ parts[2].t()).abs() @ parts[3].abs().t() * 2.0 ** -8
    check(y4, y, tol + lr + round_tol(y, F32), "w4a4")


@pytest.mark.parametrize("exponent", [-30, -20, 20, 30])
def test_linear_a16_over_the_range_of_x(exponent):
    """X scaled by 10^e: the terms of Xh keep their relative precision (every
    term and product stays a normal number)."""
    m, k, n = 5, 256, 64
    d, parts = svdq_layer(n, k, 16, "int4", 37)
    g = torch.Generator("cuda").manual_seed(38)
    x = torch.randn(m, k, generator=g, device="cuda") * 10.0 ** exponent
    y, tol = a16_ref(x, parts, None, 2.0 ** -24)
    Y = svdq.svdq_linear_w4a16(x, d)
    check(Y, y, tol + round_tol(y, F32), f"1e{exponent}")


@pytest.mark.parametrize("m", [3, 20, 64, 100, 1100])
def test_a_row_of_nans_stays_in_its_row(m):
    """NaN and infinity in one row of the input leave every other row bit for
    bit as it was, ragged ends of the reduction included."""
    k, n = 320, 336
    gate, _ = awq_layer(n, k, 91)
    up, _ = awq_layer(n, k, 92)
    d, _ = svdq_layer(n, k, 16, "nvfp4", 93)
    x, dy = bf((m, k), 94), bf((m, n), 95)
    calls = [lambda x, dy: svdq.awq_gated_w4a16(x, gate, up),
             lambda x, dy: svdq.awq_linear_w4a16_grad(dy, gate),
             lambda x, dy: svdq.awq_gated_w4a16_grad(dy, dy, dy, gate, up)[0]]
    if m <= 64:
        calls.append(lambda x, dy: svdq.svdq_linear_w4a16(x, d))
    ref = [f(x, dy) for f in calls]
    keep = torch.arange(m, device="cuda") != 1
    for bad in (float("nan"), float("inf")):
        x2, dy2 = x.clone(), dy.clone()
        x2[1], dy2[1] = bad, bad
        for f, r in zip(calls, ref):
            assert torch.equal(f(x2, dy2)[keep], r[keep])


@pytest.mark.parametrize("m,k,n", [(1, 192, 48), (5, 1088, 208), (40, 576, 304), (64, 1856, 5008),
                                   (70, 192, 80), (600, 320, 272), (1100, 192, 528)])
def test_infinite_inputs_show_in_every_output(m, k, n):
    """One infinity in a row makes the whole row of the products infinite or NaN,
    in every form, wherever it lies; the other rows stay finite."""
    gate, _ = awq_layer(n, k, 96)
    up, _ = awq_layer(n, k, 97)
    for at in (0, -3):
        x, dy = bf((m, k), 98), bf((m, n), 99)
        x[m - 1, at], dy[m - 1, at] = float("-inf"), float("inf")
        H, G, U = svdq.awq_gated_w4a16(x, gate, up, "gelu", save=True)
        ones = torch.ones_like(dy)
        out = (H, G, U, svdq.awq_linear_w4a16_grad(dy, gate),
               svdq.awq_gated_w4a16_grad(dy, ones, ones, gate, up)[0])
        for t in out:
            assert not torch.isfinite(t[m - 1]).any() and torch.isfinite(t[:m - 1]).all()


@pytest.mark.parametrize("m,k,n", [(1, 192, 48), (17, 1088, 8208), (64, 320, 272)])
@pytest.mark.parametrize("prec", ["int4", "nvfp4"])
def test_large_and_infinite_inputs_of_a16(m, k, n, prec):
    """svdq_linear_w4a16: a row with an infinity is NaN, and leaves a row with a
    finite value near the top of the range as it is."""
    d, parts = svdq_layer(n, k, 0, prec, 99)
    d["smooth"] = torch.ones_like(d["smooth"])
    x = torch.zeros(m, k, device="cuda")
    x[m - 1, 1] = 3.0e38
    if m > 1:
        x[0, k - 3] = float("inf")
    w = parts[1]
    for yt in (F32, BF):
        Y = svdq.svdq_linear_w4a16(x, d, y_dtype=yt)
        # 3e38 is a finite bf16 sum of terms; its products are in range before the
        # scale (INT4) or tensor scale (NVFP4) where the weight's code is 1 at most.
        # (Beyond that, up to 3e38 x 2688, the products of two terms of opposite
        # sign overflow both, and fp32 holds no value of the sum.)
        scale = d["wscales"][0].double() if prec == "int4" else d["w_tensor_scale"].double()
        fits = w[:, 1].abs() / scale <= 1.001
        ref = x[m - 1, 1].double() * w[:, 1]
        assert fits.any()
        check(Y[m - 1][fits], ref[fits], ref[fits].abs() * 2.0 ** -7, "large")
        if m > 1:
            assert torch.isnan(Y[0]).all() and (Y[1:m - 1] == 0).all()


def test_gate_gradient_far_out():
    """act' between -40 and -80, where it is small but no zero (1e-17 to 1e-33)."""
    m, k, n = 3, 64, 64
    gate, _ = awq_layer(n, k, 87)
    up, _ = awq_layer(n, k, 88)
    G = -torch.linspace(40, 80, m * n, device="cuda").view(m, n).to(BF)
    ones = torch.ones_like(G)
    a, da = act64(G.double(), "silu")
    # exp2's argument is rounded: 2^-24 of 116 moves the result by 116 ln 2 2^-24 < 2^-17,
    # and 1 + x is 1 / 39 of x at least
    _, dG, dU = svdq.awq_gated_w4a16_grad(ones, G, ones, gate, up)
    check(dG, da, da.abs() * 2.0 ** -15 + round_tol(da, BF), "dG")
    check(dU, a, a.abs() * 2.0 ** -15 + round_tol(a, BF), "dU")


def test_offsets_past_32_bits():
    """H and dY of more than 2^31 elements (4.4 GB): the last rows and a sample
    of the others."""
    m, k, n = 180007, 64, 12288
    assert m * n > 1 << 31
    gate, wg = awq_layer(n, k, 81)
    up, wu = awq_layer(n, k, 82)
    x = bf((m, k), 83)
    rows = torch.cat([torch.arange(0, m, 30011), torch.arange(m - 9, m)]).cuda()
    H = svdq.awq_gated_w4a16(x, gate, up)
    _, _, (h, th) = gated_ref(x[rows], wg, wu, None, None, "silu")
    check(H[rows], h, th + round_tol(h, BF) + 1e-30, "H")
    dX = svdq.awq_linear_w4a16_grad(H, gate)
    d = H[rows].double()
    check(dX[rows], d @ wg, grad_tol(d, wg) + round_tol(d @ wg, BF) + 1e-30, "dX")
    dX, dG, dU = svdq.awq_gated_w4a16_grad(H, H, H, gate, up)
    a, da = act64(d, "silu")
    check(dU[rows], d * a, round_tol(d * a, BF) + 2.0 ** -20 * (d * d).abs() + 1e-30, "dU")
    dx = dG[rows].double() @ wg + dU[rows].double() @ wu
    tol = 2 * (grad_tol(dG[rows].double(), wg) + grad_tol(dU[rows].double(), wu))
    check(dX[rows], dx, tol + round_tol(dx, BF) + 1e-30, "dX of the pair")


# ---------------------------------------------- streams, graphs, refusals

def test_zero_rows():
    lay, _ = awq_layer(32, 64, 41)
    d, _ = svdq_layer(32, 64, 16, "int4", 41)
    e = lambda w: torch.empty(0, w, dtype=BF, device="cuda")  # noqa: E731
    assert svdq.awq_gated_w4a16(e(64), lay, lay).shape == (0, 32)
    assert [t.shape for t in svdq.awq_gated_w4a16_grad(e(32), e(32), e(32), lay, lay)] == \
        [(0, 64), (0, 32), (0, 32)]
    assert svdq.awq_linear_w4a16_grad(e(32), lay).shape == (0, 64)
    assert svdq.svdq_linear_w4a16(e(64), d).shape == (0, 32)


def _all_ops(m, k, n):
    gate, _ = awq_layer(n, k, 51)
    up, _ = awq_layer(n, k, 52)
    down, _ = awq_layer(k, n, 53)
    d, _ = svdq_layer(n, k, 32, "int4", 54)
    x, dy = bf((m, k), 55), bf((m, k), 56)

    def run():
        H, G, U = svdq.awq_gated_w4a16(x, gate, up, save=True)
        y = svdq.awq_linear_w4a16(H, down)
        dH = svdq.awq_linear_w4a16_grad(dy, down)
        out = [H, G, U, y, dH, *svdq.awq_gated_w4a16_grad(dH, G, U, gate, up)]
        if m <= 64:
            out.append(svdq.svdq_linear_w4a16(x, d))
        return out
    return x, run


@pytest.mark.parametrize("m", [1, 40, 300, 1100])
def test_captured_and_replayed(m):
    """A block's forward and backward captured in one graph, replayed on
    changing inputs between eager runs of the same calls."""
    k, n = 256, 448
    x, run = _all_ops(m, k, n)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(3):
        x.copy_(bf((m, k), 60 + i))
        eager = run()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), f"replay {i}"


def test_captured_narrow_layers():
    """The forms with many slices and with most of a compute unit's LDS, captured
    with workspaces that hold NaN before every replay."""
    d, _ = svdq_layer(256, 7424, 48, "int4", 71)
    gate, _ = awq_layer(272, 8192, 72)
    up, _ = awq_layer(272, 8192, 73)
    x, x2 = bf((54, 7424), 74), bf((33, 8192), 75)
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
          (svdq.svdq_linear_w4a16_workspace_bytes(54, 7424, 256, 48),
           svdq.awq_gated_w4a16_workspace_bytes(33, 8192, 272))]

    def run():
        return (svdq.svdq_linear_w4a16(x, d, workspace=ws[0]),
                svdq.awq_gated_w4a16(x2, gate, up, workspace=ws[1]))
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(3):
        x.copy_(bf((54, 7424), 76 + i))
        x2.copy_(bf((33, 8192), 86 + i))
        eager = run()
        for w in ws:
            w.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.isfinite(a).all() and torch.equal(a, b) for a, b in zip(out, eager)), i


def test_other_stream_and_dirty_workspace():
    """On another stream than the default, and with workspaces full of NaNs."""
    m, k, n = 37, 256, 320
    x, run = _all_ops(m, k, n)
    ref = run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = run()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    for rows in (m, 300, 1100):
        gate, _ = awq_layer(n, k, 61)
        dy = bf((rows, n), 62)
        need = svdq.awq_linear_w4a16_grad_workspace_bytes(rows, k, n)
        ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(svdq.awq_linear_w4a16_grad(dy, gate),
                           svdq.awq_linear_w4a16_grad(dy, gate, workspace=ws))
        need = svdq.awq_gated_w4a16_grad_workspace_bytes(rows, k, n)
        ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")
        g = svdq.awq_gated_w4a16_grad(dy, dy, dy, gate, gate)
        assert all(torch.equal(a, b) for a, b in zip(
            g, svdq.awq_gated_w4a16_grad(dy, dy, dy, gate, gate, workspace=ws)))
        xx = bf((rows, k), 63)
        need = svdq.awq_gated_w4a16_workspace_bytes(rows, k, n)
        ws = torch.full((max(need, 256),), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(svdq.awq_gated_w4a16(xx, gate, gate),
                           svdq.awq_gated_w4a16(xx, gate, gate, workspace=ws))
