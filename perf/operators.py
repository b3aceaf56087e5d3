"""Weight-only 4-bit operators: measured cases and plain forms.

  a16          svdq_linear_w4a16: few rows times an SVDQ layer's 4-bit weights,
               activations kept in 16 or 32 bits
  gated        awq_gated_w4a16: act(X Wg^T + bg) * (X Wu^T + bu)
  gated_grad   awq_gated_w4a16_grad: its backward pass to X and to both
               projections' outputs (frozen weights)
  linear_grad  awq_linear_w4a16_grad: dX = dY W of an AWQ layer

listed() and draw() give cases, prepare() what a program holds before the
call, run() one pass: the framework's call where `own` is true, else the same
mathematics in elementary fp32 torch operations.  exact() is the definition in
64 bits.  An AWQ weight is the bf16 number bf16((q - z) s) by the format's
definition, in every form.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def listed():
    return [
        # the single-layer workload's sizes with one row: a pooled vector's projection
        dict(name="a16 int4 1 row small", op="a16", prec="int4", m=1, k=1024, n=1024, rank=16,
             x32=True, y32=True, bias=True),
        # a block's modulation layer for one image
        dict(name="a16 int4 1 row", op="a16", prec="int4", m=1, k=4096, n=24576, rank=32,
             x32=False, y32=False, bias=True),
        # the same layer type in NVFP4 for a small odd batch
        dict(name="a16 nvfp4 7 rows", op="a16", prec="nvfp4", m=7, k=4096, n=12288, rank=32,
             x32=False, y32=False, bias=False),
        # the most rows of this form, ragged sizes, a folded adapter's rank
        dict(name="a16 int4 61 rows", op="a16", prec="int4", m=61, k=2752, n=10928, rank=48,
             x32=False, y32=True, bias=True),
        # one token through a gated feed-forward block
        dict(name="gated 1 row", op="gated", act="silu", m=1, k=4096, n=12288, h32=False,
             bias=False, save=False),
        # a decoding batch
        dict(name="gated 33 rows", op="gated", act="gelu", m=33, k=2048, n=5456, h32=True,
             bias=True, save=False),
        # a short prompt of odd length, kept for a backward pass
        dict(name="gated 333 rows", op="gated", act="gelu", m=333, k=2048, n=8208, h32=False,
             bias=True, save=True),
        # a long prompt
        dict(name="gated 4096 rows", op="gated", act="silu", m=4096, k=4096, n=12288, h32=False,
             bias=False, save=False),
        # the backward pass of few rows (tuning a soft prompt)
        dict(name="gated_grad 20 rows", op="gated_grad", act="silu", m=20, k=2048, n=5456),
        # the backward pass of a training batch
        dict(name="gated_grad 4096 rows", op="gated_grad", act="gelu", m=4096, k=4096, n=12288),
        # one row back through an attention projection
        dict(name="linear_grad 1 row", op="linear_grad", m=1, k=4096, n=4096, x32=True),
        # the down-projection of the training batch
        dict(name="linear_grad 4099 rows", op="linear_grad", m=4099, k=12288, n=4096, x32=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["a16", "gated", "gated", "gated_grad", "linear_grad"])
    k = 64 * _log(rng, 4, 128)
    n = 16 * _log(rng, 16, 768)
    if op == "a16":
        # K and N of the layers above, any number of rows the form takes
        return dict(op=op, prec=rng.choice(["int4", "nvfp4"]), m=_log(rng, 1, 64), k=k, n=n,
                    rank=16 * rng.randint(0, 6), x32=rng.random() < 0.3, y32=rng.random() < 0.4,
                    bias=rng.random() < 0.5)
    m = _log(rng, 1, 4096)
    while m * k * n > 4096 * 4096 * 12288:
        m = max(1, m // 2)
    if op == "gated":
        return dict(op=op, act=rng.choice(["silu", "gelu"]), m=m, k=k, n=n,
                    h32=rng.random() < 0.3, bias=rng.random() < 0.5, save=rng.random() < 0.4)
    if op == "gated_grad":
        return dict(op=op, act=rng.choice(["silu", "gelu"]), m=m, k=k, n=n)
    return dict(op=op, m=m, k=k, n=n, x32=rng.random() < 0.4)


# ------------------------------------------------------------------ inputs

class _Gen:
    """Seeded draws on the device."""

    def __init__(self, seed):
        self.g = torch.Generator(device=DEV)
        self.g.manual_seed(seed)

    def normal(self, *shape, std=1.0):
        return torch.randn(shape, generator=self.g, device=DEV) * std

    def ints(self, lo, hi, *shape, dtype=torch.int32):
        return torch.randint(lo, hi, shape, generator=self.g, device=DEV, dtype=dtype)

    def uniform(self, lo, hi, *shape):
        return torch.rand(shape, generator=self.g, device=DEV) * (hi - lo) + lo


def _bits(t):
    return t.to(BF16).view(torch.int16)


def _activations(g, m, k):
    """N(0, 1) with one channel in a hundred scaled by 20 to 50, as the
    activations of transformer layers are."""
    x = g.normal(m, k)
    hot = torch.rand(k, generator=g.g, device=DEV) < 0.01
    return x * torch.where(hot, g.uniform(20.0, 50.0, k), torch.ones(k, device=DEV))


def _awq(g, n, k):
    """An AWQ layer whose weights have a standard deviation near 1 / sqrt(K)."""
    return dict(q=g.ints(0, 256, k // 64, n, 32, dtype=torch.uint8),
                scales=_bits(g.uniform(0.7, 1.3, k // 64, n) / (4.6 * math.sqrt(k))),
                zeros=_bits(g.ints(6, 10, k // 64, n).float()), N=n, K=k, group=64)


_GX, _GY = 0x18618618, 0x61861861


def _fold_words(mag, neg):
    """16 signed 4-bit codes (last axis) to one 8-byte chunk of the INT4 fold
    format: field f is |q| | (q < 0) << 5 at bits 6f.. of a 96-bit string
    o0 o1 o2, stored as o0 | (o1 & GX), o2 | (o1 & GY)."""
    f = mag.to(torch.int64) | ((neg & (mag > 0)).to(torch.int64) << 5)
    at = 6 * torch.arange(16, device=DEV)
    words = []
    for w in range(3):
        up = at - 32 * w
        left = torch.where((up >= 0) & (up < 32), f << up.clamp(0, 31), torch.zeros_like(f))
        right = torch.where((up < 0) & (up > -6), f >> (-up).clamp(0, 6), torch.zeros_like(f))
        words.append((left | right).sum(-1) & 0xFFFFFFFF)
    o0, o1, o2 = words
    xy = torch.stack((o0 | (o1 & _GX), o2 | (o1 & _GY)), -1)
    return torch.where(xy >= 1 << 31, xy - (1 << 32), xy).to(torch.int32).contiguous()


def _svdq(g, n, k, rank, prec):
    """An SVDQ layer as the offline quantizer leaves it: uniform codes,
    positive group scales, Gaussian low-rank factors."""
    one = torch.ones(1, device=DEV)
    d = dict(rank=rank, prec=0 if prec == "int4" else 1, N=n, K=k,
             smooth=g.uniform(0.05, 0.5, k), w_tensor_scale=one, x_tensor_scale=one.clone())
    if rank:
        d["lora_down"] = _bits(g.normal(rank, k, std=0.05))
        d["lora_up"] = _bits(g.normal(n, rank, std=0.02))
    else:
        d["lora_down"] = torch.zeros(1, dtype=torch.int16, device=DEV)
        d["lora_up"] = torch.zeros(1, dtype=torch.int16, device=DEV)
    if prec == "int4":
        words = _fold_words(g.ints(0, 8, k // 64, n, 4, 16, dtype=torch.uint8),
                            g.ints(0, 2, k // 64, n, 4, 16, dtype=torch.uint8) == 1)
        d["wcodes"] = words.view(torch.uint8).reshape(k // 64, n, 32)
        d["wscales"] = g.uniform(1e-3, 4e-3, k // 64, n)
    else:
        d["wcodes"] = g.ints(0, 256, k // 64, n, 32, dtype=torch.uint8)
        d["wscales"] = g.ints(0x58, 0x7F, k // 64, n, 4, dtype=torch.uint8)
        d["w_tensor_scale"] = g.uniform(1e-5, 2e-5, 1)
    return d


def prepare(case, seed):
    g = _Gen(seed)
    m, k, n, op = case["m"], case["k"], case["n"], case["op"]
    if op == "a16":
        x = _activations(g, m, k)
        return dict(case=case, x=x if case["x32"] else x.to(BF16),
                    layer=_svdq(g, n, k, case["rank"], case["prec"]),
                    bias=g.normal(n, std=0.02) if case["bias"] else None)
    if op == "linear_grad":
        return dict(case=case, layer=_awq(g, n, k), dy=g.normal(m, n).to(BF16))
    s = dict(case=case, gate=_awq(g, n, k), up=_awq(g, n, k))
    if op == "gated":
        s["x"] = g.normal(m, k).to(BF16)
        for b in ("bias_gate", "bias_up"):
            s[b] = g.normal(n, std=0.1).to(BF16) if case["bias"] else None
    else:
        # pre-activations of both projections as the forward pass kept them
        s["G"], s["U"] = (g.normal(m, n, std=1.5).to(BF16) for _ in range(2))
        s["dh"] = g.normal(m, n).to(BF16)
    return s


# -------------------------------------------------------------- plain forms

def _awq_weight(lay):
    """[N, K] fp32 values bf16((q - z) s)."""
    q, n, k = lay["q"], lay["N"], lay["K"]
    q = torch.stack((q & 15, q >> 4), -1).reshape(k // 64, n, 64).float()
    s = lay["scales"].view(BF16).float().unsqueeze(-1)
    z = lay["zeros"].view(BF16).float().unsqueeze(-1)
    return ((q - z) * s).to(BF16).float().permute(1, 0, 2).reshape(n, k)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _svdq_weight(lay):
    """[N, K] fp32 values of the 4-bit residual weight."""
    n, k = lay["N"], lay["K"]
    if lay["prec"] == 1:
        q = lay["wcodes"]
        c = torch.stack((q & 15, q >> 4), -1).reshape(k // 64, n, 4, 16).long()
        v = torch.tensor(_E2M1 + [-e for e in _E2M1], device=q.device)[c]
        w = v * lay["wscales"].view(torch.float8_e4m3fn).float().unsqueeze(-1)
        w = w * lay["w_tensor_scale"]
        return w.reshape(k // 64, n, 64).permute(1, 0, 2).reshape(n, k)
    xy = lay["wcodes"].contiguous().view(torch.int32).reshape(k // 64, n, 4, 2).long() & 0xFFFFFFFF
    x, y = xy[..., 0:1], xy[..., 1:2]
    o0, o1, o2 = x & ~_GX, (x & _GX) | (y & _GY), y & ~_GY
    low = 6 * torch.arange(11, device=x.device)          # fields 0..10 start in o0, o1
    high = 6 * torch.arange(11, 16, device=x.device) - 64
    first = (o0 | (o1 << 32)) >> low
    first[..., 10] = ((o1 >> 28) & 0xF | (o2 << 4))[..., 0]
    f = torch.cat((first, o2 >> high), -1) & 63
    q = (f & 7).float() * (1 - 2 * (f >> 5)).float()
    # chunk c: fields 0..7 are k = 8c + j, fields 8..15 are k = 32 + 8c + j
    q = q.reshape(k // 64, n, 4, 2, 8).permute(1, 0, 3, 2, 4).reshape(n, k // 64, 64)
    return (q * lay["wscales"].t().unsqueeze(-1)).reshape(n, k)


def _act(x, act):
    """act(x) and its derivative."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return x * s, s * (1 + x * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return (0.5 * x * (1 + t),
            0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x))


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "a16":
        lay, x = s["layer"], s["x"].float()
        y = (x * lay["smooth"]) @ _svdq_weight(lay).t()
        if lay["rank"]:
            down, up = (lay[f].view(BF16).float() for f in ("lora_down", "lora_up"))
            y = y + (x @ down.t()) @ up.t()
        if s["bias"] is not None:
            y = y + s["bias"]
        return y if case["y32"] else y.to(BF16)
    if op == "linear_grad":
        dx = s["dy"].float() @ _awq_weight(s["layer"])
        return dx if case["x32"] else dx.to(BF16)
    if op == "gated":
        x = s["x"].float()
        g, u = (x @ _awq_weight(s[f]).t() for f in ("gate", "up"))
        if case["bias"]:
            g, u = g + s["bias_gate"].float(), u + s["bias_up"].float()
        h = _act(g, case["act"])[0] * u
        h = h if case["h32"] else h.to(BF16)
        return (h, g.to(BF16), u.to(BF16)) if case["save"] else h
    dh, g, u = (s[f].float() for f in ("dh", "G", "U"))
    a, da = _act(g, case["act"])
    dg, du = dh * u * da, dh * a
    dx = dg @ _awq_weight(s["gate"]) + du @ _awq_weight(s["up"])
    return dx.to(BF16), dg.to(BF16), du.to(BF16)


def _framework(s):
    from w4a4_quantized_diffusion_amd import svdq

    case, op = s["case"], s["case"]["op"]
    if op == "a16":
        return svdq.svdq_linear_w4a16(s["x"], s["layer"], s["bias"],
                                      y_dtype=F32 if case["y32"] else BF16)
    if op == "linear_grad":
        return svdq.awq_linear_w4a16_grad(s["dy"], s["layer"],
                                          dx_dtype=F32 if case["x32"] else BF16)
    if op == "gated":
        return svdq.awq_gated_w4a16(s["x"], s["gate"], s["up"], act=case["act"],
                                    bias_gate=s["bias_gate"], bias_up=s["bias_up"],
                                    h_dtype=F32 if case["h32"] else BF16, save=case["save"])
    return svdq.awq_gated_w4a16_grad(s["dh"], s["G"], s["U"], s["gate"], s["up"],
                                     act=case["act"])


def run(state):
    return _framework(state) if own else _plain(state)


def work(case):
    m, k, n, op = case["m"], case["k"], case["n"], case["op"]
    if op == "a16":
        r = case["rank"]
        # codes, scales (one fp32 or four E4M3 per row and 64 weights), smoothing, low-rank factors
        b = n * k // 2 + n * (k // 64) * 4 + 4 * k + 2 * r * (n + k)
        b += m * k * (4 if case["x32"] else 2) + m * n * (4 if case["y32"] else 2)
        b += 4 * n if case["bias"] else 0
        return dict(bytes=b, flops=2 * m * n * k + 2 * m * r * (n + k))
    w = n * k // 2 + n * (k // 64) * 4
    if op == "linear_grad":
        return dict(bytes=w + 2 * m * n + m * k * (4 if case["x32"] else 2), flops=2 * m * n * k)
    if op == "gated":
        b = 2 * w + 2 * m * k + m * n * (4 if case["h32"] else 2)
        b += 4 * m * n if case["save"] else 0
        b += 4 * n if case["bias"] else 0
        return dict(bytes=b, flops=4 * m * n * k)
    return dict(bytes=2 * w + 6 * m * n + 4 * m * n + 2 * m * k, flops=4 * m * n * k)


# -------------------------------------------------------------- definitions

def _nibbles64(packed):
    """[K/64, N, 32] bytes to [N, K] codes, even k in the low half."""
    g, n, _ = packed.shape
    out = torch.empty(n, g, 64, dtype=torch.float64, device=packed.device)
    out[:, :, 0::2] = (packed % 16).transpose(0, 1)
    out[:, :, 1::2] = torch.div(packed, 16, rounding_mode="floor").transpose(0, 1)
    return out


def _awq64(lay):
    s, z = (lay[f].view(BF16).double().t().unsqueeze(-1) for f in ("scales", "zeros"))
    w = (_nibbles64(lay["q"]) - z) * s
    return w.float().bfloat16().double().reshape(lay["N"], lay["K"])


def _svdq64(lay):
    n, k = lay["N"], lay["K"]
    if lay["prec"] == 1:
        c = _nibbles64(lay["wcodes"])
        neg = c >= 8
        c = torch.where(neg, c - 8, c)
        # E2M1: 0, 1/2 subnormal, then (1 + m / 2) 2^(e - 1)
        e, f = torch.div(c, 2, rounding_mode="floor"), c % 2
        v = torch.where(e == 0, f / 2, (1 + f / 2) * 2.0 ** (e - 1))
        v = torch.where(neg, -v, v).reshape(n, k // 16, 16)
        b = lay["wscales"].double().permute(1, 0, 2).reshape(n, k // 16, 1)
        e, f = torch.div(b, 8, rounding_mode="floor"), b % 8   # E4M3, no sign
        b = torch.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e - 7))
        return (v * b).reshape(n, k) * lay["w_tensor_scale"].double()
    raw = lay["wcodes"].cpu().numpy().view("<u4").reshape(k // 64, n, 4, 2)
    x, y = raw[..., 0], raw[..., 1]
    o = (x & np.uint32(~_GX & 0xFFFFFFFF), (x & np.uint32(_GX)) | (y & np.uint32(_GY)),
         y & np.uint32(~_GY & 0xFFFFFFFF))
    q = np.empty((k // 64, n, 64), dtype=np.int8)
    for c in range(4):
        for f in range(16):
            w, b = divmod(6 * f, 32)
            v = o[w][:, :, c] >> np.uint32(b)
            if b > 26:
                v = v | (o[w + 1][:, :, c] << np.uint32(32 - b))
            mag = (v & np.uint32(7)).astype(np.int8)
            at = 8 * c + f if f < 8 else 32 + 8 * c + f - 8
            q[:, :, at] = np.where((v >> np.uint32(5)) & np.uint32(1), -mag, mag)
    q = torch.from_numpy(q).to(lay["wcodes"].device).double()
    return (q * lay["wscales"].double().unsqueeze(-1)).transpose(0, 1).reshape(n, k)


def _act64(x, act):
    if act == "silu":
        s = torch.sigmoid(x)
        return x * s, s + x * s * (1 - s)
    # gelu(x) = x sigmoid(2u)
    c = math.sqrt(8 / math.pi)
    s = torch.sigmoid(c * (x + 0.044715 * x ** 3))
    return x * s, s + x * s * (1 - s) * c * (1 + 0.134145 * x ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "a16":
        lay, x = s["layer"], s["x"].double()
        y = torch.mm(x * lay["smooth"].double(), _svdq64(lay).t().contiguous())
        if lay["rank"]:
            down, up = (lay[f].view(BF16).double().t().contiguous() for f in ("lora_down", "lora_up"))
            y += torch.mm(torch.mm(x, down), up)
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "linear_grad":
        return torch.mm(s["dy"].double(), _awq64(s["layer"]))
    if op == "gated":
        x = s["x"].double()
        g = torch.mm(x, _awq64(s["gate"]).t().contiguous())
        u = torch.mm(x, _awq64(s["up"]).t().contiguous())
        if case["bias"]:
            g += s["bias_gate"].double()
            u += s["bias_up"].double()
        h = _act64(g, case["act"])[0] * u
        return (h, g, u) if case["save"] else h
    dh, g, u = (s[f].double() for f in ("dh", "G", "U"))
    a, da = _act64(g, case["act"])
    dg, du = dh * u * da, dh * a
    return torch.mm(dg, _awq64(s["gate"])) + torch.mm(du, _awq64(s["up"])), dg, du
