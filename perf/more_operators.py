"""What a block puts around its 4-bit layers: measured cases and plain forms.

  norm       svdq_block_norm: x' = x + gate * t, y = n(x') * weight * (1 + scale)
             + shift, with t = h or n(h) * post
  norm_grad  svdq_block_norm_grad: its backward pass, to both inputs and to
             every vector
  res        awq_linear_w4a16_res: R + gate * act(X W^T + bias) on AWQ weights
  res_grad   awq_linear_w4a16_res_grad: its backward pass (frozen weights)
  moe        awq_moe_w4a16: a mixture-of-experts layer on AWQ experts, from the
             router's logits, for few tokens

listed() and draw() give cases, prepare() what a program holds before the
call, run() one pass: the framework's call where `own` is true, else the same
mathematics in elementary fp32 torch operations.  exact() is the definition in
64 bits.  An AWQ weight is the bf16 number bf16((q - z) s) by the format's
definition, in every form.
"""

import math

import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def listed():
    return [
        # one decoded token between two blocks
        dict(name="norm 1 row", op="norm", kind="rms", images=1, rows=1, d=4096, x32=False,
             y32=False, h=True, post=False, gate=False, weight=True, scale=False, shift=False,
             v32=False),
        # a short prompt of odd length, norms before and after the block, an fp32 stream
        # of a width that no vector load divides
        dict(name="norm 333 rows sandwich", op="norm", kind="rms", images=1, rows=333, d=5455,
             x32=True, y32=False, h=True, post=True, gate=True, weight=True, scale=True,
             shift=False, v32=True),
        # two images through a diffusion transformer's block: modulation per image
        dict(name="norm 2 x 4608 rows modulated", op="norm", kind="layer", images=2, rows=4608,
             d=4096, x32=False, y32=False, h=True, post=False, gate=True, weight=False,
             scale=True, shift=True, v32=False),
        # the backward pass of a few rows (tuning a soft prompt)
        dict(name="norm_grad 20 rows", op="norm_grad", kind="rms", images=1, rows=20, d=2048,
             x32=True, y32=False, h=True, post=False, gate=False, weight=True, scale=False,
             shift=False, v32=True),
        # the backward pass of the modulated block, everything in use
        dict(name="norm_grad 2 x 4608 rows", op="norm_grad", kind="layer", images=2, rows=4608,
             d=4096, x32=False, y32=False, h=True, post=True, gate=True, weight=True,
             scale=True, shift=True, v32=False),
        # one token through an output projection, added to the stream
        dict(name="res 1 row", op="res", act="none", images=1, rows=1, k=4096, n=4096,
             bias=False, gate=False, res=True, r32=False, y32=False, save=False),
        # a short prompt of odd length through a down-projection, an fp32 stream
        dict(name="res 333 rows", op="res", act="none", images=1, rows=333, k=8192, n=2064,
             bias=True, gate=True, res=True, r32=True, y32=True, save=False),
        # two images' up-projection with its activation, kept for a backward pass
        dict(name="res 2 x 2304 rows", op="res", act="gelu", images=2, rows=2304, k=4096,
             n=12288, bias=True, gate=False, res=False, r32=False, y32=False, save=True),
        # the backward pass of few rows
        dict(name="res_grad 20 rows", op="res_grad", act="gelu", images=1, rows=20, k=2048,
             n=5456, gate=False),
        # the backward pass of two images through a gated projection
        dict(name="res_grad 2 x 2304 rows", op="res_grad", act="silu", images=2, rows=2304,
             k=4096, n=12288, gate=True),
        # one decoded token through a layer of experts
        dict(name="moe 1 token", op="moe", act="silu", m=1, e=32, top=4, k=2048, n=1024,
             renorm=True, l32=True),
        # a decoding batch that reaches every expert
        dict(name="moe 61 tokens", op="moe", act="gelu", m=61, e=40, top=6, k=4096, n=1408,
             renorm=False, l32=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "res", "res_grad", "moe"])
    flip = lambda p: rng.random() < p
    if op == "moe":
        e = _log(rng, 2, 64)
        case = dict(op=op, act=rng.choice(["silu", "gelu"]), m=_log(rng, 1, 64), e=e,
                    top=rng.randint(1, min(8, e)), k=64 * _log(rng, 4, 64),
                    n=64 * _log(rng, 2, 40), renorm=flip(0.5), l32=flip(0.5))
        while case["e"] * case["k"] * case["n"] > 40 * 4096 * 1408:
            case["k"] = 64 * max(1, case["k"] // 128)
        return case
    images = rng.randint(1, 4)
    rows = max(1, _log(rng, 1, 9216) // images)
    if op in ("norm", "norm_grad"):
        d = _log(rng, 64, 8192)
        if flip(0.6):
            d = (d + 7) // 8 * 8                  # a layer's width, mostly
        while images * rows * d > 2 * 4608 * 4096:
            rows = max(1, rows // 2)
        x32 = flip(0.4)
        h = flip(0.85)
        return dict(op=op, kind=rng.choice(["layer", "rms"]), images=images, rows=rows, d=d,
                    x32=x32, y32=flip(0.3), h=h, post=h and flip(0.5), gate=h and flip(0.6),
                    weight=flip(0.5), scale=flip(0.6), shift=flip(0.5), v32=flip(0.5))
    k, n = 64 * _log(rng, 4, 192), 16 * _log(rng, 16, 768)
    while images * rows * k * n > 4608 * 4096 * 12288:
        rows = max(1, rows // 2)
    act = rng.choice(["none", "silu", "gelu"])
    if op == "res":
        return dict(op=op, act=act, images=images, rows=rows, k=k, n=n, bias=flip(0.5),
                    gate=flip(0.5), res=flip(0.7), r32=flip(0.3), y32=flip(0.3), save=flip(0.4))
    return dict(op=op, act=act, images=images, rows=rows, k=k, n=n,
                gate=flip(0.5) or act == "none")


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


def _hot(g, m, k):
    """N(0, 1) with one channel in a hundred scaled by 20 to 50, as the residual
    stream of a transformer is."""
    x = g.normal(m, k)
    hot = torch.rand(k, generator=g.g, device=DEV) < 0.01
    return x * torch.where(hot, g.uniform(20.0, 50.0, k), torch.ones(k, device=DEV))


def _awq(g, n, k, experts=None):
    """AWQ weights whose standard deviation is near 1 / sqrt(K); `experts` of them
    behind one another."""
    lead = () if experts is None else (experts,)
    bits = lambda t: t.to(BF16).view(torch.int16)
    lay = dict(q=g.ints(0, 256, *lead, k // 64, n, 32, dtype=torch.uint8),
               scales=bits(g.uniform(0.7, 1.3, *lead, k // 64, n) / (4.6 * math.sqrt(k))),
               zeros=bits(g.ints(6, 10, *lead, k // 64, n).float()), N=n, K=k, group=64)
    if experts is not None:
        lay["E"] = experts
    return lay


def prepare(case, seed):
    g = _Gen(seed)
    op = case["op"]
    if op == "moe":
        m, e, k, n = case["m"], case["e"], case["k"], case["n"]
        logits = g.normal(m, e, std=1.5)
        return dict(case=case, x=g.normal(m, k).to(BF16),
                    logits=logits if case["l32"] else logits.to(BF16),
                    gate=_awq(g, n, k, e), up=_awq(g, n, k, e), down=_awq(g, k, n, e))
    images, m = case["images"], case["images"] * case["rows"]
    s = dict(case=case)
    if op in ("norm", "norm_grad"):
        d = case["d"]
        xt = F32 if case["x32"] else BF16
        s["x"] = _hot(g, m, d).to(xt)
        s["h"] = g.normal(m, d).to(xt) if case["h"] else None
        # the modulation layer's output for every image: views of one tensor
        vt = F32 if case["v32"] else BF16
        mod = g.normal(images, 3 * d, std=0.3).to(vt)
        for i, f in enumerate(("gate", "scale", "shift")):
            s[f] = mod[:, i * d:(i + 1) * d] if case[f] else None
        for f in ("post", "weight"):
            s[f] = (1 + g.normal(d, std=0.2)).to(vt) if case[f] else None
        if op == "norm_grad":
            s["dy"] = g.normal(m, d).to(F32 if case["y32"] else BF16)
            s["dx_new"] = g.normal(m, d).to(xt) if case["h"] else None
        return s
    k, n = case["k"], case["n"]
    s["layer"] = _awq(g, n, k)
    s["gate"] = g.normal(images, n, std=0.5).to(BF16) if case["gate"] else None
    if op == "res":
        s["x"] = g.normal(m, k).to(BF16)
        s["bias"] = g.normal(n, std=0.1).to(BF16) if case["bias"] else None
        s["res"] = g.normal(m, n).to(F32 if case["r32"] else BF16) if case["res"] else None
    else:
        # the layer's outputs before the activation, as the forward pass kept them
        s["z"] = g.normal(m, n, std=1.5).to(BF16)
        s["dy"] = g.normal(m, n).to(BF16)
    return s


# -------------------------------------------------------------- plain forms

def _awq_weight(lay):
    """[.., N, K] fp32 values bf16((q - z) s)."""
    q, n, k = lay["q"], lay["N"], lay["K"]
    lead = q.shape[:-3]
    q = torch.stack((q & 15, q >> 4), -1).reshape(*lead, k // 64, n, 64).float()
    s = lay["scales"].view(BF16).float().unsqueeze(-1)
    z = lay["zeros"].view(BF16).float().unsqueeze(-1)
    return ((q - z) * s).to(BF16).float().transpose(-3, -2).reshape(*lead, n, k)


def _act(x, act):
    """act(x) and its derivative."""
    if act == "none":
        return x, torch.ones_like(x)
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return x * s, s * (1 + x * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return (0.5 * x * (1 + t),
            0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x))


def _per_row(v, images, m):
    """A vector [images, D] or [D] for every row, in fp32."""
    if v is None:
        return None
    v = v.float()
    if v.dim() == 1:
        return v
    return v.unsqueeze(1).expand(images, m // images, v.shape[1]).reshape(m, v.shape[1])


def _norm(x, kind):
    """n(x) and the reciprocal deviation."""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _norm_back(dn, n, r, kind):
    out = dn - n * (dn * n).mean(-1, keepdim=True)
    if kind == "layer":
        out = out - dn.mean(-1, keepdim=True)
    return out * r


def _plain_norm(s):
    c = s["case"]
    images, m = c["images"], c["images"] * c["rows"]
    gate, scale, shift = (_per_row(s[f], images, m) for f in ("gate", "scale", "shift"))
    post, weight = (None if s[f] is None else s[f].float() for f in ("post", "weight"))
    x, t = s["x"].float(), None
    if c["h"]:
        t = s["h"].float()
        if post is not None:
            nh, rh = _norm(t, c["kind"])
            t = nh * post
        x = x + (t if gate is None else gate * t)
    n, r = _norm(x, c["kind"])
    a = torch.ones_like(n) if weight is None else weight.expand_as(n)
    if c["op"] == "norm":
        y = n * (a if scale is None else a * (1 + scale))
        y = y if shift is None else y + shift
        y = y if c["y32"] else y.to(BF16)
        return (x if c["x32"] else x.to(BF16), y) if c["h"] else y
    dy = s["dy"].float()
    b = torch.ones_like(n) if scale is None else 1 + scale
    g = _norm_back(dy * a * b, n, r, c["kind"])
    if c["h"]:
        g = g + s["dx_new"].float()
    total = lambda v: v.reshape(images, m // images, -1).sum(1)
    out = dict(dx=g)
    if c["h"]:
        dt = g if gate is None else gate * g
        out["dh"] = dt if post is None else _norm_back(dt * post, nh, rh, c["kind"])
    xt = F32 if c["x32"] else BF16
    out = {f: v.to(xt) for f, v in out.items()}
    if post is not None:
        out["dpost"] = (dt * nh).sum(0)
    if gate is not None:
        out["dgate"] = total(g * t)
    if weight is not None:
        out["dweight"] = (dy * n * b).sum(0)
    if scale is not None:
        out["dscale"] = total(dy * n * a)
    if shift is not None:
        out["dshift"] = total(dy)
    return out


def _plain_res(s):
    c = s["case"]
    images, m = c["images"], c["images"] * c["rows"]
    gate = _per_row(s["gate"], images, m)
    if c["op"] == "res":
        z = s["x"].float() @ _awq_weight(s["layer"]).t()
        if c["bias"]:
            z = z + s["bias"].float()
        y = _act(z, c["act"])[0]
        y = y if gate is None else gate * y
        y = y + s["res"].float() if c["res"] else y
        y = y if c["y32"] else y.to(BF16)
        return (y, z.to(BF16)) if c["save"] else y
    dy, z = s["dy"].float(), s["z"].float()
    a, da = _act(z, c["act"])
    dz = dy * da if gate is None else dy * gate * da
    out = dict(dx=(dz @ _awq_weight(s["layer"])).to(BF16), dz=dz.to(BF16))
    if gate is not None:
        out["dgate"] = (dy * a).reshape(images, m // images, -1).sum(1)
    return out


def _plain_moe(s):
    c = s["case"]
    x, logits = s["x"].float(), s["logits"].float()
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    # equal logits in the order of their indices
    ids = torch.sort(logits, dim=-1, descending=True, stable=True)[1][:, :c["top"]]
    w = torch.gather(p, 1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    dense = torch.zeros_like(p).scatter(1, ids, w)                  # [T, E]
    g, u = (torch.matmul(x.unsqueeze(0), _awq_weight(s[f]).transpose(1, 2).contiguous())
            for f in ("gate", "up"))                                # [E, T, N]
    h = _act(g, c["act"])[0] * u * dense.t().unsqueeze(-1)
    y = torch.matmul(h, _awq_weight(s["down"]).transpose(1, 2).contiguous()).sum(0)
    return y.to(BF16), ids.to(torch.int32), w


def _framework(s):
    from w4a4_quantized_diffusion_amd import svdq

    c, op = s["case"], s["case"]["op"]
    if op == "moe":
        return svdq.awq_moe_w4a16(s["x"], s["logits"], s["gate"], s["up"], s["down"], c["top"],
                                  act=c["act"], renorm=c["renorm"], routing=True)
    if op == "res":
        return svdq.awq_linear_w4a16_res(s["x"], s["layer"], s["bias"], act=c["act"],
                                         gate=s["gate"], residual=s["res"],
                                         y_dtype=F32 if c["y32"] else BF16, save=c["save"])
    if op == "res_grad":
        dx, dz, dgate = svdq.awq_linear_w4a16_res_grad(s["dy"], s["z"], s["layer"], act=c["act"],
                                                       gate=s["gate"])
        return dict(dx=dx, dz=dz) if dgate is None else dict(dx=dx, dz=dz, dgate=dgate)
    vectors = {f: s[f] for f in ("post", "gate", "weight", "scale", "shift")}
    if op == "norm":
        return svdq.svdq_block_norm(s["x"], s["h"], kind=c["kind"], eps=EPS, **vectors,
                                    y_dtype=F32 if c["y32"] else BF16)
    grads = svdq.svdq_block_norm_grad(s["dy"], s["x"], s["h"], s["dx_new"], kind=c["kind"],
                                      eps=EPS, **vectors)
    return {f: v for f, v in zip(("dx", "dh", "dpost", "dgate", "dweight", "dscale", "dshift"),
                                 grads) if v is not None}


def run(state):
    if own:
        return _framework(state)
    op = state["case"]["op"]
    return (_plain_moe if op == "moe" else _plain_res if op.startswith("res")
            else _plain_norm)(state)


def work(case):
    op = case["op"]
    if op == "moe":
        m, e, top, k, n = (case[f] for f in ("m", "e", "top", "k", "n"))
        # experts that tokens choose at random are expected to reach
        active = min(e, e * (1 - (1 - top / e) ** m))
        w = 3 * (n * k // 2 + n * k // 64 * 4)
        return dict(bytes=int(active * w) + m * e * (4 if case["l32"] else 2) + 4 * m * k
                    + 8 * m * top, flops=6 * m * top * k * n)
    images, m = case["images"], case["images"] * case["rows"]
    if op in ("norm", "norm_grad"):
        d = case["d"]
        xs, ys = (4 if case["x32"] else 2), (4 if case["y32"] else 2)
        vs = 4 if case["v32"] else 2
        v = d * (images * (case["gate"] + case["scale"] + (case["shift"] and op == "norm"))
                 + case["post"] + case["weight"])
        if op == "norm":
            b = m * d * (xs * (3 if case["h"] else 1) + ys) + v * vs
            return dict(bytes=b, flops=12 * m * d)
        gv = d * (images * (case["gate"] + case["scale"] + case["shift"])
                  + case["post"] + case["weight"])
        return dict(bytes=m * d * (xs * (5 if case["h"] else 2) + ys) + v * vs + 4 * gv,
                    flops=30 * m * d)
    k, n = case["k"], case["n"]
    b = n * k // 2 + n * (k // 64) * 4 + 2 * m * k + 2 * images * n * case["gate"]
    if op == "res":
        b += 2 * n * case["bias"] + m * n * ((4 if case["y32"] else 2) + 2 * case["save"])
        b += m * n * (4 if case["r32"] else 2) if case["res"] else 0
    else:
        b += 6 * m * n + 4 * images * n * case["gate"]
    return dict(bytes=b, flops=2 * m * n * k)


# -------------------------------------------------------------- definitions

def _awq64(lay, expert=None):
    pick = (lambda t: t) if expert is None else (lambda t: t[expert])
    q = pick(lay["q"])
    g, n, _ = q.shape
    out = torch.empty(n, g, 64, dtype=torch.float64, device=q.device)
    out[:, :, 0::2] = (q % 16).transpose(0, 1)
    out[:, :, 1::2] = torch.div(q, 16, rounding_mode="floor").transpose(0, 1)
    s, z = (pick(lay[f]).view(BF16).double().t().unsqueeze(-1) for f in ("scales", "zeros"))
    return ((out - z) * s).float().bfloat16().double().reshape(n, g * 64)


def _act64(x, act):
    if act == "none":
        return x
    if act == "silu":
        return x * torch.sigmoid(x)
    # gelu(x) = x sigmoid(2u)
    return x * torch.sigmoid(math.sqrt(8 / math.pi) * (x + 0.044715 * x ** 3))


def _norm64(x, kind):
    mu = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    return (x - mu) * torch.rsqrt(((x - mu) ** 2).mean(-1, keepdim=True) + EPS)


def _exact_norm(s):
    c = s["case"]
    images, rows, d = c["images"], c["rows"], c["d"]
    leaf = {f: s[f].double().requires_grad_(c["op"] == "norm_grad")
            for f in ("x", "h", "post", "gate", "weight", "scale", "shift") if s[f] is not None}
    cube = lambda f: leaf[f].reshape(images, rows, d) if f in ("x", "h") else (
        leaf[f].unsqueeze(1) if leaf[f].dim() == 2 else leaf[f])
    x = cube("x")
    if c["h"]:
        t = cube("h")
        if c["post"]:
            t = _norm64(t, c["kind"]) * cube("post")
        x = x + (cube("gate") * t if c["gate"] else t)
    y = _norm64(x, c["kind"])
    if c["weight"]:
        y = y * cube("weight")
    if c["scale"]:
        y = y * (1 + cube("scale"))
    if c["shift"]:
        y = y + cube("shift")
    if c["op"] == "norm":
        return (x.reshape(-1, d), y.reshape(-1, d)) if c["h"] else y.reshape(-1, d)
    value = (y.reshape(-1, d) * s["dy"].double()).sum()
    if c["h"]:
        value = value + (x.reshape(-1, d) * s["dx_new"].double()).sum()
    grads = dict(zip(leaf, torch.autograd.grad(value, list(leaf.values()))))
    return {"d" + f: grads[f] for f in ("x", "h", "post", "gate", "weight", "scale", "shift")
            if f in grads}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        return _exact_norm(s)
    if op == "moe":
        y = torch.zeros(case["m"], case["k"], dtype=torch.float64, device=DEV)
        logits = s["logits"].double()
        ids = torch.argsort(-logits, dim=-1, stable=True)[:, :case["top"]]
        w = torch.softmax(logits, -1).gather(1, ids)
        if case["renorm"]:
            w = torch.softmax(logits.gather(1, ids), -1)
        for e in range(case["e"]):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if not len(t):
                continue
            x = s["x"][t].double()
            gate, up, down = (_awq64(s[f], e).t().contiguous() for f in ("gate", "up", "down"))
            h = _act64(torch.mm(x, gate), case["act"]) * torch.mm(x, up)
            y.index_add_(0, t, w[t, j].unsqueeze(1) * torch.mm(h, down))
        return y, ids.to(torch.int32), w
    images = case["images"]
    gate = None if s["gate"] is None else s["gate"].double().repeat_interleave(case["rows"], 0)
    if op == "res":
        z = torch.mm(s["x"].double(), _awq64(s["layer"]).t().contiguous())
        if case["bias"]:
            z += s["bias"].double()
        y = _act64(z, case["act"])
        if gate is not None:
            y = y * gate
        if case["res"]:
            y = y + s["res"].double()
        return (y, z) if case["save"] else y
    z = s["z"].double().requires_grad_()
    a = _act64(z, case["act"])
    dy = s["dy"].double()
    dz, = torch.autograd.grad(a, z, dy if gate is None else dy * gate)
    out = dict(dx=torch.mm(dz, _awq64(s["layer"])), dz=dz)
    if gate is not None:
        out["dgate"] = (dy * a.detach()).reshape(images, case["rows"], -1).sum(1)
    return out
