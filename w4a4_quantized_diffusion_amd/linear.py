"""Runtime nn.Linear replacement over the C ABI: the patching shim and the
quantized-layer file format.

The lite integration does not ship model-specific fused kernels: it swaps
the nn.Linear modules of an ordinary model for runtime SVDQ (W4A4) or AWQ
(W4A16) layers (chaosnode.de page, "Nunchaku Lite vs. Original";
aiphreaks.com page, "Bringing Nunchaku 4-bit Diffusion Inference to
Diffusers", Technical Breakdown and Performance Metrics).  Here:

  SVDQLinear      one quantized layer held as device tensors; forward runs
                  svdq_linear_w4a4 (or its GELU-input form) on the current
                  stream.
  AWQLinear       one AWQ W4A16 layer; forward runs awq_linear_w4a16, the
                  gradient of its input awq_linear_w4a16_grad.
  AWQGatedLinear  the gate and up projections of a gated feed-forward block
                  with the activation and the product; forward runs
                  awq_gated_w4a16, backward awq_gated_w4a16_grad.
  calibrate       per-input-channel max|x| of every nn.Linear's inputs
                  (svdq_act_absmax), for the smoothing step.
  quantize_linears  swaps every eligible nn.Linear of a module in place.
  save_quantized / load_quantized
                  the quantized layers of a module in one safetensors file:
                  tensors "<module name>.<field>" and a JSON header entry
                  "svdq" = {"format", "version", "layers": {name: {...}}}.

This module is marshalling only: every step of a layer runs in the HIP
library, and without it the calls raise.
"""

import json

import torch
from torch import nn
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import svdq

FORMAT = "svdq-w4a4-layers"
# version 2: INT4 codes in the fold format (include/svdq.h), written by
# the library's quantizer; version-1 files held textbook nibbles
VERSION = 2

_SVDQ_FIELDS = ("smooth", "lora_down", "lora_up", "wcodes", "wscales", "w_tensor_scale",
                "x_tensor_scale")
_AWQ_FIELDS = ("q", "scales", "zeros")
_GATED_FIELDS = tuple(f"{p}_{f}" for p in ("gate", "up") for f in _AWQ_FIELDS)
_PREC_NAME = {svdq.INT4: "int4", svdq.NVFP4: "nvfp4"}


def _shapes_svdq(n, k, rank, prec):
    """The field shapes and dtypes of one SVDQ layer."""
    ws = ((k // 64, n), torch.float32) if prec == svdq.INT4 else ((k // 64, n, 4), torch.uint8)
    r = max(rank, 1)
    return {"smooth": ((k,), torch.float32), "lora_down": ((r, k) if rank else (1,), torch.int16),
            "lora_up": ((n, r) if rank else (1,), torch.int16),
            "wcodes": ((k // 64, n, 32), torch.uint8), "wscales": ws,
            "w_tensor_scale": ((1,), torch.float32), "x_tensor_scale": ((1,), torch.float32)}


def _shapes_awq(n, k, group):
    return {"q": ((k // group, n, 32), torch.uint8), "scales": ((k // group, n), torch.int16),
            "zeros": ((k // group, n), torch.int16)}


class _BiasCache:
    """The bias in bf16 (awq_linear_w4a16 reads a bf16 bias).  One copy is kept, for
    one tensor, its version and the stream that wrote the copy.  Inside a graph
    capture none is used or left behind: the conversion is captured with the call."""

    source, key, value = None, None, None

    def get(self, bias, dtype):
        if bias is None:
            return None
        if bias.is_inference():                  # has no version to go by
            return bias.to(dtype).contiguous()
        stream = None
        if bias.is_cuda:
            if torch.cuda.is_current_stream_capturing():
                return bias.detach().to(dtype).contiguous()
            stream = svdq._raw_stream(bias.get_device())
        key = (bias.data_ptr(), bias._version, dtype, stream)
        if self.source is not bias or self.key != key:
            self.value = bias.detach().to(dtype).contiguous()
            self.source, self.key = bias, key
        return self.value


def _rows(x, width):
    """x as a contiguous [M, width] matrix at a 16-byte address, as the library takes
    it (autograd hands on expanded and strided gradients, and slices of others)."""
    x = x.reshape(-1, width).contiguous()
    return x.clone() if x.data_ptr() % 16 else x


class SVDQLinear(nn.Module):
    """An SVDQuant W4A4 layer in place of nn.Linear(K, N).

    `layer` is a dict as returned by svdq.svdq_quantize_weights or
    svdq.svdq_fold_lora (device tensors plus rank, prec, N, K).  The bias is
    kept in fp32 and added in fp32 by the library.  With gelu_input the
    layer computes Linear(GELU(x)) (tanh GELU fused into the activation pass;
    x must be bf16).  Inputs of any leading shape [..., K] in fp32 or bf16;
    the output has x's dtype.  The workspace is kept between calls and
    reused on the calling stream: one module must not run on two streams at
    once.  A call captured into a graph has a workspace of its own (the kept one is
    replaced, and freed, by a later call on more rows).

    Inputs of at most `a16_rows` rows (0 to 64, default 0) run
    svdq_linear_w4a16 instead: the same layer with x kept in its own precision,
    for the layers that see a row per image or token (with a workspace of its own
    for every call)."""

    a16_rows = 0                # of layers pickled without it

    def __init__(self, layer, bias=None, gelu_input=False, a16_rows=0):
        super().__init__()
        self.a16_rows = int(a16_rows)
        if not 0 <= self.a16_rows <= 64:
            raise ValueError("a16_rows must be in [0, 64]")
        if self.a16_rows and gelu_input:
            raise ValueError("a16_rows does not go with gelu_input")
        self.in_features, self.out_features = int(layer["K"]), int(layer["N"])
        self.rank, self.prec = int(layer["rank"]), int(svdq._PREC[layer["prec"]])
        self.gelu_input = bool(gelu_input)
        shapes = _shapes_svdq(self.out_features, self.in_features, self.rank, self.prec)
        for f in _SVDQ_FIELDS:
            t = layer[f]
            if self.rank == 0 and f in ("lora_down", "lora_up"):
                t = torch.zeros(1, dtype=torch.int16, device=layer["smooth"].device)
            shape, dt = shapes[f]
            if tuple(t.shape) != shape or t.dtype != dt:
                raise ValueError(f"{f}: expected {shape} {dt}, got {tuple(t.shape)} {t.dtype}")
            self.register_buffer(f, t)
        if bias is not None:
            bias = bias.detach().to(torch.float32).reshape(self.out_features).contiguous()
        self.register_buffer("bias", bias)
        self._ws = None

    @classmethod
    def from_linear(cls, linear, act_amax=None, rank=32, prec="int4", gelu_input=False,
                    a16_rows=0):
        """Quantize an nn.Linear on its (HIP) device with the library's
        offline quantizer; act_amax is its inputs' per-channel max|x| (None:
        no smoothing)."""
        w = linear.weight.detach().to(torch.float32).contiguous()
        lay = svdq.svdq_quantize_weights(w, act_amax, rank, prec)
        return cls(lay, linear.bias, gelu_input, a16_rows)

    def layer(self):
        d = {f: getattr(self, f) for f in _SVDQ_FIELDS}
        d.update(rank=self.rank, prec=self.prec, N=self.out_features, K=self.in_features)
        return d

    def fold_lora(self, A, B, scale=1.0):
        """Carry a LoRA adapter scale * B A in the low-rank branch from now on
        (svdq_fold_lora)."""
        lay = svdq.svdq_fold_lora(self.layer(), A, B, scale)
        self.rank = int(lay["rank"])
        self.lora_down, self.lora_up = lay["lora_down"], lay["lora_up"]
        self._ws = None

    def forward(self, x):
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected [..., {self.in_features}] input, got {tuple(x.shape)}")
        lead = x.shape[:-1]
        x2 = _rows(x, self.in_features)
        m = x2.shape[0]
        if 0 < m <= self.a16_rows:
            # (a workspace of its own for every call: one captured into a graph must
            # outlive the larger one that a later call on more rows brings)
            y = svdq.svdq_linear_w4a16(x2, self.layer(), self.bias, y_dtype=x2.dtype)
            return y.reshape(*lead, self.out_features)
        ws = None
        if not (x2.is_cuda and torch.cuda.is_current_stream_capturing()):
            need = max(svdq.svdq_workspace_bytes(m, self.in_features, self.rank, self.prec), 256)
            if self._ws is None or self._ws.numel() < need or self._ws.device != x2.device:
                self._ws = torch.empty(need, dtype=torch.uint8, device=x2.device)
            ws = self._ws
        fn = svdq.svdq_linear_w4a4_gelu if self.gelu_input else svdq.svdq_linear_w4a4
        y = fn(x2, self.layer(), self.bias, y_dtype=x2.dtype, workspace=ws)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self):
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"rank={self.rank}, prec={_PREC_NAME[self.prec]}, bias={self.bias is not None}, "
                f"gelu_input={self.gelu_input}"
                + (f", a16_rows={self.a16_rows}" if self.a16_rows else ""))


def _save(ctx, *tensors):
    """save_for_backward, which takes no tensors made under inference mode: those (a
    layer's, never changed outside it) are kept as they are."""
    ctx.inference = [t if t.is_inference() else None for t in tensors]
    ctx.save_for_backward(*(None if t.is_inference() else t for t in tensors))


def _saved(ctx):
    return [t if t is not None else i for t, i in zip(ctx.saved_tensors, ctx.inference)]


class _AWQLinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, q, scales, zeros, bias, dims):
        _save(ctx, q, scales, zeros)
        ctx.dims = dims
        return svdq.awq_linear_w4a16(x, dict(dims, q=q, scales=scales, zeros=zeros), bias)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        q, scales, zeros = _saved(ctx)
        lay = dict(ctx.dims, q=q, scales=scales, zeros=zeros)
        dx = svdq.awq_linear_w4a16_grad(_rows(dy, lay["N"]), lay)
        return dx, None, None, None, None, None


class _AWQGatedFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, act, bias_gate, bias_up, dims, *fields):
        n = len(_AWQ_FIELDS)
        gate, up = (dict(dims, **dict(zip(_AWQ_FIELDS, f))) for f in (fields[:n], fields[n:]))
        h, g, u = svdq.awq_gated_w4a16(x, gate, up, act, bias_gate, bias_up, save=True)
        _save(ctx, g, u, *fields)
        ctx.act, ctx.dims = act, dims
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        g, u, *fields = _saved(ctx)
        n = len(_AWQ_FIELDS)
        gate, up = (dict(ctx.dims, **dict(zip(_AWQ_FIELDS, f))) for f in (fields[:n], fields[n:]))
        dx, _, _ = svdq.awq_gated_w4a16_grad(_rows(dh, ctx.dims["N"]), g, u, gate, up, ctx.act)
        return (dx,) + (None,) * (4 + 2 * n)


_FROZEN = "the weights and biases of a quantized layer are frozen: they have no gradient"


def _frozen(*tensors):
    for t in tensors:
        if t is not None and t.requires_grad:
            raise RuntimeError(_FROZEN)


class _FrozenBiasFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, *biases):
        ctx.mark_dirty(y)
        return y

    @staticmethod
    def backward(ctx, dy):
        raise RuntimeError(_FROZEN)


def _frozen_bias(y, *biases):
    """y, whose backward pass raises if a bias is to get a gradient from it."""
    if not torch.is_grad_enabled():
        return y
    leaves = [b for b in biases if b is not None and b.requires_grad]
    return _FrozenBiasFn.apply(y, *leaves) if leaves else y


def _reverse_only(x):
    # (unpack_dual looks at the level too, in 1.5 us)
    if getattr(forward_ad, "_current_level", 0) >= 0 and forward_ad.unpack_dual(x).tangent is not None:
        raise RuntimeError("an AWQ layer has no forward-mode derivative")


class AWQLinear(nn.Module):
    """An AWQ W4A16 layer (asymmetric INT4 weights in groups of 64, bf16
    activations) in place of nn.Linear(K, N).  Inputs bf16 [..., K]; output
    bf16.  Differentiable once in its input, in reverse mode; weights and bias are
    frozen (a gradient asked of the bias raises)."""

    def __init__(self, layer, bias=None):
        super().__init__()
        self.in_features, self.out_features = int(layer["K"]), int(layer["N"])
        self.group = int(layer["group"])
        shapes = _shapes_awq(self.out_features, self.in_features, self.group)
        for f in _AWQ_FIELDS:
            t = layer[f]
            shape, dt = shapes[f]
            if tuple(t.shape) != shape or t.dtype != dt:
                raise ValueError(f"{f}: expected {shape} {dt}, got {tuple(t.shape)} {t.dtype}")
            self.register_buffer(f, t)
        if bias is not None:
            bias = bias.detach().to(torch.float32).reshape(self.out_features).contiguous()
        self.register_buffer("bias", bias)
        self._bias = _BiasCache()

    @classmethod
    def from_linear(cls, linear, group=64):
        lay = svdq.awq_quantize_weights(linear.weight.detach().to(torch.float32).contiguous(), group)
        return cls(lay, linear.bias)

    def forward(self, x):
        if x.dtype != torch.bfloat16:
            raise TypeError("AWQLinear takes bf16 activations")
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected [..., {self.in_features}] input, got {tuple(x.shape)}")
        _reverse_only(x)
        lead = x.shape[:-1]
        x2 = _rows(x, self.in_features)
        lay = dict(q=self.q, scales=self.scales, zeros=self.zeros, N=self.out_features,
                   K=self.in_features, group=self.group)
        bias = self._bias.get(self.bias, torch.bfloat16)
        if torch.is_grad_enabled() and x2.requires_grad:
            _frozen(self.bias)
            fields = [lay.pop(f) for f in _AWQ_FIELDS]
            y = _AWQLinearFn.apply(x2, *fields, bias, lay)
        else:
            y = _frozen_bias(svdq.awq_linear_w4a16(x2, lay, bias), self.bias)
        return y.reshape(*lead, self.out_features)

    def extra_repr(self):
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"group={self.group}, bias={self.bias is not None}")


class AWQGatedLinear(nn.Module):
    """The first half of a gated feed-forward block on two AWQ layers of one
    shape: act(x gate^T + bias_gate) * (x up^T + bias_up), in place of the two
    nn.Linear(K, N), the activation and the product.  act: "silu" or "gelu"
    (tanh form).  Inputs bf16 [..., K]; output bf16.  Differentiable once in its
    input, in reverse mode (the forward pass then keeps both pre-activations in bf16);
    weights and biases are frozen (a gradient asked of a bias raises).  An
    AWQLinear(N, K) behind it completes the block.

    Forward and backward can be captured into a graph together.  A backward pass
    that is captured needs leaves of its own: torch ends the process when an eager
    graph of the same leaves is still alive then."""

    def __init__(self, gate, up, bias_gate=None, bias_up=None, act="silu"):
        super().__init__()
        self.in_features, self.out_features = int(gate["K"]), int(gate["N"])
        self.group = int(gate["group"])
        if (up["K"], up["N"], up["group"]) != (gate["K"], gate["N"], gate["group"]):
            raise ValueError("gate and up must have one shape")
        if act not in ("silu", "gelu"):
            raise ValueError(f"act must be 'silu' or 'gelu', got {act!r}")
        self.act = act
        shapes = _shapes_awq(self.out_features, self.in_features, self.group)
        for p, lay in (("gate", gate), ("up", up)):
            for f in _AWQ_FIELDS:
                t, (shape, dt) = lay[f], shapes[f]
                if tuple(t.shape) != shape or t.dtype != dt:
                    raise ValueError(f"{p}_{f}: expected {shape} {dt}, got {tuple(t.shape)} {t.dtype}")
                self.register_buffer(f"{p}_{f}", t)
        for p, b in (("gate", bias_gate), ("up", bias_up)):
            if b is not None:                    # as awq_gated_w4a16 reads it
                b = b.detach().to(torch.bfloat16).reshape(self.out_features).contiguous()
            self.register_buffer(f"bias_{p}", b)

    @classmethod
    def from_linears(cls, gate, up, act="silu", group=64):
        """Quantize the block's two nn.Linear on their (HIP) device."""
        lays = [svdq.awq_quantize_weights(l.weight.detach().to(torch.float32).contiguous(), group)
                for l in (gate, up)]
        return cls(*lays, gate.bias, up.bias, act)

    def forward(self, x):
        if x.dtype != torch.bfloat16:
            raise TypeError("AWQGatedLinear takes bf16 activations")
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected [..., {self.in_features}] input, got {tuple(x.shape)}")
        _reverse_only(x)
        lead = x.shape[:-1]
        x2 = _rows(x, self.in_features)
        dims = dict(N=self.out_features, K=self.in_features, group=self.group)
        fields = [getattr(self, f) for f in _GATED_FIELDS]
        bg, bu = (b if b is None or b.dtype is torch.bfloat16 else b.detach().to(torch.bfloat16)
                  for b in (self.bias_gate, self.bias_up))
        if torch.is_grad_enabled() and x2.requires_grad:
            _frozen(self.bias_gate, self.bias_up)
            h = _AWQGatedFn.apply(x2, self.act, bg, bu, dims, *fields)
        else:
            n = len(_AWQ_FIELDS)
            gate, up = (dict(dims, **dict(zip(_AWQ_FIELDS, f))) for f in (fields[:n], fields[n:]))
            h = svdq.awq_gated_w4a16(x2, gate, up, self.act, bg, bu)
            h = _frozen_bias(h, self.bias_gate, self.bias_up)
        return h.reshape(*lead, self.out_features)

    def extra_repr(self):
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"group={self.group}, act={self.act}, "
                f"bias={(self.bias_gate is not None, self.bias_up is not None)}")


# ------------------------------------------------------------ patching shim

def eligible(linear, rank=0):
    """Whether the kernels take this nn.Linear: K a multiple of 64, N of 16,
    rank at most min(N, K)."""
    return (isinstance(linear, nn.Linear) and linear.in_features % 64 == 0
            and linear.out_features % 16 == 0 and rank <= min(linear.in_features,
                                                              linear.out_features))


def calibrate(module, run):
    """Per-input-channel max|x| of the inputs of every nn.Linear in `module`
    while `run()` executes (fp32 or bf16 inputs).  Returns {name: amax}."""
    amax, hooks = {}, []

    def hook(name):
        def f(mod, args):
            x = args[0]
            x2 = x.reshape(-1, x.shape[-1]).contiguous()
            if name not in amax:
                amax[name] = torch.zeros(x2.shape[-1], dtype=torch.float32, device=x2.device)
            svdq.svdq_act_absmax(x2, amax[name])
        return f

    for name, mod in module.named_modules():
        if isinstance(mod, nn.Linear):
            hooks.append(mod.register_forward_pre_hook(hook(name)))
    try:
        with torch.no_grad():
            run()
    finally:
        for h in hooks:
            h.remove()
    return amax


def _set_child(root, name, new):
    parent = root
    parts = name.split(".")
    for p in parts[:-1]:
        parent = getattr(parent, p)
    setattr(parent, parts[-1], new)


def quantize_linears(module, act_amax=None, rank=32, prec="int4", awq=(), gelu_input=(),
                     skip=(), a16_rows=0):
    """Swap the nn.Linear modules of `module` in place: names in `awq` become
    AWQLinear, names in `skip` stay, the other eligible ones become
    SVDQLinear (gelu_input for names in `gelu_input`).  act_amax: {name:
    amax} from calibrate (a missing name quantizes without smoothing).
    a16_rows: SVDQLinear's, for the layers without gelu_input.
    Returns {name: kind}."""
    if rank < 0 or rank > 256 or rank % 16:
        raise ValueError("rank must be a multiple of 16 in [0, 256]")
    if not 0 <= int(a16_rows) <= 64:
        raise ValueError("a16_rows must be in [0, 64]")
    act_amax = act_amax or {}
    done = {}
    targets = [(n, m) for n, m in module.named_modules() if isinstance(m, nn.Linear)]
    for name, lin in targets:
        if name in skip:
            continue
        if name in awq:
            if not eligible(lin):
                raise ValueError(f"{name}: shape {lin.out_features}x{lin.in_features} not supported")
            _set_child(module, name, AWQLinear.from_linear(lin))
            done[name] = "awq"
        elif eligible(lin, rank):
            gelu = name in gelu_input
            _set_child(module, name, SVDQLinear.from_linear(lin, act_amax.get(name), rank, prec,
                                                            gelu, 0 if gelu else a16_rows))
            done[name] = "svdq"
    return done


# ------------------------------------------------------------- file format

def _biases(mod, *names):
    return tuple(n for n in names if getattr(mod, n) is not None)


def save_quantized(module, path):
    """Write every SVDQLinear / AWQLinear / AWQGatedLinear of `module` to a
    safetensors file."""
    from safetensors.torch import save_file
    tensors, layers = {}, {}
    for name, mod in module.named_modules():
        if isinstance(mod, SVDQLinear):
            layers[name] = {"kind": "svdq", "prec": _PREC_NAME[mod.prec], "rank": mod.rank,
                            "N": mod.out_features, "K": mod.in_features,
                            "gelu_input": mod.gelu_input, "bias": mod.bias is not None}
            if mod.a16_rows:
                layers[name]["a16_rows"] = mod.a16_rows
            fields = _SVDQ_FIELDS + _biases(mod, "bias")
        elif isinstance(mod, AWQLinear):
            layers[name] = {"kind": "awq", "group": mod.group, "N": mod.out_features,
                            "K": mod.in_features, "bias": mod.bias is not None}
            fields = _AWQ_FIELDS + _biases(mod, "bias")
        elif isinstance(mod, AWQGatedLinear):
            biases = _biases(mod, "bias_gate", "bias_up")
            layers[name] = {"kind": "awq_gated", "group": mod.group, "N": mod.out_features,
                            "K": mod.in_features, "act": mod.act, "biases": list(biases)}
            fields = _GATED_FIELDS + biases
        else:
            continue
        for f in fields:
            tensors[f"{name}.{f}"] = getattr(mod, f).detach().cpu().contiguous()
    meta = {"format": FORMAT, "version": VERSION, "layers": layers}
    save_file(tensors, path, metadata={"svdq": json.dumps(meta)})
    return list(layers)


def load_quantized(module, path, device=None):
    """Put the layers stored by save_quantized into `module` (usually the
    unquantized model's skeleton), replacing the modules of the same names.
    Every tensor is checked against the shapes its header entry implies."""
    from safetensors import safe_open
    with safe_open(path, framework="pt", device="cpu") as f:
        raw = (f.metadata() or {}).get("svdq")
        if raw is None:
            raise ValueError(f"{path}: no svdq header entry")
        meta = json.loads(raw)
        if meta.get("format") != FORMAT or meta.get("version") != VERSION:
            raise ValueError(f"{path}: format {meta.get('format')} v{meta.get('version')} "
                             f"is not {FORMAT} v{VERSION}")
        keys = set(f.keys())

        def take(name, field):
            k = f"{name}.{field}"
            if k not in keys:
                raise ValueError(f"{path}: missing tensor {k}")
            t = f.get_tensor(k)
            return t.to(device) if device is not None else t

        for name, d in meta["layers"].items():
            n, k = int(d["N"]), int(d["K"])
            bias = take(name, "bias") if d.get("bias") else None
            if d["kind"] == "svdq":
                lay = {fld: take(name, fld) for fld in _SVDQ_FIELDS}
                lay.update(rank=int(d["rank"]), prec=svdq._PREC[d["prec"]], N=n, K=k)
                new = SVDQLinear(lay, bias, bool(d.get("gelu_input", False)),
                                 int(d.get("a16_rows", 0)))
            elif d["kind"] == "awq":
                lay = {fld: take(name, fld) for fld in _AWQ_FIELDS}
                lay.update(N=n, K=k, group=int(d["group"]))
                new = AWQLinear(lay, bias)
            elif d["kind"] == "awq_gated":
                lays = [dict({f: take(name, f"{p}_{f}") for f in _AWQ_FIELDS}, N=n, K=k,
                             group=int(d["group"])) for p in ("gate", "up")]
                biases = {b: take(name, b) for b in d["biases"]}
                for b, t in biases.items():
                    if tuple(t.shape) != (n,):
                        raise ValueError(f"{name}.{b}: expected ({n},)")
                new = AWQGatedLinear(*lays, act=d["act"], **biases)
            else:
                raise ValueError(f"{path}: unknown layer kind {d['kind']!r}")
            if bias is not None and tuple(bias.shape) != (n,):
                raise ValueError(f"{name}.bias: expected ({n},)")
            _set_child(module, name, new)
    return list(meta["layers"])
