"""GPU parity of svdq_block_norm and its backward pass with the formulas in float64.

Tolerances, per element, to first order in u = 2^-24 (one fp32 rounding):
  * sums over a row have at most 16 terms in a thread, 6 levels in a wave and 16
    waves one after another: a chain of 38 roundings, 40 u sum |terms|;
  * n = (x' - mean) r: r (40 u mean|x'| + 4 u |x'| + e) + |n| (24 u + r mean(|n| e)),
    e the error of x' (r carries half the variance's 40 u, and 4 of its own roundings);
  * the backward pass's row form dn - mean dn - n mean(dn n) likewise, 64 u of the
    magnitudes it adds, plus what the errors of n put in;
  * sums over rows: the rows of one workgroup one after another, then the workgroups
    in four chains: (rows + workgroups + 8) u sum |terms|, plus the terms' own errors;
  * an output rounded to bf16: 2^-8 of the value (half a step).
"""

import pytest
import torch

from w4a4_quantized_diffusion_amd import svdq

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
NAMES = ("post", "gate", "weight", "scale", "shift")


def draw(g, shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def problem(m, d, kind="layer", images=1, xt=BF, ht=BF, yt=BF, vt=BF, h=True, vectors=NAMES,
            seed=0, x_mean=0.0, shared=()):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1000 * d + m)
    hot = torch.rand(d, generator=g, device="cuda") < 0.02
    p = dict(kind=kind, images=images, yt=yt)
    p["x"] = (draw(g, (m, d), F32, 1.0, x_mean) * torch.where(hot, 30.0, 1.0)).to(xt)
    p["h"] = draw(g, (m, d), ht, 1.3, 0.2) if h else None
    mod = draw(g, (images, 3 * d), vt, 0.4)
    for i, f in enumerate(("gate", "scale", "shift")):
        p[f] = mod[:, i * d:(i + 1) * d] if f in vectors and (h or f != "gate") else None
        if p[f] is not None and f in shared:
            p[f] = p[f][0]
    for f in ("post", "weight"):
        p[f] = draw(g, (d,), vt, 0.3, 1.0) if f in vectors and (h or f != "post") else None
    p["dy"] = draw(g, (m, d), yt)
    p["dx_out"] = draw(g, (m, d), xt) if h else None
    return p


def rows_of(p, f):
    v = p[f]
    if v is None:
        return None
    v = v.double()
    return v if v.dim() == 1 else v.repeat_interleave(len(p["x"]) // v.shape[0], 0)


def norm64(v, e, kind, eps):
    """n, r and the error bound of n, from v with error e."""
    mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    r = ((v - mean).square().mean(-1, keepdim=True) + eps).rsqrt()
    n = (v - mean) * r
    layer = 40 * U * v.abs().mean(-1, keepdim=True) if kind == "layer" else 0.0
    a = r * (layer + 4 * U * v.abs() + e)
    return n, r, a + n.abs() * (24 * U + (n.abs() * a).mean(-1, keepdim=True))


def forward64(p, eps):
    x = p["x"].double()
    z = torch.zeros_like(x)
    s = dict(t=z, e=z)
    if p["h"] is not None:
        t, e = p["h"].double(), z
        if p["post"] is not None:
            s["nh"], s["rh"], s["enh"] = norm64(t, z, p["kind"], eps)
            w = rows_of(p, "post")
            t = s["nh"] * w
            e = s["enh"] * w.abs() + 2 * U * t.abs()
        gate = rows_of(p, "gate")
        gate = torch.ones_like(x[:1]) if gate is None else gate
        s["t"], s["e"] = t, e
        x = x + gate * t
        s["ex"] = gate.abs() * e + 2 * U * (x.abs() + (gate * t).abs())
    else:
        s["ex"] = z
    s["x"] = x
    s["n"], s["r"], s["en"] = norm64(x, s["ex"], p["kind"], eps)
    one = torch.ones_like(x[:1])
    w, sc = rows_of(p, "weight"), rows_of(p, "scale")
    s["w"], s["m"] = one if w is None else w, one if sc is None else 1 + sc
    y = s["n"] * s["w"] * s["m"]
    s["ey"] = s["en"] * (s["w"] * s["m"]).abs() + 4 * U * y.abs()
    sh = rows_of(p, "shift")
    if sh is not None:
        y = y + sh
        s["ey"] = s["ey"] + U * (y.abs() + sh.abs())
    s["y"] = y
    return s


def half_step(v, dtype):
    return v.abs() * (2.0 ** -8 if dtype is BF else U)


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance, worst "
                           f"{float((err / tol.clamp_min(1e-300)).max()):.2f} times it")


def call(p, eps=1e-6, **kw):
    return svdq.svdq_block_norm(p["x"], p["h"], p["kind"], eps, *(p[f] for f in NAMES),
                                y_dtype=p["yt"], **kw)


def call_grad(p, eps=1e-6, **kw):
    return svdq.svdq_block_norm_grad(p["dy"], p["x"], p["h"], p["dx_out"], p["kind"], eps,
                                     *(p[f] for f in NAMES), **kw)


def check_forward(p, eps=1e-6, **kw):
    s = forward64(p, eps)
    out = call(p, eps, **kw)
    if p["h"] is not None:
        xo, y = out
        assert xo.dtype == p["x"].dtype
        check(xo, s["x"], s["ex"] + half_step(s["x"], xo.dtype), "x'")
    else:
        y = out
    assert y.dtype == p["yt"]
    check(y, s["y"], s["ey"] + half_step(s["y"], y.dtype), "y")


def back64(dn, edn, n, r, en, kind):
    """r (dn - [mean dn] - n mean(dn n)) and its error."""
    mean = lambda v: v.mean(-1, keepdim=True)
    m1 = mean(dn) if kind == "layer" else torch.zeros_like(dn[:, :1])
    m2 = mean(dn * n)
    v = r * (dn - m1 - n * m2)
    size = r * (dn.abs() + mean(dn.abs()) + n.abs() * mean((dn * n).abs()))
    e = 64 * U * size + r * (edn + mean(edn) + n.abs() * mean(edn * n.abs()))
    # r's relative error is at most that of n's common factor
    rel = 24 * U + mean(n.abs() * en)
    e = e + r * (en * m2.abs() + n.abs() * mean(dn.abs() * en)) + rel * v.abs()
    return v, e


def check_grad(p, eps=1e-6, **kw):
    s = forward64(p, eps)
    got = dict(zip(("dx", "dh") + tuple("d" + f for f in NAMES), call_grad(p, eps, **kw)))
    m, images = len(p["x"]), p["images"]
    dy = p["dy"].double()
    dn = dy * s["w"] * s["m"]
    g, eg = back64(dn, 3 * U * dn.abs(), s["n"], s["r"], s["en"], p["kind"])
    if p["dx_out"] is not None:
        g = g + p["dx_out"].double()
        eg = eg + U * (g.abs() + p["dx_out"].double().abs())
    check(got["dx"], g, eg + half_step(g, p["x"].dtype), "dx")
    terms = dict(dweight=(dy * s["n"] * s["m"], (dy * s["m"]).abs() * s["en"]),
                 dscale=(dy * s["n"] * s["w"], (dy * s["w"]).abs() * s["en"]),
                 dshift=(dy, 0 * dy))
    if p["h"] is not None:
        gate = rows_of(p, "gate")
        gate = torch.ones_like(g[:1]) if gate is None else gate
        dt, edt = gate * g, gate.abs() * eg + U * (gate * g).abs()
        terms["dgate"] = (g * s["t"], eg * s["t"].abs() + g.abs() * s["e"])
        if p["post"] is not None:
            terms["dpost"] = (dt * s["nh"], edt * s["nh"].abs() + dt.abs() * s["enh"])
            w = rows_of(p, "post")
            dh, edh = back64(dt * w, edt * w.abs() + U * (dt * w).abs(), s["nh"], s["rh"], s["enh"],
                             p["kind"])
        else:
            dh, edh = dt, edt
        check(got["dh"], dh, edh + half_step(dh, p["h"].dtype), "dh")
    else:
        assert got["dh"] is None
    for f in NAMES:
        v = p[f]
        if v is None:
            assert got["d" + f] is None
            continue
        term, e = terms["d" + f]
        each = v.shape[0] if v.dim() == 2 else 1
        total = lambda a: a.reshape(each, m // each, -1).sum(1).reshape(v.shape)
        assert got["d" + f].dtype == F32 and got["d" + f].shape == v.shape
        check(got["d" + f], total(term), total(e) + (min(m, 2048) + 8 + 6) * U * total(term.abs()),
              "d" + f)


SHAPES = [(1, 1), (3, 2), (2, 7), (5, 63), (1, 64), (7, 200), (33, 1000), (4, 1155), (65, 2048),
          (3, 4096), (9, 5455), (2, 8192), (3, 8200), (2, 12288), (1, 16384), (2, 16383), (2, 1025)]


@pytest.mark.parametrize("m,d", SHAPES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_shapes(m, d, kind):
    for xt, yt in ((BF, BF), (F32, F32)):
        p = problem(m, d, kind, xt=xt, ht=xt, yt=yt, vt=xt)
        check_forward(p, 1e-5)
        check_grad(p, 1e-5)


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("ht", [BF, F32])
@pytest.mark.parametrize("yt", [BF, F32])
@pytest.mark.parametrize("vt", [BF, F32])
def test_types(xt, ht, yt, vt):
    p = problem(12, 520, "layer", 3, xt, ht, yt, vt)
    check_forward(p)
    check_grad(p)


@pytest.mark.parametrize("bits", range(32))
def test_vectors(bits):
    vectors = [f for i, f in enumerate(NAMES) if bits >> i & 1]
    kind = "rms" if bits % 3 else "layer"
    for h in (True, False):
        p = problem(10, 328, kind, 2, F32, BF, F32, F32, h=h, vectors=vectors)
        check_forward(p)
        check_grad(p)


@pytest.mark.parametrize("images,rows", [(1, 700), (2, 333), (7, 31), (600, 2), (1030, 1)])
def test_images(images, rows):
    """Vectors of every image, of all rows, and both in one call; more images than
    workgroups, one row an image."""
    for shared in ((), ("scale",), ("gate", "scale", "shift")):
        p = problem(images * rows, 264, "layer", images, shared=shared)
        check_forward(p)
        check_grad(p)


def test_vectors_of_mixed_types_and_places():
    """fp32 and bf16 vectors in one call, rows at odd distances and addresses."""
    p = problem(6, 512, "layer", 3, vt=F32)
    g = torch.Generator(device="cuda").manual_seed(5)
    p["scale"] = draw(g, (3, 1031), BF)[:, 7:519]
    p["gate"] = draw(g, (3, 517), F32)[:, 3:515]
    p["post"] = draw(g, (513,), BF)[1:]
    check_forward(p)
    check_grad(p)
    p["shift"] = draw(g, (1, 512), BF)             # one row: for all rows
    check_forward(p)
    check_grad(p)


def test_odd_addresses():
    """Matrices that start between 16-byte addresses (D a multiple of 8)."""
    p = problem(5, 264, "rms")
    for f in ("x", "h", "dy", "dx_out"):
        t = torch.zeros(5 * 264 + 1, dtype=p[f].dtype, device="cuda")[1:].view(5, 264)
        p[f] = t.copy_(p[f])
    check_forward(p)
    check_grad(p)


def test_large_mean():
    """Layer norm of rows with a mean 10^4 times their deviation."""
    p = problem(4, 4096, "layer", xt=F32, ht=F32, yt=F32, vt=F32, x_mean=1e4)
    check_forward(p)
    check_grad(p)


def test_equal_values():
    p = problem(2, 1024, "layer", h=False, vectors=("shift",))
    p["x"] = torch.full((2, 1024), 3.0, dtype=BF, device="cuda")
    assert torch.equal(call(p), p["shift"].expand(2, -1))
    p["x"].zero_()
    p["kind"] = "rms"
    assert torch.equal(call(p), p["shift"].expand(2, -1))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_bad_rows_stay_in_their_rows(bad):
    p = problem(6, 600, "layer", xt=F32, ht=F32)
    clean = call(p) + call_grad(p)[:2]
    p["x"][1, 7] = bad
    p["h"][4, 599] = bad
    dirty = call(p) + call_grad(p)[:2]
    for a, b in zip(clean, dirty):
        for r in (0, 2, 3, 5):
            assert torch.equal(a[r], b[r])
    for r in (1, 4):
        assert not torch.isfinite(dirty[1][r]).any()


def test_zero_rows():
    p = problem(0, 96, images=1)
    xo, y = call(p)
    assert xo.shape == y.shape == (0, 96)
    got = call_grad(p)
    assert got[0].shape == got[1].shape == (0, 96)
    for v in got[2:]:
        assert not v.any()


def test_given_outputs_and_rows_behind():
    p = problem(5, 256, "layer")
    buf = torch.full((2, 8, 256), 7.0, dtype=BF, device="cuda")
    xo, y = call(p, X_out=buf[0, :5], Y=buf[1, :5])
    want = call(p)
    assert torch.equal(xo, want[0]) and torch.equal(y, want[1])
    assert bool((buf[:, 5:] == 7).all())


def test_need():
    p = problem(40, 300, "rms", 2)
    full = call_grad(p)
    some = call_grad(p, need=(False, True, False, True, False))
    for i, f in enumerate(NAMES):
        if f in ("gate", "scale"):
            assert torch.equal(full[2 + i], some[2 + i])
        else:
            assert some[2 + i] is None
    assert torch.equal(full[0], some[0]) and torch.equal(full[1], some[1])


def test_same_bits_again():
    p = problem(700, 1032, "layer", 2)
    a = call(p) + call_grad(p)
    b = call(p) + call_grad(p)
    for s, t in zip(a, b):
        assert torch.equal(s, t)


def test_differences():
    """The gradient against central differences of the formula in float64, along random
    directions of every input."""
    p = problem(6, 40, "layer", 2, F32, F32, F32, F32)
    names = ("x", "h") + NAMES
    got = dict(zip(names, call_grad(p)))

    def value(q):
        s = forward64(q, 1e-6)
        return float((s["y"] * p["dy"].double()).sum() + (s["x"] * p["dx_out"].double()).sum())

    g = torch.Generator(device="cuda").manual_seed(3)
    for f in names:
        v = torch.randn(p[f].shape, generator=g, device="cuda", dtype=torch.float64)
        step = 1e-5
        hi, lo = (value({**p, f: p[f].double() + s * step * v}) for s in (1, -1))
        want = (hi - lo) / (2 * step)
        have = float((got[f].double() * v).sum())
        # the differences' own error is about step^2 of the third derivative and 1e-16 of
        # the value over the step; the gradient's 64 u of its terms
        size = float((got[f].double() * v).abs().sum())
        assert abs(want - have) <= 256 * U * size + 1e-6 * max(1.0, abs(want)), f


def test_other_stream_and_graph():
    p = problem(37, 1024, "layer")
    want = call(p) + call_grad(p)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = call(p) + call_grad(p)
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call(p) + call_grad(p)
    for i in range(3):
        p["x"].copy_(torch.roll(p["x"], 1, 0))
        p["dy"].copy_(torch.roll(p["dy"], 1, 0))
        graph.replay()
        want = call(p) + call_grad(p)
        torch.cuda.synchronize()
        for a, b in zip(want, held):
            assert torch.equal(a, b), i


def test_offsets_past_32_bits():
    """Matrices of more than 2^31 elements: the last rows as in a small call."""
    m, d = 270000, 8192
    x, h = (torch.empty((m, d), dtype=BF, device="cuda").normal_() for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    scale = draw(g, (2, d), BF, 0.3)
    xo, y = svdq.svdq_block_norm(x, h, "rms", scale=scale)
    a, b = svdq.svdq_block_norm(x[-5:], h[-5:], "rms", scale=scale[1])
    assert torch.equal(xo[-5:], a) and torch.equal(y[-5:], b)
    a, b = svdq.svdq_block_norm(x[:5], h[:5], "rms", scale=scale[0])
    assert torch.equal(xo[:5], a) and torch.equal(y[:5], b)
    del xo
    dx, dh, _, _, _, dscale, _ = svdq.svdq_block_norm_grad(y, x, h, h, "rms", scale=scale)
    small = svdq.svdq_block_norm_grad(y[-5:].contiguous(), x[-5:], h[-5:], h[-5:], "rms",
                                      scale=scale[1])
    assert torch.equal(dx[-5:], small[0]) and torch.equal(dh[-5:], small[1])
    assert torch.isfinite(dscale).all()


def test_gradient_without_the_stream_s():
    """dx_out None with h counts as zeros."""
    p = problem(7, 264, "layer")
    p["dx_out"] = torch.zeros_like(p["x"])
    want = call_grad(p)
    p["dx_out"] = None
    for a, b in zip(want, call_grad(p)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [4100, 5120, 9000, 12288, 16384])
def test_long_rows_of_every_type(d):
    """Two pieces a thread and factors in LDS, whole and with a moved last piece."""
    for xt, ht, yt in ((BF, BF, BF), (F32, BF, F32), (F32, F32, BF)):
        p = problem(6, d, "layer" if xt is BF else "rms", 2, xt, ht, yt, F32)
        check_forward(p)
        check_grad(p)
