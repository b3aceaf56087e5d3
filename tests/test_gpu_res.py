"""GPU parity of awq_linear_w4a16_res (AWQ product with bias, activation, gate and
residual in its epilogue) and its backward pass with the formulas in float64.

Tolerances, per element (u = 2^-24, one fp32 rounding):
  * Z: an fp32 sum of K exact products in any order, K u sum |terms|;
  * act(Z): the slope of SiLU and GELU is at most 1.13 in size, and exp, reciprocal and
    the few products are 16 u of the argument (a dozen roundings);
  * Y: what gate makes of that, and 3 u of the terms added;
  * dZ: 16 u of |dY gate| (1 + |Z|), the activation's derivative being a sum of products
    of the sigmoid and its argument, and half a bf16 step;
  * dX: against the float64 product of the dZ that the call returned: N u sum |terms|;
  * dgate: 16 u |dY| |Z| a term, rows in chains of 16 and 4 in a workgroup and of its
    parts behind: (32 + parts) u sum |terms|;
  * an output rounded to bf16: 2^-8 of the value (half a step).
"""

import pytest
import torch

from oracle import awq as OA
from w4a4_quantized_diffusion_amd import svdq
from tests.gpu_helpers import gm_codes, t_bf16_bits, t_u8
from tests.test_gpu_w4a16 import awq_layer, bf

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def act64(x, act):
    """act and act' in float64."""
    if act == "none":
        return x, torch.ones_like(x)
    if act == "silu":
        s = torch.sigmoid(x)
        return x * s, s + x * s * (1 - s)
    c = (8 / torch.pi) ** 0.5
    s = torch.sigmoid(c * (x + 0.044715 * x ** 3))
    return x * s, s + x * s * (1 - s) * c * (1 + 0.134145 * x ** 2)


def half_step(v, dtype):
    return v.abs() * (2.0 ** -8 if dtype is BF else U)


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance, worst "
                           f"{float((err / tol.clamp_min(1e-300)).max()):.2f} times it")


def per_row(v, m):
    v = v.double()
    return v if v.dim() == 1 else v.repeat_interleave(m // v.shape[0], 0)


def problem(m, k, n, images=1, bias=True, gate=BF, res=BF, seed=0):
    p = dict(x=bf((m, k), 3 + seed), bias=bf((n,), 4 + seed, 0.3) if bias else None, gate=None,
             residual=None, w=awq_layer(n, k, seed))
    if gate is not None:
        p["gate"] = (bf((images, n + 5), 5 + seed).to(gate)[:, 3:3 + n] if images > 1
                     else bf((n,), 5 + seed).to(gate))
    if res is not None:
        p["residual"] = (bf((m, n), 6 + seed).float() * 3.1).to(res)
    return p


def reference(p, act):
    lay, w = p["w"]
    x = p["x"].double()
    z = x @ w.t()
    tz = (x.abs() @ w.abs().t())
    if p["bias"] is not None:
        z, tz = z + p["bias"].double(), tz + p["bias"].double().abs()
    tz = tz * len(w[0]) * U
    y = act64(z, act)[0]
    ty = 1.13 * tz + 16 * U * z.abs()
    if p["gate"] is not None:
        g = per_row(p["gate"], len(x))
        y, ty = y * g, ty * g.abs()
    size = y.abs()
    if p["residual"] is not None:
        y = y + p["residual"].double()
        size = size + p["residual"].double().abs()
    return z, tz, y, ty + 3 * U * (size + y.abs())


def call(p, act, **kw):
    return svdq.awq_linear_w4a16_res(p["x"], p["w"][0], p["bias"], act, p["gate"], p["residual"],
                                     **kw)


def check_forward(p, act, yt=BF, save=True, **kw):
    z, tz, y, ty = reference(p, act)
    out = call(p, act, y_dtype=yt, save=save, **kw)
    got, gz = out if save else (out, None)
    assert got.dtype == yt and got.shape == y.shape
    check(got, y, ty + half_step(y, yt), "Y")
    if save:
        check(gz, z, tz + half_step(z, BF), "Z")


# one launch and two, one to four tiles of rows; 128 x 128 tiles with and without
# slices; 256 x 256 tiles with rows left over for both other forms
SIZES = [(1, 64, 16), (1, 4096, 4096), (3, 128, 48), (16, 704, 272), (17, 512, 1024),
         (33, 8192, 512), (40, 1024, 2064), (64, 64, 16), (64, 4096, 1024), (64, 4160, 8208),
         (65, 256, 144), (130, 1088, 400), (333, 2048, 4112), (500, 64, 16), (1025, 512, 1040),
         (2311, 1024, 4352), (4099, 2048, 4096)]


@pytest.mark.parametrize("m,k,n", SIZES)
def test_sizes(m, k, n):
    act = ("none", "silu", "gelu")[(m + n) % 3]
    check_forward(problem(m, k, n), act)
    check_forward(problem(m, k, n, gate=None, res=F32, bias=False), act, F32, save=False)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("m,k,n,images", [(12, 192, 80, 3), (60, 4096, 512, 60), (300, 512, 272, 2),
                                          (2312, 512, 1040, 8)])
@pytest.mark.parametrize("gate,res,yt", [(BF, BF, BF), (F32, F32, F32), (None, BF, F32),
                                         (BF, None, BF), (F32, BF, BF), (None, None, BF)])
def test_epilogues(act, m, k, n, images, gate, res, yt):
    p = problem(m, k, n, images, gate=gate, res=res, bias=gate is not BF)
    check_forward(p, act, yt)


@pytest.mark.parametrize("m,k,n", [(1, 4096, 64), (50, 2048, 256), (64, 4096, 1024),
                                   (200, 2048, 256), (2048, 2048, 4096)])
def test_exact_sums(m, k, n):
    """Small integers: every partial sum is exact, so is the fp32 output."""
    g = torch.Generator(device="cuda").manual_seed(m)
    q = torch.randint(0, 16, (n, k), generator=g, device="cuda")
    z = torch.randint(0, 16, (n, k // 64), generator=g, device="cuda")
    s = torch.ones(n, k // 64, dtype=torch.float64)
    lay = dict(N=n, K=k, group=64, q=t_u8(gm_codes(OA.pack_nibbles(q.cpu().numpy().astype("uint8")))),
               scales=t_bf16_bits(s.t().contiguous().numpy()),
               zeros=t_bf16_bits(z.double().t().contiguous().cpu().numpy()))
    w = q.double() - z.double().repeat_interleave(64, 1)
    x = torch.randint(-2, 3, (m, k), generator=g, device="cuda").to(BF)
    r = torch.randint(-9, 10, (m, n), generator=g, device="cuda").float()
    y = svdq.awq_linear_w4a16_res(x, lay, residual=r, y_dtype=F32)
    assert torch.equal(y.double(), x.double() @ w.t() + r.double())


def check_grad(m, k, n, images, act, dyt=BF, gate=BF, seed=0):
    p = problem(m, k, n, images, gate=gate, seed=seed)
    lay, w = p["w"]
    dy = (bf((m, n), 11).float() * 1.3).to(dyt)
    z = bf((m, n), 12, 1.5)
    dx, dz, dgate = svdq.awq_linear_w4a16_res_grad(dy, z, lay, act, p["gate"])
    a, da = act64(z.double(), act)
    g = per_row(p["gate"], m) if gate is not None else torch.ones_like(a[:1])
    ref = dy.double() * g * da
    check(dz, ref, 16 * U * (dy.double() * g).abs() * (1 + z.double().abs()) + half_step(ref, BF),
          "dZ")
    d = dz.double()
    ref = d @ w
    check(dx, ref, n * U * (d.abs() @ w.abs()) + half_step(ref, BF), "dX")
    if gate is None:
        assert dgate is None
        return
    each = p["gate"].shape[0] if p["gate"].dim() == 2 else 1
    total = lambda t: t.reshape(each, m // each, n).sum(1).reshape(p["gate"].shape)
    term = dy.double() * a
    parts = images * -(-(m // images) // 64) // each
    assert dgate.dtype == F32 and dgate.shape == p["gate"].shape
    check(dgate, total(term), total((32 + parts) * U * term.abs()
                                    + 16 * U * (dy.double() * z.double()).abs()), "dgate")


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("m,k,n,images", [(1, 64, 16, 1), (20, 2048, 5456, 1), (64, 512, 528, 4),
                                          (130, 256, 144, 1), (600, 512, 1040, 3),
                                          (2304, 1024, 4096, 2), (90, 192, 80, 90)])
def test_grad(act, m, k, n, images):
    check_grad(m, k, n, images, act)
    check_grad(m, k, n, images, act, F32, F32)
    check_grad(m, k, n, images, act, gate=None)


def test_grad_differences():
    """Gradients against central differences of the formula in float64."""
    p = problem(6, 128, 48, 2, gate=F32, res=F32)
    lay, w = p["w"]
    for act in ("none", "silu", "gelu"):
        _, z = call(p, act, y_dtype=F32, save=True)
        dy = bf((6, 48), 21)
        dx, dz, dgate = svdq.awq_linear_w4a16_res_grad(dy, z, lay, act, p["gate"])

        def value(x, gate, bias):
            y = act64(x @ w.t() + bias, act)[0] * gate.repeat_interleave(3, 0)
            return float((y * dy.double()).sum())

        at = [p["x"].double(), p["gate"].double(), p["bias"].double()]
        g = torch.Generator(device="cuda").manual_seed(9)
        for i, got in enumerate((dx.double(), dgate.double(), dz.double().sum(0))):
            v = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
            h = 1e-5
            hi, lo = (value(*[t + s * h * v if j == i else t for j, t in enumerate(at)])
                      for s in (1, -1))
            # Z is rounded to bf16 between the passes (act'' is below 1.2 and |act'| below
            # 1.13: 2 half steps of |dY Z|), dZ and dX are rounded to bf16
            size = float((got * v).abs().sum())
            zs = (dy.double() * per_row(p["gate"], 6) * z.double()).abs()
            extra = [(zs @ w.abs() * v.abs()).sum() if i == 0 else
                     ((dy.double() * z.double()).reshape(2, 3, -1).abs().sum(1) * v.abs()).sum()
                     if i == 1 else (zs.sum(0) * v.abs()).sum()][0]
            # the rounding of dZ reaches dX through the product
            through = (dz.double().abs() @ w.abs() * v.abs()).sum() if i == 0 else 0.0
            tol = 2.0 ** -8 * (size + 2 * float(extra) + float(through)) + 1e-6
            assert abs((hi - lo) / (2 * h) - float((got * v).sum())) <= tol, (act, i)


def test_grad_without_z():
    p = problem(70, 256, 144, 2)
    dy = bf((70, 144), 3)
    full = svdq.awq_linear_w4a16_res_grad(dy, bf((70, 144), 4), p["w"][0], "none", p["gate"])
    none = svdq.awq_linear_w4a16_res_grad(dy, None, p["w"][0], "none", p["gate"], need_dgate=False)
    assert torch.equal(full[0], none[0]) and torch.equal(full[1], none[1]) and none[2] is None


def test_zero_rows():
    p = problem(0, 128, 48)
    y, z = call(p, "gelu", save=True)
    assert y.shape == z.shape == (0, 48)
    dx, dz, dgate = svdq.awq_linear_w4a16_res_grad(y, z, p["w"][0], "gelu", p["gate"])
    assert dx.shape == (0, 128) and not dgate.any() and dgate.shape == (48,)


@pytest.mark.parametrize("m", [1, 40, 100, 2100])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_bad_rows_stay_in_their_rows(m, bad):
    p = problem(m, 512, 1040, res=F32)
    clean = call(p, "silu")
    p["x"][m // 2, 5] = bad
    dirty = call(p, "silu")
    keep = torch.arange(m, device="cuda") != m // 2
    assert torch.equal(clean[keep], dirty[keep])
    assert not torch.isfinite(dirty[m // 2]).any()
    p["x"][m // 2, 5] = 0
    clean = call(p, "silu")
    p["residual"][m // 2, 7] = bad
    dirty = call(p, "silu")
    assert not torch.isfinite(dirty[m // 2, 7])
    dirty[m // 2, 7] = clean[m // 2, 7]
    assert torch.equal(clean, dirty)


@pytest.mark.parametrize("m", [2, 50, 200, 2300])
def test_given_outputs_odd_addresses_and_rows_behind(m):
    n = 1040
    p = problem(m, 512, n, 2 if m > 50 else 1, gate=F32)
    want = call(p, "gelu")
    buf = torch.full((m + 3, n), 7.0, dtype=BF, device="cuda")
    ws = torch.full((svdq.awq_linear_w4a16_res_workspace_bytes(m, 512, n) + 256,), 255,
                    dtype=torch.uint8, device="cuda")
    got = call(p, "gelu", Y=buf[:m], workspace=ws[:-256])
    assert torch.equal(got, want)
    assert bool((buf[m:] == 7).all()) and bool((ws[-256:] == 255).all())
    p["bias"] = torch.cat([p["bias"][:1], p["bias"]])[1:]
    assert torch.equal(call(p, "gelu"), want)


@pytest.mark.parametrize("m", [1, 50, 64, 200, 2300])
def test_stream_graph_and_same_bits(m):
    p = problem(m, 1024, 1040)
    dy, z = bf((m, 1040), 8), bf((m, 1040), 9)
    both = lambda: (call(p, "silu"),) + svdq.awq_linear_w4a16_res_grad(dy, z, p["w"][0], "silu",
                                                                       p["gate"])
    want = both()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = both()
    torch.cuda.current_stream().wait_stream(st)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for i in range(3):
        p["x"].copy_(torch.roll(p["x"], 1, 1))
        dy.copy_(torch.roll(dy, 1, 1))
        graph.replay()
        want = both()
        torch.cuda.synchronize()
        for a, b in zip(want, held):
            assert torch.equal(a, b), i


def split_bytes(m, rows, stages, weights):
    """The workspace of a product whose last round of 256 x 256 tiles is split over the
    reduction: the dequantized weights and S fp32 tiles for each left over."""
    left = -(-m // 256) * -(-rows // 256) % 256
    return weights + left * min(256 // left, 8, stages // 16) * 256 * 256 * 4


# no whole round before the split tiles, and three; ragged edges in both directions
@pytest.mark.parametrize("m,k,n,images", [(1467, 8192, 4112, 3), (4599, 4096, 12304, 9)])
def test_split_rounds(m, k, n, images):
    weights = -(-n // 256) * (k // 32) * 16384
    assert svdq.awq_linear_w4a16_res_workspace_bytes(m, k, n) == split_bytes(m, n, k // 32, weights)
    check_forward(problem(m, k, n, images, gate=F32), "silu")
    check_forward(problem(m, k, n, gate=None, res=F32, bias=False), "none", F32, save=False)


@pytest.mark.parametrize("m,k,n,images", [(2310, 2048, 4112, 2), (1200, 4096, 12304, 3),
                                          (4608, 1024, 4096, 2)])
def test_grad_split_rounds(m, k, n, images):
    pad = -(-n // 64) * 64
    weights = -(-k // 256) * (pad // 32) * 16384
    both = svdq.awq_linear_w4a16_res_grad_workspace_bytes(m, k, n, images)
    assert both > split_bytes(m, k, pad // 32, weights)
    assert both < split_bytes(m, k, pad // 32, weights) + (64 << 20)
    check_grad(m, k, n, images, "gelu")


# few rows and a long reduction: 9 to 16 slices, joined in two turns
@pytest.mark.parametrize("m,k,n,slices", [(18, 5632, 64, 11), (64, 8192, 144, 16), (33, 4672, 16, 9)])
def test_many_slices_of_few_rows(m, k, n, slices):
    assert svdq.awq_linear_w4a16_res_workspace_bytes(m, k, n) == -(-slices * m * n * 4 // 256) * 256
    check_forward(problem(m, k, n, gate=F32), "silu")
    check_forward(problem(m, k, n, gate=None, res=F32, bias=False), "none", F32, save=False)


# a long reduction with few tiles: `slices` of it, joined in two turns or more
@pytest.mark.parametrize("m,length,width,slices",
                         [(65, 8192, 128, 16), (66, 11264, 64, 22), (200, 16384, 192, 32)])
def test_many_slices(m, length, width, slices):
    assert svdq.awq_linear_w4a16_res_workspace_bytes(m, length, width) == slices * m * width * 4
    check_forward(problem(m, length, width, gate=F32), "gelu")
    check_forward(problem(m, length, width, gate=None, res=F32, bias=False), "none", F32, save=False)
    assert svdq.awq_linear_w4a16_res_grad_workspace_bytes(m, width, length, 1) >= slices * m * width * 4
    check_grad(m, width, length, 1, "gelu")


# two sets of waves a tile, with as many chunks and one less; `sums` slices (0: no second
# launch), of two chunks and more
@pytest.mark.parametrize("m,k,n,sums", [(130, 704, 400, 5), (390, 960, 8064, 0), (150, 1088, 2048, 4),
                                        (333, 8192, 2064, 5), (257, 12352, 1040, 9)])
def test_two_sets_of_waves(m, k, n, sums):
    assert svdq.awq_linear_w4a16_res_workspace_bytes(m, k, n) == -(-sums * m * n * 4 // 256) * 256
    check_forward(problem(m, k, n, gate=F32), "silu")
    check_forward(problem(m, k, n, gate=None, res=F32, bias=False), "none", F32, save=False)
    p = problem(m, k, n)
    want = call(p, "gelu")
    p["x"][m // 2, k // 2] = float("inf")
    got = call(p, "gelu")
    keep = torch.arange(m, device=got.device) != m // 2
    assert torch.equal(got[keep], want[keep]) and not got[m // 2].isfinite().any()


@pytest.mark.parametrize("m,k,n", [(333, 8192, 2064), (390, 960, 8064), (64, 8192, 144), (65, 8192, 128)])
def test_two_at_once_and_replayed(m, k, n):
    """Calls on two streams and in a graph that share nothing but their inputs."""
    p = problem(m, k, n)
    dy, z = bf((m, n), 8), bf((m, n), 9)
    both = lambda: (call(p, "gelu"),) + svdq.awq_linear_w4a16_res_grad(dy, z, p["w"][0], "gelu",
                                                                       p["gate"])
    want = both()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(both())
    torch.cuda.synchronize()
    for other in got:
        assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for i in range(3):
        p["x"].copy_(torch.roll(p["x"], 1, 1))
        dy.copy_(torch.roll(dy, 1, 1))
        graph.replay()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held)), i


@pytest.mark.parametrize("m,k,n,images", [(130, 384, 704, 2), (390, 8064, 960, 3), (333, 2048, 8208, 1),
                                          (150, 2048, 1104, 1)])
def test_grad_two_sets_of_waves(m, k, n, images):
    check_grad(m, k, n, images, "gelu")
    check_grad(m, k, n, images, "none", dyt=F32, gate=None)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("m,images", [(1, 1), (20, 4), (64, 2)])
def test_grad_of_few_rows_with_and_without_dgate(act, m, images):
    """Without dgate dZ is formed in the product's launch: the same bits."""
    for gate in (BF, F32):
        p = problem(m, 512, 1040, images, gate=gate)
        dy, z = bf((m, 1040), 3), bf((m, 1040), 4, 1.5)
        full = svdq.awq_linear_w4a16_res_grad(dy, z, p["w"][0], act, p["gate"])
        some = svdq.awq_linear_w4a16_res_grad(dy, z, p["w"][0], act, p["gate"], need_dgate=False)
        assert torch.equal(full[0], some[0]) and torch.equal(full[1], some[1]) and some[2] is None


def test_offsets_past_32_bits():
    """Y, R and Z of more than 2^31 elements; the gate of the last image."""
    m, k, n = 140000, 64, 16384
    lay, w = awq_layer(n, k, 3)
    x = bf((m, k), 1)
    r = torch.empty((m, n), dtype=BF, device="cuda").normal_()
    gate = bf((2, n), 2)
    y, z = svdq.awq_linear_w4a16_res(x, lay, act="silu", gate=gate, residual=r, save=True)
    at = torch.tensor([0, 69999, 70000, 131071, 131072, m - 1], device="cuda")
    ref = x[at].double() @ w.t()
    tol = k * U * (x[at].double().abs() @ w.abs().t())
    check(z[at], ref, tol + half_step(ref, BF), "Z")
    g = gate[(at >= 70000).long()].double()
    a = act64(ref, "silu")[0] * g
    out = a + r[at].double()
    check(y[at], out, (1.13 * tol + 16 * U * ref.abs()) * g.abs() + 4 * U * (a.abs() + out.abs())
          + half_step(out, BF), "Y")
    dx, dz, dgate = svdq.awq_linear_w4a16_res_grad(r, z, lay, "silu", gate)
    d = r[at].double() * g * act64(z[at].double(), "silu")[1]
    check(dz[at], d, 16 * U * (r[at].double() * g).abs() * (1 + z[at].double().abs())
          + half_step(d, BF), "dZ")
    d = dz[at].double()
    check(dx[at], d @ w, n * U * (d.abs() @ w.abs()) + half_step(d @ w, BF), "dX")
    assert torch.isfinite(dgate).all() and dgate.abs().sum() > 0
