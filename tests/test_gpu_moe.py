"""GPU parity of awq_moe_w4a16 (a mixture-of-experts layer for few tokens) with the
formulas in float64.

Tolerances, per element (u = 2^-24, one fp32 rounding): G and U are fp32 sums of K exact
products, K u sum |terms|; act has a slope of at most 1.13 and 16 u of its own (exp,
reciprocal, a few products); H = act(G) U is rounded to bf16, 2^-8 of it; the
down-projection sums N products, N u sum |terms|; a weight p is a quotient of
exponentials and a sum of at most E of them, (E + 16) u of it (exp's argument, a
difference of logits below 2^5 in size, is off by at most 2^5 u); Y adds top of those
terms and is rounded, 2^-8.  Choices are exact.
"""

import pytest
import torch

from w4a4_quantized_diffusion_amd import svdq

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def experts(e, n, k, seed):
    g = gen(seed)
    bits = lambda t: t.to(BF).view(torch.int16)
    rand = lambda *s: torch.rand(s, generator=g, device="cuda")
    return dict(E=e, N=n, K=k, group=64,
                q=torch.randint(0, 256, (e, k // 64, n, 32), generator=g, device="cuda",
                                dtype=torch.uint8),
                scales=bits((0.5 + rand(e, k // 64, n)) / (4.6 * k ** 0.5)),
                zeros=bits(torch.randint(5, 11, (e, k // 64, n), generator=g, device="cuda").float()))


def weight(lay, e):
    q = lay["q"][e]
    c = torch.stack((q & 15, q >> 4), -1).reshape(q.shape[0], q.shape[1], 64).double()
    s, z = (lay[f][e].view(BF).double().unsqueeze(-1) for f in ("scales", "zeros"))
    return ((c - z) * s).float().to(BF).double().transpose(0, 1).reshape(lay["N"], lay["K"])


def act64(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    return x * torch.sigmoid((8 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3))


def problem(t, e, top, k, n, lt=F32, seed=0, std=1.5):
    g = gen(seed + t)
    return dict(x=torch.randn(t, k, generator=g, device="cuda").to(BF), top=top,
                logits=(torch.randn(t, e, generator=g, device="cuda") * std).to(lt),
                gate=experts(e, n, k, seed + 1), up=experts(e, n, k, seed + 2),
                down=experts(e, k, n, seed + 3))


def reference(p, act, renorm):
    x, logits, top = p["x"].double(), p["logits"].double(), p["top"]
    (t, k), e, n = x.shape, logits.shape[1], p["gate"]["N"]
    ids = torch.sort(logits, dim=-1, descending=True, stable=True)[1][:, :top]
    w = torch.softmax(logits, -1).gather(1, ids)
    if renorm:
        w = w / w.sum(-1, keepdim=True)
    y, ty = torch.zeros_like(x), torch.zeros_like(x)
    for i in range(e):
        at, j = torch.nonzero(ids == i, as_tuple=True)
        if not len(at):
            continue
        wg, wu, wd = (weight(p[f], i) for f in ("gate", "up", "down"))
        xs, ws = x[at], w[at, j].unsqueeze(1)
        g, u = xs @ wg.t(), xs @ wu.t()
        tg, tu = (k * U * (xs.abs() @ m.abs().t()) for m in (wg, wu))
        a = act64(g, act)
        h = a * u
        th = (1.13 * tg + 16 * U * g.abs()) * u.abs() + a.abs() * tu
        th = th * (1 + 2.0 ** -8) + 2.0 ** -8 * h.abs()
        size = h.abs() @ wd.abs().t()
        y.index_add_(0, at, ws * (h @ wd.t()))
        ty.index_add_(0, at, ws * (th @ wd.abs().t() + ((n + e + 32 + top) * U) * size))
    return y, ty, ids, w


def check(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance, worst "
                           f"{float((err / tol.clamp_min(1e-300)).max()):.2f} times it")


def call(p, act="silu", renorm=True, **kw):
    return svdq.awq_moe_w4a16(p["x"], p["logits"], p["gate"], p["up"], p["down"], p["top"], act,
                              renorm, **kw)


def check_all(p, act="silu", renorm=True):
    y, ty, ids, w = reference(p, act, renorm)
    gy, gi, gw = call(p, act, renorm, routing=True)
    assert gi.dtype == torch.int32 and torch.equal(gi.long(), ids)
    check(gw, w, (p["logits"].shape[1] + 48) * U * w + 1e-44, "weights")
    check(gy, y, ty + 2.0 ** -8 * y.abs(), "Y")
    assert torch.equal(call(p, act, renorm), gy)


# one token; more waves than chunks and experts than waves; every tile height; one
# expert for all; the most of everything
SIZES = [(1, 4, 2, 64, 64), (1, 1, 1, 128, 64), (2, 3, 3, 192, 128), (5, 8, 2, 1024, 320),
         (16, 16, 4, 256, 64), (17, 5, 2, 576, 192), (33, 2, 2, 320, 128), (40, 3, 1, 128, 704),
         (64, 64, 8, 128, 64), (64, 1, 1, 256, 64), (61, 40, 6, 512, 192), (64, 256, 16, 64, 64),
         (1, 256, 8, 128, 64), (31, 17, 5, 4096, 64), (7, 100, 3, 64, 2048)]


@pytest.mark.parametrize("t,e,top,k,n", SIZES)
def test_sizes(t, e, top, k, n):
    act = "gelu" if (t + e) % 2 else "silu"
    check_all(problem(t, e, top, k, n), act, True)
    check_all(problem(t, e, top, k, n, BF, seed=7), act, False)


@pytest.mark.parametrize("t,used", [(64, 1), (64, 2), (50, 1), (30, 1), (64, 16)])
def test_uneven_loads(t, used):
    """Every token's choices among the first few experts: tiles of up to 64 rows."""
    p = problem(t, 24, min(used, 2), 256, 128)
    p["logits"][:, used:] -= 100
    check_all(p)


def test_ties_go_to_the_lower_expert():
    p = problem(9, 70, 4, 64, 64, BF)
    p["logits"][:4] = 0.5                       # all equal
    p["logits"][4, ::3] = 3.0                   # 24 equal ones
    p["logits"][5] = 0.0
    p["logits"][5, 1::2] = -0.0                 # a zero is a zero
    p["logits"][6] = float("-inf")
    p["logits"][6, 60] = 1.0                    # one left: then the masked ones in order
    check_all(p)
    ids = call(p, routing=True)[1]
    assert ids[0].tolist() == [0, 1, 2, 3] and ids[5].tolist() == [0, 1, 2, 3]
    assert ids[6].tolist() == [60, 0, 1, 2]
    # (expert 52 drew more than 3)
    assert p["logits"][4, 52] > 3 and ids[4].tolist() == [52, 0, 3, 6]


def test_large_logits():
    p = problem(6, 12, 3, 64, 64)
    p["logits"] = p["logits"] * 3 + torch.tensor([[3e38], [-3e38], [1e4], [-1e4], [80.], [0.]],
                                                 device="cuda")
    check_all(p, renorm=False)


def test_infinite_logits():
    """+infinity is a tie for the first place or alone there, and makes its token NaN as
    the softmax does; the other tokens are not touched."""
    p = problem(5, 10, 3, 128, 64)
    clean, _, cw = call(p, routing=True)
    p["logits"][1, 4] = float("inf")
    p["logits"][3, [2, 6]] = float("inf")
    for renorm in (True, False):
        y, ids, w = call(p, renorm=renorm, routing=True)
        assert ids[1, 0] == 4 and ids[3, :2].tolist() == [2, 6]
        assert torch.isnan(w[1]).any() and torch.isnan(y[1]).all() and torch.isnan(y[3]).all()
        if renorm:
            for r in (0, 2, 4):
                assert torch.equal(y[r], clean[r]) and torch.equal(w[r], cw[r])


def test_weights_past_32_bits():
    """Experts whose codes lie more than 2^32 bytes behind the first one's."""
    e, k, n = 130, 4096, 16384
    p = problem(3, e, 2, k, n)
    p["logits"] -= 100
    p["logits"][0, [129, 3]] = 1.0
    p["logits"][1, [128, 127]] = 2.0
    p["logits"][2, [0, 129]] = torch.tensor([3.0, 1.0], device="cuda")
    check_all(p)


def test_masked_tokens():
    """A token without an expert has weights of zero and a row of zeros; a NaN stays in
    its token."""
    p = problem(6, 10, 3, 128, 64)
    clean, _, cw = call(p, routing=True)
    p["logits"][2] = float("-inf")
    p["logits"][4, 7] = float("nan")
    y, ids, w = call(p, routing=True)
    assert not w[2].any() and not y[2].any() and ids[2].tolist() == [0, 1, 2]
    assert ids[4, 0] == 7 and torch.isnan(w[4]).all() and torch.isnan(y[4]).all()
    for r in (0, 1, 3, 5):
        assert torch.equal(y[r], clean[r]) and torch.equal(w[r], cw[r])


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_bad_tokens_stay_in_their_rows(bad):
    p = problem(40, 6, 2, 192, 128)
    clean = call(p)
    p["x"][13, 77] = bad
    dirty = call(p)
    keep = torch.arange(40, device="cuda") != 13
    assert torch.equal(clean[keep], dirty[keep]) and not torch.isfinite(dirty[13]).any()


def test_zero_tokens():
    p = problem(0, 4, 2, 64, 64)
    y, ids, w = call(p, routing=True)
    assert y.shape == (0, 64) and ids.shape == w.shape == (0, 2)


def test_given_output_workspace_and_rows_behind():
    p = problem(21, 9, 3, 192, 128)
    want = call(p)
    buf = torch.full((24, 192), 7.0, dtype=BF, device="cuda")
    need = svdq.awq_moe_w4a16_workspace_bytes(21, 9, 3, 192, 128)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(call(p, Y=buf[:21], workspace=ws[:need]), want)
    assert bool((buf[21:] == 7).all()) and bool((ws[need:] == 255).all())


@pytest.mark.parametrize("t", [1, 37])
def test_stream_graph_and_same_bits(t):
    p = problem(t, 12, 4, 512, 192)
    want = call(p, routing=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = call(p, routing=True)
    torch.cuda.current_stream().wait_stream(st)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call(p, routing=True)
    for i in range(3):
        p["x"].copy_(torch.roll(p["x"], 1, 1))
        p["logits"].copy_(torch.roll(p["logits"], 5, 1))
        graph.replay()
        want = call(p, routing=True)
        torch.cuda.synchronize()
        for a, b in zip(want, held):
            assert torch.equal(a, b), i
