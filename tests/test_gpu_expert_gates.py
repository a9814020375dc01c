"""SwiGLU over the whole range of its gates: where the exponential overflows and underflows, where the slope
goes to 0 and to 1, and beyond.

A row holds its gate as binary digits, each a power of two in a block of 32 channels of its own: exact in
every form of rows, and so are the sums, of fewer than 24 bits.  The bounds then count the activation alone."""
import pytest
import torch

import expert_ref as R
from combine_get_dispatch_04_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMS = [R.FP4, R.E4M3, R.E5M2, "bf16"]
TOP, DIGITS, UP = 8, 14, 14             # digits 2^8 .. 2^-5 in blocks 0 .. 13, the up's value in block 14
I = 32
H = 32 * (DIGITS + 1)
TIMES = [1.0, 0.5, 1.5, 2.0]            # a column's gate is the row's times one of these
UPS = [1.0, -2.0, 0.5, 3.0, -1.5, 4.0, 6.0]


def gates():
    """Around the exponential's overflow (-88.7229) every 32nd, steps of 1/2 up to 300, steps of 1 up to 500."""
    near = torch.arange(-91 * 32, -86 * 32 + 1)
    wide = torch.arange(-600, 601) * 16
    far = torch.cat([torch.arange(-500, -300), torch.arange(301, 501)]) * 32
    few = torch.tensor([-2839, -2840, -2841, 2839, 2840, 0])       # -88.72 .. -88.78
    return torch.cat([near, wide, far, few]).double() / 32


def rows(v, u):
    """x [n, H] in float64: v's digits, and u."""
    x = torch.zeros((v.numel(), H), dtype=torch.float64)
    left = v.abs()
    for j in range(DIGITS):
        d = 2.0 ** (TOP - j)
        bit = left >= d
        left = left - d * bit
        x[:, 32 * j] = torch.where(bit, d * torch.sign(v), 0.0)
    assert not left.any()
    x[:, 32 * UP] = u
    return x


def weight():
    w = torch.zeros((1, 2 * I, H), dtype=torch.float64)
    for i in range(I):
        w[0, i, :32 * DIGITS:32] = TIMES[i % len(TIMES)]
        w[0, I + i, 32 * UP] = UPS[i % len(UPS)]
    return w


def coded(x, form):
    if form == "bf16":
        q, s = x.to(torch.bfloat16), None
    else:
        q, s = R.quantize(x, form)
    assert torch.equal(R.values(q, s), x)
    return q, s


def on(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def bounds(a, d=None):
    """R.gated and R.gated_grad of exact sums, with the sigmoid s within 2^-20 of its value and 0 below 2^-128 (so a
    product with it is off by that much times its other factors), each product in fp32 off by 2^-24 more."""
    g, u = a.chunk(2, -1)
    h, _ = R.gated(a, torch.zeros_like(a))
    off = 2.0 ** -19 * h.abs() + 2.0 ** -128 * (g * u).abs()
    if d is None:
        return h, off
    back, _ = R.gated_grad(a, torch.zeros_like(a), d)
    s = 1 / (1 + torch.exp(-g))
    low = torch.cat([(d * u).abs() * (1 + g.abs()), (d * g).abs()], -1)
    return h, off, back, low * (2.0 ** -19 * torch.cat([s, s], -1) + 2.0 ** -128)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("parts", [1, 3, 200])
def test_every_gate_forward_and_back(form, parts):
    """One expert has all rows, or three, or 200 (the tiles of many and of few rows)."""
    v = gates()
    n = v.numel()
    x = rows(v, torch.tensor([1.0, -0.5, 4.0])[torch.arange(n) % 3].double())
    d = torch.tensor([1.0, -2.0, 0.25, 1.5])[torch.arange(n * I).view(n, I) % 4].to(torch.bfloat16)
    w = weight()
    q, s = coded(x, form)
    wc, ws = coded(w, R.FP4)
    off = torch.linspace(0, n, parts + 1).round().to(torch.int32)
    dx_, ds_, dw_, dws_, doff, dd = on(q, s, wc.expand(parts, -1, -1).contiguous(), ws.expand(parts, -1, -1).contiguous(), off, d)
    y, _, h = api.expert_product(dx_, ds_, dw_, dws_, offsets=doff, activation="swiglu")
    dx = api.expert_product_backward(dd, h)
    a = x @ w[0].T
    want, tol, back, dback = bounds(a, d.double())
    R.assert_close(y, want, tol, "y")
    dback = dback + R.HALF * (back.abs() + dback)               # rounded to bf16 for its product
    R.assert_close(dx, back @ w[0], (R.steps(2 * I) * (1 + 2 * R.HALF)) * (back.abs() @ w[0].abs()) + dback @ w[0].abs(), "dx")


@pytest.mark.parametrize("quant", [R.FP4, R.E4M3, R.E5M2])
@pytest.mark.parametrize("form", FORMS)
def test_every_gate_quantised(form, quant):
    """Scales and codes lie between those of the bound's ends."""
    v = gates()
    x, w = rows(v, torch.full((v.numel(),), 2.0, dtype=torch.float64)), weight()
    q, s = coded(x, form)
    wc, ws = coded(w, R.FP4)
    off = torch.tensor([0, v.numel()], dtype=torch.int32)
    y, sc, _ = api.expert_product(*on(q, s, wc, ws), offsets=off.to(DEV), activation="swiglu", quant=quant)
    want, tol = bounds(x @ w[0].T)
    got, sc = R.values(y.cpu(), sc.cpu()), sc.cpu()
    spread = lambda t: R.scale_codes(t.amax(-1, keepdim=True).repeat_interleave(32, -1), quant)  # noqa: E731
    assert (sc >= spread((want.abs() - tol).clamp(min=0))).all() and (sc <= spread(want.abs() + tol)).all()
    ends = [R.values(R.pack(R.codes_of(t, sc, quant), quant), sc) for t in (want - tol, want + tol)]
    assert (got >= ends[0]).all() and (got <= ends[1]).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("size", [1e4, 2.0 ** 100, 1e30, 1.5 * 2.0 ** 127])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_gates_of_any_size(form, size, sign):
    """Up to the largest that every form of rows holds (beyond 2.36e38 times log2(e) is infinite)."""
    size = float(R.values(*R.quantize(torch.full((1, 32), size), R.FP4))[0, 0])
    x, w = torch.zeros((5, H), dtype=torch.float64), weight()
    w[0, :I] = torch.where(w[0, :I] != 0, 1.0, 0.0)
    x[:, 0], x[:, 32 * UP] = sign * size, 2.0 ** -20
    d = torch.full((5, I), 2.0 ** -20, dtype=torch.bfloat16)
    q, s = coded(x, form)
    wc, ws = coded(w, R.FP4)
    dx_, ds_, dw_, dws_, dd = on(q, s, wc, ws, d)
    y, _, h = api.expert_product(dx_, ds_, dw_, dws_, offsets=torch.tensor([0, 5], dtype=torch.int32, device=DEV),
                                 activation="swiglu")
    dx = api.expert_product_backward(dd, h)
    # the sigmoid is exactly 0 or 1: three products in fp32 are left
    want, _, back, _ = bounds(x @ w[0].T, d.double())
    tol, dback = 2.0 ** -22 * want.abs(), 2.0 ** -22 * back.abs()
    R.assert_close(y, want, tol, "y")
    dback = dback + R.HALF * (back.abs() + dback)
    R.assert_close(dx, back @ w[0], (R.steps(2 * I) * (1 + 2 * R.HALF)) * (back.abs() @ w[0].abs()) + dback @ w[0].abs(), "dx")


def test_gates_that_are_not_finite():
    """+inf stays, NaN stays; silu(inf) * inf = inf."""
    x = torch.ones((4, 32), dtype=torch.bfloat16)
    x[1, 3], x[2, 5] = float("inf"), float("nan")
    w, ws = R.quantize(torch.ones((1, 2 * I, 32)), R.FP4)
    dx_, dw_, dws_ = on(x, w, ws)
    y, _, _ = api.expert_product(dx_, None, dw_, dws_, offsets=torch.tensor([0, 4], dtype=torch.int32, device=DEV),
                                 activation="swiglu")
    y = y.float().cpu()
    assert (y[1] == float("inf")).all() and torch.isnan(y[2]).all() and torch.isfinite(y[[0, 3]]).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("by", [40.0, 300.0])
@pytest.mark.parametrize("counts", [[7, 0, 30], [90, 60], [400]], ids=str)
def test_random_rows_with_large_gates(form, by, counts):
    """Gates of about `by`: forward, the gradient, and quantised results, held as products of small gates are."""
    Hr, Ir = 352, 64
    g = torch.Generator().manual_seed(int(by) + len(counts))
    x = (torch.randn((sum(counts), Hr), generator=g) * by).to(torch.bfloat16)
    x, xs = (x, None) if form == "bf16" else R.quantize(x, form)
    w, ws = R.quantize((torch.randn((len(counts), 2 * Ir, Hr), generator=g) * Hr ** -0.5).to(torch.bfloat16), R.FP4)
    d = torch.randn((sum(counts), Ir), generator=g).to(torch.bfloat16)
    off = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32)
    dx_, ds_, dw_, dws_, doff, dd = on(x, xs, w, ws, off, d)
    y, _, h = api.expert_product(dx_, ds_, dw_, dws_, offsets=doff, activation="swiglu")
    dx = api.expert_product_backward(dd, h)
    X, W = R.values(x, xs), R.values(w, ws)
    assert float((X[:counts[0]] @ W[0, :Ir].T).min()) < -89
    coded_y = {q: api.expert_product(dx_, ds_, dw_, dws_, offsets=doff, activation="swiglu", quant=q)[:2]
               for q in (R.FP4, R.E4M3, R.E5M2)}
    for e in range(len(counts)):
        at = slice(int(off[e]), int(off[e + 1]))
        if at.start == at.stop:
            continue
        want, tol, back, dback = R.product(X[at], W[e], True, d[at].double(), None if form == "bf16" else form)
        R.assert_close(y[at], want, tol, "y")
        R.assert_close(dx[at], back, dback, "dx")
        for quant, (c, sc) in coded_y.items():
            sc = sc[at].cpu()
            got = R.values(c[at].cpu(), sc)
            ends = [R.values(R.pack(R.codes_of(t, sc, quant), quant), sc) for t in (want - tol, want + tol)]
            assert (got >= ends[0]).all() and (got <= ends[1]).all(), quant


@pytest.mark.parametrize("form", ["bf16", R.FP4])
@pytest.mark.parametrize("T,K,E,Hl,Il", [(5, 2, 4, 352, 96), (128, 8, 16, 352, 96)])
@pytest.mark.parametrize("by", [40.0, 300.0])
def test_few_tokens_with_large_gates(form, T, K, E, Hl, Il, by):
    g = torch.Generator().manual_seed(T)
    bf = lambda *s, by=1.0: (torch.randn(s, generator=g) * by).to(torch.bfloat16)  # noqa: E731
    x, up, down = bf(T, Hl, by=by), bf(E, 2 * Il, Hl, by=Hl ** -0.5), bf(E, Hl, Il, by=Il ** -0.5)
    us = ds = None
    if form == R.FP4:
        (up, us), (down, ds) = R.quantize(up, form), R.quantize(down, form)
    idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).to(torch.int32)
    w = torch.softmax(torch.randn((T, K), generator=g), 1)
    dx_, di, dw, du, dd, dus, dds = on(x, idx, w, up, down, us, ds)
    out, _ = api.low_latency_experts(dx_, di, dw, du, dd, up_scales=dus, down_scales=dds)
    R.assert_close(out, *R.layer(x.double(), idx.long(), w, R.values(up, us), R.values(down, ds)))
