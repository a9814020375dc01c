"""The experts' products against the definition in 64 bits."""
import pytest
import torch

import expert_ref as R
from combine_get_dispatch_04_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
FORMS = [R.FP4, R.E4M3, R.E5M2, "bf16"]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def bf(g, *shape, by=1.0):
    return (torch.randn(shape, generator=g) * by).to(torch.bfloat16)


def make(form, counts, H, O, seed=0, extra=0):
    """Rows of every expert one after the other (`extra` more behind them), a weight, on the CPU."""
    g = gen(seed)
    n = sum(counts) + extra
    x = bf(g, n, H)
    x, xs = (x, None) if form == "bf16" else R.quantize(x, form)
    w, ws = R.quantize(bf(g, len(counts), O, H, by=H ** -0.5), R.FP4)
    off = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)
    return x, xs, w, ws, off


def on(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def form_of(x):
    return {v: k for k, v in R.TYPES.items()}.get(x.dtype)


def want(x, xs, w, ws, off, act, d=None):
    """Per expert: (slice, product's results)."""
    X, W = R.values(x, xs), R.values(w, ws)
    for e in range(w.shape[0]):
        at = slice(int(off[e]), int(off[e + 1]))
        if at.stop > at.start:
            yield at, R.product(X[at], W[e], act, None if d is None else d[at].double(), form_of(x))


def check(form, counts, H, O, act, seed=0, back=True):
    x, xs, w, ws, off = make(form, counts, H, O, seed)
    n, width = x.shape[0], O // 2 if act else O
    d = bf(gen(seed + 100), n, width)
    dx_, ds_, dw_, dws_, doff, dd = on(x, xs, w, ws, off, d)
    y, none, h = api.expert_product(dx_, ds_, dw_, dws_, offsets=doff, activation=act)
    assert none is None and y.shape == (n, width)
    dx = api.expert_product_backward(dd, h) if back else None
    for at, r in want(x, xs, w, ws, off, act, d if back else None):
        R.assert_close(y[at], r[0], r[1], ("y", form, at))
        if back:
            R.assert_close(dx[at], r[2], r[3], ("dx", form, at))


# rows per expert: few (the narrow tile), some, many; none, one, tiles that end anywhere
SPREADS = [[1], [0, 3, 0, 17, 1, 0], [5, 33, 0, 64, 31], [50, 129, 1, 90], [160, 0, 400], [257, 255, 513]]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("counts", SPREADS, ids=str)
@pytest.mark.parametrize("H,O", [(32, 16), (96, 48), (256, 128), (608, 272), (1024, 544)])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_products_and_gradients(form, counts, H, O, act):
    check(form, counts, H, O, act, seed=len(counts) + H)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_long_rows(form, act):
    check(form, [3, 0, 40], 7168, 64, act)
    check(form, [200, 30], 2080, 4128, act, back=False)


@pytest.mark.parametrize("H", [32 * i for i in range(1, 18)])
def test_every_length_of_the_last_stage(H):
    for form in FORMS:
        check(form, [70, 2], H, 80, None, seed=H)
        check(form, [200], H, 32, "swiglu", seed=H)


@pytest.mark.parametrize("O", [8, 24, 40, 72, 120, 136, 248, 264])
def test_every_width_of_the_last_tile(O):
    for form in FORMS:
        check(form, [6, 40], 64, O, None, seed=O)
        check(form, [170], 64, O, None, seed=O)
        check(form, [170, 3], 64, 2 * O, "swiglu", seed=O)


# enough blocks for the large tiles: 256 x 256 (128 x 256 with 8-bit rows) and 128 x 256 (128 x 128 with bf16)
LARGE = [[200, 0, 300], [60, 0, 70, 50]]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("counts", LARGE, ids=str)
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("H", [96, 288])
def test_large_tiles(form, counts, act, H):
    check(form, counts, H, 24656, act, seed=H, back=False)


@pytest.mark.parametrize("counts", LARGE, ids=str)
@pytest.mark.parametrize("act,O", [(None, 40), (None, 200), ("swiglu", 80)])
def test_large_tiles_of_the_gradient(counts, act, O):
    for form in ("bf16", R.FP4):
        check(form, counts, 24640, O, act, seed=O)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_large_tiles_of_long_rows(form, act):
    check(form, [600, 0, 700, 1500], 2080, 4160, act, seed=3, back=act is None and form == "bf16")


@pytest.mark.parametrize("form", [R.FP4, R.E4M3, "bf16"])
@pytest.mark.parametrize("counts", LARGE, ids=str)
def test_large_tiles_write_their_rows_only(form, counts):
    """Rows that no expert has, and what lies behind a row's last column, in every tile's way of storing."""
    E, cap, H, O = len(counts), max(counts) + 5, 64, 24640
    g = gen(31)
    x = bf(g, E, cap, H)
    x, xs = (x, None) if form == "bf16" else R.quantize(x, form)
    w, ws = R.quantize(bf(g, E, O, H, by=0.1), R.FP4)
    cnt = torch.tensor(counts, dtype=torch.int32)
    dx_, ds_, dw_, dws_, dc = on(x, xs, w, ws, cnt)
    for act in (None, "swiglu"):
        y = torch.full((E, cap, O // 2 if act else O), 7.0, dtype=torch.bfloat16, device=DEV)
        api.expert_product(dx_, ds_, dw_, dws_, counts=dc, activation=act, out=y)
        q, s, _ = api.expert_product(dx_, ds_, dw_, dws_, counts=dc, activation=act, quant=R.E4M3)
        for e in range(E):
            n = counts[e]
            assert (y[e, n:] == 7).all() and not (y[e, :n] == 7).all(dim=1).any()
            if n:       # the codes are those of the same sums, of which y are the nearest bf16
                v = api.mx_dequantize(q[e, :n].contiguous(), s[e, :n].contiguous()).float()
                top = y[e, :n].float().abs().unflatten(-1, (-1, 32)).amax(-1, keepdim=True)
                # half a step of e4m3 (2^-4 of a value, or of the largest's 2^-14), saturation (512 to 448), bf16's own
                tol = y[e, :n].float().abs().unflatten(-1, (-1, 32)) * (2.0 ** -3 + 2.0 ** -7) + top * 2.0 ** -14
                assert ((v - y[e, :n].float()).abs().unflatten(-1, (-1, 32)) <= tol).all()


@pytest.mark.parametrize("quant", [R.FP4, R.E4M3, R.E5M2])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("counts", [[4, 0, 9], [60, 100], [300]], ids=str)
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_quantised_results(quant, form, counts, act):
    """The scale is that of a maximum within the sums' bound, and each code lies between those of the bound's ends."""
    H, O = 352, 320
    x, xs, w, ws, off = make(form, counts, H, O, 5)
    dx_, ds_, dw_, dws_, doff = on(x, xs, w, ws, off)
    y, s, _ = api.expert_product(dx_, ds_, dw_, dws_, offsets=doff, activation=act, quant=quant)
    width = O // 2 if act else O
    assert y.dtype == R.TYPES[quant] and s.shape == (x.shape[0], width // 32)
    got, s = R.values(y.cpu(), s.cpu()), s.cpu()
    for at, (v, off_) in want(x, xs, w, ws, off, act):
        a = v.abs().unflatten(-1, (-1, 32))
        o = off_.unflatten(-1, (-1, 32))
        low, high = (a - o).clamp(min=0).amax(-1), (a + o).amax(-1)
        spread = lambda t: R.scale_codes(t.repeat_interleave(32, -1), quant)  # noqa: E731
        assert (s[at] >= spread(low)).all() and (s[at] <= spread(high)).all()
        ends = [R.values(R.pack(R.codes_of(t, s[at], quant), quant), s[at]) for t in (v - off_, v + off_)]
        assert (got[at] >= ends[0]).all() and (got[at] <= ends[1]).all()


@pytest.mark.parametrize("quant", [R.FP4, R.E4M3, R.E5M2])
def test_quantised_results_of_exact_sums(quant):
    """Small whole numbers: the sums are exact in fp32, the codes those of the definition, bit for bit."""
    g = gen(2)
    n, H, O, E = 90, 128, 96, 2
    x = torch.randint(-3, 4, (n, H), generator=g).to(torch.bfloat16)
    w, ws = R.quantize(torch.randint(-2, 3, (E, O, H), generator=g).to(torch.bfloat16), R.FP4)
    off = torch.tensor([0, 41, 90], dtype=torch.int32)
    dx_, dw_, dws_, doff = on(x, w, ws, off)
    y, s, _ = api.expert_product(dx_, None, dw_, dws_, offsets=doff, quant=quant)
    W = R.values(w, ws)
    v = torch.cat([x[:41].double() @ W[0].T, x[41:].double() @ W[1].T])
    c, sc = R.quantize(v, quant)
    assert torch.equal(s.cpu(), sc) and torch.equal(y.cpu().view(torch.uint8), c.view(torch.uint8))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("counts,cap", [([0, 3, 9, 40], 9), ([64, 200, 0], 128), (None, 5), (None, 200), ([0, 0], 7), ([-4, 3], 4)])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_padded_rows(form, counts, cap, act):
    """Counts beyond the capacity are cut off; rows without a token are not written, nor read (they hold NaN)."""
    E = 3 if counts is None else len(counts)
    H, O = 160, 96
    g = gen(9)
    x = bf(g, E, cap, H)
    held = [cap if counts is None else max(0, min(c, cap)) for c in (counts or [0] * E)]
    x, xs = (x, None) if form == "bf16" else R.quantize(x, form)
    w, ws = R.quantize(bf(g, E, O, H, by=0.1), R.FP4)
    width = O // 2 if act else O
    d = bf(g, E, cap, width)
    for e in range(E):
        d[e, held[e]:] = float("nan")
        if form == "bf16":
            x[e, held[e]:] = float("nan")
        else:
            xs[e, held[e]:] = 255
    cnt = None if counts is None else torch.tensor(counts, dtype=torch.int32)
    dx_, ds_, dw_, dws_, dc, dd = on(x, xs, w, ws, cnt, d)
    y = torch.full((E, cap, width), 7.0, dtype=torch.bfloat16, device=DEV)
    dx = torch.full((E, cap, H), 7.0, dtype=torch.bfloat16, device=DEV)
    _, _, h = api.expert_product(dx_, ds_, dw_, dws_, counts=dc, activation=act, out=y)
    api.expert_product_backward(dd, h, out=dx)
    W = R.values(w, ws)
    for e in range(E):
        n = held[e]
        assert (y[e, n:] == 7).all() and (dx[e, n:] == 7).all()
        if n:
            X = R.values(x[e, :n], None if xs is None else xs[e, :n])
            r = R.product(X, W[e], act, d[e, :n].double(), form)
            R.assert_close(y[e, :n], r[0], r[1])
            R.assert_close(dx[e, :n], r[2], r[3])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("per", [8, 90, 300])
def test_rows_behind_the_last_expert_and_broken_offsets(form, per):
    """What no expert has is left as it was; offsets that reach beyond the buffer are cut off."""
    counts = [per, per + 3]
    x, xs, w, ws, off = make(form, counts, 64, 32, 3, extra=5)
    dx_, ds_, dw_, dws_, doff = on(x, xs, w, ws, off)
    y = torch.full((x.shape[0], 32), 7.0, dtype=torch.bfloat16, device=DEV)
    api.expert_product(dx_, ds_, dw_, dws_, offsets=doff, out=y)
    assert (y[-5:] == 7).all() and not (y[:-5] == 7).all(dim=1).any()
    n = x.shape[0]
    for bad in ([0, per, n + 1000], [-50, per, n], [0, 2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, per, per]):
        z = torch.full_like(y, 7.0)
        api.expert_product(dx_, ds_, dw_, dws_, offsets=torch.tensor(bad, dtype=torch.int32, device=DEV), out=z)
        cut = [min(max(v, 0), n) for v in bad]
        torch.cuda.synchronize()
        for e in range(2):
            a, b = cut[e], min(cut[e + 1], int(off[e + 1]))
            if b > a and int(off[e]) <= a:
                assert torch.equal(z[a:b], y[a:b])
    # decreasing: values without meaning, nothing outside the arrays
    api.expert_product(dx_, ds_, dw_, dws_, offsets=torch.tensor([n, 0, n], dtype=torch.int32, device=DEV), out=y)
    torch.cuda.synchronize()


@pytest.mark.parametrize("form", FORMS)
def test_offsets_that_overlap_ask_for_no_more_than_there_is(form):
    """Every second expert has all rows: more tiles than the rows make; nothing outside the arrays."""
    E, n, H, O = 300, 700, 64, 128
    g = gen(12)
    x = bf(g, n, H)
    x, xs = (x, None) if form == "bf16" else R.quantize(x, form)
    w, ws = R.quantize(bf(g, E, O, H), R.FP4)
    dx_, ds_, dw_, dws_ = on(x, xs, w, ws)
    off = torch.tensor([0, n] * (E // 2) + [0], dtype=torch.int32, device=DEV)
    guard = torch.full((n + 64, O), 7.0, dtype=torch.bfloat16, device=DEV)
    api.expert_product(dx_, ds_, dw_, dws_, offsets=off, out=guard[:n])
    torch.cuda.synchronize()
    assert (guard[n:] == 7).all() and torch.isfinite(guard.float()).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("counts", [[3, 4], [80, 70], [300, 200]], ids=str)
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_what_is_not_finite_stays_in_its_row(form, counts, act):
    H, O = 320, 64
    x, xs, w, ws, off = make(form, counts, H, O, 4)
    d = bf(gen(1), x.shape[0], O // 2 if act else O)
    dx_, ds_, dw_, dws_, doff, dd = on(x, xs, w, ws, off, d)

    def run():
        y, _, h = api.expert_product(dx_, ds_, dw_, dws_, offsets=doff, activation=act)
        return y, api.expert_product_backward(dd, h)
    y, g = run()
    row = counts[0] // 2
    if form == "bf16":
        dx_[row, 33] = float("nan")
    else:
        ds_[row, 1] = 255
    dd[row + 1, 3] = float("inf")
    y2, g2 = run()
    keep = torch.ones(x.shape[0], dtype=torch.bool)
    keep[row] = False
    assert torch.equal(y2.cpu()[keep], y.cpu()[keep]) and torch.isnan(y2[row].float()).all()
    keep[row + 1] = False
    assert torch.equal(g2.cpu()[keep], g.cpu()[keep])
    assert not torch.isfinite(g2[row + 1].float()).any()


@pytest.mark.parametrize("form", FORMS)
def test_the_same_calls_give_the_same_bits_and_no_rows_give_nothing(form):
    x, xs, w, ws, off = make(form, [100, 0, 77], 512, 256, 6)
    dx_, ds_, dw_, dws_, doff = on(x, xs, w, ws, off)
    first = api.expert_product(dx_, ds_, dw_, dws_, offsets=doff, activation="swiglu")[0]
    for _ in range(3):
        assert torch.equal(first, api.expert_product(dx_, ds_, dw_, dws_, offsets=doff, activation="swiglu")[0])
    none = None if ds_ is None else ds_[:0]
    y, _, h = api.expert_product(dx_[:0], none, dw_, dws_, offsets=torch.zeros(4, dtype=torch.int32, device=DEV))
    assert y.shape == (0, 256) and api.expert_product_backward(y, h).shape == (0, 512)


def test_gradient_against_differences():
    """SwiGLU's gradient of the definition that the tests above hold the kernel to, against differences of it."""
    g = gen(8)
    x, w, d = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((3, 32), (16, 32), (3, 8)))
    f = lambda v: (R.product(v, w, True)[0] * d).sum()  # noqa: E731
    dx = R.product(x, w, True, d)[2]
    for i in range(3):
        for j in range(0, 32, 5):
            e = torch.zeros_like(x)
            e[i, j] = 1e-5
            assert abs(float((f(x + e) - f(x - e)) / 2e-5 - dx[i, j])) < 1e-7 * float(1 + dx.abs().max())
