"""The router, the balance loss and their gradients on the GPU against the
64-bit definitions (router_ref.py, which derives the bounds): choices and
counts equal, weights, losses and gradients within the rounding of fp32 (and
of bf16 where that is the logits' type)."""
import numpy as np
import pytest
import torch

import router_ref as R
from combine_get_dispatch_04_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
LOWEST = float(np.finfo(np.float32).min)


def say(*a):
    print("[case]", *a, flush=True)


def make(seed, T, E, dtype, kind="plain"):
    """Logits on the GPU and the same values in 64 bits."""
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((T, E)) + 0.5 * rng.standard_normal(E)
    if kind == "masked":
        z[rng.random((T, E)) < 0.5] = -np.inf
        z[::3] = -np.inf
        z[1::7, 1:] = -np.inf
    elif kind == "lowest":
        z[rng.random((T, E)) < 0.5] = LOWEST
        z[::4] = LOWEST
    elif kind == "bad":
        z[rng.random((T, E)) < 0.1] = np.nan
        z[rng.random((T, E)) < 0.1] = np.inf
        z[0] = np.nan
    elif kind == "ties":
        z = np.round(z)
        z[::2] = -z[::2]                      # -0 and +0 side by side
    elif kind == "wide":
        z = z * 40.0
    elif kind == "deep":
        z = z * 3.0 - 200.0                   # sigmoid underflows in fp32
    elif kind == "high":
        z = np.round(z * 8.0) + 60.0          # sigmoid is 1 in fp32 and in fp64
    t = torch.from_numpy(z.astype(np.float32)).to(dtype)
    return t.to(DEV), t.double().numpy()


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (67, 64, 6), (33, 65, 3), (50, 129, 8), (128, 256, 8),
          (41, 384, 16), (20, 513, 64), (9, 1000, 10), (5, 2049, 33), (4, 4096, 64)]
KINDS = ["plain", "masked", "lowest", "bad", "ties", "wide", "deep", "high"]


def check_route(z_d, z, K, score, bias, renorm, scale=1.5):
    b_d = None if bias is None else torch.from_numpy(bias).to(DEV)
    rt = api.route(z_d, K, score=score, bias=b_d, renormalise=renorm, scale=scale)
    idx, w, bad = R.route(z, K, score, bias, renorm, scale)
    assert np.array_equal(rt.topk_idx.cpu().numpy(), idx)
    assert np.array_equal(rt.num_invalid.cpu().numpy(), bad)
    got = rt.topk_weights.cpu().numpy().astype(np.float64)
    err = np.abs(got - w)
    assert (err <= R.weight_bound(z) * np.abs(w) + R.TINY).all(), err.max()
    return rt, idx


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_route_and_its_gradient(T, E, K, dtype, score, renorm):
    say("route", T, E, K, dtype, score, renorm)
    z_d, z = make(T * 1000 + E, T, E, dtype)
    rt, idx = check_route(z_d, z, K, score, None, renorm)
    d_w = np.random.default_rng(7).standard_normal((T, K)).astype(np.float32)
    check_grad(z, rt, idx, d_w)


def check_grad(z, rt, idx, d_w):
    d = api.route_backward(torch.from_numpy(d_w).to(DEV), rt)
    assert d.dtype == rt.logits.dtype
    want, size = R.route_grad(z, idx, d_w, rt.score, rt.renormalise, rt.scale)
    err = np.abs(d.double().cpu().numpy() - want)
    bound = R.grad_bound(z) * size + R.TINY
    if d.dtype == torch.bfloat16:
        bound = bound + R.BF16 * (np.abs(want) + bound)
    assert (err <= bound).all(), (err - bound).max()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_route_masks_and_ranges(kind, dtype, score, renorm):
    T, E, K = 37, 96, 8
    say("route", kind, dtype, score, renorm)
    z_d, z = make(11, T, E, dtype, kind)
    rt, idx = check_route(z_d, z, K, score, None, renorm)
    d_w = np.random.default_rng(8).standard_normal((T, K)).astype(np.float32)
    check_grad(z, rt, idx, d_w)


@pytest.mark.parametrize("kind", ["plain", "masked", "bad", "ties", "deep", "high"])
@pytest.mark.parametrize("T,E,K", [(300, 256, 8), (25, 384, 16), (7, 1000, 64), (10, 9, 9)])
@pytest.mark.parametrize("steps", [None, 8])
def test_route_with_selection_bias(kind, T, E, K, steps):
    """The order of sigmoid + bias is that of 64 bits, ties and near-ties among
    them: `steps` draws the biases from few values, so that equal logits tie."""
    say("bias", kind, T, E, K, steps)
    z_d, z = make(5, T, E, torch.float32, kind)
    rng = np.random.default_rng(6)
    bias = 0.1 * rng.standard_normal(E)
    if steps:
        bias = np.round(bias * steps) / steps
    bias = bias.astype(np.float32)
    check_route(z_d, z, K, "sigmoid", bias, True)
    check_route(z_d, z, K, "sigmoid", bias, False)


def test_route_order_next_to_a_border():
    """Keys that differ by less than fp32 resolves: 64 bits decide."""
    rng = np.random.default_rng(3)
    T, E, K = 200, 128, 8
    z = rng.standard_normal((T, E)).astype(np.float32)
    base = z[:, :1].repeat(E, 1)
    z = np.nextafter(base, base + rng.choice([-1.0, 1.0], (T, E)).astype(np.float32))
    for _ in range(3):
        z = np.where(rng.random((T, E)) < 0.5, np.nextafter(z, np.float32(10)), z)
    bias = np.zeros(E, np.float32)
    check_route(torch.from_numpy(z).to(DEV), z.astype(np.float64), K, "sigmoid", bias, True)


def test_route_bias_that_is_not_finite_masks_its_expert():
    z_d, z = make(4, 16, 32, torch.float32)
    bias = np.zeros(32, np.float32)
    bias[3], bias[7], bias[9] = -np.inf, np.nan, np.inf
    rt, idx = check_route(z_d, z, 29, "sigmoid", bias, True)
    assert not np.isin(idx, [3, 7, 9]).any()


def test_route_no_tokens():
    rt = api.route(torch.empty((0, 16), device=DEV), 4)
    assert rt.topk_idx.shape == (0, 4) and rt.topk_weights.shape == (0, 4)
    assert api.route_backward(torch.empty((0, 4), device=DEV), rt).shape == (0, 16)


def test_route_matches_the_drawn_router():
    """workloads.router_topk draws the same choice and weights."""
    from combine_get_dispatch_04_amd import workloads as W
    rng = np.random.default_rng(1)
    z = rng.standard_normal((64, 256)).astype(np.float32)
    idx, w = W.router_topk(z, None, 8)
    rt = api.route(torch.from_numpy(z).to(DEV), 8)
    assert np.array_equal(rt.topk_idx.cpu().numpy(), idx)
    assert np.abs(rt.topk_weights.cpu().numpy() - w).max() <= R.weight_bound(z)


# ------------------------------------------------------------ the balance loss
def offsets(kind, T, S, rng):
    if kind == "one":
        return None
    cuts = np.sort(rng.integers(0, T + 1, S + 1))
    if kind == "whole":
        cuts[0], cuts[-1] = 0, T
    elif kind == "inside":                     # tokens before and behind
        cuts[0], cuts[-1] = min(2, T), max(min(2, T), T - 3)
        cuts = np.maximum.accumulate(np.clip(cuts, cuts[0], cuts[-1]))
    elif kind == "empty":
        cuts[:] = T // 2
    elif kind == "single":                     # every token its own
        cuts = np.arange(T + 1)
    return cuts.astype(np.int32)


def check_balance(z_d, z, idx, score, coef=0.5, seq=None, d_loss=0.7):
    s_d = None if seq is None else torch.from_numpy(seq).to(DEV)
    bal = api.balance_loss(z_d, torch.from_numpy(idx).to(DEV), score=score, coef=coef, seq_offsets=s_d)
    loss, counts, bad, grad = R.balance(z, idx, score, coef, seq)
    assert np.array_equal(bal.num_tokens_per_expert.cpu().numpy(), counts)
    assert np.array_equal(bal.num_invalid.cpu().numpy(), bad)
    # sums of at most 64 rows per wave in fp32 (T <= 2^14 here), the rest in fp64
    assert abs(float(bal.loss) - loss) <= (R.weight_bound(z) + 66 * R.U) * abs(loss) + R.TINY
    d = api.balance_loss_backward(torch.full((1,), d_loss, device=DEV), bal)
    want, size = grad(float(np.float32(d_loss)))
    err = np.abs(d.double().cpu().numpy() - want)
    bound = R.grad_bound(z) * size + R.TINY
    if d.dtype == torch.bfloat16:
        bound = bound + R.BF16 * (np.abs(want) + bound)
    assert (err <= bound).all(), (err - bound).max()
    return bal


def choice(rng, T, E, K, drop=0.1, invalid=0.02):
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :K].astype(np.int32)
    if K > E:
        idx = rng.integers(0, E, (T, K)).astype(np.int32)
    u = rng.random(idx.shape)
    idx[u < drop] = -1
    idx[(u >= drop) & (u < drop + invalid)] = rng.choice([E, -2, 1 << 30])
    return np.ascontiguousarray(idx)


@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (17, 8, 2), (128, 8, 2), (300, 65, 6), (130, 256, 8),
                                   (70, 384, 16), (40, 600, 5), (33, 1025, 4), (18, 4096, 9), (5000, 24, 3)])
@pytest.mark.parametrize("kind,S", [("one", 1), ("whole", 3), ("whole", 40), ("inside", 4), ("empty", 2),
                                    ("single", 0)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_loss_and_its_gradient(T, E, K, kind, S, score):
    if kind == "single" and T * E > 20000:
        pytest.skip("a table of every token's counts")
    dtype = torch.bfloat16 if (T + E) % 2 else torch.float32
    say("balance", T, E, K, kind, S, score, dtype)
    rng = np.random.default_rng(T + E + S)
    z_d, z = make(T + 3 * E, T, E, dtype)
    check_balance(z_d, z, choice(rng, T, E, K), score, seq=offsets(kind, T, S, rng))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_masks_and_ranges(kind, score):
    say("balance", kind, score)
    if kind == "deep" and score == "sigmoid":
        pass                                   # the stand-in for underflowing scores
    rng = np.random.default_rng(2)
    T, E, K = 61, 70, 4
    z_d, z = make(12, T, E, torch.float32, kind)
    check_balance(z_d, z, choice(rng, T, E, K), score, seq=np.array([0, 1, 30, 61], np.int32))


def test_balance_all_masked_and_no_tokens():
    z = torch.full((9, 16), float("-inf"), device=DEV)
    idx = torch.zeros((9, 2), dtype=torch.int32, device=DEV)
    bal = api.balance_loss(z, idx)
    assert float(bal.loss) == 0.0 and int(bal.num_tokens_per_expert[0, 0]) == 18
    d = api.balance_loss_backward(torch.ones(1, device=DEV), bal)
    assert torch.equal(d, torch.zeros_like(d))
    bal = api.balance_loss(z[:0], idx[:0], seq_offsets=torch.zeros(4, dtype=torch.int32, device=DEV))
    assert float(bal.loss) == 0.0 and not bal.num_tokens_per_expert.any()
    assert api.balance_loss_backward(torch.ones(1, device=DEV), bal).shape == (0, 16)


def test_balance_offsets_that_decrease_stay_inside():
    """Bad offsets: unspecified values, every access inside the arrays."""
    z_d, _ = make(1, 100, 32, torch.float32)
    idx = torch.zeros((100, 2), dtype=torch.int32, device=DEV)
    seq = torch.tensor([50, -5, 1 << 30, 7, 100], dtype=torch.int32, device=DEV)
    bal = api.balance_loss(z_d, idx, seq_offsets=seq)
    api.balance_loss_backward(torch.ones(1, device=DEV), bal)
    torch.cuda.synchronize()


def test_balance_gradient_against_differences():
    """The kernel's gradient against central differences of the 64-bit loss
    (error of a difference with step h: h^2 / 6 of the third derivative, below
    1e-8 here, and 2^-52 / h = 2e-12 of rounding)."""
    T, E, K = 6, 12, 3
    rng = np.random.default_rng(9)
    for score in ("softmax", "sigmoid"):
        z_d, z = make(21, T, E, torch.float32)
        idx = choice(rng, T, E, K, 0.0, 0.0)
        bal = api.balance_loss(z_d, torch.from_numpy(idx).to(DEV), score=score)
        d = api.balance_loss_backward(torch.ones(1, device=DEV), bal).double().cpu().numpy()
        h = 1e-4
        for t in range(T):
            for e in range(E):
                hi, lo = z.copy(), z.copy()
                hi[t, e] += h
                lo[t, e] -= h
                num = (R.balance(hi, idx, score)[0] - R.balance(lo, idx, score)[0]) / (2 * h)
                assert abs(num - d[t, e]) <= 1e-8 + 1e-5 * abs(num), (score, t, e)


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                          ("sigmoid", False)])
def test_route_gradient_against_differences(score, renorm):
    T, E, K = 5, 10, 3
    z_d, z = make(22, T, E, torch.float32)
    rt = api.route(z_d, K, score=score, renormalise=renorm, scale=1.5)
    idx = rt.topk_idx.cpu().numpy()
    g = np.random.default_rng(1).standard_normal((T, K)).astype(np.float32)
    d = api.route_backward(torch.from_numpy(g).to(DEV), rt).double().cpu().numpy()

    def value(z):
        got, w, _ = R.route(z, K, score, None, renorm, 1.5)
        assert np.array_equal(got, idx)
        return float((w * g).sum())

    h = 1e-5
    for t in range(T):
        for e in range(E):
            hi, lo = z.copy(), z.copy()
            hi[t, e] += h
            lo[t, e] -= h
            num = (value(hi) - value(lo)) / (2 * h)
            assert abs(num - d[t, e]) <= 1e-8 + 1e-5 * abs(num), (t, e)


# ------------------------------------------------------------------- together
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_one_pass_for_both_gradients(dtype, score, renorm):
    T, E, K = 203, 256, 8
    z_d, z = make(30, T, E, dtype)
    seq = np.array([0, 50, 50, 190], np.int32)
    rt, idx = check_route(z_d, z, K, score, None, renorm)
    bal = check_balance(z_d, z, idx, score, seq=seq)
    g = np.random.default_rng(1).standard_normal((T, K)).astype(np.float32)
    d_loss = torch.full((1,), 3.0, device=DEV)
    d = api.route_backward(torch.from_numpy(g).to(DEV), rt, balance=bal, d_loss=d_loss)
    a, sa = R.route_grad(z, idx, g, score, renorm, 1.5)
    b, sb = R.balance(z, idx, score, 0.5, seq)[3](3.0)
    want, bound = a + b, R.grad_bound(z) * (sa + sb) + R.U * (sa + sb) + R.TINY
    if dtype == torch.bfloat16:
        bound = bound + R.BF16 * (np.abs(want) + bound)
    assert (np.abs(d.double().cpu().numpy() - want) <= bound).all()


def test_router_layout_dispatch_combine():
    """The layer's path: choice, counts, dispatch, combine with the weights."""
    T, E, K, H = 150, 32, 4, 256
    z_d, _ = make(40, T, E, torch.float32)
    x = torch.randn((T, H), device=DEV).to(torch.bfloat16)
    rt = api.route(z_d, K)
    bal = api.balance_loss(z_d, rt.topk_idx)
    L = api.get_dispatch_layout(rt.topk_idx, E)
    assert torch.equal(bal.num_tokens_per_expert[0], L.num_tokens_per_expert)
    recv, _, h = api.dispatch(x, L)
    out = api.combine(recv, h, rt.topk_weights)
    # identity experts and weights that sum to 1: K products and sums in fp32, one rounding to bf16
    x64 = x.double()
    assert ((out.double() - x64).abs() <= (R.BF16 + 200 * R.U) * x64.abs()).all()


def test_same_bits_every_time_and_on_another_stream():
    T, E, K = 3000, 200, 8
    z_d, _ = make(50, T, E, torch.float32)
    g = torch.randn((T, K), device=DEV)
    one = torch.ones(1, device=DEV)

    def all_of_it():
        rt = api.route(z_d, K, score="sigmoid")
        bal = api.balance_loss(z_d, rt.topk_idx, score="sigmoid")
        d = api.route_backward(g, rt, balance=bal, d_loss=one)
        return rt.topk_idx, rt.topk_weights, bal.loss, bal.num_tokens_per_expert, d

    first = all_of_it()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = all_of_it()
    torch.cuda.current_stream().wait_stream(side)
    third = all_of_it()
    for a, b, c in zip(first, again, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_captured_step_replays():
    """Route, loss and gradient captured once, replayed on new inputs with eager
    work between the replays: the eager results every time."""
    T, E, K = 500, 64, 6
    z_in = torch.empty((T, E), device=DEV)
    g = torch.randn((T, K), device=DEV)
    one = torch.ones(1, device=DEV)

    def step(z):
        rt = api.route(z, K)
        bal = api.balance_loss(z, rt.topk_idx)
        return rt.topk_idx, rt.topk_weights, bal.loss, bal.num_tokens_per_expert, api.route_backward(
            g, rt, balance=bal, d_loss=one)

    z_in.copy_(make(60, T, E, torch.float32)[0])
    step(z_in)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(z_in)
    for seed in range(61, 65):
        z = make(seed, T, E, torch.float32)[0]
        z_in.copy_(z)
        graph.replay()
        want = step(z)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_refusals():
    z = torch.zeros((4, 8), device=DEV)
    with pytest.raises(ValueError):
        api.route(z, 9)
    with pytest.raises(ValueError):
        api.route(z, 2, bias=torch.zeros(8, device=DEV))
    with pytest.raises(ValueError):
        api.route(z, 2, score="sigmoid", bias=torch.zeros(7, device=DEV))
    with pytest.raises(ValueError):
        api.route(z.half(), 2)
    with pytest.raises(ValueError):
        api.route(z.t(), 2)
    with pytest.raises(ValueError):
        api.route(torch.zeros((4, 100), device=DEV), 65)          # more choices than lanes
    rt = api.route(z, 2)
    with pytest.raises(ValueError):
        api.route_backward(torch.zeros((4, 3), device=DEV), rt)
    with pytest.raises(ValueError):
        api.balance_loss(z, torch.zeros((3, 2), dtype=torch.int32, device=DEV))
    bal = api.balance_loss(z, rt.topk_idx)
    with pytest.raises(ValueError):
        api.route_backward(torch.zeros((4, 2), device=DEV), rt, balance=bal)
    with pytest.raises(ValueError):
        api.route_backward(torch.zeros((4, 2), device=DEV), rt, d_loss=torch.ones(1, device=DEV))
    other = api.balance_loss(z, rt.topk_idx, score="sigmoid")
    with pytest.raises(ValueError):
        api.route_backward(torch.zeros((4, 2), device=DEV), rt, balance=other,
                           d_loss=torch.ones(1, device=DEV))
