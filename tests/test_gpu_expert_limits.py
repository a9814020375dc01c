"""The experts at the ends of what a call may hold: gradients whose factors overflow between them, weights that
are infinite, a token among any others."""
import pytest
import torch

import expert_ref as R
from combine_get_dispatch_04_amd import api
from test_gpu_expert_few import call, make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("g,u,d", [(-2.0 ** 30, 1.0, 2.0 ** 100), (-200.0, 2.0 ** 30, 2.0 ** 100),
                                   (-60.0, 2.0 ** 40, 2.0 ** 100), (-90.0, 2.0 ** 60, -2.0 ** 120),
                                   (-2.0 ** 100, 2.0 ** 100, 2.0 ** 100), (1.0, 1.0, 2.0 ** 100)])
def test_gradients_whose_factors_overflow_between_them(g, u, d):
    """d u and d g may be beyond fp32 where their products with the sigmoid are not."""
    I, H = 16, 64
    x = torch.zeros((3, H), dtype=torch.bfloat16)
    x[:, 0], x[:, 32] = g, u
    w = torch.zeros((1, 2 * I, H))
    w[0, :I, 0], w[0, I:, 32] = 1.0, 1.0
    wc, ws = R.quantize(w, R.FP4)
    dy = torch.full((3, I), d, dtype=torch.bfloat16)
    _, _, h = api.expert_product(x.to(DEV), None, wc.to(DEV), ws.to(DEV), activation="swiglu",
                                 offsets=torch.tensor([0, 3], dtype=torch.int32, device=DEV))
    dx = api.expert_product_backward(dy.to(DEV), h).cpu()
    back, _ = R.gated_grad(x.double() @ w[0].double().T, torch.zeros(3, 2 * I, dtype=torch.float64), dy.double())
    # the sigmoid within 2^-20 and 0 below 2^-128; d_g and d_u rounded to bf16; sums of equal terms
    s = 1 / (1 + torch.exp(torch.tensor(-g, dtype=torch.float64)))
    off = 2.0 ** -19 * back.abs() + (0 if s >= 2.0 ** -128 else back.abs())
    off = off + R.HALF * (back.abs() + off)
    R.assert_close(dx, back @ w[0].double(), R.steps(2 * I) * (back.abs() @ w[0].double()) + off @ w[0].double())


@pytest.mark.parametrize("T,K,E,H,I", [(6, 2, 3, 96, 64), (24, 2, 5, 352, 264), (128, 8, 8, 72, 264), (64, 16, 16, 136, 1032)])
@pytest.mark.parametrize("sign", [1, -1])
def test_an_infinite_weight_of_the_second_product(T, K, E, H, I, sign):
    """h goes into the product as two parts: what the second one makes of an infinite weight is not part of the result."""
    x, idx, w, up, us, down, ds = make(T, K, E, H, I, "bf16", seed=T)
    w = w + 0.1
    finite, _ = call(x, idx, w, up, us, down, ds)
    down[1, 5, 3] = sign * float("inf")
    out, _ = call(x, idx, w, up, us, down, ds)
    out, finite = out.cpu().float(), finite.cpu().float()
    named = (idx == 1).any(1)
    assert named.any()
    other = torch.ones(H, dtype=torch.bool)
    other[5] = False
    assert torch.equal(out[:, other], finite[:, other]) and torch.equal(out[~named], finite[~named])
    h = R.gated(x.double() @ up[1].double().T, torch.zeros(T, 2 * I, dtype=torch.float64))[0][:, 3]
    assert (h[named] != 0).all()
    assert torch.equal(out[named, 5], (sign * torch.sign(h[named])).float() * float("inf"))


# (narrow and wide forms of both kinds of weights)
@pytest.mark.parametrize("form,T,K,E,H,I", [("bf16", 16, 4, 9, 256, 160), (R.FP4, 16, 4, 9, 256, 160),
                                            ("bf16", 128, 8, 100, 200, 256), (R.FP4, 128, 8, 100, 1184, 160),
                                            ("bf16", 128, 1, 64, 96, 72), (R.FP4, 33, 2, 3, 4096, 96)])
def test_a_token_gives_the_same_bits_in_any_company(form, T, K, E, H, I):
    """One token's row, entries and weights stay; all others get other values, other experts, the same ones, or none."""
    x, idx, w, up, us, down, ds = make(T, K, E, H, I, form, seed=H)
    t = T // 2
    first = call(x, idx, w, up, us, down, ds)[0][t]
    g = torch.Generator().manual_seed(1)
    for kind in ("values", "experts", "the same experts", "none"):
        x2 = (torch.randn((T, H), generator=g) * 3).to(torch.bfloat16)
        w2, idx2 = torch.randn((T, K), generator=g), idx.clone()
        if kind == "experts":
            idx2 = torch.randint(-1, E, (T, K), generator=g, dtype=torch.int32)
        elif kind == "the same experts":
            idx2[:] = idx[t]
        elif kind == "none":
            idx2[:] = -1
        x2[t], w2[t], idx2[t] = x[t], w[t], idx[t]
        out = call(x2, idx2, w2, up, us, down, ds)[0]
        assert torch.equal(out[t], first), kind
        assert kind == "none" or not torch.equal(out[t - 1], first)
