"""The router and the balance loss over very many tokens: the sums' rounding
does not grow with the number of tokens."""
import pytest
import torch

import router_ref as R
from combine_get_dispatch_04_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,E", [(1 << 24, 3), (1 << 22, 66)])
def test_balance_sums_over_millions_of_tokens(T, E):
    """Equal logits and one expert chosen throughout: p = 1 / E, f = E there, so
    the loss is 1.  Equal addends round the same way each time, so that a long
    sum in fp32 drifts: 200 u and more here.  The bound is that of sums of 64
    values in fp32 and of those in fp64, of a row's own (spread 0), and of the
    loss's rounding."""
    print("[case] balance, long", T, E, flush=True)
    z = torch.zeros((T, E), dtype=torch.bfloat16, device=DEV)
    idx = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    bal = api.balance_loss(z, idx)
    assert int(bal.num_tokens_per_expert[0, 0]) == T
    assert abs(float(bal.loss) - 1.0) <= (80 + 66) * R.U


@pytest.mark.parametrize("E,K,score", [(8, 3, "softmax"), (66, 2, "sigmoid")])
def test_more_rows_than_waves(E, K, score):
    """Past 2^22 rows a wave takes several: the same bits as calls of fewer rows."""
    T, part = (1 << 22) + 12345, 1 << 21
    print("[case] rows", T, E, flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(T + E)
    z = torch.randn((T, E), generator=g, device=DEV).to(torch.bfloat16)
    d_w = torch.randn((T, K), generator=g, device=DEV)
    z[5::1001] = float("-inf")
    for renorm in (True, False):
        rt = api.route(z, K, score=score, renormalise=renorm)
        d = api.route_backward(d_w, rt)
        for lo in range(0, T, part):
            at = slice(lo, min(T, lo + part))
            few = api.route(z[at], K, score=score, renormalise=renorm)
            assert torch.equal(rt.topk_idx[at], few.topk_idx)
            assert torch.equal(rt.topk_weights[at], few.topk_weights)
            assert torch.equal(rt.num_invalid[at], few.num_invalid)
            assert torch.equal(d[at], api.route_backward(d_w[at], few))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", [((1 << 20) + 77, 5, 2), (300001, 96, 3), (40000, 1500, 4)])
def test_balance_loss_with_many_rows_per_wave(T, E, K, score):
    """Up to 256 rows per wave, three sequences, against 64 bits.  Logits within
    [-4, 4], so that `spread` is at most 8."""
    print("[case] balance, many rows", T, E, score, flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(T + E)
    z = torch.randn((T, E), generator=g, device=DEV).clamp(-4, 4)
    idx = torch.randint(0, E, (T, K), generator=g, device=DEV, dtype=torch.int32)
    cuts = [0, T // 7, T // 7, T - 1000]
    bal = api.balance_loss(z, idx, score=score, seq_offsets=torch.tensor(cuts, dtype=torch.int32, device=DEV))
    d = api.balance_loss_backward(torch.ones(1, device=DEV), bal)
    z64 = z.double()
    s = torch.exp(z64) if score == "softmax" else 1 / (1 + torch.exp(-z64))
    p = s / s.sum(dim=1, keepdim=True)
    del z64
    loss, want, size = 0.0, torch.zeros_like(p), torch.zeros_like(p)
    live = 2
    for i, (lo, hi) in enumerate(zip(cuts, cuts[1:])):
        counts = torch.bincount(idx[lo:hi].flatten().long(), minlength=E)
        assert torch.equal(bal.num_tokens_per_expert[i].long(), counts)
        if lo == hi:
            continue
        n = hi - lo
        f = E * counts.double() / (K * n)
        loss += float((f * p[lo:hi].sum(dim=0)).sum()) / n / live
        dot = (p[lo:hi] * f).sum(dim=1, keepdim=True)
        slope = 1 - s[lo:hi] if score == "sigmoid" else 1.0
        want[lo:hi] = p[lo:hi] * (f - dot) * slope / (n * live)
        size[lo:hi] = p[lo:hi] * (f + dot) * slope / (n * live)
    assert abs(float(bal.loss) - loss) <= (8 + 80 + 66) * R.U * loss
    assert ((d.double() - want).abs() <= (2 * 88 + 70) * R.U * size + R.TINY).all()
