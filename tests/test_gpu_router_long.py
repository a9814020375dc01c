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
