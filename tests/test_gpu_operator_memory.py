"""What the results of the router and the adapters keep alive: what their
backward reads, and no scratch memory."""
import pytest
import torch

from combine_get_dispatch_04_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda"
BLOCK = 512                                     # torch hands out memory in multiples of this


def held(make):
    """Bytes that stay allocated while only make()'s result is alive."""
    make()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    kept = make()
    return torch.cuda.memory_allocated() - before, kept


@pytest.mark.parametrize("T", [1, 100, 128])
def test_a_small_adapter_call_keeps_no_workspace(T):
    H, O, E, r = 512, 1024, 4, 16
    bf = lambda *s: torch.randn(s, device=DEV).to(torch.bfloat16)  # noqa: E731
    x, W, a, b, dy = bf(T, H), bf(O, H), bf(E, r, H), bf(E, O, r), bf(T, O)
    idx = torch.arange(T, dtype=torch.int32, device=DEV).view(T, 1) % E
    n, h = held(lambda: api.adapter_project(x, W, a, b, idx)[1])
    assert n <= 2 * BLOCK                       # the count of bad entries, and at most a stub of a state
    first = api.adapter_project_backward(dy, h)
    second = api.adapter_project_backward(dy, h)
    for p, q in zip(first, second):
        assert torch.equal(p, q)


def test_the_balance_loss_keeps_no_workspace():
    T, E, K, S = 5000, 256, 8, 3
    z = torch.randn((T, E), device=DEV)
    idx = torch.randint(0, E, (T, K), device=DEV, dtype=torch.int32)
    seq = torch.tensor([0, 100, 3000, T], dtype=torch.int32, device=DEV)
    n, bal = held(lambda: api.balance_loss(z, idx, seq_offsets=seq))
    # counts, the gradient's table, loss and num_invalid
    assert n <= 4 * S * E + 4 * (S * E + 1) + 4 * BLOCK
    d = api.balance_loss_backward(torch.ones(1, device=DEV), bal)
    assert torch.equal(d, api.balance_loss_backward(torch.ones(1, device=DEV), bal))
