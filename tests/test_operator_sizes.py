"""The adapters' workspaces hold what their kernels write, and no multiple of it."""
import pytest

import combine_get_dispatch_04_amd._native as N


def depth(D):
    """Parts that a sum over D channels is split into at most: one below 512, else of 256."""
    return 1 if D < 512 else D // 256


@pytest.mark.parametrize("T,H,O,E,K,r", [(129, 256, 256, 64, 64, 128), (4001, 512, 512, 30, 4, 64),
                                         (1001, 4096, 1032, 32, 1, 24), (300, 504, 8192, 9, 2, 16),
                                         (40000, 128, 7168, 64, 8, 16)])
def test_workspaces_are_sized_by_the_splits_there_can_be(T, H, O, E, K, r):
    entries = 4 * T * K * r
    slots = max(4, min(64, 512 // ((T + 127) // 128)), min(64, 512 // ((T + 63) // 64)))
    fwd = N.ep_adapter_workspace_bytes(T, H, O, E, K, r, 0)
    assert entries <= fwd <= min(slots, depth(H)) * entries + 1024
    # backward: the splits' sums (or those of the two gradients, up to 16 each), V in fp32 and as a dense matrix
    dense = N.ep_adapter_state_bytes(T, H, O, E, K, r) - entries
    grads = sum(16 * 4 * E * r * n for n in (H, O))
    bwd = N.ep_adapter_workspace_bytes(T, H, O, E, K, r, 1)
    assert bwd <= max(min(slots, max(depth(H), depth(O))) * entries, grads) + entries + dense + 2048
