"""The choice of experts over rows whose keys have no range to divide, or one that
fp32 cannot hold: every step of its histogram is then the same, or not a number."""
import numpy as np
import pytest
import torch

from test_gpu_router import DEV, check_route, say

pytestmark = pytest.mark.gpu


def rows(kind, T, E, rng):
    if kind == "equal":
        z = np.repeat(rng.standard_normal((T, 1)), E, axis=1)
    elif kind == "huge":                        # max - min overflows
        z = rng.choice([-3.0e38, -1.0, 0.0, 2.0, 3.0e38], (T, E))
    elif kind == "one_huge":
        z = rng.standard_normal((T, E))
        z[:, E // 2] = 3.3e38
        z[::2, 0] = -3.3e38
    else:                                       # "tiny": 1 / (max - min) overflows
        z = rng.integers(0, 5, (T, E)) * 2.0 ** -149 + 0.0
    z = z.astype(np.float32)
    z[rng.random((T, E)) < 0.1] = -np.inf
    return z


@pytest.mark.parametrize("kind", ["equal", "huge", "one_huge", "tiny"])
@pytest.mark.parametrize("T,E,K", [(70, 8, 3), (33, 64, 64), (40, 96, 8), (9, 512, 20), (5, 1500, 64)])
def test_rows_without_a_usable_range(kind, T, E, K):
    say("range", kind, T, E, K)
    z = rows(kind, T, E, np.random.default_rng(T + E))
    z_d = torch.from_numpy(z).to(DEV)
    z64 = z.astype(np.float64)
    for score in ("softmax", "sigmoid"):
        check_route(z_d, z64, K, score, None, True)
    bias = np.where(np.arange(E) % 3 == 0, np.float32(-3.0e38), np.float32(0.5)).astype(np.float32)
    check_route(z_d, z64, K, "sigmoid", bias, True)
    check_route(z_d, z64, K, "sigmoid", np.zeros(E, np.float32), False)
