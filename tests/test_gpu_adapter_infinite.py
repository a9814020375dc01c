"""An infinity or a NaN in an operand of the adapters: every result is infinite,
NaN or finite where the definition's is, with its sign, and the finite ones
have their values."""
import numpy as np
import pytest
import torch

import adapter_ref as R
from combine_get_dispatch_04_amd import api
from test_gpu_adapter import Case, say

pytestmark = pytest.mark.gpu
DEV = "cuda"


def same_kind(name, got, broken, clean, bound):
    """`broken`: the definition on the broken operands, `clean` on the whole
    ones, which is the value of whatever is still finite."""
    got = got.double().cpu().numpy()
    fine = np.isfinite(broken)
    assert np.array_equal(np.isnan(got), np.isnan(broken)), name
    assert np.array_equal(got[~fine & ~np.isnan(broken)], broken[~fine & ~np.isnan(broken)]), name
    err = np.abs(got[fine] - clean[fine])
    assert (err <= bound[fine]).all(), (name, err.max())
    return not fine.all()


@pytest.mark.parametrize("where", ["x", "dy", "a", "b"])
@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("T,K", [(8, 1), (150, 1), (150, 3), (300, 1)])
def test_an_infinity_has_the_definitions_sign(where, what, T, K):
    say("infinite", where, what, T, K)
    H, O, E, r = 136, 72, 6, 24
    clean, c = (Case(31, T, H, O, E, K, r, weights=False) for _ in range(2))
    named = (c.idx >= 0) & (c.idx < E)
    t = T // 2 + int(np.argmax(named[T // 2:].any(axis=1)))
    e = int(c.idx[t][named[t]][0])
    at = dict(x=(t, 9), dy=(t, 4), a=(e, 3, 5), b=(e, 7, 2))[where]
    getattr(c, where)[at] = what
    setattr(c, where + "64", getattr(c, where).double().numpy())
    out, h = api.adapter_project(*c.gpu(), scale=c.scale)
    grads = dict(zip(("dx", "da", "db", "dw"), api.adapter_project_backward(c.dy.to(DEV), h)))
    value, bound, saved = clean.ref()
    back = clean.ref_back(saved)
    with np.errstate(invalid="ignore", over="ignore"):
        value_b, _, saved_b = c.ref()
        back_b = c.ref_back(saved_b)
    reached = [same_kind("out", out, value_b, value, bound)]
    for name, (g, b) in back.items():
        reached.append(same_kind(name, grads[name], back_b[name][0], g, b))
    assert any(reached)
