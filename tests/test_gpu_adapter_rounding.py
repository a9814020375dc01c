"""The adapters round to bf16 once, at the result, whatever the call's size:
scale * w * (A x) and scale * w * (B^T d) go into their products in two parts
of bf16, which leave 2^-16 of a value, not 2^-8 (adapter_ref.py, carried)."""
import numpy as np
import pytest
import torch

import adapter_ref as R
from combine_get_dispatch_04_amd import api
from test_gpu_adapter import Case, close, say

pytestmark = pytest.mark.gpu
DEV = "cuda"
TWO_PARTS = R.H * R.H


@pytest.mark.parametrize("T,H,O,E,K,r,kind", [
    (96, 64, 72, 6, 2, 24, "mixed"),            # the form for a few tokens
    (129, 64, 72, 6, 1, 16, "mixed"),
    (300, 64, 72, 6, 1, 16, "mixed"),           # more values than one part was kept for before
    (600, 72, 40, 5, 2, 24, "mixed"),
    (700, 64, 64, 40, 1, 64, "requests"),
    (24600, 64, 64, 5, 1, 16, "requests"),      # tiles of 128 tokens
    (49200, 64, 64, 3, 1, 8, "one"),            # tiles of 256 tokens
])
def test_results_are_rounded_once(T, H, O, E, K, r, kind):
    say("rounded once", T, H, O, E, K, r, kind)
    c = Case(T + r, T, H, O, E, K, r, kind, weights=K > 1)
    out, h = api.adapter_project(*c.gpu(), scale=c.scale)
    grads = dict(zip(("dx", "da", "db", "dw"), api.adapter_project_backward(c.dy.to(DEV), h)))
    args = (c.x64, c.W64, c.a64, c.b64, c.idx, c.w, c.scale)
    want, bound, saved = R.forward(*args, carried=TWO_PARTS)
    wrong = []
    for name, got, g, b in [("out", out, want, bound)] + [
            (n, grads[n], *v) for n, v in R.backward(*args, c.dy64, saved, carried=TWO_PARTS).items()]:
        try:
            close(name, got, g, b)
        except AssertionError as e:
            wrong.append(str(e)[:80])
    assert not wrong, wrong
