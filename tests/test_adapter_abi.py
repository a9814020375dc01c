"""Argument errors of the adapters' entry points, on the CPU (fake addresses:
every call is refused by the host's checks), the sizes, and the reference's
gradients against differences."""
import numpy as np
import pytest
import torch

import adapter_ref as R
import combine_get_dispatch_04_amd._native as N
from combine_get_dispatch_04_amd import api

A, WS = 0x10000, 0x100000
BAD, UNS, WSP = N.EP_ERR_INVALID_ARG, N.EP_ERR_UNSUPPORTED, N.EP_ERR_WORKSPACE


def _fwd(**kw):
    a = dict(x=A, T=16, H=64, weight=A, O=64, a=A, b=A, E=4, r=16, topk_idx=A, topk_weights=A, K=2, scale=1.0,
             out=A, num_invalid=A, state=WS, state_bytes=1 << 24, ws=WS, ws_bytes=1 << 24, stream=None)
    a.update(kw)
    return N.ep_adapter_project(**a, check=False)


def _bwd(**kw):
    a = dict(d_out=A, x=A, T=16, H=64, weight=A, O=64, a=A, b=A, E=4, r=16, topk_idx=A, topk_weights=A, K=2,
             scale=1.0, state=WS, state_bytes=1 << 24, dx=A, da=A, db=A, d_weights=A, ws=WS, ws_bytes=1 << 24,
             stream=None)
    a.update(kw)
    return N.ep_adapter_project_backward(**a, check=False)


COMMON = [(dict(T=-1), BAD), (dict(K=0), BAD), (dict(E=0), BAD), (dict(H=60), BAD), (dict(H=0), BAD),
          (dict(O=60), BAD), (dict(r=12), BAD), (dict(r=0), BAD), (dict(T=1 << 30, K=2), BAD),
          (dict(r=136), UNS), (dict(E=4097), UNS), (dict(K=65), UNS), (dict(H=(1 << 20) + 8), UNS),
          (dict(O=(1 << 20) + 8), UNS), (dict(T=1 << 29, K=1), UNS), (dict(x=None), BAD), (dict(x=A + 8), BAD),
          (dict(weight=None), BAD), (dict(weight=A + 8), BAD), (dict(a=None), BAD), (dict(a=A + 8), BAD),
          (dict(b=None), BAD), (dict(b=A + 8), BAD), (dict(topk_idx=None), BAD), (dict(topk_idx=A + 2), BAD),
          (dict(topk_weights=A + 2), BAD), (dict(state=None), WSP), (dict(state=WS + 128), BAD),
          (dict(state_bytes=64), WSP), (dict(ws=None), WSP), (dict(ws=WS + 128), WSP), (dict(ws_bytes=64), WSP)]


@pytest.mark.parametrize("kw,status", COMMON + [(dict(out=None), BAD), (dict(out=A + 8), BAD),
                                                (dict(num_invalid=None), BAD), (dict(num_invalid=A + 2), BAD)])
def test_forward_refuses(kw, status):
    assert _fwd(**kw) == status


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(d_out=None), BAD), (dict(d_out=A + 8), BAD), (dict(dx=A + 8), BAD), (dict(da=A + 8), BAD),
    (dict(db=A + 8), BAD), (dict(d_weights=A + 2), BAD), (dict(dx=None, da=None, db=None, d_weights=None), BAD)])
def test_backward_refuses(kw, status):
    assert _bwd(**kw) == status


def test_sizes():
    s, w = N.ep_adapter_state_bytes, N.ep_adapter_workspace_bytes
    # the sums of every entry in fp32
    assert s(300, 64, 64, 4, 2, 16) >= 300 * 2 * 16 * 4
    assert w(100, 64, 64, 4, 2, 16, 0) >= 100 * 2 * 16 * 4 and w(100, 64, 64, 4, 2, 16, 1) > 0
    assert s(0, 64, 64, 4, 2, 16) > 0 and w(0, 64, 64, 4, 2, 16, 1) > 0
    assert s(-1, 64, 64, 4, 2, 16) == 0 and w(1, 60, 64, 4, 2, 16, 0) == 0 and s(1, 64, 64, 4, 2, 200) == 0


def test_reference_gradients_against_differences():
    """<dy, out> is linear in x, a, b and w each: a difference with step 1 is
    exact up to rounding in 64 bits."""
    rng = np.random.default_rng(0)
    T, H, O, E, K, r = 5, 16, 8, 3, 2, 8
    v = dict(x=rng.standard_normal((T, H)), a=rng.standard_normal((E, r, H)), b=rng.standard_normal((E, O, r)),
             w=rng.standard_normal((T, K)))
    W, dy = rng.standard_normal((O, H)), rng.standard_normal((T, O))
    idx = rng.integers(-1, E, (T, K)).astype(np.int32)
    idx[0] = 1                                   # the same adapter twice

    def value():
        return R.forward(v["x"], W, v["a"], v["b"], idx, v["w"], 0.7)

    saved = value()[2]
    back = R.backward(v["x"], W, v["a"], v["b"], idx, v["w"], 0.7, dy, saved)
    for name, arr in v.items():
        g = back["d" + name][0]
        for at in np.ndindex(arr.shape):
            if name in "ab" and rng.random() < 0.8:
                continue
            d = []
            for s in (1.0, -1.0):
                arr[at] += s
                d.append(float((value()[0] * dy).sum()))
                arr[at] -= s
            assert abs((d[0] - d[1]) / 2 - g[at]) < 1e-10 * (1 + abs(d[0]) + abs(d[1]))


def test_an_output_inside_an_operand_is_refused():
    buf = torch.zeros(64, 8, dtype=torch.bfloat16)
    api._apart(buf[:32], x=buf[32:], topk_weights=None)        # neighbours
    api._apart(buf[8:8], x=buf)                                # nothing to write
    for out, x in ((buf, buf), (buf[:32], buf[31:]), (buf[31:], buf[:32]), (buf[8:16], buf)):
        with pytest.raises(ValueError, match="must not overlap x"):
            api._apart(out, topk_weights=None, x=x)
