"""The adapters' projection in every form of its tiles, forward and for the
gradient of x, with lengths that no tile divides, and with an infinite value in an
adapter, which a wave's second pass keeps apart.  test_operators_sanitize.py holds
the shapes below to the forms that they name."""
import numpy as np
import pytest
import torch

import adapter_ref as R
from combine_get_dispatch_04_amd import api
from test_gpu_adapter import Case, close, say
from test_gpu_adapter_infinite import same_kind

pytestmark = pytest.mark.gpu
DEV = "cuda"

# (T, H, O, E, K, r): tokens of a tile, columns of the forward's tiles, and of those of dx
FORMS = {
    (333, 200, 136, 5, 2, 24): (64, 64, 64),
    (1001, 640, 2056, 9, 1, 24): (64, 96, 64),
    (1001, 520, 4088, 7, 1, 24): (64, 128, 64),
    (1001, 4088, 520, 7, 2, 40): (64, 64, 128),
    (12300, 264, 280, 30, 1, 16): (128, 128, 128),
    (6200, 2048, 2056, 6, 1, 16): (256, 256, 256),
}


def run(c):
    out, h = api.adapter_project(*c.gpu(), scale=c.scale)
    return out, dict(zip(("dx", "da", "db", "dw"), api.adapter_project_backward(c.dy.to(DEV), h)))


@pytest.mark.parametrize("shape", FORMS)
def test_every_form(shape):
    say("form", *shape)
    c = Case(sum(shape), *shape, "requests" if shape[4] == 1 else "mixed", shape[4] > 1)
    out, grads = run(c)
    want, bound, saved = c.ref()
    close("out", out, want, bound)
    for name, (g, b) in c.ref_back(saved).items():
        close(name, grads[name], g, b)


@pytest.mark.parametrize("where", ["a", "b"])
@pytest.mark.parametrize("shape", [s for s, f in FORMS.items() if f[0] == 64])
def test_an_infinite_adapter_in_every_form_of_64(shape, where):
    say("form, infinite", where, *shape)
    clean, c = (Case(sum(shape), *shape, "mixed", weights=False) for _ in range(2))
    e = int(np.bincount(c.idx[(c.idx >= 0) & (c.idx < shape[3])]).argmax())
    at = (e, 3, shape[1] - 2) if where == "a" else (e, shape[2] - 3, 2)
    getattr(c, where)[at] = float("-inf")
    setattr(c, where + "64", getattr(c, where).double().numpy())
    out, grads = run(c)
    value, bound, saved = clean.ref()
    back = clean.ref_back(saved)
    with np.errstate(invalid="ignore", over="ignore"):
        value_b, _, saved_b = c.ref()
        back_b = c.ref_back(saved_b)
    reached = [same_kind("out", out, value_b, value, bound)]
    for name, (g, b) in back.items():
        reached.append(same_kind(name, grads[name], back_b[name][0], g, b))
    assert reached[0] and reached[1]


def test_a_dense_matrix_past_32_bits():
    """Every tile names about a thousand adapters: each part of the dense matrix
    takes more than 2^32 bytes.  All tiles are the same small problem."""
    n, H, O, E, K, r = 547, 64, 64, 1024, 16, 16
    say("dense matrix", n * 256, H, O, E, K, r)
    c = Case(17, 256, H, O, E, K, r)
    x, W, a, b, idx, w = c.gpu()
    many = lambda t: t.repeat(n, 1).contiguous()  # noqa: E731
    out, h = api.adapter_project(many(x), W, a, b, many(idx), many(w), scale=c.scale)
    dx, da, db, dw = api.adapter_project_backward(many(c.dy.to(DEV)), h)
    assert h.state.numel() > 1 << 33
    want, bound, saved = c.ref()
    back = c.ref_back(saved)
    for i in (0, n // 2, n - 1):
        at = slice(256 * i, 256 * (i + 1))
        close("out", out[at], want, bound)
        close("dx", dx[at], *back["dx"])
        close("dw", dw[at], *back["dw"])
    # n times the small problem's sums; the order of n * 256 additions in fp32 besides
    mag_a, mag_b = np.zeros(c.a64.shape), np.zeros(c.b64.shape)
    for t, e, ks, coef, cm, u, eu, ec in saved["entries"]:
        mag_a[e] += np.outer(np.abs(coef * (c.b64[e].T @ c.dy64[t])), np.abs(c.x64[t]))
        mag_b[e] += np.outer(np.abs(c.dy64[t]), np.abs(coef * u))
    for name, got, mag in (("da", da, mag_a), ("db", db, mag_b)):
        g, e = back[name]
        e = n * e + 2 * n * 256 * R.U * n * mag
        close(name, got, n * g, e + R.H * (np.abs(n * g) + e))
