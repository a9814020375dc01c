"""Sizes that a 32-bit argument cannot hold: refused by the front end, where the C call would get what is left
of them (tensors without memory stand for those of the GPU)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import combine_get_dispatch_04_amd._native as N
from combine_get_dispatch_04_amd import api

BF, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
FAR = 1 << 32


def fake(shape, dtype):
    with FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device="cuda")


def refused(call):
    with pytest.raises(N.EpError) as e:
        call()
    assert e.value.status == N.EP_ERR_UNSUPPORTED


@pytest.mark.parametrize("shape", [(FAR + 64,), (FAR + 5, 32), (1 << 31, 32), (1 << 20, 1 << 12, 32)])
def test_quantisation(shape):
    refused(lambda: api.mx_quantize(fake(shape, BF)))
    c, s = (*shape[:-1], shape[-1] // 2), (*shape[:-1], shape[-1] // 32)
    refused(lambda: api.mx_dequantize(fake(c, U8), fake(s, U8)))


def _rows(rows=8, E=2, O=32, H=64, cap=None):
    x = (fake((E, cap, H), BF) if cap else fake((rows, H), BF), None)
    w = fake((E, O, H // 2), U8), fake((E, O, H // 32), U8)
    off = {} if cap else dict(offsets=fake((E + 1,), I32))
    return x, w, off


@pytest.mark.parametrize("kw", [dict(rows=FAR + 5), dict(rows=1 << 31), dict(E=FAR + 2), dict(O=FAR + 32),
                                dict(H=FAR + 64), dict(E=1 << 12, cap=1 << 20), dict(E=1, cap=FAR + 8)])
def test_products(kw):
    x, w, off = _rows(**kw)
    refused(lambda: api.expert_product(*x, *w, **off))
    h = api.ExpertHandle(*x, *w, off.get("offsets"), None, None)
    refused(lambda: api.expert_product_backward(fake((*x[0].shape[:-1], w[0].shape[1]), BF), h))


@pytest.mark.parametrize("kw", [dict(T=FAR + 1), dict(T=1 << 31), dict(K=FAR + 2), dict(E=FAR + 4), dict(H=FAR + 64),
                                dict(I=FAR + 32)])
def test_a_few_tokens(kw):
    d = dict(T=2, K=1, E=4, H=64, I=32)
    d.update(kw)
    T, K, E, H, I = d.values()
    refused(lambda: api.low_latency_experts(fake((T, H), BF), fake((T, K), I32), fake((T, K), F32), fake((E, 2 * I, H), BF),
                                            fake((E, H, I), BF)))
