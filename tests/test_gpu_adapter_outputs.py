"""The adapters' backward with some of its outputs left out (NULL at the C entry
point): the others are the same, bit for bit."""
import itertools

import pytest
import torch

import combine_get_dispatch_04_amd._native as N
from combine_get_dispatch_04_amd import api
from test_gpu_adapter import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T", [0, 5, 300, 2100])
def test_backward_without_some_of_its_outputs(T):
    H, O, E, K, r = 264, 200, 6, 2, 24
    c = Case(T + 3, T, H, O, E, K, r)
    x, W, a, b, idx, w = c.gpu()
    dy = c.dy.to(DEV)
    _, h = api.adapter_project(x, W, a, b, idx, w, scale=0.5)
    want = api.adapter_project_backward(dy, h)
    state_bytes = N.ep_adapter_state_bytes(T, H, O, E, K, r)
    state = torch.empty(state_bytes, dtype=torch.uint8, device=DEV) if h.state is None else h.state
    ws = torch.empty(N.ep_adapter_workspace_bytes(T, H, O, E, K, r, 1), dtype=torch.uint8, device=DEV)
    stream = torch.cuda.current_stream().cuda_stream
    for on in itertools.product([False, True], repeat=4):
        if not any(on):
            continue
        print("[case] outputs", T, on, flush=True)
        got = [torch.empty_like(t) if f else None for t, f in zip(want, on)]
        ws.fill_(255)
        N.ep_adapter_project_backward(dy.data_ptr(), x.data_ptr(), T, H, W.data_ptr(), O, a.data_ptr(), b.data_ptr(),
                                      E, r, idx.data_ptr(), w.data_ptr(), K, 0.5, state.data_ptr(), state_bytes,
                                      *[None if g is None else g.data_ptr() for g in got], ws.data_ptr(), ws.numel(),
                                      stream)
        for g, t in zip(got, want):
            assert g is None or torch.equal(g, t)
