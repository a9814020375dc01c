"""The experts as they are used: between dispatch and combine, replayed from a HIP graph, from several threads and
streams, what their results keep alive, and what the front end refuses."""
import threading

import pytest
import torch

import expert_ref as R
from combine_get_dispatch_04_amd import api

pytestmark = pytest.mark.gpu
DEV = "cuda"


def layer(T, K, E, H, I, seed=0):
    g = torch.Generator().manual_seed(seed)
    bf = lambda *s, by=1.0: (torch.randn(s, generator=g) * by).to(torch.bfloat16)  # noqa: E731
    x, up, down = bf(T, H), bf(E, 2 * I, H, by=H ** -0.5), bf(E, H, I, by=I ** -0.5)
    idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).to(torch.int32)
    idx[torch.rand((T, K), generator=g) < 0.1] = -1
    return [t.to(DEV) for t in (x, up, down, idx, torch.softmax(torch.randn((T, K), generator=g), 1))]


def chain(x, up, us, down, ds, idx, w, E, quant="bf16", between="bf16"):
    L = api.get_dispatch_layout(idx, E)
    recv, scales, h = api.dispatch(x, L, quant=quant)
    a, s, h1 = api.expert_product(recv, scales, up, us, offsets=L.offsets, activation="swiglu", quant=between)
    y, _, h2 = api.expert_product(a, s, down, ds, offsets=L.offsets)
    return api.combine(y, h, w), (L, h, h1, h2)


@pytest.mark.parametrize("T,K,E,H,I", [(1, 2, 4, 64, 32), (37, 3, 6, 256, 160), (128, 4, 12, 544, 352)])
def test_dispatch_products_combine_beside_the_few_tokens_layer(T, K, E, H, I):
    x, up, down, idx, w = layer(T, K, E, H, I)
    (uc, us), (dc, ds) = api.mx_quantize(up), api.mx_quantize(down)
    out, _ = chain(x, uc, us, dc, ds, idx, w, E)
    few, bad = api.low_latency_experts(x, idx, w, uc, dc, up_scales=us, down_scales=ds)
    U, D = R.values(uc.cpu(), us.cpu()), R.values(dc.cpu(), ds.cpu())
    ref, off = R.layer(x.cpu().double(), idx.cpu().long(), w.cpu(), U, D)
    R.assert_close(few, ref, off)
    assert int(bad) == 0
    # the chain rounds h and the products to bf16 as well
    more = torch.zeros_like(ref)
    for t in range(T):
        for k in range(K):
            e = int(idx[t, k])
            if e >= 0:
                h = R.gated(x[t:t + 1].cpu().double() @ U[e].T, torch.zeros(1, 2 * I, dtype=torch.float64))[0]
                y = h @ D[e].T
                more[t] += float(w[t, k]) * (R.HALF * (h.abs() @ D[e].abs().T) * (1 + R.HALF) + R.HALF * y.abs())[0]
    R.assert_close(out, ref, off * (1 + 3 * R.HALF) + more)


@pytest.mark.parametrize("quant", [R.FP4, R.E4M3, R.E5M2])
def test_quantised_rows_all_the_way(quant):
    """Each link of the chain on what the one before it really made."""
    T, K, E, H, I = 200, 2, 5, 320, 192
    x, up, down, idx, w = layer(T, K, E, H, I, 3)
    (uc, us), (dc, ds) = api.mx_quantize(up), api.mx_quantize(down)
    out, (L, h, h1, h2) = chain(x, uc, us, dc, ds, idx, w, E, quant, quant)
    off = L.offsets.cpu()
    n = int(off[-1])
    recv, a = (R.values(t.cpu()[:n], s.cpu()[:n]) for t, s in ((h1.x, h1.x_scales), (h2.x, h2.x_scales)))
    src = h.recv_src[:n].long().cpu()
    want, want_s = R.quantize(x.cpu()[src], quant)
    assert torch.equal(recv, R.values(want, want_s))
    U, D = R.values(uc.cpu(), us.cpu()), R.values(dc.cpu(), ds.cpu())
    y = api.expert_product(h2.x, h2.x_scales, dc, ds, offsets=L.offsets)[0]
    for e in range(E):
        at = slice(int(off[e]), int(off[e + 1]))
        v, tol = R.product(recv[at], U[e], True, quant=quant)
        ends = [R.values(R.pack(R.codes_of(t, h2.x_scales.cpu()[at], quant), quant), h2.x_scales.cpu()[at])
                for t in (v - tol, v + tol)]
        assert (a[at] >= ends[0]).all() and (a[at] <= ends[1]).all()
        v, tol = R.product(a[at], D[e], False, quant=quant)
        R.assert_close(y[at], v, tol)
    assert torch.equal(out, api.combine(y, h, w))


def test_low_latency_dispatch_and_expert_choice_rows():
    T, K, E, H, I = 60, 3, 7, 256, 96
    x, up, down, idx, w = layer(T, K, E, H, I, 5)
    (uc, us), (dc, ds) = api.mx_quantize(up), api.mx_quantize(down)
    U = R.values(uc.cpu(), us.cpu())
    recv, scales, h = api.low_latency_dispatch(x, idx, 20, E, quant=R.FP4)
    y = torch.full((E, 20, I), 3.0, dtype=torch.bfloat16, device=DEV)
    api.expert_product(recv, scales, uc, us, counts=h.recv_count, activation="swiglu", out=y)
    cnt = h.recv_count.cpu().tolist()
    assert max(cnt) == 20 and min(cnt) < 20
    for e in range(E):
        r = R.product(R.values(recv[e, :cnt[e]].cpu(), scales[e, :cnt[e]].cpu()), U[e], True)
        R.assert_close(y[e, :cnt[e]], *r)
        assert (y[e, cnt[e]:] == 3).all()
    ti = torch.randint(0, T, (E, 9), dtype=torch.int32, device=DEV)
    rows, _ = api.dispatch_expert_choice(x, ti, torch.rand((E, 9), device=DEV))
    y, _, _ = api.expert_product(rows, None, uc, us)
    for e in range(E):
        R.assert_close(y[e], *R.product(rows[e].cpu().double(), U[e], False))


def step(x, up, us, down, ds, idx, w, d, E, quant):
    """Forward through both products, the rows' gradient, and the few tokens' layer on the first 128."""
    out, (L, h, h1, h2) = chain(x, up, us, down, ds, idx, w, E, quant)
    dx = api.expert_product_backward(d, h1)
    codes, scales = api.mx_quantize(x, R.E4M3)
    few, n = api.low_latency_experts(x[:128], idx[:128], w[:128], up, down, up_scales=us, down_scales=ds)
    return dict(out=out, few=few, n=n, codes=codes, scales=scales, dx=dx), L.offsets


@pytest.mark.parametrize("T,K,E,H,I,quant", [(200, 2, 6, 256, 160, "bf16"), (600, 4, 5, 512, 256, R.FP4),
                                             (128, 4, 4, 288, 96, R.E5M2)])
def test_graph_replays(T, K, E, H, I, quant):
    x, up, down, idx, w = layer(T, K, E, H, I, 7)
    (uc, us), (dc, ds) = api.mx_quantize(up), api.mx_quantize(down)
    d = torch.randn((T * K, I), device=DEV).to(torch.bfloat16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(x, uc, us, dc, ds, idx, w, d, E, quant)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _ = step(x, uc, us, dc, ds, idx, w, d, E, quant)
    for r in range(4):
        x2, _, _, idx2, w2 = layer(T, K, E, H, I, 20 + r)
        x.copy_(x2)
        idx.copy_(idx2)
        w.copy_(w2)
        graph.replay()
        torch.cuda.synchronize()
        want, off = step(x2, uc, us, dc, ds, idx2, w2, d, E, quant)
        torch.cuda.synchronize()
        n = int(off[-1])
        for k in want:
            a, b = (got[k], want[k]) if k != "dx" else (got[k][:n], want[k][:n])
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (r, k)


def test_two_captured_calls_share_no_workspace():
    """Two graphs of the few tokens' layer, replayed on two streams at once."""
    jobs = []
    for seed in (1, 2):
        x, up, down, idx, w = layer(100, 3, 5, 512, 256, seed)
        want, _ = api.low_latency_experts(x, idx, w, up, down)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got, _ = api.low_latency_experts(x, idx, w, up, down)
        jobs.append((g, got, want, torch.cuda.Stream(), (x, up, down, idx, w)))
    for _ in range(5):
        for g, _, _, s, _ in jobs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, got, want, _, _ in jobs:
            assert torch.equal(got, want)


def test_calls_from_several_threads():
    jobs, want = [], []
    for seed, (T, K, E, H, I, quant) in enumerate([(90, 2, 5, 256, 96, "bf16"), (128, 8, 16, 192, 64, R.FP4),
                                                   (400, 1, 3, 320, 128, R.E4M3)]):
        x, up, down, idx, w = layer(T, K, E, H, I, seed)
        (uc, us), (dc, ds) = api.mx_quantize(up), api.mx_quantize(down)
        d = torch.randn((T * K, I), device=DEV).to(torch.bfloat16)
        jobs.append((x, uc, us, dc, ds, idx, w, d, E, quant))
        want.append(step(*jobs[-1]))
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(5):
                    got, off = step(*jobs[i])
                    s.synchronize()
                    n = int(off[-1])
                    for k, v in want[i][0].items():
                        a, b = (got[k][:n], v[:n]) if k == "dx" else (got[k], v)
                        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k
        except Exception as e:      # noqa: BLE001
            errors.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_results_keep_no_scratch_memory():
    x, up, down, idx, w = layer(300, 2, 4, 512, 256, 2)
    (uc, us), (dc, ds) = api.mx_quantize(up), api.mx_quantize(down)
    L = api.get_dispatch_layout(idx, 4)
    recv, _, _ = api.dispatch(x, L)

    def held(make, own):
        make()
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        kept = make()
        assert torch.cuda.memory_allocated() - before <= own + 2 * 512, kept
    held(lambda: api.expert_product(recv, None, uc, us, offsets=L.offsets, activation="swiglu"), 600 * 256 * 2)
    _, _, h = api.expert_product(recv, None, uc, us, offsets=L.offsets, activation="swiglu")
    d = torch.randn((600, 256), device=DEV).to(torch.bfloat16)
    held(lambda: api.expert_product_backward(d, h), 600 * 512 * 2)
    held(lambda: api.low_latency_experts(x[:128], idx[:128], w[:128], up, down), 128 * 512 * 2)


def test_refusals():
    E, H, O = 3, 64, 32
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    w, ws, x, off = u8(E, O, H // 2), u8(E, O, H // 32), bf(5, H), i32(E + 1)
    p = lambda x=x, xs=None, w=w, ws=ws, **k: api.expert_product(x, xs, w, ws, **{"offsets": off, **k})  # noqa: E731
    bad = [lambda: p(x=bf(5, H, 1)), lambda: p(x=bf(5, 2 * H)), lambda: p(x=x.float()), lambda: p(x=x.t()),
           lambda: p(xs=u8(5, 2)), lambda: p(x=u8(5, 32)), lambda: p(x=u8(5, 32), xs=u8(5, 1)),
           lambda: p(x=u8(5, 8), xs=u8(5, 0)), lambda: p(ws=u8(E, O, 1)), lambda: p(w=w[:, :, :16].contiguous()),
           lambda: p(w=torch.zeros((E, O, H), dtype=torch.float8_e4m3fn, device=DEV)), lambda: p(offsets=i32(E)),
           lambda: p(offsets=off.long()), lambda: p(counts=i32(E)), lambda: p(activation="gelu"),
           lambda: p(quant="int8"), lambda: p(quant=R.FP4, out=bf(5, O)), lambda: p(out=bf(5, O + 1)),
           lambda: p(out=x.view(-1)[:5 * O].view(5, O)), lambda: p(activation="swiglu", quant=R.FP4),
           lambda: p(offsets=None), lambda: p(x=bf(E + 1, 4, H), offsets=None),
           lambda: p(x=bf(E, 4, H), offsets=None, counts=i32(E + 1)), lambda: p(w=u8(E, 12, 32), ws=u8(E, 12, 2)),
           lambda: p(w=u8(E, 24, 32), ws=u8(E, 24, 2), activation="swiglu"), lambda: p(out=bf(5, O).cpu())]
    _, _, h = p()
    bad += [lambda: api.expert_product_backward(bf(5, O + 8), h), lambda: api.expert_product_backward(x.float(), h),
            lambda: api.expert_product_backward(bf(5, O), h, out=bf(5, O)),
            lambda: api.expert_product_backward(bf(5, O), h, out=x)]
    bad += [lambda: api.mx_quantize(bf(4, 48)), lambda: api.mx_quantize(bf(4, 0)), lambda: api.mx_quantize(bf(64, 4).t()),
            lambda: api.mx_quantize(x.half()), lambda: api.mx_quantize(bf(4, 64), "fp8_e4m3_g128"),
            lambda: api.mx_dequantize(u8(4, 32), u8(4, 1)), lambda: api.mx_dequantize(u8(4, 32), u8(4, 2).float()),
            lambda: api.mx_dequantize(bf(4, 32), u8(4, 1)), lambda: api.mx_dequantize(u8(4, 0), u8(4, 0))]
    up, down, idx, tw = bf(E, 2 * O, H), bf(E, H, O), i32(5, 2), torch.zeros((5, 2), device=DEV)
    few = lambda x=x, idx=idx, tw=tw, up=up, down=down, **k: api.low_latency_experts(x, idx, tw, up, down, **k)  # noqa: E731
    bad += [lambda: few(idx=i32(4, 2)), lambda: few(tw=tw[:, :1].contiguous()), lambda: few(tw=tw.half()),
            lambda: few(up=bf(E, O, H)), lambda: few(up=bf(E, 2 * O, 2 * H)), lambda: few(down=bf(E + 1, H, O)),
            lambda: few(up_scales=u8(E, 2 * O, 2)), lambda: few(up=u8(E, 2 * O, H // 2)), lambda: few(out=x),
            lambda: few(out=bf(5, H + 8)), lambda: few(x=bf(129, H), idx=i32(129, 2), tw=None),
            lambda: few(idx=i32(5, 65), tw=None), lambda: few(up=u8(E, 2 * O, 32), down=u8(E, H, 16),
                                                             up_scales=u8(E, 2 * O, 2), down_scales=u8(E, H, 2))]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            print("not refused:", i)
    torch.cuda.synchronize()


def test_arrays_past_4_gib():
    g = torch.Generator().manual_seed(1)
    bf = lambda *s, by=1.0: (torch.randn(s, generator=g) * by).to(torch.bfloat16)  # noqa: E731
    # rows
    n, H, O, last = 600_000, 4096, 64, 301
    x = torch.zeros((n, H), dtype=torch.bfloat16, device=DEV)
    tail = bf(last, H)
    x[-last:] = tail.to(DEV)
    w, ws = R.quantize(bf(2, O, H, by=H ** -0.5), R.FP4)
    off = torch.tensor([0, n - last, n], dtype=torch.int32, device=DEV)
    want = R.product(tail.double(), R.values(w, ws)[1], False)
    y, _, h = api.expert_product(x, None, w.to(DEV), ws.to(DEV), offsets=off)
    R.assert_close(y[-last:], *want)
    assert not y[:-last].any()
    d = torch.zeros((n, O), dtype=torch.bfloat16, device=DEV)
    d[-last:] = bf(last, O).to(DEV)
    dx = api.expert_product_backward(d, h)
    R.assert_close(dx[-last:], *R.product(tail.double(), R.values(w, ws)[1], False, d[-last:].cpu().double())[2:])
    assert not dx[:-last].any()
    codes, scales = api.mx_quantize(x)
    del x, y, d, dx, h
    big = torch.zeros((4 * n, H // 2), dtype=torch.uint8, device=DEV)
    big_s = torch.zeros((4 * n, H // 32), dtype=torch.uint8, device=DEV)
    big[-last:], big_s[-last:] = codes[-last:], scales[-last:]
    off = torch.tensor([0, last, 4 * n], dtype=torch.int32, device=DEV)
    y, _, _ = api.expert_product(big[-2 * last:], big_s[-2 * last:], w.to(DEV), ws.to(DEV),
                                 offsets=torch.tensor([0, last, 2 * last], dtype=torch.int32, device=DEV))
    z, _, _ = api.expert_product(big, big_s, w.to(DEV), ws.to(DEV), offsets=off)
    v, tol = R.product(R.values(codes[-last:].cpu(), scales[-last:].cpu()), R.values(w, ws)[1], False)
    R.assert_close(y[-last:], v, tol)
    R.assert_close(z[-last:], v, tol)
    del big, big_s, y, z
    # weights
    E, H, I = 200, 4096, 2048
    up = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device=DEV)
    down = torch.zeros((E, H, I), dtype=torch.bfloat16, device=DEV)
    up[-1], down[-1] = bf(2 * I, H, by=H ** -0.5).to(DEV), bf(H, I, by=I ** -0.5).to(DEV)
    xs, idx = bf(1, H).to(DEV), torch.tensor([[E - 1]], dtype=torch.int32, device=DEV)
    out, _ = api.low_latency_experts(xs, idx, None, up, down)
    one, _ = api.low_latency_experts(xs, idx * 0, None, up[-1:], down[-1:])
    assert torch.equal(out, one) and out.any()
    uc, us = api.mx_quantize(up[-1:])
    codes = torch.zeros((600, 2 * I, H // 2), dtype=torch.uint8, device=DEV)
    sc = torch.zeros((600, 2 * I, H // 32), dtype=torch.uint8, device=DEV)
    codes[-1], sc[-1] = uc[0], us[0]
    rows = xs.repeat(3, 1)
    off = torch.zeros(601, dtype=torch.int32, device=DEV)
    off[-1] = 3
    y, _, _ = api.expert_product(rows, None, codes, sc, offsets=off)
    one, _, _ = api.expert_product(rows, None, uc, us, offsets=torch.tensor([0, 3], dtype=torch.int32, device=DEV))
    assert torch.equal(y, one) and y.any()


@pytest.mark.parametrize("fp4,T,K,E,H,I", [(True, 128, 8, 40, 288, 608), (False, 128, 8, 16, 136, 1032),
                                           (True, 2, 8, 12, 1056, 4128), (True, 100, 2, 3, 96, 32)])
def test_few_tokens_layers_in_a_graph(fp4, T, K, E, H, I):
    """Replayed with other tokens and other numbers of them for each expert, eager calls in between."""
    x, up, down, idx, w = layer(T, K, E, H, I, 3)
    us = ds = None
    if fp4:
        (up, us), (down, ds) = api.mx_quantize(up), api.mx_quantize(down)
    run = lambda x, idx, w: api.low_latency_experts(x, idx, w, up, down, up_scales=us, down_scales=ds)  # noqa: E731
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(x, idx, w)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, bad = run(x, idx, w)
    for r in range(5):
        x2, _, _, idx2, w2 = layer(T, K, E, H, I, 50 + r)
        if r == 2:
            idx2[:] = -1
        if r == 3:
            idx2[:] = idx2[:1]          # all tokens at the same experts
            idx2[-1, 0] = E
        x.copy_(x2)
        idx.copy_(idx2)
        w.copy_(w2)
        graph.replay()
        torch.cuda.synchronize()
        want, n = run(x2, idx2, w2)
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and int(bad) == int(n) == (r == 3), r
