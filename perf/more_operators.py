"""The experts' products in microscaled floating point, and a whole layer of
experts for a few tokens: what they are measured on.

Conventions of the token dispatch: topk_idx is int32 [T, K] with -1 for an
entry that is not used; an expert's rows stand together, at offsets[e] of a
contiguous buffer or at e * cap of a padded one; MX codes have one e8m0 scale
per 32 channels (e2m1: two codes per byte, the lower channel in the low nibble).

- quantise: bf16 to MX codes and scales, and back to bf16.
- product: y = W_e x for every row of every expert, W in MXFP4 [E, O, H], rows
  in MXFP4, MXFP8 or bf16; with "swiglu" silu(y[:O/2]) * y[O/2:]; training:
  also the rows' gradient (W is frozen).
- chain: the two products of an expert, the hidden rows quantised in between.
- layer: out_t = sum_k w_tk W2_e (silu(Wg_e x_t) * (Wu_e x_t)) for a few
  tokens, weights in bf16 or MXFP4.
"""
import math

import torch

own = False

DEV = "cuda"
FP4, E4M3, E5M2 = "mxfp4_e2m1", "mxfp8_e4m3", "mxfp8_e5m2"
EMAX = {FP4: 2, E4M3: 8, E5M2: 15}
MOST = {FP4: 6.0, E4M3: 448.0, E5M2: 57344.0}
CODES = {FP4: torch.uint8, E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}


# ------------------------------------------------------------------ the cases
def _quantise(name, E, rows, H, quant):
    return dict(name=name, op="quantise", E=E, rows=rows, H=H, quant=quant)


def _product(name, T, K, E, H, O, rows, act, train, padded):
    return dict(name=name, op="product", T=T, K=K, E=E, H=H, O=O, rows=rows, act=act, train=train, padded=padded)


def _chain(name, T, K, E, H, I, rows):
    return dict(name=name, op="chain", T=T, K=K, E=E, H=H, I=I, rows=rows)


def _layer(name, T, K, E, H, I, weights, none):
    return dict(name=name, op="layer", T=T, K=K, E=E, H=H, I=I, weights=weights, none=none)


def listed():
    return [
        # the rows of a decode batch, before an experts' product: latency alone
        _quantise("quantise_decode", 1, 128, 7168, E4M3),
        # the weights of 16 experts, once when a model is loaded, or at each step of one trained through its rounding
        _quantise("quantise_weights", 16, 4096, 7168, FP4),
        # a decode batch's rows in the padded buffer, few for each expert: the weights' bytes
        _product("product_decode", 128, 8, 64, 7168, 4096, E4M3, "", False, True),
        # prefill, rows as the dispatch quantises them, the gated half of an expert
        _product("product_prefill", 4096, 8, 64, 4096, 4096, FP4, "swiglu", False, False),
        # bf16 rows of uneven experts, sizes that fill no tile, forward and backward
        _product("product_odd", 1001, 2, 12, 1120, 1032, "bf16", "", True, False),
        # fine-tuning in front of frozen experts: through the gated half and back
        _product("product_train", 4096, 2, 8, 4096, 4096, "bf16", "swiglu", True, False),
        # prefill through both products of the experts
        _chain("chain_prefill", 4096, 8, 64, 7168, 2048, FP4),
        # a toy layer, one token: latency alone
        _layer("layer_toy", 1, 2, 8, 1024, 512, "bf16", 0.0),
        # decode, one request
        _layer("layer_one_token", 1, 8, 64, 4096, 2048, "bf16", 0.0),
        # the same with 4-bit weights, wider
        _layer("layer_one_token_4bit", 1, 8, 64, 7168, 2048, FP4, 0.0),
        # decode, 32 requests: nearly every expert, a few rows each
        _layer("layer_batch", 32, 8, 64, 4096, 2048, "bf16", 0.05),
        # decode, 128 requests over few experts, more rows than a tile has
        _layer("layer_batch_4bit", 128, 2, 8, 4096, 4096, FP4, 0.0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "product", "product", "chain", "layer", "layer"])
    if op == "quantise":
        return _quantise("", rng.choice([1, 1, 3, 8]), _spread(rng, 1, 4096), 32 * _spread(rng, 2, 224),
                         rng.choice([FP4, FP4, E4M3, E5M2]))
    E = _spread(rng, 1, 64)
    K = rng.randint(1, min(8, E))
    if op == "product":
        rows = rng.choice([FP4, FP4, E4M3, E5M2, "bf16", "bf16"])
        H, O = 32 * _spread(rng, 4, 128), 16 * _spread(rng, 8, 256)
        return _product("", _spread(rng, 1, 4096), K, E, H, O, rows, rng.choice(["", "swiglu"]), rng.random() < 0.5,
                        rng.random() < 0.4)
    if op == "chain":
        return _chain("", _spread(rng, 16, 4096), K, E, 32 * _spread(rng, 8, 128), 32 * _spread(rng, 4, 64),
                      rng.choice([FP4, FP4, E4M3]))
    return _layer("", _spread(rng, 1, 128), K, E, 32 * _spread(rng, 8, 128), 32 * _spread(rng, 4, 64),
                  rng.choice(["bf16", FP4]), rng.choice([0.0, 0.1]))


# --------------------------------------------------- microscaled numbers, plain
def _pow2(n):
    """2^n in fp32 for whole n in [-127, 127]."""
    n = n.to(torch.int32)
    return torch.where(n > -127, (n + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _to_mx(v, quant):
    """fp32 values [..., H] -> codes, e8m0 scales."""
    H = v.shape[-1]
    b = v.view(*v.shape[:-1], H // 32, 32)
    top = b.abs().amax(dim=-1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 1 - EMAX[quant], -127).clamp(-127, 127)
    s = (b * _pow2(-e).unsqueeze(-1)).clamp(-MOST[quant], MOST[quant])
    if quant == FP4:
        a = s.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        q = torch.round(a / step) * step                                   # to the nearest, ties to even
        code = torch.where(q < 2, 2 * q, torch.where(q < 4, q + 2, q / 2 + 4)).to(torch.uint8)
        code = (code + 8 * torch.signbit(s).to(torch.uint8)).view(*v.shape)
        codes = code[..., 0::2] + 16 * code[..., 1::2]
    else:
        codes = s.view(*v.shape).to(CODES[quant])
    return codes.contiguous(), (e + 127).to(torch.uint8).contiguous()


def _values(codes, scales):
    """fp32 values of MX codes."""
    if codes.dtype == torch.uint8:
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                             device=DEV)
        both = torch.stack([codes & 15, codes >> 4], dim=-1).to(torch.int32)
        v = table.index_select(0, both.view(-1)).view(*codes.shape[:-1], 2 * codes.shape[-1])
    else:
        v = codes.float()
    b = v.view(*v.shape[:-1], scales.shape[-1], 32)
    return (b * _pow2(scales.to(torch.int32) - 127).unsqueeze(-1)).view(v.shape)


# ----------------------------------------------------------------- the inputs
def _choice(g, T, E, K):
    """K different experts for each token, some experts busier than others."""
    z = torch.randn((T, E), generator=g, device=DEV) + 0.5 * torch.randn(E, generator=g, device=DEV)
    return torch.sort(z, dim=1, descending=True, stable=True)[1][:, :K].to(torch.int32).contiguous()


def _capacity(T, K, E):
    """Rows of an expert in a padded buffer: 2.5 times the average, at most one for each token."""
    return min(T, 16 + 5 * T * K // (2 * E))


def _randn(g, *shape, by=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * by).to(torch.bfloat16)


def _weight(g, E, O, H, quant):
    """[E, O, H] in bf16, or its codes and scales; expert after expert, for their size."""
    if quant == "bf16":
        return torch.stack([_randn(g, O, H, by=H ** -0.5) for _ in range(E)]), None
    parts = [_to_mx(_randn(g, O, H, by=H ** -0.5).float(), quant) for _ in range(E)]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])


def _rows(g, n, H, quant):
    x = _randn(g, n, H)
    return (x, None) if quant == "bf16" else _to_mx(x.float(), quant)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    c = case
    s = dict(case=dict(c))
    if c["op"] == "quantise":
        shape = (c["rows"], c["H"]) if c["E"] == 1 else (c["E"], c["rows"], c["H"])
        s["x"] = _randn(g, *shape)
        return s
    T, K, E, H = c["T"], c["K"], c["E"], c["H"]
    idx = _choice(g, T, E, K)
    if c["op"] == "layer":
        if c["none"] > 0:
            idx = torch.where(torch.rand((T, K), generator=g, device=DEV) < c["none"], -1, idx)
        s["idx"] = idx.to(torch.int32).contiguous()
        s["w"] = torch.softmax(torch.randn((T, K), generator=g, device=DEV), dim=1).contiguous()
        s["x"] = _randn(g, T, H)
        s["up"], s["up_scales"] = _weight(g, E, 2 * c["I"], H, c["weights"])
        s["down"], s["down_scales"] = _weight(g, E, H, c["I"], c["weights"])
        return s
    padded = c["op"] == "product" and c["padded"]
    counts = torch.bincount(idx.flatten().long(), minlength=E)
    if padded:                                          # what an expert gets beyond the capacity is dropped
        counts = counts.clamp(max=_capacity(T, K, E))
    s["most"] = _capacity(T, K, E) if padded else int(counts.max())
    s["counts"] = counts.to(torch.int32)
    s["offsets"] = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)]).to(torch.int32)
    O = 2 * c["I"] if c["op"] == "chain" else c["O"]
    s["weight"], s["weight_scales"] = _weight(g, E, O, H, FP4)
    n = E * s["most"] if padded else T * K
    x, xs = _rows(g, n, H, c["rows"])
    if padded:
        x = x.view(E, s["most"], -1)
        xs = None if xs is None else xs.view(E, s["most"], -1)
    s["x"], s["x_scales"] = x, xs
    if c["op"] == "chain":
        s["down"], s["down_scales"] = _weight(g, E, H, c["I"], FP4)
        return s
    width = O // 2 if c["act"] else O
    if padded:                                          # rows without a token stay as they are
        s["y"] = torch.zeros((E, s["most"], width), dtype=torch.bfloat16, device=DEV)
    if c["train"]:
        s["d_y"] = _randn(g, *x.shape[:-1], width)
        if padded:
            s["dx"] = torch.zeros((E, s["most"], H), dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------ the plain forms
def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _gated(y):
    half = y.shape[-1] // 2
    return y[..., :half] * _sigmoid(y[..., :half]) * y[..., half:]


def _gated_grad(y, d):
    half = y.shape[-1] // 2
    gate, up = y[..., :half], y[..., half:]
    s = _sigmoid(gate)
    return torch.cat([d * up * s * (1.0 + gate * (1.0 - s)), d * gate * s], dim=-1)


def _places(s):
    """Of contiguous rows: each row's expert and place in it; of the padded ones: which row stands there, and whether one does."""
    E, most = s["case"]["E"], s["most"]
    off = s["offsets"].long()
    n = s["case"]["T"] * s["case"]["K"]
    row = torch.arange(n, device=DEV)
    expert = torch.searchsorted(off, row, right=True) - 1
    at = off[:E].view(E, 1) + torch.arange(most, device=DEV)
    live = at < off[1:].view(E, 1)
    return expert, row - off[expert], at.clamp(max=n - 1), live


def _plain_product(s):
    c = s["case"]
    w = _values(s["weight"], s["weight_scales"]).transpose(1, 2)
    x = s["x"].float() if s["x_scales"] is None else _values(s["x"], s["x_scales"])
    d = s["d_y"].float() if c["op"] == "product" and c["train"] else None
    if s["x"].dim() == 2:
        expert, place, at, live = _places(s)
        x = x[at]
        d = None if d is None else d[at]
        back = lambda v: v[expert, place]  # noqa: E731
    else:
        live = torch.arange(s["most"], device=DEV) < s["counts"].view(-1, 1)
        back = lambda v: torch.where(live.unsqueeze(2), v, 0.0)  # noqa: E731
    y = torch.bmm(x, w)
    if c["op"] == "chain":
        h = _values(*_to_mx(_gated(y), c["rows"]))
        y = torch.bmm(h, _values(s["down"], s["down_scales"]).transpose(1, 2))
        return dict(y=back(y).to(torch.bfloat16))
    out = dict(y=back(_gated(y) if c["act"] else y).to(torch.bfloat16))
    if d is not None:
        d = _gated_grad(y, d) if c["act"] else d
        out["dx"] = back(torch.bmm(d, w.transpose(1, 2))).to(torch.bfloat16)
    return out


def _plain_layer(s):
    c = s["case"]
    T, K, E = c["T"], c["K"], c["E"]
    x, idx = s["x"].float(), s["idx"]
    wide = lambda v, sc, e: (v[e].float() if sc is None else _values(v[e], sc[e]))  # noqa: E731
    w = torch.where(idx >= 0, s["w"], 0.0)
    at = torch.where(idx >= 0, idx, 0).long()
    if T * K <= E:      # the entries' own experts
        e = at.view(-1)
        xe = x.view(T, 1, 1, -1).expand(T, K, 1, -1).reshape(T * K, 1, -1)
        h = _gated(torch.bmm(xe, wide(s["up"], s["up_scales"], e).transpose(1, 2)))
        y = torch.bmm(h, wide(s["down"], s["down_scales"], e).transpose(1, 2)).view(T, K, -1)
        return (y * w.unsqueeze(2)).sum(dim=1).to(torch.bfloat16)
    e = torch.arange(E, device=DEV)
    h = _gated(torch.matmul(x, wide(s["up"], s["up_scales"], e).transpose(1, 2)))       # [E, T, I]
    y = torch.bmm(h, wide(s["down"], s["down_scales"], e).transpose(1, 2))
    coef = torch.zeros((T, E), device=DEV).scatter_add_(1, at, w)
    return (y * coef.t().unsqueeze(2)).sum(dim=0).to(torch.bfloat16)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "quantise":
        codes, scales = _to_mx(s["x"].float(), c["quant"])
        return dict(values=_values(codes, scales).to(torch.bfloat16), scales=scales)
    if c["op"] == "layer":
        return dict(out=_plain_layer(s))
    return _plain_product(s)


# ------------------------------------------------------- the framework's calls
def _run_own(s):
    from combine_get_dispatch_04_amd import api
    c = s["case"]
    if c["op"] == "quantise":
        codes, scales = api.mx_quantize(s["x"], quant=c["quant"])
        return dict(values=api.mx_dequantize(codes, scales), scales=scales)
    if c["op"] == "layer":
        out, _ = api.low_latency_experts(s["x"], s["idx"], s["w"], s["up"], s["down"], up_scales=s["up_scales"],
                                         down_scales=s["down_scales"])
        return dict(out=out)
    if c["op"] == "chain":
        h, hs, _ = api.expert_product(s["x"], s["x_scales"], s["weight"], s["weight_scales"], offsets=s["offsets"],
                                      activation="swiglu", quant=c["rows"])
        y, _, _ = api.expert_product(h, hs, s["down"], s["down_scales"], offsets=s["offsets"])
        return dict(y=y)
    where = dict(counts=s["counts"], out=s["y"]) if c["padded"] else dict(offsets=s["offsets"])
    y, _, handle = api.expert_product(s["x"], s["x_scales"], s["weight"], s["weight_scales"],
                                      activation=c["act"] or None, **where)
    out = dict(y=y)
    if c["train"]:
        out["dx"] = api.expert_product_backward(s["d_y"], handle, out=s.get("dx"))
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------- what a pass cannot avoid
def _used(E, n):
    """Experts that n entries name, on average."""
    return E * (1.0 - (1.0 - 1.0 / E) ** n) if E > 1 else 1.0


def _bytes(quant):
    return {"bf16": 2.0, FP4: 0.5 + 1 / 32, E4M3: 1 + 1 / 32, E5M2: 1 + 1 / 32}[quant]


def work(case):
    c = case
    if c["op"] == "quantise":
        n = float(c["E"] * c["rows"] * c["H"])
        return {"bytes": n * (4 + 1 / 32), "flops": 4 * n}
    n, H = float(c["T"] * c["K"]), c["H"]
    used = _used(c["E"], n)
    if c["op"] == "layer":
        n *= 1.0 - c["none"]
        weights = 3.0 * H * c["I"]
        return {"bytes": used * weights * _bytes(c["weights"]) + 4 * c["T"] * H + 8 * c["T"] * c["K"],
                "flops": 2 * n * weights}
    if c["op"] == "chain":
        weights = 3.0 * H * c["I"]
        return {"bytes": used * weights * _bytes(FP4) + n * H * (2 + _bytes(c["rows"])), "flops": 2 * n * weights}
    O, width = c["O"], c["O"] // 2 if c["act"] else c["O"]
    b = used * O * H * _bytes(FP4) + n * (H * _bytes(c["rows"]) + 2 * width)
    f = 2.0 * n * H * O
    if c["train"]:
        b += n * 2 * (width + H)
        f *= 2
    return {"bytes": b, "flops": f}


# --------------------------------------------------- the definition in 64 bits
def _exact_quantise(x, quant):
    """Codes' values by distance: the nearest of all that the format has, ties to the even one."""
    v = x.double()
    b = v.view(*v.shape[:-1], -1, 32)
    top = b.abs().max(dim=-1, keepdim=True).values
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - EMAX[quant]
    scale = torch.pow(torch.tensor(2.0, dtype=torch.float64, device=DEV), torch.clamp(e, -127, 127))
    z = (b / scale).abs()
    if quant == FP4:
        grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    else:
        bits, bias = (3, 7) if quant == E4M3 else (2, 15)
        grid = [m * 2.0 ** (1 - bias - bits) for m in range(1 << bits)]
        grid += [(1 + m / (1 << bits)) * 2.0 ** (p - bias) for p in range(1, 32) for m in range(1 << bits)]
        grid = [q for q in grid if q <= MOST[quant]]
    grid = torch.tensor(grid, dtype=torch.float64, device=DEV)
    middle = (grid[1:] + grid[:-1]) / 2
    low = torch.bucketize(z, middle)                     # middles below z
    tie = (low < middle.numel()) & (z == middle[low.clamp(max=middle.numel() - 1)])
    low = torch.where(tie & (low % 2 == 1), low + 1, low)
    return (torch.copysign(grid[low], b) * scale).view(v.shape)


def _exact_values(codes, scales, quant):
    if quant == "bf16":
        return codes.double()
    if quant == FP4:
        n = torch.stack([codes % 16, torch.div(codes, 16, rounding_mode="floor")], dim=-1).flatten(-2).double()
        mag = n % 8
        small = mag / 2
        mag = torch.where(mag < 4, small, torch.where(mag < 6, mag - 2, 2 * mag - 8))
        v = torch.where(n >= 8, -mag, mag)
    else:
        v = codes.double()
    two = torch.tensor(2.0, dtype=torch.float64, device=DEV)
    return v * torch.pow(two, scales.double() - 127).repeat_interleave(32, dim=-1)


def _exact_expert(s, e, x):
    """An expert's y in front of the activation, and its weight."""
    w = _exact_values(s["weight"][e], s["weight_scales"][e], FP4)
    return torch.matmul(x, w.T), w


def _exact_gate(y):
    a, b = y.chunk(2, dim=-1)
    return a / (1 + torch.exp(-a)) * b


def _exact_product(s):
    c = s["case"]
    E, padded = c["E"], s["x"].dim() == 3
    x = _exact_values(s["x"], s["x_scales"], c["rows"])
    off = s["offsets"].tolist()
    width = c["H"] if c["op"] == "chain" else c["O"] // 2 if c["act"] else c["O"]
    out = dict(y=torch.zeros((*x.shape[:-1], width), dtype=torch.float64, device=DEV))
    train = c["op"] == "product" and c["train"]
    if train:
        out["dx"] = torch.zeros_like(x)
    for e in range(E):
        at = (e, slice(0, off[e + 1] - off[e])) if padded else slice(off[e], off[e + 1])
        y, w = _exact_expert(s, e, x[at])
        if c["op"] == "chain":
            h = _exact_quantise(_exact_gate(y), c["rows"])
            out["y"][at] = torch.matmul(h, _exact_values(s["down"][e], s["down_scales"][e], FP4).T)
            continue
        out["y"][at] = _exact_gate(y) if c["act"] else y
        if train:
            d = s["d_y"][at].double()
            if c["act"]:
                a, b = y.chunk(2, dim=-1)
                p = 1 / (1 + torch.exp(-a))
                d = torch.cat([d * b * (p + a * p * (1 - p)), d * a * p], dim=-1)
            out["dx"][at] = torch.matmul(d, w)
    return out


def _exact_layer(s):
    c = s["case"]
    x, idx = s["x"].double(), s["idx"].long()
    out = torch.zeros_like(x)
    for e in torch.unique(idx[idx >= 0]).tolist():
        t, k = torch.nonzero(idx == e, as_tuple=True)
        up = _exact_values(s["up"][e], None if s["up_scales"] is None else s["up_scales"][e], c["weights"])
        down = _exact_values(s["down"][e], None if s["down_scales"] is None else s["down_scales"][e], c["weights"])
        h = _exact_gate(torch.matmul(x[t], up.T))
        out.index_add_(0, t, torch.matmul(h, down.T) * s["w"][t, k].double().unsqueeze(1))
    return dict(out=out)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        return dict(values=_exact_quantise(s["x"], case["quant"]), scales=None)
    if case["op"] == "layer":
        return _exact_layer(s)
    return _exact_product(s)
