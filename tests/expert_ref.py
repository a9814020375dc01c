"""Microscaled tensors, the experts' products and the few tokens' layer in 64 bits,
with the bounds their kernels are held to.

The bounds count roundings: half a step of the result's type, and for a sum of n
products in fp32 at most (n + 8) steps of 2^-23 of the sum of their magnitudes
(the matrix units' additions may truncate: a whole step each, not half of one)."""
import torch

FP4, E4M3, E5M2 = "mxfp4_e2m1", "mxfp8_e4m3", "mxfp8_e5m2"
TYPES = {FP4: torch.uint8, E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
EMAX = {FP4: 2, E4M3: 8, E5M2: 15}
TOP = {FP4: 6.0, E4M3: 448.0, E5M2: 57344.0}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
HALF = 2.0 ** -8            # bf16: half a step, relative


def grid(quant):
    """The format's non-negative values, ascending: value i has code i."""
    if quant == FP4:
        return torch.tensor(E2M1, dtype=torch.float64)
    n = 0x7F if quant == E4M3 else 0x7C
    return torch.arange(n, dtype=torch.uint8).view(TYPES[quant]).double()


def codes_of(x, scale_code, quant):
    """Codes (one per value, sign above) of x [..., H] by given scales [..., H/32]: the nearest, ties to the even code."""
    g = grid(quant)
    two = torch.pow(torch.tensor(2.0, dtype=torch.float64), 127.0 - scale_code.double())
    z = x.double() * two.repeat_interleave(32, -1)
    a = z.abs().clamp(max=TOP[quant])
    i = torch.searchsorted(g, a).clamp(max=g.numel() - 1)            # g[i] >= a
    lo = (i - 1).clamp(min=0)
    below, above = a - g[lo], g[i] - a
    pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, i)
    return pick + torch.where(torch.signbit(z), 8 if quant == FP4 else 128, 0)


def scale_codes(x, quant):
    """e8m0 codes of the blocks of x [..., H]."""
    top = x.double().abs().unflatten(-1, (-1, 32)).amax(-1)
    e = torch.frexp(top)[1] - 1 - EMAX[quant]
    return torch.where(top > 0, e.clamp(-127, 127), -127) + 127


def pack(codes, quant):
    c = codes.to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4) if quant == FP4 else c.view(TYPES[quant])


def quantize(x, quant):
    s = scale_codes(x, quant)
    return pack(codes_of(x, s, quant), quant).contiguous(), s.to(torch.uint8).contiguous()


def values(codes, scales):
    """float64 values of codes (on the CPU)."""
    if codes.dtype == torch.bfloat16:
        return codes.double()
    if codes.dtype == torch.uint8:
        both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        v = torch.tensor(E2M1 + [-q for q in E2M1], dtype=torch.float64)[both.long()]
    else:
        v = codes.double()
    return v * torch.pow(torch.tensor(2.0, dtype=torch.float64), scales.double() - 127).repeat_interleave(32, -1)


def silu(a):
    return a / (1 + torch.exp(-a))


def steps(n):
    return (n + 8) * 2.0 ** -23


def lost(x, w, quant):
    """What the matrix unit drops of x [n, H] by w [O, H] with 8-bit x and 4-bit w.  It lines up the products of 8
    (e4m3) or 16 (e5m2) neighbouring channels, which share their scales, with the largest of them and cuts each off at
    u = 2^-13 of it.  A product has 4 + 2 (3 + 2) significant bits, its lowest at least 2^-5 (2^-4) of its leading one,
    so only one below 64 u (32 u) loses anything, and then less than u, and less than itself."""
    if quant not in (E4M3, E5M2):
        return 0.0
    n, bits = (8, 64.0) if quant == E4M3 else (16, 32.0)
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    a, b = x.abs().float().to(dev), w.abs().float().to(dev)
    H, O = x.shape[1], w.shape[0]
    rows = max(1, (1 << 27) // (O * H))
    out = []
    for i in range(0, x.shape[0], rows):
        t = (a[i:i + rows, None, :] * b[None]).view(-1, O, H // n, n)
        u = t.amax(-1, keepdim=True) * 2.0 ** -13
        out.append(torch.where(t < bits * u, torch.minimum(t, u), 0.0).sum((-1, -2)).double().cpu())
    return torch.cat(out) * (1 + 2.0 ** -12) if out else 0.0


def sums(x, w, quant=None):
    """x [n, H] by w [O, H]: values and how far fp32 sums may be off."""
    return x @ w.T, steps(x.shape[1]) * (x.abs() @ w.abs().T) + lost(x, w, quant)


def gated(a, da):
    """silu(a0) * a1 and its bound from the sums' (|silu'| < 1.1; the rest for the exponential and the products in fp32)."""
    (g, u), (dg, du) = a.chunk(2, -1), da.chunk(2, -1)
    h = silu(g) * u
    return h, 1.1 * dg * (u.abs() + du) + g.abs() * du + 2.0 ** -20 * h.abs()


def gated_grad(a, da, d):
    """The gradient of gated's sums, and its bound (|silu''| <= 0.5)."""
    (g, u), (dg, du) = a.chunk(2, -1), da.chunk(2, -1)
    s = 1 / (1 + torch.exp(-g))
    slope = s * (1 + g * (1 - s))
    out = torch.cat([d * u * slope, d * g * s], -1)
    off = torch.cat([d.abs() * (1.1 * du + 0.5 * dg * (u.abs() + du)), d.abs() * 1.1 * dg], -1)
    # sigmoid's own rounding meets 1 + g (1 - s), where it counts |g| times
    loose = torch.cat([(d * u).abs() * (1 + g.abs()), (d * g).abs()], -1)
    return out, off + 2.0 ** -20 * loose


def product(x, w, act, d=None, quant=None):
    """One expert's rows: y and its bound in fp32; with d the gradient and its bound, unrounded."""
    a, da = sums(x, w, quant)
    y, dy = gated(a, da) if act else (a, da)
    if d is None:
        return y, dy
    back, dback = d, torch.zeros_like(d)
    if act:
        back, dback = gated_grad(a, da, d)
        dback = dback + HALF * (back.abs() + dback)           # rounded to bf16 for its product
    dx, off = sums(back, w.T)
    return y, dy, dx, off * (1 + 2 * HALF) + dback @ w.abs()


def layer(x, idx, weights, up, down):
    """out [T, H] and its bound in fp32."""
    T, K = idx.shape
    E, out = up.shape[0], torch.zeros_like(x)
    off, mass = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(E):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        if t.numel() == 0:
            continue
        h, dh = product(x[t], up[e], True)
        dh = dh + 2.0 ** -16 * h.abs()
        y, dy = sums(h, down[e])
        dy = dy * (1 + 2.0 ** -15) + dh @ down[e].abs().T
        c = torch.ones(t.numel(), dtype=torch.float64) if weights is None else weights[t, k].double()
        out.index_add_(0, t, y * c[:, None])
        off.index_add_(0, t, dy * c.abs()[:, None])
        mass.index_add_(0, t, (y * c[:, None]).abs())
    return out, off + steps(K) * mass


def assert_close(got, want, off, what=""):
    """bf16 results within the bound and half a step; NaN fails."""
    got = got.double().cpu()
    tol = off + HALF * (want.abs() + off) + 1e-37
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:3].tolist(),
                           float(((got - want).abs() / tol).max()))
