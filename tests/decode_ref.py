"""Plain 64-bit definitions of the layer with 16-bit activations, the 4-bit
cache and the attention over it, and bounds of the error of a 32-bit evaluation,
for the tests (torch, no code of the library)."""

import math

import torch

U32 = 2.0 ** -24   # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half of the smallest subnormal: the absolute rounding error near zero."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ the linear
def w4a16_64(X, codes, sw, lam, L1, L2, bias, residual, group, y_dtype):
    """(Y, tolerance after the store).

    The residual's product is taken as x (24 + code) less 24 sum x, both fp32
    sums of exact products: each of the K additions of either is off by one unit
    at most (2 U32) of at most 32 |x| times the scale.  With lambda, x is off by
    three roundings of fp32 and that of its fp16 terms: 2^-11 (one, for a bf16 Y)
    or 2^-22 of itself, not below 2^-37 of its group's largest; in the rank branch
    too.  Its codes are then subnormal numbers, of which the matrix unit keeps no
    more than 2^-24 of 2^-14 times the largest x: a term of the sum of the codes or of
    the constant, codes of 2^-24 (2^-18 against two terms), is cut at 2^-14
    (2^-20) of it."""
    x = X.double()
    ex, cut = torch.zeros_like(x), torch.zeros_like(x)
    M, K = x.shape
    if lam is not None:
        x = x / lam.double()
        top = x.abs().view(M, K // group, group).amax(2).repeat_interleave(group, 1)
        ex = x.abs() * (4 * U32 + (2.0 ** -11 if y_dtype == torch.bfloat16 else 2.0 ** -22)) + top * 2.0 ** -37
        cut = 2 * top * (2.0 ** -14 if y_dtype == torch.bfloat16 else 2.0 ** -20)
    ys, ts = [], []
    for b in range(codes.shape[0]):
        s = sw[b].double().repeat_interleave(group, 0)
        w = codes[b].double() * s
        y = torch.mm(x, w)
        t = torch.mm(ex, w.abs()) + torch.mm(cut, s) + 2 * (K + 4) * U32 * 2 * 32 * torch.mm(x.abs(), s)
        if L1 is not None:
            u = torch.mm(x, L1[b].double())
            au = torch.mm(x.abs(), L1[b].double().abs())
            y = y + torch.mm(u, L2[b].double())
            t = t + torch.mm(2 * (K + 4) * U32 * au + torch.mm(ex, L1[b].double().abs()), L2[b].double().abs())
            t = t + 2 * (L1.shape[2] + 1) * U32 * torch.mm(au, L2[b].double().abs())
        if bias is not None:
            y = y + bias[b].double()
        if residual is not None:
            y = y + residual[b].double()
            t = t + U32 * residual[b].double().abs()
        t = t + 3 * U32 * y.abs()
        ys.append(y)
        ts.append(t + half_step(y_dtype) * (y.abs() + t) + tiny(y_dtype))
    return torch.stack(ys), torch.stack(ts)


# ------------------------------------------------------------------ the cache
def held64(x, quant):
    """The values that the cache holds of x (T, H, D), fp64."""
    T, H, D = x.shape
    v = x.double().view(T, H, D // 64, 64)
    bad = ~torch.isfinite(v).all(-1, keepdim=True)
    v = torch.where(bad, torch.zeros_like(v), v)
    lo, hi = v.amin(-1, keepdim=True).clamp(max=0), v.amax(-1, keepdim=True).clamp(min=0)
    if quant == "asym":
        s = ((hi - lo) / 15).clamp(max=65504).half().double()
    else:
        s = (torch.maximum(hi, -lo) / 7).clamp(max=65504).half().double()
    d = torch.where(s == 0, torch.full_like(s, math.inf), s)
    if quant == "asym":
        z = torch.round(-lo / d).clamp(0, 15)
        n = (torch.round(v / d) + z).clamp(0, 15)
    else:
        z = torch.full_like(s, 8.0)
        n = torch.round(v / d).clamp(-8, 7) + 8
    out = s * (n - z)
    return torch.where(bad, torch.full_like(out, math.nan), out).view(T, H, D)


# ------------------------------------------------------------------ attention
def attention64(Q, k, v, ks, vs, pos, scale, causal, window, y_dtype):
    """One sequence: Q (n, Hq, D), the values held k, v (len, H, D) fp64, their
    scales ks, vs (len, H, D / 64), pos the position of the first query.

    Returns (y, lse, tolerance of y after the store, tolerance of lse).  With U
    half a unit: a group's score is the difference of two sums of 64 terms below
    31 |q|, each addition off by 2 U, then a few roundings; the codes are subnormal
    numbers, whose exponent the matrix unit takes to be that of 2^-14, so that 64
    terms and the sum before each instruction, 16 at most, are cut at 2^-20 of the
    largest |q| with codes of 2^-18; exp2's argument is off
    by U (4 |e| log2(e) + 64) and its result by two units (so eta, relative);
    p s is rounded to fp16 (2^-11) or to two (2^-21), not below 2^-32 of the row's
    largest; the sums over N tokens add 2 N U: of |v|, or, where the result has 16
    bits, of p s n and p s z apart, 30 p s in all; and their terms, N and an instruction's
    start every four, are cut likewise at 2^-14 (codes of 2^-24; 2^-20 where the result is
    fp32) of the largest p s."""
    n, Hq, D = Q.shape
    N, H, _ = k.shape
    G = D // 64
    q = Q.double()
    dev = Q.device
    t = torch.arange(N, device=dev)[None]
    i = torch.arange(n, device=dev)[:, None] + pos
    seen = (t <= i) if causal else torch.ones(n, N, dtype=torch.bool, device=dev)
    if window:
        seen = seen & (t > i - window)
    y = torch.zeros(n, Hq, D, dtype=torch.float64, device=dev)
    ty = torch.zeros_like(y)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=dev)
    tl = torch.zeros_like(lse)
    h = 2.0 ** -21 if y_dtype == torch.float32 else 2.0 ** -11
    unit = 2.0 ** -20 if y_dtype == torch.float32 else 2.0 ** -14
    if N == 0:
        return y, lse, ty, tl
    for hq in range(Hq):
        hk = hq // (Hq // H)
        e = scale * torch.mm(q[:, hq], k[:, hk].t().contiguous())
        e = torch.where(seen, e, torch.full_like(e, -math.inf))
        some = seen.any(1)
        top = torch.where(some, e.amax(1), torch.zeros(n, dtype=torch.float64, device=dev))
        p = torch.exp(e - top[:, None])
        tot = p.sum(1, keepdim=True)
        div = torch.where(tot > 0, tot, torch.ones_like(tot))
        vh = torch.where(seen.any(0)[:, None], v[:, hk], torch.zeros_like(v[:, hk]))   # what no row sees is not there
        yy = torch.mm(p, vh) / div
        aa = torch.mm(p, vh.abs()) / div
        a = q[:, hq].abs().view(n, G, 64).sum(2)
        most = q[:, hq].abs().view(n, G, 64).amax(2)
        de = scale * torch.mm(31 * 264 * U32 * a + 80 * 2.0 ** -20 * most, ks[:, hk].double().t().contiguous())
        de = torch.where(seen, de, torch.zeros_like(de)).amax(1, keepdim=True)
        big = torch.where(seen, e.abs(), torch.zeros_like(e)).amax(1, keepdim=True)
        eta = de + U32 * (4 * 1.45 * big + 64) * 0.7 + 8 * U32
        ps = p[:, :, None] * vs[None, :, hk].double()                                 # n, N, G
        cut = unit * ps.amax(1, keepdim=True)
        cut = 2 * (torch.minimum(15 * ps, cut).sum(1) + (N / 4 + 8) * cut[:, 0]) / div
        cut = cut.repeat_interleave(64, 1)
        ps = ps.amax(1)                                                               # n, G
        floor = (15 * N * 2.0 ** -32 * ps / div).repeat_interleave(64, 1)
        apart = 0.0
        if y_dtype != torch.float32:
            sums = (torch.mm(p, vs[:, hk].double()) / div).repeat_interleave(64, 1)
            apart = 30 * sums * 2 * (N + 64) * U32
        t1 = aa * (eta + h + 2 * (N + 64) * U32) + apart + yy.abs() * (eta + 2 * (N + 64) * U32 + 8 * U32) + floor + cut
        y[:, hq] = yy
        ty[:, hq] = t1 + half_step(y_dtype) * (yy.abs() + t1) + tiny(y_dtype)
        l = torch.log(tot[:, 0]) + top
        lse[:, hq] = torch.where(some, l, torch.full_like(l, -math.inf))
        tl[:, hq] = eta[:, 0] + 2 * (N + 64) * U32 + 4 * U32 * (l.abs() + 64)
    return y, lse, ty, tl


def scales64(x, quant):
    T, H, D = x.shape
    v = x.double().view(T, H, D // 64, 64)
    if quant == "asym":
        return ((v.amax(-1).clamp(min=0) - v.amin(-1).clamp(max=0)) / 15).clamp(max=65504).half().double()
    return (v.abs().amax(-1) / 7).clamp(max=65504).half().double()
