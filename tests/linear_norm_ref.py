"""Plain 64-bit definitions of the 16-bit linear and the layer normalisation,
and the error bounds of a 32-bit evaluation with 16-bit operands, for the
tests (torch, no code of the library)."""

import math

import torch

U32 = 2.0 ** -24   # half a step of fp32, relative
K = math.sqrt(2.0 / math.pi)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny_step(dtype):
    """Half of the smallest subnormal: the absolute rounding error near zero."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def act64(z, act):
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(K * (z + 0.044715 * z ** 3)))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z.clone()


def act_grad64(z, act):
    if act == "gelu_tanh":
        t = torch.tanh(K * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * K * (1 + 3 * 0.044715 * z * z)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def linear64(X, W, bias, residual, act):
    """(Y, Z, tolerance of Y in fp32, tolerance of Z in fp32).

    The K products are exact in fp32; each of at most K additions is off by one
    unit at most (2 U32: no assumption on the matrix unit's rounding).  The
    activations have slope below 1.2, and are evaluated as z times a factor in
    [0, 1] whose error is below 8 U32: its argument x is off by |x| U32, which
    a factor e^-|x| keeps below U32, and five operations add theirs."""
    x, w = X.double(), W.double()
    z = torch.mm(x, w)
    mag = torch.mm(x.abs(), w.abs())
    tz = 2 * X.shape[1] * U32 * mag
    if bias is not None:
        z = z + bias.double()
        tz = tz + U32 * z.abs() * 2
    y = act64(z, act)
    ty = 1.2 * tz + (8 * U32 * z.abs() if act != "identity" else 0)
    if residual is not None:
        y = y + residual.double()
        ty = ty + U32 * (y.abs() + ty)
    return y, z, ty, tz


def linear_backward64(dY, X, W, Z, act):
    """(dX, dW, db) and their tolerances before the last rounding.

    act' is below 1.2 and evaluated to 16 U32 (see linear64); dZ is rounded
    to X's type as an operand of the two products; the sums are bounded as
    in linear64."""
    h, tiny = half_step(X.dtype), tiny_step(X.dtype)
    x, w, dy = X.double(), W.double(), dY.double()
    dz = dy if act == "identity" else dy * act_grad64(Z.double(), act)
    ez = torch.zeros_like(dz) if act == "identity" else 17 * U32 * dy.abs()
    rounded = act != "identity" or dY.dtype != X.dtype
    ez2 = ez + (h * (dz.abs() + ez) + tiny if rounded else 0)
    wt, xt = w.t().contiguous(), x.t().contiguous()
    M, N = dY.shape
    dX = torch.mm(dz, wt)
    tX = torch.mm(ez2 + 2 * N * U32 * (dz.abs() + ez2), wt.abs())
    dW = torch.mm(xt, dz)
    tW = torch.mm(xt.abs(), ez2 + 2 * M * U32 * (dz.abs() + ez2))
    db = dz.sum(0)
    tb = (ez + 2 * M * U32 * (dz.abs() + ez)).sum(0)
    return (dX, dW, db), (tX, tW, tb)


def layer_norm64(x, w, b, eps):
    x = x.double()
    M = x.shape[0]
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if w is not None:
        y = y * w.double().reshape(-1, x.shape[1]).repeat_interleave(M // (w.numel() // x.shape[1]), 0)
    if b is not None:
        y = y + b.double().reshape(-1, x.shape[1]).repeat_interleave(M // (b.numel() // x.shape[1]), 0)
    return y, mean, rstd


def layer_norm_backward64(dy, x, mean, rstd, w, groups=1):
    dy, x = dy.double(), x.double()
    M, C = x.shape
    groups = groups if w is None else w.numel() // C
    xh = (x - mean.double()[:, None]) * rstd.double()[:, None]
    g = dy if w is None else dy * w.double().reshape(-1, C).repeat_interleave(M // groups, 0)
    dx = rstd.double()[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    dw = (dy * xh).reshape(groups, M // groups, C).sum(1)
    db = dy.reshape(groups, M // groups, C).sum(1)
    return dx, dw, db
