"""Operands whose sums come out exact in fp32, so that a test needs no tolerance.

The values are -1, 0 and 1: products and sums are whole numbers below 2^24,
which fp32 holds whatever the order.  The share of zeros keeps the spread of
an output at 35 at most, so that 16 bits hold nearly all outputs too (bf16 up to
256): a lost or doubled term shows, however long the reduction.  An output
that 16 bits do not hold has one rounding."""

import torch


def signs(g, share, shape, dt):
    """-1 and 1 with probability share / 2 each, otherwise 0."""
    u = torch.rand(shape, generator=g, device=g.device, dtype=torch.float32)
    return (u < share / 2).to(dt) - (u > 1 - share / 2).to(dt)


def operands(g, M, K, N, dt):
    """X, W, bias, residual and dY of a linear layer.  A sum of n products has the
    spread sqrt(n times the shares of both operands)."""
    def operand(m, n, longest):
        return signs(g, 1.0 if m * n < 64 else min(0.6, 35 / longest ** 0.5), (m, n), dt)

    X, W, dY = operand(M, K, max(M, K)), operand(K, N, max(K, N)), operand(M, N, max(M, N))
    b, R = (torch.randint(-3, 4, s, generator=g, device=g.device).to(dt) for s in ((N,), (M, N)))
    return X, W, b, R, dY


def same(got, ref, what):
    """ref in 64 bits: whole numbers below 2^24."""
    assert ref.abs().max() < 2 ** 24
    want = ref.to(torch.float32).to(got.dtype)
    bad = got != want
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}, "
                           f"got {got[bad][0].item()}, want {want[bad][0].item()}")
