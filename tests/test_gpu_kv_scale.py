"""The scale of a group of the 4-bit cache is the real quotient rounded once, where
two roundings would end elsewhere."""

from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from test_gpu_kv_cache import DEV, DT, i32, pages_for  # noqa: E402


def to_half(q):
    """A real number to fp16, ties to even (torch's own cast of fp64 goes through fp32)."""
    h = np.float16(float(q))
    near = [np.nextafter(h, np.float16(-np.inf)), h, np.nextafter(h, np.float16(np.inf))]
    return min(near, key=lambda c: (abs(Fraction(float(c)) - q), int(c.view(np.uint16)) & 1))


def held(x):
    """What an asymmetric group holds of x (floats), in real numbers."""
    x = [Fraction(v) for v in x]
    lo, hi = min(0, *x), max(0, *x)
    s = Fraction(float(to_half((hi - lo) / 15)))
    if s == 0:
        return [0.0] * len(x)
    z = min(max(round(-lo / s), 0), 15)
    return [float(s * (min(max(round(v / s) + z, 0), 15) - z)) for v in x]


def near_ties():
    """(hi, lo) of fp16 whose range is next to 15 times the middle of two fp16 numbers."""
    out = [(1.888671875, -1023 * 2.0 ** -24)]
    for e in (-14, -9, -1, 0, 1):
        for m in range(1024, 2048, 7):
            wide = 15 * Fraction(2 * m + 1, 2048) * Fraction(2) ** e
            for hi in {np.float16(float(wide)), np.nextafter(np.float16(float(wide)), np.float16(0))}:
                rest = wide - Fraction(float(hi))
                for j in (-2, -1, 0, 1, 2):
                    lo = rest + Fraction(j, 2 ** 24)
                    if lo > 0 and Fraction(float(np.float16(float(lo)))) == lo:
                        out.append((float(hi), -float(lo)))
    return out


# of bf16: the middles of subnormal scales, and a low end that fp32 loses beside the high one
BF16_TIES = [(15 * k * 2.0 ** -25, -(2.0 ** -e)) for k in (1, 3, 5, 9, 17) for e in (40, 49, 50, 60, 100)]


@pytest.mark.parametrize("dt,pairs", [("f16", near_ties()), ("bf16", BF16_TIES)], ids=["f16", "bf16"])
@pytest.mark.parametrize("sign", [1, -1])
def test_scale_is_rounded_once(dt, pairs, sign):
    T, D = len(pairs), 64
    x = np.zeros((T, D))
    for t, (hi, lo) in enumerate(pairs):
        x[t] = np.linspace(lo, hi, D)
        x[t, 5], x[t, 40] = hi, lo
    x = torch.from_numpy(sign * x).to(DT[dt])
    assert all(float(x[t, 5]) == sign * hi and float(x[t, 40]) == sign * lo for t, (hi, lo) in enumerate(pairs))
    k = x[:, None].to(DEV)
    table, n = pages_for([T], 32)
    cache = hsq.kv_cache(n, 1, D, 32)
    hsq.kv_cache_write(k, k, cache, table, i32(T))
    a, b = hsq.kv_cache_read(cache, table, i32(T), tokens=T, head_dim=D, dtype="f32")
    want = torch.tensor([held(row) for row in x.double().tolist()], dtype=torch.float64, device=DEV)
    bad = (a[:, 0].double() != want).any(1)
    assert torch.equal(a, b)
    assert not bad.any(), (int(bad.sum()), T, pairs[int(bad.nonzero()[0])])
