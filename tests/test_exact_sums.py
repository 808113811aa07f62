"""The exact comparison of the GPU tests, on the host: it takes a right sum and
rejects one with a mistake in it, at the lengths where a bound that grows with
the length would not."""

import pytest
import torch

from exact_sums import operands, same, signs

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("dt", [BF, F16, F32])
@pytest.mark.parametrize("n", [12288, 262136, 1 << 24])
def test_mistakes_are_seen(n, dt):
    g = torch.Generator().manual_seed(n)
    m = 9
    a, b = (signs(g, min(0.6, 35 / n ** 0.5), s, torch.float64) for s in ((m, n), (n, 7)))
    ref = a @ b
    same(ref.to(F32).to(dt), ref, "itself")
    last = int((a[0] * b[:, 0]).nonzero()[-1])                # the last term that counts
    wrong = {"zeros": torch.zeros_like(ref), "half of the sum": a[:, :n // 2] @ b[:n // 2],
             "one split of sixteen lost": ref - a[:, :n // 16] @ b[:n // 16], "one split twice": ref + a[:, -n // 16:] @ b[-n // 16:]}
    less = ref.clone()
    less[0, 0] -= a[0, last] * b[last, 0]
    wrong["one term lost"] = less
    for name, value in wrong.items():
        with pytest.raises(AssertionError):
            same(value.to(F32).to(dt), ref, name)


def test_spread_of_the_outputs():
    # nearly all of them are held by bf16, and are not zero
    g = torch.Generator().manual_seed(1)
    X, W, b, R, dY = operands(g, 300, 4096, 520, BF)
    for p in (X.double() @ W.double(), dY.double() @ W.double().t(), X.double().t() @ dY.double()):
        assert 5 < p.std() < 50 and (p.abs() <= 256).double().mean() > 0.999
    assert b.abs().max() <= 3 and R.abs().max() <= 3 and set(X.unique().tolist()) == {-1, 0, 1}
