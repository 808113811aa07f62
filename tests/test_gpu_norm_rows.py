"""The norm's forward pass where a workgroup goes from row to row: two turns and
a part of one for every width of the kernel, groups that change on the way, and
rows of one value."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from linear_norm_ref import layer_norm64  # noqa: E402
from test_gpu_layer_norm import BF, DEV, F16, F32, NAME, close, forward_bound, make, say  # noqa: E402

# Rows of a turn: 512 above 4096 channels (a workgroup of eight waves each), 1024
# above 1536 (four waves), 4096 below (four rows to a workgroup).
ROWS = [
    (1100, 4100, 11, F32, F32, F32),
    (1089, 8192, 1, BF, BF, BF),
    (1100, 8191, 5, F16, F16, F16),
    (1025, 8200, 5, F32, BF, F32),
    (1300, 12288, 13, F32, F32, F32),
    (1100, 12281, 4, BF, BF, F32),
    (1030, 12296, 10, F32, F16, F16),
    (1027, 16384, 1, BF, BF, F32),
    (2100, 2048, 7, F32, F32, F32),
    (2301, 4096, 3, F16, F16, F32),
    (8200, 512, 8, BF, BF, BF),
    (9001, 1000, 1, F32, BF, F32),
    (8203, 1536, 13, F16, F16, F16),
]


@pytest.mark.parametrize("M,C,G,xdt,ydt,pdt", ROWS)
def test_rows_in_turn(M, C, G, xdt, ydt, pdt):
    say(f"[norm turns] M={M} C={C} groups={G} {xdt} {ydt} {pdt}")
    X, w, b, _ = make(M + 3 * C, M, C, G, xdt, ydt, pdt)
    eps = 1e-6
    y, mean, rstd = hsq.layer_norm(X, w, b, eps=eps, y_dtype=NAME[ydt], return_stats=True)
    ry, rm, rr = layer_norm64(X, w, b, eps)
    ty, tm, tr = forward_bound(X, w, b, ry, rm, rr, eps)
    close(y, ry, ty, ydt, "Y")
    close(mean, rm, tm, F32, "mean")
    close(rstd, rr, tr, F32, "rstd")
    # a row's bits depend on the row alone: the same ones in a launch without a second turn
    n = M // G
    step = 300 if G == 1 else max(n, 300) // n * n
    for lo in range(0, M, step):
        part = slice(lo, min(M, lo + step))
        params = (w, b) if G == 1 else (t[lo // n:part.stop // n].clone() for t in (w, b))
        assert torch.equal(hsq.layer_norm(X[part].clone(), *params, eps=eps, y_dtype=NAME[ydt]), y[part])
    if xdt == ydt:
        assert torch.equal(hsq.layer_norm(X, w, b, eps=eps, out=X), y)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("C", [1, 9, 512, 700, 1024, 1152, 1537, 2240, 4096, 6000, 8192, 9000, 12288, 16384])
def test_rows_of_one_value(C, dt):
    """A row of one power of two: its sum, its mean, and so the differences are
    exact, and y is the bias.  Other values: within the bound of the mean's error,
    which the rstd of 1 / sqrt(eps) magnifies."""
    say(f"[norm constant] C={C} {dt}")
    M = 5
    _, w, b, _ = make(C, M, C, 1, F32, F32, F32)
    value = torch.tensor([4.0, -0.5, 0.0, 1024.0, 2.0 ** -20], device=DEV)
    X = value[:, None].expand(M, C).to(dt).contiguous()
    y, mean, rstd = hsq.layer_norm(X, w, b, eps=1e-6, y_dtype=NAME[dt], return_stats=True)
    assert torch.equal(mean, value) and torch.equal(y, b.to(dt).expand(M, C))
    X = torch.tensor([0.1, -3.3, 7.7, 1e-3, 1e3], device=DEV)[:, None].expand(M, C).to(dt).contiguous()
    y, mean, rstd = hsq.layer_norm(X, w, b, eps=1e-2, y_dtype=NAME[dt], return_stats=True)
    ry, rm, rr = layer_norm64(X, w, b, 1e-2)
    ty, tm, tr = forward_bound(X, w, b, ry, rm, rr, 1e-2)
    close(y, ry, ty, dt, "Y")
    close(mean, rm, tm, F32, "mean")
    close(rstd, rr, tr, F32, "rstd")


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("C", [64, 1152, 4096, 16384])
def test_rows_beyond_the_range_of_their_squares(C, dt):
    """Rows of +-2^k: mean 0 and variance 2^2k, whose sum of C leaves fp32 from
    C 2^2k = 2^128 on.  Then rstd is 0 and y the bias; below, y is w + b or b - w."""
    say(f"[norm large values] C={C} {dt}")
    _, w, b, _ = make(C, 2, C, 1, F32, F32, F32)
    sign = torch.ones(C, device=DEV)
    sign[1::2] = -1
    held, beyond = 2.0 ** 56, 2.0 ** 64
    X = torch.stack([sign * held, sign * beyond, -sign * held]).to(dt)
    y, mean, rstd = hsq.layer_norm(X, w, b, eps=1e-6, y_dtype=NAME[dt], return_stats=True)
    assert not mean.any() and rstd.tolist() == [1 / held, 0.0, 1 / held]
    for row, s in ((0, sign), (1, torch.zeros_like(sign)), (2, -sign)):
        assert torch.equal(y[row], (s * w + b).to(dt))
