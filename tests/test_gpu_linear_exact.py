"""Sums of the 16-bit linear and of the norm's parameter gradients that come out
exact (exact_sums): every output has one right value, however long the reduction."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from exact_sums import operands, same, signs  # noqa: E402
from linear_cases import DEEP, units  # noqa: E402
from test_gpu_linear import BACKWARD, FORWARD, LARGE  # noqa: E402

DEV = torch.device("cuda:0")
BF, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
DEPTHS = [(1, 4096, 12288), (16, 12288, 4096), (64, 12288, 4096), (200, 12288, 520)]


def say(msg):
    print(msg, flush=True)


def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def forward(M, K, N, dt, seed):
    X, W, b, R, _ = operands(generator(seed), M, K, N, dt)
    z = torch.mm(X.double(), W.double()) + b.double()
    if M * N > 64:
        assert (z != 0).any()              # an output of zeros is wrong
    Y, Z = hsq.linear(X, W, b, R.float(), y_dtype="f32", return_preact=True)
    same(Y, z + R.double(), "Y")
    same(Z, z, "Z")
    same(hsq.linear(X, W), z - b.double(), "Y without its bias")


def backward(M, K, N, dt, seed):
    X, W, _, _, dY = operands(generator(seed), M, K, N, dt)
    dX, dW, db = hsq.linear_backward(dY, X, W)
    rX = torch.mm(dY.double(), W.double().t().contiguous())
    rW = torch.mm(X.double().t().contiguous(), dY.double())
    if M * N > 64:
        assert (rX != 0).any() and (rW != 0).any()
    for got, ref, what in ((dX, rX, "dX"), (dW, rW, "dW"), (db, dY.sum(0, dtype=F64), "db")):
        same(got, ref, what)
    # dY in fp32, whose dZ is formed by a pass of its own; the products launched apart
    same(hsq.linear_backward(dY.float(), X, W, need_weight=False, need_bias=False)[0], rX, "dX from fp32")
    same(hsq.linear_backward(dY.float(), X, W, need_input=False, need_bias=False)[1], rW, "dW from fp32")


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("M,K,N,product,tiles", DEEP)
def test_every_kind_of_tile(M, K, N, product, tiles, dt):
    assert units(M, K, N, product)[0] == tiles
    say(f"[exact] {product} {tiles}: M={M} K={K} N={N} {dt}")
    (forward if product == "fwd" else backward)(M, K, N, dt, M + K + N)


@pytest.mark.parametrize("M,K,N,dt", [c[:4] for c in FORWARD] + [(*s, BF) for s in DEPTHS])
def test_forward(M, K, N, dt):
    say(f"[exact forward] M={M} K={K} N={N} {dt}")
    forward(M, K, N, dt, 2 * M + K + N)


@pytest.mark.parametrize("M,K,N,dt", [c[:4] for c in BACKWARD] + [(*s, BF) for s in DEPTHS])
def test_backward(M, K, N, dt):
    say(f"[exact backward] M={M} K={K} N={N} {dt}")
    backward(M, K, N, dt, 3 * M + K + N)


@pytest.mark.parametrize("act", ["identity", "silu"])
def test_range_of_an_fp16_dz(act):
    """dZ is an fp16 operand of dX and dW, whatever dY's type: what lies outside
    fp16 is lost there, not in dbias, and a loss scaled by a power of two brings
    it back."""
    say(f"[fp16 dZ] {act}")
    M, K, N = 4096, 96, 136
    X, W, _, _, dY = operands(generator(3), M, K, N, F16)
    Z = torch.full((M, N), 100.0, device=DEV, dtype=F16)    # silu' = 1 there, to within 2^-80

    def grads(scale):
        return hsq.linear_backward(dY.float() * scale, X, W, Z, act=act)

    def check(got, scale):
        for t, ref in zip(got, (dY.double() @ W.double().t().contiguous(), X.double().t().contiguous() @ dY.double(),
                                dY.sum(0, dtype=F64))):
            assert (ref != 0).any() and torch.equal(t, (ref * scale).to(F32).to(F16))

    check(grads(1.0), 1.0)
    check(grads(2.0 ** -14), 2.0 ** -14)                     # the least normal value
    check(grads(2.0 ** -24), 2.0 ** -24)                     # the least subnormal one
    dX, dW, db = grads(2.0 ** -25)                           # half of it: to even, zero
    assert not dX.any() and not dW.any()
    same(db.double() * 2.0 ** 24, (dY.sum(0, dtype=F64) / 2).round(), "db")
    dX, dW, db = grads(65536.0)
    # every term of a hit row or column is an infinity or NaN
    assert not torch.isfinite(dX[(dY != 0).any(1)]).any() and not torch.isfinite(dW[:, (dY != 0).any(0)]).any()


@pytest.mark.parametrize("M,K,N", LARGE)
def test_longest_sums(M, K, N):
    """Every output through its row and column sums, some rows and columns one by
    one."""
    say(f"[exact large] M={M} K={K} N={N}")
    X, W, _, _, dY = operands(generator(9), M, K, N, F16)       # fp16 holds whole numbers up to 2048
    rows, mid, cols = ([*range(0, n, max(1, n // 20)), n - 1] for n in (M, K, N))

    def sums(got, left, right, what):
        """got = left right, one factor at a time."""
        assert got.abs().max() <= 2048 and (got != 0).any()
        assert torch.equal(got.sum(0, dtype=F64), left.sum(0, dtype=F64) @ right.double()), what
        assert torch.equal(got.sum(1, dtype=F64), left.double() @ right.sum(1, dtype=F64)), what

    Y = hsq.linear(X, W, y_dtype="f32")
    same(Y[rows][:, cols], X[rows].double() @ W[:, cols].double().contiguous(), "Y")
    sums(Y, X, W, "Y")
    del Y
    dX, dW, db = hsq.linear_backward(dY, X, W)
    same(dX[rows][:, mid], dY[rows].double() @ W[mid].double().t().contiguous(), "dX")
    same(dW[mid][:, cols], X[:, mid].double().t().contiguous() @ dY[:, cols].double().contiguous(), "dW")
    same(db, dY.sum(0, dtype=F64), "db")
    sums(dX, dY, W.t(), "dX")
    sums(dW, X.t(), dY, "dW")


@pytest.mark.parametrize("M,K,N", [(1, 3, 1 << 24), (1, 1 << 24, 3), (60, (1 << 24) - 8, 3), (60, 3, (1 << 24) - 8)])
def test_widest_rows(M, K, N):
    say(f"[exact wide] M={M} K={K} N={N}")
    X, W, b, _, dY = operands(generator(13), M, K, N, F16)
    z = X.double() @ W.double()
    assert (z != 0).any()
    same(hsq.linear(X, W, b, y_dtype="f32"), z + b.double(), "Y")
    dX, dW, db = hsq.linear_backward(dY, X, W)
    same(dX, dY.double() @ W.double().t().contiguous(), "dX")
    same(dW, X.double().t().contiguous() @ dY.double(), "dW")
    same(db, dY.sum(0, dtype=F64), "db")


@pytest.mark.parametrize("M,C,G", [(1 << 25, 61, 1), (1 << 25, 61, 64), (131071, 16384, 1), (70000, 1152, 7),
                                   (5000, 2241, 1), (4096, 9000, 4)])
def test_parameter_gradients_of_the_norm(M, C, G):
    # mean 0 and rstd 1 given: xh = x, so that dy xh is whole too
    say(f"[exact norm] M={M} C={C} groups={G}")
    g = generator(6)
    n = M // G
    X, dY = (signs(g, min(0.6, 35 / n ** 0.5), (M, C), BF) for _ in range(2))
    dw = (dY * X).view(G, n, C).sum(1, dtype=F64)
    assert (dw != 0).any()
    stats = torch.zeros(M, device=DEV), torch.ones(M, device=DEV)
    got = hsq.layer_norm_backward(dY, X, *stats, groups=G, need_input=False)
    same(got[1], dw, "dw")
    same(got[2], dY.view(G, n, C).sum(1, dtype=F64), "db")
