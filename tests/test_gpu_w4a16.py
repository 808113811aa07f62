"""The layer with 16-bit activations: element by element against 64 bits within
derived bounds, and sums that come out exact, so that every output of every shape
has one right value."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from decode_ref import w4a16_64  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def layer(M, K, N, batch, group, r, dt, smooth, bias, residual, ydt, seed=1):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(M, K, generator=g) * (0.3 + torch.rand(K, generator=g))
    X[:, :: max(1, K // 5)] *= 8
    s = dict(X=X.to(DT[dt]), codes=torch.randint(-8, 8, (batch, K, N), generator=g, dtype=torch.int8),
             sw=(0.02 * (0.5 + torch.rand(batch, K // group, N, generator=g))).half(),
             lam=(0.25 + 3 * torch.rand(K, generator=g)).half() if smooth else None,
             L1=(torch.randn(batch, K, r, generator=g) / math.sqrt(K)).to(DT[dt]) if r else None,
             L2=torch.randn(batch, r, N, generator=g).to(DT[dt]) if r else None,
             bias=torch.randn(batch, N, generator=g).to(DT[dt]) if bias else None,
             residual=torch.randn(batch, M, N, generator=g).to(DT[ydt]) if residual else None)
    return {k: None if v is None else v.to(DEV) for k, v in s.items()}


def call(s, group, ydt, **kw):
    batch, K, N = s["codes"].shape
    packed = torch.cat([hsq.pack_weights(c)[0] for c in s["codes"]])
    return hsq.w4a16_lowrank_linear(s["X"], packed, s["sw"], s["lam"], s["L1"], s["L2"], s["bias"], s["residual"], N=N,
                                    batch=batch, group=group, y_dtype=ydt, **kw)


SHAPES = [
    # M, K, N, batch, group, r
    (1, 64, 1, 1, 64, 0), (1, 64, 16, 1, 64, 1), (1, 128, 17, 1, 128, 4), (2, 192, 33, 1, 64, 0),
    (3, 320, 100, 2, 64, 5), (1, 4096, 1024, 1, 64, 16), (16, 4096, 256, 1, 128, 4), (15, 1088, 77, 3, 64, 32),
    (17, 640, 130, 1, 64, 3), (33, 1152, 48, 1, 128, 8), (31, 576, 65, 2, 64, 0), (48, 512, 31, 1, 64, 7),
    (49, 448, 97, 1, 64, 1), (64, 1024, 160, 2, 128, 32), (64, 12288, 16, 1, 64, 4), (1, 12288, 9000, 1, 64, 0),
    (5, 128, 9001, 1, 64, 2), (64, 64, 15, 1, 64, 31), (4, 2112, 8200, 1, 64, 0),
    # up to four rows: U in the same launch with 2, 3 and 4 column tiles, in one before it,
    # no room for xh in LDS, too many columns
    (1, 128, 8000, 1, 64, 8), (2, 192, 12000, 1, 64, 3), (1, 256, 4000, 3, 128, 16), (1, 4096, 100, 2, 64, 32),
    (2, 8320, 40, 1, 64, 16), (4, 12288, 33, 1, 64, 7), (3, 256, 12000, 1, 128, 4), (4, 128, 4096, 1, 64, 32),
]


@pytest.mark.parametrize("dt,ydt", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_against_64_bits(shape, smooth, dt, ydt):
    M, K, N, batch, group, r = shape
    print(f"[w4a16] {shape} smooth={smooth} {dt} {ydt}", flush=True)
    s = layer(M, K, N, batch, group, r, dt, smooth, N % 2 == 1, M % 2 == 0 or N == 17, ydt)
    y = call(s, group, ydt).double()
    want, tol = w4a16_64(s["X"], s["codes"], s["sw"], s["lam"], s["L1"], s["L2"], s["bias"], s["residual"], group,
                         DT[ydt])
    assert bool(((y - want).abs() <= tol).all()), ((y - want).abs() / tol).max().item()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("smooth", [False, True])
def test_exact_sums(shape, smooth):
    # x in {-1, 0, 1} / lambda in {1/2, 1, 2}, scales 1 and 1/2, small factors: every partial
    # sum is a multiple of 2^-2 below 2^22
    M, K, N, batch, group, r = shape
    g = torch.Generator().manual_seed(5)
    pick = lambda vals, *sh: torch.tensor(vals)[torch.randint(0, len(vals), sh, generator=g)]  # noqa: E731
    s = dict(X=pick([-1.0, 0.0, 0.0, 1.0], M, K).bfloat16(), lam=pick([0.5, 1.0, 2.0], K).half() if smooth else None,
             codes=torch.randint(-8, 8, (batch, K, N), generator=g, dtype=torch.int8),
             sw=pick([0.5, 1.0], batch, K // group, N).half(),
             L1=pick([-1.0, 0.0, 0.0, 0.0, 1.0], batch, K, r).bfloat16() if r else None,
             L2=pick([-1.0, 0.0, 0.0, 1.0], batch, r, N).bfloat16() if r else None,
             bias=pick([-3.0, 2.0], batch, N).bfloat16(), residual=pick([-7.0, 5.0], batch, M, N))
    s = {k: None if v is None else v.to(DEV) for k, v in s.items()}
    y = call(s, group, "f32").double()
    x = s["X"].double() / (s["lam"].double() if smooth else 1.0)
    for b in range(batch):
        want = torch.mm(x, s["codes"][b].double() * s["sw"][b].double().repeat_interleave(group, 0))
        if r:
            want = want + torch.mm(torch.mm(x, s["L1"][b].double()), s["L2"][b].double())
        want = want + s["bias"][b].double() + s["residual"][b].double()
        assert torch.equal(y[b], want)


def test_every_code_and_column_in_its_place():
    # one channel at a time: Y row m is the dequantized weight's row k
    K, N = 256, 70
    g = torch.Generator().manual_seed(6)
    codes = torch.randint(-8, 8, (1, K, N), generator=g, dtype=torch.int8).to(DEV)
    sw = (0.5 + torch.rand(1, K // 64, N, generator=g)).half().to(DEV)
    packed = hsq.pack_weights(codes[0])[0]
    for dt in (torch.bfloat16, torch.float16):
        for k0 in range(0, K, 64):
            X = torch.zeros(64, K, dtype=dt, device=DEV)
            X[torch.arange(64), torch.arange(k0, k0 + 64)] = 1.0
            y = hsq.w4a16_lowrank_linear(X, packed, sw, N=N, y_dtype="f32")
            assert torch.equal(y[0].double(), codes[0, k0:k0 + 64].double() * sw[0, k0 // 64].double())


def test_ranges():
    # tiny and large activations, lambdas that move them far, and rows that are not finite
    K, N = 192, 40
    for dt, top in (("bf16", 1e30), ("f16", 6e4)):
        s = layer(6, K, N, 1, 64, 3, dt, True, True, False, "f32", seed=9)
        X = s["X"].float()
        X[0] *= top / X[0].abs().max()
        X[1] *= 1e-7 / X[1].abs().max()
        X[2] = 0.0
        X[3, 64:128] *= 1e-6
        s["X"] = X.to(DT[dt])
        s["lam"] = torch.where(torch.rand(K) < 0.3, 6e-4, 40.0).half().to(DEV)
        y = call(s, 64, "f32")
        want, tol = w4a16_64(s["X"], s["codes"], s["sw"], s["lam"], s["L1"], s["L2"], s["bias"], None, 64, DT["f32"])
        assert bool(((y.double() - want).abs() <= tol).all())
        for bad in (math.nan, math.inf, -math.inf):
            for smooth in (True, False):
                s2 = dict(s, X=s["X"].clone())
                s2["X"][4, 7] = bad
                if not smooth:
                    s2["lam"] = None
                a = call(s2, 64, "f32")
                b = call(dict(s, lam=s2["lam"]), 64, "f32")
                assert bool(torch.isnan(a[0, 4]).all())
                keep = [0, 1, 2, 3, 5]
                assert torch.equal(a[0, keep], b[0, keep])


def test_residual_in_place_and_same_bits():
    s = layer(16, 1024, 300, 2, 64, 4, "bf16", True, True, True, "f32")
    y = call(s, 64, "f32")
    for _ in range(3):
        assert torch.equal(call(s, 64, "f32"), y)
    out = s["residual"].clone()
    got = call(dict(s, residual=out), 64, "f32", out=out)
    assert got is out and torch.equal(out, y)
    # the workspace's contents do not matter
    need = hsq.w4a16_workspace_bytes(16, 1024, 300, 4, 2, 64, True, "f32")
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    assert torch.equal(call(s, 64, "f32", workspace=ws[:need]), y) and bool((ws[need:] == 0xFF).all())


def test_layer_object_weight_only():
    g = torch.Generator().manual_seed(12)
    K, N, r = 512, 96, 4
    qw = torch.randint(-7, 8, (1, K, N), generator=g, dtype=torch.int8).to(DEV)
    sw = (0.01 + 0.01 * torch.rand(1, K // 64, N, generator=g)).half().to(DEV)
    lam = (0.5 + torch.rand(K, generator=g)).half().to(DEV)
    L1 = (0.05 * torch.randn(1, K, r, generator=g)).bfloat16().to(DEV)
    L2 = torch.randn(1, r, N, generator=g).bfloat16().to(DEV)
    X = torch.randn(5, K, generator=g).bfloat16().to(DEV)
    lay = hsq.Layer(lam, qw, sw, L1, L2, max_tokens=64)
    y = lay(X, "f32", weight_only=True)
    want, tol = w4a16_64(X, qw, sw, lam, L1, L2, None, None, 64, torch.float32)
    assert bool(((y.double() - want).abs() <= tol).all())
    # the quantized form of the same layer: 4-bit activations, a few percent away
    q = lay(X, "f32")
    assert float((q.double() - want).norm() / want.norm()) < 0.15


@pytest.mark.parametrize("M", [1, 3, 16, 40])
@pytest.mark.parametrize("smooth", [False, True])
def test_small_channels_count_beside_a_large_one(M, smooth):
    # one channel of 1 in each group and the others 2^-19, codes 7 against -8: an fp32 result
    # holds them.  The sums of the codes and of the constant cut their terms, 64 and 64 of two
    # parts each, at 2^-20 of the largest product's unit
    K, N = 256, 48
    X = torch.full((M, K), 2.0 ** -19)
    X[:, ::64] = 1.0
    codes = torch.full((1, K, N), 7, dtype=torch.int8)
    codes[:, ::64] = -8
    s = dict(X=X.bfloat16(), codes=codes, sw=torch.ones(1, K // 64, N).half(), lam=torch.ones(K).half() if smooth else None,
             L1=None, L2=None, bias=None, residual=None)
    s = {k: None if v is None else v.to(DEV) for k, v in s.items()}
    y = call(s, 64, "f32").double()
    want = 4 * (-8 + 63 * 7 * 2.0 ** -19)
    assert bool(((y - want).abs() <= 4 * 256 * 2.0 ** -20).all()), (y - want).abs().max().item()
