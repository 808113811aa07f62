"""Layer normalisation and its backward pass on the GPU against the 64-bit
definition, element by element within derived bounds, and the norm, the 16-bit
linear and the W4A4 layer run together as a transformer's MLP."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from linear_norm_ref import (U32, act64, act_grad64, half_step, layer_norm64, layer_norm_backward64,  # noqa: E402
                             tiny_step)

DEV = torch.device("cuda:0")
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAME = {BF: "bf16", F16: "f16", F32: "f32"}
# additions on the way to a row's sum: at most 32 in a lane, 6 across a wave, 8 across waves
DEPTH = 46


def say(msg):
    print(msg, flush=True)


def close(got, ref, tol, dt, what):
    lim = tol + half_step(dt) * (ref.abs() + tol) + tiny_step(dt)
    bad = ~((got.double() - ref).abs() <= lim)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}, got "
                           f"{got[bad][0].item()}, want {ref[bad][0].item()}, limit {lim[bad][0].item()}")


def make(seed, M, C, G, xdt, ydt, pdt, offset=0.5):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, generator=g, device=DEV)

    X = (rnd(M, C) * (0.5 + torch.rand(C, generator=g, device=DEV)) + offset * rnd(M, 1)).to(xdt)
    w = b = None
    if pdt is not None:
        shape = (C,) if G == 1 else (G, C)
        w, b = (1 + 0.3 * rnd(*shape)).to(pdt), (0.3 * rnd(*shape)).to(pdt)
    return X, w, b, rnd(M, C).to(ydt)


def forward_bound(X, w, b, y, mean, rstd, eps):
    """Tolerances of y (before its rounding), mean and rstd.

    The mean of DEPTH rounded additions is off by DEPTH U32 of the mean
    magnitude (plus its division); x - mean and the product round once each;
    the variance's own sum gives rstd (DEPTH + 4) / 2 U32 relative, and the
    mean's error e adds e^2 / var to it."""
    x = X.double()
    C = x.shape[1]
    em = (DEPTH + 1) * U32 * x.abs().mean(1) + U32 * mean.abs()
    er = rstd * ((DEPTH + 8) * U32 + (em * rstd) ** 2)
    d = (x - mean[:, None]).abs()
    M = x.shape[0]
    W = torch.ones_like(x) if w is None else w.double().reshape(-1, C).repeat_interleave(M // (w.numel() // C), 0).abs()
    ty = W * ((em[:, None] + U32 * d) * (rstd + er)[:, None] + d * (er + 4 * U32 * rstd)[:, None])
    return ty + U32 * 2 * y.abs(), em, er + U32 * rstd


CASES = [
    # M, C, groups, X, Y, parameters
    (1, 1, 1, BF, BF, BF),
    (1, 4096, 1, BF, BF, BF),
    (3, 7, 3, F16, F16, F32),
    (5, 64, 1, F32, F32, F32),
    (64, 511, 1, BF, BF, F32),
    (64, 512, 2, F16, F16, F16),
    (70, 513, 1, BF, BF, None),
    (33, 1024, 1, F32, BF, BF),
    (40, 1152, 4, BF, BF, F32),
    (41, 1536, 1, F16, F16, F16),
    (10, 1537, 5, F32, F16, F32),
    (12, 2048, 1, BF, BF, BF),
    (13, 2241, 1, F32, BF, F32),
    (300, 4099, 3, BF, BF, BF),
    (7, 8192, 1, F32, F32, None),
    (6, 8193, 2, F16, F16, F32),
    (9, 12288, 1, BF, BF, BF),
    (3, 16384, 1, F32, F32, F32),
    (2, 16383, 2, BF, BF, F32),
    (5000, 72, 1, BF, BF, BF),
    (4100, 1152, 2, BF, BF, F32),
    (2500, 2240, 1, F32, F16, F16),
]


@pytest.mark.parametrize("M,C,G,xdt,ydt,pdt", CASES)
def test_layer_norm(M, C, G, xdt, ydt, pdt):
    say(f"[norm] M={M} C={C} groups={G} {xdt} {ydt} {pdt}")
    X, w, b, _ = make(M + C, M, C, G, xdt, ydt, pdt)
    buf = torch.full((M * C + 128,), 7.0, dtype=ydt, device=DEV)
    out = buf[64:64 + M * C].view(M, C)
    eps = 1e-6
    y, mean, rstd = hsq.layer_norm(X, w, b, eps=eps, y_dtype=NAME[ydt], out=out, return_stats=True)
    torch.cuda.synchronize()
    assert (buf[:64] == 7).all() and (buf[64 + M * C:] == 7).all()
    ry, rm, rr = layer_norm64(X, w, b, eps)
    ty, tm, tr = forward_bound(X, w, b, ry, rm, rr, eps)
    close(y, ry, ty, ydt, "Y")
    close(mean, rm, tm, F32, "mean")
    close(rstd, rr, tr, F32, "rstd")
    assert torch.equal(hsq.layer_norm(X, w, b, eps=eps, y_dtype=NAME[ydt]), y)
    if xdt == ydt:
        inplace = X.clone()
        assert torch.equal(hsq.layer_norm(inplace, w, b, eps=eps, out=inplace), y)
    if w is not None:   # either parameter alone
        close(hsq.layer_norm(X, w, None, eps=eps, y_dtype=NAME[ydt]), *_alone(X, w, None, eps), ydt, "weight alone")
        close(hsq.layer_norm(X, None, b, eps=eps, y_dtype=NAME[ydt]), *_alone(X, None, b, eps), ydt, "bias alone")


def _alone(X, w, b, eps):
    y, m, r = layer_norm64(X, w, b, eps)
    return y, forward_bound(X, w, b, y, m, r, eps)[0]


@pytest.mark.parametrize("M,C,G,xdt,ydt,pdt", CASES)
def test_layer_norm_backward(M, C, G, xdt, ydt, pdt):
    say(f"[norm backward] M={M} C={C} groups={G} {xdt} {ydt} {pdt}")
    X, w, b, dY = make(2 * M + C, M, C, G, xdt, ydt, pdt)
    _, m64, r64 = layer_norm64(X, None, None, 1e-6)
    mean, rstd = m64.float(), r64.float()
    need = hsq.layer_norm_backward_workspace_bytes(M, C, G)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    ws[need:] = 90
    dX, dw, db = hsq.layer_norm_backward(dY, X, mean, rstd, w, groups=G, workspace=ws)
    torch.cuda.synchronize()
    assert (ws[need:] == 90).all()
    rX, rw, rb = layer_norm_backward64(dY, X, mean, rstd, w, G)
    # xh is off by 3 U32 |xh|, g by U32; the two means by (DEPTH + 4) U32 of their magnitudes
    x, dy, r = X.double(), dY.double(), rstd.double()[:, None]
    xh = ((x - mean.double()[:, None]) * r).abs()
    g = dy.abs() if w is None else dy.abs() * w.double().reshape(-1, C).repeat_interleave(M // G, 0).abs()
    tX = (DEPTH + 12) * U32 * r * (g + g.mean(1, keepdim=True) + xh * (g * xh).mean(1, keepdim=True))
    close(dX, rX, tX, xdt, "dX")
    n = M // G
    tw = (n + 12) * U32 * (dy.abs() * xh).view(G, n, C).sum(1)
    tb = (n + 12) * U32 * dy.abs().view(G, n, C).sum(1)
    p = F32 if w is None else w.dtype
    assert dw.dtype == p and dw.shape == (w.shape if w is not None else (G, C))
    close(dw.view(G, C), rw, tw, p, "dw")
    close(db.view(G, C), rb, tb, p, "db")
    # each kind alone: the same bits
    only = hsq.layer_norm_backward(dY, X, mean, rstd, w, groups=G, need_params=False)
    assert torch.equal(only[0], dX) and only[1] is None
    only = hsq.layer_norm_backward(dY, X, mean, rstd, w, groups=G, need_input=False)
    assert only[0] is None and torch.equal(only[1], dw) and torch.equal(only[2], db)


@pytest.mark.parametrize("C", [700, 1152, 2240, 6000, 9000])
def test_offset_constant_and_bad_rows(C):
    say(f"[norm rows] C={C}")
    M = 9
    X, w, b, dY = make(C, M, C, 1, F32, F32, F32)
    ref = hsq.layer_norm(X, w, b)
    bad = X.clone()
    bad[2, C - 1] = float("nan")
    bad[5, 0] = float("inf")
    got, mean, rstd = hsq.layer_norm(bad, w, b, return_stats=True)
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[2] = keep[5] = False
    assert torch.equal(got[keep], ref[keep]) and got[2].isnan().all()
    # a row of one value: the bias, whatever the value (its mean is exact for a power of two)
    const = torch.full((M, C), 4.0, device=DEV)
    got, mean, rstd = hsq.layer_norm(const, w, b, eps=1e-6, return_stats=True)
    if C == 700:
        assert (got - b).abs().max() <= 4.0 * DEPTH * U32 * 1e3 * w.abs().max() + 1e-6
    # a large offset: the variance is summed around the mean, not from squares
    off = X + 1000.0
    got = hsq.layer_norm(off, w, b)
    y, m, r = layer_norm64(off, w, b, 1e-5)
    close(got, y, forward_bound(off, w, b, y, m, r, 1e-5)[0], F32, "offset")


def test_gradient_against_differences():
    M, C, G = 12, 1000, 3
    say("[norm differences]")
    X, w, b, dY = make(3, M, C, G, F32, F32, F32)
    _, mean, rstd = hsq.layer_norm(X, w, b, eps=1e-5, return_stats=True)
    dX, dw, db = hsq.layer_norm_backward(dY, X, mean, rstd, w)
    g = torch.Generator(device=DEV).manual_seed(4)
    h = 1e-4
    for i, (t, grad) in enumerate(((X, dX), (w, dw), (b, db))):
        v = torch.randn(t.shape, generator=g, device=DEV, dtype=torch.float64)
        vals = []
        for s in (h, -h):
            a = [X.double(), w.double(), b.double()]
            a[i] = a[i] + s * v
            vals.append((layer_norm64(a[0], a[1], a[2], 1e-5)[0] * dY.double()).sum())
        num = (vals[0] - vals[1]) / (2 * h)
        # the statistics carry (DEPTH + 8) U32, the sums DEPTH more: relative to the sum of magnitudes,
        # and a row's gradient is a difference of terms a few times its size
        tol = 8 * (2 * DEPTH + 8) * U32 * (grad.double().abs() * v.abs()).sum() + 1e-6 * num.abs()
        assert abs((grad.double() * v).sum() - num) <= tol


def test_replay_streams_and_repeats():
    for M, C, G in [(1, 4096, 1), (600, 1152, 2), (50, 9000, 1), (31, 333, 31)]:
        say(f"[norm graph] {M} {C} {G}")
        X, w, b, dY = make(17, M, C, G, BF, BF, F32)

        def run():
            y, m, r = hsq.layer_norm(X, w, b, return_stats=True)
            return (y, m, r) + hsq.layer_norm_backward(dY, X, m, r, w)

        ref = run()
        torch.cuda.synchronize()
        graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        cap.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(cap):
            with torch.cuda.graph(graph, stream=cap):
                outs = run()
        torch.cuda.synchronize()
        for rep in range(4):
            for o in outs:
                o.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, c) for a, c in zip(outs, ref)), rep
            assert all(torch.equal(a, c) for a, c in zip(run(), ref))
        got = []
        for s in (torch.cuda.Stream(), torch.cuda.Stream()):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(run())
        torch.cuda.synchronize()
        for o in got:
            assert all(torch.equal(a, c) for a, c in zip(o, ref))


@pytest.mark.parametrize("M,C", [(131071, 16384), (1 << 25, 61)])
def test_largest_sizes(M, C):
    # rows sampled over the whole range; the parameter gradients of all rows
    say(f"[norm large] {M} {C}")
    g = torch.Generator(device=DEV).manual_seed(6)
    X = torch.empty(M, C, device=DEV, dtype=BF).normal_(generator=g)
    dY = torch.empty(M, C, device=DEV, dtype=BF).normal_(generator=g)
    w, b = torch.rand(C, generator=g, device=DEV) + 0.5, torch.rand(C, generator=g, device=DEV)
    rows = torch.cat([torch.arange(0, M, M // 60, device=DEV), torch.tensor([M - 1], device=DEV)])
    y, mean, rstd = hsq.layer_norm(X, w, b, return_stats=True)
    ry, rm, rr = layer_norm64(X[rows], w, b, 1e-5)
    close(y[rows], ry, forward_bound(X[rows], w, b, ry, rm, rr, 1e-5)[0], BF, "Y")
    del y
    dX, dw, db = hsq.layer_norm_backward(dY, X, mean, rstd, w)
    x, dy, r = X[rows].double(), dY[rows].double(), rstd[rows].double()[:, None]
    rX = layer_norm_backward64(dy, x, mean[rows], rstd[rows], w)[0]
    xh, gr = ((x - mean[rows].double()[:, None]) * r).abs(), dy.abs() * w.double()
    close(dX[rows], rX, (DEPTH + 12) * U32 * r * (gr + gr.mean(1, keepdim=True) + xh * (gr * xh).mean(1, keepdim=True)),
          BF, "dX")
    del dX
    # a workgroup adds its share of the rows one by one, 256 shares (8 rows side by side in short rows)
    for c in (0, C // 2, C - 1):
        col, wx = dY[:, c].double(), (X[:, c].double() - mean.double()) * rstd.double()
        n = M // 256 + 300
        assert abs(db[c] - col.sum()) <= n * U32 * col.abs().sum() + U32 * db[c].abs()
        assert abs(dw[c] - (col * wx).sum()) <= (n + 12) * U32 * (col * wx).abs().sum() + U32 * dw[c].abs()


def test_more_rows_than_a_launch_has_threads_for_are_refused():
    X = torch.zeros((1 << 26) - 1, 1, device=DEV, dtype=BF)
    with pytest.raises(hsq.HsqError) as e:
        hsq.layer_norm(X)
    assert e.value.status == hsq.E_INVAL


def rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("M", [1, 37, 260])
def test_pre_norm_mlp_forward_and_backward(M):
    """x + down(gelu(up(norm(x)))) in 16 bits, and its gradients: every stored
    tensor is off by half a bf16 step of itself (2^-8 at most, 2^-9 in the
    mean), so a chain of n roundings stays below n 2^-8 in norm."""
    say(f"[mlp] M={M}")
    C, H = 320, 1288
    g = torch.Generator(device=DEV).manual_seed(M)

    def rnd(*s):
        return torch.randn(*s, generator=g, device=DEV)

    x, dy = rnd(M, C).to(BF), rnd(M, C).to(BF)
    w, b = (1 + 0.2 * rnd(C)).to(BF), (0.2 * rnd(C)).to(BF)
    W1, b1 = (rnd(C, H) / C ** 0.5).to(BF), (0.1 * rnd(H)).to(BF)
    W2, b2 = (rnd(H, C) / H ** 0.5).to(BF), (0.1 * rnd(C)).to(BF)
    n, mean, rstd = hsq.layer_norm(x, w, b, return_stats=True)
    hid, z = hsq.linear(n, W1, b1, act="gelu_tanh", return_preact=True)
    y = hsq.linear(hid, W2, b2, x)
    dh, dW2, db2 = hsq.linear_backward(dy, hid, W2)
    dn, dW1, db1 = hsq.linear_backward(dh, n, W1, z, act="gelu_tanh")
    dx, dw, db = hsq.layer_norm_backward(dn, x, mean, rstd, w)
    dx = dx + dy                                # the residual's own gradient
    xd = x.double()
    rn, rm, rr = layer_norm64(x, w, b, 1e-5)
    rz = rn @ W1.double() + b1.double()
    rh = act64(rz, "gelu_tanh")
    ry = rh @ W2.double() + b2.double() + xd
    rdh = dy.double() @ W2.double().t()
    rdz = rdh * act_grad64(rz, "gelu_tanh")
    rdn = rdz @ W1.double().t()
    rdx, rdw, rdb = layer_norm_backward64(rdn, x, rm, rr, w)
    step = 2.0 ** -8
    for got, ref, roundings in ((y, ry, 3), (dW2, rh.t() @ dy.double(), 3), (db2, dy.double().sum(0), 1),
                                (dW1, rn.t() @ rdz, 5), (db1, rdz.sum(0), 4), (dw, rdw[0], 6), (db, rdb[0], 6),
                                (dx, rdx + dy.double(), 7)):
        # act' and act take their argument's error with a slope below 1.2 and |act''| < 1.2
        assert rel(got, ref) <= 1.5 * roundings * step


def test_norm_feeds_the_w4a4_layer():
    """The norm's bf16 output is the W4A4 layer's X, and the 16-bit linear on the
    same layer's dequantized weight stays as close to it as its 4-bit codes allow."""
    from synth import make_random_layer

    M, K, N = 150, 512, 256
    say("[norm -> w4a4]")
    lay = make_random_layer(811, M, K, N, r=4)

    def d16(a):
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).to(DEV)

    X = d16(lay["X"]).view(BF)
    packed, _ = hsq.pack_weights(torch.from_numpy(lay["qw"][0]).to(DEV))
    lam, sw, L1, L2, bias = d16(lay["lam"]), d16(lay["sw"]), d16(lay["L1"]), d16(lay["L2"]), d16(lay["bias"])
    n = hsq.layer_norm(X, eps=1e-6)
    y = hsq.w4a4_lowrank_linear(n, lam, packed, sw, L1, L2, bias, N=N, y_dtype="f32")[0]
    # the layer in 64 bits on the same input, activations not quantized
    scale = sw.view(F16).double()[0].repeat_interleave(64, 0)
    Wd = torch.from_numpy(lay["qw"][0]).to(DEV).double() * scale + L1.view(BF).double()[0] @ L2.view(BF).double()[0]
    Wd = Wd / lam.view(F16).double()[:, None]
    ref = n.double() @ Wd + bias.view(BF).double()[0]
    lin = hsq.linear(n, Wd.to(BF).contiguous(), bias.view(BF)[0].contiguous(), y_dtype="f32")
    # one weight rounding: 2^-8 of |n| |W| at most, in norm far below
    tol = (half_step(BF) + 2 * K * U32) * torch.mm(n.double().abs(), Wd.abs()) + U32 * 2 * ref.abs()
    close(lin, ref, tol, F32, "16-bit layer")
    # a 4-bit code is half a step of absmax / 7 away at most, per element of X / lambda
    xh = (n.double() / lam.view(F16).double()).abs()
    step = xh.view(M, K // 64, 64).amax(2, keepdim=True).expand(M, K // 64, 64).reshape(M, K) / 7 * (0.5 + 7 * 2.0 ** -11)
    q = torch.from_numpy(lay["qw"][0]).to(DEV).double().abs() * scale
    lim = torch.mm(step * (1 + 1e-3), q) + 1e-4 * ref.abs() + 1e-4 * torch.mm(xh, Wd.abs() * lam.view(F16).double()[:, None])
    assert ((y.double() - ref).abs() <= lim).all()
