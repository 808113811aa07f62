"""The 16-bit linear and its backward pass on the GPU against the 64-bit
definition, element by element, within bounds derived from the formats and
the number of additions (linear_norm_ref)."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # collected on CPU-only hosts, never run there
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from linear_norm_ref import act_grad64, half_step, linear64, linear_backward64, tiny_step  # noqa: E402

DEV = torch.device("cuda:0")
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def say(msg):
    print(msg, flush=True)


def make(seed, M, K, N, dt, bias=True):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, generator=g, device=DEV)

    X, W = rnd(M, K).to(dt), (rnd(K, N) / K ** 0.5).to(dt)
    return X, W, (0.5 * rnd(N)).to(dt) if bias else None, rnd


def guarded(shape, dt):
    """A tensor whose surroundings show a write out of its bounds."""
    n = 1
    for s in shape:
        n *= s
    buf = torch.full((n + 128,), 7.0, dtype=dt, device=DEV)
    t = buf[64:64 + n].view(shape)
    t.fill_(float("nan"))

    def check():
        assert (buf[:64] == 7).all() and (buf[64 + n:] == 7).all(), "write outside the output"

    return t, check


def close(got, ref, tol, dt, what):
    """tol: before the last rounding to dt."""
    lim = tol + half_step(dt) * (ref.abs() + tol) + tiny_step(dt)
    bad = ~((got.double() - ref).abs() <= lim)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}, got "
                           f"{got[bad][0].item()}, want {ref[bad][0].item()}, limit {lim[bad][0].item()}")


def stale(nbytes):
    return torch.full((max(nbytes, 16),), 255, dtype=torch.uint8, device=DEV)   # NaN in every type


FORWARD = [
    # M, K, N, type, act, bias, residual, fp32 output
    (1, 1, 1, BF, "identity", True, True, False),
    (1, 64, 16, BF, "identity", False, False, True),
    (1, 4096, 12288, BF, "silu", False, False, False),
    (1, 1000, 1001, F16, "gelu", True, True, True),
    (2, 33, 7, F16, "gelu_tanh", True, True, False),
    (5, 2240, 130, BF, "silu", True, False, True),
    (16, 12288, 4096, BF, "identity", False, True, False),
    (17, 1152, 136, F16, "identity", True, False, False),
    (33, 515, 1023, BF, "gelu_tanh", True, True, True),
    (48, 256, 200, F16, "silu", False, True, False),
    (64, 777, 300, BF, "gelu", True, True, False),
    (64, 4096, 513, F16, "identity", True, True, True),
    (65, 40, 64, BF, "identity", False, False, True),
    (65, 7, 3, F16, "gelu_tanh", True, True, False),
    (100, 31, 1000, BF, "silu", True, False, True),
    (128, 128, 128, BF, "identity", False, False, True),
    (129, 1001, 777, F16, "gelu", True, True, True),
    (300, 4096, 520, BF, "gelu_tanh", True, True, False),     # few tiles: the reduction is split
    (333, 1001, 777, F16, "gelu", True, True, True),
    (2049, 72, 4100, BF, "silu", True, True, False),          # many tiles, ragged in all three
    (2048, 1152, 4608, BF, "gelu_tanh", True, False, True),
    (4096, 8, 8200, F16, "identity", True, True, True),
    (1000, 1, 999, BF, "gelu", True, True, True),
    # few rows at the ends of X and W: loads there move back by up to seven elements
    (5, 3867, 119, BF, "gelu", False, False, False),
    (48, 33, 9, F16, "silu", True, True, True),
    (2, 4, 2, BF, "identity", True, False, True),
    (1, 8, 1, BF, "identity", False, False, True),
    (1, 7, 1, BF, "identity", False, False, True),
    (7, 1, 7, F16, "gelu_tanh", True, False, True),
    (49, 300, 131, BF, "identity", True, False, True),
    # ragged rows read as they are (short reductions, few tiles) and from padded copies
    (130, 8, 3, BF, "identity", True, False, True),
    (1000, 4001, 201, BF, "silu", True, True, False),
    (900, 2500, 1201, F16, "identity", False, False, True),
] + [(150 + i, 95 + i, 241 + 3 * i, BF, "identity", False, False, True) for i in range(8)
] + [(3, 31 + i, 121 + i, BF, "identity", False, False, True) for i in range(8)]


@pytest.mark.parametrize("M,K,N,dt,act,bias,res,y32", FORWARD)
def test_linear(M, K, N, dt, act, bias, res, y32):
    say(f"[linear] M={M} K={K} N={N} {dt} {act}")
    X, W, b, rnd = make(M + K + N, M, K, N, dt, bias)
    ydt = F32 if y32 else dt
    R = rnd(M, N).to(ydt) if res else None
    out, chk = guarded((M, N), ydt)
    Z, chkz = guarded((M, N), dt)
    ws = stale(hsq.linear_workspace_bytes(M, K, N))
    got = hsq.linear(X, W, b, R, act=act, y_dtype="f32" if y32 else None, out=out, preact_out=Z, workspace=ws)
    assert got is out
    torch.cuda.synchronize()
    chk()
    chkz()
    y, z, ty, tz = linear64(X, W, b, R, act)
    close(out, y, ty, ydt, "Y")
    close(Z, z, tz, dt, "Z")
    # without Z, in place of the residual, without a workspace of the caller's: the same bits
    inplace = R.clone() if res else None
    again = hsq.linear(X, W, b, inplace, act=act, y_dtype="f32" if y32 else None, out=inplace)
    assert torch.equal(again, out)


BACKWARD = [
    # M, K, N, type, act, bias, fp32 dY
    (1, 1, 1, BF, "identity", True, False),
    (1, 64, 128, F16, "silu", True, False),
    (3, 4096, 1000, BF, "gelu_tanh", True, False),
    (16, 33, 7, F16, "gelu", True, True),
    (64, 515, 1023, BF, "identity", True, False),
    (65, 2240, 64, BF, "silu", False, False),
    (128, 128, 128, BF, "identity", False, False),
    (200, 1152, 520, F16, "gelu_tanh", True, False),
    (257, 515, 1023, F16, "silu", True, False),
    (300, 48, 4096, BF, "identity", True, True),
    (1000, 999, 31, BF, "gelu", True, False),
    (40, 2049, 4104, BF, "identity", True, False),           # many tiles of dW, a short reduction
    (2049, 4100, 72, F16, "silu", True, False),              # many tiles of dX
    (1500, 1023, 1401, BF, "identity", True, False),         # ragged rows read as they are
    (700, 1503, 5001, F16, "gelu", False, False),            # W padded for dX, X too
    (2, 2240, 4001, BF, "gelu_tanh", True, False),           # few rows against a long, split reduction
    (9, 1, 9, BF, "identity", True, False),
    (4096, 256, 300, BF, "gelu_tanh", True, False),          # a long reduction into few tiles of dW
]


@pytest.mark.parametrize("M,K,N,dt,act,bias,dy32", BACKWARD)
def test_linear_backward(M, K, N, dt, act, bias, dy32):
    say(f"[linear backward] M={M} K={K} N={N} {dt} {act}")
    X, W, b, rnd = make(3 * M + K + N, M, K, N, dt, bias)
    dY = rnd(M, N).to(F32 if dy32 else dt)
    Z = (2 * rnd(M, N)).to(dt)
    ws = stale(hsq.linear_backward_workspace_bytes(M, K, N))
    dX, dW, db = hsq.linear_backward(dY, X, W, Z, act=act, need_bias=bias, workspace=ws)
    (rX, rW, rb), (tX, tW, tb) = linear_backward64(dY, X, W, Z, act)
    close(dX, rX, tX, dt, "dX")
    close(dW, rW, tW, dt, "dW")
    assert (db is None) == (not bias)
    if bias:
        close(db, rb, tb, dt, "db")
    # each output alone: the same bits
    for i, kw in enumerate((dict(need_weight=False, need_bias=False), dict(need_input=False, need_bias=False),
                            dict(need_input=False, need_weight=False))):
        alone = hsq.linear_backward(dY, X, W, Z, act=act, **kw)
        assert [t is not None for t in alone] == [i == 0, i == 1, i == 2]
        if i < 2 or bias:
            assert torch.equal(alone[i], (dX, dW, db)[i])


@pytest.mark.parametrize("dt", [BF, F16])
@pytest.mark.parametrize("K,N", [(64, 64), (97, 61)])
@pytest.mark.parametrize("M", [20, 70, 300])
def test_outputs_stay_inside_their_buffers(M, K, N, dt):
    # through the C ABI, which takes the buffers from the caller
    say(f"[linear buffers] M={M} K={K} N={N} {dt}")
    X, W, b, rnd = make(5, M, K, N, dt)
    dY = rnd(M, N).to(dt)
    lib, P, code = hsq._load(), hsq._ptr, hsq._t().code[dt]
    outs = [guarded(s, dt) for s in ((M, K), (K, N), (N,))]
    need = hsq.linear_backward_workspace_bytes(M, K, N)
    ws = torch.full((need + 256,), 90, dtype=torch.uint8, device=DEV)
    st = lib.hsq_linear_backward(P(dY), code, P(X), M, K, N, code, P(W), None, 0, P(outs[0][0]), P(outs[1][0]),
                                 P(outs[2][0]), P(ws), need, hsq._stream())
    torch.cuda.synchronize()
    assert st == hsq.OK
    for t, chk in outs:
        chk()
        assert torch.isfinite(t).all()
    assert (ws[need:] == 90).all()
    need = hsq.linear_workspace_bytes(M, K, N)
    ws = torch.full((need + 256,), 90, dtype=torch.uint8, device=DEV)
    Y, chk = guarded((M, N), dt)
    st = lib.hsq_linear(P(X), M, K, N, code, P(W), P(b), 0, None, P(Y), code, None, P(ws), need, hsq._stream())
    torch.cuda.synchronize()
    assert st == hsq.OK and torch.isfinite(Y).all() and (ws[need:] == 90).all()
    chk()


@pytest.mark.parametrize("M", [5, 40, 130, 2100])
def test_a_bad_row_stays_in_its_row(M):
    # NaN and infinity in one token: the other rows' bits do not change, and
    # neither does the padding of ragged rows bring them anywhere else
    K, N = 333, 4099 if M > 1000 else 205
    say(f"[linear rows] M={M}")
    X, W, b, rnd = make(11, M, K, N, BF)
    ref = hsq.linear(X, W, b, act="silu")
    bad = X.clone()
    bad[3, K - 1] = float("nan")
    bad[1, 0] = float("inf")
    got = hsq.linear(bad, W, b, act="silu")
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[3] = keep[1] = False
    assert torch.equal(got[keep], ref[keep])
    assert got[3].isnan().all()
    # and in the weights: a bad input channel k reaches every output, a bad column only its own
    w2 = W.clone()
    w2[K - 1, N - 1] = float("nan")
    got = hsq.linear(X, w2, b, act="silu")
    assert torch.equal(got[:, :-1], ref[:, :-1]) and got[:, -1].isnan().all()
    dY = rnd(M, N).to(BF)
    r = hsq.linear_backward(dY, X, W)
    d2 = dY.clone()
    d2[M - 1, N - 1] = float("nan")
    g = hsq.linear_backward(d2, X, W)
    assert torch.equal(g[0][:-1], r[0][:-1]) and g[0][-1].isnan().all()
    assert torch.equal(g[1][:, :-1], r[1][:, :-1]) and g[1][:, -1].isnan().all()
    assert torch.equal(g[2][:-1], r[2][:-1]) and g[2][-1].isnan()


@pytest.mark.parametrize("act", ["gelu_tanh", "gelu", "silu"])
def test_activations_over_their_range(act):
    # every bf16 value as Z through a 1 x 1 product with W = 1 (and its derivative)
    bits = torch.arange(65536, device=DEV, dtype=torch.int32).to(torch.int16)
    z = bits.view(BF)
    z = z[torch.isfinite(z) & (z.abs() < 1e18)]
    M = z.numel()
    say(f"[activation] {act} on {M} values")
    X, W = z.view(M, 1).contiguous(), torch.ones(1, 1, dtype=BF, device=DEV)
    Y, Z = hsq.linear(X, W, act=act, y_dtype="f32", return_preact=True)
    assert torch.equal(Z, X)
    y, _, ty, _ = linear64(X, W, None, None, act)
    close(Y, y, ty, F32, "act")
    big = X.abs() > 30
    # |act(z)| <= |z| e^-|z| < 3e-12 below z = -30 (silu the largest), within 3e-12 of z above 30
    assert torch.equal(Y[big & (X > 0)], X[big & (X > 0)].float()) and (Y[big & (X < 0)].abs() < 3e-12).all()
    dY = torch.ones(M, 1, dtype=F32, device=DEV)
    dX = hsq.linear_backward(dY, X, W, X, act=act, need_weight=False, need_bias=False)[0]
    ref = act_grad64(X.double().clamp(-1e4, 1e4), act)
    close(dX, ref, torch.full_like(ref, 17 * 2.0 ** -24) + half_step(BF) * ref.abs(), BF, "act'")


@pytest.mark.parametrize("act", ["gelu_tanh", "gelu", "silu"])
def test_activations_at_the_ends(act):
    # where squares and cubes of z leave fp32: z or 0, slope 1 or 0; NaN stays NaN
    say(f"[activation] {act} at the ends")
    z = torch.tensor([11, 17, 65, 89, 1e4, 1e13, 1e18, 1e20, 1e30, 3e38], device=DEV).to(BF)
    z = torch.cat([z, -z, torch.tensor([float("nan")], device=DEV, dtype=BF)])
    X, W = z.view(-1, 1).contiguous(), torch.ones(1, 1, dtype=BF, device=DEV)
    Y = hsq.linear(X, W, act=act, y_dtype="f32")
    dX = hsq.linear_backward(torch.ones_like(X), X, W, X, act=act, need_weight=False, need_bias=False)[0]
    assert torch.equal(Y[:10], torch.where(X[:10] > 17, X[:10].float(), Y[:10])) and (dX[:10] == 1).all()
    # silu(-11) = -11 e^-11, silu'(-11) = -10 e^-11
    assert (Y[10:20].abs() <= 2e-4).all() and (dX[10:20].abs() <= 2e-4).all()
    assert (Y[12:20].abs() <= 1e-20).all() and (dX[12:20].abs() <= 1e-20).all()
    assert Y[20].isnan() and dX[20].isnan()


@pytest.mark.parametrize("act", ["gelu_tanh", "gelu", "silu"])
def test_slope_at_a_stored_infinity(act):
    # a Z beyond fp16 is stored as an infinity: its slope is 1 or 0, not NaN
    X = torch.tensor([[float("inf")], [float("-inf")]], device=DEV, dtype=F16)
    W, dY = torch.ones(1, 1, dtype=F16, device=DEV), torch.ones(2, 1, dtype=F16, device=DEV)
    dX = hsq.linear_backward(dY, X, W, X, act=act, need_weight=False, need_bias=False)[0]
    # below -64 the slope is at most 65 e^-64 < 1e-25, below fp16's smallest value (6e-8) by far
    assert dX[0] == 1 and dX[1] == 0


@pytest.mark.parametrize("M,K,N", [(8, 512, 384), (100, 512, 384), (333, 130, 257)])
def test_gradient_against_differences(M, K, N):
    # L = sum(dY * Y): the library's gradient along a direction v against the
    # central difference of the 64-bit forward pass (truncation below 1e-9 here)
    say(f"[linear differences] {M} {K} {N}")
    X, W, b, rnd = make(23, M, K, N, F16)
    dY = rnd(M, N).to(F16)
    _, Z = hsq.linear(X, W, b, act="gelu", return_preact=True)
    grads = hsq.linear_backward(dY, X, W, Z, act="gelu")
    # dZ is taken at Z as it was stored: half a step of fp16 away at most, with |act''| < 1.2
    (rX, rW, rb), tols = linear_backward64(dY, X, W, Z, "gelu")
    slack = 1.2 * (half_step(F16) * Z.double().abs() + 2 * K * 2.0 ** -24 * torch.mm(X.double().abs(), W.double().abs()) + tiny_step(F16)) * dY.double().abs()
    slacks = (torch.mm(slack, W.double().abs().t().contiguous()), torch.mm(X.double().abs().t().contiguous(), slack),
              slack.sum(0))
    h = 1e-4
    for i, t in enumerate((X, W, b)):
        v = rnd(*t.shape).double()
        args = [X.double(), W.double(), b.double()]
        vals = []
        for s in (h, -h):
            a = list(args)
            a[i] = args[i] + s * v
            vals.append((linear64(a[0], a[1], a[2], None, "gelu")[0] * dY.double()).sum())
        num = (vals[0] - vals[1]) / (2 * h)
        tol = ((tols[i] + slacks[i] + half_step(F16) * grads[i].double().abs() + tiny_step(F16)) * v.abs()).sum()
        assert abs((grads[i].double() * v).sum() - num) <= tol + 1e-6 * num.abs() + 1e-6


def test_replay_streams_and_repeats():
    """Captured and replayed with other work in between, on two streams at
    once with a workspace each, and over again: the same bits."""
    cases = [(1, 4096, 1024), (40, 512, 300), (200, 1030, 257), (2048, 64, 4096)]
    for M, K, N in cases:
        say(f"[linear graph] {M} {K} {N}")
        X, W, b, rnd = make(31, M, K, N, BF)
        dY = rnd(M, N).to(BF)
        R = rnd(M, N).to(BF)

        def run(wsf, wsb):
            y, z = hsq.linear(X, W, b, R, act="silu", return_preact=True, workspace=wsf)
            return (y, z) + hsq.linear_backward(dY, X, W, z, act="silu", workspace=wsb)

        def spaces():
            return (stale(hsq.linear_workspace_bytes(M, K, N)), stale(hsq.linear_backward_workspace_bytes(M, K, N)))

        ref = run(*spaces())
        torch.cuda.synchronize()
        for _ in range(3):
            assert all(torch.equal(a, c) for a, c in zip(run(*spaces()), ref))
        graph, cap, sp = torch.cuda.CUDAGraph(), torch.cuda.Stream(), spaces()
        cap.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(cap):
            with torch.cuda.graph(graph, stream=cap):
                outs = run(*sp)
        torch.cuda.synchronize()
        for rep in range(4):
            for o in outs:
                o.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, c) for a, c in zip(outs, ref)), rep
            assert all(torch.equal(a, c) for a, c in zip(run(*spaces()), ref))
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        got = []
        for s in (s1, s2):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(run(None, None))
        torch.cuda.synchronize()
        for g in got:
            assert all(torch.equal(a, c) for a, c in zip(g, ref))


LARGE = [
    # each of the three matrices in turn close to 2^30 elements
    (262143, 4088, 72),
    (3, 4088, 262136),
    (70, 4088, 262136),
    (262143, 16, 4088),
]


@pytest.mark.parametrize("M,K,N", LARGE)
def test_largest_sizes(M, K, N):
    # rows and columns sampled over the whole range, the last ones among them
    say(f"[linear large] {M} {K} {N}")
    g = torch.Generator(device=DEV).manual_seed(9)
    X = torch.empty(M, K, device=DEV, dtype=BF).normal_(generator=g)
    W = torch.empty(K, N, device=DEV, dtype=BF).normal_(generator=g)
    rows = torch.cat([torch.arange(0, M, max(1, M // 50), device=DEV), torch.tensor([M - 1], device=DEV)])
    cols = torch.cat([torch.arange(0, N, max(1, N // 50), device=DEV), torch.tensor([N - 1], device=DEV)])
    Y = hsq.linear(X, W, y_dtype="f32")
    Xs, Ws = X[rows], W[:, cols].contiguous()
    y, _, ty, _ = linear64(Xs, Ws, None, None, "identity")
    close(Y[rows][:, cols], y, ty, F32, "Y")
    del Y
    dY = torch.empty(M, N, device=DEV, dtype=BF).normal_(generator=g)
    dX, dW, db = hsq.linear_backward(dY, X, W)
    kc = torch.cat([torch.arange(0, K, max(1, K // 20), device=DEV), torch.tensor([K - 1], device=DEV)])
    d = dY[rows].double()
    w = W[kc].double()
    close(dX[rows][:, kc], d @ w.t(), 2 * N * 2.0 ** -24 * (d.abs() @ w.abs().t()), BF, "dX")
    x, d = X[:, kc].double(), dY[:, cols].double()
    xt = x.t().contiguous()
    close(dW[kc][:, cols], xt @ d, 2 * M * 2.0 ** -24 * (xt.abs() @ d.abs()), BF, "dW")
    close(db[cols], d.sum(0), 2 * M * 2.0 ** -24 * d.abs().sum(0), BF, "db")


def test_wide_rows():
    # the widest N and K, one token
    say("[linear wide]")
    for K, N in ((3, 1 << 24), (1 << 24, 3)):
        X, W, b, rnd = make(13, 1, K, N, BF)
        y, _, ty, _ = linear64(X, W, b, None, "identity")
        close(hsq.linear(X, W, b, y_dtype="f32"), y, ty, F32, "Y")
        dY = rnd(1, N).to(BF)
        (rX, rW, rb), (tX, tW, tb) = linear_backward64(dY, X, W, None, "identity")
        dX, dW, db = hsq.linear_backward(dY, X, W)
        close(dX, rX, tX, BF, "dX")
        close(dW, rW, tW, BF, "dW")
        close(db, rb, tb, BF, "db")


def test_host_threads():
    """Calls from several host threads at once, a stream and buffers each."""
    import threading

    say("[linear threads]")
    M, K, N = 150, 700, 333
    X, W, b, rnd = make(19, M, K, N, F16)
    dY = rnd(M, N).to(F16)
    ref = hsq.linear_backward(dY, X, W) + (hsq.linear(X, W, b),)
    torch.cuda.synchronize()
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = hsq.linear_backward(dY, X, W) + (hsq.linear(X, W, b),)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, c) for a, c in zip(got, ref)):
                    bad.append(1)

    ts = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


def test_two_graphs_share_a_workspace():
    """Two captured calls of different sizes on one workspace, replayed in turn:
    neither relies on what it left there."""
    say("[linear graphs, one workspace]")
    cases = [(300, 4096, 520), (333, 1001, 4777), (20, 3000, 500), (70, 515, 1023)]
    ws = stale(max(max(hsq.linear_workspace_bytes(*c), hsq.linear_backward_workspace_bytes(*c)) for c in cases))
    runs = []
    for M, K, N in cases:
        X, W, b, rnd = make(M, M, K, N, BF)
        dY = rnd(M, N).to(BF)

        def run(X=X, W=W, b=b, dY=dY):
            return (hsq.linear(X, W, b, act="gelu", workspace=ws),) + hsq.linear_backward(dY, X, W, workspace=ws)

        ref = [t.clone() for t in run()]
        torch.cuda.synchronize()
        graph, cap = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        cap.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(cap):
            with torch.cuda.graph(graph, stream=cap):
                outs = run()
        torch.cuda.synchronize()
        # `run` holds the inputs: a graph reads their memory at every replay, and
        # the next capture returns the memory of dropped tensors to the device
        runs.append((graph, outs, ref, run))
    for rep in range(3):
        for graph, outs, ref, _ in runs:
            for o in outs:
                o.fill_(float("nan"))
            graph.replay()
        torch.cuda.synchronize()
        for graph, outs, ref, _ in runs:
            assert all(torch.equal(a, c) for a, c in zip(outs, ref)), rep
