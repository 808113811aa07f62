"""Calls of the 16-bit linear and the layer normalisation that the interface
does not allow, on the host: sizes beyond a C int, outputs over other operands."""

import pytest
import torch

import w4a4_rank_assisted_amd as hsq

lib = hsq._load()
BIG = 1 << 32          # its low 32 bits are zero


# ------------------------------------------------------- sizes beyond a C int
@pytest.mark.parametrize("big", [(BIG + 333, 1001, 777), (333, BIG + 1001, 777), (333, 1001, BIG + 777),
                                 (-BIG + 333, 1001, 777)])
def test_workspaces_of_sizes_beyond_an_int(big):
    # what the low 32 bits name is another, small shape
    assert hsq.linear_workspace_bytes(333, 1001, 777) > 0 and hsq.linear_workspace_bytes(*big) == 0
    assert hsq.linear_backward_workspace_bytes(333, 1001, 777) > 0 and hsq.linear_backward_workspace_bytes(*big) == 0
    M, C, _ = big
    assert hsq.layer_norm_backward_workspace_bytes(M, C) == 0 or (M, C) == (333, 1001)
    assert hsq.layer_norm_backward_workspace_bytes(333, 1001, BIG + 1) == 0


class Recorder:
    """Stands for the library: every call succeeds and is kept."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name == "hsq_status_string":
            return lib.hsq_status_string
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture
def recorder(monkeypatch):
    # tensors without memory stand for device tensors of sizes no host holds
    r = Recorder()
    monkeypatch.setattr(hsq, "_load", lambda: r)
    monkeypatch.setattr(hsq, "_device", lambda T, t, name: -1)
    monkeypatch.setattr(hsq._t(), "stream", lambda dev: 0)
    return r


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def test_calls_of_sizes_beyond_an_int_are_refused(recorder):
    many, few, wide = meta(BIG + 5, 8), meta(8, 16), meta(8, BIG + 16)
    stat = meta(BIG + 5, dtype=torch.float32)
    for call in (lambda: hsq.linear(many, few), lambda: hsq.linear(meta(4, 8), wide),
                 lambda: hsq.linear(meta(4, BIG + 8), meta(BIG + 8, 16)),
                 lambda: hsq.linear_backward(meta(BIG + 5, 16), many, few),
                 lambda: hsq.linear_backward(meta(4, BIG + 16), meta(4, 8), wide),
                 lambda: hsq.layer_norm(many), lambda: hsq.layer_norm(meta(4, BIG + 8)),
                 lambda: hsq.layer_norm(meta(4, 8), meta(BIG + 1, 8)),
                 lambda: hsq.layer_norm_backward(many, many, stat, stat),
                 lambda: hsq.layer_norm_backward(meta(4, 8), meta(4, 8), stat[:4], stat[:4], groups=BIG + 1)):
        with pytest.raises(hsq.HsqError) as e:
            call()
        assert e.value.status == hsq.E_INVAL
    assert recorder.calls == []
    hsq.linear(meta(4, 8), few)
    assert recorder.calls[-1][0] == "hsq_linear" and recorder.calls[-1][1][1:4] == (4, 8, 16)


# ------------------------------------------------------- outputs over other operands
# Where a call is not refused it reaches the launch, which fails without a GPU
# (E_HIP); with one the fake addresses must not get that far, so only refused
# calls run there.
NO_GPU = not torch.cuda.is_available()
GAP = 1 << 24          # operands of these sizes are below 2^24 bytes


def at(i):
    return 0x10000000 + i * GAP


def _status(fn, args, refused):
    if not refused and not NO_GPU:
        pytest.skip("a launch on made-up addresses")
    st = fn(*args)
    assert st == (hsq.E_INVAL if refused else hsq.E_HIP)


def linear_args(dt=hsq.BF16, ydt=hsq.BF16, M=64, K=256, N=256, **kw):
    a = dict(X=at(0), W=at(1), bias=at(2), res=at(3), Y=at(4), Z=at(5), ws=at(6))
    a.update(kw)
    need = lib.hsq_linear_workspace_bytes(M, K, N)
    return (a["X"], M, K, N, dt, a["W"], a["bias"], 0, a["res"], a["Y"], ydt, a["Z"], a["ws"], need, None)


END = 64 * 256 * 2     # bytes of X, Y, Z and the residual in 16 bits


@pytest.mark.parametrize("kw,refused", [
    (dict(), False), (dict(Y=at(3)), False),                            # all apart; added in place
    (dict(Y=at(0)), True), (dict(Y=at(1)), True), (dict(Y=at(2) - END + 16), True), (dict(Y=at(5)), True),
    (dict(Y=at(3) + 16), True), (dict(Y=at(3) - 16), True), (dict(Y=at(3) + END), False), (dict(Y=at(3) - END), False),
    (dict(Z=at(0)), True), (dict(Z=at(1) + 256 * 256 * 2 - 16), True), (dict(Z=at(1) + 256 * 256 * 2), False),
    (dict(Z=at(3)), True), (dict(Z=at(3), Y=at(3)), True),
    (dict(ydt=hsq.F32, Y=at(5) - END), True), (dict(ydt=hsq.F32, Y=at(5) - 2 * END), False),
    (dict(X=at(1)), False), (dict(res=at(1)), False),                   # two inputs may share memory
    (dict(ws=at(0) + 16), False),                                       # no workspace is needed here
    (dict(M=300, K=2048, N=256, ws=at(4)), True), (dict(M=300, K=2048, N=256, ws=at(1)), True),
])
def test_linear_outputs_over_operands(kw, refused):
    _status(lib.hsq_linear, linear_args(**kw), refused)


@pytest.mark.parametrize("kw,refused", [
    (dict(), False), (dict(dX=at(1)), True), (dict(dX=at(0)), True), (dict(dW=at(2)), True), (dict(dW=at(3)), True),
    (dict(db=at(0) + 16), True), (dict(dX=at(5)), True), (dict(ws=at(4)), True), (dict(ws=at(0)), True),
    (dict(dX=None, dW=at(2)), False),      # W is not read without dX
    (dict(dX=at(3), act=0), False),        # nor Z for the identity
    (dict(X=at(2)), False),
])
def test_linear_backward_outputs_over_operands(kw, refused):
    a = dict(dY=at(0), X=at(1), W=at(2), Z=at(3), act=1, dX=at(4), dW=at(5), db=at(6), ws=at(7))
    a.update(kw)
    need = lib.hsq_linear_backward_workspace_bytes(64, 256, 256)
    _status(lib.hsq_linear_backward, (a["dY"], hsq.BF16, a["X"], 64, 256, 256, hsq.BF16, a["W"], a["Z"], a["act"],
                                      a["dX"], a["dW"], a["db"], a["ws"], need, None), refused)


@pytest.mark.parametrize("kw,refused", [
    (dict(), False), (dict(Y=at(0)), False), (dict(xdt=hsq.F32, Y=at(0)), True), (dict(Y=at(0) + 512), True),
    (dict(Y=at(1)), True), (dict(Y=at(2)), True), (dict(mean=at(5)), True), (dict(mean=at(0)), True),
    (dict(rstd=at(4) + 240), True), (dict(rstd=at(4) + 256), False), (dict(rstd=at(3)), True), (dict(w=at(2)), False),
])
def test_layer_norm_outputs_over_operands(kw, refused):
    a = dict(X=at(0), xdt=hsq.BF16, w=at(1), b=at(2), Y=at(3), mean=at(4), rstd=at(5))
    a.update(kw)
    _status(lib.hsq_layer_norm, (a["X"], a["xdt"], 64, 256, 1, a["w"], a["b"], hsq.F32, 1e-5, a["Y"], hsq.BF16,
                                 a["mean"], a["rstd"], None), refused)


@pytest.mark.parametrize("kw,refused", [
    (dict(), False), (dict(dX=at(0)), True), (dict(dX=at(1)), True), (dict(dw=at(2)), True), (dict(db=at(3)), True),
    (dict(dw=at(7)), True), (dict(db=at(4)), True), (dict(ws=at(5)), True), (dict(ws=at(1)), True),
    (dict(dw=None, db=None, ws=at(1)), False),       # the workspace is not used then
])
def test_layer_norm_backward_outputs_over_operands(kw, refused):
    a = dict(dY=at(0), X=at(1), mean=at(2), rstd=at(3), w=at(4), dX=at(5), dw=at(6), db=at(7), ws=at(8))
    a.update(kw)
    need = lib.hsq_layer_norm_backward_workspace_bytes(64, 256, 1)
    _status(lib.hsq_layer_norm_backward, (a["dY"], hsq.BF16, a["X"], hsq.BF16, 64, 256, 1, a["mean"], a["rstd"],
                                          a["w"], hsq.F32, a["dX"], a["dw"], a["db"], a["ws"], need, None), refused)
