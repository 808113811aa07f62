"""The 16-bit linear and the layer normalisation on the host: sizes,
refusals of the C ABI and of the binding before anything is enqueued, and the
definitions that the GPU tests compare with, checked against differences."""

import ctypes
import math

import pytest
import torch

import w4a4_rank_assisted_amd as hsq
from linear_norm_ref import act64, act_grad64, layer_norm64, layer_norm_backward64

lib = hsq._load()
A = 0x100000  # a 16-byte aligned fake device address: validation rejects before use


def _linear(**kw):
    a = dict(X=A, M=64, K=256, N=256, dt=hsq.BF16, W=A, bias=A, act=0, res=A, Y=A, ydt=hsq.BF16, Z=A, ws=A, wsb=0)
    a.update(kw)
    return lib.hsq_linear(a["X"], a["M"], a["K"], a["N"], a["dt"], a["W"], a["bias"], a["act"], a["res"], a["Y"],
                          a["ydt"], a["Z"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), hsq.E_INVAL), (dict(W=None), hsq.E_INVAL), (dict(Y=None), hsq.E_INVAL),
    (dict(M=0), hsq.E_INVAL), (dict(K=0), hsq.E_INVAL), (dict(N=-1), hsq.E_INVAL),
    (dict(dt=hsq.F32), hsq.E_INVAL), (dict(dt=3), hsq.E_INVAL), (dict(ydt=hsq.F16), hsq.E_INVAL),
    (dict(ydt=7), hsq.E_INVAL), (dict(act=4), hsq.E_INVAL), (dict(act=-1), hsq.E_INVAL),
    (dict(X=A + 2), hsq.E_ALIGN), (dict(W=A + 8), hsq.E_ALIGN), (dict(bias=A + 4), hsq.E_ALIGN),
    (dict(res=A + 2), hsq.E_ALIGN), (dict(Y=A + 8), hsq.E_ALIGN), (dict(Z=A + 2), hsq.E_ALIGN),
    (dict(ws=A + 1), hsq.E_ALIGN),
    (dict(M=1 << 18, K=1 << 12), hsq.E_INVAL),             # M * K = 2^30
    (dict(K=1 << 15, N=1 << 15, M=1), hsq.E_INVAL),        # K * N = 2^30
    (dict(M=1 << 27, K=1, N=1), hsq.E_INVAL),              # rows of 1 rounded up to 8: 2^30
    (dict(M=1, K=1, N=(1 << 24) + 1), hsq.E_INVAL), (dict(M=1, K=(1 << 24) + 1, N=1), hsq.E_INVAL),
    (dict(M=4333, K=1001, N=4777, wsb=0), hsq.E_WORKSPACE),  # many ragged rows are staged
    (dict(M=4333, K=1001, N=4777, ws=None, wsb=1 << 30), hsq.E_WORKSPACE),
])
def test_linear_refusals(kw, code):
    assert _linear(**kw) == code


def _linear_backward(**kw):
    a = dict(dY=A, ydt=hsq.BF16, X=A, M=64, K=256, N=256, dt=hsq.BF16, W=A, Z=A, act=1, dX=A, dW=A, db=A, ws=A,
             wsb=1 << 30)
    a.update(kw)
    return lib.hsq_linear_backward(a["dY"], a["ydt"], a["X"], a["M"], a["K"], a["N"], a["dt"], a["W"], a["Z"],
                                   a["act"], a["dX"], a["dW"], a["db"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dY=None), hsq.E_INVAL), (dict(dX=None, dW=None, db=None), hsq.E_INVAL),
    (dict(W=None), hsq.E_INVAL), (dict(X=None), hsq.E_INVAL), (dict(Z=None), hsq.E_INVAL),
    (dict(ws=None), hsq.E_INVAL), (dict(act=4), hsq.E_INVAL), (dict(dt=0), hsq.E_INVAL),
    (dict(ydt=hsq.F16), hsq.E_INVAL), (dict(M=0), hsq.E_INVAL), (dict(M=1 << 27, N=1), hsq.E_INVAL),
    (dict(dY=A + 2), hsq.E_ALIGN), (dict(dX=A + 2), hsq.E_ALIGN), (dict(dW=A + 4), hsq.E_ALIGN),
    (dict(db=A + 8), hsq.E_ALIGN), (dict(Z=A + 8), hsq.E_ALIGN), (dict(wsb=1000), hsq.E_WORKSPACE),
])
def test_linear_backward_refusals(kw, code):
    assert _linear_backward(**kw) == code


def _norm(**kw):
    a = dict(X=A, xdt=hsq.BF16, M=64, C=256, G=1, w=A, b=A, pdt=hsq.F32, eps=1e-5, Y=A, ydt=hsq.BF16, mean=A, rstd=A)
    a.update(kw)
    return lib.hsq_layer_norm(a["X"], a["xdt"], a["M"], a["C"], a["G"], a["w"], a["b"], a["pdt"], a["eps"], a["Y"],
                              a["ydt"], a["mean"], a["rstd"], None)


SIZES = [
    (dict(M=0), hsq.E_INVAL), (dict(C=0), hsq.E_INVAL), (dict(C=16385), hsq.E_INVAL), (dict(G=0), hsq.E_INVAL),
    (dict(G=65536, M=65536), hsq.E_INVAL), (dict(G=5), hsq.E_SHAPE), (dict(M=1 << 20, C=1 << 11), hsq.E_INVAL),
    (dict(M=(1 << 25) + 1, C=2), hsq.E_INVAL),
    (dict(xdt=3), hsq.E_INVAL), (dict(ydt=hsq.F32), hsq.E_INVAL), (dict(ydt=hsq.F16), hsq.E_INVAL),
    (dict(pdt=hsq.F16), hsq.E_INVAL), (dict(xdt=hsq.F32, ydt=hsq.F32, pdt=hsq.BF16), hsq.E_INVAL),
    (dict(X=None), hsq.E_INVAL), (dict(X=A + 2), hsq.E_ALIGN), (dict(w=A + 4), hsq.E_ALIGN),
    (dict(mean=A + 4), hsq.E_ALIGN),
]


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(Y=None), hsq.E_INVAL), (dict(eps=-1.0), hsq.E_INVAL), (dict(eps=float("nan")), hsq.E_INVAL),
    (dict(eps=float("inf")), hsq.E_INVAL), (dict(b=A + 8), hsq.E_ALIGN), (dict(Y=A + 2), hsq.E_ALIGN),
])
def test_layer_norm_refusals(kw, code):
    assert _norm(**kw) == code


def _norm_backward(**kw):
    a = dict(dY=A, ydt=hsq.BF16, X=A, xdt=hsq.BF16, M=64, C=256, G=1, mean=A, rstd=A, w=A, pdt=hsq.F32, dX=A, dw=A,
             db=A, ws=A, wsb=1 << 30)
    a.update(kw)
    return lib.hsq_layer_norm_backward(a["dY"], a["ydt"], a["X"], a["xdt"], a["M"], a["C"], a["G"], a["mean"],
                                       a["rstd"], a["w"], a["pdt"], a["dX"], a["dw"], a["db"], a["ws"], a["wsb"],
                                       None)


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(dY=None), hsq.E_INVAL), (dict(mean=None), hsq.E_INVAL), (dict(rstd=None), hsq.E_INVAL),
    (dict(dX=None, dw=None, db=None), hsq.E_INVAL), (dict(ws=None), hsq.E_WORKSPACE), (dict(wsb=0), hsq.E_WORKSPACE),
    (dict(dX=A + 2), hsq.E_ALIGN), (dict(dw=A + 2), hsq.E_ALIGN), (dict(db=A + 2), hsq.E_ALIGN),
])
def test_layer_norm_backward_refusals(kw, code):
    assert _norm_backward(**kw) == code


def test_workspace_sizes():
    f, b, n = (lib.hsq_linear_workspace_bytes, lib.hsq_linear_backward_workspace_bytes,
               lib.hsq_layer_norm_backward_workspace_bytes)
    assert f(0, 64, 64) == 0 and b(64, 0, 64) == 0 and n(0, 64, 1) == 0 and n(6, 64, 4) == 0
    assert f(4096, 1152, 4608) == 0                       # whole rows, enough tiles: nothing to stage
    assert f(4333, 1001, 4777) >= 2 * (4333 * 1008 + 1001 * 4784)
    assert b(4333, 4001, 4777) >= 2 * (4333 * 4008 + 4001 * 4784 + 4333 * 4784)
    assert n(8192, 1152, 2) % (2 * 2 * 1152 * 4) == 0 and n(8192, 1152, 2) > 0
    for M, K, N in [(1, 1, 1), (1, 4096, 12288), (64, 12288, 4096), (65, 7, 9), (8192, 12288, 4096)]:
        assert f(M, K, N) < 1 << 31 and 0 < b(M, K, N) < 1 << 33


def test_chain_refuses_the_linear_only_activations():
    for act in (2, 3):
        assert lib.hsq_w4a4_lowrank_mlp(A, 64, 256, 512, 256, A, A, A, A, A, 4, A, act, A, A, A, A, A, 4, A, A,
                                        hsq.BF16, None, A, 1 << 30, None) == hsq.E_INVAL


def test_constants_match_header():
    import re

    consts = dict((k, int(v)) for k, v in re.findall(r"#define (HSQ_\w+)\s+(-?\d+)", open(hsq.HEADER).read()))
    assert consts["HSQ_F16"] == hsq.F16 and consts["HSQ_ACT_GELU"] == hsq.ACT_GELU
    assert consts["HSQ_ACT_SILU"] == hsq.ACT_SILU


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="HIP device"):
        hsq.linear(x, torch.zeros(8, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="HIP device"):
        hsq.linear_backward(x, x, x)
    with pytest.raises(ValueError, match="HIP device"):
        hsq.layer_norm(x)
    with pytest.raises(ValueError, match="HIP device"):
        hsq.layer_norm_backward(x, x, x, x)


def test_binding_refuses_shapes_and_types(monkeypatch):
    # host tensors stand for device tensors up to the call: both are on "device" -1
    monkeypatch.setattr(hsq, "_device", lambda T, t, name: -1)
    bf, f16, f32 = torch.bfloat16, torch.float16, torch.float32
    x, w = torch.zeros(4, 8, dtype=bf), torch.zeros(8, 16, dtype=bf)
    for bad in (torch.zeros(7, 16, dtype=bf), torch.zeros(8, dtype=bf)):
        with pytest.raises(ValueError):
            hsq.linear(x, bad)
        with pytest.raises(ValueError):
            hsq.linear_backward(x, x, bad)
    with pytest.raises(TypeError):
        hsq.linear(x, w.to(f16))
    with pytest.raises(TypeError):
        hsq.linear(x.float(), w.float())
    with pytest.raises(ValueError):
        hsq.linear(x, w, act="relu")
    with pytest.raises(ValueError):
        hsq.linear(x, w, y_dtype="f64")
    with pytest.raises(TypeError):
        hsq.linear(x, w, y_dtype="f16")
    with pytest.raises(ValueError):
        hsq.linear(x, w, torch.zeros(8, dtype=bf))
    with pytest.raises(TypeError):
        hsq.linear(x, w, residual=torch.zeros(4, 16, dtype=f32))
    with pytest.raises(ValueError):
        hsq.linear(x.t(), w)
    with pytest.raises(ValueError):
        hsq.layer_norm(x, torch.zeros(7, dtype=bf))
    with pytest.raises(ValueError):
        hsq.layer_norm(x, torch.zeros(2, 8, dtype=bf), torch.zeros(8, dtype=bf))
    with pytest.raises(ValueError):
        hsq.layer_norm(x, torch.zeros(8, dtype=bf), torch.zeros(8, dtype=f32))
    with pytest.raises(TypeError):
        hsq.layer_norm(x, torch.zeros(8, dtype=f16))
    with pytest.raises(TypeError):
        hsq.layer_norm(x, y_dtype="f32")
    st = torch.zeros(4)
    with pytest.raises(TypeError):
        hsq.layer_norm_backward(x.float(), x, st, st)
    with pytest.raises(ValueError):
        hsq.layer_norm_backward(x, x, st[:3], st)
    with pytest.raises(ValueError):
        hsq.layer_norm_backward(x, x, st, st, torch.zeros(2, 8, dtype=bf), groups=4)


def test_binding_refuses_another_device(monkeypatch):
    class T(torch.Tensor):
        def get_device(self):
            return 1

    other = torch.zeros(4, 8, dtype=torch.bfloat16).as_subclass(T)
    monkeypatch.setattr(hsq._t(), "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        hsq.layer_norm(other)
    with pytest.raises(ValueError, match="current device"):
        hsq.linear(other, other)
    monkeypatch.setattr(hsq._t(), "current_device", lambda: 1)
    with pytest.raises(ValueError, match="HIP device 1"):      # X there, W on the host
        hsq.linear(other, torch.zeros(8, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="HIP device 1"):
        hsq.layer_norm(other, torch.zeros(8, dtype=torch.bfloat16))


# ------------------------------------------------------- the definitions
@pytest.mark.parametrize("act", ["identity", "gelu_tanh", "gelu", "silu"])
def test_activation_derivative_against_differences(act):
    # central differences of step h: truncation h^2 |f'''| / 6 with |f'''| < 4,
    # rounding 2^-52 (|f| + 1) / h
    z = torch.linspace(-9, 9, 2001, dtype=torch.float64)
    h = 1e-5
    num = (act64(z + h, act) - act64(z - h, act)) / (2 * h)
    tol = h * h + 16 * 2.0 ** -52 * (z.abs() + 1) / h
    assert ((num - act_grad64(z, act)).abs() <= tol).all()


@pytest.mark.parametrize("groups", [1, 3])
def test_layer_norm_gradient_against_differences(groups):
    g = torch.Generator().manual_seed(7)
    M, C = 6, 13
    x, dy = (torch.randn(M, C, generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(groups, C, generator=g, dtype=torch.float64) for _ in range(2))
    y, mean, rstd = layer_norm64(x, w, b, 1e-5)
    dx, dw, db = layer_norm_backward64(dy, x, mean, rstd, w)
    h = 1e-5
    for t, grad in ((x, dx), (w, dw), (b, db)):
        v = torch.randn(t.shape, generator=g, dtype=torch.float64)
        out = []
        for sgn in (1, -1):
            t += sgn * h * v
            out.append((layer_norm64(x, w, b, 1e-5)[0] * dy).sum())
            t -= sgn * h * v
        num = (out[0] - out[1]) / (2 * h)
        assert abs(num - (grad * v).sum()) <= 1e-6 * (1 + (grad.abs() * v.abs()).sum())


def test_layer_norm_of_a_hand_row():
    x = torch.tensor([[1.0, 2.0, 3.0, 6.0]], dtype=torch.float64)     # mean 3, variance (4 + 1 + 0 + 9) / 4
    y, mean, rstd = layer_norm64(x, None, None, 0.5)
    assert mean.item() == 3.0 and rstd.item() == 0.5                  # 3.5 + 0.5 = 4
    assert y.tolist() == [[-1.0, -0.5, 0.0, 1.5]]


def test_gelu_values():
    z = torch.tensor([0.0, 1.0, -1.0], dtype=torch.float64)
    phi = 0.5 * (1 + math.erf(1 / math.sqrt(2)))
    assert torch.allclose(act64(z, "gelu"), torch.tensor([0.0, phi, phi - 1], dtype=torch.float64))
    assert ctypes.c_float(act64(z, "silu")[1].item()).value == pytest.approx(1 / (1 + math.exp(-1)), rel=1e-7)
