"""The layer with 16-bit activations, the 4-bit cache and the attention over it
on the host: sizes, refusals of the C ABI and of the binding before anything is
enqueued, and the definitions that the GPU tests compare with."""

import math
import re

import pytest
import torch

import w4a4_rank_assisted_amd as hsq
from decode_ref import attention64, held64, scales64

lib = hsq._load()
GAP = 1 << 28
A = 0x10000000         # fake device addresses, far apart: validation rejects before use
NO_GPU = not torch.cuda.is_available()


def at(i):
    return A + i * GAP


def refused(st, code):
    if code is None:
        if not NO_GPU:
            pytest.skip("a launch on made-up addresses")
        assert st == hsq.E_HIP        # reached the launch, which fails without a GPU
    else:
        assert st == code


def w4a16(**kw):
    a = dict(X=at(0), M=16, K=256, N=96, b=1, group=64, dt=hsq.BF16, lam=at(1), w=at(2), sw=at(3), L1=at(4), L2=at(5),
             r=4, bias=at(6), res=at(7), Y=at(8), ydt=hsq.BF16, ws=at(9), wsb=1 << 20)
    a.update(kw)
    return lib.hsq_w4a16_lowrank_linear(a["X"], a["M"], a["K"], a["N"], a["b"], a["group"], a["dt"], a["lam"], a["w"],
                                        a["sw"], a["L1"], a["L2"], a["r"], a["bias"], a["res"], a["Y"], a["ydt"],
                                        a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(), None), (dict(lam=None, r=0, L1=None, L2=None, ws=None, wsb=0), None), (dict(res=None, bias=None), None),
    (dict(Y=at(7)), None),                                                   # added in place
    (dict(X=None), hsq.E_INVAL), (dict(w=None), hsq.E_INVAL), (dict(sw=None), hsq.E_INVAL), (dict(Y=None), hsq.E_INVAL),
    (dict(L1=None), hsq.E_INVAL), (dict(L2=None), hsq.E_INVAL), (dict(M=0), hsq.E_INVAL), (dict(M=65), hsq.E_INVAL),
    (dict(N=0), hsq.E_INVAL), (dict(K=0), hsq.E_INVAL), (dict(K=100), hsq.E_SHAPE), (dict(K=192, group=128), hsq.E_SHAPE),
    (dict(group=32), hsq.E_INVAL), (dict(b=0), hsq.E_INVAL), (dict(b=17), hsq.E_INVAL), (dict(r=33), hsq.E_INVAL),
    (dict(r=-1), hsq.E_INVAL), (dict(dt=hsq.F32), hsq.E_INVAL), (dict(ydt=hsq.F16), hsq.E_INVAL),
    (dict(K=1 << 16, N=1 << 15), hsq.E_INVAL), (dict(ws=None), hsq.E_WORKSPACE), (dict(wsb=100), hsq.E_WORKSPACE),
    (dict(X=at(0) + 2), hsq.E_ALIGN), (dict(lam=at(1) + 8), hsq.E_ALIGN), (dict(Y=at(8) + 4), hsq.E_ALIGN),
    (dict(res=at(7) + 2), hsq.E_ALIGN), (dict(ws=at(9) + 8), hsq.E_ALIGN),
    (dict(Y=at(0)), hsq.E_INVAL), (dict(Y=at(2)), hsq.E_INVAL), (dict(Y=at(7) + 16), hsq.E_INVAL),
    (dict(Y=at(9)), hsq.E_INVAL), (dict(ws=at(4)), hsq.E_INVAL), (dict(X=at(3)), None),
])
def test_w4a16(kw, code):
    refused(w4a16(**kw), code)


def kv_where(a):
    return (a["table"], a["width"], a["lens"], a["cu"], a["b"])


KV = dict(T=12, H=2, D=64, quant=1, cache=at(0), pages=8, page=64, table=at(1), width=4, lens=at(2), cu=at(3), b=3,
          top=12)


def write(**kw):
    a = dict(KV, K=at(4), ks=128, V=at(5), vs=128, dt=hsq.BF16)
    a.update(kw)
    return lib.hsq_kv_cache_write(a["K"], a["ks"], a["V"], a["vs"], a["T"], a["dt"], a["H"], a["D"], a["quant"],
                                  a["cache"], a["pages"], a["page"], *kv_where(a), a["top"], None)


def read(**kw):
    a = dict(KV, K=at(4), V=at(5), dt=hsq.F32)
    a.update(kw)
    return lib.hsq_kv_cache_read(a["cache"], a["pages"], a["page"], a["H"], a["D"], *kv_where(a), a["T"], a["top"],
                                 a["K"], a["V"], a["dt"], None)


def attend(**kw):
    a = dict(KV, Q=at(4), qs=256, Hq=4, dt=hsq.BF16, scale=0.125, causal=1, window=0, Y=at(5), ydt=hsq.BF16, lse=at(6),
             ws=at(7), wsb=1 << 24)
    a.update(kw)
    return lib.hsq_kv_attention(a["Q"], a["qs"], a["T"], a["dt"], a["Hq"], a["cache"], a["pages"], a["page"], a["H"],
                                a["D"], *kv_where(a), a["top"], a["scale"], a["causal"], a["window"], a["Y"], a["ydt"],
                                a["lse"], a["ws"], a["wsb"], None)


WHERE = [
    (dict(T=0), hsq.E_INVAL), (dict(T=(1 << 24) + 1), hsq.E_INVAL), (dict(b=0), hsq.E_INVAL),
    (dict(b=65536, T=65536), hsq.E_INVAL), (dict(H=0), hsq.E_INVAL), (dict(D=96), hsq.E_SHAPE), (dict(D=0), hsq.E_SHAPE),
    (dict(D=32), hsq.E_SHAPE), (dict(page=16), hsq.E_SHAPE), (dict(page=96), hsq.E_SHAPE), (dict(page=1 << 21), hsq.E_SHAPE),
    (dict(page=0), hsq.E_SHAPE), (dict(page=-64), hsq.E_SHAPE), (dict(pages=0), hsq.E_INVAL), (dict(width=0), hsq.E_INVAL),
    (dict(width=1 << 25), hsq.E_INVAL), (dict(cu=None, T=13), hsq.E_SHAPE), (dict(top=0), hsq.E_INVAL),
    (dict(top=-13), hsq.E_INVAL), (dict(cache=None), hsq.E_INVAL), (dict(table=None), hsq.E_INVAL),
    (dict(lens=None), hsq.E_INVAL), (dict(cache=at(0) + 8), hsq.E_ALIGN), (dict(table=at(1) + 2), hsq.E_ALIGN),
    (dict(lens=at(2) + 1), hsq.E_ALIGN), (dict(cu=at(3) + 2), hsq.E_ALIGN), (dict(table=at(1) + 4), None),
    (dict(cu=None, top=-9), None), (dict(b=65535, T=1 << 24, top=1 << 24), hsq.E_INVAL),
]


@pytest.mark.parametrize("kw,code", WHERE + [
    (dict(), None), (dict(K=None), hsq.E_INVAL), (dict(V=None), hsq.E_INVAL), (dict(dt=hsq.F32), hsq.E_INVAL),
    (dict(quant=2), hsq.E_INVAL), (dict(quant=-1), hsq.E_INVAL), (dict(ks=127), hsq.E_SHAPE), (dict(vs=120), hsq.E_SHAPE),
    (dict(ks=132), hsq.E_SHAPE), (dict(ks=136, vs=4096), None), (dict(K=at(4) + 2), hsq.E_ALIGN), (dict(K=at(0)), hsq.E_INVAL),
    (dict(V=at(0) + 8 * 64 * 2 * 70 - 16), hsq.E_INVAL), (dict(V=at(0) + 8 * 64 * 2 * 70), None),
    (dict(table=at(0)), hsq.E_INVAL), (dict(K=at(4), V=at(4)), None),
])
def test_kv_cache_write(kw, code):
    refused(write(**kw), code)


@pytest.mark.parametrize("kw,code", WHERE + [
    (dict(), None), (dict(dt=hsq.F16), None), (dict(K=None), hsq.E_INVAL), (dict(V=None), hsq.E_INVAL),
    (dict(dt=3), hsq.E_INVAL), (dict(K=at(4) + 4), hsq.E_ALIGN), (dict(K=at(5)), hsq.E_INVAL), (dict(K=at(0)), hsq.E_INVAL),
    (dict(K=at(2)), hsq.E_INVAL),
])
def test_kv_cache_read(kw, code):
    refused(read(**kw), code)


@pytest.mark.parametrize("kw,code", WHERE + [
    (dict(), None), (dict(lse=None), None), (dict(Q=None), hsq.E_INVAL), (dict(Y=None), hsq.E_INVAL),
    (dict(Hq=3), hsq.E_SHAPE), (dict(Hq=0), hsq.E_INVAL), (dict(Hq=4098), hsq.E_INVAL), (dict(dt=hsq.F32), hsq.E_INVAL),
    (dict(ydt=hsq.F16), hsq.E_INVAL), (dict(ydt=hsq.F32), None), (dict(scale=0.0), hsq.E_INVAL), (dict(scale=-1.0), hsq.E_INVAL),
    (dict(scale=math.nan), hsq.E_INVAL), (dict(scale=math.inf), hsq.E_INVAL), (dict(causal=2), hsq.E_INVAL),
    (dict(window=-1), hsq.E_INVAL), (dict(window=5), None), (dict(window=5, causal=0), hsq.E_INVAL), (dict(causal=0), None),
    (dict(qs=255), hsq.E_SHAPE), (dict(qs=260), hsq.E_SHAPE), (dict(Q=at(4) + 8), hsq.E_ALIGN), (dict(Y=at(5) + 8), hsq.E_ALIGN),
    (dict(lse=at(6) + 4), hsq.E_ALIGN), (dict(ws=at(7) + 4), hsq.E_ALIGN), (dict(Y=at(4)), hsq.E_INVAL),
    (dict(Y=at(0)), hsq.E_INVAL), (dict(lse=at(5)), hsq.E_INVAL), (dict(lse=at(1)), hsq.E_INVAL),
    (dict(width=400, page=1024, top=1, ws=None), hsq.E_WORKSPACE), (dict(width=400, page=1024, top=1, wsb=1000), hsq.E_WORKSPACE),
    (dict(width=400, page=1024, top=1, ws=at(4)), hsq.E_INVAL),
])
def test_kv_attention(kw, code):
    refused(attend(**kw), code)


def test_sizes():
    assert [lib.hsq_kv_page_bytes(32, 1, d) for d in (64, 128, 256)] == [2240, 4480, 8960]
    assert lib.hsq_kv_page_bytes(64, 8, 128) == 64 * 8 * 140
    for bad in ((16, 1, 64), (48, 1, 64), (32, 0, 64), (32, 1, 80), (32, 5000, 64), (1 << 21, 1, 64), (-32, 1, 64)):
        assert lib.hsq_kv_page_bytes(*bad) == 0
    f = lib.hsq_w4a16_workspace_bytes
    assert f(1, 4096, 4096, 0, 1, 64, 0, hsq.BF16) == f(1, 4096, 4096, 4, 1, 64, 1, hsq.F32) == 0   # one launch
    assert 0 < f(16, 4096, 4096, 4, 1, 64, 0, hsq.BF16) < f(16, 4096, 4096, 4, 1, 64, 1, hsq.BF16) < f(
        16, 4096, 4096, 4, 1, 64, 1, hsq.F32)
    for bad in ((65, 4096, 64, 4, 1, 64), (0, 64, 64, 4, 1, 64), (1, 96, 64, 4, 1, 64), (1, 192, 64, 4, 1, 128),
                (1, 64, 64, 33, 1, 64), (1, 64, 64, 4, 17, 64)):
        assert f(*bad, 1, hsq.F32) == 0
    for K in (64, 4096, 12288, 1 << 20, 1 << 24):
        assert f(64, K, 64, 32, 16, 64, 1, hsq.F32) < 1 << 35
    g = lib.hsq_kv_attention_workspace_bytes
    assert g(1, 32, 8, 128, 1, 1, 131072) > 0            # one sequence is split
    assert g(1024, 32, 8, 128, 1024, 1, 131072) == 0     # a large batch fills the chip
    assert g(2048, 32, 8, 128, 1, 2048, 131072) == 0     # and so does a prompt
    assert g(0, 32, 8, 128, 1, 1, 64) == 0 and g(1, 32, 5, 128, 1, 1, 64) == 0 and g(1, 32, 8, 96, 1, 1, 64) == 0
    # a bound on the rows that is larger never needs more
    for D in (64, 128, 256):
        for B in (1, 3, 16):
            last = None
            for m in (1, 2, 3, 5, 8, 13, 16, 40, 64, 200):
                n = g(200 * B, 8, 2, D, B, m, 1 << 17)
                assert last is None or n <= last
                last = n
    # above the rows there are it is their number
    assert g(5, 8, 2, 128, 1, 5, 1 << 17) == g(5, 8, 2, 128, 1, 6, 1 << 17) == g(5, 8, 2, 128, 1, 1 << 30, 1 << 17) > 0


def test_sizes_beyond_an_int():
    big = 1 << 32
    assert hsq.kv_page_bytes(big + 64, 8, 128) == 0 and hsq.w4a16_workspace_bytes(big + 1, 64, 64, 4) == 0
    assert hsq.kv_attention_workspace_bytes(big + 1, 32, 8, 128, 1, 1, 1024) == 0


def test_constants_match_header():
    consts = dict((k, int(v)) for k, v in re.findall(r"#define (HSQ_\w+)\s+(-?\d+)", open(hsq.HEADER).read()))
    assert consts["HSQ_W4A16_MAX_M"] == hsq.W4A16_MAX_M


def test_binding_refuses(monkeypatch):
    x, c = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 1, 2240, dtype=torch.uint8)
    t, n = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    k = torch.zeros(4, 1, 64, dtype=torch.bfloat16)
    for call in (lambda: hsq.w4a16_lowrank_linear(x, c, x, N=64), lambda: hsq.kv_cache_write(k, k, c, t, n),
                 lambda: hsq.kv_cache_read(c, t, n, tokens=4, head_dim=64), lambda: hsq.kv_attention(q, c, t, n)):
        with pytest.raises(ValueError, match="HIP device"):
            call()
    # host tensors stand for device tensors up to the call
    monkeypatch.setattr(hsq, "_device", lambda T, t, name: -1)
    blob = torch.zeros(hsq.packed_weight_bytes(64, 16), dtype=torch.uint8)
    sw = torch.zeros(1, 1, 16, dtype=torch.float16)
    for kw in (dict(packed_w=blob[:-1]), dict(sw=sw[:, :, :8]), dict(lam=torch.zeros(32, dtype=torch.float16)),
               dict(N=17), dict(group=32), dict(bias=torch.zeros(16, dtype=torch.bfloat16)), dict(batch=2),
               dict(residual=torch.zeros(4, 16, dtype=torch.bfloat16)), dict(y_dtype="f64")):
        a = dict(packed_w=blob, sw=sw, N=16)
        a.update(kw)
        with pytest.raises(ValueError):
            hsq.w4a16_lowrank_linear(x, **a)
    for kw in (dict(sw=sw.float()), dict(L1=torch.zeros(1, 64, 4), L2=torch.zeros(1, 4, 16)), dict(y_dtype="f16"),
               dict(bias=torch.zeros(1, 16))):
        a = dict(packed_w=blob, sw=sw, N=16)
        a.update(kw)
        with pytest.raises(TypeError):
            hsq.w4a16_lowrank_linear(x, **a)
    for a in ((k, k, c[0], t, n), (k, k, c[:, :, :100].contiguous(), t, n), (k, k, c, t[0], n), (k, k, c, t, n[:0]),
              (q, q, c, t, n), (k, k[:3], c, t, n), (torch.zeros(4, 1, 128, dtype=torch.bfloat16)[:, :, ::2], k, c, t, n), (k, k, c, t, n, n)):
        with pytest.raises(ValueError):
            hsq.kv_cache_write(*a)
    for a in ((k, k, c.int(), t, n), (k, k, c, t.long(), n), (k, k.half(), c, t, n), (k.float(), k.float(), c, t, n)):
        with pytest.raises(TypeError):
            hsq.kv_cache_write(*a)
    with pytest.raises(ValueError):
        hsq.kv_cache_write(k, k, c, t, n, quant="int4")
    with pytest.raises(hsq.HsqError):
        hsq.kv_cache_read(c, t, n, tokens=4, head_dim=80)
    with pytest.raises(ValueError):
        hsq.kv_cache_read(c, t, n, tokens=4, head_dim=64, dtype="f64")
    with pytest.raises(ValueError):
        hsq.kv_attention(torch.zeros(4, 4, 64, dtype=torch.bfloat16)[:, ::2], c, t, n)    # heads apart
    with pytest.raises(ValueError):
        hsq.kv_attention(torch.zeros(4, 132, dtype=torch.bfloat16)[:, :128].unflatten(1, (2, 64)), c, t, n)
    with pytest.raises(TypeError):
        hsq.kv_attention(q, c, t, n, y_dtype="f16")
    with pytest.raises(hsq.HsqError):
        hsq.kv_attention(q, c, t, n, window=-1)
    with pytest.raises(hsq.HsqError):
        hsq.kv_cache(0, 1, 64)
    with pytest.raises(hsq.HsqError):
        hsq.kv_cache(1, 1, 64, 48)


def test_binding_refuses_another_device(monkeypatch):
    class T(torch.Tensor):
        def get_device(self):
            return 1

    other = torch.zeros(4, 1, 64, dtype=torch.bfloat16).as_subclass(T)
    t, n, c = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, 2240, dtype=torch.uint8)
    monkeypatch.setattr(hsq._t(), "current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        hsq.kv_attention(other, c, t, n)
    monkeypatch.setattr(hsq._t(), "current_device", lambda: 1)
    with pytest.raises(ValueError, match="HIP device 1"):
        hsq.kv_cache_write(other, other, c, t, n)


# ------------------------------------------------------- the definitions
def test_held_values_of_a_hand_group():
    x = torch.zeros(1, 1, 64)
    x[0, 0, :5] = torch.tensor([-4.0, 11.0, 0.5, 1.5, 2.6])      # scale 1, zero 4
    assert held64(x, "asym")[0, 0, :6].tolist() == [-4.0, 11.0, 0.0, 2.0, 3.0, 0.0]
    assert scales64(x, "asym").item() == 1.0
    x[0, 0, :5] = torch.tensor([-7.0, 3.5, 2.5, -0.6, 6.4])      # scale 1
    assert held64(x, "sym")[0, 0, :5].tolist() == [-7.0, 4.0, 2.0, -1.0, 6.0]


@pytest.mark.parametrize("quant,levels", [("asym", 15), ("sym", 14)])
def test_held_values_are_near(quant, levels):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(50, 2, 128, generator=g)
    v = x.view(50, 2, 2, 64)
    span = v.amax(-1).clamp(min=0) - v.amin(-1).clamp(max=0) if quant == "asym" else 2 * v.abs().amax(-1)
    # half a step and, asymmetric, another for the zero's rounding; the scale's rounding moves 15 steps by 2^-11
    step = span.double() / levels
    err = (held64(x, quant) - x).view(50, 2, 2, 64).abs().amax(-1)
    assert bool((err <= step * ((1.0 if quant == "asym" else 0.5) + 16 * 2.0 ** -11)).all())


def test_attention_of_a_hand_row():
    k = torch.zeros(3, 1, 64, dtype=torch.float64)
    v = torch.zeros_like(k)
    k[:, 0, 0] = torch.tensor([0.0, math.log(3.0), 50.0])
    v[:, 0, 5] = torch.tensor([1.0, 5.0, 100.0])
    Q = torch.zeros(2, 1, 64)
    Q[:, 0, 0] = 1.0
    s = torch.ones(3, 1, 1)
    y, lse, _, _ = attention64(Q, k, v, s, s, 0, 1.0, True, 0, torch.float32)
    assert y[0, 0, 5] == 1.0 and y[1, 0, 5].item() == pytest.approx(4.0) and lse[1, 0].item() == pytest.approx(math.log(4))
    y, lse, _, _ = attention64(Q, k, v, s, s, -1, 1.0, True, 0, torch.float32)
    assert y[0].abs().max() == 0 and lse[0, 0] == -math.inf and y[1, 0, 5] == 1.0
    y, _, _, _ = attention64(Q, k, v, s, s, 0, 1.0, True, 1, torch.float32)
    assert y[1, 0, 5] == 5.0


def test_attention_against_a_softmax():
    g = torch.Generator().manual_seed(4)
    Q = torch.randn(5, 4, 64, generator=g)
    k, v = (torch.randn(20, 2, 64, generator=g).double() for _ in range(2))
    s = torch.ones(20, 2, 1)
    y, lse, _, _ = attention64(Q, k, v, s, s, 15, 0.125, True, 0, torch.float32)
    for h in range(4):
        e = 0.125 * Q[:, h].double() @ k[:, h // 2].T
        e = e.masked_fill(torch.arange(20)[None] > torch.arange(15, 20)[:, None], -math.inf)
        assert torch.allclose(y[:, h], torch.softmax(e, 1) @ v[:, h // 2], atol=1e-12)
        assert torch.allclose(lse[:, h], torch.logsumexp(e, 1), atol=1e-12)
