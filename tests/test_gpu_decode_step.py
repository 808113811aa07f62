"""The operators of a decoding step together, as a program uses them: projections
with 4-bit weights, keys and values into the cache, attention, the output
projection onto the residual; eager, captured and replayed, on other streams and
from several host threads."""

import math
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from decode_ref import attention64, held64, scales64, w4a16_64  # noqa: E402
from test_gpu_kv_cache import DEV, i32, pages_for  # noqa: E402

C, HQ, H, D, PAGE, R = 512, 8, 2, 64, 32, 4


class Block:
    """One attention block: joint q, k, v projection, output projection."""

    def __init__(self, seed, dt=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)

        def weights(K, N):
            w = dict(codes=torch.randint(-8, 8, (1, K, N), generator=g, dtype=torch.int8),
                     sw=(0.25 / math.sqrt(K) * (0.5 + torch.rand(1, K // 64, N, generator=g))).half(),
                     lam=(0.5 + torch.rand(K, generator=g)).half(),
                     L1=(torch.randn(1, K, R, generator=g) / math.sqrt(K)).to(dt),
                     L2=(0.3 * torch.randn(1, R, N, generator=g)).to(dt))
            w = {k: v.to(DEV) for k, v in w.items()}
            w["packed"] = hsq.pack_weights(w["codes"][0])[0]
            return w

        self.qkv, self.o = weights(C, (HQ + 2 * H) * D), weights(HQ * D, C)

    def linear(self, w, X, residual=None, **kw):
        return hsq.w4a16_lowrank_linear(X, w["packed"], w["sw"], w["lam"], w["L1"], w["L2"], None, residual,
                                        N=w["codes"].shape[2], **kw)

    def step(self, x, cache, table, lens, cu=None, top=None, **kw):
        a = self.linear(self.qkv, x)[0].unflatten(1, (HQ + 2 * H, D))
        q, k, v = a[:, :HQ], a[:, HQ:HQ + H], a[:, HQ + H:]
        hsq.kv_cache_write(k, v, cache, table, lens, cu, max_tokens=top)
        y = hsq.kv_attention(q, cache, table, lens, cu, max_tokens=top, **kw)
        return self.linear(self.o, y.flatten(1), x[None])[0], (q, k, v, y)


def inputs(seed, n):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, C, generator=g).bfloat16().to(DEV)


def test_prompt_and_tokens_against_64_bits():
    b = Block(1)
    lens = [45, 7]
    table, n = pages_for([80, 80], PAGE)
    cache = torch.full_like(hsq.kv_cache(n, H, D, PAGE), 0xFF)
    ks, vs = [[], []], [[], []]
    done = [0, 0]
    for it in range(6):                      # ragged prompts, then single tokens
        new = lens if it == 0 else [1, 1]
        done = [d + m for d, m in zip(done, new)]
        x = inputs(10 + it, sum(new))
        out, (q, k, v, y) = b.step(x, cache, table, i32(*done), i32(0, new[0], sum(new)), max(new))
        want, tol = w4a16_64(x, b.qkv["codes"], b.qkv["sw"], b.qkv["lam"], b.qkv["L1"], b.qkv["L2"], None, None, 64,
                             torch.bfloat16)
        got = torch.cat([q, k, v], 1).flatten(1)
        assert bool(((got.double() - want[0]).abs() <= tol[0]).all())
        r = 0
        for s in range(2):
            ks[s].append(k[r:r + new[s]].clone())
            vs[s].append(v[r:r + new[s]].clone())
            kk, vv = torch.cat(ks[s]), torch.cat(vs[s])
            w, _, t, _ = attention64(q[r:r + new[s]].contiguous(), held64(kk, "asym"), held64(vv, "asym"),
                                     scales64(kk, "asym"), scales64(vv, "asym"), done[s] - new[s], D ** -0.5, True, 0,
                                     torch.bfloat16)
            assert bool(((y[r:r + new[s]].double() - w).abs() <= t).all())
            r += new[s]
        want, tol = w4a16_64(y.flatten(1), b.o["codes"], b.o["sw"], b.o["lam"], b.o["L1"], b.o["L2"], None, x[None], 64,
                             torch.bfloat16)
        assert bool(((out.double() - want[0]).abs() <= tol[0]).all())


@pytest.mark.parametrize("width", [4, 400])          # one workgroup a head, and parts that are joined
def test_captured_step_follows_its_inputs(width):
    b = Block(2)
    B = 3
    table, n = pages_for([PAGE * width] * B, PAGE, spare=0)
    lens = i32(5, 33, 0)
    x, out = inputs(20, B), torch.empty(B, C, dtype=torch.bfloat16, device=DEV)
    caches = [hsq.kv_cache(n, H, D, PAGE) for _ in range(2)]
    # the histories, and a first eager step before the capture
    for c in caches:
        b.step(inputs(21, 38), c, table, i32(5, 33, 0), i32(0, 5, 38, 38), 33)
    b.step(x, hsq.kv_cache(n, H, D, PAGE), table, lens + 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lens += 1
        y, _ = b.step(x, caches[0], table, lens)
        out.copy_(y)
    lens.copy_(i32(5, 33, 0))
    ref = i32(5, 33, 0)
    for it in range(5):
        x.copy_(inputs(30 + it, B))
        graph.replay()
        ref += 1
        want, _ = b.step(x, caches[1], table, ref)
        torch.cuda.synchronize()
        assert torch.equal(lens, ref) and torch.equal(out, want) and torch.equal(caches[0], caches[1])


def test_two_graphs_share_a_workspace():
    b = Block(3)
    table, n = pages_for([20000], 1024)
    cache = hsq.kv_cache(n, H, D, 1024)
    g = torch.Generator(device=DEV).manual_seed(1)
    k = torch.randn(20000, H, D, generator=g, device=DEV).bfloat16()
    hsq.kv_cache_write(k, k, cache, table, i32(20000))
    need = max(hsq.kv_attention_workspace_bytes(1, HQ, H, D, 1, 1, table.shape[1] * 1024),
               hsq.w4a16_workspace_bytes(1, C, (HQ + 2 * H) * D, R, smooth=True))
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    x, q = inputs(40, 1), k[:1].repeat(1, HQ // H, 1).contiguous()
    outs, graphs = [None, None], [torch.cuda.CUDAGraph() for _ in range(2)]
    fns = [lambda: hsq.kv_attention(q, cache, table, i32_20000, workspace=ws),
           lambda: b.linear(b.qkv, x, workspace=ws)]
    i32_20000 = i32(20000)
    want = [f().clone() for f in fns]
    torch.cuda.synchronize()
    for i in (0, 1):
        with torch.cuda.graph(graphs[i]):
            outs[i] = fns[i]()
    for it in range(6):
        graphs[it % 2].replay()
        if it == 3:
            ws.fill_(0xFF)
        torch.cuda.synchronize()
        assert torch.equal(outs[it % 2], want[it % 2])
        outs[it % 2].zero_()


def test_other_streams_and_threads():
    b = Block(4)
    table, n = pages_for([300], PAGE)
    x, hist = inputs(50, 1), inputs(51, 300)[:64]

    def one(stream, out, i):
        with torch.cuda.stream(stream):
            cache = hsq.kv_cache(n, H, D, PAGE)
            for j in range(4):
                b.step(hist, cache, table, i32(64 * (j + 1)))
            y, _ = b.step(x, cache, table, i32(257))
            out[i] = y.clone()
        stream.synchronize()

    want = [None]
    one(torch.cuda.current_stream(), want, 0)
    got, ts = [None] * 4, []
    for i in range(4):
        ts.append(threading.Thread(target=one, args=(torch.cuda.Stream(), got, i)))
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    for y in got:
        assert torch.equal(y, want[0])


def test_chunks_of_a_prompt_equal_the_whole():
    # the same tokens written at once or in pieces: the same cache, the same attention up to its rounding
    g = torch.Generator().manual_seed(60)
    k, v = (torch.randn(300, H, D, generator=g).bfloat16().to(DEV) for _ in range(2))
    Q = torch.randn(300, HQ, D, generator=g).bfloat16().to(DEV)
    table, n = pages_for([300], PAGE)
    c1, c2 = hsq.kv_cache(n, H, D, PAGE), hsq.kv_cache(n, H, D, PAGE)
    hsq.kv_cache_write(k, v, c1, table, i32(300))
    whole, l1 = hsq.kv_attention(Q, c1, table, i32(300), y_dtype="f32", return_lse=True)
    at = 0
    for m in (1, 30, 2, 200, 64, 3):
        s = slice(at, at + m)
        at += m
        hsq.kv_cache_write(k[s], v[s], c2, table, i32(at))
        y, l2 = hsq.kv_attention(Q[s], c2, table, i32(at), y_dtype="f32", return_lse=True)
        assert torch.allclose(y, whole[s], rtol=0, atol=2e-5) and torch.allclose(l1[s], l2, rtol=0, atol=2e-5)
    assert torch.equal(c1, c2)
