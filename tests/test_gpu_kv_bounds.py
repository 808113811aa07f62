"""max_tokens of the 4-bit cache's calls: rows of a sequence beyond it are left alone,
whatever tile or block they lie in."""

import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from decode_ref import held64  # noqa: E402
from test_gpu_kv_attention import fill  # noqa: E402
from test_gpu_kv_cache import DEV, i32, pages_for, rows, same  # noqa: E402


@pytest.mark.parametrize("D,page", [(64, 32), (128, 64), (256, 32)])
@pytest.mark.parametrize("start", [0, 5, 32, 40])
@pytest.mark.parametrize("top,counts", [(1, (5, 1)), (4, (30, 3)), (32, (100, 33)), (33, (70, 90))])
def test_write_and_read(D, page, start, top, counts):
    H, T = 2, sum(counts)
    k, v = rows(201, T, H, D, torch.bfloat16), rows(202, T, H, D, torch.bfloat16)
    lens = [start + c for c in counts]
    table, n = pages_for(lens, page)
    cu = i32(0, counts[0], T)
    got = torch.full_like(hsq.kv_cache(n, H, D, page), 0xA5)
    want = got.clone()
    hsq.kv_cache_write(k, v, got, table, i32(*lens), cu, max_tokens=top)
    # the same rows alone, at the same positions
    few = [min(c, top) for c in counts]
    sel = torch.cat([torch.arange(few[0]), counts[0] + torch.arange(few[1])]).to(DEV)
    hsq.kv_cache_write(k[sel], v[sel], want, table, i32(*(start + f for f in few)), i32(0, few[0], sum(few)))
    assert torch.equal(got, want)
    hsq.kv_cache_write(k, v, got, table, i32(*lens), cu)
    out = tuple(torch.full((T, H, D), 9.0, dtype=torch.float32, device=DEV) for _ in range(2))
    hsq.kv_cache_read(got, table, i32(*lens), cu, tokens=T, head_dim=D, dtype="f32", max_tokens=top, out=out)
    for o, x in zip(out, (k, v)):
        full = held64(x, "asym")
        for at, c, f in ((0, counts[0], few[0]), (counts[0], counts[1], few[1])):
            assert same(o[at:at + f].double(), full[at:at + f]) and bool((o[at + f:at + c] == 9).all())


@pytest.mark.parametrize("spare", [1, 200])                 # one part, and several
@pytest.mark.parametrize("ydt", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,H,D,top,count", [
    (4, 1, 64, 1, 9), (4, 2, 128, 1, 3), (4, 1, 256, 1, 2), (4, 1, 64, 2, 6), (8, 2, 128, 2, 9), (3, 1, 128, 2, 4),
    (4, 1, 256, 3, 20), (4, 1, 128, 5, 30), (4, 1, 64, 7, 25), (2, 1, 64, 33, 80), (4, 1, 128, 40, 200), (4, 2, 256, 40, 66),
])
def test_attention(Hq, H, D, top, count, ydt, spare):
    n = 1500
    k, v = rows(211, n, H, D, torch.bfloat16), rows(212, n, H, D, torch.bfloat16)
    cache, table = fill(k, v, [n], 32, spare=spare)
    T = count + 3
    Q = rows(213, T, Hq, D, torch.bfloat16)
    # two sequences of one history: `count` rows and three
    table = table.repeat(2, 1).contiguous()
    out = torch.full((T, Hq, D), 5.0, dtype=torch.float32 if ydt == "f32" else torch.bfloat16, device=DEV)
    _, lse = hsq.kv_attention(Q, cache, table, i32(n, n), i32(0, count, T), max_tokens=top, y_dtype=ydt, out=out, return_lse=True)
    assert bool((out[top:count] == 5).all()) and bool((out[count + min(top, 3):] == 5).all())
    few = [top, min(top, 3)]
    sel = torch.cat([torch.arange(few[0]), count + torch.arange(few[1])]).to(DEV)
    y, l = hsq.kv_attention(Q[sel], cache, table, i32(n - count + few[0], n - 3 + few[1]), i32(0, few[0], sum(few)),
                            max_tokens=top, y_dtype=ydt, return_lse=True)
    # the same rows, tokens and parts: the same bits
    assert torch.equal(out[sel], y) and torch.equal(lse[sel], l)
