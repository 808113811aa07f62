"""Ragged batches given without a bound on their rows, as many sequences as a batch of
prompts has."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from decode_ref import attention64, held64, scales64  # noqa: E402
from test_gpu_kv_cache import DEV, i32, rows, same  # noqa: E402


def batch(B, most, D, H, seed):
    """Rows of 0 .. most - 1 each, behind up to 40 that are held already."""
    g = torch.Generator().manual_seed(seed)
    counts = torch.randint(0, most, (B,), generator=g)
    counts[0], counts[1], counts[-1] = 0, most - 1, 0
    held = torch.randint(0, 41, (B,), generator=g)
    lens = held + counts
    page = 32
    need = (lens + page - 1) // page
    table = torch.full((B, int(need.max()) + 1), -1, dtype=torch.int32)
    perm = torch.randperm(int(need.sum()), generator=g).to(torch.int32)
    at = 0
    for b in range(B):
        m = int(need[b])
        table[b, :m] = perm[at:at + m]
        at += m
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32)
    T = int(counts.sum())
    k, v = rows(seed + 1, T, H, D, torch.bfloat16), rows(seed + 2, T, H, D, torch.bfloat16)
    cache = torch.zeros_like(hsq.kv_cache(at, H, D, page))
    return k, v, cache, table.to(DEV), lens.to(torch.int32).to(DEV), cu.to(DEV), counts.tolist()


@pytest.mark.parametrize("B,most,D,H", [(2048, 17, 64, 8), (300, 400, 128, 8), (7, 90, 256, 2)])
def test_without_a_bound(B, most, D, H):
    k, v, cache, table, lens, cu, counts = batch(B, most, D, H, 400)
    T = k.shape[0]
    print(f"[ragged] B={B} T={T}", flush=True)
    bounded = cache.clone()
    hsq.kv_cache_write(k, v, cache, table, lens, cu)
    hsq.kv_cache_write(k, v, bounded, table, lens, cu, max_tokens=most)
    assert torch.equal(cache, bounded)
    a, b = hsq.kv_cache_read(cache, table, lens, cu, tokens=T, head_dim=D, dtype="f32")
    assert same(a.double(), held64(k, "asym")) and same(b.double(), held64(v, "asym"))
    Q = rows(409, T, 2 * H, D, torch.bfloat16)
    out = torch.full((T, 2 * H, D), 3.0, device=DEV)
    hsq.kv_attention(Q, cache, table, lens, cu, y_dtype="f32", out=out)
    # the tokens held before are zeros (a cache of zeros has scales of zero)
    at = cu.tolist()
    for s in sorted({1, 2, B // 3, B // 2, B - 2}):
        n, c = int(lens[s]), counts[s]
        if c == 0:
            continue
        r = slice(at[s], at[s + 1])
        full = torch.zeros(2, n, H, D, dtype=torch.float64, device=DEV)
        full[0, n - c:], full[1, n - c:] = held64(k[r], "asym"), held64(v[r], "asym")
        sc = torch.zeros(2, n, H, D // 64, dtype=torch.float64, device=DEV)
        sc[0, n - c:], sc[1, n - c:] = scales64(k[r], "asym"), scales64(v[r], "asym")
        want, _, tol, _ = attention64(Q[r], full[0], full[1], sc[0], sc[1], n - c, 1 / math.sqrt(D), True, 0, torch.float32)
        assert bool(((out[r].double() - want).abs() <= tol).all()), s
    assert bool((out != 3).all())


def test_one_row_each_without_a_bound():
    # 64 single tokens by cu_tokens
    B, H, D = 64, 2, 128
    k, v, cache, table, lens, cu, counts = batch(B, 60, D, H, 420)
    hsq.kv_cache_write(k, v, cache, table, lens, cu)
    Q = rows(421, B, 8, D, torch.bfloat16)
    each = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    y, lse = hsq.kv_attention(Q, cache, table, lens, each, y_dtype="f32", return_lse=True)
    z, l = hsq.kv_attention(Q, cache, table, lens, each, y_dtype="f32", return_lse=True, max_tokens=1)
    assert torch.equal(z, hsq.kv_attention(Q, cache, table, lens, y_dtype="f32"))
    for b in range(0, B, 5):
        n = int(lens[b])
        if n == 0:
            assert not y[b].any() and not z[b].any()
            continue
        x = [t.double() for t in hsq.kv_cache_read(cache, table[b:b + 1], lens[b:b + 1], tokens=n, head_dim=D, dtype="f32")]
        c = counts[b]
        sc = torch.zeros(2, n, H, D // 64, dtype=torch.float64, device=DEV)
        r = slice(int(cu[b]), int(cu[b + 1]))
        if c:
            sc[0, n - c:], sc[1, n - c:] = scales64(k[r], "asym"), scales64(v[r], "asym")
        want, wl, tol, tl = attention64(Q[b:b + 1], *x, sc[0], sc[1], n - 1, 1 / math.sqrt(D), True, 0, torch.float32)
        for got, gl in ((y, lse), (z, l)):
            assert bool(((got[b].double() - want[0]).abs() <= tol[0]).all())
            assert bool(((gl[b].double() - wl[0]).abs() <= tl[0]).all())


def test_starts_that_are_wrong_stay_inside():
    H, D, B = 1, 64, 40
    T = 4000
    k = rows(430, T, H, D, torch.bfloat16)
    guard = torch.full((3, T, H, D), 3.0, dtype=torch.float32, device=DEV)
    g = torch.Generator().manual_seed(431)
    table = torch.arange(B * 4, dtype=torch.int32, device=DEV).view(B, 4)
    cache = hsq.kv_cache(B * 4, H, D, 32)
    lens = torch.full((B,), 128, dtype=torch.int32, device=DEV)
    for _ in range(6):
        cu = torch.randint(-200, T + 300, (B + 1,), generator=g).to(torch.int32).to(DEV)
        hsq.kv_cache_write(k, k, cache, table, lens, cu)
        hsq.kv_cache_read(cache, table, lens, cu, tokens=T, head_dim=D, dtype="f32", out=(guard[1], torch.empty_like(guard[1])))
        hsq.kv_attention(k, cache, table, lens, cu, y_dtype="f32", out=guard[1])
    torch.cuda.synchronize()
    assert bool((guard[0] == 3).all()) and bool((guard[2] == 3).all())
