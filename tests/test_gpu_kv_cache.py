"""The 4-bit cache on the GPU: what is read back is the definition's value, bit
for bit, and nothing else of the cache or of the outputs is touched."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from decode_ref import held64  # noqa: E402

DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def pages_for(lens, page, seed=0, spare=1):
    """A block table of shuffled pages, and their number (one more than used)."""
    need = [max(1, -(-n // page)) for n in lens]
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(sum(need) + 1, generator=g)[:sum(need)].to(torch.int32)
    table = torch.full((len(lens), max(need) + spare), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    return table.to(DEV), sum(need) + 1


def rows(seed, T, H, D, dt):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g) * (0.3 + torch.rand(H, D, generator=g))
    x[:, :, ::17] += 4.0
    return x.to(dt).to(DEV)


def same(a, b):
    """Equal, NaN where NaN."""
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("quant", ["asym", "sym"])
@pytest.mark.parametrize("H,D,page,lens", [
    (1, 64, 32, [1]), (2, 64, 32, [31, 32, 33]), (5, 64, 128, [1, 257, 64]), (8, 128, 64, [65, 1000]),
    (3, 128, 32, [500, 7, 95]), (1, 256, 256, [300]), (2, 256, 32, [33, 64]),
])
def test_values_read_back(H, D, page, lens, quant, dt):
    print(f"[kv] H={H} D={D} page={page} lens={lens} {quant} {dt}", flush=True)
    T = sum(lens)
    k, v = rows(1, T, H, D, DT[dt]), rows(2, T, H, D, DT[dt])
    table, n = pages_for(lens, page)
    cache = hsq.kv_cache(n, H, D, page)
    cu = i32(0, *lens).cumsum(0).to(torch.int32)
    hsq.kv_cache_write(k, v, cache, table, i32(*lens), cu, quant=quant)
    for out in ("f32", "bf16", "f16"):
        a, b = hsq.kv_cache_read(cache, table, i32(*lens), cu, tokens=T, head_dim=D, dtype=out)
        for got, x in ((a, k), (b, v)):
            want = held64(x, quant)
            assert same(got, want.to(DT["f32"]).to(DT[out]))
            if out == "f32":
                assert same(got.double(), want)     # 16 bits: fp32 holds the product


@pytest.mark.parametrize("quant", ["asym", "sym"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_ties_extremes_and_what_is_not_finite(quant, dt):
    D, T = 64, 24
    x = torch.zeros(T, 1, D)
    step = torch.arange(64) % 16
    x[0, 0] = (step - 7.5).clamp(-7, 7) + 0.0          # halves: ties at scale 1 (sym)
    x[1, 0] = step * 1.0                               # scale 1 (asym)
    x[2, 0] = (step - 0.5).clamp(0, 15)                # ties at scale 1 (asym)
    x[2, 0, 0] = 15.0
    x[3, 0] = (step - 4.5)                             # ties about a zero point
    x[3, 0, 0], x[3, 0, 1] = -4.0, 11.0
    x[4, 0] = 6e4                                      # one value
    x[5, 0] = -6e4
    x[6, 0, 3] = 2.0 ** -24
    x[7, 0, 5] = -(2.0 ** -20)
    x[8, 0] = torch.linspace(-6e4, 6e4, 64)
    x[9, 0, 7] = math.inf
    x[10, 0, 8] = -math.inf
    x[11, 0, 9] = math.nan
    x[11, 0, 10] = 5.0
    x[12, 0] = torch.linspace(1e-6, 9e-6, 64)          # subnormal scales
    x[13, 0] = -torch.linspace(0.5, 1.0, 64)           # all of one sign
    x[14, 0] = torch.linspace(0.25, 0.75, 64)
    if dt == "bf16":
        x[15, 0] = torch.linspace(-3e38, 3e38, 64)     # the scale saturates
        x[16, 0] = 1e-38
        x[17, 0] = torch.linspace(-1e6, 3e6, 64)
    x[18:] = torch.randint(-28, 29, (6, 1, D)).float() / 4   # many ties
    x[18:, 0, 0] = 7.0
    k = x.to(DT[dt]).to(DEV)
    v = k.flip(0).contiguous()
    table, n = pages_for([T], 32)
    cache = hsq.kv_cache(n, 1, D, 32)
    hsq.kv_cache_write(k, v, cache, table, i32(T), quant=quant)
    a, b = hsq.kv_cache_read(cache, table, i32(T), tokens=T, head_dim=D, dtype="f32")
    assert same(a.double(), held64(k, quant)) and same(b.double(), held64(v, quant))


@pytest.mark.parametrize("D,page", [(64, 32), (128, 64), (256, 32)])
def test_piecewise_equals_whole_and_leaves_the_rest(D, page):
    H, lens = 3, [97, 200]
    T = sum(lens)
    k, v = rows(3, T, H, D, torch.bfloat16), rows(4, T, H, D, torch.bfloat16)
    table, n = pages_for(lens, page)
    whole, parts = (torch.full_like(hsq.kv_cache(n, H, D, page), 0xA5) for _ in range(2))
    cu = i32(0, *lens).cumsum(0).to(torch.int32)
    hsq.kv_cache_write(k, v, whole, table, i32(*lens), cu)
    done = [0, 0]
    for steps in ([1, 1], [30, 33], [1, 0], [2, 95], [40, 1], [23, 70]):
        sel = torch.cat([torch.arange(off + d, off + d + s) for off, d, s in zip((0, lens[0]), done, steps)])
        done = [d + s for d, s in zip(done, steps)]
        hsq.kv_cache_write(k[sel], v[sel], parts, table, i32(*done), i32(0, steps[0], sum(steps)),
                           max_tokens=max(steps))
    assert done == lens and torch.equal(whole, parts)
    # pages of no sequence, and tokens after the last, are as they were
    used = set(table[table >= 0].tolist())
    for p in set(range(n)) - used:
        assert bool((whole[p] == 0xA5).all())
    a, b = hsq.kv_cache_read(parts, table, i32(50, 200), i32(0, 13, 20), tokens=20, head_dim=D, dtype="f32")
    sel = torch.cat([torch.arange(37, 50), torch.arange(lens[0] + 193, lens[0] + 200)])
    assert same(a.double(), held64(k[sel], "asym")) and same(b.double(), held64(v[sel], "asym"))


def test_a_token_writes_its_own_bytes_alone():
    H, D, page = 2, 128, 32
    table, n = pages_for([32], page)
    k, v = rows(5, 32, H, D, torch.bfloat16), rows(6, 32, H, D, torch.bfloat16)
    base = torch.full_like(hsq.kv_cache(n, H, D, page), 0x5A)
    count = torch.zeros(base.shape, dtype=torch.int32, device=DEV)
    other = torch.full_like(base, 0xA5)
    for t in range(32):
        a, b = base.clone(), other.clone()
        for c in (a, b):
            hsq.kv_cache_write(k[t:t + 1], v[t:t + 1], c, table, i32(t + 1))
        count += (a == b).int()           # written: the same over both backgrounds
        assert int(((a != base) & (a != b)).sum()) == 0
    p = int(table[0, 0])
    assert bool((count[p] == 1).all()) and int(count.sum()) == count[p].numel()


def test_strided_rows_and_guarded_outputs():
    H, D, T = 4, 64, 70
    joint = rows(7, T, 10 * H // 4 + 2 * H, D, torch.float16).reshape(T, -1)      # T x (q k v) of one projection
    nq = joint.shape[1] - 2 * H * D
    k = joint[:, nq:nq + H * D].unflatten(1, (H, D))
    v = joint[:, nq + H * D:].unflatten(1, (H, D))
    table, n = pages_for([T], 32)
    c1, c2 = hsq.kv_cache(n, H, D, 32), hsq.kv_cache(n, H, D, 32)
    hsq.kv_cache_write(k, v, c1, table, i32(T))
    hsq.kv_cache_write(k.contiguous(), v.contiguous(), c2, table, i32(T))
    assert torch.equal(c1, c2)
    # rows of no sequence, and beyond max_tokens' tiles, are left alone
    out = tuple(torch.full((T + 5, H, D), 7.0, dtype=torch.float32, device=DEV) for _ in range(2))
    hsq.kv_cache_read(c1, table, i32(T), i32(3, T - 2), tokens=T + 5, head_dim=D, dtype="f32", out=out)
    want = held64(k.contiguous(), "asym")
    assert same(out[0][3:T - 2].double(), want[5:])
    for o in out:
        assert bool((o[:3] == 7).all()) and bool((o[T - 2:] == 7).all())


def test_positions_that_are_not_there():
    H, D, page = 2, 64, 32
    k, v = rows(8, 40, H, D, torch.bfloat16), rows(9, 40, H, D, torch.bfloat16)
    cache = torch.full_like(hsq.kv_cache(3, H, D, page), 0x11)
    before = cache.clone()
    # pages outside the cache, negative lengths and positions, a table that ends early
    for table, lens in ((i32(3, -1)[None], i32(40)), (i32(-2 ** 31, 2 ** 31 - 1)[None], i32(40)),
                        (i32(1, 2)[None], i32(-5)), (i32(1, 2)[None], i32(-2 ** 31)),
                        (i32(1, 2)[None], i32(2 ** 31 - 1)), (i32(0, 1)[None], i32(104))):
        hsq.kv_cache_write(k, v, cache, table, lens)
        assert torch.equal(cache, before)
        a, b = hsq.kv_cache_read(cache, table, lens, tokens=40, head_dim=D, dtype="f32")
        assert not a.any() and not b.any()
    # rows 0 .. 9 at negative positions; the rest on page 2 alone
    hsq.kv_cache_write(k, v, cache, i32(2, -1)[None], i32(30))
    a, b = hsq.kv_cache_read(cache, i32(2, -1)[None], i32(30), tokens=40, head_dim=D, dtype="f32")
    assert not a[:10].any() and same(a[10:].double(), held64(k[10:], "asym"))
    assert same(b[10:].double(), held64(v[10:], "asym")) and torch.equal(cache[:2], before[:2])
    # the last positions of a table, some of them past it
    hsq.kv_cache_write(k, v, cache, i32(0, 1)[None], i32(70))
    a, _ = hsq.kv_cache_read(cache, i32(0, 1)[None], i32(70), tokens=40, head_dim=D, dtype="f32")
    assert same(a[:34].double(), held64(k[:34], "asym")) and not a[34:].any()


def test_cu_tokens_that_are_wrong_stay_inside():
    H, D = 1, 64
    k = rows(10, 16, H, D, torch.bfloat16)
    guard = torch.full((3, 16, H, D), 3.0, dtype=torch.float32, device=DEV)
    table, n = pages_for([64, 64], 32)
    cache = hsq.kv_cache(n, H, D, 32)
    for cu in (i32(-5, 8, 100), i32(10, 4, 12), i32(20, 30, 40), i32(0, 16, 3)):
        hsq.kv_cache_write(k, k, cache, table, i32(64, 64), cu)
        out = (guard[1], torch.empty_like(guard[1]))
        hsq.kv_cache_read(cache, table, i32(64, 64), cu, tokens=16, head_dim=D, dtype="f32", out=out)
    torch.cuda.synchronize()
    assert bool((guard[0] == 3).all()) and bool((guard[2] == 3).all())


def test_many_pages_beyond_32_bits():
    # 4.5 GB of cache: page numbers times page bytes pass 2^32
    H, D, page = 8, 128, 1024
    per = hsq.kv_page_bytes(page, H, D)
    n = (1 << 32) // per + 40
    cache = torch.empty((n, H, per // H), dtype=torch.uint8, device=DEV)
    k, v = rows(11, 70, H, D, torch.bfloat16), rows(12, 70, H, D, torch.bfloat16)
    for p in (n - 1, n // 2, 0):
        cache[p].zero_()
        hsq.kv_cache_write(k, v, cache, i32(p)[None], i32(1000))
        a, b = hsq.kv_cache_read(cache, i32(p)[None], i32(1000), tokens=70, head_dim=D, dtype="f32")
        assert same(a.double(), held64(k, "asym")) and same(b.double(), held64(v, "asym"))
    del cache
    torch.cuda.empty_cache()
