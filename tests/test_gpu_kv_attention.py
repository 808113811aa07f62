"""Attention over the 4-bit cache: element by element against 64 bits within
derived bounds, exact sums in which every token counts once, one-token softmax
that names the token, and what is not seen."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from decode_ref import U32, attention64, half_step, held64, scales64  # noqa: E402
from test_gpu_kv_cache import DEV, DT, i32, pages_for, rows  # noqa: E402


def fill(k, v, lens, page, quant="asym", spare=1):
    """A cache of the sequences, their tokens one after the other in k, v."""
    _, H, D = k.shape
    table, n = pages_for(lens, page, spare=spare)
    cache = torch.full_like(hsq.kv_cache(n, H, D, page), 0xFF)    # what is not written: NaN scales
    cu = i32(0, *lens).cumsum(0).to(torch.int32)
    if sum(lens):
        hsq.kv_cache_write(k, v, cache, table, i32(*lens), cu, quant=quant)
    return cache, table


def compare(Q, cache, table, k, v, lens, qn, quant, scale, causal, window, y_dtype, uniform):
    cu = None if uniform else i32(0, *qn).cumsum(0).to(torch.int32)
    y, lse = hsq.kv_attention(Q, cache, table, i32(*lens), cu, scale=scale, causal=causal, window=window,
                              y_dtype=y_dtype, return_lse=True, max_tokens=max(qn))
    kd, vd = held64(k, quant), held64(v, quant)
    ks, vs = scales64(k, quant), scales64(v, quant)
    r = t = 0
    for n, m in zip(lens, qn):
        s = slice(t, t + n)
        want, wl, ty, tl = attention64(Q[r:r + m], kd[s], vd[s], ks[s], vs[s], n - m, scale, causal, window,
                                       DT[y_dtype])
        got, gl = y[r:r + m].double(), lse[r:r + m].double()
        assert bool(((got - want).abs() <= ty).all()), (n, m, ((got - want).abs() / ty).max().item())
        dead = torch.isinf(wl)
        assert torch.equal(torch.isinf(gl) & (gl < 0), dead)
        assert bool(((gl - wl).abs() <= tl)[~dead].all())
        assert not got[dead].any()
        r, t = r + m, t + n


CASES = [
    # Hq, H, D, page, lens, queries, causal, window
    (4, 1, 64, 32, [1], [1], True, 0),
    (1, 1, 64, 32, [33], [1], True, 0),
    (32, 8, 128, 64, [777], [1], True, 0),
    (8, 2, 128, 32, [5, 64, 300], [1, 1, 1], True, 0),
    (16, 16, 64, 64, [100, 31], [1, 1], True, 0),
    (5, 1, 256, 32, [130], [1], True, 0),
    (24, 1, 128, 64, [95], [1], True, 0),               # more heads than a tile of rows
    (12, 4, 128, 64, [700, 40], [3, 7], True, 0),
    (7, 7, 64, 32, [1001, 5, 64], [4, 1, 3], True, 50),
    (4, 4, 128, 32, [2100], [1], True, 33),
    (6, 2, 64, 64, [40, 90], [40, 60], True, 0),        # prompts
    (8, 2, 128, 64, [500], [200], True, 0),
    (4, 2, 256, 32, [150], [90], True, 0),
    (4, 2, 128, 32, [333, 64], [100, 1], False, 0),
    (2, 1, 64, 32, [300], [130], True, 7),
    (2, 1, 128, 32, [3, 70], [9, 75], True, 0),         # more rows than tokens: some see nothing
    (4, 1, 64, 32, [0, 40], [1, 1], True, 0),           # a sequence without tokens
    (3, 1, 128, 1024, [5000], [1], True, 0),            # split over workgroups
    (8, 4, 64, 128, [4097, 20, 900], [2, 1, 5], True, 0),
    (4, 2, 256, 64, [3000], [2], True, 0),
    (2, 2, 64, 32, [2500], [3], False, 0),
]


@pytest.mark.parametrize("dt,ydt", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
def test_against_64_bits(case, dt, ydt):
    Hq, H, D, page, lens, qn, causal, window = case
    print(f"[attn] {case} {dt} {ydt}", flush=True)
    T, quant = sum(lens), "asym" if Hq % 2 == 0 else "sym"
    k, v = rows(20, max(T, 1), H, D, DT[dt])[:T], rows(21, max(T, 1), H, D, DT[dt])[:T]
    Q = rows(22, sum(qn), Hq, D, DT[dt])
    cache, table = fill(k, v, lens, page, quant)
    uniform = len(set(qn)) == 1 and len(qn) % 2 == 1
    compare(Q, cache, table, k, v, lens, qn, quant, 1.3 / math.sqrt(D), causal, window, ydt, uniform)


# Queries of zero weigh all tokens alike; values of whole numbers under scales of
# powers of two then have exact sums, whatever their order: y is the sum over the
# number of tokens, three roundings from the real one.
EXACT = [
    # Hq, H, D, page, lens, queries, causal, window
    (4, 1, 128, 64, [1, 31, 32, 33, 1000], 1, True, 0),
    (32, 8, 128, 64, [100000], 1, True, 0),
    (8, 8, 64, 32, [70000, 3], 1, True, 0),
    (16, 1, 256, 256, [20000], 1, True, 0),
    (8, 2, 128, 64, [9000, 600], 2, True, 1234),
    (4, 2, 128, 64, [3001, 999], 401, True, 0),
    (4, 2, 64, 32, [2001], 301, True, 500),
    (2, 1, 256, 32, [801], 201, True, 0),
    (6, 3, 128, 32, [1777], 100, False, 0),
    (8, 1, 128, 32, [513 * 32 + 7], 2, False, 0),
]


@pytest.mark.parametrize("case", EXACT, ids=lambda c: "-".join(str(x) for x in c).replace(" ", ""))
@pytest.mark.parametrize("ydt", ["f32", "bf16"])
def test_every_token_counts_once(case, ydt):
    Hq, H, D, page, lens, q, causal, window = case
    print(f"[attn exact] {case} {ydt}", flush=True)
    g = torch.Generator().manual_seed(31)
    T = sum(lens)
    v = torch.randint(-7, 8, (T, H, D), generator=g).float()
    v[:, :, ::64] = 7.0
    v *= torch.exp2(torch.randint(-2, 3, (T, H, 1), generator=g).float())
    k = torch.randn(T, H, D, generator=g).to(torch.bfloat16).to(DEV)
    v = v.to(torch.bfloat16).to(DEV)
    cache, table = fill(k, v, lens, page, "sym")
    Q = torch.zeros(len(lens) * q, Hq, D, dtype=torch.bfloat16, device=DEV)
    y, lse = hsq.kv_attention(Q, cache, table, i32(*lens), causal=causal, window=window, y_dtype=ydt, return_lse=True)
    t = 0
    for b, n in enumerate(lens):
        c = torch.cat([torch.zeros(1, H, D, dtype=torch.float64, device=DEV), v[t:t + n].double().cumsum(0)])
        i = torch.arange(n - q, n, device=DEV)
        hi = i + 1 if causal else torch.full_like(i, n)
        lo = (i - window + 1).clamp(min=0) if window else torch.zeros_like(i)
        want = ((c[hi] - c[lo]) / (hi - lo)[:, None, None]).repeat_interleave(Hq // H, 1)
        got = y[b * q:(b + 1) * q].double()
        tol = want.abs() * (3 * U32 + (half_step(torch.bfloat16) * (1 + 4 * U32) if ydt == "bf16" else 0))
        assert bool(((got - want).abs() <= tol).all()), (n, ((got - want).abs() - tol).max().item())
        wl = torch.log((hi - lo).double())[:, None]
        assert bool(((lse[b * q:(b + 1) * q].double() - wl).abs() <= 8 * U32 * (wl + 1)).all())
        t += n


@pytest.mark.parametrize("Hq,H,D,page,n,q", [(8, 2, 64, 32, 1500, 1), (4, 2, 128, 64, 700, 64), (8, 8, 128, 64, 90, 2),
                                            (2, 1, 256, 64, 400, 70), (3, 1, 64, 64, 5000, 3)])
def test_one_token_softmax(Hq, H, D, page, n, q):
    # a query along one key, so long that the others weigh less than 2^-40: y is that value
    g = torch.Generator().manual_seed(41)
    k = torch.where(torch.rand(n, H, D, generator=g) < 0.5, -7.0, 7.0).to(torch.bfloat16).to(DEV)   # codes hold them
    v = rows(42, n, H, D, torch.bfloat16)
    cache, table = fill(k, v, [n], page, "sym")
    pick = torch.randint(0, n - q + 1, (q, Hq), generator=g).to(DEV)
    Q = k[pick, (torch.arange(Hq, device=DEV) // (Hq // H))[None]] / 7
    # scores: scale D 7 for the token itself; another agrees in D/2 + 4.5 sqrt(D) channels at most here
    scale = 1.0
    agree = torch.einsum("thd,shd->hts", k.cpu().double() / 7, k.cpu().double() / 7)
    agree.diagonal(dim1=1, dim2=2).fill_(-D)
    assert float(agree.max()) <= D - 6           # 7 (D - (D - 6)) > 40 / log2(e) + ...: p < 2^-60
    y = hsq.kv_attention(Q.contiguous(), cache, table, i32(n), scale=scale, y_dtype="f32", causal=False)
    want = held64(v, "sym")[pick, (torch.arange(Hq, device=DEV) // (Hq // H))[None]]
    assert bool(((y.double() - want).abs() <= want.abs() * (8 * U32 + 2.0 ** -21) + 1e-9).all())


def test_growing_scores_move_the_offset():
    # scores rise along the sequence, and scales span 2^-20 .. 2^10
    D, n = 64, 600
    g = torch.Generator().manual_seed(51)
    k = torch.randn(n, 1, D, generator=g) * torch.linspace(0.01, 6.0, n)[:, None, None]
    v = torch.randn(n, 1, D, generator=g) * torch.exp2(torch.randint(-20, 11, (n, 1, 1), generator=g).float())
    v[100:140] = 0.0
    for kk in (k, k.flip(0)):
        kk, vv = kk.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV)
        cache, table = fill(kk, vv, [n], 32)
        Q = rows(52, 3, 4, D, torch.bfloat16)
        for ydt in ("bf16", "f32"):
            compare(Q, cache, table, kk, vv, [n], [3], "asym", 2.0, True, 0, ydt, True)


def test_values_of_zero_still_weigh():
    D, n = 64, 100
    k = rows(53, n, 1, D, torch.float16)
    v = torch.zeros(n, 1, D, dtype=torch.float16, device=DEV)
    v[:3] = 1.0
    cache, table = fill(k, v, [n], 32)
    Q = rows(54, 1, 2, D, torch.float16)
    for ydt in ("f16", "f32"):
        compare(Q, cache, table, k, v, [n], [1], "asym", 0.5, True, 0, ydt, True)
    v.zero_()
    cache, table = fill(k, v, [n], 32)
    y, lse = hsq.kv_attention(Q, cache, table, i32(n), scale=8.0, return_lse=True)
    assert not y.any() and bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("Hq,H,D,q", [(4, 1, 64, 1), (4, 2, 128, 3), (4, 1, 128, 70)])
def test_nan_where_it_is_not_seen(Hq, H, D, q):
    n, bad = 200, 150
    k, v = rows(61, n, H, D, torch.bfloat16), rows(62, n, H, D, torch.bfloat16)
    cache, table = fill(k, v, [n], 32)
    Q = rows(63, q, Hq, D, torch.bfloat16)
    # all sequences of one length, with a bad token behind the queries' end
    want = hsq.kv_attention(Q, cache, table, i32(bad), y_dtype="f32")
    for x in (math.nan, math.inf, -math.inf):
        for part in (0, 1):
            kk, vv = k.clone(), v.clone()
            (kk if part == 0 else vv)[bad:] = x
            c2, t2 = fill(kk, vv, [n], 32)
            assert torch.equal(hsq.kv_attention(Q, c2, t2, i32(bad), y_dtype="f32"), want)
            # queries that end behind it: those that see it are NaN, the others as they were
            y = hsq.kv_attention(Q, c2, t2, i32(bad + 1), y_dtype="f32")
            assert bool(torch.isnan(y[-1]).any(-1).all())
            if q > 1:
                clean = hsq.kv_attention(Q, cache, table, i32(bad + 1), y_dtype="f32")
                assert torch.equal(y[:-1], clean[:-1])
            # outside the window
            w = hsq.kv_attention(Q[-1:].contiguous(), c2, t2, i32(n), window=5, y_dtype="f32")
            assert bool(torch.isnan(w).any())
            vv2 = v.clone()
            vv2[:bad] = x
            c3, t3 = fill(k, vv2, [n], 32)
            w3 = hsq.kv_attention(Q[-1:].contiguous(), c3, t3, i32(n), window=n - bad, y_dtype="f32")
            assert torch.equal(w3, hsq.kv_attention(Q[-1:].contiguous(), cache, table, i32(n), window=n - bad,
                                                    y_dtype="f32"))
    # a query that is not finite keeps to its own row
    Q2 = Q.clone()
    Q2[0, 0, 0] = math.nan
    y, clean = (hsq.kv_attention(t, cache, table, i32(bad), y_dtype="f32") for t in (Q2, Q))
    assert bool(torch.isnan(y[0, 0]).all())
    assert torch.equal(y[0, 1:], clean[0, 1:]) and torch.equal(y[1:], clean[1:])


def test_pages_that_are_not_there_take_no_part():
    H, D, page, n = 2, 64, 32, 160
    k, v = rows(71, n, H, D, torch.bfloat16), rows(72, n, H, D, torch.bfloat16)
    cache, table = fill(k, v, [n], page, spare=0)
    Q = rows(73, 1, 4, D, torch.bfloat16)
    for bad in (-1, cache.shape[0], 2 ** 31 - 1, -2 ** 31):
        t2 = table.clone()
        t2[0, 1] = bad
        y = hsq.kv_attention(Q, cache, t2, i32(n), y_dtype="f32")
        keep = torch.cat([torch.arange(32), torch.arange(64, n)])
        c3, t3 = fill(k[keep], v[keep], [n - 32], page)
        assert torch.allclose(y, hsq.kv_attention(Q, c3, t3, i32(n - 32), y_dtype="f32"), rtol=1e-5, atol=1e-6)
    # lengths past the table's end count what the table holds; the queries sit past it
    y = hsq.kv_attention(Q, cache, table, i32(n + 1000), y_dtype="f32")
    assert torch.equal(y, hsq.kv_attention(Q, cache, table, i32(n), y_dtype="f32"))
    for lens in (0, -7, -2 ** 31):
        y, lse = hsq.kv_attention(Q, cache, table, i32(lens), return_lse=True)
        assert not y.any() and bool((lse == -math.inf).all())


def test_rows_of_no_sequence_and_strides():
    H, D = 2, 128
    k, v = rows(81, 100, H, D, torch.bfloat16), rows(82, 100, H, D, torch.bfloat16)
    cache, table = fill(k, v, [60, 40], 32)
    joint = rows(83, 9, 3 * 4, D, torch.bfloat16)
    Q = joint[:, 4:8]
    cu = i32(2, 3, 7)
    out = torch.full((9, 4, D), 5.0, dtype=torch.bfloat16, device=DEV)
    y = hsq.kv_attention(Q, cache, table, i32(60, 40), cu, max_tokens=4, out=out)
    assert y is out and bool((y[:2] == 5).all()) and bool((y[7:] == 5).all())
    y2 = hsq.kv_attention(Q[2:7].contiguous(), cache, table, i32(60, 40), cu - 2, max_tokens=4)
    assert torch.equal(y[2:7], y2)


@pytest.mark.parametrize("T", [1, 5, 40])
def test_a_bound_above_the_rows(T):
    H, D, n = 2, 128, 300
    k, v = rows(85, n, H, D, torch.bfloat16), rows(86, n, H, D, torch.bfloat16)
    Q, cu = rows(87, T, 4, D, torch.bfloat16), i32(0, T)
    cache, table = fill(k, v, [n], 32)
    want = hsq.kv_attention(Q, cache, table, i32(n), cu, y_dtype="f32")
    whole = hsq.kv_cache_read(cache, table, i32(n), cu, tokens=T, head_dim=D)
    for top in (T + 1, 1000, 2 ** 31 - 1):
        assert torch.equal(hsq.kv_attention(Q, cache, table, i32(n), cu, y_dtype="f32", max_tokens=top), want)
        again = cache.clone()
        hsq.kv_cache_write(k[n - T:], v[n - T:], again, table, i32(n), cu, max_tokens=top)
        assert torch.equal(again, cache)
        got = hsq.kv_cache_read(again, table, i32(n), cu, tokens=T, head_dim=D, max_tokens=top)
        assert torch.equal(got[0], whole[0]) and torch.equal(got[1], whole[1])


def test_result_does_not_depend_on_the_rest():
    # the same bits alone, in a batch, and from call to call
    H, D, lens = 2, 128, [900, 77, 3000]
    T = sum(lens)
    k, v = rows(91, T, H, D, torch.bfloat16), rows(92, T, H, D, torch.bfloat16)
    cache, table = fill(k, v, lens, 64)
    Q = rows(93, 3, 8, D, torch.bfloat16)
    y = hsq.kv_attention(Q, cache, table, i32(*lens))
    for _ in range(5):
        assert torch.equal(y, hsq.kv_attention(Q, cache, table, i32(*lens)))


@pytest.mark.parametrize("y_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads", [1, 4, 8, 16, 80])
def test_small_channels_count_beside_a_large_one(D, heads, y_dtype):
    # one channel of 1 and the others 2^-19, their codes 15 and the large one's 0, over
    # zeros from 0 to 8: the small ones are not lost from the scores.  Each of up to 16
    # instructions a group and the steps around them rounds at 2^-20 of the largest product
    # per term: 80 terms and 16 steps
    q = torch.full((1, heads, D), 2.0 ** -19)
    q[..., ::64] = 1.0
    k = torch.empty(9, 1, D)
    for z in range(9):
        k[z] = float(15 - z)
        k[z, :, ::64] = float(-z)
    k, v = k.bfloat16().to(DEV), torch.ones(9, 1, D, dtype=torch.bfloat16, device=DEV)
    for z in range(9):
        cache, table = fill(k[z:z + 1], v[z:z + 1], [1], 32)
        y, lse = hsq.kv_attention(q.bfloat16().to(DEV), cache, table, i32(1), scale=1.0, y_dtype=y_dtype, return_lse=True)
        want = D // 64 * (-z + 63 * (15 - z) * 2.0 ** -19)
        assert bool(((lse.double() - want).abs() <= D // 64 * 96 * 2.0 ** -20 + 4 * U32 * abs(want)).all()), z
        held = held64(v[z:z + 1], "asym")                # 15 times the fp16 scale 1 / 15
        assert bool(((y.double() - held.view(-1)[0]).abs() <= (2.0 ** -20 if y_dtype == "f32" else 2.0 ** -7)).all())
