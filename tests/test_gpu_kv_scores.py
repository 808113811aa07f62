"""Attention over the 4-bit cache at the ends of the scores' range: scales that take
a query to nothing, scores far from zero, scores beyond the whole numbers of fp32."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from decode_ref import U32, half_step, held64  # noqa: E402
from test_gpu_kv_attention import fill  # noqa: E402
from test_gpu_kv_cache import DEV, DT, i32  # noqa: E402

# Hq, H, D, rows of queries, tokens: every form of the kernels, whole and split
FORMS = [
    (4, 1, 64, 1, 77), (4, 2, 128, 1, 45), (2, 1, 256, 2, 100), (8, 1, 64, 1, 90), (8, 1, 128, 1, 45), (16, 2, 256, 1, 70),
    (6, 2, 64, 3, 130), (12, 2, 128, 3, 99), (4, 2, 64, 40, 170), (4, 2, 128, 40, 170), (2, 1, 256, 70, 140),
    (4, 1, 128, 1, 5003), (8, 1, 64, 4, 5003), (4, 2, 256, 2, 3333),
]
ids = dict(ids=lambda c: "-".join(map(str, c)))


def whole_values(g, n, H, D):
    """Whole numbers from -7 to 7 times powers of two, which the symmetric cache holds."""
    v = torch.randint(-7, 8, (n, H, D), generator=g).float()
    v[:, :, ::64] = 7.0
    return (v * torch.exp2(torch.randint(-2, 3, (n, H, 1), generator=g).float())).to(torch.bfloat16).to(DEV)


def means(v, q, G):
    """The mean of the values that each of the last q tokens sees, and their number."""
    n = v.shape[0]
    seen = torch.arange(n - q + 1, n + 1, device=DEV)
    return (v.double().cumsum(0)[n - q:] / seen[:, None, None]).repeat_interleave(G, 1), seen.double()[:, None]


def check_means(y, v, q, G, ydt):
    # every token weighs the same power of two: the sums are exact, three roundings remain
    want, _ = means(v, q, G)
    tol = want.abs() * (3 * U32 + (half_step(torch.bfloat16) * (1 + 4 * U32) if ydt == "bf16" else 0))
    assert bool(((y.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("form", FORMS, **ids)
@pytest.mark.parametrize("ydt", ["f32", "bf16"])
def test_queries_of_zero_under_a_tiny_scale(form, ydt):
    Hq, H, D, q, n = form
    g = torch.Generator().manual_seed(101)
    v = whole_values(g, n, H, D)
    k = torch.randn(n, H, D, generator=g).to(torch.bfloat16).to(DEV)
    cache, table = fill(k, v, [n], 32, "sym", spare=160)
    Q = torch.zeros(q, Hq, D, dtype=torch.bfloat16, device=DEV)
    for scale in (1e-12, 1e-14, 1e-25, 1e-38, 1e-45):
        print(f"[scores] {form} {ydt} scale {scale}", flush=True)
        y, lse = hsq.kv_attention(Q, cache, table, i32(n), scale=scale, y_dtype=ydt, return_lse=True)
        check_means(y, v, q, Hq // H, ydt)
        wl = torch.log(means(v, q, Hq // H)[1])
        assert bool(((lse.double() - wl).abs() <= 8 * U32 * (wl + 1)).all())


def one_channel_keys(g, codes, H, D):
    """Keys that the symmetric cache holds as they are: channel 0 as given (n, H), the others any."""
    k = torch.randint(-7, 8, (codes.shape[0], H, D), generator=g).float()
    k[:, :, 1::64] = 7.0
    k[:, :, 0] = codes
    return k.to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q", [1, 6, 70])
def test_the_largest_queries_and_scales(D, q):
    # one token of score scale |q| among others of 0: its value, and lse while the product
    # is below 2^122
    n = 50
    g = torch.Generator().manual_seed(105)
    codes = torch.zeros(n, 1)
    codes[n // 2 - q // 4 if q < 40 else 0] = 1.0
    k = one_channel_keys(g, codes, 1, D)
    v = whole_values(g, n, 1, D)
    n2 = n + q                                       # all rows see the token
    k, v = torch.cat([k, k[1:2].expand(q, -1, -1)]), torch.cat([v, v[1:2].expand(q, -1, -1)])
    cache, table = fill(k, v, [n2], 32, "sym")
    at = int(codes.argmax())
    for power, scale in ((121, 1.0), (121, 2.0 ** -20), (100, 2.0 ** 21), (60, 2.0 ** 61), (22, 2.0 ** 99), (124, 1.0),
                         (127, 1.0), (120, 2.0 ** 60)):
        Q = torch.zeros(q, 4, D, dtype=torch.bfloat16, device=DEV)
        Q[:, :, 0] = 2.0 ** power
        print(f"[scores] {D} {q} 2^{power} {scale}", flush=True)
        y, lse = hsq.kv_attention(Q, cache, table, i32(n2), scale=scale, y_dtype="f32", return_lse=True)
        want = v[at].double()[None].expand(q, 4, D)
        assert bool(((y.double() - want).abs() <= want.abs() * (8 * U32 + 2.0 ** -21)).all())
        wl = 2.0 ** power * scale
        if wl < 2.0 ** 122:
            assert bool(((lse.double() - wl).abs() <= 8 * U32 * wl).all())


# Channel 0 of the queries is 2^p, p another for every row and head, so that rows of
# scores near zero and far ones share a wave; one key a head holds 7 there and the others
# less, by 1 at least, which for 2^7 and more is a weight below 2^-180: y is its value.  The
# values' scales are powers of two from 2^-14 to 2^12.  A weight times its scale is rounded
# once to fp16 for bf16 results, to two terms for the others (2^-21); the rest is a few
# roundings of fp32.
@pytest.mark.parametrize("form", FORMS, **ids)
@pytest.mark.parametrize("ydt", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_one_token_at_every_distance(form, ydt, where):
    Hq, H, D, q, n = form
    G, last = Hq // H, n - q + 1
    g = torch.Generator().manual_seed(103)
    v = torch.randint(-7, 8, (n, H, D), generator=g).float()
    v[:, :, ::64] = 7.0
    v = (v * torch.exp2(torch.randint(-14, 13, (n, H, 1), generator=g).float())).to(torch.bfloat16).to(DEV)
    # the others rise along the sequence, so that offsets move
    codes = (torch.linspace(-7.0, 6.49, n).round()[:, None]).repeat(1, H)
    at = {"first": 0, "middle": last // 2, "last": last - 1}[where]
    pick = torch.tensor([max(0, at - 7 * h) for h in range(H)])
    codes[pick, torch.arange(H)] = 7.0
    k = one_channel_keys(g, codes, H, D)
    cache, table = fill(k, v, [n], 32, "sym", spare=160)
    powers = [7, 13, 20, 22, 24, 26, 27, 28, 30, 45, 61, 99, 110]
    p = torch.tensor([[powers[(3 * i + h) % len(powers)] for h in range(Hq)] for i in range(q)]).double()
    Q = torch.zeros(q, Hq, D, dtype=torch.bfloat16, device=DEV)
    Q[:, :, 0] = torch.exp2(p).to(torch.bfloat16).to(DEV)
    print(f"[scores] {form} {ydt} {where}", flush=True)
    y, lse = hsq.kv_attention(Q, cache, table, i32(n), scale=1.0, y_dtype=ydt, return_lse=True)
    want = held64(v, "sym")[pick.to(DEV), torch.arange(H, device=DEV)].repeat_interleave(G, 0)[None].expand(q, -1, -1)
    rel = 8 * U32 + (2.0 ** -21 if ydt == "f32" else 2.0 ** -11 + half_step(DT[ydt]) * (1 + 2.0 ** -10))
    assert bool(((y.double() - want).abs() <= want.abs() * rel + 1e-30).all())
    wl = 7 * torch.exp2(p).to(DEV)
    assert bool(((lse.double() - wl).abs() <= 8 * U32 * wl.abs()).all())


@pytest.mark.parametrize("form", FORMS, **ids)
@pytest.mark.parametrize("power", [24, 28, 33, 100])
def test_many_tokens_far_above_zero(form, power):
    # tokens of one score count alike, however far it is
    Hq, H, D, q, n = form
    g = torch.Generator().manual_seed(104)
    v = whole_values(g, n, H, D)
    k = one_channel_keys(g, torch.full((n, H), 7.0), H, D)
    cache, table = fill(k, v, [n], 32, "sym", spare=160)
    Q = torch.zeros(q, Hq, D, dtype=torch.bfloat16, device=DEV)
    Q[:, :, 0] = 2.0 ** power
    print(f"[scores] {form} 2^{power}", flush=True)
    y, lse = hsq.kv_attention(Q, cache, table, i32(n), scale=1.0, y_dtype="f32", return_lse=True)
    check_means(y, v, q, Hq // H, "f32")
    wl = 7 * 2.0 ** power + torch.log(means(v, q, Hq // H)[1])
    assert bool(((lse.double() - wl).abs() <= 8 * U32 * wl.abs()).all())


@pytest.mark.parametrize("form", FORMS, **ids)
def test_a_far_row_that_rises_to_zero(form):
    # the tokens of score 0 come behind others of -7 |q|, which are far below
    Hq, H, D, q, n = form
    g = torch.Generator().manual_seed(106)
    v = whole_values(g, n, H, D)
    codes = torch.full((n, H), -7.0)
    codes[n - q - 2:] = 0.0
    k = one_channel_keys(g, codes, H, D)
    cache, table = fill(k, v, [n], 32, "sym", spare=160)
    for power in (23, 40, 90):
        Q = torch.zeros(q, Hq, D, dtype=torch.bfloat16, device=DEV)
        Q[:, :, 0] = 2.0 ** power
        print(f"[scores] {form} 2^{power}", flush=True)
        y, lse = hsq.kv_attention(Q, cache, table, i32(n), scale=1.0, y_dtype="f32", return_lse=True)
        check_means(y, v[n - q - 2:], q, Hq // H, "f32")
        wl = torch.log(means(v[n - q - 2:], q, Hq // H)[1])
        assert bool(((lse.double() - wl).abs() <= 8 * U32 * (wl + 1)).all())


@pytest.mark.parametrize("form", FORMS, **ids)
@pytest.mark.parametrize("ydt", ["f32", "bf16"])
def test_scores_far_below_zero(form, ydt):
    # all tokens of one score: -7 |q|.  lse: three roundings in the score, and those of the
    # logarithm's sum and product
    Hq, H, D, q, n = form
    g = torch.Generator().manual_seed(102)
    v = whole_values(g, n, H, D)
    k = one_channel_keys(g, torch.full((n, H), -7.0), H, D)
    cache, table = fill(k, v, [n], 32, "sym", spare=160)
    for power in (20, 60, 97, 100, 112):
        print(f"[scores] {form} {ydt} 2^{power}", flush=True)
        Q = torch.zeros(q, Hq, D, dtype=torch.bfloat16, device=DEV)
        Q[:, :, 0] = 2.0 ** power
        y, lse = hsq.kv_attention(Q, cache, table, i32(n), scale=1.0, y_dtype=ydt, return_lse=True)
        check_means(y, v, q, Hq // H, ydt)
        wl = -7 * 2.0 ** power + torch.log(means(v, q, Hq // H)[1])
        assert bool(((lse.double() - wl).abs() <= 8 * U32 * wl.abs()).all())
