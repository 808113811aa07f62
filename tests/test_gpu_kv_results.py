"""What results of the attention over the 4-bit cache keep: fp16 ones as many bits as
their type has, groups of channels beside others of larger values."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from decode_ref import U32, half_step, held64, tiny  # noqa: E402
from test_gpu_kv_attention import fill  # noqa: E402
from test_gpu_kv_cache import DEV, DT, i32, rows  # noqa: E402


# Hq, H, D, rows of queries, tokens: every form, rows of one token and of many
@pytest.mark.parametrize("Hq,H,D,q,n", [
    (4, 1, 64, 1, 1), (4, 2, 128, 1, 1), (4, 1, 256, 1, 1), (8, 1, 64, 2, 2), (8, 1, 128, 1, 33), (16, 1, 64, 3, 40),
    (8, 1, 128, 4, 60), (4, 1, 256, 9, 50), (4, 1, 64, 70, 70), (4, 1, 128, 70, 100), (2, 1, 256, 70, 90), (4, 1, 128, 1, 1500),
])
def test_fp16_results(Hq, H, D, q, n):
    # one key for all tokens: their scores and weights are alike, whatever the scores' own
    # error, and y is the mean of the values.  A weight times a scale is held in two terms of
    # fp16 (2^-21); the sums add 2 units a token, and cut their terms, N and an
    # instruction's start every four, at 2^-20 of the largest; then one rounding to fp16.
    k = rows(301, 1, H, D, torch.float16).expand(n, -1, -1).contiguous()
    v = rows(302, n, H, D, torch.float16)
    Q = rows(303, q, Hq, D, torch.float16)
    cache, table = fill(k, v, [n], 32, spare=160)
    y = hsq.kv_attention(Q, cache, table, i32(n), scale=1.3 / math.sqrt(D)).double()
    held = held64(v, "asym")
    seen = torch.arange(n - q + 1, n + 1, device=DEV).double()[:, None, None]
    want, most = (t.cumsum(0)[n - q:] / seen for t in (held, held.abs()))
    s = (v.double().view(n, H, D // 64, 64).amax(3).clamp(min=0) - v.double().view(n, H, D // 64, 64).amin(3).clamp(max=0)) / 15
    cut = 2 * (n / 4 + 8 + n) * 2.0 ** -20 * (1 + 2.0 ** -11) * s.cummax(0).values[n - q:].repeat_interleave(64, 2) / seen
    tol = most * (2.0 ** -21 + 2 * (n + 64) * U32) + cut
    tol, want = tol.repeat_interleave(Hq // H, 1), want.repeat_interleave(Hq // H, 1)
    tol = tol + half_step(torch.float16) * (want.abs() + tol) + tiny(torch.float16)
    assert bool(((y - want).abs() <= tol).all()), ((y - want).abs() / tol).max().item()


# Hq, H, D, rows of queries, tokens
@pytest.mark.parametrize("Hq,H,D,q,n", [(4, 1, 128, 1, 1), (4, 1, 256, 1, 5), (8, 1, 128, 2, 40), (8, 2, 256, 4, 30),
                                        (8, 1, 128, 4, 60), (4, 1, 128, 70, 100), (2, 1, 256, 70, 90), (4, 1, 128, 1, 1500)])
@pytest.mark.parametrize("apart", [8, 16, 24, 40])
@pytest.mark.parametrize("ydt", ["f32", "bf16", "f16"])
def test_groups_of_other_scales(Hq, H, D, q, n, apart, ydt):
    # as above, with the values' groups 2^apart from each other: all groups of a row share an
    # offset, that takes the row's largest weight times scale to 2^7 at least, where fp16 ends at
    # 2^-24.  So a weight times a scale is also off by 2^-32 of the row's largest, fifteen
    # codes of it a token, and where the codes are of 2^-24 their sums by 2^-35 a term.
    half = torch.float16 if ydt == "f16" else torch.bfloat16
    k = rows(311, 1, H, D, half).expand(n, -1, -1).contiguous()
    G, lower = D // 64, torch.arange(D // 64) % 2
    by = torch.exp2(torch.where(lower == 1, -float(apart) + 2, 2.0)).repeat_interleave(64).to(DEV)
    v = (rows(312, n, H, D, torch.float32) * by).to(half)
    Q = rows(313, q, Hq, D, half)
    cache, table = fill(k, v, [n], 32, spare=160)
    y = hsq.kv_attention(Q, cache, table, i32(n), scale=1.3 / math.sqrt(D), y_dtype=ydt).double()
    held = held64(v, "asym")
    seen = torch.arange(n - q + 1, n + 1, device=DEV).double()[:, None, None]
    want, most = (t.cumsum(0)[n - q:] / seen for t in (held, held.abs()))
    x = v.double().view(n, H, G, 64)
    s = (x.amax(3).clamp(min=0) - x.amin(3).clamp(max=0)) / 15 * (1 + 2.0 ** -11)
    split = ydt != "bf16"
    top = s.cummax(0).values[n - q:]
    cut = 2 * (n / 4 + 8 + n) * (2.0 ** -20 if split else 2.0 ** -14) * top.repeat_interleave(64, 2) / seen
    floor = (15 * n * 2.0 ** -32 + 2 * (n / 4 + 8 + n) * 2.0 ** -35) * top.amax(2, keepdim=True) / seen
    # 16-bit sums of p s n and p s z apart: 30 p s in all
    apart_sums = 0.0 if split else 30 * s.cumsum(0)[n - q:].repeat_interleave(64, 2) / seen * 2 * (n + 64) * U32
    tol = most * ((2.0 ** -21 if split else 2.0 ** -11) + 2 * (n + 64) * U32) + cut + floor + apart_sums
    tol, want = tol.repeat_interleave(Hq // H, 1), want.repeat_interleave(Hq // H, 1)
    if ydt != "f32":
        tol = tol + half_step(DT[ydt]) * (want.abs() + tol) + tiny(DT[ydt])
    assert bool(((y - want).abs() <= tol).all()), ((y - want).abs() / tol).max().item()
