"""A sequence's attention does not depend on the others of its batch."""

import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import w4a4_rank_assisted_amd as hsq  # noqa: E402
from test_gpu_kv_attention import fill  # noqa: E402
from test_gpu_kv_cache import DEV, i32, rows  # noqa: E402


@pytest.mark.parametrize("ydt", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,H,D,q", [(8, 2, 128, 1), (8, 1, 64, 1), (2, 1, 256, 3), (8, 2, 128, 3), (4, 2, 64, 40), (4, 1, 256, 20)])
def test_alone_and_in_a_batch(Hq, H, D, q, ydt):
    # tables of one part's width, so that both calls are planned alike: the same bits
    lens = [900, 77, 1000, 45]
    T = sum(lens)
    k, v = rows(501, T, H, D, torch.bfloat16), rows(502, T, H, D, torch.bfloat16)
    cache, table = fill(k, v, lens, 32, spare=0)
    assert table.shape[1] == 32
    Q = rows(503, q * len(lens), Hq, D, torch.bfloat16)
    y, lse = hsq.kv_attention(Q, cache, table, i32(*lens), y_dtype=ydt, return_lse=True)
    for b, n in enumerate(lens):
        r = slice(b * q, (b + 1) * q)
        a, l = hsq.kv_attention(Q[r].contiguous(), cache, table[b:b + 1].contiguous(), i32(n), y_dtype=ydt, return_lse=True)
        assert torch.equal(a, y[r]) and torch.equal(l, lse[r])
