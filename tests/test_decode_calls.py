"""Calls of the 4-bit cache and of the weight-only layer on the host: batches whose
bound on the rows is loose, a choice that there is not."""

import pytest

import w4a4_rank_assisted_amd as hsq
from test_decode_abi import attend, read, refused, write

# made-up addresses, further apart than the operands are long
FAR = dict(cache=1 << 40, table=1 << 41, lens=1 << 42, cu=1 << 43, width=256, H=8, D=64)


@pytest.mark.parametrize("b,T,code", [(64, 64 * 8192, None), (2048, 2048 * 8, None), (65535, 70000, None),
                                      (256, 1 << 22, None), (4096, 1 << 24, hsq.E_INVAL)])
def test_a_ragged_batch_without_a_bound(b, T, code):
    # max_tokens is T, of every sequence: what is launched follows the rows there are
    refused(write(b=b, T=T, top=T, K=1 << 44, ks=512, V=1 << 45, vs=512, **FAR), code)
    refused(read(b=b, T=T, top=T, K=1 << 44, V=1 << 45, **FAR), code)
    refused(attend(b=b, T=T, top=T, Q=1 << 44, Hq=32, qs=2048, Y=1 << 45, lse=1 << 46, ws=None, wsb=0, **FAR), code)


@pytest.mark.parametrize("kernel", ["tiled", "skinny", "other"])
def test_a_weight_only_layer_has_one_kernel(kernel):
    layer = object.__new__(hsq.Layer)
    with pytest.raises(ValueError, match="weight_only has one kernel"):
        layer(None, kernel=kernel, weight_only=True)
