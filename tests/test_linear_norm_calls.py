"""Calls of the 16-bit linear and the layer normalisation that the interface
does not allow, on the host: sizes beyond a C int."""

import pytest
import torch

import w4a4_rank_assisted_amd as hsq

lib = hsq._load()
BIG = 1 << 32          # its low 32 bits are zero


# ------------------------------------------------------- sizes beyond a C int
@pytest.mark.parametrize("big", [(BIG + 333, 1001, 777), (333, BIG + 1001, 777), (333, 1001, BIG + 777),
                                 (-BIG + 333, 1001, 777)])
def test_workspaces_of_sizes_beyond_an_int(big):
    # what the low 32 bits name is another, small shape
    assert hsq.linear_workspace_bytes(333, 1001, 777) > 0 and hsq.linear_workspace_bytes(*big) == 0
    assert hsq.linear_backward_workspace_bytes(333, 1001, 777) > 0 and hsq.linear_backward_workspace_bytes(*big) == 0
    M, C, _ = big
    assert hsq.layer_norm_backward_workspace_bytes(M, C) == 0 or (M, C) == (333, 1001)
    assert hsq.layer_norm_backward_workspace_bytes(333, 1001, BIG + 1) == 0


class Recorder:
    """Stands for the library: every call succeeds and is kept."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name == "hsq_status_string":
            return lib.hsq_status_string
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture
def recorder(monkeypatch):
    # tensors without memory stand for device tensors of sizes no host holds
    r = Recorder()
    monkeypatch.setattr(hsq, "_load", lambda: r)
    monkeypatch.setattr(hsq, "_device", lambda T, t, name: -1)
    monkeypatch.setattr(hsq._t(), "stream", lambda dev: 0)
    return r


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def test_calls_of_sizes_beyond_an_int_are_refused(recorder):
    many, few, wide = meta(BIG + 5, 8), meta(8, 16), meta(8, BIG + 16)
    stat = meta(BIG + 5, dtype=torch.float32)
    for call in (lambda: hsq.linear(many, few), lambda: hsq.linear(meta(4, 8), wide),
                 lambda: hsq.linear(meta(4, BIG + 8), meta(BIG + 8, 16)),
                 lambda: hsq.linear_backward(meta(BIG + 5, 16), many, few),
                 lambda: hsq.linear_backward(meta(4, BIG + 16), meta(4, 8), wide),
                 lambda: hsq.layer_norm(many), lambda: hsq.layer_norm(meta(4, BIG + 8)),
                 lambda: hsq.layer_norm(meta(4, 8), meta(BIG + 1, 8)),
                 lambda: hsq.layer_norm_backward(many, many, stat, stat),
                 lambda: hsq.layer_norm_backward(meta(4, 8), meta(4, 8), stat[:4], stat[:4], groups=BIG + 1)):
        with pytest.raises(hsq.HsqError) as e:
            call()
        assert e.value.status == hsq.E_INVAL
    assert recorder.calls == []
    hsq.linear(meta(4, 8), few)
    assert recorder.calls[-1][0] == "hsq_linear" and recorder.calls[-1][1][1:4] == (4, 8, 16)
