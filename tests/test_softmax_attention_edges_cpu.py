"""What the bindings of softmax attention, rotary positions and the chunked mixer do around the library's call: no GPU
is used, the calls are stood in for."""
import pytest
import torch
from torch.autograd import forward_ad

import gated_linear_attention_local_b200 as sg
from gated_linear_attention_local_b200 import attention


@pytest.fixture
def plain(monkeypatch):
    """The entry points without the library: outputs of zeros."""
    monkeypatch.setattr(attention, "_forward", lambda q, k, v, *a, **kw: (torch.zeros_like(q), torch.zeros(q.shape[:-1])))
    monkeypatch.setattr(attention, "_rotary", lambda q, k, *a, **kw: (q * 0, None if k is None else k * 0))
    for name in ("simple_gla_fwd", "simple_gla_chunk"):
        monkeypatch.setattr(sg, name, lambda q, *a, **kw: (torch.zeros_like(q), None))


def calls():
    pos, freq = torch.zeros(1, 4, dtype=torch.int64), torch.ones(4)
    return {"softmax_attention": lambda q, k, v: sg.softmax_attention(q, k, v),
            "multi_axis_rotary": lambda q, k, v: sg.multi_axis_rotary(q, k, pos, freq)[0],
            "chunk_simple_gla": lambda q, k, v: sg.chunk_simple_gla(q, k, v)[0]}


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("name", sorted(calls()))
def test_forward_mode_tangents_are_not_dropped(plain, name, which):
    """A dual tensor requires no gradient; its tangent must not be taken for zero without a word."""
    x = [torch.randn(1, 4, 2, 8) for _ in range(3)]
    call = calls()[name]
    assert float(call(*x).abs().max()) == 0.0
    with forward_ad.dual_level():
        assert float(call(*x).abs().max()) == 0.0  # no tangent: as ever
        x[which] = forward_ad.make_dual(x[which], torch.ones_like(x[which]))
        with pytest.raises(RuntimeError):
            call(*x)
        with torch.no_grad(), pytest.raises(RuntimeError):  # which stops reverse mode only
            call(*x)
